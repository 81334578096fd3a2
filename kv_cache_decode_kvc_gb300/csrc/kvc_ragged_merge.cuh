// kvc_ragged_merge.cuh -- merge of the pieces of split streams (see kvc_ragged.cuh), launched
// behind an attention kernel with the split R.
#pragma once

#include "kvc_ragged.cuh"

namespace kvc {

// One warp merges np pieces of one output row: state(i, o, ml) gives piece i's address.
// out = sum_i w_i o_i / sum_i w_i l_i, w_i = 2^(m_i - max m); a piece that saw nothing (l = 0)
// has weight 0.  NaN scores reach l and o and stay NaN.
template <typename T, class F>
__device__ __forceinline__ void merge_row(const RaggedParams& p, int np, T* out, int lane, F&& state) {
    float M = -INFINITY;
    for (int i = lane; i < np; i += 32) {
        const float *o, *ml;
        state(i, o, ml);
        M = fmaxf(M, __ldcg(ml));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    if (M == -INFINITY) M = 0.f;
    float den = 0.f;
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
        const float *o, *ml;
        state(i, o, ml);
        const float2 s = __ldcg(reinterpret_cast<const float2*>(ml));
        const float w = s.y == 0.f ? 0.f : fast_exp2(s.x - M);
        den += w == 0.f && s.y == s.y ? 0.f : w * s.y;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int d = lane * 4 + v * 128;
            if (d < p.D) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(o + d));
                if (s.y != 0.f) {
                    acc[v].x = fmaf(w, x.x, acc[v].x);
                    acc[v].y = fmaf(w, x.y, acc[v].y);
                    acc[v].z = fmaf(w, x.z, acc[v].z);
                    acc[v].w = fmaf(w, x.w, acc[v].w);
                }
            }
        }
    }
    const float inv = 1.f / den;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int d = lane * 4 + v * 128;
        if (d < p.D) {
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint2*>(out + d) = make_uint2(bf16x2_rn(acc[v].x * inv, acc[v].y * inv),
                                                                bf16x2_rn(acc[v].z * inv, acc[v].w * inv));
            } else {
                *reinterpret_cast<float4*>(out + d) =
                    make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
            }
        }
    }
}

constexpr int MERGE_WARPS = 8, MERGE_SLICES = 8;

// Without groups: block (c, s) takes the c-th possible cut; if a stream was cut there first, its
// warps merge every MERGE_SLICES-th eight rows of the stream's tile.
template <typename T, class R>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_cuts_kernel(const RaggedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 a = __ldcg(p.cuts + 2 * blockIdx.x), b = __ldcg(p.cuts + 2 * blockIdx.x + 1);
    if (a.x == 0) return;
    const int G = 1 << p.lgG;
    for (int r = blockIdx.y * MERGE_WARPS + warp; r < b.x; r += MERGE_SLICES * MERGE_WARPS) {
        const int64_t row = a.w + (r >> p.lgG);
        T* out = static_cast<T*>(p.out) + row * p.out_ts + (int64_t)(b.y * G + (r & (G - 1))) * p.D;
        merge_row<T>(p, a.x, out, lane, [&](int q, const float*& o, const float*& ml) {
            const int64_t at = (int64_t)R::slot(a.z, a.y + q, q > 0) * R::SLOT_ROWS + r;
            o = p.slot_o + at * p.D;
            ml = p.slot_ml + at * 2;
        });
    }
}

// With groups: block (row, KV head), a warp per query head of the group in turn; the row's
// pieces are those of its prefix stream and of its sequence's own stream.
template <typename T, class R>
__global__ void __launch_bounds__(128) merge_rows_kernel(const RaggedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const typename R::Split sp = R::planned(p);
    if (!sp.valid) return;
    const int row = blockIdx.x, h = blockIdx.y, G = 1 << p.lgG;
    if (row >= __ldg(p.cu + p.B)) return;
    int lo = 0, hi = p.B - 1;  // the sequence: largest b with cu[b] <= row
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.cu + mid) <= row) lo = mid; else hi = mid - 1;
    }
    const typename R::Stream own = R::of_row(p, sp, p.plan, p.NG + lo, h, row);
    if (!own.s.ok) return;
    const int of = R::owner(sp, own.u0 + RAGGED_C0), ol = R::owner(sp, own.u0 + RAGGED_C0 + own.n - 1);
    const bool joint = own.s.pfx > 0;
    if (!joint && of == ol) return;  // written by its worker
    int pf = 0, pl = -1, pr = 0, pc = 0;
    const int oc = R::cls(p, own.s);
    if (joint) {
        int a = 0, b = p.NG - 1;
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            if (__ldg(p.groups + mid) <= lo) a = mid; else b = mid - 1;
        }
        const typename R::Stream pre = R::of_row(p, sp, p.plan, a, h, row);
        pf = R::owner(sp, pre.u0 + RAGGED_C0);
        pl = R::owner(sp, pre.u0 + RAGGED_C0 + pre.n - 1);
        pr = ((row - pre.s.row0) << p.lgG) & (R::RT - 1);
        pc = R::cls(p, pre.s);
    }
    const int orow = ((row - own.s.row0) << p.lgG) & (R::RT - 1);
    const int n0 = pl - pf + 1, np = n0 + ol - of + 1;
    for (int g = warp; g < G; g += 4) {
        const int j = h * G + g;
        T* out = static_cast<T*>(p.out) + row * p.out_ts + (int64_t)j * p.D;
        merge_row<T>(p, np, out, lane, [&](int q, const float*& o, const float*& ml) {
            const bool pre = q < n0;
            const int c = pre ? q : q - n0;
            int64_t at;
            if (c == 0 && joint) {
                at = ((int64_t)(pre ? 0 : 1) * p.N + row) * p.H_q + j;
                o = p.row_o + at * p.D;
                ml = p.row_ml + at * 2;
            } else {
                at = (int64_t)R::slot(pre ? pc : oc, (pre ? pf : of) + c, c > 0) * R::SLOT_ROWS + (pre ? pr : orow) + g;
                o = p.slot_o + at * p.D;
                ml = p.slot_ml + at * 2;
            }
        });
    }
}

// Launch behind the attention kernel; starts as that one ends.
template <typename T, class R>
inline int launch_merge(const RaggedParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (p.NG == 0) {
        cfg.gridDim = dim3((unsigned)(3 * p.P), MERGE_SLICES);
        cfg.blockDim = dim3(MERGE_WARPS * 32);
        e = cudaLaunchKernelEx(&cfg, merge_cuts_kernel<T, R>, p);
    } else {
        cfg.gridDim = dim3((unsigned)p.N, (unsigned)p.H_kv);
        cfg.blockDim = dim3(128);
        e = cudaLaunchKernelEx(&cfg, merge_rows_kernel<T, R>, p);
    }
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

}  // namespace kvc
