// kvc_ragged.cu -- attention of ragged new tokens over a paged cache on CUDA cores, in fp32: fp32
// caches, the head dimensions the tensor-core kernel does not take, and math mode 1.
//
// A block walks its share of the streams (kvc_ragged.cuh).  Per key tile: scores of RT rows x
// KT keys, the online softmax of each row, then the weighted sum of V, all from shared memory;
// a thread holds a 4 x (KT / 16) patch of scores and 4 rows x D / 16 columns of the output in
// registers, so each shared-memory vector feeds four products.
#include <type_traits>

#include "kvc_ragged_merge.cuh"

namespace kvc {

template <int D_, bool JOINT>
struct CcCfg {
    static constexpr int D = D_;
    static constexpr int LKT = D > 64 ? 5 : 6;
    static constexpr int RT = 64;
    static constexpr int KT = 1 << LKT;
    using R = Ragged<6, LKT, false, JOINT>;
    static constexpr int NC = KT / 16;           // score columns of a thread
    static constexpr int NV = D < 64 ? 1 : D / 64;  // float4 output columns of a thread
    static constexpr int QS = D + 4, KS = D + 4, PS = KT + 4;  // row strides (floats)
    static constexpr int TILES = (RT * QS + KT * KS + KT * D + RT * PS) * 4;
    static constexpr int PLAN = R::work_ints(MAX_B, MAX_B) * 4;  // the split's arrays lie under the tiles
    static constexpr int SMEM = TILES > PLAN ? TILES : PLAN;
};

// 16 bytes of the cache as floats.
template <typename T>
__device__ __forceinline__ void store_row16(float* dst, const uint4& v, float scale) {
    float f[Elem<T>::VEC];
    Elem<T>::unpack(v, f);
#pragma unroll
    for (int i = 0; i < Elem<T>::VEC; i += 4)
        *reinterpret_cast<float4*>(dst + i) =
            make_float4(f[i] * scale, f[i + 1] * scale, f[i + 2] * scale, f[i + 3] * scale);
}

template <typename T, int D, bool JOINT>
__global__ void __launch_bounds__(256) ragged_cc_kernel(const RaggedParams p) {
    using C = CcCfg<D, JOINT>;
    using R = typename C::R;
    extern __shared__ __align__(16) char smem[];
    __shared__ typename R::Seg seg_s;
    __shared__ typename R::Split split_s;
    float* qs = reinterpret_cast<float*>(smem);
    float* ks = qs + C::RT * C::QS;
    float* vs = ks + C::KT * C::KS;
    float* ps = vs + C::KT * D;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    const typename R::Work work = R::work(p, smem);
    if (tid < 32) {
        const typename R::Split sp = R::scan(p, work, tid);
        if (tid == 0) split_s = sp;
    }
    __syncthreads();
    const typename R::Split sp = split_s;
    if (blockIdx.x == 0) {
        const int n = 2 * (R::groups(p) + p.B + 1);
        for (int i = tid; i < n; i += 256) p.plan[i] = sp.valid ? work.c[i] : 0;
        if (!sp.valid && tid == 0) atomicOr(p.err, DEV_BAD_SEQ);
    }
    if (tid < 6) p.cuts[6 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
    if (sp.valid) ragged_zero_rows<T, JOINT>(p, tid, 256);
    typename R::Walk wk;
    if (tid == 0) wk = R::walk(p, sp, work, blockIdx.x, 1);

    while (true) {
        __syncthreads();  // the prefix sums (or the last segment's tiles) are read
        if (tid == 0) {
            seg_s = R::next_seg(p, wk);
            if (wk.cut) R::leave_cut(p, sp, wk, blockIdx.x, 1, seg_s);
        }
        __syncthreads();
        const typename R::Seg g = seg_s;
        if (g.n == 0) return;
        const int G = 1 << p.lgG, nrow = g.ntok << p.lgG;
        constexpr int VPR = D * Elem<T>::BYTES / 16;  // 16-byte vectors of a row
        for (int i = tid; i < C::RT * VPR; i += 256) {
            const int r = i / VPR, v = i - r * VPR;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < nrow) {
                const T* src = static_cast<const T*>(p.q) + (int64_t)(g.row0 + (r >> p.lgG)) * p.q_ts +
                               (int64_t)(g.h * G + (r & (G - 1))) * D;
                w = __ldg(reinterpret_cast<const uint4*>(src) + v);
            }
            store_row16<T>(qs + r * C::QS + v * Elem<T>::VEC, w, p.qscale);
        }
        float m[4], l[4];
        float4 acc[4][C::NV];
        int lim[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            lim[i] = min(g.kv_end, g.lim0 + g.causal * ((ty + 16 * i) >> p.lgG));
#pragma unroll
            for (int v = 0; v < C::NV; ++v) acc[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int j = 0; j < g.n; ++j) {
            const int t0 = g.kv0 + j * C::KT;
            if (j > 0) __syncthreads();
            for (int i = tid; i < C::KT * VPR; i += 256) {
                const int t = i / VPR, v = i - t * VPR;
                uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
                if (t0 + t < g.kv_end) {
                    const int64_t row = cache_row_rd(p.table, p.bs, p.max_blocks, p.num_blocks, p.H_kv, p.T_max, g.seq,
                                                     g.h, t0 + t, p.err);
                    kw = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.K) + row * D) + v);
                    vw = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.V) + row * D) + v);
                }
                store_row16<T>(ks + t * C::KS + v * Elem<T>::VEC, kw, 1.f);
                store_row16<T>(vs + t * D + v * Elem<T>::VEC, vw, 1.f);
            }
            __syncthreads();
            float s[4][C::NC];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < C::NC; ++c) s[i][c] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 kv[C::NC];
#pragma unroll
                for (int c = 0; c < C::NC; ++c) kv[c] = *reinterpret_cast<const float4*>(ks + (tx + 16 * c) * C::KS + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ty + 16 * i >= nrow) continue;
                    const float4 q = *reinterpret_cast<const float4*>(qs + (ty + 16 * i) * C::QS + d);
#pragma unroll
                    for (int c = 0; c < C::NC; ++c)
                        s[i][c] = fmaf(q.x, kv[c].x, fmaf(q.y, kv[c].y, fmaf(q.z, kv[c].z, fmaf(q.w, kv[c].w, s[i][c]))));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < C::NC; ++c) {
                    if (t0 + tx + 16 * c >= lim[i]) s[i][c] = -INFINITY;
                    mx = fmaxf(mx, s[i][c]);
                }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                mx = fmaxf(mx, m[i]);
                const float mu = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: weights 2^-inf = 0
                const float corr = fast_exp2(m[i] - mu);
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < C::NC; ++c) {
                    const float w = fast_exp2(s[i][c] - mu);
                    sum += w;
                    ps[(ty + 16 * i) * C::PS + tx + 16 * c] = w;
                }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
                l[i] = l[i] * corr + sum;
                m[i] = mx;
#pragma unroll
                for (int v = 0; v < C::NV; ++v) {
                    acc[i][v].x *= corr;
                    acc[i][v].y *= corr;
                    acc[i][v].z *= corr;
                    acc[i][v].w *= corr;
                }
            }
            __syncwarp();  // a row's weights come from its own half-warp
            const bool masked = t0 + C::KT > g.lim0;  // some row does not see the whole tile
            if (D >= 64 || tx == 0) {
                // A weight of an unseen position is 0, but 0 times an infinite or NaN value is NaN: in
                // masked tiles such products are left out.
                auto sum_tile = [&](auto guard) {
#pragma unroll 2
                    for (int t = 0; t < C::KT; t += 4) {
                        float4 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = *reinterpret_cast<const float4*>(ps + (ty + 16 * i) * C::PS + t);
#pragma unroll
                        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                            for (int v = 0; v < C::NV; ++v) {
                                const float4 x = *reinterpret_cast<const float4*>(vs + (t + tt) * D + v * 64 + tx * 4);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if (ty + 16 * i >= nrow) continue;
                                    if (guard && t0 + t + tt >= lim[i]) continue;
                                    const float f = tt == 0 ? w[i].x : tt == 1 ? w[i].y : tt == 2 ? w[i].z : w[i].w;
                                    acc[i][v].x = fmaf(f, x.x, acc[i][v].x);
                                    acc[i][v].y = fmaf(f, x.y, acc[i][v].y);
                                    acc[i][v].z = fmaf(f, x.z, acc[i][v].z);
                                    acc[i][v].w = fmaf(f, x.w, acc[i][v].w);
                                }
                            }
                    }
                };
                if (masked) sum_tile(std::true_type{});
                else sum_tile(std::false_type{});
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            if (r >= nrow || (D < 64 && tx > 0)) continue;
            const int64_t row = g.row0 + (r >> p.lgG);
            const int head = g.h * G + (r & (G - 1));
            if (g.dst == -1) {
                const float inv = 1.f / l[i];
                T* out = static_cast<T*>(p.out) + row * p.out_ts + (int64_t)head * D;
#pragma unroll
                for (int v = 0; v < C::NV; ++v) {
                    const int d = v * 64 + tx * 4;
                    if constexpr (sizeof(T) == 2) {
                        *reinterpret_cast<uint2*>(out + d) =
                            make_uint2(bf16x2_rn(acc[i][v].x * inv, acc[i][v].y * inv),
                                       bf16x2_rn(acc[i][v].z * inv, acc[i][v].w * inv));
                    } else {
                        *reinterpret_cast<float4*>(out + d) = make_float4(acc[i][v].x * inv, acc[i][v].y * inv,
                                                                          acc[i][v].z * inv, acc[i][v].w * inv);
                    }
                }
            } else {
                float *o, *ml;
                ragged_dst(p, g.dst, R::SLOT_ROWS, r, row, head, o, ml);
#pragma unroll
                for (int v = 0; v < C::NV; ++v) *reinterpret_cast<float4*>(o + v * 64 + tx * 4) = acc[i][v];
                if (tx == 0) *reinterpret_cast<float2*>(ml) = make_float2(m[i], l[i]);
            }
        }
    }
}

template <typename T, int D, bool JOINT>
static int launch_cc_as(const RaggedParams& p, cudaStream_t s) {
    using C = CcCfg<D, JOINT>;
    static PerDeviceOnce once;
    const int e0 = once.run([] {
        return (int)cudaFuncSetAttribute(ragged_cc_kernel<T, D, JOINT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e0 != 0) return e0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)p.P);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ragged_cc_kernel<T, D, JOINT>, p);
    if (e != cudaSuccess) return (int)e;
    return launch_merge<T, typename C::R, JOINT>(p, s);
}
template <typename T, int D>
static int launch_cc(const RaggedParams& p, cudaStream_t s) {
    return p.NG > 0 ? launch_cc_as<T, D, true>(p, s) : launch_cc_as<T, D, false>(p, s);
}

int launch_ragged_cc(int dtype, const RaggedParams& p, cudaStream_t s) {
    if (dtype == 0) switch (p.D) {
        case 64: return launch_cc<__nv_bfloat16, 64>(p, s);
        case 128: return launch_cc<__nv_bfloat16, 128>(p, s);
        case 256: return launch_cc<__nv_bfloat16, 256>(p, s);
        default: return (int)cudaErrorInvalidValue;
    }
    switch (p.D) {
        case 4: return launch_cc<float, 4>(p, s);
        case 64: return launch_cc<float, 64>(p, s);
        case 128: return launch_cc<float, 128>(p, s);
        case 256: return launch_cc<float, 256>(p, s);
        default: return (int)cudaErrorInvalidValue;
    }
}

}  // namespace kvc
