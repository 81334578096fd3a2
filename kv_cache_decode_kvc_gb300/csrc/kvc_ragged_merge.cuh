// kvc_ragged_merge.cuh -- merge of the pieces of split streams (see kvc_ragged.cuh), launched
// behind an attention kernel with the split R.
//
// States (m_i, l_i, o_i) of disjoint key sets merge to M = max m_i, sum 2^(m_i - M) l_i, sum 2^(m_i - M) o_i,
// here in the fixed order of the pieces.  Bound by latency, not by bytes (two to three states of D + 2
// floats per cut row, mostly from L2): a chain of lookups, then the pieces' loads all in flight.  So few
// dependent loads count: finding a row's sequence and group by two warp-wide loads instead of by halving
// took 256 tokens behind a prefix from 132.1 to 130.3 us and 64 MQA drafts from 42.4 to 41.3 us.
#pragma once

#include <type_traits>

#include "kvc_ragged.cuh"

namespace kvc {

constexpr int MERGE_WARPS = 8;
// More pieces than this: the block's warps share a row (one sequence of 131,000 positions on one KV head,
// 304 pieces of 32 rows: 38 us in all, a warp to a row 105; 4 to 16 take the same).
constexpr int MERGE_WIDE = 16;

// Softmax state of one output row, a warp's lanes holding columns 4 lane .. and 128 + 4 lane ..
struct MergeAcc {
    float m, l;
    float4 o[2];
};

// Pieces i0, i0 + step, .. below np of one row, in order: state(i, o, ml) gives piece i's address.
// Their merged state is (M, sum w_i l_i, sum w_i o_i) with M = max m_i, w_i = 2^(m_i - M); a piece that
// saw nothing (l = 0) has weight 0; NaN scores reach l and o and stay NaN.  The lanes fetch the
// pieces' (m, l) together, then the outputs are independent loads.
template <class F>
__device__ __forceinline__ MergeAcc merge_pieces(const RaggedParams& p, int np, int i0, int step, int lane, F&& state) {
    MergeAcc a;
    a.m = -INFINITY;
    a.l = 0.f;
    a.o[0] = a.o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = i0; i < np; i += 32 * step) {
        const int n = min(32, (np - i + step - 1) / step);
        float2 s = make_float2(-INFINITY, 0.f);
        if (lane < n) {
            const float *o, *ml;
            state(i + lane * step, o, ml);
            s = __ldcg(reinterpret_cast<const float2*>(ml));
        }
        float M = fmaxf(a.m, s.x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
        const float mu = M == -INFINITY ? 0.f : M;
        const float f = fast_exp2(a.m - mu);  // 0 while nothing has been added
        const float w = s.y == 0.f ? 0.f : fast_exp2(s.x - mu);
        float wl = s.y == 0.f ? 0.f : w * s.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) wl += __shfl_xor_sync(0xFFFFFFFFu, wl, off);
        a.l = a.l * f + wl;
        a.m = M;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            a.o[v].x *= f;
            a.o[v].y *= f;
            a.o[v].z *= f;
            a.o[v].w *= f;
        }
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float *o, *ml;
            state(i + k * step, o, ml);
            const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
            const bool any = __shfl_sync(0xFFFFFFFFu, s.y, k) != 0.f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int d = lane * 4 + v * 128;
                if (d < p.D) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(o + d));
                    if (any) {
                        a.o[v].x = fmaf(wk, x.x, a.o[v].x);
                        a.o[v].y = fmaf(wk, x.y, a.o[v].y);
                        a.o[v].z = fmaf(wk, x.z, a.o[v].z);
                        a.o[v].w = fmaf(wk, x.w, a.o[v].w);
                    }
                }
            }
        }
    }
    return a;
}
template <typename T>
__device__ __forceinline__ void merge_store(const RaggedParams& p, const MergeAcc& a, T* out, int lane) {
    const float inv = 1.f / a.l;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int d = lane * 4 + v * 128;
        if (d < p.D) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2*>(out + d) = make_uint2(bf16x2_rn(a.o[v].x * inv, a.o[v].y * inv),
                                                                bf16x2_rn(a.o[v].z * inv, a.o[v].w * inv));
            else
                *reinterpret_cast<float4*>(out + d) = make_float4(a.o[v].x * inv, a.o[v].y * inv, a.o[v].z * inv, a.o[v].w * inv);
        }
    }
}
// All warps of the block on one row (every thread takes part): warp w of n merges pieces w, w + n,
// .., the first warp their states in order.
template <typename T, class F>
__device__ __forceinline__ void merge_row_wide(const RaggedParams& p, int np, T* out, int warp, int lane, F&& state) {
    __shared__ float so[MERGE_WARPS][256], sml[MERGE_WARPS][2];
    const int nw = blockDim.x >> 5;
    const MergeAcc a = merge_pieces(p, np, warp, nw, lane, state);
#pragma unroll
    for (int v = 0; v < 2; ++v)
        if (lane * 4 + v * 128 < p.D) *reinterpret_cast<float4*>(&so[warp][lane * 4 + v * 128]) = a.o[v];
    if (lane == 0) {
        sml[warp][0] = a.m;
        sml[warp][1] = a.l;
    }
    __syncthreads();
    if (warp == 0) {
        float M = -INFINITY;
        for (int w = 0; w < nw; ++w) M = fmaxf(M, sml[w][0]);
        const float mu = M == -INFINITY ? 0.f : M;
        MergeAcc b;
        b.m = M;
        b.l = 0.f;
        b.o[0] = b.o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < nw; ++w) {
            if (sml[w][1] == 0.f) continue;
            const float f = fast_exp2(sml[w][0] - mu);
            b.l += f * sml[w][1];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (lane * 4 + v * 128 >= p.D) continue;
                const float4 x = *reinterpret_cast<const float4*>(&so[w][lane * 4 + v * 128]);
                b.o[v].x = fmaf(f, x.x, b.o[v].x);
                b.o[v].y = fmaf(f, x.y, b.o[v].y);
                b.o[v].z = fmaf(f, x.z, b.o[v].z);
                b.o[v].w = fmaf(f, x.w, b.o[v].w);
            }
        }
        merge_store<T>(p, b, out, lane);
    }
    __syncthreads();
}

// NP pieces, two to four, the common cuts: a warp merges ILP rows at once (all their loads in flight).  Three and four in
// the order and with the roundings of merge_pieces; of two, the second denominator is added to the first by one fma (products
// and sums are written out: left to the compiler, which of them become one fma is its choice).  (Three and four pieces taken so as well: 24 sequences, 4 with chunks of up to 300 tokens, over an 8-bit
// cache 165 -> 156 us.)
template <int NP, int ILP, typename T, class Out, class At>
__device__ __forceinline__ void merge_few(const RaggedParams& p, int r0, int step, int rows, int lane, Out&& out_of, At&& at_row) {
    float4 x[ILP][NP][2];
    float2 s[ILP][NP];
#pragma unroll
    for (int k = 0; k < ILP; ++k)
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const int r = min(r0 + k * step, rows - 1);
            const float *o, *ml;
            at_row(r)(q, o, ml);
            s[k][q] = __ldcg(reinterpret_cast<const float2*>(ml));
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (lane * 4 + v * 128 < p.D) x[k][q][v] = __ldcg(reinterpret_cast<const float4*>(o + lane * 4 + v * 128));
        }
#pragma unroll
    for (int k = 0; k < ILP; ++k) {
        if (r0 + k * step >= rows) break;
        float M = s[k][0].x;
#pragma unroll
        for (int q = 1; q < NP; ++q) M = fmaxf(M, s[k][q].x);
        const float mu = M == -INFINITY ? 0.f : M;
        MergeAcc a;
        a.m = M;
        a.o[0] = a.o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        float l[4] = {};
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            if (s[k][q].y == 0.f) continue;
            const float w = fast_exp2(s[k][q].x - mu);
            l[q] = NP == 2 && q == 1 ? fmaf(w, s[k][q].y, l[0]) : __fmul_rn(w, s[k][q].y);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (lane * 4 + v * 128 >= p.D) continue;
                a.o[v].x = fmaf(w, x[k][q][v].x, a.o[v].x);
                a.o[v].y = fmaf(w, x[k][q][v].y, a.o[v].y);
                a.o[v].z = fmaf(w, x[k][q][v].z, a.o[v].z);
                a.o[v].w = fmaf(w, x[k][q][v].w, a.o[v].w);
            }
        }
        if constexpr (NP == 2) a.l = s[k][1].y == 0.f ? l[0] : l[1];
        else a.l = (l[0] + l[2]) + (l[1] + l[3]);
        merge_store<T>(p, a, out_of(r0 + k * step), lane);
    }
}

// Blocks that share the rows of a cut.  (One for 16 or 32 rows, which its warps hold at once: all cuts' blocks then run
// in one go.)
template <class R>
constexpr int MERGE_SLICES = R::SLOT_ROWS < 8 * MERGE_WARPS ? 1 : 8;
// Without groups: block (c, y) takes the c-th possible cut; if a stream was cut there first, its
// warps merge the rows of the stream's tile from row 8 y on, every 64th eight of them.  With many pieces
// the blocks of all its cuts take its rows in turn, one by one.
template <typename T, class R>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_cuts_kernel(const RaggedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = R::SLOTS > 2 ? blockIdx.x : 3 * blockIdx.x + 1;
    const int4 a = __ldcg(p.cuts + 2 * e), b = __ldcg(p.cuts + 2 * e + 1);
    if (a.x == 0 || (a.x <= MERGE_WIDE && b.z > 0)) return;
    const int G = 1 << p.lgG;
    auto out_of = [&](int r) {
        return static_cast<T*>(p.out) + (int64_t)(a.w + (r >> p.lgG)) * p.out_ts + (int64_t)(b.y * G + (r & (G - 1))) * p.D;
    };
    auto at_row = [&](int r) {
        return [&p, &a, r](int q, const float*& o, const float*& ml) {
            const int64_t at = (int64_t)R::slot(a.z, a.y + q, q > 0) * R::SLOT_ROWS + r;
            o = p.slot_o + at * p.D;
            ml = p.slot_ml + at * 2;
        };
    };
    auto few = [&](auto np, auto ilp) {
        constexpr int NP = decltype(np)::value, ILP = decltype(ilp)::value, STEP = MERGE_SLICES<R> * MERGE_WARPS;
        for (int r = blockIdx.y * MERGE_WARPS + warp; r < b.x; r += ILP * STEP)
            merge_few<NP, ILP, T>(p, r, STEP, b.x, lane, out_of, at_row);
    };
    using std::integral_constant;
    if (a.x == 2) return few(integral_constant<int, 2>{}, integral_constant<int, 4>{});
    if (a.x == 3) return few(integral_constant<int, 3>{}, integral_constant<int, 2>{});
    if (a.x == 4) return few(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    if (a.x > MERGE_WIDE) {
        for (int r = b.z * MERGE_SLICES<R> + blockIdx.y; r < b.x; r += (a.x - 1) * MERGE_SLICES<R>)
            merge_row_wide<T>(p, a.x, out_of(r), warp, lane, at_row(r));
        return;
    }
    for (int r = blockIdx.y * MERGE_WARPS + warp; r < b.x; r += MERGE_SLICES<R> * MERGE_WARPS)
        merge_store<T>(p, merge_pieces(p, a.x, 0, 1, lane, at_row(r)), out_of(r), lane);
}

// The last i < n <= MAX_B with a[i] <= x of an ascending array with a[0] <= x, by a converged warp in two
// loads one behind the other (halving it takes up to ten).
__device__ __forceinline__ int last_at(const int* a, int n, int x, int lane) {
    static_assert(MAX_B <= 32 * 32);
    const int b = 32 * (__popc(__ballot_sync(0xFFFFFFFFu, 32 * lane < n && __ldg(a + 32 * lane) <= x)) - 1);
    return b + __popc(__ballot_sync(0xFFFFFFFFu, b + lane < n && __ldg(a + b + lane) <= x)) - 1;
}

// With groups: block (row, KV head, y), a warp per query head 8 y + warp of the group; the row's
// pieces are those of its prefix stream and of its sequence's own stream.
template <typename T, class R>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_rows_kernel(const RaggedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const typename R::Split sp = R::planned(p);
    if (!sp.valid) return;
    const int row = blockIdx.x, h = blockIdx.y, G = 1 << p.lgG;
    if (row >= __ldg(p.cu + p.B)) return;
    const int lo = last_at(p.cu, p.B, row, lane);  // the sequence
    const int a = last_at(p.groups, p.NG, lo, lane), b0 = __ldg(p.groups + a), b1 = __ldg(p.groups + a + 1);
    const int P = __ldg(p.prefix + a), used = prefix_used(p, b0, b1, P);
    const typename R::Stream own =
        R::of_row(p, sp, p.plan, p.NG + lo, seq_entry(p, lo, __ldg(p.cu + lo), __ldg(p.cu + lo + 1), __ldg(p.lens + lo), P, used), h, row);
    if (!own.s.ok) return;
    const int oc = R::cls(p, own.s);
    const int of = R::owner_of(sp, own, oc, 0), ol = R::owner_of(sp, own, oc, own.n - 1);
    const bool joint = own.s.pfx > 0;
    if (!joint && of == ol) return;  // written by its worker
    int pf = 0, pl = -1, pr = 0, pc = 0;
    if (joint) {
        const typename R::Stream pre =
            R::of_row(p, sp, p.plan, a, group_entry(b0, __ldg(p.cu + b0), __ldg(p.cu + b1), used), h, row);
        pc = R::cls(p, pre.s);
        pf = R::owner_of(sp, pre, pc, 0);
        pl = R::owner_of(sp, pre, pc, pre.n - 1);
        pr = ((row - pre.s.row0) << p.lgG) & (R::RT - 1);
    }
    const int orow = ((row - own.s.row0) << p.lgG) & (R::RT - 1);
    const int n0 = pl - pf + 1, np = n0 + ol - of + 1;
    auto out_of = [&](int g) { return static_cast<T*>(p.out) + (int64_t)row * p.out_ts + (int64_t)(h * G + g) * p.D; };
    auto at_head = [&](int g) {
        return [&, g](int q, const float*& o, const float*& ml) {
            const bool pre = q < n0;
            const int c = pre ? q : q - n0;
            if (c == 0 && joint) {
                const int64_t at = ((int64_t)(pre ? 0 : 1) * p.N + row) * p.H_q + h * G + g;
                o = p.row_o + at * p.D;
                ml = p.row_ml + at * 2;
            } else {
                const int64_t at = (int64_t)R::slot(pre ? pc : oc, (pre ? pf : of) + c, c > 0) * R::SLOT_ROWS + (pre ? pr : orow) + g;
                o = p.slot_o + at * p.D;
                ml = p.slot_ml + at * 2;
            }
        };
    };
    const int g0 = blockIdx.z * MERGE_WARPS;
    if (np > MERGE_WIDE) {
        for (int g = g0; g < min(g0 + MERGE_WARPS, G); ++g) merge_row_wide<T>(p, np, out_of(g), warp, lane, at_head(g));
    } else if (g0 + warp < G) {
        merge_store<T>(p, merge_pieces(p, np, 0, 1, lane, at_head(g0 + warp)), out_of(g0 + warp), lane);
    }
}

// With groups, where entries of many rows were attended by the kernel with split RA (parameters pa) and the others by
// that with split RB (pb): as merge_rows_kernel, each of the row's two streams from its own kernel's pieces.  (The row
// buffers are one.)
template <typename T, class RA, class RB>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_parts_kernel(const RaggedParams pa, const RaggedParams pb) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RaggedParams& p = pb;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const typename RA::Split spa = RA::planned(pa);
    const typename RB::Split spb = RB::planned(pb);
    if (!spa.valid && !spb.valid) return;
    const int row = blockIdx.x, h = blockIdx.y, G = 1 << p.lgG;
    if (row >= __ldg(p.cu + p.B)) return;
    const int lo = last_at(p.cu, p.B, row, lane);  // the sequence
    const int a = last_at(p.groups, p.NG, lo, lane), b0 = __ldg(p.groups + a), b1 = __ldg(p.groups + a + 1);
    const int P = __ldg(p.prefix + a), used = prefix_used(p, b0, b1, P);
    // A stream's pieces: how many, the first one's owner, class, the row's place in its tile, which kernel's.
    struct Pieces {
        int n, first, cl, row;
        bool many;
    };
    auto pieces = [&](int e, const Entry& s) {
        Pieces x;
        x.many = !in_part(pb, s);
        x.n = 0;
        auto find = [&](auto r, const auto& sp, const RaggedParams& q) {
            if (!sp.valid) return;  // (a part that was refused as too large has left no split)
            using R = decltype(r);
            const typename R::Stream st = R::of_row(q, sp, q.plan, e, s, h, row);
            x.cl = R::cls(q, s);
            x.first = R::owner_of(sp, st, x.cl, 0);
            x.n = R::owner_of(sp, st, x.cl, st.n - 1) - x.first + 1;
            x.row = ((row - s.row0) << p.lgG) & (R::RT - 1);
        };
        if (x.many) find(RA{}, spa, pa);
        else find(RB{}, spb, pb);
        return x;
    };
    const Entry own = seq_entry(p, lo, __ldg(p.cu + lo), __ldg(p.cu + lo + 1), __ldg(p.lens + lo), P, used);
    if (!own.ok) return;
    const Pieces po = pieces(p.NG + lo, own);
    const bool joint = own.pfx > 0;
    if (po.n == 0 || (!joint && po.n == 1)) return;  // (written by its worker)
    Pieces pp;
    pp.n = 0;
    if (joint) {
        pp = pieces(a, group_entry(b0, __ldg(p.cu + b0), __ldg(p.cu + b1), used));
        if (pp.n == 0) return;
    }
    const int np = pp.n + po.n;
    auto out_of = [&](int g) { return static_cast<T*>(p.out) + (int64_t)row * p.out_ts + (int64_t)(h * G + g) * p.D; };
    auto at_head = [&](int g) {
        return [&, g](int q, const float*& o, const float*& ml) {
            const bool pre = q < pp.n;
            const int c = pre ? q : q - pp.n;
            if (c == 0 && joint) {
                const int64_t at = ((int64_t)(pre ? 0 : 1) * p.N + row) * p.H_q + h * G + g;
                o = p.row_o + at * p.D;
                ml = p.row_ml + at * 2;
                return;
            }
            const int cl = pre ? pp.cl : po.cl, owner = (pre ? pp.first : po.first) + c, r = (pre ? pp.row : po.row) + g;
            const bool many = pre ? pp.many : po.many;
            const RaggedParams& k = many ? pa : pb;
            const int64_t at = (many ? (int64_t)RA::slot(cl, owner, c > 0) * RA::SLOT_ROWS
                                     : (int64_t)RB::slot(cl, owner, c > 0) * RB::SLOT_ROWS) + r;
            o = k.slot_o + at * p.D;
            ml = k.slot_ml + at * 2;
        };
    };
    const int g0 = blockIdx.z * MERGE_WARPS;
    if (np > MERGE_WIDE) {
        for (int g = g0; g < min(g0 + MERGE_WARPS, G); ++g) merge_row_wide<T>(p, np, out_of(g), warp, lane, at_head(g));
    } else if (g0 + warp < G) {
        merge_store<T>(p, merge_pieces(p, np, 0, 1, lane, at_head(g0 + warp)), out_of(g0 + warp), lane);
    }
}
template <typename T, class RA, class RB>
inline int launch_merge_parts(const RaggedParams& pa, const RaggedParams& pb, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int G = 1 << pb.lgG;
    cfg.gridDim = dim3((unsigned)pb.N, (unsigned)pb.H_kv, (unsigned)((G + MERGE_WARPS - 1) / MERGE_WARPS));
    cfg.blockDim = dim3((unsigned)((G < 4 ? 4 : (G < MERGE_WARPS ? G : MERGE_WARPS)) * 32));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, merge_parts_kernel<T, RA, RB>, pa, pb);
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

// Launch behind the attention kernel; starts as that one ends.  (Released early, by the attention kernel or the merge, what
// follows is no sooner done and takes the SMs from blocks not yet begun: 256 tokens behind 16,384 common positions 191 us
// against 155, 24 tokens behind 2048 on an 8-bit cache 51.5 against 47.7.)
template <typename T, class R, bool JOINT>
inline int launch_merge(const RaggedParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if constexpr (!JOINT) {
        cfg.gridDim = dim3((unsigned)(R::SLOTS > 2 ? 3 * p.P : p.P), MERGE_SLICES<R>);
        cfg.blockDim = dim3(MERGE_WARPS * 32);
        e = cudaLaunchKernelEx(&cfg, merge_cuts_kernel<T, R>, p);
    } else {
        const int G = 1 << p.lgG;
        cfg.gridDim = dim3((unsigned)p.N, (unsigned)p.H_kv, (unsigned)((G + MERGE_WARPS - 1) / MERGE_WARPS));
        cfg.blockDim = dim3((unsigned)((G < 4 ? 4 : (G < MERGE_WARPS ? G : MERGE_WARPS)) * 32));
        e = cudaLaunchKernelEx(&cfg, merge_rows_kernel<T, R>, p);
    }
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

}  // namespace kvc
