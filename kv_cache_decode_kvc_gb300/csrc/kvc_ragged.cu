// kvc_ragged.cu -- attention of ragged new tokens over a paged cache on CUDA cores, in fp32: fp32
// caches, the head dimensions the tensor-core kernel does not take, and math mode 1.
//
// A block walks its share of the streams (kvc_ragged.cuh), found one ahead by a warp of its own.  Per key
// tile: scores of RT rows x KT keys, the online softmax of each row, then the weighted sum of V, all from
// shared memory, the next tile's copies in flight meanwhile (cp.async, two buffers).  A thread holds a
// patch of 4 rows x KT / 8 scores and 4 rows x D / 8 columns of the output in registers (/ 16 at D = 256,
// where the output would not fit), each shared-memory vector feeds four or eight products, and two
// products are one instruction (fma.rn.f32x2).
//
// Bound by the fp32 units at about half their rate: 16 x 333 fp32 tokens behind 1700 positions, 8 heads on
// 2, D = 64 take 602 us, 34 TFLOP/s (fma pipe 50 % busy, shared memory 61 %; stalls: fixed latencies, then
// the barrier of a tile, with 8 warps an SM).  4 x 4 patches of 256 threads took 667, loads without the
// second buffer and single products 698; D = 256 in bf16 2465 against 4870.
#include <type_traits>

#include "kvc_ragged_merge.cuh"

namespace kvc {

template <typename T, int D_, bool JOINT>
struct CcCfg {
    static constexpr int D = D_;
    static constexpr int LKT = D > 64 ? 5 : 6;
    static constexpr int RT = 64;
    static constexpr int KT = 1 << LKT;
    using R = Ragged<6, LKT, false, JOINT>;
    static constexpr int LTX = D > 128 ? 4 : 3, TX = 1 << LTX;  // threads of a row
    static constexpr int NT = RT / 4 * TX;                      // threads that attend
    static constexpr int NC = KT / TX;                          // score columns of a thread
    static constexpr int NV = D < 4 * TX ? 1 : D / (4 * TX);    // output columns of a thread, by fours
    static constexpr int PAD = 16 / sizeof(T);
    static constexpr int QS = D + PAD, KS = D + PAD, PS = KT + 4;  // row strides (elements)
    static constexpr int KV = KT * KS + KT * D;                    // a K and a V tile (elements)
    static constexpr int TILES = (RT * QS + 2 * KV) * (int)sizeof(T) + RT * PS * 4;
    static constexpr int PLAN = R::work_ints(MAX_B, MAX_B) * 4;  // the split's arrays lie under the tiles
    static constexpr int SMEM = TILES > PLAN ? TILES : PLAN;
    static constexpr int THREADS = NT + 32;  // a warp finds the segments
};

// 16 bytes to shared memory behind the caller's back; zeros where there is nothing to read.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two products at once: two fp32 multiply-adds are one instruction.
union Two {
    float2 f;
    uint64_t u;
};
__device__ __forceinline__ void fma_two(Two& d, const Two& a, const Two& b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d.u) : "l"(a.u), "l"(b.u));
}
__device__ __forceinline__ void mul_two(Two& d, const Two& a) {
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d.u) : "l"(a.u));
}
struct Four {
    Two lo, hi;
};
__device__ __forceinline__ Four load4(const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    Four r;
    r.lo.f = make_float2(v.x, v.y);
    r.hi.f = make_float2(v.z, v.w);
    return r;
}
__device__ __forceinline__ Four load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    Four r;
    r.lo.f = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    r.hi.f = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
    return r;
}

template <typename T, int D, bool JOINT>
__global__ void __launch_bounds__(CcCfg<T, D, JOINT>::THREADS, D > 128 ? 1 : 2) ragged_cc_kernel(const RaggedParams p) {
    using C = CcCfg<T, D, JOINT>;
    using R = typename C::R;
    extern __shared__ __align__(16) char smem[];
    __shared__ typename R::Seg seg_s[2];
    __shared__ typename R::Split split_s;
    T* qs = reinterpret_cast<T*>(smem);
    T* kvs = qs + C::RT * C::QS;
    float* ps = reinterpret_cast<float*>(kvs + 2 * C::KV);
    const int tid = threadIdx.x, tx = tid & (C::TX - 1), ty = tid >> C::LTX;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    const typename R::Work work = R::work(p, smem);
    if (tid >= C::NT) {
        const typename R::Split sp = R::scan(p, work, tid - C::NT);
        if (tid == C::NT) split_s = sp;
    }
    __syncthreads();
    const typename R::Split sp = split_s;
    if (blockIdx.x == 0) {
        const int n = 2 * (R::groups(p) + p.B + 1);
        for (int i = tid; i < n; i += C::THREADS) p.plan[i] = sp.valid ? work.c[i] : 0;
        if (!sp.valid && tid == 0) atomicOr(p.err, sp.why);
    }
    if (tid >= C::NT) {  // the segments, one ahead of the threads that attend them
        // The block's cuts start out empty.  The warp that leaves them (leave_cut) empties them: from another
        // warp nothing would order the two writes, and a cut that is lost is a stream that is never merged.
        if (tid - C::NT < 6) p.cuts[6 * blockIdx.x + tid - C::NT] = make_int4(0, 0, 0, 0);
        __syncwarp();
        typename R::Walk wk;
        if (tid == C::NT) wk = R::walk(p, sp, work, blockIdx.x, 1);
        for (int s = 0;; ++s) {
            if (tid == C::NT) {
                seg_s[s & 1] = R::next_seg(p, wk);
                if (wk.cut) R::leave_cut(p, sp, wk, blockIdx.x, 1, seg_s[s & 1]);
            }
            __syncwarp();
            const bool last = *(volatile int*)&seg_s[s & 1].n == 0;
            __syncthreads();
            if (last) return;
        }
    }
    if (sp.valid) ragged_zero_rows<T, JOINT>(p, tid, C::NT);

    constexpr int VPR = D * (int)sizeof(T) / 16, VEC = 16 / (int)sizeof(T);  // 16-byte vectors of a row
    for (int seg = 0;; ++seg) {
        __syncthreads();  // the prefix sums (or the last segment's tiles) are read, the segment is there
        const typename R::Seg& g = seg_s[seg & 1];  // read there: copies would not fit the registers
        if (g.n == 0) return;
        const int G = 1 << p.lgG, nrow = g.ntok << p.lgG;
        auto fetch = [&](int j) {
            T* ks = kvs + (j & 1) * C::KV;
            T* vs = ks + C::KT * C::KS;
            const int t0 = g.kv0 + j * C::KT;
            for (int i = tid; i < C::KT * VPR; i += C::NT) {
                const int t = i / VPR, v = (i - t * VPR) * VEC;
                const bool there = t < g.kv_end - t0;  // (t0 + t may pass 2^31)
                int64_t row = 0;
                if (there)
                    row = cache_row_rd(p.table, p.bs, p.max_blocks, p.num_blocks, p.H_kv, p.T_max, g.seq, g.h, t0 + t, p.err);
                copy16(ks + t * C::KS + v, static_cast<const T*>(p.K) + row * D + v, there);
                copy16(vs + t * D + v, static_cast<const T*>(p.V) + row * D + v, there);
            }
        };
        for (int i = tid; i < C::RT * VPR; i += C::NT) {
            const int r = i / VPR, v = (i - r * VPR) * VEC;
            const int rr = min(r, nrow - 1);
            copy16(qs + r * C::QS + v,
                   static_cast<const T*>(p.q) + (int64_t)(g.row0 + (rr >> p.lgG)) * p.q_ts +
                       (int64_t)(g.h * G + (rr & (G - 1))) * D + v,
                   r < nrow);
        }
        fetch(0);
        const bool live = (tid >> 5) * (128 >> C::LTX) < nrow;  // alike in a warp
        float m[4], l[4];
        Four acc[4][C::NV];
        unsigned lim[4];  // (as positions of a tile: unsigned, they may pass 2^31)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
            lim[i] = g.sees((ty * 4 + i) >> p.lgG);
#pragma unroll
            for (int v = 0; v < C::NV; ++v) acc[i][v].lo.f = acc[i][v].hi.f = make_float2(0.f, 0.f);
        }
        for (int j = 0; j < g.n; ++j) {
            const unsigned t0 = g.kv0 + j * C::KT;
            const T* ks = kvs + (j & 1) * C::KV;
            const T* vs = ks + C::KT * C::KS;
            copies_done();
            named_bar_sync(1, C::NT);  // tile j is there, tile j - 1 is read
            if (j + 1 < g.n) fetch(j + 1);
            if (!live) continue;
            Two s[4][C::NC];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < C::NC; ++c) s[i][c].f = make_float2(0.f, 0.f);
#pragma unroll 2
            for (int d = 0; d < D; d += 4) {
                Four kv[C::NC];
#pragma unroll
                for (int c = 0; c < C::NC; ++c) kv[c] = load4(ks + (tx + C::TX * c) * C::KS + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Four q = load4(qs + (ty * 4 + i) * C::QS + d);
#pragma unroll
                    for (int c = 0; c < C::NC; ++c) {
                        fma_two(s[i][c], q.lo, kv[c].lo);
                        fma_two(s[i][c], q.hi, kv[c].hi);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY, x[C::NC];
#pragma unroll
                for (int c = 0; c < C::NC; ++c) {
                    x[c] = t0 + tx + C::TX * c < lim[i] ? (s[i][c].f.x + s[i][c].f.y) * p.qscale : -INFINITY;
                    mx = fmaxf(mx, x[c]);
                }
#pragma unroll
                for (int off = C::TX / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                mx = fmaxf(mx, m[i]);
                const float mu = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: weights 2^-inf = 0
                Two corr;
                corr.f.x = corr.f.y = fast_exp2(m[i] - mu);
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < C::NC; ++c) {
                    const float w = fast_exp2(x[c] - mu);
                    sum += w;
                    ps[(ty * 4 + i) * C::PS + tx + C::TX * c] = w;
                }
#pragma unroll
                for (int off = C::TX / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
                l[i] = l[i] * corr.f.x + sum;
                m[i] = mx;
#pragma unroll
                for (int v = 0; v < C::NV; ++v) {
                    mul_two(acc[i][v].lo, corr);
                    mul_two(acc[i][v].hi, corr);
                }
            }
            __syncwarp();  // a row's weights come from its own half-warp
            if (D >= 4 * C::TX || tx == 0) {
                // A weight of an unseen position is 0, but 0 times an infinite or NaN value is NaN: from the
                // first key that not all of a thread's rows see such products are left out, and no row sees a
                // key behind the last.
                auto sum_tile = [&](int t, auto guard) {
                    float4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (ty * 4 + i) * C::PS + t);
#pragma unroll
                    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                        for (int v = 0; v < C::NV; ++v) {
                            const Four x = load4(vs + (t + tt) * D + (v * C::TX + tx) * 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (decltype(guard)::value && t0 + t + tt >= lim[i]) continue;
                                Two f;
                                f.f.x = f.f.y = tt == 0 ? w[i].x : tt == 1 ? w[i].y : tt == 2 ? w[i].z : w[i].w;
                                fma_two(acc[i][v].lo, f, x.lo);
                                fma_two(acc[i][v].hi, f, x.hi);
                            }
                        }
                };
                const int all = min(C::KT, (int)(lim[0] - t0)), some = min(C::KT, (int)(lim[3] - t0));
                int t = 0;
#pragma unroll 1
                for (; t + 4 <= all; t += 4) sum_tile(t, std::false_type{});
#pragma unroll 1
                for (; t < some; t += 4) sum_tile(t, std::true_type{});
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= nrow || (D < 4 * C::TX && tx > 0)) continue;
            const int64_t row = g.row0 + (r >> p.lgG);
            const int head = g.h * G + (r & (G - 1));
            if (g.dst == -1) {
                const float inv = 1.f / l[i];
                T* out = static_cast<T*>(p.out) + row * p.out_ts + (int64_t)head * D;
#pragma unroll
                for (int v = 0; v < C::NV; ++v) {
                    const int d = (v * C::TX + tx) * 4;
                    if constexpr (sizeof(T) == 2) {
                        *reinterpret_cast<uint2*>(out + d) =
                            make_uint2(bf16x2_rn(acc[i][v].lo.f.x * inv, acc[i][v].lo.f.y * inv),
                                       bf16x2_rn(acc[i][v].hi.f.x * inv, acc[i][v].hi.f.y * inv));
                    } else {
                        *reinterpret_cast<float4*>(out + d) = make_float4(acc[i][v].lo.f.x * inv, acc[i][v].lo.f.y * inv,
                                                                          acc[i][v].hi.f.x * inv, acc[i][v].hi.f.y * inv);
                    }
                }
            } else {
                float *o, *ml;
                ragged_dst(p, g.dst, R::SLOT_ROWS, r, row, head, o, ml);
#pragma unroll
                for (int v = 0; v < C::NV; ++v)
                    *reinterpret_cast<float4*>(o + (v * C::TX + tx) * 4) = make_float4(acc[i][v].lo.f.x, acc[i][v].lo.f.y,
                                                                                  acc[i][v].hi.f.x, acc[i][v].hi.f.y);
                if (tx == 0) *reinterpret_cast<float2*>(ml) = make_float2(m[i], l[i]);
            }
        }
    }
}

template <typename T, int D, bool JOINT>
static int launch_cc_as(const RaggedParams& p, cudaStream_t s) {
    using C = CcCfg<T, D, JOINT>;
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
    cfg.blockDim = dim3(C::THREADS);
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
