// kvc_ragged_q8.cu -- attention of ragged new tokens over a paged cache held in 8 bits (kvc_q8.cuh), on the
// 5th-generation tensor cores and on the codes as they are (D = 64 or 128, bf16 queries).
//
// With k_t = 2^{a_t} c_t and v_t = 2^{b_t} d_t (codes c, d; a, b per block) a row's output is
//     sum_t 2^{x_t} 2^{b_t} d_t / sum_t 2^{x_t},   x_t = log2(e) / sqrt(D) 2^{a_t} (q . c_t),
// so both products take E4M3 operands: keys and values go from memory to the tensor cores untouched, and
// everything else enters through the small operand:
//   - S^T = K Q^T (A = a tile of codes, K-major, B = the rows): a query row is scaled by a power of two to
//     [128, 256) and split into two codes, q = 2^e (t0 + t1 / 16).  Two 4-bit significands hold bf16's 8 bits:
//     exact but for elements below 2^-13 of the row's largest (off by 2^-21 of that).  Each term has columns of its own.
//   - O^T += V^T W (A = the same tile of V read MN-major, B = the weights): w_t = 2^{x_t - m} 2^{b_t} 2^{m - M + 4} as
//     three E5M2 terms with columns of their own, w = u0 + u1 / 8 + u2 / 64: the top byte of w in f16, that of 8 times what
//     is left, and of 8 times what is then left, rounded: within 2^-9 + 2^-11 of w (the last term's rounding and f16's; 1.09 2^-9
//     at worst), or 2^-23 + 2^-25 absolute with the row's largest above 2^3.  (A byte mask, a subtraction and a product each; E4M3 terms took conversions, and a weight had 2 binades
//     to grow until its reference had to be raised, here 10.)  m >= max x_t and M >= max(x_t + b_t) are integers: all
//     factors between references are exact.  The denominator sums 2^{x_t - m} in fp32.
// A thread is a key position (lane of S^T), its columns the rows.  The references are raised only if a weight
// passes 2^14: per tile one vote over the four warps instead of a maximum over the positions.
// S has two places: the scores of the next tile are computed while this one's are weighed.
//
// D = 64: a 128-byte row of the tile holds two tokens, tile rows are token pairs.  The operand has columns for
// either token of the pair (the other half of a query row's 128 bytes is 0), and of O^T, whose 128 rows are
// (token of the pair, d), each lane uses its own token's columns; the two halves are added at the end.
//
// What bounds it: for few rows the memory's bytes, half of a bf16 cache's (24 sequences of 3000 to 6000 positions on 8 KV
// heads of 128 take 45 to 48 us, 4.7 to 5.0 TB/s; of 12,000 to 24,000 144 us, 6.3 TB/s: 6 us of start, 4 to 8 of merge and end),
// for more the softmax warps: 2.2 us a tile of 32 rows by 128 positions (256 of D = 64), two CTAs an SM at work, of
// which the products take a tenth; conversions, three terms a weight and the exponentials are its chain (64 sequences of
// 32 to 160 rows on one KV head of 64: 110 us against 7 of memory).  Two groups of softmax warps a CTA took as long.
// So entries of many rows go to the kernel of plain pools (kvc_ragged_host.cu).
//
// The streams, their split over the CTAs and the merge are those of kvc_ragged.cuh (tiles of RT rows, all of
// class 1, one worker a CTA).  Warps: 0 copies, 1 issues the products, 2 computes the split and walks the
// streams, 3 writes the rows of invalid sequences, 4-7 softmax and output.
#include <type_traits>

#include "kvc_decode_tc5.cuh"
#include "kvc_q8.cuh"
#include "kvc_ragged_merge.cuh"

namespace kvc {

// TOK tokens per 128-byte row (D = 128 / TOK), RT = 2^LRT query rows.  Up to 2 64 + 96 columns of tensor memory
// fit two CTAs an SM; D = 64 with 32 rows takes one.
template <int TOK_, int LRT, bool JOINT>
struct Q8Cfg {
    static constexpr int TOK = TOK_, D = 128 / TOK, RT = 1 << LRT, LKT = TOK == 2 ? 8 : 7, KT = 1 << LKT;
    using R = Ragged<LRT, LKT, false, JOINT, 8>;
    using Seg = typename R::Seg;
    static constexpr int CTAS = TOK * RT > 32 ? 1 : 2;  // an SM
    static constexpr int TILE = 128 * 128;
    static constexpr int QROWS = 2 * TOK * RT;  // columns of S
    static constexpr int PCOLS = 3 * TOK * RT;  // columns of O
    static constexpr int QBYTES = QROWS * 128, PBYTES = PCOLS * 128;
    static constexpr int MISC = 6 << 10;
    static constexpr int BUDGET = CTAS == 2 ? 115712 : 232448;
    static constexpr int NSLOT_A = (BUDGET - QBYTES - PBYTES - MISC) / TILE;
    static constexpr int NSLOT = NSLOT_A > 12 ? 12 : NSLOT_A;
    static constexpr int SMEM = NSLOT * TILE + QBYTES + PBYTES + MISC;
    static constexpr int TMEM_COLS = CTAS == 2 ? 256 : 512;
    static constexpr int OCOL = 2 * QROWS;  // two places of S, then O
    static constexpr int NSEG = 4;      // segments known ahead (a power of two; see the copies)
    static constexpr int NSC = 8;       // tiles whose scales are held
    static constexpr int THREADS = 256;
    static_assert(2 * QROWS + PCOLS <= TMEM_COLS, "tensor memory");
    static_assert(NSLOT >= 4 && NSLOT / 2 + 2 <= NSC, "ring");
    static_assert(NSLOT * TILE >= R::work_ints(MAX_B, MAX_B) * 4, "the split's arrays lie under the ring");
    static_assert(PBYTES >= RT * 64 * 4 || TOK == 1, "the halves' exchange lies in the weights' place");
    struct Misc {
        uint64_t full[12], empty[12];
        uint64_t sfull[2], kfix[2], pfull, odone, qfull, drain;
        uint64_t segfull[NSEG], segempty[NSEG];
        Seg seg[NSEG];
        float2 scale[NSC][16];  // (K, V) scales of a tile's boxes
        // per row: the queries' scales (of two segments in turn), references m and M, what the weights
        // use of them, factors of a raise
        alignas(16) float qs[2][32];  // (read four at a time)
        alignas(16) float mu[32];
        alignas(16) float b[32];
        float m[32], M[32], fo[32], fl[32];
        char* dst[32];  // where a row's output or piece goes
        float2 red[4][32];
        uint32_t knan[2][4];  // (TOK = 2, of two tiles in turn) second tokens whose key has NaN codes
        uint32_t over[2];  // (of two tiles in turn) groups of eight rows whose references have to be raised
        int nonfinite;  // NaN codes were taken out of V in this segment
        int abort;
        uint32_t tmem;
        int valid;
    };
    static_assert(sizeof(Misc) <= MISC, "misc area");
};

struct Q8Attn {
    RaggedParams r;
    const float *Ksc, *Vsc;
    int once;  // every tile is read by one CTA: it leaves L2 first
};

// Polls a barrier until the phase has completed, for at most WAIT_LIMIT_NS (false: gave up, see mbar_wait); ns: sleep
// between polls.
__device__ __noinline__ bool q8_poll(uint64_t* bar, uint32_t parity, uint32_t ns, volatile int* abort_flag, uint32_t* err) {
    const uint64_t t0 = global_ns();
    while (true) {
        if (ns) __nanosleep(ns);
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_ns() - t0 > WAIT_LIMIT_NS) {
            *abort_flag = 1;
            atomicOr(err, DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

// ---- operands
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46;
}
__device__ __forceinline__ void q8_mma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ bool q8_elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Eight columns at each of two or three places of this thread's lane, loaded when it returns.
__device__ __forceinline__ void tm_ld8x2(uint32_t t0, uint32_t t1, float (&a)[8], float (&b)[8]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t0), "r"(t1)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = __uint_as_float(r[i]);
        b[i] = __uint_as_float(r[8 + i]);
    }
}
__device__ __forceinline__ void tm_ld8x3(uint32_t t0, uint32_t t1, uint32_t t2, float (&a)[8], float (&b)[8], float (&c)[8]) {
    uint32_t r[24];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%24];"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%25];"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%26];"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
        : "r"(t0), "r"(t1), "r"(t2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = __uint_as_float(r[i]);
        b[i] = __uint_as_float(r[8 + i]);
        c[i] = __uint_as_float(r[16 + i]);
    }
}
__device__ __forceinline__ void tm_st8(uint32_t t, const float (&a)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
                 "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                 "r"(__float_as_uint(a[3])), "r"(__float_as_uint(a[4])), "r"(__float_as_uint(a[5])),
                 "r"(__float_as_uint(a[6])), "r"(__float_as_uint(a[7]))
                 : "memory");
}
// A barrier of n threads that ors a predicate.
__device__ __forceinline__ bool any_of(int id, int n, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_from(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
// Largest of a value over a warp, as an ordered integer.
__device__ __forceinline__ float warp_max(float x) {
    const int i = __float_as_int(x), o = i >= 0 ? i : i ^ 0x7FFFFFFF;
    const int r = __reduce_max_sync(0xFFFFFFFFu, o);
    return __int_as_float(r >= 0 ? r : r ^ 0x7FFFFFFF);
}
// The smaller of two, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Eight values summed over the warp: each halving exchanges what the other half keeps, so lane i ends with sum i / 4.
__device__ __forceinline__ float rows_of_warp(const float (&sum)[8], int lane) {
    float h4[4], h2[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        const float keep = up ? sum[4 + i] : sum[i], give = up ? sum[i] : sum[4 + i];
        h4[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        const float keep = up ? h4[2 + i] : h4[i], give = up ? h4[i] : h4[2 + i];
        h2[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 8);
    }
    const bool up = lane & 4;
    float v = (up ? h2[1] : h2[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? h2[0] : h2[1], 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 1);
}
// 0xFF in the bytes that are NaN codes (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t u) {
    return ((((u & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
}
// NaN in column `dim` of the rows r0 .. that see a NaN code there which was taken out of V: of positions that not all
// rows see, up to `end`, the last that the segment's tiles hold.
template <class Seg>
__device__ __noinline__ void add_nan(const RaggedParams& p, const Seg& g, int end, int r0, int dim, int D, float (&o)[8]) {
    for (int t = max(g.lim0, g.kv0); t < end; ++t) {
        const int64_t vr = cache_row_rd(p.table, p.bs, p.max_blocks, p.num_blocks, p.H_kv, p.T_max, g.seq, g.h, t, p.err);
        if ((__ldg(static_cast<const uint8_t*>(p.V) + vr * D + dim) & 0x7F) != 0x7F) continue;
        for (int i = 0; i < 8; ++i)
            if (t < g.sees((r0 + i) >> p.lgG)) o[i] = __uint_as_float(0x7FFFFFFFu);
    }
}
// 2^d for an integer-valued d, clamped to the normal floats.
__device__ __forceinline__ float pow2_of(float d) { return exp2i((int)fminf(fmaxf(d, -126.f), 127.f)); }

template <int TOK, int LRT, bool JOINT>
__global__ void __launch_bounds__(256, (Q8Cfg<TOK, LRT, JOINT>::CTAS))
ragged_q8_kernel(const Q8Attn pa, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = Q8Cfg<TOK, LRT, JOINT>;
    using R = typename C::R;
    using Seg = typename C::Seg;
    using Misc = typename C::Misc;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    constexpr int D = C::D;
    const RaggedParams& p = pa.r;
    extern __shared__ __align__(1024) char q8_smem[];
    static_assert(alignof(Misc) == 16 && (C::QBYTES | C::PBYTES) % 1024 == 0);
    char* ring = q8_smem;
    char* qop = ring + C::NSLOT * C::TILE;
    char* wop = qop + C::QBYTES;
    Misc& M = *reinterpret_cast<Misc*>(wop + C::PBYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = 1 << p.lgG;
    volatile int* ab = &M.abort;
    auto wait_on = [&](uint64_t* bar, uint32_t parity, uint32_t ns = 0) {
        return mbar_try_wait(bar, parity) || q8_poll(bar, parity, ns, ab, p.err);
    };
    if (smem_addr(q8_smem) & 1023) {  // (the swizzled tiles need it; the declaration asks for it)
        if (tid == 0) atomicOr(p.err, DEV_WAIT_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&M.full[i], 1);
            mbar_init(&M.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M.sfull[i], 1);
            mbar_init(&M.kfix[i], 1);
        }
        mbar_init(&M.pfull, 4);
        mbar_init(&M.odone, 1);
        mbar_init(&M.qfull, 4);
        mbar_init(&M.drain, 1);
        for (int i = 0; i < C::NSEG; ++i) {
            mbar_init(&M.segfull[i], 1);
            mbar_init(&M.segempty[i], 6);  // copies, products, four softmax warps
        }
        M.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&M.tmem)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc5_fence_before();
    }
    if (warp == 0 && lane < 2) {
        const CUtensorMap* m = lane == 0 ? &tmK : &tmV;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    typename R::Split sp;
    typename R::Walk wk;
    if (warp == 2) {
        const typename R::Work work = R::work(p, ring);
        sp = R::scan(p, work, lane);
        if (lane == 0) M.valid = sp.valid;
        if (blockIdx.x == 0) {
            const int n = 2 * (R::groups(p) + p.B + 1);
            for (int i = lane; i < n; i += 32) p.plan[i] = sp.valid ? work.c[i] : 0;
            if (!sp.valid && lane == 0) atomicOr(p.err, sp.why);
        }
        // The block's cuts start out empty (the warp that leaves them empties them).
        if (lane < 6) p.cuts[6 * blockIdx.x + lane] = make_int4(0, 0, 0, 0);
        __syncwarp();
        if (lane < 2) wk = R::walk(p, sp, work, blockIdx.x, lane);  // class 0, then class 1
        fence_async_smem();  // (the split's arrays are overwritten by copies)
    }
    __syncthreads();
    tc5_fence_after();
    const uint32_t tmem = M.tmem;
    uint32_t issued = 0;  // copies / products begun (copy and product warps)

    if (warp == 2) {
        // ====================================================== streams
        // Lane 0 leaves the segments of class 0, then lane 1 those of class 1 and the end.
        int s = 0;
        bool ok = true;
        for (int cl = 0; cl < 2; ++cl) {
            if (lane == cl) {
                while (ok) {
                    const Seg g = R::next_seg(p, wk);
                    if (g.n == 0 && cl == 0) break;
                    if (s >= C::NSEG) ok = wait_on(&M.segempty[s % C::NSEG], (s / C::NSEG - 1) & 1, 500);
                    if (!ok) break;
                    M.seg[s % C::NSEG] = g;
                    mbar_arrive(&M.segfull[s % C::NSEG]);
                    if (wk.cut) R::leave_cut(p, sp, wk, blockIdx.x, 1, g);
                    if (g.n == 0) break;
                    ++s;
                }
            }
            s = __shfl_sync(ALL, s, 0);
            ok = __shfl_sync(ALL, ok, 0);
        }
    } else if (warp == 3) {
        if (M.valid) ragged_zero_rows<__nv_bfloat16, JOINT>(p, lane, 32);
    } else if (warp == 0) {
        // ====================================================== copies
        // Lane i copies box i of a tile: min(bs, KT) tokens.  Three places in the streams: block numbers are
        // looked up two tiles ahead, scales one ahead.  (Four segments are known ahead: the first place is at
        // most two segments past the third, whose predecessors end without this warp.)
        const uint64_t pol = pa.once ? policy_evict_first() : 0;
        uint64_t pol_n;
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol_n));
        const uint64_t policy = pa.once ? pol : pol_n;
        const int lgb = min(p.lgbs, C::LKT);  // log2 of a box's tokens
        const int bt = lane << lgb;           // this lane's box begins at this token of a tile
        const int box_bytes = (1 << lgb) * D;
        const uint32_t ring_s = smem_addr(ring);
        struct At {
            Seg g;
            int s, j;
        };
        auto next_of = [&](At& a) {  // the next tile (g.n = 0: none)
            if (a.j + 1 < a.g.n) {
                ++a.j;
                return true;
            }
            ++a.s;
            a.j = 0;
            const int i = a.s % C::NSEG;
            const bool ok = __all_sync(ALL, wait_on(&M.segfull[i], (a.s / C::NSEG) & 1)) != 0;
            if (!ok) return false;
            a.g = M.seg[i];
            __syncwarp();
            if (lane == 0) mbar_arrive(&M.segempty[i]);
            return true;
        };
        auto there = [&](const At& a) {
            return a.g.n > 0 && bt < C::KT && (unsigned)a.g.kv0 + a.j * C::KT + bt < (unsigned)a.g.kv_end;
        };
        auto look_up = [&](const At& a) {
            if (!there(a)) return 0;
            return __ldg(p.table + (size_t)a.g.seq * p.max_blocks + (((unsigned)a.g.kv0 + a.j * C::KT + bt) >> p.lgbs));
        };
        auto scales_of = [&](const At& a, int e) {
            if (!there(a)) return make_float2(1.f, 1.f);  // (-inf times it stays that)
            const int64_t at = (int64_t)((unsigned)e < (unsigned)p.num_blocks ? e : 0) * p.H_kv + a.g.h;
            return make_float2(__ldg(pa.Ksc + at), __ldg(pa.Vsc + at));
        };
        At a, b, c;  // block numbers, scales, copies
        a.g.n = 0;
        a.s = -1;
        a.j = 0;
        bool ok = next_of(a);
        int ea = 0, eb = 0, ec = 0;
        float2 sb, sc;
        if (ok) {
            b = a;
            ea = look_up(a);
            eb = ea;
            if (a.g.n > 0) {
                ok = next_of(a);
                if (ok) ea = look_up(a);
            }
            sb = scales_of(b, eb);
        }
        uint32_t slot = 0, use = 0, tile = 0;
        while (ok && b.g.n > 0) {
            c = b;
            ec = eb;
            sc = sb;
            b = a;
            eb = ea;
            if (a.g.n > 0) {
                ok = next_of(a);
                if (!ok) break;
                ea = look_up(a);
            }
            sb = scales_of(b, eb);
            const int t0 = c.g.kv0 + c.j * C::KT;
            const int rows = min(c.g.kv_end - t0, C::KT), nbox = (rows + (1 << lgb) - 1) >> lgb;
            if (lane < nbox && (unsigned)ec >= (unsigned)p.num_blocks) {
                atomicOr(p.err, DEV_BAD_BLOCK);
                ec = 0;
            }
            const int row = (int)(((((int64_t)ec * p.H_kv + c.g.h) << p.lgbs) + ((t0 + bt) & (p.bs - 1))) / TOK);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if (issued >= C::NSLOT) ok = __all_sync(ALL, lane != 0 || wait_on(&M.empty[slot], use & 1 ^ 1)) != 0;
                if (!ok) break;
                __syncwarp();
                // (the bytes may land before they are announced: the phase ends with lane 0's arrival, and V's comes
                // behind the scales, which were looked up a tile ago)
                if (lane < nbox)
                    tma_load_2d(ring_s + slot * C::TILE + lane * box_bytes, kv ? &tmV : &tmK, 0, row, &M.full[slot], policy);
                if (kv == 1 && lane < 16) {
                    // Blocks never written have scales of 0, whose logarithm the weights cannot take, and codes of 0.
                    // (Looked at here: next to their loads it took 24 single tokens from 46.5 to 51 us.)
                    const float least = exp2i(Q8_EMIN);
                    M.scale[tile % C::NSC][lane] = make_float2(sc.x < least ? least : sc.x, sc.y < least ? least : sc.y);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&M.full[slot], (uint32_t)(nbox * box_bytes));
                ++issued;
                if (++slot == C::NSLOT) {
                    slot = 0;
                    ++use;
                }
            }
            if (!ok) break;
            ++tile;
        }
    } else if (warp == 1) {
        // ====================================================== products (the whole warp, one elected thread issues)
        const uint64_t dK = smem_desc_sw128(smem_addr(ring), 16u, 1024u);
        const uint64_t dV = smem_desc_sw128(smem_addr(ring), 1024u, 1024u);
        const uint64_t dQ = smem_desc_sw128(smem_addr(qop), 16u, 1024u);
        const uint64_t dW = smem_desc_plain(smem_addr(wop), 128u, 2048u);
        const uint32_t tm = __shfl_sync(ALL, tmem, 0);
        uint32_t item = 0, tile = 0, fixes = 0;
        auto uni = [&](uint32_t x) { return __shfl_sync(ALL, x, 0); };
        bool ok = true;
        for (int s = 0; ok; ++s) {
            const int si = s % C::NSEG;
            ok = __all_sync(ALL, wait_on(&M.segfull[si], (s / C::NSEG) & 1)) != 0;
            if (!ok) break;
            const int n = uni(M.seg[si].n), nrow = uni(M.seg[si].ntok) << p.lgG;
            const int kv0 = M.seg[si].kv0, lim0 = M.seg[si].lim0, kv_end = M.seg[si].kv_end;
            __syncwarp();
            if (lane == 0) mbar_arrive(&M.segempty[si]);
            if (n == 0) break;
            const int Rp = nrow <= 8 ? 8 : nrow <= 16 ? 16 : 32;
            const int NS = 2 * TOK * Rp, NO = (3 * TOK * Rp + 15) & ~15;
            const uint32_t idS = uni((1u << 4) | ((uint32_t)(NS >> 3) << 17) | (8u << 24));
            const uint32_t idO = uni((1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(NO >> 3) << 17) | (8u << 24));
            ok = __all_sync(ALL, wait_on(&M.qfull, s & 1)) != 0;
            for (int j = 0; ok && j <= n; ++j) {
                if (j < n) {
                    // S^T = K Q^T of tile j, into the place of the tile before the last, whose weights are in
                    const uint32_t ks = item % C::NSLOT;
                    ok = __all_sync(ALL, wait_on(&M.full[ks], (item / C::NSLOT) & 1)) != 0;
                    if (!ok) break;
                    if constexpr (TOK == 2) {
                        // A pair's scores share a product, in which a 0 meets the other token's codes: a second token that
                        // some row does not see, while it sees the first, must not hold NaN.  The rows that see it are told.
                        const int t0 = kv0 + j * C::KT;
                        if (lim0 - t0 < C::KT) {
                            if (lane < 4) M.knan[tile & 1][lane] = 0;
                            __syncwarp();
                            const int first = max(lim0 - t0, 0) | 1, last = min(kv_end - t0, C::KT - 1);
                            for (int i = lane; first + 2 * (i >> 2) <= last; i += 32) {
                                const int tr = (first >> 1) + (i >> 2);  // tile row; chunk 4 + i % 4 of it
                                uint4* a = reinterpret_cast<uint4*>(ring + ks * C::TILE + tr * 128 + (((4 + (i & 3)) ^ (tr & 7)) << 4));
                                const uint4 v = *a, z = make_uint4(nan_bytes(v.x), nan_bytes(v.y), nan_bytes(v.z), nan_bytes(v.w));
                                if ((z.x | z.y | z.z | z.w) == 0) continue;
                                *a = make_uint4(v.x & ~z.x, v.y & ~z.y, v.z & ~z.z, v.w & ~z.w);
                                atomicOr(&M.knan[tile & 1][tr >> 5], 1u << (tr & 31));
                            }
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&M.kfix[fixes & 1]);
                            ++fixes;
                        }
                    }
                    tc5_fence_after();
                    issued = 1;
                    const uint32_t ka = uni((uint32_t)dK + ks * (C::TILE >> 4)), at = uni(tm + (tile & 1) * C::QROWS);
                    if (q8_elect()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            q8_mma(at, ka + k * 2, (uint32_t)(dK >> 32), (uint32_t)dQ + k * 2, (uint32_t)(dQ >> 32), idS, k > 0);
                        tc5_commit(&M.sfull[tile & 1]);
                        tc5_commit(&M.empty[ks]);
                    }
                    __syncwarp();
                    item += 2;
                    ++tile;
                }
                if (j > 0) {
                    // O^T (+)= V^T W of tile j - 1
                    const uint32_t back = j < n ? 2 : 1, vi = item + 1 - 2 * back, vs = vi % C::NSLOT;
                    ok = __all_sync(ALL, wait_on(&M.pfull, (tile - back) & 1) && wait_on(&M.full[vs], (vi / C::NSLOT) & 1));
                    if (!ok) break;
                    tc5_fence_after();
                    const uint32_t va = uni((uint32_t)dV + vs * (C::TILE >> 4)), acc = uni(j > 1 ? 1u : 0u);
                    if (q8_elect()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            q8_mma(tm + C::OCOL, va + k * 256, (uint32_t)(dV >> 32), (uint32_t)dW + k * 32, (uint32_t)(dW >> 32),
                                   idO, k > 0 ? 1u : acc);
                        tc5_commit(&M.odone);
                        tc5_commit(&M.empty[vs]);
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ====================================================== softmax and output
        const int sw = warp - 4, r = tid - 128;  // tile row of this thread, and its lane of O^T
        const uint32_t lanes = (uint32_t)(sw * 32) << 16;
        const uint32_t tS0 = tmem + lanes, tO = tmem + C::OCOL + lanes;
        const int own_par = TOK == 2 ? r >> 6 : 0, dim = r & (D - 1);
        const int my_row = 8 * (lane & 3) + (lane >> 2);  // the row whose denominator this lane sums
        auto sync4 = [&] { named_bar_sync(1, 128); };
        // The segment's rows as the operand of S (all four warps).
        constexpr int VPR = D / 8;  // 16-byte vectors of a row
        auto load_q = [&](const Seg& g, int i) {
            const int rr = i / VPR, v = i & (VPR - 1);
            if (rr >= (g.ntok << p.lgG)) return make_uint4(0, 0, 0, 0);
            return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                        (int64_t)(g.row0 + (rr >> p.lgG)) * p.q_ts +
                                                        (int64_t)(g.h * G + (rr & (G - 1))) * D) +
                         v);
        };
        constexpr int QV = (C::RT * VPR + 127) / 128;  // a thread's vectors
        auto write_q = [&](const Seg& g, int s, uint4 x0) {  // x0: this thread's first vector
            const int nrow = g.ntok << p.lgG, Rp = nrow <= 8 ? 8 : nrow <= 16 ? 16 : 32;
            uint4 xs[QV];
            xs[0] = x0;
#pragma unroll
            for (int k = 1; k < QV; ++k)
                if (r + 128 * k < Rp * VPR) xs[k] = load_q(g, r + 128 * k);
#pragma unroll
            for (int k = 0; k < QV; ++k) {
                const int i = r + 128 * k;
                if (i >= Rp * VPR) continue;
                const int rr = i / VPR, v = i & (VPR - 1);
                const uint4 x = xs[k];
                float f[8];
                Elem<__nv_bfloat16>::unpack(x, f);
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t u = __float_as_uint(f[k]) & 0x7FFFFFFFu;
                    if (u < 0x7F800000u) top = max(top, u);
                }
#pragma unroll
                for (int off = VPR / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(ALL, top, off));
                // the row's largest goes to [128, 256); a NaN takes an infinity's place (the row is NaN either way)
                int e = (int)(top >> 23) - 127 - 7;
                e = top == 0 ? 0 : e < -119 ? -119 : e;
                if (v == 0) M.qs[s & 1][rr] = rr < nrow ? p.qscale * exp2i(e) : 1.f;
                uint32_t c0[4], c1[4];
                const float down = exp2i(-e);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float y0 = isfinite(f[2 * k]) ? f[2 * k] * down : __uint_as_float(0x7FFFFFFFu);
                    const float y1 = isfinite(f[2 * k + 1]) ? f[2 * k + 1] * down : __uint_as_float(0x7FFFFFFFu);
                    c0[k] = e4m3x2(y0, y1);
                    const float2 t = e4m3x2_value(c0[k]);
                    c1[k] = e4m3x2((y0 - t.x) * 16.f, (y1 - t.y) * 16.f);
                }
#pragma unroll
                for (int par = 0; par < TOK; ++par)
#pragma unroll
                    for (int term = 0; term < 2; ++term) {
                        const int n = (par * 2 + term) * Rp + rr;
                        const uint32_t(&c)[4] = term ? c1 : c0;
#pragma unroll
                        for (int half = 0; half < TOK; ++half) {  // (the other token's half of the row is 0)
                            const int byte = half * D + v * 8, ch = byte >> 4;
                            const bool mine = half == par;
                            *reinterpret_cast<uint2*>(qop + n * 128 + ((ch ^ (n & 7)) << 4) + (byte & 8)) =
                                make_uint2(mine ? c[0] | c[1] << 16 : 0u, mine ? c[2] | c[3] << 16 : 0u);
                        }
                    }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&M.qfull);
        };
        auto fetch = [&](int s, Seg& g) {
            const bool ok = __all_sync(ALL, wait_on(&M.segfull[s % C::NSEG], (s / C::NSEG) & 1)) != 0;
            if (ok) g = M.seg[s % C::NSEG];
            return ok;
        };
        // (A wait that gave up: every later wait of the CTA gives up too, and the four warps keep their barriers.)
        uint32_t tile = 0, item = 0, fixes = 0;
        Seg g;
        g.n = 0;
        bool live = !any_of(1, 128, !fetch(0, g));
        if (live && g.n > 0) write_q(g, 0, load_q(g, r));
        for (int s = 0; live && g.n > 0; ++s) {
            const int nrow = g.ntok << p.lgG, Rp = nrow <= 8 ? 8 : nrow <= 16 ? 16 : 32;
            const float* qs = M.qs[s & 1];
            // Denominators: this thread's part of each row, and of row my_row what raises have added up over the warp.
            constexpr int NG8 = C::RT / 8;  // groups of eight rows
            float l = 0.f;
            float2 ls[NG8][4];
#pragma unroll
            for (int c = 0; c < NG8; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) ls[c][i] = make_float2(0.f, 0.f);
            if (r == 0) M.nonfinite = M.over[0] = M.over[1] = 0;
            sync4();
            bool ok = true, known = false;
            Seg g2;  // the next segment, fetched with this one's last tile, and a vector of its rows
            g2.n = 0;
            uint4 x2 = make_uint4(0, 0, 0, 0);
            for (int j = 0; j < g.n; ++j, ++tile, item += 2) {
                const int t0 = g.kv0 + j * C::KT;
                if (j + 1 == g.n) {
                    known = fetch(s + 1, g2);
                    if (known && g2.n > 0) x2 = load_q(g2, r);
                }
                ok = wait_on(&M.sfull[tile & 1], (tile >> 1) & 1) && ok;
                const uint32_t tS = tS0 + (tile & 1) * C::QROWS;
                // The scales lie there with the tile's copies.  (V's barrier, whose place is held until this tile's
                // product; K's may be two uses on by now, which its parity does not tell.)
                const bool whole = g.lim0 - t0 >= C::KT;
                const uint32_t vslot = (item + 1) % C::NSLOT;
                ok = wait_on(&M.full[vslot], ((item + 1) / C::NSLOT) & 1) && ok;
                bool knan = false;  // (TOK = 2) this row's second token has a NaN key
                if (TOK == 2 && !whole) {
                    ok = wait_on(&M.kfix[fixes & 1], (fixes >> 1) & 1) && ok;
                    ++fixes;
                    knan = (M.knan[tile & 1][r >> 5] >> (r & 31) & 1) != 0;
                }
                __syncwarp();
                tc5_fence_after();
                const float2 sc = M.scale[tile % C::NSC][(TOK * r) >> min(p.lgbs, C::LKT)];
                if (!whole) {
                    // Scores of positions that a row does not see become -inf in their place.
#pragma unroll 1
                    for (int i = 0; i < TOK * Rp / 8; ++i) {
                        const int par = TOK == 2 ? i & 1 : 0, c = i / TOK;
                        const uint32_t at = tS + par * 2 * Rp + 8 * c;
                        const unsigned t = (unsigned)t0 + TOK * r + par;
                        float s0[8], s1[8];
                        tm_ld8x2(at, at + Rp, s0, s1);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (TOK == 2 && par == 1 && knan) s0[k] = __uint_as_float(0x7FFFFFFFu);
                            const bool see = t < (unsigned)g.sees((8 * c + k) >> p.lgG);
                            s0[k] = see ? s0[k] : -INFINITY;
                            s1[k] = see ? s1[k] : 0.f;
                        }
                        tm_st8(at, s0);
                        tm_st8(at + Rp, s1);
                    }
                    tc5_wait_st();
                }
                // What a score's factor, (a row's scale) (a block's scale), is at least, added to it: the product of two tiny scales
                // is 0, and a masked score of -inf times 0 NaN.  (Nothing for factors from 2^-101 on; below, scores of up to 2^24
                // times it are 0 next to 1 with and without it.)
                constexpr float LEAST = 0x1p-126f;
                // Scores of eight rows at token par, in log2 units.
                auto scores = [&](int c, int par, float (&x)[8]) {
                    float s0[8], s1[8];
                    const uint32_t at = tS + par * 2 * Rp + 8 * c;
                    tm_ld8x2(at, at + Rp, s0, s1);
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 q4 = *reinterpret_cast<const float4*>(qs + 8 * c + i);
                        x[i] = fmaf(s1[i], 0.0625f, s0[i]) * fmaf(q4.x, sc.x, LEAST);
                        x[i + 1] = fmaf(s1[i + 1], 0.0625f, s0[i + 1]) * fmaf(q4.y, sc.x, LEAST);
                        x[i + 2] = fmaf(s1[i + 2], 0.0625f, s0[i + 2]) * fmaf(q4.z, sc.x, LEAST);
                        x[i + 3] = fmaf(s1[i + 3], 0.0625f, s0[i + 3]) * fmaf(q4.w, sc.x, LEAST);
                    }
                };
                // References of the rows 8 c .. of each bit c of `which` at or above everything in this tile, rounded up to
                // integers; O and l follow.
                auto raise = [&](uint32_t which) {
                    const float la = (float)((int)((__float_as_uint(sc.y) >> 23) & 0xFFu) - 127);
                    const bool alike = __all_sync(ALL, la == __shfl_sync(ALL, la, 0));  // (one block's positions, mostly)
#pragma unroll 1
                    for (int c = 0; c < Rp / 8; ++c) {
                        if (!(which >> c & 1)) continue;
                        float top[8], x[8];
                        scores(c, 0, top);
#pragma unroll
                        for (int par = 1; par < TOK; ++par) {
                            scores(c, par, x);
#pragma unroll
                            for (int i = 0; i < 8; ++i) top[i] = fmaxf(top[i], x[i]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float v = top[i] == top[i] ? top[i] : -INFINITY;
                            const float mx = warp_max(v), Mx = alike ? mx + la : warp_max(v + la);
                            if (lane == 0) M.red[sw][8 * c + i] = make_float2(mx, Mx);
                        }
                    }
                    sync4();
                    if (r < Rp && !(which >> (r >> 3) & 1)) M.fl[r] = 1.f;
                    if (r < Rp && (which >> (r >> 3) & 1)) {
                        float m = j == 0 ? -INFINITY : M.m[r], MM = j == 0 ? -INFINITY : M.M[r];
                        const float m0 = m, M0 = MM;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            m = fmaxf(m, ceilf(M.red[w][r].x));
                            MM = fmaxf(MM, ceilf(M.red[w][r].y));
                        }
                        M.m[r] = m;
                        M.M[r] = MM;
                        M.mu[r] = m == -INFINITY ? 0.f : -m;
                        M.b[r] = m == -INFINITY ? 1.f : pow2_of(m - MM + 4.f);
                        M.fl[r] = m0 == -INFINITY || m == m0 ? 1.f : m0 - m < -126.f ? 0.f : pow2_of(m0 - m);
                        M.fo[r] = M0 == -INFINITY || MM == M0 ? 1.f : M0 - MM < -126.f ? 0.f : pow2_of(M0 - MM);
                    }
                    sync4();
                    l *= my_row < Rp ? M.fl[my_row] : 1.f;
                    if (j > 0) {
                        // (the weights' first writes have waited for the products into O so far)
#pragma unroll 1
                        for (int k = 0; k < 3 * Rp / 8; ++k) {
                            const int row0 = (8 * k) % Rp;
                            if (!(which >> (row0 >> 3) & 1)) continue;
                            const uint32_t at = tO + own_par * 3 * Rp + 8 * k;
                            float o[8];
                            tc5_ld8(at, o);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= M.fo[row0 + i];
                            tm_st8(at, o);
                        }
                        tc5_wait_st();
                    }
                };
                // Eight rows' weights: their terms into the operand, each pair of rows'
                // 2^{x - m}, added to `sum`, and whether a weight is too large for its terms.  (Pairs of rows: two
                // products or sums are one instruction.  2^{x - m} is held below 2^60, where it stays finite until a
                // raise has taken it out again.)
                bool free_w = false;
                auto weigh = [&](int c, float2 (&sum)[4]) {
                    __half2 top = __float2half2_rn(0.f);
                    const __half2 eight = __float2half2_rn(8.f);
                    const float2 a2 = make_float2(sc.y, sc.y), k2 = make_float2(sc.x, sc.x), s16 = make_float2(0.0625f, 0.0625f),
                                 least = make_float2(LEAST, LEAST);
#pragma unroll
                    for (int par = 0; par < TOK; ++par) {
                        float s0[8], s1[8];
                        const uint32_t at = tS + par * 2 * Rp + 8 * c;
                        tm_ld8x2(at, at + Rp, s0, s1);
                        uint32_t u[3][4];
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float4 q4 = *reinterpret_cast<const float4*>(qs + 8 * c + 2 * i);
                            const float4 m4 = *reinterpret_cast<const float4*>(M.mu + 8 * c + 2 * i);
                            const float4 b4 = *reinterpret_cast<const float4*>(M.b + 8 * c + 2 * i);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int n = i + k;
                                const float2 f = __ffma2_rn(k ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y), k2, least);
                                float2 e = __ffma2_rn(make_float2(s1[2 * n], s1[2 * n + 1]), s16, make_float2(s0[2 * n], s0[2 * n + 1]));
                                e = __ffma2_rn(e, f, k ? make_float2(m4.z, m4.w) : make_float2(m4.x, m4.y));
                                e = make_float2(fast_exp2(min_nan(e.x, 60.f)), fast_exp2(min_nan(e.y, 60.f)));
                                sum[n] = __fadd2_rn(sum[n], e);
                                // (in this order: 2^{b_t} of a block with large values times b may pass the largest float, which 0, the
                                // weight of a position that a row does not see, must not meet)
                                const float2 w = __fmul2_rn(__fmul2_rn(e, k ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y)), a2);
                                __half2 h = __floats2half2_rn(w.x, w.y);
                                top = __hmax2(top, h);
                                u[0][n] = half2_bits(h);
                                h = __hmul2(__hsub2(h, half2_from(u[0][n] & 0xFF00FF00u)), eight);
                                u[1][n] = half2_bits(h);
                                h = __hmul2(__hsub2(h, half2_from(u[1][n] & 0xFF00FF00u)), eight);
                                u[2][n] = half2_bits(h) + 0x00800080u;
                            }
                        }
                        if (!free_w) {  // the product of the tile before has read its weights
                            ok = (tile == 0 || wait_on(&M.odone, (tile - 1) & 1)) && ok;
                            free_w = true;
                        }
#pragma unroll
                        for (int term = 0; term < 3; ++term) {
                            const int col = (par * 3 + term) * Rp + 8 * c;
                            *reinterpret_cast<uint2*>(wop + (col >> 4) * 2048 + r * 16 + (col & 8)) =
                                make_uint2(__byte_perm(u[term][0], u[term][1], 0x7531), __byte_perm(u[term][2], u[term][3], 0x7531));
                        }
                    }
                    // (a sum of 2^59 is one whose value may have been held, or soon: that row's m is raised too)
                    const float2 all = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                    return all.x + all.y > 0x1p59f || __hgt(__hmax(__low2half(top), __high2half(top)), __float2half_rn(0x1p14f));
                };
                if (!whole) {
                    // A weight of 0 times NaN is NaN: V of tokens behind the end (stale, or never loaded) is zeroed, and
                    // NaN codes of tokens that some row does not see, which those that do add at the end.
                    char* row = ring + vslot * C::TILE + r * 128;
#pragma unroll
                    for (int par = 0; par < TOK; ++par) {
                        const unsigned t = (unsigned)t0 + TOK * r + par;
                        const bool gone = t >= (unsigned)g.kv_end;
                        if (!gone && t < (unsigned)g.lim0) continue;
                        bool found = false;
#pragma unroll 1
                        for (int ch = par * (8 / TOK); ch < (par + 1) * (8 / TOK); ++ch) {
                            uint4* a = reinterpret_cast<uint4*>(row + ((ch ^ (r & 7)) << 4));
                            uint4 v = gone ? make_uint4(0, 0, 0, 0) : *a;
                            if (!gone) {
                                const uint4 n = make_uint4(nan_bytes(v.x), nan_bytes(v.y), nan_bytes(v.z), nan_bytes(v.w));
                                if ((n.x | n.y | n.z | n.w) == 0) continue;
                                found = true;
                                v = make_uint4(v.x & ~n.x, v.y & ~n.y, v.z & ~n.z, v.w & ~n.w);
                            }
                            *a = v;
                        }
                        if (found) M.nonfinite = 1;
                    }
                }
                if (j == 0) raise((1u << NG8) - 1);
                uint32_t over = 0;
                auto weigh_all = [&](auto groups) {
#pragma unroll
                    for (int c = 0; c < decltype(groups)::value; ++c)
                        if (weigh(c, ls[c])) over |= 1u << c;
                };
                if (Rp == 8) weigh_all(std::integral_constant<int, 1>{});
                else if (Rp == 16) weigh_all(std::integral_constant<int, 2>{});
                else if constexpr (C::RT == 32) weigh_all(std::integral_constant<int, 4>{});
                if (j > 0 && over) atomicOr(&M.over[j & 1], over);
                if (any_of(1, 128, j > 0 && over)) {
                    // The groups' sums go to l, this tile's are taken out of them (their size is at most that of the sums to come,
                    // and so is what rounding leaves of them), the references raised, the weights computed again.
                    const uint32_t which = *(volatile uint32_t*)&M.over[j & 1];
                    auto add_to_l = [&](int c, const float2 (&v)[4], float sign) {
                        const float flat[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
                        const float x = rows_of_warp(flat, lane);
                        if ((lane & 3) == c) l = fmaf(sign, x, l);
                    };
#pragma unroll
                    for (int c = 0; c < NG8; ++c)
                        if (which >> c & 1) {
                            add_to_l(c, ls[c], 1.f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) ls[c][i] = make_float2(0.f, 0.f);
                        }
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {
                        if (pass == 1) raise(which);
#pragma unroll 1
                        for (int c = 0; c < Rp / 8; ++c) {
                            if (!(which >> c & 1)) continue;
                            float2 sum[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
                            weigh(c, sum);
                            add_to_l(c, sum, pass == 0 ? -1.f : 1.f);
                        }
                    }
                }
                // (read by all before raise's barriers; the next tile's votes go to the other word)
                if (r == 0) M.over[j & 1] = 0;
                fence_async_smem();
                tc5_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&M.pfull);
            }
            // ---- the next segment's rows, while this one's last product runs
            live = !any_of(1, 128, !known);
            if (live && g2.n > 0) write_q(g2, s + 1, x2);
            // ---- the segment's state: written out, or left as a piece
#pragma unroll
            for (int c = 0; c < NG8; ++c)
                if (8 * c < Rp) {
                    const float flat[8] = {ls[c][0].x, ls[c][0].y, ls[c][1].x, ls[c][1].y,
                                           ls[c][2].x, ls[c][2].y, ls[c][3].x, ls[c][3].y};
                    const float x = rows_of_warp(flat, lane);
                    if ((lane & 3) == c) l += x;
                }
            M.red[sw][my_row].x = l;
            ok = wait_on(&M.odone, (tile - 1) & 1) && ok;
            __syncwarp();
            tc5_fence_after();
            ok = !any_of(1, 128, !ok);
            if (r < Rp) {
                const float sum = (M.red[0][r].x + M.red[1][r].x) + (M.red[2][r].x + M.red[3][r].x);
                M.fo[r] = 1.f / M.b[r] * (g.dst == -1 ? 1.f / sum : 1.f);
                const int64_t row = g.row0 + (r >> p.lgG);
                const int head = g.h * G + (r & (G - 1));
                if (g.dst == -1) {
                    M.dst[r] = static_cast<char*>(p.out) + (row * p.out_ts + (int64_t)head * D) * 2;
                } else {
                    float *po, *pml;
                    ragged_dst(p, g.dst, R::SLOT_ROWS, r, row, head, po, pml);
                    M.dst[r] = reinterpret_cast<char*>(po);
                    if (r < nrow && ok) *reinterpret_cast<float2*>(pml) = make_float2(M.m[r], sum);
                }
            }
            sync4();
            const bool nonfin = M.nonfinite != 0;
            float* half = reinterpret_cast<float*>(wop);  // (TOK = 2) [row][64] of the pairs' second tokens
            auto outputs = [&](int c, float (&o)[8]) {
                float o1[8], o2[8];
                const uint32_t at = tO + own_par * 3 * Rp + 8 * c;
                tm_ld8x3(at, at + Rp, at + 2 * Rp, o, o1, o2);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(fmaf(o2[i], 0.125f, o1[i]), 0.125f, o[i]) * M.fo[8 * c + i];
            };
            if constexpr (TOK == 2) {
                if (own_par == 1) {
#pragma unroll 1
                    for (int c = 0; c < Rp / 8; ++c) {
                        float o[8];
                        outputs(c, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) half[(8 * c + i) * 64 + dim] = o[i];
                    }
                }
                sync4();
            }
            if (own_par == 0 && ok) {
#pragma unroll 1
                for (int c = 0; c < (nrow + 7) / 8; ++c) {
                    float o[8];
                    outputs(c, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (TOK == 2) o[i] += half[(8 * c + i) * 64 + dim];
                    }
                    if (nonfin) add_nan(p, g, g.n > (g.kv_end - 1 - g.kv0) / C::KT ? g.kv_end : g.kv0 + g.n * C::KT, 8 * c, dim, D, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (8 * c + i >= nrow) continue;
                        char* to = M.dst[8 * c + i];
                        if (g.dst == -1) reinterpret_cast<__nv_bfloat16*>(to)[dim] = __float2bfloat16_rn(o[i]);
                        else reinterpret_cast<float*>(to)[dim] = o[i];
                    }
                }
            }
            tc5_fence_before();
            sync4();  // the state is read before the next segment's first raise
            if (lane == 0) mbar_arrive(&M.segempty[s % C::NSEG]);
            g = g2;
        }
    }
    __syncwarp();
    __syncthreads();  // every role is out of its loop (all waits are bounded)
    if (*ab) {
        // a wait timed out: let issued copies and products land, bounded
        if (tid == 0)
            for (uint32_t it = issued > C::NSLOT ? issued - C::NSLOT : 0; it < issued; ++it) {
                const uint64_t t = global_ns();
                while (!mbar_try_wait(&M.full[it % C::NSLOT], (it / C::NSLOT) & 1) && global_ns() - t < WAIT_LIMIT_NS) {
                }
            }
        if (warp == 1 && issued > 0) {
            if (q8_elect()) tc5_commit(&M.drain);
            const uint64_t t = global_ns();
            while (!mbar_try_wait(&M.drain, 0) && global_ns() - t < WAIT_LIMIT_NS) {
            }
        }
    }
    tc5_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc5_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
    }
}

template <int TOK, int LRT, bool JOINT>
static int launch_q8_as(const Q8Attn& pa, const RaggedParams* many, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    using C = Q8Cfg<TOK, LRT, JOINT>;
    static PerDeviceOnce once;
    const int e0 = once.run([] {
        return (int)cudaFuncSetAttribute(ragged_q8_kernel<TOK, LRT, JOINT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e0 != 0) return e0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)pa.r.P);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ragged_q8_kernel<TOK, LRT, JOINT>, pa, k, v);
    if (e != cudaSuccess) return (int)e;
    if constexpr (JOINT)
        if (many) return launch_merge_parts<__nv_bfloat16, RaggedTc5<true>, typename C::R>(*many, pa.r, s);
    return launch_merge<__nv_bfloat16, typename C::R, JOINT>(pa.r, s);
}

// Rows of a stream's tile and CTAs an SM of the instantiation for D and G.
void q8_shape(int D, int G, int* rows, int* ctas) {
    *rows = D == 64 && G <= 16 ? 16 : 32;
    *ctas = D == 64 && G > 16 ? 1 : 2;
}

int launch_ragged_q8(const RaggedParams& p, const RaggedParams* many, const float* Ksc, const float* Vsc,
                     const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    int rows, ctas;
    q8_shape(p.D, 1 << p.lgG, &rows, &ctas);
    Q8Attn pa{p, Ksc, Vsc, 0};
    // (a batch of at most one tile of rows per sequence and no shared prefixes)
    pa.once = p.NG == 0 && ((int64_t)p.N << p.lgG) <= (int64_t)p.B * rows;
    auto go = [&](auto tok, auto lrt) {
        constexpr int TOK = decltype(tok)::value, LRT = decltype(lrt)::value;
        return p.NG > 0 ? launch_q8_as<TOK, LRT, true>(pa, many, k, v, s) : launch_q8_as<TOK, LRT, false>(pa, many, k, v, s);
    };
    using std::integral_constant;
    if (p.D == 128) return go(integral_constant<int, 1>{}, integral_constant<int, 5>{});
    if (rows == 16) return go(integral_constant<int, 2>{}, integral_constant<int, 4>{});
    return go(integral_constant<int, 2>{}, integral_constant<int, 5>{});
}

}  // namespace kvc
