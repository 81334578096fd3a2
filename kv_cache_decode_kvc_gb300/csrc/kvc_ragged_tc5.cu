// kvc_ragged_tc5.cu -- attention of ragged new tokens over a paged bf16 cache on the 5th-generation
// tensor cores (D = 64 or 128).
//
// The streams and their split over the CTAs are those of kvc_ragged.cuh: a tile of query rows (tokens
// x heads of a group) against key tiles of 128.  A CTA has two sets of eight softmax warps, each
// with its own scores S (128 x 128 fp32, 128 columns of tensor memory), output O (128 x D fp32) and
// running state:
//   - class 0 (more than 64 rows): set s takes rows [128 s, 128 s + 128) of the stream's 256; both
//     read every K / V tile from the same shared-memory copy;
//   - class 1 (up to 64 rows: single tokens, drafts): each set walks streams of its own.
// While one set does its softmax the tensor cores work for the other.  Per tile and set:
// S = Q K^T (A = Q, B = K, both K-major); two threads per row load 64 scores each and agree on
// the row's maximum through shared memory; the reference maximum is raised only if it grew by more
// than 2^8 (then O is rescaled in place); the weights are written as bf16 over the scores'
// columns (each half over its own); O += P V (A = P from tensor memory, B = V read MN-major).
// Weights enter O += P V in bf16.  Class 1, which waits for memory, takes each as two terms, the leading bits
// and the rounded rest: off by 2^-15 of it.  (24 tokens at 3000 to 6000 positions: the second term's products are
// hidden, its arithmetic takes 4 us of 91.)  Class 0 takes one, off by at most half a step, 2^-8, as the output
// itself is after the division: there the tensor core and the softmax bound it, and the second term costs 40 % (a
// chunk of 4096 tokens behind 12,288 positions 1276 us -> 1796, six prompts 222 -> 305).  The denominator sums the
// unrounded weights in fp32.
//
// What bounds it.  Class 0: the chain of a set, from the S product's issue to its sight by the softmax 870
// cycles (512 of the tensor core), softmax 1300 (64 scores a thread; arithmetic of two warps on one
// sub-partition 594, of it exponentials 513), 430 to the P product's issue, 640 to the next S product's:
// 3250 per key tile of both sets, in which the tensor core works 2048 and the products and copies move 256 KB
// through shared memory.  Tensor memory holds S and O of two sets and no more.  1216 tokens of 32 heads at
// 16,384 positions: tensor pipe 65 % busy; a chunk of 4096 tokens of 64 heads behind 12,288 positions:
// 1276 us, 1.51 PFLOP/s (0.78 of cuBLAS's burst rate).  Weights signalled in two parts (their product begins
// earlier) took a fifth longer; without the maximum's search past the first tile (the sum shows that the
// reference holds), with products issued back to back or with other polling the period stayed as it is.
// A change of streams costs about 9 k cycles from the last weights to the next scores: the output's way
// out, the segments' hand-over and the first products are code that has left the instruction cache.
// Class 1, long streams: memory (24 single tokens at 3000 positions: a pair of 32 KB tiles per set every 6.9 k
// cycles, 5.4 TB/s).  Class 1, streams of a tile or two: the roles' code, run in turns, exceeds the 32 KB
// instruction cache (4700 misses per SM in 87 us at 256 tokens of 251 positions, no-instruction stalls ahead
// of all but the waits): its 2048 streams of two tiles take the 304 sets some 20 k cycles each.
//
// Warps: 0 copies (TMA), 1 issues the products, 2 computes the split and walks the streams, 3 guards
// masked values, 4-11 set 0 and 12-19 set 1 (four warps per half of the columns).  K and V tiles
// [8-row group][column block][8 rows][128 B] (128-byte swizzle), one ring slot each, in the order the
// products use them; every role replays that order from the same segments.
//
// Masked values: a weight of an unseen position is 0, but 0 times an infinite or NaN value is
// NaN.  Warp 3 zeroes V rows behind the stream's end (stale or never loaded), and in the tiles of the
// causal diagonal the non-finite values of positions that some row does not see; rows that do
// see them add them at the end of the segment (a finite sum plus an infinity or NaN is that).
#include <type_traits>

#include "kvc_decode_tc5.cuh"
#include "kvc_ragged_merge.cuh"

namespace kvc {

// What the polling loops need beside the barrier: at a fixed place of shared memory.
struct Give {
    int abort;  // a wait gave up: the others follow
    int pad;
    uint32_t* err;
};

template <int D_, bool JOINT>
struct RtCfg {
    static constexpr int D = D_;
    using R = RaggedTc5<JOINT>;
    using Seg = typename R::Seg;
    static constexpr int KT = R::KT;
    static constexpr int CB = D / 64;                // 128-byte column blocks of a row
    static constexpr int QSET = 128 * D * 2;         // a set's query bytes: 128 rows
    static constexpr int TILE = KT * D * 2;          // bytes of a K or V tile
    static constexpr int GSTR = 1024 * CB;           // 8-row group stride of a K / V tile
    static constexpr int MISC = 3 << 10;             // barriers, segments, exchanged maxima
    static constexpr int BUDGET = 232448;            // 227 KB
    static constexpr int NSLOT_A = (BUDGET - MISC - 2 * QSET) / TILE;
    static constexpr int NSLOT = NSLOT_A > 10 ? 10 : NSLOT_A;
    static constexpr int SMEM = 2 * QSET + NSLOT * TILE + MISC;
    static constexpr int HD = D / 2;                 // output columns of a thread
    static constexpr int THREADS = 640;
    // tensor memory columns: S of set s at 128 s, O of set s at 256 + D s
    static constexpr int TMEM_COLS = 512;
    static_assert(NSLOT >= 4, "ring too shallow");
    static_assert(NSLOT * TILE >= R::work_ints(MAX_B, MAX_B) * 4, "the split's arrays lie under the ring");
    struct Misc {
        uint64_t full[10], empty[10], vfix[10];
        uint64_t qpair, qfree;      // class 0: query rows landed; last product with them done
        uint64_t qfull[2][2];       // class 1: a set's query tile (two places in turn) landed
        uint64_t sfull[2], pfull[2], ofull[2], segfull[2][2], segempty[2][2], drain;
        Seg seg[2][2];              // [set][place]
        float xm[2][2][128];        // [set][column half][row] maxima, then denominators
        int nonfinite[2][2];        // [set][place]: warp 3 took non-finite values out of V
        int valid;
        uint32_t tmem, nq[5];       // nq: copies of query rows begun per barrier (qpair, qfull)
        Give give;
    };
    static_assert(sizeof(Misc) <= MISC, "misc area");
};

// 32 consecutive 32-bit columns of this thread's tensor-memory lane, loaded when it returns.
__device__ __forceinline__ void tc5_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32]; "
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 64 consecutive 32-bit columns of this thread's tensor-memory lane, loaded when it returns.
__device__ __forceinline__ void tc5_ld64(uint32_t taddr, float* v) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, "
        "%36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, "
        "%53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64]; "
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
// ... and stored (completion: tc5_wait_st).
__device__ __forceinline__ void tc5_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 "
        "[%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}; "
        :
        : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
          "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tc5_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Query rows of the smaller copied box: 16, or a token's if it has more (the same batch: 80.6 us against
// 82.6 with 64 always).
__host__ __device__ constexpr int few_rows(int G) { return G > 16 ? G : 16; }
// First row, of the set's 128, of its sc-th segment of class 1: its places are rows 0-63 and 64-127 in
// turn.  A warp reads the tensor-memory lanes of its quarter and a quarter's warps sit on one
// sub-partition of the SM, so a smaller box of up to 32 rows of set 1 takes the places' upper halves: the
// sets work on sub-partitions of their own (256 tokens x 4 heads of 251 positions: 80.6 us against 84.6).
// (The box of 64 rows fills a place.)
__device__ __forceinline__ int class1_row(int q, int sc, int rows, int G) {
    return (sc & 1) * 64 + (rows <= min(few_rows(G), 32) ? q * 32 : 0);
}
// 3-D copy of query rows: box (64 columns, G heads, tokens).
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* map, int col, int head, int token,
                                           uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(token), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// 32 bytes of a row at once (a whole sector per thread) or, where rows are only 16-byte aligned, two
// vectors.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// A row's two threads sit in different warps: 64 threads of named barrier id, and-reducing a predicate.
__device__ __forceinline__ bool pair_all(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, 64, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(id)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}
// One thread of the converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// The products with the varying halves of the descriptors as 32-bit values: computed warp-uniformly
// they stay in uniform registers, which halved the instructions per product (a product is 64 cycles of
// the tensor core at M = N = 128; issued from a divergent lane it took 60 cycles alone and over 100
// beside the softmax warps).
__device__ __forceinline__ void tc5_mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                           uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tc5_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                           uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
        : "memory");
}

// The kernel's roles and their unrolled tiles together exceed the instruction cache if each use of a
// helper is its own copy: the waits' polling, the rare paths and the roles' bodies are kept in one
// place each.
__device__ __forceinline__ bool try_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Has the phase completed?  Returns at once: try_wait may hold its thread for thousands of cycles, which is
// what a thread that waits wants and one with other work does not.
__device__ __forceinline__ bool done_at(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Polls until the phase has completed or the limit has passed (then the flag and the error word are
// set).  ns: sleep between polls.  The softmax warps wait most of the time, up to sixteen of them at
// once; asleep they leave the issue slots to the warps that work (a guarded tile took warp 3 up to 7 k
// cycles beside polling warps).
__device__ __noinline__ bool poll_at(uint32_t bar, uint32_t parity, uint32_t ns, Give* give) {
    volatile int* flag = &give->abort;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (true) {
        if (ns) __nanosleep(ns);
        if (try_at(bar, parity)) return true;
        if (*flag) return false;
        if (global_ns() - t0 > WAIT_LIMIT_NS) {
            *flag = 1;
            atomicOr(give->err, DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}
template <bool JOINT>
__device__ __noinline__ void zero_rows(const RaggedParams& p, int tid, int n) {
    ragged_zero_rows<__nv_bfloat16, JOINT>(p, tid, n);
}
// sum += 0 x, two bf16 values each: stays 0 but for an infinite or NaN x.
__device__ __forceinline__ void add_zero_times(uint32_t& sum, uint32_t x) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
}
// Adds the non-finite V values of positions [a, b) to a row's stored columns [col, col + n): out (bf16,
// already divided; the sum is the value or NaN either way) or a piece.
__device__ __noinline__ void add_nonfinite(const RaggedParams& p, int seq, int h, int a, int b, int col, int n,
                                           __nv_bfloat16* out, float* po) {
    for (int t = a; t < b; ++t) {
        const int64_t vr = cache_row_rd(p.table, p.bs, p.max_blocks, p.num_blocks, p.H_kv, p.T_max, seq, h, t, p.err);
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.V) + vr * p.D;
        for (int d = col; d < col + n; ++d) {
            const float x = __bfloat162float(v[d]);
            if (isfinite(x)) continue;
            if (po) po[d] += x;
            else out[d] = __float2bfloat16_rn(__bfloat162float(out[d]) + x);
        }
    }
}

// The order of the ring's items, replayed by the copy, product and guard warps.  fetch(l) loads the next
// segment of lane l.  A segment of class 0, which both sets walk together, is handled by whole(l): K of
// its tiles 0 ..  each followed by V (K0 V0 K1 V1 ..).  In class 1 each set is a lane and the lanes
// alternate: turn(l, v, k) handles V of tile l.j if v and K of the tile after it (0 if not v) if k; a
// segment's last V and the next segment's first K are turns of their own, one behind the other.
// All return false to stop (a wait gave up).
template <class Seg>
struct Lane {
    Seg g;
    int q, s, j;
    bool begun;      // K of tile j has been handled
    int ent, next;   // (copies) this CUDA lane's block of tile j and of the tile after it
    bool peeked;     // .. which is the next segment's first
};
template <class Seg, class Fetch, class Turn, class Whole>
__device__ __forceinline__ void replay(Fetch&& fetch, Turn&& turn, Whole&& whole) {
    Lane<Seg> a, b;
    a.q = a.s = a.j = b.s = b.j = 0;
    b.q = 1;
    a.begun = b.begun = a.peeked = b.peeked = false;
    bool both = true, more = true;  // class 0; lane a needs its next segment
    while (true) {
        if (more) {
            if (!fetch(a)) return;
            if (both) {
                if (!fetch(b)) return;  // (class 0: the same segment)
                ++b.s;
                both = a.g.n > 0 && a.g.cl == 0;
            }
            ++a.s;
        }
        more = false;
        if (both) {
            if (!whole(a)) return;
            more = true;
            continue;
        }
        if (a.g.n > 0) {
            const bool last = a.begun && a.j + 1 == a.g.n;
            if (!turn(a, a.begun, !last)) return;
            more = last;
            a.j = last || !a.begun ? 0 : a.j + 1;
            a.begun = !last;
            if (more) continue;
        }
        if (!both) {
            if (a.g.n == 0 && b.g.n == 0) return;
            const Lane<Seg> t = a;
            a = b;
            b = t;
        }
    }
}

template <int D, bool JOINT>
__global__ void __launch_bounds__(640, 1)
ragged_tc5_kernel(const RaggedParams p, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = RtCfg<D, JOINT>;
    using R = typename C::R;
    using Seg = typename C::Seg;
    using Misc = typename C::Misc;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    extern __shared__ __align__(1024) char rt_smem[];
    char* qbuf = rt_smem;
    char* ring = rt_smem + 2 * C::QSET;
    Misc& M = *reinterpret_cast<Misc*>(ring + C::NSLOT * C::TILE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = 1 << p.lgG;
    volatile int* ab = &M.give.abort;
    // Waits for a barrier's phase (false: gave up); sleep: ns between polls.
    auto wait_on = [&](uint64_t* bar, uint32_t parity, uint32_t sleep = 0) {
        const uint32_t at = smem_addr(bar);
        return try_at(at, parity) || poll_at(at, parity, sleep, &M.give);
    };
    if (smem_addr(rt_smem) & 1023) {  // (the swizzled tiles need it; the declaration asks for it)
        if (tid == 0) atomicOr(p.err, DEV_WAIT_TIMEOUT);
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&M.full[i], 1);
            mbar_init(&M.empty[i], 2);  // the products, and warp 3, which looks at every item
            mbar_init(&M.vfix[i], 1);
        }
        mbar_init(&M.qpair, 1);
        mbar_init(&M.qfree, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M.sfull[i], 1);
            mbar_init(&M.pfull[i], 8);
            mbar_init(&M.ofull[i], 1);
            for (int k = 0; k < 2; ++k) {
                mbar_init(&M.qfull[i][k], 1);
                mbar_init(&M.segfull[i][k], 1);
                mbar_init(&M.segempty[i][k], 11);  // copies, products, guard, the set's 8 warps
            }
        }
        mbar_init(&M.drain, 1);
        for (int i = 0; i < 5; ++i) M.nq[i] = 0;
        M.give.abort = 0;
        M.give.err = p.err;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&M.tmem)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc5_fence_before();
    }
    if (warp == 0 && lane < 4) {
        const CUtensorMap* m = lane == 0 ? &tmQ : lane == 1 ? &tmQ1 : lane == 2 ? &tmK : &tmV;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    // Warp 2 begins with the split at once and joins the others (barrier 9) before it hands out segments.
    if (warp != 2) named_bar_sync(10, C::THREADS - 32);
    tc5_fence_after();
    const uint32_t tmem = warp != 2 ? M.tmem : 0;
    uint32_t issued = 0;  // copies / products begun (copy and product threads)
    if (warp != 2) named_bar_arrive(9, C::THREADS);
    // Before any wait: a kernel that releases its dependents early may run for longer than a wait's limit.
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // A role's segment s of set q, as soon as it is known (the caller releases the place).
    auto fetch_seg = [&](int q, int s, Seg& g) {
        const bool ok = wait_on(&M.segfull[q][s & 1], (s >> 1) & 1);
        if (ok) g = M.seg[q][s & 1];
        return ok;
    };
    // ... by a whole warp that keeps its own copy and needs the place no longer.
    auto take_seg = [&](Lane<Seg>& l) {
        const bool ok = __all_sync(ALL, fetch_seg(l.q, l.s, l.g)) != 0;
        __syncwarp();  // (a vote orders no memory: all lanes have read it)
        if (ok && lane == 0) mbar_arrive(&M.segempty[l.q][l.s & 1]);
        return ok;
    };

    if (warp == 2) {
        // ====================================================== split and streams
        const typename R::Work work = R::work(p, ring);
        if (lane < 6) p.cuts[6 * blockIdx.x + lane] = make_int4(0, 0, 0, 0);
        const typename R::Split sp = R::scan(p, work, lane);
        if (lane == 0) M.valid = sp.valid;
        if (blockIdx.x == 0) {
            const int n = 2 * (R::groups(p) + p.B + 1);
            for (int i = lane; i < n; i += 32) p.plan[i] = sp.valid ? work.c[i] : 0;
            if (!sp.valid && lane == 0) atomicOr(p.err, sp.why);
        }
        typename R::Walk wk;
        if (lane < 3) wk = R::walk(p, sp, work, blockIdx.x, lane);
        fence_async_smem();
        named_bar_sync(9, C::THREADS);  // the split's arrays are read, the barriers set up
        // Lane 0 leaves the segments of class 0 to both sets, then lanes 1 and 2 those of class 1 to
        // theirs and the end.
        int s = 0;
        bool done = lane > 2, have = false;
        Seg g;
        g.n = 0;
        // When this lane first found its segment's place taken, 0: not yet.  (Counted from then on only: lanes 1 and 2
        // look for the first time when class 0 is over, which may take longer than a wait's limit.)
        uint64_t t0 = 0;
        while (__any_sync(ALL, !done)) {
            const bool pairs = (__ballot_sync(ALL, !done) & 1) != 0;
            const int s0 = __shfl_sync(ALL, s, 0);
            if (done) continue;
            if (!have) {
                g = R::next_seg(p, wk);
                have = true;
            }
            if (lane == 0 && g.n == 0) {
                done = true;
                continue;
            }
            if (lane > 0 && pairs) continue;
            if (lane > 0 && s < s0) s = s0;
            const int q0 = lane == 2 ? 1 : 0, q1 = lane == 1 ? 0 : 1;
            const uint32_t ph = ((s - 2) >> 1) & 1;
            if (s < 2 || (done_at(&M.segempty[q0][s & 1], ph) && done_at(&M.segempty[q1][s & 1], ph))) {
                for (int q = q0; q <= q1; ++q) {
                    M.seg[q][s & 1] = g;
                    mbar_arrive(&M.segfull[q][s & 1]);
                }
                if (wk.cut) R::leave_cut(p, sp, wk, blockIdx.x, lane, g);
                done = g.n == 0;
                have = false;
                ++s;
                t0 = 0;
            } else if (*ab) {
                done = true;
            } else {
                const uint64_t now = global_ns();
                if (t0 == 0) t0 = now;
                if (now - t0 > WAIT_LIMIT_NS) {
                    *ab = 1;
                    atomicOr(p.err, DEV_WAIT_TIMEOUT);
                }
            }
        }
    } else if (warp == 0) {
        // ====================================================== copies
        // tiles of class 1 are read once: they leave L2 first (the kernel's code and the batch's arrays, which
        // the next call needs from there, stay: 24 tokens at 3000 positions 58.6 us against 67.2)
        const uint64_t pol0 = policy_evict_normal(), pol1 = policy_evict_first();
        const int lgr = min(p.lgbs, 7);  // log2 of the rows of a copied box
        const int bt = lane << lgr;      // this lane's box of a tile begins at this row
        const uint32_t ring_s = smem_addr(ring), q_s = smem_addr(qbuf), to = bt * D * 2;
        uint32_t slot = 0, filled = 0;    // the next item's slot; parity of the slots' uses
        int npair = 0, sc0 = 0, sc1 = 0;  // segments begun: of class 0, of class 1 by set
        auto entry = [&](const Seg& g, int j) {  // this lane's block of key tile j
            const unsigned t = (unsigned)g.kv0 + j * C::KT + bt;  // (of the last tiles it may pass 2^31)
            return bt < C::KT && t < (unsigned)g.kv_end ? __ldg(p.table + (size_t)g.seq * p.max_blocks + (t >> p.lgbs)) : 0;
        };
        // K (isv false) or V of key tile j, whose block this CUDA lane knows
        auto copy = [&](const Seg& g, int j, int e, bool isv) {
            const int t0 = g.kv0 + j * C::KT, rows = min(g.kv_end - t0, C::KT), nbox = (rows + (1 << lgr) - 1) >> lgr;
            bool ok = true;
            if (lane == 0) {
                if (issued >= C::NSLOT) ok = wait_on(&M.empty[slot], filled & 1 ^ 1);
                if (ok) mbar_arrive_expect_tx(&M.full[slot], (uint32_t)((nbox << lgr) * D * 2));
            }
            if (!__all_sync(ALL, ok)) return false;
            __syncwarp();  // lane 0 has seen the slot empty
            ++issued;
            if (lane < nbox) {
                if ((unsigned)e >= (unsigned)p.num_blocks) {
                    atomicOr(p.err, DEV_BAD_BLOCK);
                    e = 0;
                }
                const int row = (int)((((int64_t)e * p.H_kv + g.h) << p.lgbs) + ((t0 + bt) & (p.bs - 1)));
                const uint32_t dst = ring_s + slot * C::TILE + to;
                const CUtensorMap* map = isv ? &tmV : &tmK;
                const uint64_t pol = g.cl == 0 ? pol0 : pol1;
                if constexpr (D == 128) tma_load_4d(dst, map, row >> 3, 0, &M.full[slot], pol);
                else tma_load_2d(dst, map, 0, row, &M.full[slot], pol);
            }
            if (++slot == C::NSLOT) {
                slot = 0;
                ++filled;
            }
            return true;
        };
        replay<Seg>(
            [&](Lane<Seg>& l) {
                const bool ok = take_seg(l);
                if (ok && !l.peeked && l.g.n > 0) l.next = entry(l.g, 0);
                l.peeked = false;
                return ok;
            },
            [&](Lane<Seg>& l, bool v, bool k) {  // class 1
                const Seg& g = l.g;
                if (!v) {
                    // the segment's query rows, into the set's places in turn: a place comes free with the
                    // segment before the last, the first ones with class 0's last products
                    const int rows = g.ntok << p.lgG, few = few_rows(G), sc = l.q ? sc1 : sc0, place = sc & 1;
                    const bool small = rows <= few;
                    bool ok = true;
                    if (lane == 0 && npair > 0 && sc == 0) ok = wait_on(&M.qfree, (npair - 1) & 1);
                    if (lane == 0 && ok) {
                        M.nq[1 + 2 * l.q + place] = (sc >> 1) + 1;
                        mbar_arrive_expect_tx(&M.qfull[l.q][place], C::CB * (small ? few * 128 : 8192));
                        for (int cb = 0; cb < C::CB; ++cb)
                            tma_load_q(q_s + l.q * C::QSET + cb * 16384 + class1_row(l.q, sc, rows, G) * 128, small ? &tmQ1 : &tmQ,
                                       cb * 64, g.h * G, g.row0, &M.qfull[l.q][place]);
                    }
                    if (l.q) ++sc1;
                    else ++sc0;
                    if (!__all_sync(ALL, ok)) return false;
                }
#pragma unroll 1
                for (int i = v ? 0 : 1; i < (k ? 2 : 1); ++i) {
                    const int j = l.j + (i && v ? 1 : 0);
                    if (i) {
                        l.ent = l.next;
                        if (j + 1 < g.n) l.next = entry(g, j + 1);
                    }
                    if (!copy(g, j, l.ent, i == 0)) return false;
                }
                // the segment after this one may be known: its first blocks are looked up ahead
                if (k && (v ? l.j + 2 : 1) == g.n &&
                    __all_sync(ALL, done_at(&M.segfull[l.q][l.s & 1], (l.s >> 1) & 1))) {
                    const Seg& n = M.seg[l.q][l.s & 1];
                    l.next = n.n > 0 ? entry(n, 0) : 0;
                    l.peeked = true;
                }
                return true;
            },
            [&](Lane<Seg>& l) {  // class 0
                const Seg& g = l.g;
                // query rows in boxes of 64 (set q's are 2 q, 2 q + 1), once the products with the last ones are
                // done
                const int boxes = ((g.ntok << p.lgG) + 63) / 64;
                bool ok = true;
                if (lane == 0 && npair > 0) ok = wait_on(&M.qfree, (npair - 1) & 1);
                ++npair;
                if (lane == 0 && ok) {
                    M.nq[0] = npair;
                    mbar_arrive_expect_tx(&M.qpair, boxes * C::CB * 8192);
#pragma unroll 1
                    for (int i = 0; i < boxes * C::CB; ++i) {
                        const int b = i / C::CB, cb = i - b * C::CB;
                        tma_load_q(q_s + (b >> 1) * C::QSET + (b & 1) * 8192 + cb * 16384, &tmQ, cb * 64, g.h * G,
                                   g.row0 + (b * 64 >> p.lgG), &M.qpair);
                    }
                }
                if (!__all_sync(ALL, ok)) return false;
                int e = 0;
#pragma unroll 1
                for (int i = 0; i < 2 * g.n; ++i) {
                    if ((i & 1) == 0) {
                        e = l.next;
                        l.next = entry(g, (i >> 1) + 1);
                    }
                    if (!copy(g, i >> 1, e, i & 1)) return false;
                }
                return true;
            });
    } else if (warp == 1) {
        // ====================================================== products
        // (the whole warp runs this, one elected thread issues)
        constexpr uint32_t ID1 = instr_desc_bf16(128, C::KT, 0, 0);
        constexpr uint32_t ID2 = instr_desc_bf16(128, D, 0, 1);
        const uint64_t dQ = smem_desc_sw128(smem_addr(qbuf), 16u, 1024u);
        const uint64_t dK = smem_desc_sw128(smem_addr(ring), 16u, C::GSTR);
        const uint64_t dV = smem_desc_sw128(smem_addr(ring), 1024u, C::GSTR);
        const uint32_t tm = __shfl_sync(ALL, tmem, 0);
        uint32_t item = 0, fix = 0, np = 0;  // parities: each slot's next guarded use, each set's weights
        int npair = 0, sc0 = 0, sc1 = 0;
        auto wait_item = [&](uint32_t it) { return wait_on(&M.full[it % C::NSLOT], (it / C::NSLOT) & 1); };
        // a V tile that some row does not see all of has passed warp 3
        auto wait_v = [&](const Seg& g, int j) {
            bool ok = wait_item(item);
            if (ok && g.lim0 - (g.kv0 + j * C::KT) < C::KT) {
                const uint32_t sl = item % C::NSLOT;
                ok = wait_on(&M.vfix[sl], (fix >> sl) & 1);
                fix ^= 1u << sl;
            }
            return ok;
        };
        auto uni = [&](uint32_t x) { return __shfl_sync(ALL, x, 0); };
        // O[q] (+)= P[q] V, V's descriptor vb; its commits.  (one elected thread issues)  The weights of 16
        // keys are 8 columns: in class 0 one behind the other in the first half of their scores' columns, in class 1
        // in the first half of those 16 keys' and their second terms in the second.
        auto apply = [&](auto cl, uint32_t q, uint32_t vb, uint32_t acc, uint64_t* done, uint64_t* freed) {
            tc5_fence_after();
            if (elect_one()) {
                // (unrolled in class 1 as well, 256 tokens at 251 positions take 100 us against 96: instruction fetch)
                constexpr int UNROLL = decltype(cl)::value == 0 ? C::KT / 16 : 2;
#pragma unroll UNROLL
                for (int kk = 0; kk < C::KT / 16; ++kk) {
                    const uint32_t a = tm + q * 128 + (cl == 0 ? (kk >> 2) * 64 + (kk & 3) * 8 : kk * 16);
                    const uint32_t b = vb + ((kk * 2 * C::GSTR) >> 4);
                    tc5_mma_ts(tm + 256 + q * D, a, b, (uint32_t)(dV >> 32), ID2, kk > 0 ? 1u : acc);
                    if (cl != 0) tc5_mma_ts(tm + 256 + q * D, a + 8, b, (uint32_t)(dV >> 32), ID2, 1u);
                }
                if (done) tc5_commit(done);
                if (freed) tc5_commit(freed);
            }
            __syncwarp();
        };
        // S[q] = Q K^T, descriptors qb and kb.  (In class 1 the rows of the other place come along unused.)
        auto score = [&](uint32_t q, uint32_t qb, uint32_t kb, uint64_t* freed, uint64_t* qfreed) {
            tc5_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc5_mma_ss(tm + q * 128, qb + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), (uint32_t)(dQ >> 32),
                               kb + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), (uint32_t)(dK >> 32), ID1, kk > 0);
                tc5_commit(&M.sfull[q]);
                if (freed) tc5_commit(freed);
                if (qfreed) tc5_commit(qfreed);
            }
            __syncwarp();
        };
        replay<Seg>(
            take_seg,
            [&](Lane<Seg>& l, bool v, bool k) {  // class 1
                const Seg& g = l.g;
                const int sc = l.q ? sc1 : sc0, place = sc & 1;
                const uint32_t vs = item % C::NSLOT, ki = item + (v ? 1 : 0), ks = ki % C::NSLOT;
                issued = 1;
                const uint32_t vb = (uint32_t)dV + uni(vs) * (C::TILE >> 4), kb = (uint32_t)dK + uni(ks) * (C::TILE >> 4);
                const uint32_t q = uni(l.q), acc = uni(l.j > 0 ? 1u : 0u);
                const uint32_t qb = (uint32_t)dQ + ((q * C::QSET) >> 4);
                if (v) {
                    bool ok = wait_v(g, l.j) && wait_on(&M.pfull[q], (np >> q) & 1);
                    np ^= 1u << q;
                    if (!__all_sync(ALL, ok)) return false;
                    apply(std::integral_constant<int, 1>{}, q, vb, acc, k ? nullptr : &M.ofull[q], &M.empty[vs]);
                }
                if (k) {
                    bool ok = v || wait_on(&M.qfull[q][place], (sc >> 1) & 1);
                    ok = ok && wait_item(ki);
                    if (!__all_sync(ALL, ok)) return false;
                    score(q, qb, kb, &M.empty[ks], nullptr);
                }
                item += (v ? 1 : 0) + (k ? 1 : 0);
                if (v && !k) {
                    if (l.q) ++sc1;
                    else ++sc0;
                }
                return true;
            },
            [&](Lane<Seg>& l) {  // class 0: V of tile j, K of tile j + 1, set by set
                // (written out for each set: with the set as a loop's variable a chunk of 4096 tokens takes a
                // quarter longer)
                const Seg& g = l.g;
                constexpr std::integral_constant<int, 0> class0;
                const int sets = (g.ntok << p.lgG) > 128 ? 2 : 1, n = g.n;
                const uint32_t qb = (uint32_t)dQ;
                auto v_desc = [&](uint32_t it) { return (uint32_t)dV + uni(it % C::NSLOT) * (C::TILE >> 4); };
                auto k_desc = [&](uint32_t it) { return (uint32_t)dK + uni(it % C::NSLOT) * (C::TILE >> 4); };
                auto ready = [&](int q) {
                    const bool ok = wait_on(&M.pfull[q], (np >> q) & 1);
                    np ^= 1u << q;
                    return __all_sync(ALL, ok) != 0;
                };
                if (!__all_sync(ALL, wait_on(&M.qpair, npair++ & 1) && wait_item(item))) return false;
                issued = 1;
                const uint32_t k0 = k_desc(item);
                score(0, qb, k0, sets == 1 ? &M.empty[item % C::NSLOT] : nullptr, sets == 1 && n == 1 ? &M.qfree : nullptr);
                if (sets == 2) score(1, qb + (C::QSET >> 4), k0, &M.empty[item % C::NSLOT], n == 1 ? &M.qfree : nullptr);
                ++item;
#pragma unroll 1
                for (int j = 0; j + 1 < n; ++j) {
                    const uint32_t vb = v_desc(item), kb = k_desc(item + 1), acc = uni(j > 0 ? 1u : 0u);
                    uint64_t *ve = &M.empty[item % C::NSLOT], *ke = &M.empty[(item + 1) % C::NSLOT];
                    uint64_t* qf = j + 2 == n ? &M.qfree : nullptr;
                    if (!__all_sync(ALL, wait_v(g, j)) || !ready(0)) return false;
                    apply(class0, 0, vb, acc, nullptr, sets == 1 ? ve : nullptr);
                    if (!__all_sync(ALL, wait_item(item + 1))) return false;
                    score(0, qb, kb, sets == 1 ? ke : nullptr, sets == 1 ? qf : nullptr);
                    if (sets == 2) {
                        if (!ready(1)) return false;
                        apply(class0, 1, vb, acc, nullptr, ve);
                        score(1, qb + (C::QSET >> 4), kb, ke, qf);
                    }
                    item += 2;
                }
                if (!__all_sync(ALL, wait_v(g, n - 1))) return false;
                const uint32_t vb = v_desc(item), acc = uni(n > 1 ? 1u : 0u);
                if (!ready(0)) return false;
                apply(class0, 0, vb, acc, &M.ofull[0], sets == 1 ? &M.empty[item % C::NSLOT] : nullptr);
                if (sets == 2) {
                    if (!ready(1)) return false;
                    apply(class0, 1, vb, acc, &M.ofull[1], &M.empty[item % C::NSLOT]);
                }
                ++item;
                return true;
            });
    } else if (warp == 3) {
        // ====================================================== masked values
        uint32_t item = 0;
        // Every item is waited for in turn and held until it has been seen: a barrier's parity tells
        // only neighbouring uses apart.  j: V of key tile j, -1: K.
        auto look = [&](const Lane<Seg>& l, int j) {
            const Seg& g = l.g;
            const uint32_t slot = item % C::NSLOT;
            if (!__all_sync(ALL, wait_on(&M.full[slot], (item / C::NSLOT) & 1))) return false;
            const int t0 = g.kv0 + j * C::KT;
            if (j >= 0 && g.lim0 - t0 < C::KT) {
                char* tile = ring + slot * C::TILE;
                const int end = min(g.kv_end - t0, C::KT), first = max(g.lim0 - t0, 0);
                constexpr int W = C::CB * 8;  // 16-byte pieces of a row
                uint32_t found = 0;
                auto piece = [&](int r, int w) {
                    return reinterpret_cast<uint4*>(tile + (r >> 3) * C::GSTR + (w >> 3) * 1024 + (r & 7) * 128 + (w & 7) * 16);
                };
                // Are there any?  The sum of all values times 0 is NaN if so (a test of each value here took 6 k cycles
                // for 64 rows, which the tile's product waits for).
                uint32_t sum = 0;
#pragma unroll 2
                for (int r = first + lane / W; r < end; r += 32 / W) {
                    const uint4 d = *piece(r, lane % W);
                    add_zero_times(sum, d.x);
                    add_zero_times(sum, d.y);
                    add_zero_times(sum, d.z);
                    add_zero_times(sum, d.w);
                }
                const bool some = __any_sync(ALL, (sum & 0x7F807F80u) != 0);
#pragma unroll 1
                for (int r = first + lane / W; some && r < end; r += 32 / W) {
                    uint4* a = piece(r, lane % W);
                    const uint4 d = *a;
                    // an all-ones exponent in either half of a word
                    auto bad = [](uint32_t u) {
                        return ((u & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((u & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
                    };
                    const uint4 b = make_uint4(bad(d.x), bad(d.y), bad(d.z), bad(d.w));
                    const uint32_t any = b.x | b.y | b.z | b.w;
                    found |= any;
                    if (any != 0) *a = make_uint4(d.x & ~b.x, d.y & ~b.y, d.z & ~b.z, d.w & ~b.w);
                }
                // rows behind the end: those of its 8-row group, then the whole groups
                if (end < C::KT) {
                    const int g8 = (end + 7) & ~7;
                    for (int c = end * W + lane; c < g8 * W; c += 32) {
                        *piece(c / W, c % W) = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll 4
                    for (int at = (g8 >> 3) * C::GSTR + lane * 16; at < C::TILE; at += 512)
                        *reinterpret_cast<uint4*>(tile + at) = make_uint4(0, 0, 0, 0);
                }
                if (found) {
                    M.nonfinite[l.q][(l.s - 1) & 1] = 1;
                    if (g.cl == 0) M.nonfinite[1][(l.s - 1) & 1] = 1;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&M.vfix[slot]);
            }
            if (lane == 0) mbar_arrive(&M.empty[slot]);
            ++item;
            return true;
        };
        replay<Seg>(
            [&](Lane<Seg>& l) {
                const bool ok = __all_sync(ALL, fetch_seg(l.q, l.s, l.g)) != 0;
                __syncwarp();
                if (ok && lane == 0) {
                    M.nonfinite[l.q][l.s & 1] = 0;
                    mbar_arrive(&M.segempty[l.q][l.s & 1]);
                }
                __syncwarp();
                return ok;
            },
            [&](Lane<Seg>& l, bool v, bool k) {
#pragma unroll 1
                for (int i = v ? 0 : 1; i < (k ? 2 : 1); ++i)
                    if (!look(l, i ? -1 : l.j)) return false;
                return true;
            },
            [&](Lane<Seg>& l) {
#pragma unroll 1
                for (int i = 0; i < 2 * l.g.n; ++i)
                    if (!look(l, i & 1 ? i >> 1 : -1)) return false;
                return true;
            });
    } else {
        // ====================================================== softmax and output
        const int set = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quad = warp & 3;
        const int r128 = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + set * 128 + lanes, tO = tmem + 256 + set * D + half * C::HD + lanes;
        const float c = p.qscale;
        // Binades that a row's maximum may grow by before its reference follows.  (Weights against a lower reference keep
        // their relative precision; only the room for sums of large values shrinks.  An 8-bit cache's keys differ
        // in size from block to block: with 8 there a chunk of 2048 tokens behind 12,288 positions took 866 us in all, with 16 656.)
        const float slack = p.part == 2 ? 16.f : 8.f;
        const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_ts * 2)) & 31) == 0;
        uint32_t ns = 0, no = 0;
        int sc = 0;  // segments of class 1 begun
        float* mine = &M.xm[set][half][r128];
        const float* other = &M.xm[set][half ^ 1][r128];
        // Both warps of a row's halves run the same loops to the end (a wait that gave up only skips the
        // stores), so the barrier between them always completes.
        const int bar = 1 + set * 4 + quad;
        auto fetch_dozing = [&](int q, int s, Seg& g) {
            const bool ok = wait_on(&M.segfull[q][s & 1], (s >> 1) & 1, 40);
            if (ok) g = M.seg[q][s & 1];
            return ok;
        };
        for (int s = 0;; ++s) {
            Seg g;
            if (!pair_all(bar, fetch_dozing(set, s, g))) break;
            if (s == 0 && M.valid) zero_rows<JOINT>(p, tid - 128, C::THREADS - 128);
            if (g.n == 0) break;
            const int nrow = g.ntok << p.lgG;
            const int r0 = g.cl == 0 ? set * 128 : -class1_row(set, sc, nrow, G);  // the set's lane 0 is row r0
            if (g.cl != 0) ++sc;
            const int r = r0 + r128, rw = r - lane;                             // the warp's first row sees least
            const bool idle = rw < 0 || rw >= nrow;
            bool ok = true;
            if (r0 < nrow) {
                // Warps without rows: with at most 64 rows the others arrive for them, else they keep
                // the protocol.
                const int quads = (min(nrow - max(r0, 0), 128) + 31) >> 5;
                const uint32_t count = quads == 1 ? 4 : quads == 2 ? 2 : 1;
                const int limit = g.sees(r >> p.lgG), limit_w = g.sees(rw >> p.lgG);
                float m = -INFINITY, l = 0.f;  // reference maximum of the raw scores, sum of this half's weights
                // Tile j's scores are in: waits, and gives its first position.
                auto begin = [&](int j) {
                    ok = wait_on(&M.sfull[set], ns++ & 1, 20) && ok;
                    __syncwarp();
                    tc5_fence_after();
                    return g.kv0 + j * C::KT;
                };
                // The row's maximum so far from this half's `top`; the reference is raised, and O with it, only if
                // it grew by more than `slack` binades.
                // Returns the weights' offset.
                auto agree = [&](float top, int j) {
                    *mine = top;
                    named_bar_sync(bar, 64);
                    top = fmaxf(top, *other);
                    const bool raise = (top - m) * c > slack;
                    if (__any_sync(ALL, raise)) {
                        const float mn = raise ? top : m;
                        const float f = raise ? fast_exp2((m - mn) * c) : 1.f;
                        if (j > 0) {
                            // the products into O so far are complete (S of this tile came behind them)
#pragma unroll 1
                            for (int d = 0; d < C::HD; d += 32) {
                                float o[32];
                                tc5_ld32(tO + d, o);
                                uint32_t u[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
                                tc5_st32(tO + d, u);
                            }
                        }
                        l *= f;
                        m = mn;
                    }
                    return m == -INFINITY ? 0.f : -m * c;  // nothing seen yet: weights 2^-inf = 0
                };
                // All 8 warps arrive for a segment's first tile, each of them once its rows of the segment before are
                // stored (its first product overwrites O, of all rows); later tiles' idle ones are arrived for.
                auto finish = [&](const float2& s, int j) {
                    l += s.x + s.y;
                    tc5_wait_st();
                    tc5_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(&M.pfull[set], j == 0 ? 1 : count);
                };
                if (idle) {
                    if (count > 1) {
                        if (lane == 0) mbar_arrive(&M.pfull[set]);
                        ns += g.n;
                    } else {
                        for (int j = 0; j < g.n; ++j) {
                            ok = wait_on(&M.sfull[set], ns++ & 1, 20) && ok;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&M.pfull[set]);
                        }
                    }
                } else if (g.cl == 0) {
                    for (int j = 0; j < g.n; ++j) {
                        const int t0 = begin(j);
                        float v[64];
                        tc5_ld64(tS + half * 64, v);
                        if (limit_w - t0 < half * 64 + 64) {
                            const int see = limit - t0 - half * 64;
#pragma unroll
                            for (int i = 0; i < 64; ++i) v[i] = i < see ? v[i] : -INFINITY;
                        }
                        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                        for (int i = 4; i < 64; i += 4) {
                            mx[0] = fmaxf(mx[0], v[i]);
                            mx[1] = fmaxf(mx[1], v[i + 1]);
                            mx[2] = fmaxf(mx[2], v[i + 2]);
                            mx[3] = fmaxf(mx[3], v[i + 3]);
                        }
                        const float mc = agree(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), j);
                        const float2 c2 = make_float2(c, c), mc2 = make_float2(mc, mc);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 a = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), c2, mc2);
                            const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                            sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                            w[i] = bf16x2_rn(e.x, e.y);
                        }
                        tc5_st32(tS + half * 64, w);
                        finish(__fadd2_rn(sum[0], sum[1]), j);
                    }
                } else {
                    // Few rows: the loop is kept short instead, 16 columns at a time, loaded again for the weights (all
                    // roles' code runs in turns here and has to fit the instruction cache).
                    for (int j = 0; j < g.n; ++j) {
                        // In a tile some row does not see all of, scores are masked in place first: the two loops do
                        // without comparisons, which cost 4 to 8 % of every tile (24 tokens at 3000 to 6000 positions
                        // 91.6 us, without them 85.6; 24 behind a common prompt, D = 64, 49.9 and 45.9).
                        const int t0 = begin(j) + half * 64;
                        if (limit_w - t0 < 64) {
                            const int see = limit - t0;
#pragma unroll 1
                            for (int d = 0; d < 64; d += 16) {
                                float x[16];
                                uint32_t u[16];
                                tc5_ld16(tS + half * 64 + d, x);
#pragma unroll
                                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(d + i < see ? x[i] : -INFINITY);
                                tc5_st16(tS + half * 64 + d, u);
                            }
                            tc5_wait_st();
                        }
                        float top = -INFINITY;
#pragma unroll 1
                        for (int d = 0; d < 64; d += 16) {
                            float x[16];
                            tc5_ld16(tS + half * 64 + d, x);
#pragma unroll
                            for (int i = 0; i < 16; ++i) top = fmaxf(top, x[i]);
                        }
                        const float mc = agree(top, j);
                        const float2 c2 = make_float2(c, c), mc2 = make_float2(mc, mc);
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
                        for (int d = 0; d < 64; d += 16) {
                            float x[16];
                            tc5_ld16(tS + half * 64 + d, x);
                            // The weight as two bf16 terms, in the place of the 16 scores.  The first is cut off from a
                            // little less than the weight, so both are positive where it is: an infinite value times
                            // them stays that infinity (a second term of 0 or below would make it NaN).
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float2 a = __ffma2_rn(make_float2(x[i], x[i + 1]), c2, mc2);
                                const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                                sum = __fadd2_rn(sum, e);
                                const float2 h = __fmul2_rn(e, make_float2(1.f - 0x1p-16f, 1.f - 0x1p-16f));
                                w[i / 2] = __byte_perm(__float_as_uint(h.x), __float_as_uint(h.y), 0x7632);
                                const float2 f = __ffma2_rn(make_float2(bf16_lo(w[i / 2]), bf16_hi(w[i / 2])), make_float2(-1.f, -1.f), e);
                                w[8 + i / 2] = bf16x2_rn(f.x, f.y);
                            }
                            tc5_st16(tS + half * 64 + d, w);
                        }
                        finish(sum, j);
                    }
                }
                // ---- the segment's state: written out, or left as a piece
                ok = wait_on(&M.ofull[set], no++ & 1, idle ? 100 : 20) && ok;
                if (!idle) {
                    __syncwarp();
                    tc5_fence_after();
                    *mine = l;
                    ok = pair_all(bar, ok);
                    l += *other;
                    named_bar_sync(bar, 64);  // read on both sides before the next segment's maxima
                    const bool nonfin = *(volatile int*)&M.nonfinite[set][s & 1] != 0;
                    const int64_t row = g.row0 + (r >> p.lgG);
                    const int head = g.h * G + (r & (G - 1));
                    const float inv = g.dst == -1 ? 1.f / l : 1.f;
                    float *po = nullptr, *pml = nullptr;
                    if (g.dst != -1) {
                        ragged_dst(p, g.dst, R::SLOT_ROWS, r, row, head, po, pml);
                        if (r < nrow && half == 0 && ok) *reinterpret_cast<float2*>(pml) = make_float2(m * c, l);
                    }
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_ts + (int64_t)head * D;
#pragma unroll 1
                    for (int d = 0; d < C::HD; d += 32) {
                        const int col = half * C::HD + d;
                        float o[32];
                        __syncwarp();
                        tc5_ld32(tO + d, o);
                        if (r < nrow && ok) {
                            if (g.dst == -1) {
#pragma unroll
                                for (int i = 0; i < 32; i += 16) {
                                    uint32_t w[8];
#pragma unroll
                                    for (int k = 0; k < 8; ++k) w[k] = bf16x2_rn(o[i + 2 * k] * inv, o[i + 2 * k + 1] * inv);
                                    store32(out + col + i, w, wide);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; i += 8) {
                                    uint32_t w[8];
#pragma unroll
                                    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(o[i + k]);
                                    store32(po + col + i, w, true);
                                }
                            }
                        }
                    }
                    if (nonfin && r < nrow && ok) {
                        // the values warp 3 took out of tiles this row sees part of
                        const int end = g.n > (limit - g.kv0) / C::KT ? limit : g.kv0 + g.n * C::KT;
                        add_nonfinite(p, g.seq, g.h, max(g.lim0, g.kv0), end, half * C::HD, C::HD, out,
                                      g.dst == -1 ? nullptr : po);
                    }
                    tc5_fence_before();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&M.segempty[set][s & 1]);
        }
    }
    __syncwarp();
    __syncthreads();  // every role is out of its loop (all waits are bounded)
    if (*ab) {
        // a wait timed out: let issued copies and products land, bounded
        if (tid == 0) {
            auto land = [&](uint64_t* bar, uint32_t uses) {
                const uint64_t t = global_ns();
                while (uses > 0 && !mbar_try_wait(bar, (uses - 1) & 1) && global_ns() - t < WAIT_LIMIT_NS) {
                }
            };
            land(&M.qpair, M.nq[0]);
            for (int i = 0; i < 4; ++i) land(&M.qfull[i >> 1][i & 1], M.nq[1 + i]);
            for (uint32_t it = issued > C::NSLOT ? issued - C::NSLOT : 0; it < issued; ++it)
                land(&M.full[it % C::NSLOT], it / C::NSLOT + 1);
        }
        if (warp == 1 && issued > 0) {
            if (elect_one()) tc5_commit(&M.drain);
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

template <int D, bool JOINT>
static int launch_rt(const RaggedParams& p, const CUtensorMap& q, const CUtensorMap& q1, const CUtensorMap& k,
                     const CUtensorMap& v, cudaStream_t s) {
    using C = RtCfg<D, JOINT>;
    static PerDeviceOnce once;
    const int e0 = once.run([] {
        return (int)cudaFuncSetAttribute(ragged_tc5_kernel<D, JOINT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ragged_tc5_kernel<D, JOINT>, p, q, q1, k, v);
    if (e != cudaSuccess) return (int)e;
    if (JOINT && p.part != 0) return 0;  // (merged with the pieces of the kernel on codes)
    return launch_merge<__nv_bfloat16, typename C::R, JOINT>(p, s);
}

int launch_ragged_tc5(const RaggedParams& p, const CUtensorMap& q, const CUtensorMap& q1, const CUtensorMap& k,
                      const CUtensorMap& v, cudaStream_t s) {
    if (p.NG > 0) return p.D == 128 ? launch_rt<128, true>(p, q, q1, k, v, s) : launch_rt<64, true>(p, q, q1, k, v, s);
    return p.D == 128 ? launch_rt<128, false>(p, q, q1, k, v, s) : launch_rt<64, false>(p, q, q1, k, v, s);
}

}  // namespace kvc
