// kvc_ragged.cuh -- attention of ragged new tokens over a paged cache: the work split shared by
// its kernels, and the merge of split streams.
//
// Row i of sequence b (T_b new tokens, lens[b] = L_b positions) sees positions [0, L_b - T_b + i]
// (the lower-right causal mask of "第 1 周 · Day 4：KV Cache 与 MQA / GQA" §3.3).  A softmax over
// a set of positions is a state (m, l, o) = (max s, sum e^(s-m), sum e^(s-m) v), and the states of
// disjoint sets merge exactly, so a row's positions may be cut anywhere and any rows may walk
// the same keys together:
//   - a stream is a tile of up to RT query rows of one KV head (TQ = RT / G consecutive tokens
//     times the G heads of the group, row r = (token r / G, head r % G)) and the keys they see, in
//     tiles of KT;
//   - a group of sequences with a common prefix of P positions has streams over [0, P) whose
//     rows come from all of its sequences (packed consecutively), no mask; each of its
//     sequences has streams over [P, L_b) as any sequence has over [0, L_b).  Groups and
//     sequences are the entries e in [0, NG + B) of the batch;
//   - all streams are laid end to end, each costing so much per key tile and for its start, and CTA
//     i of P takes the cost units [i U / P, (i + 1) U / P): equal work whatever the lengths, no
//     CTA waits for another, the same split on every run (results are reproducible);
//   - streams of class 0 come first, then those of class 1.  The tensor-core kernel has two
//     softmax sets per CTA: they share the streams of entries with more than PAIR_ROWS query
//     rows per head (class 0: each K / V tile feeds both), and halve the CTA's range of the
//     others (class 1) between them, each walking streams of its own.  Elsewhere all
//     streams are class 1 and a CTA is one worker.
// Everything is computed on the device from cu_seqlens, lens and the groups.
//
// A stream that one worker holds whole and that no other stream shares rows with is written to
// out.  Otherwise its pieces go to scratch and are merged (kvc_ragged_merge.cuh): the first piece of
// a stream of a sequence with a shared prefix to a row buffer (one for prefix streams, one for
// the sequences' own); of other streams, and all later pieces, to slots of their worker.
#pragma once

#include <math.h>

#include "kvc_internal.cuh"

namespace kvc {

// Entries with more query rows per head than this are class 0.  (Class 1 holds 64 at most; as class 0, 24
// sequences of 16 tokens x 4 heads at 3000 positions take 74.2 us against 68.5, 100 of them at 300 61.9
// against 54.3: one set of two would work on a stream, and idle at its start.)
constexpr int PAIR_ROWS = 64;

struct RaggedParams {
    const void* K;  // layer base, pools [num_blocks, H_kv, bs, D]
    const void* V;
    const void* q;  // [N, H_q, D], tokens q_ts elements apart
    void* out;      // [N, H_q, D], tokens out_ts elements apart
    int64_t q_ts, out_ts;
    const int32_t* table;  // [B, max_blocks]
    const int32_t* cu;     // [B + 1]
    const int32_t* lens;   // [B]
    const int32_t* groups; // [NG + 1], nullptr: no shared prefixes
    const int32_t* prefix; // [NG]
    uint32_t* err;
    int* plan;       // [2][NG + B + 1] per-head cost prefix sums of the classes, for the merge
    int4* cuts;      // [3 P][2] streams cut between workers (no groups), for the merge
    float* row_o;    // [2][N H_q][D] unnormalised outputs of first pieces (groups only)
    float* row_ml;   // [2][N H_q][2] (max in log2 units, denominator)
    float* slot_o;   // [P][slots][slot rows][D]
    float* slot_ml;  // [P][slots][slot rows][2]
    int B, N, H_q, H_kv, lgG, NG, D;
    int bs, lgbs, max_blocks, num_blocks, T_max;
    int P;          // CTAs at most
    float qscale;   // log2(e) / sqrt(D)
    // 8-bit caches: entries with more than `wide` query rows per head are attended by the kernel of plain pools, the
    // others by that on codes.  part: 0 all entries, 1 those with few rows, 2 the others: set by take().
    int wide, part;
    unsigned T0, T1;  // this call's entries have T0 .. T0 + T1 new tokens
    void take(int which, int rows) {
        wide = rows;
        part = which;
        const unsigned few = (unsigned)rows >> lgG;
        T0 = which == 2 ? few + 1 : 0;
        T1 = which == 1 ? few : ~0u - T0;
    }
};

// Scratch layout (bytes, 256-byte aligned parts), host side: P CTAs with `slots` slots of `rows` rows.
struct RaggedScratch {
    uint64_t plan, cuts, row_o, row_ml, slot_o, slot_ml, total;
};
inline RaggedScratch ragged_scratch(int B, int N, int NG, int H_q, int D, int P, int slots, int rows) {
    auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
    RaggedScratch s;
    uint64_t at = 0;
    s.plan = at;
    at += up(2 * (uint64_t)(B + NG + 1) * 4);
    s.cuts = at;
    at += up(3 * (uint64_t)P * 32);
    const uint64_t joint = NG > 0 ? 2ull * (uint64_t)N * (uint64_t)H_q : 0;
    s.row_o = at;
    at += up(joint * (uint64_t)D * 4);
    s.row_ml = at;
    at += up(joint * 8);
    const uint64_t held = (uint64_t)P * slots * rows;
    s.slot_o = at;
    at += up(held * (uint64_t)D * 4);
    s.slot_ml = at;
    at += up(held * 8);
    s.total = at;
    return s;
}

#ifdef __CUDACC__

// ------------------------------------------------------------------ entries and streams
struct Entry {
    int row0, T;  // packed rows [row0, row0 + T)
    int L, pfx;   // positions; shared prefix in effect (whole blocks, 0: none)
    int seq;      // table row
    bool group;   // a group's prefix: positions [0, pfx); else a sequence: [pfx, L)
    bool ok;      // has streams
    bool bad;     // a sequence with rows that cannot be attended (its outputs are zero)
};

// Shared prefix of group g of sequences [b0, b1): in effect (whole blocks; a group of one shares
// nothing); P as given may be out of range.
__device__ __forceinline__ int prefix_used(const RaggedParams& p, int b0, int b1, int P) {
    return (b1 - b0 < 2 || P < 0 || P > p.T_max) ? 0 : P >> p.lgbs << p.lgbs;
}
__device__ __forceinline__ Entry seq_entry(const RaggedParams& p, int b, int row0, int row1, int L, int P, int used) {
    Entry s;
    s.row0 = row0;
    s.T = row1 - row0;
    s.L = L;
    s.pfx = used;
    s.seq = b;
    s.group = false;
    s.ok = s.T > 0 && L >= s.T && L <= p.T_max && P >= 0 && P <= p.T_max && L - s.T >= P;
    s.bad = s.T > 0 && !s.ok;
    return s;
}
__device__ __forceinline__ Entry group_entry(int b0, int row0, int row1, int used) {
    Entry s;
    s.row0 = row0;
    s.T = row1 - row0;
    s.L = s.pfx = used;
    s.seq = b0;
    s.group = true;
    s.ok = s.T > 0 && used > 0;
    s.bad = false;
    return s;
}
// The same from the arrays in memory.
template <bool JOINT>
__device__ __forceinline__ Entry seq_entry(const RaggedParams& p, int b) {
    const int row0 = __ldg(p.cu + b), row1 = __ldg(p.cu + b + 1), L = __ldg(p.lens + b);
    int P = 0, used = 0;
    if (JOINT) {
        int lo = 0, hi = p.NG - 1;  // largest g with groups[g] <= b
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(p.groups + mid) <= b) lo = mid; else hi = mid - 1;
        }
        P = __ldg(p.prefix + lo);
        used = prefix_used(p, __ldg(p.groups + lo), __ldg(p.groups + lo + 1), P);
    }
    return seq_entry(p, b, row0, row1, L, P, used);
}
__device__ __forceinline__ Entry group_entry(const RaggedParams& p, int g) {
    const int b0 = __ldg(p.groups + g), b1 = __ldg(p.groups + g + 1), P = __ldg(p.prefix + g);
    return group_entry(b0, __ldg(p.cu + b0), __ldg(p.cu + b1), prefix_used(p, b0, b1, P));
}

// Is the entry this call's?
__device__ __forceinline__ bool in_part(const RaggedParams& p, const Entry& s) {
    return (unsigned)s.T - p.T0 <= p.T1;
}

// sum of ceil(x / 2^lg) for x = 1 .. X, modulo 2^32 (of far positions only differences fit: unsigned
// sums wrap, signed ones may not)
__host__ __device__ __forceinline__ unsigned triangle(unsigned n) { return ((n + 1) >> 1) * (n | 1); }  // 1 + .. + n
__host__ __device__ __forceinline__ unsigned ceil_sum(unsigned X, int lg) {
    const unsigned n = X >> lg;
    return (triangle(n) << lg) + (X & ((1u << lg) - 1)) * (n + 1);
}

// Work split.  LRT, LKT: log2 of a stream's rows and of a key tile; PAIRS: classes as the
// tensor-core kernel has them, and two workers per CTA for class 1; JOINT: the call has groups.
// (A CTA starts with a cold instruction cache, where code costs several times its warm time:
// the split's is kept short, and without groups their part is compiled out.)
// MANY > 0 (without PAIRS): entries with more query rows per head are class 0 of a tile's other cost; a CTA's worker
// walks its part of class 0, then that of class 1.  (At most one of its streams is cut at the end and one at the
// start: where class 0 ends in a CTA, it ends with a stream.)
template <int LRT, int LKT, bool PAIRS, bool JOINT, int MANY = 0>
struct Ragged {
    static constexpr bool CLASSES = PAIRS || MANY > 0;
    static constexpr int RT = 1 << LRT, KT = 1 << LKT;
    // scratch slots of a CTA: with PAIRS five of 128 rows (a shared stream's later piece takes 0-1,
    // its first piece 2-3 and then ends the range; set 0: 0 and 2, set 1: 3 and 4)
    static constexpr int SLOTS = PAIRS ? 5 : 2, SLOT_ROWS = PAIRS ? RT / 2 : RT;

    // Cost units of a key tile and of a stream's start, by class.  (Measured with starts of 4, 6, 8 and 10 in
    // class 0: six prompts of 700 to 4096 tokens 221, 220, 227, 234 us; of 2, 3, 4 in class 1: 256 single tokens
    // with up to 500 positions behind 16,384 common ones 181, 153, 162 us, 200 with 350 behind as many 132,
    // 139, 146: where the cuts happen to fall weighs as much as what a start costs, 3 is a middle; tiles of class 1 at
    // 1/2, 1 and 3/2 of class 0's: a batch of chunks and tokens 176, 133, 168.)
    // (MANY, the kernel on codes: a tile of 32 rows takes 1.7 to 2.2 us, one of up to 8, which comes from memory, 1.3.  Tiles of
    // 5 : 3, 7 : 3, 7 : 4 with starts of 9 : 9, 24 : 7, 24 : 9: 24 tokens behind 2048 common positions 59.3, 53.2, 51.4 us, 128
    // with 10 to 100 of their own 72.9, 69.4, 66.4; 24 tokens alone 47.0, 46.2, 46.5.)
    __host__ __device__ static constexpr int tile_cost(int cl) { return PAIRS ? 2 : MANY > 0 ? (cl == 0 ? 7 : 4) : 1; }
    __host__ __device__ static constexpr int start_cost(int cl) { return PAIRS ? (cl == 0 ? 6 : 3) : MANY > 0 ? (cl == 0 ? 24 : 9) : 1; }
    // log2 of the units a CTA takes at least: a worker between two pieces of a stream then holds a tile
    // of it (a worker's share, half of that in class 1, is a tile's cost or more).  With class 0 twice that,
    // a stream's start (one of 1 x 4000 positions 18.3 us against 20.6 with the larger share, 200 tokens at
    // 500 positions 26.5 against 31.3 with the smaller).
    __device__ static int lg_min(int W0) { return MANY > 0 ? 3 : !PAIRS ? 0 : W0 > 0 ? 3 : 2; }
    __device__ static int groups(const RaggedParams& p) { return JOINT ? p.NG : 0; }
    __device__ static Entry entry_of(const RaggedParams& p, int e) {
        if (JOINT && e < p.NG) return group_entry(p, e);
        return seq_entry<JOINT>(p, e - groups(p));
    }
    __host__ __device__ static int cls(const RaggedParams& p, const Entry& s) {
        return CLASSES && ((int64_t)s.T << p.lgG) > (PAIRS ? PAIR_ROWS : MANY) ? 0 : 1;
    }
    // Key tiles of a stream of an entry with S0 keys of its own before its new tokens, whose
    // last row is new token t1 - 1: positions [pfx, pfx + S0 + t1).
    __host__ __device__ static int tiles(int S0, int t1) { return (int)(((unsigned)S0 + (unsigned)t1 + KT - 1) >> LKT); }
    // Costs are 32-bit (a call of more than MOST units, some 12 s of work, is refused: scan).  Key tiles of an entry's first
    // k streams, all full (TQ = 2^lq tokens each): sum over i = 1 .. k of ceil((S0 + i TQ) / KT).
    __host__ __device__ static int tiles_full(int S0, int k, int lq) {
        if (lq >= LKT) return (int)((unsigned)k * (((unsigned)S0 + KT - 1) >> LKT) + (triangle(k) << (lq - LKT)));
        // ceil((S0 + i TQ) / KT) = ceil((ceil(S0 / TQ) + i) / (KT / TQ))
        const unsigned s = ((unsigned)S0 + (1u << lq) - 1) >> lq;
        return (int)(ceil_sum(s + k, LKT - lq) - ceil_sum(s, LKT - lq));
    }
    __host__ __device__ static int cost(const RaggedParams& p, const Entry& s, int cl) {
        if (!s.ok) return 0;
        const int lq = LRT - p.lgG, nk = (int)((unsigned)(s.T + (1 << lq) - 1) >> lq), S0 = s.L - s.T - s.pfx;
        const unsigned n = JOINT && s.group ? (unsigned)nk * (unsigned)tiles(s.pfx, 0)
                                            : (unsigned)tiles_full(S0, nk - 1, lq) + (unsigned)tiles(S0, s.T);
        return (int)(n * tile_cost(cl) + (unsigned)nk * start_cost(cl));
    }
    // At least that, to a few parts in a million, and at most a tile or two per stream more; does not wrap.
    __host__ __device__ static float cost_about(const RaggedParams& p, const Entry& s, int cl) {
        if (!s.ok) return 0.f;
        const int lq = LRT - p.lgG, nk = (int)(((unsigned)s.T + (1u << lq) - 1) >> lq);
        const float f = (float)nk, own = JOINT && s.group ? (float)s.pfx : (float)(s.L - s.T - s.pfx) + 0.5f * (1 << lq) * (f + 1.f);
        return f * ((own / KT + 1.f) * tile_cost(cl) + start_cost(cl));
    }
    // A call of more units is refused (2^31 less the estimate's part in a million, rounded down).
    static constexpr float MOST = 2.1e9f;

    // The batch's split: total cost U, class 0's part W0, CTAs P.
    // CTA i of P takes `each` units, the first `more` of them one more.
    struct Split {
        int U, W0, P, each, more;
        bool valid;
        uint32_t why;  // not valid: the error to flag
    };
    __device__ static void divide(const RaggedParams& p, Split& sp) {
        const int want = sp.U >> lg_min(sp.W0);
        sp.P = sp.U == 0 ? 0 : max(1, min(want, p.P));
        sp.each = sp.U == 0 ? 0 : (int)((unsigned)sp.U / (unsigned)sp.P);
        sp.more = sp.U - sp.each * sp.P;
    }
    __device__ static int begin(const Split& sp, int i) { return i * sp.each + min(i, sp.more); }
    __device__ static int cta(const Split& sp, int x) {
        const int y = x - sp.more * (sp.each + 1);
        return y < 0 ? (int)((unsigned)x / (unsigned)(sp.each + 1)) : sp.more + (int)((unsigned)y / (unsigned)sp.each);
    }
    // What one warp computes in shared memory (work_ints of it): the per-head cost prefix sums
    // c[0 .. NE], c[NE + 1 .. 2 NE + 1] of the two classes (NE = NG + B), the entries, a copy of the
    // groups.
    struct Work {
        int4* ent;  // (row0, T, L, pfx and flags: sequence ok 1)
        int *c, *groups, *prefix;
    };
    static constexpr int work_ints(int B, int NG) { return 4 * (B + NG) + 2 * (B + NG + 1) + 2 * NG + 1; }
    __device__ static Work work(const RaggedParams& p, void* smem) {
        const int NE = groups(p) + p.B;
        Work k;
        k.ent = static_cast<int4*>(smem);
        k.c = reinterpret_cast<int*>(k.ent + NE);
        k.groups = k.c + 2 * (NE + 1);
        k.prefix = k.groups + p.NG + 1;
        return k;
    }
    // ... and whether cu and the groups ascend within their bounds and the sums hold the cost.
    __device__ static Split scan(const RaggedParams& p, const Work& k, int lane) {
        const int NE = groups(p) + p.B;
        int* c = k.c;
        int carry[2] = {0, 0};
        float about = 0.f;  // the total cost
        bool bad = false;
        if (lane < 2) c[lane * (NE + 1)] = 0;
        for (int g = lane; JOINT && g <= p.NG; g += 32) {
            const int b0 = __ldg(p.groups + g);
            bad |= b0 < 0 || b0 > p.B || (g == 0 && b0 != 0) || (g == p.NG && b0 != p.B);
            k.groups[g] = b0;
            if (g < p.NG) k.prefix[g] = __ldg(p.prefix + g);
        }
        if (JOINT) {
            bad = __any_sync(0xFFFFFFFFu, bad);
            __syncwarp();  // the copies are read by other lanes below, and a vote orders no memory
        }
        for (int e0 = 0; e0 < NE && !bad; e0 += 32) {
            const int e = e0 + lane;
            Entry s;
            s.ok = false;
            bool fine = e >= NE;
            if (JOINT && e < p.NG) {
                const int b0 = k.groups[e], b1 = k.groups[e + 1];
                fine = b1 >= b0;
                if (fine) s = group_entry(b0, __ldg(p.cu + b0), __ldg(p.cu + b1), prefix_used(p, b0, b1, k.prefix[e]));
            } else if (e < NE) {
                const int b = e - groups(p), c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), L = __ldg(p.lens + b);
                fine = c0 >= 0 && c1 >= c0 && c1 <= p.N && (b > 0 || c0 == 0);
                int P = 0, used = 0;
                if (JOINT) {
                    int lo = 0, hi = p.NG - 1;  // largest g with groups[g] <= b
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (k.groups[mid] <= b) lo = mid; else hi = mid - 1;
                    }
                    P = k.prefix[lo];
                    used = prefix_used(p, k.groups[lo], k.groups[lo + 1], P);
                }
                s = seq_entry(p, b, c0, c1, L, P, used);
            }
            bad |= !fine;
            int x[2] = {0, 0};
            if (fine && e < NE) {
                const int cl = cls(p, s);
                if (in_part(p, s)) {
                    x[cl] = cost(p, s, cl);
                    about += cost_about(p, s, cl);
                }
                k.ent[e] = make_int4(s.row0, s.T, s.L, s.pfx);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t1 = __shfl_up_sync(0xFFFFFFFFu, x[1], o);
                const int t0 = CLASSES ? __shfl_up_sync(0xFFFFFFFFu, x[0], o) : 0;
                if (lane >= o) {
                    x[0] += t0;
                    x[1] += t1;
                }
            }
            if (e < NE) {
                c[e + 1] = carry[0] + x[0];
                c[NE + 1 + e + 1] = carry[1] + x[1];
            }
            carry[0] += CLASSES ? __shfl_sync(0xFFFFFFFFu, x[0], 31) : 0;
            carry[1] += __shfl_sync(0xFFFFFFFFu, x[1], 31);
            bad = __any_sync(0xFFFFFFFFu, bad);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) about += __shfl_xor_sync(0xFFFFFFFFu, about, o);
        Split sp;
        sp.why = bad ? DEV_BAD_SEQ : DEV_TOO_LARGE;
        sp.valid = !bad && about * (float)p.H_kv <= MOST;
        sp.W0 = sp.valid ? carry[0] * p.H_kv : 0;
        sp.U = sp.valid ? sp.W0 + carry[1] * p.H_kv : 0;
        divide(p, sp);
        __syncwarp();
        return sp;
    }
    // The split as the attention kernel left it in p.plan.
    __device__ static Split planned(const RaggedParams& p) {
        const int NE = groups(p) + p.B;
        Split sp;
        sp.W0 = p.plan[NE] * p.H_kv;
        sp.U = sp.W0 + p.plan[2 * NE + 1] * p.H_kv;
        sp.valid = sp.U > 0;
        divide(p, sp);
        return sp;
    }

    // Worker w of CTA i: 0 the CTA as a whole (class 0), 1 and 2 its sets (class 1; without
    // PAIRS only 1).  Cost units [a, b).
    __device__ static void range(const Split& sp, int i, int w, int& a, int& b) {
        a = b = 0;
        if (i >= sp.P) return;
        const int x0 = begin(sp, i), x1 = begin(sp, i + 1);
        if (w == 0) {
            a = x0;
            b = x1 < sp.W0 ? x1 : sp.W0;
            return;
        }
        a = x0 > sp.W0 ? x0 : sp.W0;
        b = x1;
        if (PAIRS && b > a) {
            const int mid = a + (b - a + 1) / 2;
            if (w == 1) b = mid; else a = mid;
        }
    }
    // The worker that owns unit x, as a position in the order of its class: CTA for class 0,
    // 2 CTA + set (CTA without PAIRS) for class 1.
    __device__ static int owner(const Split& sp, int x) {
        const int i = cta(sp, x);
        if (!PAIRS || x < sp.W0) return i;
        int a, b;
        range(sp, i, 2, a, b);
        return 2 * i + (x >= a ? 1 : 0);
    }
    // The worker of key tile j of a stream of class cl.
    template <class S>
    __device__ static int owner_of(const Split& sp, const S& st, int cl, int j) {
        return owner(sp, st.u0 + start_cost(cl) + j * tile_cost(cl));
    }
    // Slot of a worker's piece: `later` piece of a stream (it opens the worker's range) or its first.
    __device__ static int slot(int cl, int own, bool later) {
        if (!PAIRS) return own * 2 + (later ? 0 : 1);
        if (cl == 0) return own * 5 + (later ? 0 : 2);
        return (own >> 1) * 5 + ((own & 1) ? (later ? 3 : 4) : (later ? 0 : 2));
    }

    struct Stream {
        Entry s;
        int e, h, k;
        int u0;  // its first cost unit
        int n;   // key tiles
    };
    __device__ static void fill(const RaggedParams& p, Stream& st) {
        const int lq = LRT - p.lgG;
        if (JOINT && st.s.group) {
            st.n = tiles(st.s.pfx, 0);
        } else {
            const int64_t t1 = (int64_t)(st.k + 1) << lq;
            st.n = tiles(st.s.L - st.s.T - st.s.pfx, t1 < st.s.T ? (int)t1 : st.s.T);
        }
    }
    // The stream holding cost unit x.
    __device__ static Stream locate(const RaggedParams& p, const Split& sp, const Work& k, int x) {
        const int NE = groups(p) + p.B, lq = LRT - p.lgG;
        const int* c = k.c;
        Stream st;
        const int base = x < sp.W0 ? 0 : sp.W0, tc = tile_cost(x < sp.W0 ? 0 : 1), sc = start_cost(x < sp.W0 ? 0 : 1);
        if (x >= sp.W0) c += NE + 1;
        int lo = 0, hi = NE - 1;  // largest e with H_kv c[e] <= x - base
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (c[mid] * p.H_kv <= x - base) lo = mid; else hi = mid - 1;
        }
        st.e = lo;
        const int4 w = k.ent[lo];
        st.s.row0 = w.x;
        st.s.T = w.y;
        st.s.L = w.z;
        st.s.pfx = w.w;
        st.s.group = JOINT && lo < p.NG;
        st.s.seq = JOINT && st.s.group ? k.groups[lo] : lo - groups(p);
        st.s.ok = true;
        st.s.bad = false;
        const int per = c[lo + 1] - c[lo];
        int r = x - base - c[lo] * p.H_kv;
        st.h = (int)((unsigned)r / (unsigned)per);
        r -= st.h * per;
        st.u0 = base + c[lo] * p.H_kv + st.h * per;
        if (JOINT && st.s.group) {
            const int one = tiles(st.s.pfx, 0) * tc + sc;
            st.k = (int)((unsigned)r / (unsigned)one);
            st.u0 += st.k * one;
        } else {
            // largest k with k streams costing at most r: by the real root of
            // tc (k^2 TQ / 2 + k (S0 + KT / 2)) + k sc KT = r KT, then steps (the ceilings differ from the half
            // tile by less than one stream's cost)
            const int S0 = st.s.L - st.s.T - st.s.pfx, last = (int)((unsigned)(st.s.T + (1 << lq) - 1) >> lq) - 1;
            int a = 0;
            if (last > 0) {
                const float TQ = (float)(1 << lq), b1 = (float)S0 + 0.5f * TQ + KT * ((float)sc / tc + 0.5f);
                const float root = (sqrtf(b1 * b1 + 2.f * TQ * KT * (float)r / tc) - b1) / TQ;
                a = min(max((int)root, 0), last);
                while (a > 0 && tiles_full(S0, a, lq) * tc + a * sc > r) --a;
                while (a < last && tiles_full(S0, a + 1, lq) * tc + (a + 1) * sc <= r) ++a;
            }
            st.k = a;
            st.u0 += tiles_full(S0, a, lq) * tc + a * sc;
        }
        fill(p, st);
        return st;
    }
    // The stream of packed row `row` of entry e.
    __device__ static Stream of_row(const RaggedParams& p, const Split& sp, const int* c, int e, const Entry& s, int h, int row) {
        const int NE = groups(p) + p.B, lq = LRT - p.lgG;
        Stream st;
        st.e = e;
        st.h = h;
        st.s = s;
        st.k = (row - st.s.row0) >> lq;
        const int cl = cls(p, st.s);
        c += cl * (NE + 1);
        st.u0 = (cl == 0 ? 0 : sp.W0) + c[e] * p.H_kv + h * (c[e + 1] - c[e]);
        const int n = JOINT && st.s.group ? st.k * tiles(st.s.pfx, 0)
                                          : tiles_full(st.s.L - st.s.T - st.s.pfx, st.k, lq);
        st.u0 += n * tile_cost(cl) + st.k * start_cost(cl);
        fill(p, st);
        return st;
    }
    // The next stream of class cl after st; false if there is none.
    __device__ static bool next(const RaggedParams& p, Stream& st, int cl) {
        const int lq = LRT - p.lgG;
        st.u0 += st.n * tile_cost(cl) + start_cost(cl);
        if (((int64_t)(st.k + 1) << lq) < st.s.T) {
            ++st.k;
        } else {
            const bool one = st.k == 0;
            st.k = 0;
            if (++st.h < p.H_kv && one) return true;  // the same keys of the next head
            if (st.h == p.H_kv) {
                st.h = 0;
                do {
                    if (++st.e == groups(p) + p.B) return false;
                    st.s = entry_of(p, st.e);
                } while (!st.s.ok || cls(p, st.s) != cl || !in_part(p, st.s));
            }
        }
        fill(p, st);
        return true;
    }

    // A worker's piece of a stream.
    struct Seg {
        int n;           // key tiles (0: no more segments)
        int seq, h;      // table row, KV head
        int row0, ntok;  // packed rows of the tile
        int kv0;         // position of its first key tile
        int kv_end;      // positions [kv0, kv_end) exist for the stream
        int lim0;        // row of token i sees positions below sees(i); all see those below lim0
        // (no sum here passes kv_end, which may be close to 2^31)
        __device__ int sees(int i) const { return lim0 + min(i, kv_end - lim0); }
        int dst;         // -1 out, -2 / -3 row buffer 0 / 1, else the slot
        int cl;          // class
    };
    // The part [x, x1) of stream st as a segment (n = 0 if it holds no tile).  own: the worker
    // (as `owner` counts).
    __device__ static Seg segment(const RaggedParams& p, const Stream& st, int cl, int own, int x, int x1) {
        const int lq = LRT - p.lgG;
        Seg g;
        // a tile belongs to the worker that owns its first unit
        const int tc = tile_cost(cl), first = st.u0 + start_cost(cl);
        const int j0 = (int)((unsigned)max(x - first + tc - 1, 0) / (unsigned)tc);
        const int j1 = min((int)((unsigned)max(x1 - first + tc - 1, 0) / (unsigned)tc), st.n);
        g.n = j1 - j0;
        g.cl = cl;
        g.seq = st.s.seq;
        g.h = st.h;
        g.row0 = st.s.row0 + (st.k << lq);
        g.ntok = min(1 << lq, st.s.T - (st.k << lq));
        g.kv0 = (JOINT && st.s.group ? 0 : st.s.pfx) + (j0 << LKT);
        if (JOINT && st.s.group) {
            g.kv_end = st.s.pfx;
            g.lim0 = st.s.pfx;
        } else {
            const int S = st.s.L - st.s.T + (st.k << lq);  // position of the tile's first token
            g.kv_end = S + g.ntok;
            g.lim0 = S + 1;
        }
        if (j0 > 0) g.dst = slot(cl, own, true);
        else if (JOINT && st.s.pfx > 0) g.dst = st.s.group ? -2 : -3;  // rows shared with another stream
        else g.dst = j1 == st.n ? -1 : slot(cl, own, false);
        return g;
    }

    // A worker's segments, in order.
    struct Walk {
        Stream st;
        int x, x1, own, cl;
        bool cut;   // the last segment is a piece, not the last, of a stream that others share no rows with
        bool step;  // st is done: the next segment is in the stream after it
    };
    __device__ static Walk walk(const RaggedParams& p, const Split& sp, const Work& wk, int i, int w) {
        Walk k;
        range(sp, i, w, k.x, k.x1);
        k.cl = w == 0 ? 0 : 1;
        k.own = PAIRS && w > 0 ? 2 * i + (w - 1) : i;
        k.cut = k.step = false;
        if (k.x < k.x1) k.st = locate(p, sp, wk, k.x);
        return k;
    }
    __device__ static Seg next_seg(const RaggedParams& p, Walk& k) {
        Seg g;
        g.n = 0;
        g.cl = k.cl;
        k.cut = false;
        while (g.n == 0 && k.x < k.x1) {
            if (k.step && !next(p, k.st, k.cl)) break;
            g = segment(p, k.st, k.cl, k.own, k.x, k.x1);
            k.cut = k.st.s.pfx == 0 && g.dst >= 0 && g.n > 0 && (g.kv0 == 0 || (g.kv0 >> LKT) + g.n < k.st.n);
            k.x = k.st.u0 + start_cost(k.cl) + k.st.n * tile_cost(k.cl);
            k.step = true;
        }
        return g;
    }
    // Leaves the cut stream that ends worker w's range (k.cut, g its last segment) for the merge:
    // entry 3 i + w is (pieces, first owner, class, packed row), (rows of the tile, KV head, this piece).
    __device__ static void leave_cut(const RaggedParams& p, const Split& sp, const Walk& k, int i, int w, const Seg& g) {
        const int first = g.kv0 == 0 ? k.own : owner_of(sp, k.st, k.cl, 0), last = owner_of(sp, k.st, k.cl, k.st.n - 1);
        p.cuts[2 * (3 * i + w)] = make_int4(last - first + 1, first, k.cl, g.row0);
        p.cuts[2 * (3 * i + w) + 1] = make_int4(g.ntok << p.lgG, g.h, k.own - first, 0);
    }
};

// The split of the tensor-core kernel of plain pools.
template <bool JOINT>
using RaggedTc5 = Ragged<8, 7, true, JOINT>;

// Zero output rows of the sequences that cannot be attended (CTA-strided over sequences, thread tid
// of n).
template <typename T, bool JOINT>
__device__ __forceinline__ void ragged_zero_rows(const RaggedParams& p, int tid, int n) {
    const int vecs = p.H_q * p.D * Elem<T>::BYTES / 16;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const Entry s = seq_entry<JOINT>(p, b);
        if (!s.bad) continue;
        if (tid == 0) atomicOr(p.err, DEV_BAD_LENS);
        for (int64_t i = tid; i < (int64_t)s.T * vecs; i += n) {
            const int64_t r = i / vecs;
            char* row = static_cast<char*>(p.out) + (s.row0 + r) * p.out_ts * Elem<T>::BYTES;
            reinterpret_cast<uint4*>(row)[i - r * vecs] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Where the state of packed row `row`, head j (query row r of its tile) of a segment with dst != -1
// goes.
__device__ __forceinline__ void ragged_dst(const RaggedParams& p, int dst, int slot_rows, int r, int64_t row, int j,
                                           float*& o, float*& ml) {
    if (dst < 0) {
        const int64_t at = ((int64_t)(-2 - dst) * p.N + row) * p.H_q + j;
        o = p.row_o + at * p.D;
        ml = p.row_ml + at * 2;
    } else {
        const int64_t at = (int64_t)dst * slot_rows + r;
        o = p.slot_o + at * p.D;
        ml = p.slot_ml + at * 2;
    }
}

#endif  // __CUDACC__

// Launchers (kvc_ragged.cu, kvc_ragged_tc5.cu, kvc_rope.cu); each returns a cudaError_t.
int launch_ragged_cc(int dtype, const RaggedParams& p, cudaStream_t s);
// bf16, D = 64 or 128; q, q1: make_q_tensor_map with boxes of 64 rows and of max(16, G); k / v: the
// pool's maps with min(bs, 128)-row boxes.
int launch_ragged_tc5(const RaggedParams& p, const CUtensorMap& q, const CUtensorMap& q1, const CUtensorMap& k,
                      const CUtensorMap& v, cudaStream_t s);
// Radians per position as turns per position modulo 1 (whole turns change nothing), in 2^-64 turns.
// 1 / (2 pi) and the product are sums of two doubles, so the result is within 2^-62 of a turn for rates
// up to 2^44 (an angle at position 2^31 within 2^-31); a negative rate is the negated fraction, not the
// rest to the next turn, which a double would round.
inline uint64_t rope_turns(double rate) {
    const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;  // 1 / (2 pi)
    const double a = fabs(rate);
    const volatile double rounded = a * hi;  // (volatile: not fused into the difference below where hosts have fma)
    const double p = rounded, e = fma(a, hi, -p) + a * lo;
    const double pf = p - floor(p), ef = fmod(e, 1.0);  // both exact
    uint64_t t = (uint64_t)ldexp(pf, 64);
    if (ef < 0) t -= (uint64_t)ldexp(-ef, 64);
    else t += (uint64_t)ldexp(ef, 64);
    return rate < 0 ? 0 - t : t;
}
struct RopeTable {
    uint64_t freq[128];  // rope_turns of inv_freq
    uint8_t axis[128];
    int rot_dim, adjacent, n_axes;
    float scale;
};
struct RopeParams {
    const void *q, *k, *v;
    void *q_out, *Kc, *Vc;
    int64_t q_ts, qo_ts, k_ts, v_ts, pos_ts;  // elements between tokens (positions: between axes)
    const int32_t *positions, *table, *cu, *lens;
    uint32_t* err;
    int B, N, H_q, H_kv, D, bs, max_blocks, num_blocks, T_max;
    const void *q_norm, *k_norm;  // [D] weights of the heads' norms, nullptr: not normalised
    float eps;
    float *Ksc, *Vsc;  // 8-bit cache: scales [num_blocks, H_kv] (Kc, Vc: E4M3 codes)
};
int launch_append_rope(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s);
// The queries' half of an 8-bit cache's append of many rows, behind the keys' (see LATE in kvc_rope.cuh).
int launch_late_queries(int dtype, const RopeParams& p, const RopeTable& t, cudaStream_t s);

}  // namespace kvc
