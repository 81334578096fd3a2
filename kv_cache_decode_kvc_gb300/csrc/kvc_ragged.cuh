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
//     sequences has streams over [P, L_b) as any sequence has over [0, L_b);
//   - all streams are laid end to end, each costing its tiles and C0 more for its start, and CTA
//     i of P takes the cost units [i U / P, (i + 1) U / P): equal work whatever the lengths, no
//     CTA waits for another, the same split on every run (results are reproducible).
// Everything is computed on the device from cu_seqlens, lens and the groups.
//
// A stream that one CTA holds whole and that no other stream shares rows with is written to out.
// Otherwise its pieces go to scratch and combine_ragged_kernel merges them: the first piece of a
// stream of a sequence with a shared prefix to a row buffer (one for prefix streams, one for
// the sequences' own), of other streams to slot 1 of its CTA; later pieces, which open their
// CTA's range, to slot 0.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {

constexpr int RAGGED_C0 = 1;         // cost of a stream's start, in tiles
constexpr int RAGGED_MIN_UNITS = 4;  // fewer CTAs when a CTA's share would drop below this
constexpr int RAGGED_SLOT_ROWS = 256;

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
    int64_t* plan;   // [NG + 1] + [B + 1] per-head cost prefix sums, for the merge
    float* row_o;    // [2][N H_q][D] unnormalised outputs of first pieces (groups only)
    float* row_ml;   // [2][N H_q][2] (max in log2 units, denominator)
    float* slot_o;   // [P][2][RAGGED_SLOT_ROWS][D]
    float* slot_ml;  // [P][2][RAGGED_SLOT_ROWS][2]
    int B, N, H_q, H_kv, lgG, NG, D;
    int bs, max_blocks, num_blocks, T_max;
    int P;          // CTAs at most
    int min_units;  // 1: use all P CTAs down to one unit each
    float qscale;   // log2(e) / sqrt(D)
};

// Scratch layout (bytes, 256-byte aligned parts), host side.
struct RaggedScratch {
    uint64_t plan, row_o, row_ml, slot_o, slot_ml, total;
};
inline RaggedScratch ragged_scratch(int B, int N, int NG, int H_q, int D, int P) {
    auto up = [](uint64_t x) { return (x + 255) / 256 * 256; };
    RaggedScratch s;
    uint64_t at = 0;
    s.plan = at;
    at += up((uint64_t)(B + NG + 2) * 8);
    const uint64_t rows = NG > 0 ? 2ull * (uint64_t)N * (uint64_t)H_q : 0;
    s.row_o = at;
    at += up(rows * (uint64_t)D * 4);
    s.row_ml = at;
    at += up(rows * 8);
    const uint64_t slots = 2ull * (uint64_t)P * RAGGED_SLOT_ROWS;
    s.slot_o = at;
    at += up(slots * (uint64_t)D * 4);
    s.slot_ml = at;
    at += up(slots * 8);
    s.total = at;
    return s;
}

#ifdef __CUDACC__

// ------------------------------------------------------------------ sequences and streams
struct SeqInfo {
    int row0, T;  // packed rows [row0, row0 + T)
    int L, pfx;   // positions; shared prefix in effect (whole blocks, 0: none)
    bool ok;      // false: has rows but cannot be attended (its outputs are zero)
};

// Shared prefix of sequence b: in effect (whole blocks; a group of one shares nothing) and as
// given (-1 if out of range).
__device__ __forceinline__ int2 seq_prefix(const RaggedParams& p, int b) {
    if (p.groups == nullptr) return make_int2(0, 0);
    int lo = 0, hi = p.NG - 1;  // largest g with groups[g] <= b
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.groups + mid) <= b) lo = mid; else hi = mid - 1;
    }
    const int P = __ldg(p.prefix + lo);
    if (P < 0 || P > p.T_max) return make_int2(0, -1);
    const bool one = __ldg(p.groups + lo + 1) - __ldg(p.groups + lo) < 2;
    return make_int2(one ? 0 : P / p.bs * p.bs, P);
}

__device__ __forceinline__ SeqInfo seq_info(const RaggedParams& p, int b) {
    SeqInfo s;
    s.row0 = __ldg(p.cu + b);
    s.T = __ldg(p.cu + b + 1) - s.row0;
    s.L = __ldg(p.lens + b);
    const int2 pf = seq_prefix(p, b);
    s.pfx = pf.x;
    s.ok = s.T > 0 && s.L >= s.T && s.L <= p.T_max && pf.y >= 0 && s.L - s.T >= pf.y;
    return s;
}

// Rows of group g and its prefix in effect (0: no streams).
__device__ __forceinline__ SeqInfo group_info(const RaggedParams& p, int g) {
    const int b0 = __ldg(p.groups + g), b1 = __ldg(p.groups + g + 1);
    SeqInfo s;
    s.row0 = __ldg(p.cu + b0);
    s.T = __ldg(p.cu + b1) - s.row0;
    const int P = __ldg(p.prefix + g);
    s.pfx = (b1 - b0 < 2 || P < 0 || P > p.T_max) ? 0 : P / p.bs * p.bs;
    s.L = s.pfx;
    s.ok = s.T > 0 && s.pfx > 0;
    return s;
}

// sum of ceil(x / R) for x = 1 .. X
__device__ __forceinline__ int64_t ceil_sum(int64_t X, int R) {
    const int64_t n = X / R, r = X - n * R;
    return (int64_t)R * (n * (n + 1) / 2) + r * (n + 1);
}

template <int RT, int KT>
struct Ragged {
    // Key tiles of a stream of a sequence with S0 keys of its own before its new tokens, whose
    // last row is new token t1 - 1: positions [pfx, pfx + S0 + t1).
    __device__ static int tiles(int S0, int t1) { return (int)(((int64_t)S0 + t1 + KT - 1) / KT); }
    // Cost of its first k streams, all full (TQ tokens each):
    // sum over i = 1 .. k of ceil((S0 + i TQ) / KT), and the starts.
    __device__ static int64_t cost_full(int S0, int64_t k, int TQ) {
        if (TQ >= KT) return k * ((S0 + KT - 1) / KT) + (int64_t)(TQ / KT) * (k * (k + 1) / 2) + k * RAGGED_C0;
        const int R = KT / TQ;  // ceil((S0 + i TQ) / KT) = ceil((ceil(S0 / TQ) + i) / R)
        const int64_t s = (S0 + TQ - 1) / TQ;
        return ceil_sum(s + k, R) - ceil_sum(s, R) + k * RAGGED_C0;
    }
    __device__ static int64_t seq_cost(const SeqInfo& s, int TQ) {
        if (!s.ok) return 0;
        const int nk = (s.T + TQ - 1) / TQ, S0 = s.L - s.T - s.pfx;
        return cost_full(S0, nk - 1, TQ) + tiles(S0, s.T) + RAGGED_C0;
    }
    __device__ static int64_t group_cost(const SeqInfo& s, int TQ) {
        if (!s.ok) return 0;
        return (int64_t)((s.T + TQ - 1) / TQ) * ((s.pfx + KT - 1) / KT + RAGGED_C0);
    }

    // A stream: type 0 = a group's prefix, 1 = a sequence's own keys; idx = group or sequence.
    struct Stream {
        int type, idx, h, k;
        SeqInfo s;
        int64_t u0;  // its first cost unit
        int n;       // key tiles
    };
    __device__ static void fill(Stream& st, int TQ) {
        if (st.type == 0) {
            st.n = (st.s.pfx + KT - 1) / KT;
        } else {
            const int t1 = min(st.s.T, (st.k + 1) * TQ);
            st.n = tiles(st.s.L - st.s.T - st.s.pfx, t1);
        }
    }
    // The stream holding cost unit x, from the prefix sums gc[NG + 1], sc[B + 1] (per head).
    __device__ static Stream locate(const RaggedParams& p, const int64_t* gc, const int64_t* sc, int64_t x) {
        const int TQ = RT >> p.lgG;
        Stream st;
        const int64_t W0 = p.NG > 0 ? gc[p.NG] * p.H_kv : 0;
        st.type = x < W0 ? 0 : 1;
        const int64_t* c = st.type == 0 ? gc : sc;
        const int64_t base = st.type == 0 ? 0 : W0;
        int lo = 0, hi = (st.type == 0 ? p.NG : p.B) - 1;  // largest i with H_kv c[i] <= x - base
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (c[mid] * p.H_kv <= x - base) lo = mid; else hi = mid - 1;
        }
        st.idx = lo;
        const int64_t per = c[lo + 1] - c[lo];
        int64_t r = x - base - c[lo] * p.H_kv;
        st.h = (int)(r / per);
        r -= st.h * per;
        st.u0 = base + c[lo] * p.H_kv + st.h * per;
        st.s = st.type == 0 ? group_info(p, lo) : seq_info(p, lo);
        const int nk = (st.s.T + TQ - 1) / TQ;
        if (st.type == 0) {
            const int64_t one = (st.s.pfx + KT - 1) / KT + RAGGED_C0;
            st.k = (int)(r / one);
            st.u0 += st.k * one;
        } else {
            const int S0 = st.s.L - st.s.T - st.s.pfx;
            int a = 0, b = nk - 1;
            while (a < b) {  // largest k with cost_full(k) <= r
                const int mid = (a + b + 1) >> 1;
                if (cost_full(S0, mid, TQ) <= r) a = mid; else b = mid - 1;
            }
            st.k = a;
            st.u0 += cost_full(S0, a, TQ);
        }
        fill(st, TQ);
        return st;
    }
    // The stream of packed row `row` (a token of sequence idx, type 1, or of group idx, type 0).
    __device__ static Stream of_row(const RaggedParams& p, const int64_t* gc, const int64_t* sc, int type, int idx,
                                    int h, int row) {
        const int TQ = RT >> p.lgG;
        Stream st;
        st.type = type;
        st.idx = idx;
        st.h = h;
        st.s = type == 0 ? group_info(p, idx) : seq_info(p, idx);
        st.k = (row - st.s.row0) / TQ;
        const int64_t* c = type == 0 ? gc : sc;
        st.u0 = (type == 0 || p.NG == 0 ? 0 : gc[p.NG] * p.H_kv) + c[idx] * p.H_kv + h * (c[idx + 1] - c[idx]);
        if (type == 0)
            st.u0 += st.k * (int64_t)((st.s.pfx + KT - 1) / KT + RAGGED_C0);
        else
            st.u0 += cost_full(st.s.L - st.s.T - st.s.pfx, st.k, TQ);
        fill(st, TQ);
        return st;
    }
    // The next stream with keys after st; false if there is none.
    __device__ static bool next(const RaggedParams& p, Stream& st) {
        const int TQ = RT >> p.lgG;
        st.u0 += st.n + RAGGED_C0;
        if ((int64_t)(st.k + 1) * TQ < st.s.T) {
            ++st.k;
        } else {
            st.k = 0;
            if (++st.h == p.H_kv) {
                st.h = 0;
                while (true) {
                    if (++st.idx == (st.type == 0 ? p.NG : p.B)) {
                        if (st.type == 1) return false;
                        st.type = 1;
                        st.idx = 0;
                    }
                    st.s = st.type == 0 ? group_info(p, st.idx) : seq_info(p, st.idx);
                    if (st.s.ok) break;
                }
            }
        }
        fill(st, TQ);
        return true;
    }

    // A CTA's piece of a stream.
    struct Seg {
        int n;           // key tiles (0: no more segments)
        int seq, h;      // table row, KV head
        int row0, ntok;  // packed rows of the tile
        int kv0;         // position of its first key tile
        int kv_end;      // positions [kv0, kv_end) exist for the stream
        int lim0, causal;  // row of token i sees positions below min(kv_end, lim0 + i * causal)
        int dst;         // 0 out, 1 / 2 row buffer 0 / 1, 3 / 4 slot 0 / 1 of the CTA
    };
    // The part [x, x1) of stream st as a segment (n = 0 if it holds no tile).
    __device__ static Seg segment(const RaggedParams& p, const Stream& st, int64_t x, int64_t x1) {
        const int TQ = RT >> p.lgG;
        Seg g;
        const int64_t a = x - st.u0 - RAGGED_C0, b = x1 - st.u0 - RAGGED_C0;
        const int j0 = a < 0 ? 0 : (int)a, j1 = b < 0 ? 0 : (b > st.n ? st.n : (int)b);
        g.n = j1 - j0;
        g.seq = st.type == 0 ? __ldg(p.groups + st.idx) : st.idx;
        g.h = st.h;
        g.row0 = st.s.row0 + st.k * TQ;
        g.ntok = min(TQ, st.s.T - st.k * TQ);
        const int first = st.type == 0 ? 0 : st.s.pfx;
        g.kv0 = first + j0 * KT;
        if (st.type == 0) {
            g.kv_end = st.s.pfx;
            g.lim0 = st.s.pfx;
            g.causal = 0;
        } else {
            const int S = st.s.L - st.s.T + st.k * TQ;  // position of the tile's first token
            g.kv_end = S + g.ntok;
            g.lim0 = S + 1;
            g.causal = 1;
        }
        const bool joint = st.s.pfx > 0;  // (a prefix stream always is)
        if (j0 > 0) g.dst = 3;
        else if (joint) g.dst = 1 + st.type;
        else g.dst = j1 == st.n ? 0 : 4;
        return g;
    }
};

__device__ __forceinline__ int64_t ragged_ctas(int64_t U, int P, int min_units) {
    const int64_t want = (U + min_units - 1) / min_units;
    return want < P ? want : P;
}

// cu and groups ascend within their bounds?  Every thread of the block takes part.
__device__ __forceinline__ bool ragged_valid(const RaggedParams& p, int tid, int nthreads) {
    bool bad = false;
    for (int b = tid; b <= p.B; b += nthreads) {
        const int c = __ldg(p.cu + b);
        bad |= b == 0 ? c != 0 : c < __ldg(p.cu + b - 1);
        bad |= c > p.N;
    }
    for (int g = tid; g <= p.NG && p.NG > 0; g += nthreads) {
        const int c = __ldg(p.groups + g);
        bad |= g == 0 ? c != 0 : c < __ldg(p.groups + g - 1);
        bad |= g == p.NG ? c != p.B : c > p.B;
    }
    return __syncthreads_or(bad) == 0;
}

// Per-head cost prefix sums gc[NG + 1], sc[B + 1] in shared memory (every thread of the block;
// tmp: 32 int64).  Returns the total cost U.
template <int RT, int KT>
__device__ __forceinline__ int64_t ragged_scan(const RaggedParams& p, int64_t* gc, int64_t* sc, int64_t* tmp, int tid,
                                               int nthreads) {
    using R = Ragged<RT, KT>;
    const int TQ = RT >> p.lgG, lane = tid & 31, warp = tid >> 5, nw = nthreads >> 5;
    int64_t total[2] = {0, 0};
#pragma unroll 1
    for (int ty = 0; ty < 2; ++ty) {
        const int n = ty == 0 ? p.NG : p.B;
        int64_t* c = ty == 0 ? gc : sc;
        int64_t carry = 0;
        if (tid == 0) c[0] = 0;
        for (int i0 = 0; i0 < n; i0 += nthreads) {
            const int i = i0 + tid;
            int64_t v = 0;
            if (i < n) v = ty == 0 ? R::group_cost(group_info(p, i), TQ) : R::seq_cost(seq_info(p, i), TQ);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
                if (lane >= o) v += t;
            }
            if (lane == 31) tmp[warp] = v;
            __syncthreads();
            int64_t before = carry, all = carry;
            for (int w = 0; w < nw; ++w) {
                if (w < warp) before += tmp[w];
                all += tmp[w];
            }
            if (i < n) c[i + 1] = before + v;
            carry = all;
            __syncthreads();
        }
        total[ty] = carry;
    }
    return (total[0] + total[1]) * p.H_kv;
}

// Zero output rows of the sequences that cannot be attended (CTA-strided over sequences).
template <typename T>
__device__ __forceinline__ void ragged_zero_rows(const RaggedParams& p, int tid, int nthreads) {
    const int vecs = p.H_q * p.D * Elem<T>::BYTES / 16;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const SeqInfo s = seq_info(p, b);
        if (s.T <= 0 || s.ok) continue;
        if (tid == 0) atomicOr(p.err, DEV_BAD_LENS);
        for (int64_t i = tid; i < (int64_t)s.T * vecs; i += nthreads) {
            const int64_t r = i / vecs;
            char* row = static_cast<char*>(p.out) + (s.row0 + r) * p.out_ts * Elem<T>::BYTES;
            reinterpret_cast<uint4*>(row)[i - r * vecs] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Where the state of packed row `row`, head j (query-row r of its tile) of a segment with dst > 0
// goes.
template <typename S>
__device__ __forceinline__ void ragged_dst(const RaggedParams& p, const S& g, int cta, int r, int64_t row, int j,
                                           float*& o, float*& ml) {
    if (g.dst <= 2) {
        const int64_t at = ((int64_t)(g.dst - 1) * p.N + row) * p.H_q + j;
        o = p.row_o + at * p.D;
        ml = p.row_ml + at * 2;
    } else {
        const int64_t at = ((int64_t)cta * 2 + (g.dst - 3)) * RAGGED_SLOT_ROWS + r;
        o = p.slot_o + at * p.D;
        ml = p.slot_ml + at * 2;
    }
}

#endif  // __CUDACC__

// Launchers (kvc_ragged.cu, kvc_ragged_tc5.cu, kvc_rope.cu); each returns a cudaError_t.
int launch_ragged_cc(int dtype, const RaggedParams& p, cudaStream_t s);
// bf16, D = 64 or 128; q: make_q_tensor_map, k / v: the pool's maps with min(bs, 128)-row boxes.
int launch_ragged_tc5(const RaggedParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                      cudaStream_t s);
struct RopeTable {
    uint64_t freq[128];  // inv_freq in 2^-64 turns per position
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
};
int launch_append_rope(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s);

}  // namespace kvc
