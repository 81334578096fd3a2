// kvc_rope.cuh -- the rows of an append of ragged new tokens with rotary positions: a block of the plain cache's append
// (kvc_rope.cu), and the queries' part of the 8-bit cache's (kvc_append8.cu).
//
// Pair i of a head's first rot_dim dimensions turns by a_i = position * inv_freq[i] ("第 1 周 ·
// Day 4：KV Cache 与 MQA / GQA" §3.2: a new token's position is its place in the sequence):
//     y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a.
// The frequency is kept as a 64-bit fraction of a turn per position, within 2^-62 (rope_turns), so
// position * frequency modulo one turn is one wrapping integer product: exact at any distance, where an
// fp32 product would lose the angle's low bits (2^-24 of 10^5 radians is 0.006).  The top 32 bits give
// the half-turns in [-1, 1) that sincospif takes, rounded to fp32 (error below 2^-24 of a turn).
#pragma once

#include "kvc_ragged.cuh"

namespace kvc {

constexpr int ROPE_THREADS = 256;

// 1 / sqrt(mean x^2 + eps) of a head whose `per` pieces lie in neighbouring lanes: this lane's two vectors x and
// y.  rD = 1 / D (a power of two).  All lanes of the warp come along (shuffles of a part of them, found at run time,
// cost the compiler's search for it: 12,400 rows of 80 heads took 105 to 120 us so).
template <int VEC>
__device__ __forceinline__ float norm_factor(const float (&x)[VEC], const float (&y)[VEC], int per, float rD, float eps) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        s0 = fmaf(x[e], x[e], s0);
        s1 = fmaf(y[e], y[e], s1);
    }
    float sum = s0 + s1;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        if (off < per) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    return rsqrtf(fmaf(sum, rD, eps));
}
// The two vectors times that factor and their weights, 16-byte vectors at wx and wy.
template <typename T>
__device__ __forceinline__ void norm_piece(float (&x)[Elem<T>::VEC], float (&y)[Elem<T>::VEC], const uint4& wx, const uint4& wy,
                                           float inv) {
    float w[Elem<T>::VEC];
    Elem<T>::unpack(wx, w);
#pragma unroll
    for (int e = 0; e < Elem<T>::VEC; ++e) x[e] *= inv * w[e];
    Elem<T>::unpack(wy, w);
#pragma unroll
    for (int e = 0; e < Elem<T>::VEC; ++e) y[e] *= inv * w[e];
}

// The places of packed rows [r0, r0 + n), n at most the block's warps, which find one each: position in the sequence (-1:
// skip the row) and pool row of head 0 (-1: not stored).  Checks cu as well: true, to all threads, if it is bad, else `flag` is
// the error of this warp's row.  Ends with a barrier.
__device__ __forceinline__ bool find_rows(const RopeParams& p, int r0, int n, int64_t* krow, int* slots, uint32_t& flag) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool bad = false;
    flag = 0;  // (speaks of a row only once cu is known to be sound)
    for (int b = tid; b <= p.B; b += ROPE_THREADS) {
        const int c = __ldg(p.cu + b);
        bad |= (b == 0 ? c != 0 : c < __ldg(p.cu + b - 1)) || c > p.N;
    }
    if (warp < n) {
        // the row's sequence: the number of b with cu[b + 1] <= row
        const int row = r0 + warp;
        int b = 0;
        for (int i = 0; i < p.B; i += 32)
            b += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < p.B && __ldg(p.cu + i + lane + 1) <= row));
        if (lane == 0) {
            int slot = -1;
            int64_t kr = -1;
            if (b < p.B && row < p.N) {
                const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), L = __ldg(p.lens + b);
                if (c0 >= 0 && c0 <= row && row < c1 && c1 <= p.N) {  // (else cu does not ascend within 0 .. N)
                    if (L < c1 - c0 || L > p.T_max) {
                        flag = DEV_BAD_LENS;
                    } else {
                        slot = L - (c1 - c0) + (row - c0);
                        const int e = __ldg(p.table + (size_t)b * p.max_blocks + slot / p.bs);
                        if ((unsigned)e >= (unsigned)p.num_blocks) flag = DEV_BAD_BLOCK;
                        else kr = (int64_t)e * p.H_kv * p.bs + slot % p.bs;
                    }
                }
            }
            slots[warp] = slot;
            krow[warp] = kr;
        }
    }
    return __syncthreads_or(bad) != 0;
}
// Cosine and sine of pair j of packed row `row`, at `slot` of its sequence.
__device__ __forceinline__ void row_angle(const RopeParams& p, const RopeTable& rt, int row, int slot, int j, float& c, float& s) {
    const int pos = p.positions ? __ldg(p.positions + (int64_t)rt.axis[j] * p.pos_ts + row) : slot;
    const uint64_t turn = (uint64_t)(int64_t)pos * rt.freq[j];
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    c *= rt.scale;
    s *= rt.scale;
}

// A vector's pairs turned, with the vector of their other halves (halves) or each with its neighbour.
template <int VEC>
__device__ __forceinline__ void turn_piece(float (&x)[VEC], float (&y)[VEC], const float* co, const float* si, bool halves) {
    if (halves) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float f = x[e], g = y[e];
            x[e] = f * co[e] - g * si[e];
            y[e] = g * co[e] + f * si[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float c = co[e], s = si[e], c2 = co[e + VEC / 2], s2 = si[e + VEC / 2];
            const float f = x[2 * e], g = x[2 * e + 1], f2 = y[2 * e], g2 = y[2 * e + 1];
            x[2 * e] = f * c - g * s;
            x[2 * e + 1] = g * c + f * s;
            y[2 * e] = f2 * c2 - g2 * s2;
            y[2 * e + 1] = g2 * c2 + f2 * s2;
        }
    }
}

// A block takes TB consecutive packed rows: one warp each finds the row's sequence and slot, all
// threads compute the rows' cosines and sines once (the heads share them), then the 16-byte
// vectors of all heads are rotated and stored.  VECTOR: every rotated pair lies in whole 16-byte
// vectors (rot_dim a multiple of two vectors); a thread takes two vectors of a head, which hold
// both halves of their pairs.  Otherwise a thread takes one pair (or two unrotated values).
//
// Bound by memory: each value is read and written once, the products are a tenth of the time.
// Bytes in flight decide: 16,000 bf16 rows of 80 heads take 105 us (5.9 TB/s, 0.89 of a copy's
// rate) with two pieces ahead and 4 blocks an SM; 115 us with one piece, 110 with three (fewer
// blocks fit), 131 with 5 blocks of fewer registers.
//
// NORM: the heads of q and k are first divided by the root of their mean square (plus eps) and multiplied by a
// weight per dimension, y = x w / sqrt(mean x^2 + eps), all in fp32: a head's threads are neighbours in a warp and
// add their squares by shuffles.  The same bytes: 12,400 rows of 80 heads take 97 us with norms (5.2 TB/s), which the lanes' issue bounds as much (0.8 of its slots).
//
// LATE: the grid before on the stream is the other half of the same append, which has waited for what came before it and
// shares nothing with this one: it is waited for at the end, not at the start.  (Asked for at run time, 2100 fp32 rows of 24 heads
// took 8.2 us without it, against 7.8.)
template <typename T, int TB, bool VECTOR, bool NORM, bool LATE = false>
__device__ __forceinline__ void append_rows(const RopeParams& p, const RopeTable& rt, int bid) {
    constexpr int VEC = Elem<T>::VEC;
    // Pieces of a thread in flight: read before the rows' slots and angles are known (the rows
    // depend on neither), and from then on two ahead of the stores.
    constexpr int PRE = 2;
    __shared__ __align__(16) float cs[TB][128], sn[TB][128];
    __shared__ int64_t krow[TB];  // pool row of head 0, -1: not stored
    __shared__ int slot_s[TB];    // position of the row in its sequence, -1: skip the row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = rt.rot_dim / 2;
    const int r0 = bid * TB;

    const int heads = (p.q ? p.H_q : 0) + 2 * p.H_kv;
    const int per = VECTOR ? p.D / (2 * VEC) : p.D / 2;  // a thread's pieces of a head
    const int h0 = p.q ? p.H_q : 0;
    const int pieces = heads * per, total = min(TB, p.N - r0) * pieces;
    const int nrot = rt.rot_dim / (2 * VEC);  // (VECTOR) pieces of a head that rotate
    // the two vectors of piece u: of the two halves, or neighbours
    auto vectors = [&](int u, int& v0, int& v1) {
        const bool halves = u < nrot && !rt.adjacent;
        v0 = halves ? u : 2 * u;
        v1 = halves ? u + nrot : 2 * u + 1;
    };
    auto source = [&](int t, int head) {
        const int64_t row = r0 + t;
        if (head < h0) return static_cast<const T*>(p.q) + row * p.q_ts + (int64_t)head * p.D;
        const int h = head - h0;
        return h < p.H_kv ? static_cast<const T*>(p.k) + row * p.k_ts + (int64_t)h * p.D
                          : static_cast<const T*>(p.v) + row * p.v_ts + (int64_t)(h - p.H_kv) * p.D;
    };
    // piece i: row, head and place in the head (a power of two of them make a head of whole vectors)
    const int lg = 31 - __clz(per);
    auto piece = [&](int i, int& t, int& head, int& u) {
        t = 0;
#pragma unroll
        for (int k = 1; k < TB; ++k) t += i >= k * pieces;
        const int w = i - t * pieces;
        head = VECTOR ? w >> lg : w / per;
        u = w - head * per;
    };
    uint4 xa[PRE], xb[PRE];
    auto load = [&](int i, uint4& a, uint4& b) {
        if (i >= total) return;
        int t, head, u, v0, v1;
        piece(i, t, head, u);
        vectors(u, v0, v1);
        const uint4* src = reinterpret_cast<const uint4*>(source(t, head));
        a = src[v0];
        b = src[v1];
    };

    if constexpr (!LATE) asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (VECTOR) {
#pragma unroll
        for (int k = 0; k < PRE; ++k) load(tid + k * ROPE_THREADS, xa[k], xb[k]);
    }
    uint32_t flag;
    if (find_rows(p, r0, TB, krow, slot_s, flag)) {
        if (bid == 0 && tid == 0) atomicOr(p.err, DEV_BAD_SEQ);
        if constexpr (LATE) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (flag) atomicOr(p.err, flag);
    for (int i = tid; i < TB * pairs; i += ROPE_THREADS) {
        const int t = i / pairs, j = i - t * pairs;
        if (slot_s[t] >= 0) row_angle(p, rt, r0 + t, slot_s[t], j, cs[t][j], sn[t][j]);
    }
    __syncthreads();

    // where head `head` of row t goes, null: nowhere
    auto place = [&](int t, int head) -> T* {
        if (slot_s[t] < 0) return nullptr;
        if (head < h0) return static_cast<T*>(p.q_out) + (int64_t)(r0 + t) * p.qo_ts + (int64_t)head * p.D;
        if (krow[t] < 0) return nullptr;
        const int h = head - h0;
        return h < p.H_kv ? static_cast<T*>(p.Kc) + (krow[t] + (int64_t)h * p.bs) * p.D
                          : static_cast<T*>(p.Vc) + (krow[t] + (int64_t)(h - p.H_kv) * p.bs) * p.D;
    };
    if constexpr (VECTOR) {
        // (NORM: a warp's lanes stay together for the norms' sums)
        for (int i0 = tid; (NORM ? i0 - lane : i0) < total; i0 += PRE * ROPE_THREADS) {
#pragma unroll
            for (int k = 0; k < PRE; ++k) {
                const int i = i0 + k * ROPE_THREADS;
                if ((NORM ? i - lane : i) >= total) continue;
                int t, head, u;
                piece(NORM ? min(i, total - 1) : i, t, head, u);
                T* dst = place(t, head);
                uint4 a = xa[k], b = xb[k];
                load(i + PRE * ROPE_THREADS, xa[k], xb[k]);
                if (!NORM && !dst) continue;
                int v0, v1;
                vectors(u, v0, v1);
                if constexpr (NORM) {
                    const bool rot = head < h0 + p.H_kv && u < nrot;
                    const void* weight = head < h0 ? p.q_norm : head < h0 + p.H_kv ? p.k_norm : nullptr;
                    float x[VEC], y[VEC];
                    Elem<T>::unpack(a, x);
                    Elem<T>::unpack(b, y);
                    const float inv = norm_factor<VEC>(x, y, per, 1.f / (float)p.D, p.eps);
                    if (!dst || i >= total) continue;
                    if (rot || weight) {
                        if (weight)
                            norm_piece<T>(x, y, __ldg(static_cast<const uint4*>(weight) + v0),
                                          __ldg(static_cast<const uint4*>(weight) + v1), inv);
                        if (rot) {
                            float co[VEC], si[VEC];
#pragma unroll
                            for (int e = 0; e < VEC; e += 4) {
                                *reinterpret_cast<float4*>(co + e) = *reinterpret_cast<const float4*>(&cs[t][u * VEC + e]);
                                *reinterpret_cast<float4*>(si + e) = *reinterpret_cast<const float4*>(&sn[t][u * VEC + e]);
                            }
                            turn_piece<VEC>(x, y, co, si, !rt.adjacent);
                        }
                        a = Elem<T>::pack(x);
                        b = Elem<T>::pack(y);
                    }
                    *(reinterpret_cast<uint4*>(dst) + v0) = a;
                    *(reinterpret_cast<uint4*>(dst) + v1) = b;
                    continue;
                }
                if (head < h0 + p.H_kv && u < nrot) {
                    float x[VEC], y[VEC];
                    Elem<T>::unpack(a, x);
                    Elem<T>::unpack(b, y);
                    float co[VEC], si[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; e += 4) {
                        *reinterpret_cast<float4*>(co + e) = *reinterpret_cast<const float4*>(&cs[t][u * VEC + e]);
                        *reinterpret_cast<float4*>(si + e) = *reinterpret_cast<const float4*>(&sn[t][u * VEC + e]);
                    }
                    if (!rt.adjacent) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float c = co[e], s = si[e];
                            const float f = x[e], g = y[e];
                            x[e] = f * c - g * s;
                            y[e] = g * c + f * s;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC / 2; ++e) {
                            const float c = co[e], s = si[e], c2 = co[e + VEC / 2], s2 = si[e + VEC / 2];
                            const float f = x[2 * e], g = x[2 * e + 1], f2 = y[2 * e], g2 = y[2 * e + 1];
                            x[2 * e] = f * c - g * s;
                            x[2 * e + 1] = g * c + f * s;
                            y[2 * e] = f2 * c2 - g2 * s2;
                            y[2 * e + 1] = g2 * c2 + f2 * s2;
                        }
                    }
                    a = Elem<T>::pack(x);
                    b = Elem<T>::pack(y);
                }
                *(reinterpret_cast<uint4*>(dst) + v0) = a;
                *(reinterpret_cast<uint4*>(dst) + v1) = b;
            }
        }
    } else if constexpr (NORM) {
        // A warp takes a head: all of it is read before any of it is written (q may be rotated in place).
        const int rows = min(TB, p.N - r0);
        for (int w = warp; w < rows * heads; w += ROPE_THREADS / 32) {
            const int t = w / heads, head = w - t * heads;
            T* dst = place(t, head);
            if (!dst) continue;
            const T* src = source(t, head);
            const T* weight = static_cast<const T*>(head < h0 ? p.q_norm : head < h0 + p.H_kv ? p.k_norm : nullptr);
            T a[4], b[4];  // D <= 256: up to four pairs a lane
            float sum = 0.f;
            auto dims = [&](int u, int& d0, int& d1) {
                const bool halves = u < pairs && !rt.adjacent;
                d0 = halves ? u : 2 * u;
                d1 = halves ? u + pairs : 2 * u + 1;
            };
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int u = lane + 32 * k;
                if (u >= per) continue;
                int d0, d1;
                dims(u, d0, d1);
                a[k] = src[d0];
                b[k] = src[d1];
                sum = fmaf((float)a[k], (float)a[k], fmaf((float)b[k], (float)b[k], sum));
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            const float inv = rsqrtf(sum / (float)p.D + p.eps);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int u = lane + 32 * k;
                if (u >= per) continue;
                int d0, d1;
                dims(u, d0, d1);
                const bool turn = head < h0 + p.H_kv && u < pairs;
                if (!weight && !turn) {
                    dst[d0] = a[k];
                    dst[d1] = b[k];
                    continue;
                }
                float f = (float)a[k], g = (float)b[k];
                if (weight) {
                    f *= inv * (float)weight[d0];
                    g *= inv * (float)weight[d1];
                }
                if (turn) {
                    const float c = cs[t][u], s = sn[t][u], x = f;
                    f = x * c - g * s;
                    g = g * c + x * s;
                }
                Elem<T>::store(dst, d0, f);
                Elem<T>::store(dst, d1, g);
            }
        }
    } else {
        for (int i = tid; i < total; i += ROPE_THREADS) {
            int t, head, u;
            piece(i, t, head, u);
            T* dst = place(t, head);
            if (!dst) continue;
            const T* src = source(t, head);
            const bool turn = u < pairs;
            const int d0 = turn && !rt.adjacent ? u : 2 * u, d1 = turn && !rt.adjacent ? u + pairs : 2 * u + 1;
            const T a = src[d0], b = src[d1];
            if (head < h0 + p.H_kv && turn) {
                const float c = cs[t][u], s = sn[t][u], f = (float)a, g = (float)b;
                Elem<T>::store(dst, d0, f * c - g * s);
                Elem<T>::store(dst, d1, g * c + f * s);
            } else {
                dst[d0] = a;
                dst[d1] = b;
            }
        }
    }
    if constexpr (LATE) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace kvc
