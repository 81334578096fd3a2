// kvc_rope.cu -- append of ragged new tokens to a paged cache with rotary positions.
//
// Pair i of a head's first rot_dim dimensions turns by a_i = position * inv_freq[i] ("第 1 周 ·
// Day 4：KV Cache 与 MQA / GQA" §3.2: a new token's position is its place in the sequence):
//     y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a.
// The frequency is kept as a 64-bit fraction of a turn per position, within 2^-62 (rope_turns), so
// position * frequency modulo one turn is one wrapping integer product: exact at any distance, where an
// fp32 product would lose the angle's low bits (2^-24 of 10^5 radians is 0.006).  The top 32 bits give
// the half-turns in [-1, 1) that sincospif takes, rounded to fp32 (error below 2^-24 of a turn).
#include "kvc_ragged.cuh"

namespace kvc {

constexpr int ROPE_THREADS = 256;

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
template <typename T, int TB, bool VECTOR>
__global__ void __launch_bounds__(ROPE_THREADS, 4) append_rope_kernel(const RopeParams p, const __grid_constant__ RopeTable rt) {
    constexpr int VEC = Elem<T>::VEC;
    // Pieces of a thread in flight: read before the rows' slots and angles are known (the rows
    // depend on neither), and from then on two ahead of the stores.
    constexpr int PRE = 2;
    __shared__ __align__(16) float cs[TB][128], sn[TB][128];
    __shared__ int64_t krow[TB];  // pool row of head 0, -1: not stored
    __shared__ int slot_s[TB];    // position of the row in its sequence, -1: skip the row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = rt.rot_dim / 2;
    const int r0 = blockIdx.x * TB;

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

    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (VECTOR) {
#pragma unroll
        for (int k = 0; k < PRE; ++k) load(tid + k * ROPE_THREADS, xa[k], xb[k]);
    }
    bool bad = false;
    uint32_t flag = 0;  // of this warp's row: set once cu is known to be sound, else it speaks of no row
    for (int b = tid; b <= p.B; b += ROPE_THREADS) {
        const int c = __ldg(p.cu + b);
        bad |= (b == 0 ? c != 0 : c < __ldg(p.cu + b - 1)) || c > p.N;
    }
    if (warp < TB) {
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
            slot_s[warp] = slot;
            krow[warp] = kr;
        }
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(p.err, DEV_BAD_SEQ);
        return;
    }
    if (flag) atomicOr(p.err, flag);
    for (int i = tid; i < TB * pairs; i += ROPE_THREADS) {
        const int t = i / pairs, j = i - t * pairs;
        if (slot_s[t] < 0) continue;
        const int pos = p.positions ? __ldg(p.positions + (int64_t)rt.axis[j] * p.pos_ts + r0 + t) : slot_s[t];
        const uint64_t turn = (uint64_t)(int64_t)pos * rt.freq[j];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        cs[t][j] = c * rt.scale;
        sn[t][j] = s * rt.scale;
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
        for (int i0 = tid; i0 < total; i0 += PRE * ROPE_THREADS) {
#pragma unroll
            for (int k = 0; k < PRE; ++k) {
                const int i = i0 + k * ROPE_THREADS;
                if (i >= total) continue;
                int t, head, u;
                piece(i, t, head, u);
                T* dst = place(t, head);
                uint4 a = xa[k], b = xb[k];
                load(i + PRE * ROPE_THREADS, xa[k], xb[k]);
                if (!dst) continue;
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
                int v0, v1;
                vectors(u, v0, v1);
                *(reinterpret_cast<uint4*>(dst) + v0) = a;
                *(reinterpret_cast<uint4*>(dst) + v1) = b;
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
}

template <typename T>
static int launch_rope(const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // Rows of a block: 4 when that still gives each SM two blocks (the angles' work and the search
    // are shared: 2100 fp32 rows of 24 heads 13.0 us against 15.8 with 1), else 1 (more blocks for
    // a few rows).
    const bool many = p.N >= 8 * sms;
    const int tb = many ? 4 : 1;
    cfg.gridDim = dim3(((unsigned)p.N + tb - 1) / tb);
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool vec = t.rot_dim % (2 * Elem<T>::VEC) == 0 && p.D % (2 * Elem<T>::VEC) == 0;
    const cudaError_t e = many ? (vec ? cudaLaunchKernelEx(&cfg, append_rope_kernel<T, 4, true>, p, t)
                                      : cudaLaunchKernelEx(&cfg, append_rope_kernel<T, 4, false>, p, t))
                               : (vec ? cudaLaunchKernelEx(&cfg, append_rope_kernel<T, 1, true>, p, t)
                                      : cudaLaunchKernelEx(&cfg, append_rope_kernel<T, 1, false>, p, t));
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

int launch_append_rope(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s) {
    return dtype == 0 ? launch_rope<__nv_bfloat16>(p, t, sms, s) : launch_rope<float>(p, t, sms, s);
}

}  // namespace kvc
