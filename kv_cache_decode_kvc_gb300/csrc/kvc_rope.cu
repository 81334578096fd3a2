// kvc_rope.cu -- append of ragged new tokens to a paged cache with rotary positions.
//
// Pair i of a head's first rot_dim dimensions turns by a_i = position * inv_freq[i] ("第 1 周 ·
// Day 4：KV Cache 与 MQA / GQA" §3.2: a new token's position is its place in the sequence):
//     y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a.
// The frequency is kept as a 64-bit fraction of a turn per position, so position * frequency
// modulo one turn is one wrapping integer product: exact at any distance, where an fp32 product
// would lose the angle's low bits (2^-24 of 10^5 radians is 0.006).  The top 32 bits give the
// half-turns in [-1, 1) that sincospif takes (error below 2^-24 of a turn).
#include "kvc_ragged.cuh"

namespace kvc {

constexpr int ROPE_THREADS = 256;

// A block takes TB consecutive packed rows: one warp each finds the row's sequence and slot, all
// threads compute the rows' cosines and sines once (the heads share them), then the 16-byte
// vectors of all heads are rotated and stored.  VECTOR: every rotated pair lies in whole 16-byte
// vectors (rot_dim a multiple of two vectors); a thread takes two vectors of a head, which hold
// both halves of their pairs.  Otherwise a thread takes one pair (or two unrotated values).
template <typename T, int TB, bool VECTOR>
__global__ void __launch_bounds__(ROPE_THREADS) append_rope_kernel(const RopeParams p, const __grid_constant__ RopeTable rt) {
    constexpr int VEC = Elem<T>::VEC;
    __shared__ float cs[TB][128], sn[TB][128];
    __shared__ int64_t krow[TB];  // pool row of head 0, -1: not stored
    __shared__ int slot_s[TB];    // position of the row in its sequence, -1: skip the row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pairs = rt.rot_dim / 2;
    const int r0 = blockIdx.x * TB;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool bad = false;
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
                if (c0 <= row) {  // (else cu does not ascend)
                    if (L < c1 - c0 || L > p.T_max) {
                        atomicOr(p.err, DEV_BAD_LENS);
                    } else {
                        slot = L - (c1 - c0) + (row - c0);
                        const int e = __ldg(p.table + (size_t)b * p.max_blocks + slot / p.bs);
                        if ((unsigned)e >= (unsigned)p.num_blocks) atomicOr(p.err, DEV_BAD_BLOCK);
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

    const int heads = (p.q ? p.H_q : 0) + 2 * p.H_kv;
    const int per = VECTOR ? p.D / (2 * VEC) : p.D / 2;  // a thread's pieces of a head
    const int h0 = p.q ? p.H_q : 0;
    for (int i = tid; i < TB * heads * per; i += ROPE_THREADS) {
        const int t = i / (heads * per), w = i - t * heads * per;
        const int head = w / per, u = w - head * per;
        if (slot_s[t] < 0) continue;
        const int64_t row = r0 + t;
        const T* src;
        T* dst;
        const bool rotate = head < h0 + p.H_kv;
        if (head < h0) {
            src = static_cast<const T*>(p.q) + row * p.q_ts + (int64_t)head * p.D;
            dst = static_cast<T*>(p.q_out) + row * p.qo_ts + (int64_t)head * p.D;
        } else {
            const int h = (head - h0) % p.H_kv;
            if (krow[t] < 0) continue;
            src = rotate ? static_cast<const T*>(p.k) + row * p.k_ts : static_cast<const T*>(p.v) + row * p.v_ts;
            src += (int64_t)h * p.D;
            dst = static_cast<T*>(rotate ? p.Kc : p.Vc) + (krow[t] + (int64_t)h * p.bs) * p.D;
        }
        if constexpr (VECTOR) {
            const int nrot = rt.rot_dim / (2 * VEC);  // pieces that rotate
            const bool turn = u < nrot;
            // the two vectors of piece u: of the two halves, or neighbours
            const int v0 = turn && !rt.adjacent ? u : 2 * u, v1 = turn && !rt.adjacent ? u + nrot : 2 * u + 1;
            uint4 a = *(reinterpret_cast<const uint4*>(src) + v0), b = *(reinterpret_cast<const uint4*>(src) + v1);
            if (rotate && turn) {
                float x[VEC], y[VEC];
                Elem<T>::unpack(a, x);
                Elem<T>::unpack(b, y);
                if (!rt.adjacent) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float c = cs[t][u * VEC + e], s = sn[t][u * VEC + e];
                        const float f = x[e], g = y[e];
                        x[e] = f * c - g * s;
                        y[e] = g * c + f * s;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const int j = u * VEC + e;
                        const float c = cs[t][j], s = sn[t][j];
                        const float c2 = cs[t][j + VEC / 2], s2 = sn[t][j + VEC / 2];
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
        } else {
            const bool turn = u < pairs;
            const int d0 = turn && !rt.adjacent ? u : 2 * u, d1 = turn && !rt.adjacent ? u + pairs : 2 * u + 1;
            const T a = src[d0], b = src[d1];
            if (rotate && turn) {
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
    const bool many = p.N >= 16 * sms;
    const int tb = many ? 4 : 1;
    cfg.gridDim = dim3((unsigned)((p.N + tb - 1) / tb));
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
