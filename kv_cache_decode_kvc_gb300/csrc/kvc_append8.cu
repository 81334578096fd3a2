// kvc_append8.cu -- the paged cache held in 8 bits (kvc_q8.cuh): append of ragged new tokens with norms and
// rotary positions, reading positions back, widening of whole blocks.
#include <type_traits>

#include "kvc_q8.cuh"
#include "kvc_rope.cuh"

namespace kvc {

// Two finite values, or any, as codes: infinite and NaN values are stored as NaN (E4M3 has no infinity).
__device__ __forceinline__ uint32_t q8_codes2(float x, float y, float mul, float lim) {
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const float a = isfinite(x) ? fminf(fmaxf(x * mul, -lim), lim) : nan;
    const float b = isfinite(y) ? fminf(fmaxf(y * mul, -lim), lim) : nan;
    return e4m3x2(a, b);
}
// Four codes scaled by a power of two.
__device__ __forceinline__ uint32_t q8_rescale4(uint32_t c, float mul) {
    const float2 a = e4m3x2_value(c), b = e4m3x2_value(c >> 16);
    return e4m3x2(a.x * mul, a.y * mul) | e4m3x2(b.x * mul, b.y * mul) << 16;
}

// The new rows of one block and some of its heads, K and V: a CTA's share of the keys' and values' append.
// Sequence b's blocks are items cu[b] / bs + 2 b, .. (floor(T / bs) + 2 places hold the blocks that T rows
// touch), so no sum over the sequences is needed.  The rows' pieces (two 16-byte vectors, as in append_rows)
// are all read at once, up to Q8_HELD of a thread; the first pass finds each head's largest |x| of
// K, normalised and rotated, and of V; then the scales are settled, and the second pass, from the same
// registers, stores the codes.  A block that holds earlier rows and needs a larger scale has their codes
// moved down.
constexpr int Q8_HELD = 8;

template <typename T, bool NORM>
__device__ __forceinline__ void append8_block(const RopeParams& p, const RopeTable& rt, int item, int h_first, int nh,
                                              bool table_fits, float2* trig) {
    constexpr int VEC = Elem<T>::VEC, NT = ROPE_THREADS;
    __shared__ int found;
    __shared__ uint32_t amax[32];
    __shared__ float mul_s[32], lim_s[32], down_s[32];
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) found = 0;
    if (tid < 32) amax[tid] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    bool bad = false;
    int cnt = 0;
    for (int b = tid; b <= p.B; b += NT) {
        const int c = __ldg(p.cu + b);
        bad |= (b == 0 ? c != 0 : c < __ldg(p.cu + b - 1)) || c > p.N;
        cnt += b < p.B && c / p.bs + 2 * b <= item;
    }
    if (cnt) atomicAdd(&found, cnt);
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(p.err, DEV_BAD_SEQ);
        return;
    }
    const int b = found - 1;
    const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), L = __ldg(p.lens + b), n = c1 - c0;
    const int j = item - (c0 / p.bs + 2 * b);
    if (n == 0) return;
    if (L < n || L > p.T_max) {
        if (tid == 0 && j == 0) atomicOr(p.err, DEV_BAD_LENS);
        return;
    }
    const int H = L - n, k = H / p.bs + j;
    if (k > (L - 1) / p.bs) return;
    const int start = k * p.bs, lo = max(H, start), nrow = min(L - start, p.bs) - (lo - start), held = max(0, H - start);
    const int64_t r0 = c0 + (lo - H);
    const int e = __ldg(p.table + (size_t)b * p.max_blocks + k);
    if ((unsigned)e >= (unsigned)p.num_blocks) {
        if (tid == 0) atomicOr(p.err, DEV_BAD_BLOCK);
        return;
    }
    const int per = p.D / (2 * VEC), lg = 31 - __clz(per);
    const int half = nrow * per, total = 2 * nh * half;  // a head's K pieces, and its V pieces
    const int pairs = rt.rot_dim / 2, nrot = rt.rot_dim / (2 * VEC);
    auto piece = [&](int i, int& hk, int& row, int& u) {
        const int g = i >> lg;
        u = i & (per - 1);
        hk = g / nrow;
        row = g - hk * nrow;
    };
    auto vectors = [&](int hk, int u, int& v0, int& v1) {
        const bool halves = !(hk & 1) && u < nrot && !rt.adjacent;
        v0 = halves ? u : 2 * u;
        v1 = halves ? u + nrot : 2 * u + 1;
    };
    auto load = [&](int i, uint4& a, uint4& bb) {
        int hk, row, u, v0, v1;
        piece(i, hk, row, u);
        vectors(hk, u, v0, v1);
        const int h = h_first + (hk >> 1);
        const T* src = hk & 1 ? static_cast<const T*>(p.v) + (r0 + row) * p.v_ts + (int64_t)h * p.D
                              : static_cast<const T*>(p.k) + (r0 + row) * p.k_ts + (int64_t)h * p.D;
        a = __ldg(reinterpret_cast<const uint4*>(src) + v0);
        bb = __ldg(reinterpret_cast<const uint4*>(src) + v1);
    };
    uint4 xa[Q8_HELD], xb[Q8_HELD];
#pragma unroll
    for (int q = 0; q < Q8_HELD; ++q)
        if (tid + q * NT < total) load(tid + q * NT, xa[q], xb[q]);
    auto angle = [&](int row, int pr) {
        const int pos = p.positions ? __ldg(p.positions + (int64_t)rt.axis[pr] * p.pos_ts + r0 + row) : lo + row;
        const uint64_t turn = (uint64_t)(int64_t)pos * rt.freq[pr];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        return make_float2(c * rt.scale, s * rt.scale);
    };
    if (table_fits)
        for (int i = tid; i < nrow * pairs; i += NT) {
            const int row = i / pairs;
            trig[i] = angle(row, i - row * pairs);
        }
    __syncthreads();
    // the values that piece i stands for, in fp32
    auto values = [&](int i, const uint4& a, const uint4& bb, float (&x)[VEC], float (&y)[VEC], int& hk, int& row, int& v0,
                      int& v1) {
        int u;
        piece(i, hk, row, u);
        vectors(hk, u, v0, v1);
        Elem<T>::unpack(a, x);
        Elem<T>::unpack(bb, y);
        if (hk & 1) return;
        if (NORM && p.k_norm) norm_piece<T>(x, y, p.k_norm, v0, v1, per, p.D, p.eps);
        if (u >= nrot) return;
        const float2* tr = trig + row * pairs + u * VEC;
        auto at = [&](int q) { return table_fits ? tr[q] : angle(row, u * VEC + q); };
        if (!rt.adjacent) {
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float2 t = at(q);
                const float f = x[q], g = y[q];
                x[q] = f * t.x - g * t.y;
                y[q] = g * t.x + f * t.y;
            }
        } else {
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) {
                const float2 t = at(q), t2 = at(q + VEC / 2);
                const float f = x[2 * q], g = x[2 * q + 1], f2 = y[2 * q], g2 = y[2 * q + 1];
                x[2 * q] = f * t.x - g * t.y;
                x[2 * q + 1] = g * t.x + f * t.y;
                y[2 * q] = f2 * t2.x - g2 * t2.y;
                y[2 * q + 1] = g2 * t2.x + f2 * t2.y;
            }
        }
    };
    auto largest = [&](int i, const uint4& a, const uint4& bb) {
        float x[VEC], y[VEC];
        int hk, row, v0, v1;
        values(i, a, bb, x, y, hk, row, v0, v1);
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            const uint32_t f = __float_as_uint(x[q]) & 0x7FFFFFFFu, g = __float_as_uint(y[q]) & 0x7FFFFFFFu;
            if (f < 0x7F800000u) m = max(m, f);
            if (g < 0x7F800000u) m = max(m, g);
        }
        const uint32_t mask = (per == 32 ? 0xFFFFFFFFu : (1u << per) - 1u) << (lane & ~(per - 1));
        for (int off = per >> 1; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(mask, m, off));
        if ((lane & (per - 1)) == 0) atomicMax(&amax[hk], m);
    };
#pragma unroll
    for (int q = 0; q < Q8_HELD; ++q)
        if (tid + q * NT < total) largest(tid + q * NT, xa[q], xb[q]);
    for (int i = tid + Q8_HELD * NT; i < total; i += NT) {
        uint4 a, bb;
        load(i, a, bb);
        largest(i, a, bb);
    }
    __syncthreads();
    if (tid < 2 * nh) {
        float* sc = (tid & 1 ? p.Vsc : p.Ksc) + (int64_t)e * p.H_kv + h_first + (tid >> 1);
        int x = q8_exponent(amax[tid]);
        float down = 1.f;
        if (held > 0) {
            const int old = q8_stored(__float_as_uint(*sc));
            if (old >= x) x = old;
            else down = exp2i(max(old - x, -60));
        }
        *sc = exp2i(x);
        mul_s[tid] = exp2i(-x);
        lim_s[tid] = x == Q8_EMAX ? 240.f : 448.f;  // (256 2^120 is past the largest float)
        down_s[tid] = down;
    }
    __syncthreads();
    auto codes_of = [&](int hk) {
        char* pool = static_cast<char*>(hk & 1 ? p.Vc : p.Kc);
        return pool + (((int64_t)e * p.H_kv + h_first + (hk >> 1)) * p.bs) * p.D;
    };
    auto store = [&](int i, const uint4& a, const uint4& bb) {
        float x[VEC], y[VEC];
        int hk, row, v0, v1;
        values(i, a, bb, x, y, hk, row, v0, v1);
        const float mul = mul_s[hk], lim = lim_s[hk];
        char* dst = codes_of(hk) + (lo - start + row) * p.D;
        uint32_t w[VEC / 4], z[VEC / 4];
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
            w[q] = q8_codes2(x[4 * q], x[4 * q + 1], mul, lim) | q8_codes2(x[4 * q + 2], x[4 * q + 3], mul, lim) << 16;
            z[q] = q8_codes2(y[4 * q], y[4 * q + 1], mul, lim) | q8_codes2(y[4 * q + 2], y[4 * q + 3], mul, lim) << 16;
        }
        if constexpr (VEC == 8) {
            *reinterpret_cast<uint2*>(dst + v0 * VEC) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(dst + v1 * VEC) = make_uint2(z[0], z[1]);
        } else {
            *reinterpret_cast<uint32_t*>(dst + v0 * VEC) = w[0];
            *reinterpret_cast<uint32_t*>(dst + v1 * VEC) = z[0];
        }
    };
#pragma unroll
    for (int q = 0; q < Q8_HELD; ++q)
        if (tid + q * NT < total) store(tid + q * NT, xa[q], xb[q]);
    for (int i = tid + Q8_HELD * NT; i < total; i += NT) {
        uint4 a, bb;
        load(i, a, bb);
        store(i, a, bb);
    }
    if (held > 0)
        for (int hk = 0; hk < 2 * nh; ++hk) {
            const float down = down_s[hk];
            if (down == 1.f) continue;
            uint4* c = reinterpret_cast<uint4*>(codes_of(hk));
            for (int i = tid; i < held * (p.D / 16); i += NT) {
                const uint4 w = c[i];
                c[i] = make_uint4(q8_rescale4(w.x, down), q8_rescale4(w.y, down), q8_rescale4(w.z, down),
                                  q8_rescale4(w.w, down));
            }
        }
}

// Blocks [0, nkv) append keys and values (nkv / groups items, heads in groups of hg), the others rotate the
// queries, TB rows each.
struct Append8Grid {
    int nkv, groups, hg, table_fits;
};
template <typename T, int TB, bool NORM>
__global__ void __launch_bounds__(ROPE_THREADS, 2)
append8_kernel(const RopeParams p, const __grid_constant__ RopeTable rt, const Append8Grid g) {
    extern __shared__ __align__(16) float2 trig8[];
    if (blockIdx.x < g.nkv) {
        const int item = blockIdx.x / g.groups, h = (blockIdx.x - item * g.groups) * g.hg;
        append8_block<T, NORM>(p, rt, item, h, min(g.hg, p.H_kv - h), g.table_fits != 0, trig8);
    } else {
        RopeParams q = p;  // the queries alone
        q.H_kv = 0;
        append_rows<T, TB, true, NORM>(q, rt, blockIdx.x - g.nkv);
    }
}

template <typename T, int TB, bool NORM>
static int launch_append8_as(const RopeParams& p, const RopeTable& t, cudaStream_t s) {
    constexpr int VEC = Elem<T>::VEC, TABLE = 64 << 10;
    Append8Grid g;
    const int per_head = 2 * p.bs * (p.D / (2 * VEC));
    g.hg = Q8_HELD * ROPE_THREADS / per_head;
    g.hg = g.hg < 1 ? 1 : g.hg > 16 ? 16 : g.hg;
    if (g.hg > p.H_kv) g.hg = p.H_kv;
    g.groups = (p.H_kv + g.hg - 1) / g.hg;
    const int64_t items = p.N / p.bs + 2 * (int64_t)p.B, nkv = items * g.groups;
    const int64_t nq = p.q ? ((int64_t)p.N + TB - 1) / TB : 0;
    if (nkv + nq > 0x7FFFFFFF) return (int)cudaErrorInvalidValue;
    g.nkv = (int)nkv;
    const int table = p.bs * (t.rot_dim / 2) * (int)sizeof(float2);
    g.table_fits = table <= TABLE;
    static PerDeviceOnce once;
    const int e0 = once.run([] {
        return (int)cudaFuncSetAttribute(append8_kernel<T, TB, NORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, TABLE);
    });
    if (e0 != 0) return e0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(nkv + nq));
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.dynamicSmemBytes = g.table_fits ? table : 0;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, append8_kernel<T, TB, NORM>, p, t, g);
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}
int launch_append8(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s) {
    const bool norm = p.q_norm || p.k_norm, many = p.N >= 8 * sms;  // (as in kvc_rope.cu)
    auto go = [&](auto tp) {
        using T = decltype(tp);
        return many ? (norm ? launch_append8_as<T, 4, true>(p, t, s) : launch_append8_as<T, 4, false>(p, t, s))
                    : (norm ? launch_append8_as<T, 1, true>(p, t, s) : launch_append8_as<T, 1, false>(p, t, s));
    };
    return dtype == 0 ? go(__nv_bfloat16()) : go(float());
}

// ------------------------------------------------------------------ reading back
// 16 codes -> 16 values of the cache's dtype (exact in both but for values a float does not hold).
template <typename T>
__device__ __forceinline__ void q8_widen16(const uint4& c, float scale, uint4 (&out)[16 / Elem<T>::VEC]) {
    constexpr int VEC = Elem<T>::VEC;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = e4m3x2_value(w[i >> 1] >> (16 * (i & 1)));
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
#pragma unroll
    for (int i = 0; i < 16 / VEC; ++i) {
        float x[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) x[q] = f[i * VEC + q];
        out[i] = Elem<T>::pack(x);
    }
}

// Positions of the sequences as packed rows: a block takes READ_ROWS consecutive rows, a warp each finds
// the row's place, then all threads copy its heads.  Bound by memory: every code is read, every value
// written once.
constexpr int READ_THREADS = 256, READ_ROWS = 4;
template <typename T, bool Q8>
__global__ void __launch_bounds__(READ_THREADS) paged_read_kernel(const Q8Read p) {
    constexpr int VEC = Elem<T>::VEC, PIECE = Q8 ? 16 : VEC;
    __shared__ int block_s[READ_ROWS], off_s[READ_ROWS];  // block: -1 zeros, -2 not a row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r0 = blockIdx.x * READ_ROWS;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool bad = false;
    uint32_t flag = 0;
    for (int b = tid; b <= p.B; b += READ_THREADS) {
        const int c = __ldg(p.cu + b);
        bad |= (b == 0 ? c != 0 : c < __ldg(p.cu + b - 1)) || c > p.N;
    }
    if (warp < READ_ROWS) {
        const int row = r0 + warp;
        int b = 0;
        for (int i = 0; i < p.B; i += 32)
            b += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < p.B && __ldg(p.cu + i + lane + 1) <= row));
        if (lane == 0) {
            int block = -2, off = 0;
            if (b < p.B && row < p.N) {
                const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), L = __ldg(p.lens + b);
                if (c0 >= 0 && c0 <= row && row < c1 && c1 <= p.N) {
                    block = -1;
                    if (L < c1 - c0 || L > p.T_max) {
                        flag = DEV_BAD_LENS;
                    } else {
                        const int slot = L - (c1 - c0) + (row - c0);
                        const int e = __ldg(p.table + (size_t)b * p.max_blocks + slot / p.bs);
                        if ((unsigned)e >= (unsigned)p.num_blocks) flag = DEV_BAD_BLOCK;
                        else block = e;
                        off = slot % p.bs;
                    }
                }
            }
            block_s[warp] = block;
            off_s[warp] = off;
        }
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(p.err, DEV_BAD_SEQ);
        return;
    }
    if (flag) atomicOr(p.err, flag);
    const int per = p.D / PIECE, row_pieces = 2 * p.H_kv * per;
#pragma unroll 4
    for (int i = tid; i < READ_ROWS * row_pieces; i += READ_THREADS) {
        const int t = i / row_pieces, w = i - t * row_pieces, hk = w / per, u = w - hk * per;
        const bool isv = hk >= p.H_kv;
        const int h = isv ? hk - p.H_kv : hk, block = block_s[t];
        T* out = static_cast<T*>(isv ? p.v_out : p.k_out);
        if (block == -2 || !out) continue;
        uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)(r0 + t) * (isv ? p.v_ts : p.k_ts) + (int64_t)h * p.D + u * PIECE);
        const int64_t bh = (int64_t)max(block, 0) * p.H_kv + h;
        const char* src = static_cast<const char*>(isv ? p.Vc : p.Kc) +
                          ((bh * p.bs + off_s[t]) * p.D + u * PIECE) * (Q8 ? 1 : (int)sizeof(T));
        const uint4 c = block < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(src));
        if constexpr (Q8) {
            uint4 o[16 / VEC];
            q8_widen16<T>(c, __ldg((isv ? p.Vsc : p.Ksc) + bh), o);
#pragma unroll
            for (int q = 0; q < 16 / VEC; ++q) dst[q] = o[q];
        } else {
            *dst = c;
        }
    }
}

// The blocks that entries with more than `wide` rows read (a group's prefix, a sequence's own part), as pools of the
// cache's dtype, at the same place, for the attention kernels of plain pools.  Every CTA finds these entries, 256 at a
// time, and all share their pieces laid end to end.  Bound by memory, a byte read and two (four) written a value.
template <typename T, bool JOINT>
__global__ void __launch_bounds__(READ_THREADS) widen_kernel(const Q8Widen x) {
    constexpr int VEC = Elem<T>::VEC, ILP = 4, WARPS = READ_THREADS / 32;
    const RaggedParams& p = x.r;
    __shared__ int seq_s[READ_THREADS], j0_s[READ_THREADS], warps[WARPS];
    __shared__ int64_t end_s[READ_THREADS], sums[WARPS];  // pieces up to and with an entry's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, NE = p.B + (JOINT ? p.NG : 0);
    const int lgper = 31 - __clz(p.bs * p.D / 16), heads = 2 * p.H_kv;  // 16-code pieces of a head's block; K and V heads
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int e0 = 0; e0 < NE; e0 += READ_THREADS) {
        const int e = e0 + tid;
        Entry s;
        s.ok = false;
        if (JOINT && e < p.NG) {
            const int b0 = __ldg(p.groups + e), b1 = __ldg(p.groups + e + 1);
            if (b0 >= 0 && b0 < p.B && b1 >= b0 && b1 <= p.B) s = group_entry(p, e);  // (else the attention flags it)
        } else if (e < NE) {
            s = seq_entry<JOINT>(p, e - (JOINT ? p.NG : 0));
        }
        const bool mine = s.ok && ((int64_t)s.T << p.lgG) > p.wide;
        const int j0 = !mine || s.group ? 0 : s.pfx >> p.lgbs;
        const int64_t n = !mine ? 0 : ((int64_t)((((s.group ? s.pfx : s.L) - 1) >> p.lgbs) + 1 - j0) * heads) << lgper;
        int64_t end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xFFFFFFFFu, end, o);
            if (lane >= o) end += t;
        }
        const uint32_t those = __ballot_sync(0xFFFFFFFFu, mine);
        __syncthreads();  // (the entries before are done with)
        if (lane == 31) {
            sums[warp] = end;
            warps[warp] = __popc(those);
        }
        __syncthreads();
        int found = 0, at = __popc(those & ((1u << lane) - 1));
        int64_t total = 0;
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) {
                at += warps[w];
                end += sums[w];
            }
            found += warps[w];
            total += sums[w];
        }
        if (mine) {
            seq_s[at] = s.seq;
            j0_s[at] = j0;
            end_s[at] = end;
        }
        __syncthreads();
        for (int64_t i0 = (int64_t)blockIdx.x * (ILP * READ_THREADS) + tid; i0 < total; i0 += (int64_t)gridDim.x * (ILP * READ_THREADS)) {
            uint4 c[ILP];
            float sc[ILP];
            int64_t at_piece[ILP];
            bool isv[ILP];
#pragma unroll
            for (int q = 0; q < ILP; ++q) {
                const int64_t i = i0 + q * READ_THREADS;
                at_piece[q] = -1;
                if (i >= total) continue;
                int k = 0, hi = found - 1;  // the first entry that ends behind the piece
                while (k < hi) {
                    const int mid = (k + hi) >> 1;
                    if (end_s[mid] <= i) k = mid + 1; else hi = mid;
                }
                const int64_t w = i - (k > 0 ? end_s[k - 1] : 0);
                const unsigned g = (unsigned)(w >> lgper), j = g / (unsigned)heads, hk = g - j * heads;
                const int block = __ldg(p.table + (size_t)seq_s[k] * p.max_blocks + j0_s[k] + j);
                if ((unsigned)block >= (unsigned)p.num_blocks) continue;
                isv[q] = hk >= (unsigned)p.H_kv;
                const int64_t bh = (int64_t)block * p.H_kv + (isv[q] ? hk - p.H_kv : hk);
                at_piece[q] = (bh << lgper) + (w & ((1 << lgper) - 1));
                c[q] = __ldg(static_cast<const uint4*>(isv[q] ? p.V : p.K) + at_piece[q]);
                sc[q] = __ldg((isv[q] ? x.Vsc : x.Ksc) + bh);
            }
#pragma unroll
            for (int q = 0; q < ILP; ++q) {
                if (at_piece[q] < 0) continue;
                uint4 o[16 / VEC];
                q8_widen16<T>(c[q], sc[q], o);
#pragma unroll
                for (int v = 0; v < 16 / VEC; ++v) static_cast<uint4*>(isv[q] ? x.V : x.K)[at_piece[q] * (16 / VEC) + v] = o[v];
            }
        }
    }
}

static cudaLaunchConfig_t dependent(cudaLaunchAttribute* attr, dim3 grid, int threads, cudaStream_t s) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

int launch_paged_read(int dtype, const Q8Read& p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = dependent(attr, dim3(((unsigned)p.N + READ_ROWS - 1) / READ_ROWS), READ_THREADS, s);
    const bool q8 = p.Ksc != nullptr;
    const cudaError_t e = dtype == 0 ? (q8 ? cudaLaunchKernelEx(&cfg, paged_read_kernel<__nv_bfloat16, true>, p)
                                           : cudaLaunchKernelEx(&cfg, paged_read_kernel<__nv_bfloat16, false>, p))
                                     : (q8 ? cudaLaunchKernelEx(&cfg, paged_read_kernel<float, true>, p)
                                           : cudaLaunchKernelEx(&cfg, paged_read_kernel<float, false>, p));
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

int launch_widen(int dtype, const Q8Widen& x, int sms, cudaStream_t s) {
    const RaggedParams& p = x.r;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = dependent(attr, dim3(4 * sms), READ_THREADS, s);
    const cudaError_t e = dtype == 0 ? (p.NG > 0 ? cudaLaunchKernelEx(&cfg, widen_kernel<__nv_bfloat16, true>, x)
                                                 : cudaLaunchKernelEx(&cfg, widen_kernel<__nv_bfloat16, false>, x))
                                     : (p.NG > 0 ? cudaLaunchKernelEx(&cfg, widen_kernel<float, true>, x)
                                                 : cudaLaunchKernelEx(&cfg, widen_kernel<float, false>, x));
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

}  // namespace kvc
