// kvc_append8.cu -- the paged cache held in 8 bits (kvc_q8.cuh): append of ragged new tokens with norms and
// rotary positions, reading positions back, widening of whole blocks.
#include <type_traits>

#include "kvc_q8.cuh"
#include "kvc_rope.cuh"

namespace kvc {

// Two values as codes.  (mul: 2^-e; out of range is the largest code.)
__device__ __forceinline__ uint32_t q8_codes2(float x, float y, float mul) { return e4m3x2(x * mul, y * mul); }
// The same where infinities occur, which are stored as NaN (E4M3 has none), or where the largest code would read back as
// one.
__device__ __forceinline__ uint32_t q8_codes2_any(float x, float y, float mul, float lim) {
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
// touch), so no sum over the sequences is needed.  The angles of 4096 pairs (64 rows at D = 128) are turned into
// cosines and sines at a time, once for the CTA's heads where that is all of them.  K or V of a head is a unit of one warp (of two or four where heads are few or blocks long), which goes
// over its rows twice: first for the largest |x| of K, normalised and rotated, or of V, which settles the scale, then, from
// L1, for the codes.  Bound by its chain of lookups, first pass, maximum and second pass (0.43 of its issue slots, waits for
// memory first among its stalls): 9700 rows of 32 + 8 heads, two groups of heads, take 73 us with the queries' grid, 3.0 TB/s.  That
// grid begins as the last CTA of this one has begun, for there are 304 places, two an SM: 152 blocks of 64 rows take 69 us, 153
// 87, 304 129, 308 148.  (Values held in registers between the passes
// spilled, or left too few warps: 112 to 129 us, and 81 with a CTA's heads laid out as pieces and a maximum exchanged
// for each.)  A block that holds earlier rows and needs a larger scale has their codes moved down.
constexpr int APPEND8_THREADS = 256, APPEND8_WARPS = APPEND8_THREADS / 32;
struct Append8Grid {
    int nkv, groups, hg, rounds, wpu, chunk, two;  // CTAs of keys and values; groups of `rounds` times hg heads; warps of a unit; rows
                                           // whose angles are held; do the queries follow as a grid of their own?
};

template <typename T, bool NORM>
__device__ __forceinline__ void append8_block(const RopeParams& p, const RopeTable& rt, int item, int h_first, int h_count,
                                              const Append8Grid& grid, float* trig) {
    constexpr int VEC = Elem<T>::VEC, NT = APPEND8_THREADS;
    __shared__ int found;
    __shared__ uint32_t amax[2][APPEND8_WARPS];  // of a round's units, of two rounds in turn
    __shared__ uint64_t freq_s[128];  // (from the parameters, where each lane's is another, a warp's loads go one by one)
    __shared__ uint8_t axis_s[128];
    __shared__ float inv_s[256];  // norms of the rows of a round's heads (4 of 64 rows, 2 of 128, or 1)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pairs = rt.rot_dim / 2, nrot = rt.rot_dim / (2 * VEC);
    if (tid == 0) found = 0;
    if (tid < 2 * APPEND8_WARPS) amax[tid / APPEND8_WARPS][tid % APPEND8_WARPS] = 0;
    if (tid < pairs) {
        freq_s[tid] = rt.freq[tid];
        axis_s[tid] = rt.axis[tid];
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (grid.two) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (see LATE: 74 us against 79.5)
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
    const int chunk = min(grid.chunk, nrow), nchunk = (nrow + grid.chunk - 1) / grid.chunk;
    float* cosines = trig;
    float* sines = trig + chunk * pairs;
    // the angles of rows [row, row + chunk), by all threads
    auto angles_of = [&](int row) {
        __syncthreads();
        for (int i = tid; i < min(chunk, nrow - row) * pairs; i += NT) {
            const int t = i / pairs, pr = i - t * pairs;
            const int pos = p.positions ? __ldg(p.positions + (int64_t)axis_s[pr] * p.pos_ts + r0 + row + t) : lo + row + t;
            const uint64_t turn = (uint64_t)(int64_t)pos * freq_s[pr];
            float s, c;
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
            cosines[i] = c * rt.scale;
            sines[i] = s * rt.scale;
        }
        __syncthreads();
    };
    if (nchunk == 1) angles_of(0);
    // A unit's pieces: a lane's are at one place of the rows' heads, v0 and v1, rows `row0`, row0 + step, ..
    const int per = p.D / (2 * VEC), lg = 31 - __clz(per), u = lane & (per - 1);
    const int unit = warp / grid.wpu, part = warp - unit * grid.wpu;
    const bool isv = unit & 1, halves = !isv && u < nrot && !rt.adjacent;
    const int v0 = halves ? u : 2 * u, v1 = halves ? u + nrot : 2 * u + 1;
    const int row0 = (part << (5 - lg)) + (lane >> lg), step = grid.wpu << (5 - lg);
    const bool normed = NORM && p.k_norm && !isv, turned = !isv && u < nrot;
    uint4 wx = make_uint4(0, 0, 0, 0), wy = wx;
    if (normed) {
        wx = __ldg(static_cast<const uint4*>(p.k_norm) + v0);
        wy = __ldg(static_cast<const uint4*>(p.k_norm) + v1);
    }
    for (int rd = 0; rd < grid.rounds; ++rd) {
        const int hl = rd * grid.hg + (unit >> 1);  // the unit's head, of this CTA's
        const bool live = unit < 2 * grid.hg && hl < h_count;
        const int h = h_first + hl;
        const T* src = isv ? static_cast<const T*>(p.v) + r0 * p.v_ts + (int64_t)h * p.D
                           : static_cast<const T*>(p.k) + r0 * p.k_ts + (int64_t)h * p.D;
        const int64_t ts = isv ? p.v_ts : p.k_ts;
        // Row `row`'s values at this lane's place; the angles held begin at row `from`.
        auto values = [&](int pass, bool there, int row, int from, const uint4& a, const uint4& bb, float (&x)[VEC], float (&y)[VEC]) {
            Elem<T>::unpack(a, x);
            Elem<T>::unpack(bb, y);
            if (normed) {  // (alike in a warp, whose lanes stay together)
                float* kept = &inv_s[(unit >> 1) * p.bs + row];
                const float inv = pass == 0 ? norm_factor<VEC>(x, y, per, 1.f / (float)p.D, p.eps) : *kept;
                if (pass == 0 && there) *kept = inv;
                norm_piece<T>(x, y, wx, wy, inv);
            }
            if (!turned) return;
            const float *cr = cosines + (row - from) * pairs + u * VEC, *sr = sines + (row - from) * pairs + u * VEC;
            float co[VEC], si[VEC];
#pragma unroll
            for (int q = 0; q < VEC; q += 4) {
                *reinterpret_cast<float4*>(co + q) = *reinterpret_cast<const float4*>(cr + q);
                *reinterpret_cast<float4*>(si + q) = *reinterpret_cast<const float4*>(sr + q);
            }
            turn_piece<VEC>(x, y, co, si, !rt.adjacent);
        };
        uint32_t* tops = amax[rd & 1];
        char* codes = static_cast<char*>(isv ? p.Vc : p.Kc) + (((int64_t)e * p.H_kv + h) * p.bs) * p.D;
        char* dst = codes + (lo - start) * p.D;
        float mul = 0.f, lim = 0.f, down = 1.f;
        bool infinite = false;
        // Pass 0: the largest |x|; 1: the largest finite one, if that was none; 2: the codes.  (One copy of the code: with
        // one for each pass the values did not fit the registers.)
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            if (pass == 1 && !infinite) continue;
            float m = 0.f;
            // this lane's rows, two loaded at once; all of the block come along for the angles
            for (int from = 0; from < nrow; from += chunk) {
                if (nchunk > 1) angles_of(from);
                if (!live) continue;
                const int end = min(from + chunk, nrow);
                for (int first = from + row0 - (lane >> lg); first < end; first += 2 * step) {  // (the warp's first row)
                    uint4 a[2], bb[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int row = first + (lane >> lg) + q * step;
                        a[q] = bb[q] = make_uint4(0, 0, 0, 0);
                        if (row < end) {
                            const uint4* at = reinterpret_cast<const uint4*>(src + row * ts);
                            a[q] = __ldg(at + v0);
                            bb[q] = __ldg(at + v1);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (first + q * step >= end) continue;
                        const int row = min(first + (lane >> lg) + q * step, end - 1);
                        float x[VEC], y[VEC];
                        const bool there = first + (lane >> lg) + q * step < end;
                        values(pass, there, row, from, a[q], bb[q], x, y);
                        if (!there) continue;
                        if (pass == 0) {  // (a maximum passes NaN over)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(y[i])));
                        } else if (pass == 1) {
#pragma unroll
                            for (int i = 0; i < VEC; ++i) {
                                m = isfinite(x[i]) ? fmaxf(m, fabsf(x[i])) : m;
                                m = isfinite(y[i]) ? fmaxf(m, fabsf(y[i])) : m;
                            }
                        } else {
                            uint32_t w[VEC / 4], z[VEC / 4];
#pragma unroll
                            for (int i = 0; i < VEC / 4; ++i) {
                                const int k = 4 * i;
                                if (lim == 0.f) {
                                    w[i] = q8_codes2(x[k], x[k + 1], mul) | q8_codes2(x[k + 2], x[k + 3], mul) << 16;
                                    z[i] = q8_codes2(y[k], y[k + 1], mul) | q8_codes2(y[k + 2], y[k + 3], mul) << 16;
                                } else {
                                    w[i] = q8_codes2_any(x[k], x[k + 1], mul, lim) | q8_codes2_any(x[k + 2], x[k + 3], mul, lim) << 16;
                                    z[i] = q8_codes2_any(y[k], y[k + 1], mul, lim) | q8_codes2_any(y[k + 2], y[k + 3], mul, lim) << 16;
                                }
                            }
                            char* to = dst + row * p.D;
                            if constexpr (VEC == 8) {
                                *reinterpret_cast<uint2*>(to + v0 * VEC) = make_uint2(w[0], w[1]);
                                *reinterpret_cast<uint2*>(to + v1 * VEC) = make_uint2(z[0], z[1]);
                            } else {
                                *reinterpret_cast<uint32_t*>(to + v0 * VEC) = w[0];
                                *reinterpret_cast<uint32_t*>(to + v1 * VEC) = z[0];
                            }
                        }
                    }
                }
            }
            if (pass == 2) break;
            uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
            if (live && lane == 0) atomicMax(&tops[unit], top);
            __syncthreads();
            if (live) top = tops[unit];
            if (pass == 0) {
                if (tid < APPEND8_WARPS) amax[(rd & 1) ^ 1][tid] = 0;
                infinite = __syncthreads_or(live && top >= 0x7F800000u) != 0;
                if (infinite) {
                    if (tid < APPEND8_WARPS) tops[tid] = 0;
                    __syncthreads();
                    continue;
                }
            }
            float* sc = (isv ? p.Vsc : p.Ksc) + (int64_t)e * p.H_kv + h;
            int x = q8_exponent(top);
            if (live && held > 0) {
                const int old = q8_stored(__float_as_uint(*sc));
                if (old >= x) x = old;
                else down = exp2i(max(old - x, -60));
            }
            // (a unit's lanes, and its warps, have all read the old scale before one of them stores the new one)
            if (grid.wpu > 1) __syncthreads();
            else __syncwarp();
            if (live && part == 0 && lane == 0) *sc = exp2i(x);
            mul = exp2i(-x);
            if (infinite || x == Q8_EMAX) lim = x == Q8_EMAX ? 240.f : 448.f;  // (256 2^120 is past the largest float)
        }
        if (live && down != 1.f) {
            uint4* c = reinterpret_cast<uint4*>(codes);
            for (int i = part * 32 + lane; i < held * (p.D / 16); i += 32 * grid.wpu) {
                const uint4 w = c[i];
                c[i] = make_uint4(q8_rescale4(w.x, down), q8_rescale4(w.y, down), q8_rescale4(w.z, down),
                                  q8_rescale4(w.w, down));
            }
        }
    }
}

// Blocks [0, nkv) append keys and values (nkv / groups items), the others rotate the queries, a row each (none in the
// launch of many rows, where the queries have a kernel of their own, with more blocks an SM).
template <typename T, bool NORM>
__global__ void __launch_bounds__(APPEND8_THREADS, 2)
append8_kernel(const RopeParams p, const __grid_constant__ RopeTable rt, const Append8Grid g) {
    extern __shared__ __align__(16) float trig8[];
    if (blockIdx.x < g.nkv) {
        const int item = blockIdx.x / g.groups, each = g.hg * g.rounds, h = (blockIdx.x - item * g.groups) * each;
        append8_block<T, NORM>(p, rt, item, h, min(each, p.H_kv - h), g, trig8);
    } else {
        RopeParams q = p;  // the queries alone
        q.H_kv = 0;
        append_rows<T, 1, true, NORM>(q, rt, blockIdx.x - g.nkv);
    }
}

template <typename T, bool NORM>
static int launch_append8_as(const RopeParams& p, const RopeTable& t, int sms, bool many, cudaStream_t s) {
    Append8Grid g;
    // heads at a time: a unit's warp gets some 64 rows at most
    const int most = p.bs <= 64 ? 4 : p.bs == 128 ? 2 : 1;
    g.hg = most;
    while (g.hg > p.H_kv) g.hg /= 2;
    g.wpu = APPEND8_WARPS / (2 * g.hg);
    // the angles are shared by a CTA's heads: as many as leave the GPU some CTAs an SM
    g.rounds = 1;
    while (g.rounds * g.hg * 2 <= p.H_kv && (int64_t)(p.N / p.bs) * ((p.H_kv + 2 * g.rounds * g.hg - 1) / (2 * g.rounds * g.hg)) >= 4 * sms)
        g.rounds *= 2;
    g.groups = (p.H_kv + g.hg * g.rounds - 1) / (g.hg * g.rounds);
    const int64_t nkv = (p.N / p.bs + 2 * (int64_t)p.B) * g.groups;
    const int64_t nq = p.q && !many ? p.N : 0;
    if (nkv + nq > 0x7FFFFFFF) return (int)cudaErrorInvalidValue;
    g.nkv = (int)nkv;
    g.two = many && p.q;
    // rows whose angles are held: 4096 cosines and as many sines, 32 KB
    const int pairs = t.rot_dim > 0 ? t.rot_dim / 2 : 1;
    g.chunk = 4096 / pairs < p.bs ? 4096 / pairs : p.bs;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(nkv + nq));
    cfg.blockDim = dim3(APPEND8_THREADS);
    cfg.dynamicSmemBytes = g.chunk * pairs * 2 * sizeof(float);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, append8_kernel<T, NORM>, p, t, g);
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}
int launch_append8(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s) {
    const bool norm = p.q_norm || p.k_norm, many = p.N >= 8 * sms;
    auto go = [&](auto tp) {
        using T = decltype(tp);
        return norm ? launch_append8_as<T, true>(p, t, sms, many, s) : launch_append8_as<T, false>(p, t, sms, many, s);
    };
    const int e = dtype == 0 ? go(__nv_bfloat16()) : go(float());
    if (e != 0 || !many || !p.q) return e;
    RopeParams q = p;
    q.H_kv = 0;
    return launch_late_queries(dtype, q, t, s);
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
// written once.  (38,000 bf16 rows of 8 heads 47.2 us, 5.0 TB/s, with 8 rows, 50.3 with 4; in blocks of 16 and three times
// as many 123 against 134, 5.4 TB/s.  32 bytes a store make no difference.)
constexpr int READ_THREADS = 256, READ_ROWS = 8;
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
// time, and all share their pieces laid end to end.  Bound by memory, a byte read and two (four) written a value: 4
// sequences of 4500 positions of 8 heads 20 us.  (By entries, a CTA each, one long entry took as long as all.)
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
                const int64_t g = w >> lgper;  // (past 32 bits for 16 KV heads at 2^31 positions)
                const unsigned j = g >> 32 ? (unsigned)(g / heads) : (unsigned)g / (unsigned)heads, hk = (unsigned)g - j * heads;
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
