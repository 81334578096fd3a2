// kvc_q8.cuh -- the paged cache held in 8 bits: what its kernels share.
//
// A layer's K and V are pools of E4M3 codes [num_blocks, H_kv, bs, D] with one scale per block and
// KV head [num_blocks, H_kv], a power of two 2^e: value = code 2^e.  With amax the largest finite |x| of a
// block's rows of a head, e is the smallest exponent >= -64 with amax <= 448 2^e.  In a float format a
// power of two costs no precision (but for the lowest of its 18 binades), and makes three things exact: the
// comparison that picks e, the growth of a block's scale when a larger token joins (codes move down whole
// binades; only those that become subnormal are rounded again, by half of 2^-9 of the new scale each
// time: less than one such step in all, the sum of the halves of ever larger steps), and the values, which
// bf16 holds as they are.
#pragma once

#include "kvc_ragged.cuh"

namespace kvc {

constexpr int Q8_EMIN = -64, Q8_EMAX = 120;

// The exponent for the largest finite |x| given by its bits (448 = 1.75 2^8).
__host__ __device__ __forceinline__ int q8_exponent(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < Q8_EMIN ? Q8_EMIN : e;  // (at most Q8_EMAX: finite values are below 2^128)
}
// Exponent of a stored scale.
__host__ __device__ __forceinline__ int q8_stored(uint32_t bits) {
    const int e = (int)((bits >> 23) & 0xFFu) - 127;
    return e < Q8_EMIN ? Q8_EMIN : e > Q8_EMAX ? Q8_EMAX : e;
}

struct Q8Read {
    const void *Kc, *Vc;  // codes, or a plain cache's values (Ksc == nullptr)
    const float *Ksc, *Vsc;
    void *k_out, *v_out;  // [N, H_kv, D], either may be nullptr
    int64_t k_ts, v_ts;
    const int32_t *table, *cu, *lens;
    uint32_t* err;
    int B, N, H_kv, D, bs, max_blocks, num_blocks, T_max;
};
struct Q8Widen {
    RaggedParams r;  // (K, V: the codes)
    const float *Ksc, *Vsc;
    void *K, *V;  // pools of the same shape in the cache's dtype
};

// Attention on the codes (kvc_ragged_q8.cu; bf16, D = 64 or 128): maps of 128-byte rows (128 / D tokens) in boxes of
// q8_box tokens, scratch for P = ctas an SM with 2 slots of `rows` rows.
void q8_shape(int D, int G, int* rows, int* ctas);
constexpr int q8_box(int D, int bs) { return bs < 16384 / D ? bs : 16384 / D; }
// many: the call of the kernel of plain pools that attended the entries of many rows (p.part = 1), or nullptr.
int launch_ragged_q8(const RaggedParams& p, const RaggedParams* many, const float* Ksc, const float* Vsc,
                     const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);

// Launchers (kvc_append8.cu); each returns a cudaError_t.
int launch_append8(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s);
int launch_paged_read(int dtype, const Q8Read& p, cudaStream_t s);
int launch_widen(int dtype, const Q8Widen& p, int sms, cudaStream_t s);

}  // namespace kvc
