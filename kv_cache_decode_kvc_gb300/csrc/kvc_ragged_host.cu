// kvc_ragged_host.cu -- the C ABI of ragged batches over a paged cache: rotary tables, argument
// checks, scratch layout, dispatch (include/kvc.h).
#include <math.h>
#include <string.h>

#include <new>

#include "kvc_handle.cuh"
#include "kvc_ragged.cuh"

struct kvc_rope {
    kvc::RopeTable t;
};

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A packed tensor: 16-byte aligned rows of at least `row` elements.
bool packed_ok(const void* p, int64_t stride, int64_t row, int es) {
    return p && aligned(p, 16) && stride >= row && stride <= (int64_t(1) << 40) && (stride * es) % 16 == 0;
}

int on_device(const kvc_cache* h) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return KVC_ECUDA;
    return dev == h->device ? KVC_OK : KVC_EINVAL;
}

// The tensor-core kernel takes bf16 pools with D = 64 or 128 unless CUDA cores are asked for.
bool ragged_tc5(const kvc_cache* h) {
    return h->dtype == KVC_BF16 && h->math != 1 && (h->D == 128 ? h->tc_ok : !h->rmaps.empty());
}
// CTAs of the attention kernels at most: the tensor-core kernel fills an SM, two blocks of the
// CUDA-core kernel fit.
int ragged_p(const kvc_cache* h, bool tc5) { return h->ctas > 0 ? h->ctas : (tc5 ? 1 : 2) * h->sms; }
// Scratch of a path: the tensor-core kernel's CTAs hold five slots of 128 rows, the others' two of 64.
kvc::RaggedScratch ragged_ws(const kvc_cache* h, int N, int NG, bool tc5) {
    return kvc::ragged_scratch(h->B, N, NG, h->H_q, h->D, ragged_p(h, tc5), tc5 ? 5 : 2, tc5 ? 128 : 64);
}

int attn_ragged(kvc_t h, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride, const int32_t* table,
                const int32_t* cu, const int32_t* lens, int N, const int32_t* groups, const int32_t* prefix, int NG,
                void* ws, uint64_t ws_bytes, void* stream) {
    if (!h || !table || !cu || !lens || !ws || N < 1) return KVC_EINVAL;
    if (!h->paged || layer < 0 || layer >= h->layers) return KVC_EINVAL;
    const int64_t row = (int64_t)h->H_q * h->D;
    if (!packed_ok(q, q_stride, row, h->es) || !packed_ok(out, out_stride, row, h->es)) return KVC_EINVAL;
    if (!aligned(table, 4) || !aligned(cu, 4) || !aligned(lens, 4) || !aligned(ws, 256)) return KVC_EINVAL;
    const bool tc5 = ragged_tc5(h);
    const kvc::RaggedScratch sc = ragged_ws(h, N, NG, tc5);
    if (ws_bytes < sc.total) return KVC_EINVAL;
    const int rc = on_device(h);
    if (rc != KVC_OK) return rc;
    kvc::RaggedParams p{};
    p.K = h->slab + (size_t)(2 * layer) * h->layer_bytes;
    p.V = h->slab + (size_t)(2 * layer + 1) * h->layer_bytes;
    p.q = q;
    p.out = out;
    p.q_ts = q_stride;
    p.out_ts = out_stride;
    p.table = table;
    p.cu = cu;
    p.lens = lens;
    p.groups = NG > 0 ? groups : nullptr;
    p.prefix = NG > 0 ? prefix : nullptr;
    p.err = h->err;
    char* w = static_cast<char*>(ws);
    p.plan = reinterpret_cast<int*>(w + sc.plan);
    p.cuts = reinterpret_cast<int4*>(w + sc.cuts);
    p.row_o = reinterpret_cast<float*>(w + sc.row_o);
    p.row_ml = reinterpret_cast<float*>(w + sc.row_ml);
    p.slot_o = reinterpret_cast<float*>(w + sc.slot_o);
    p.slot_ml = reinterpret_cast<float*>(w + sc.slot_ml);
    p.B = h->B;
    p.N = N;
    p.H_q = h->H_q;
    p.H_kv = h->H_kv;
    p.NG = NG;
    p.D = h->D;
    for (p.lgG = 0; (1 << p.lgG) < h->G; ++p.lgG) {}
    p.bs = h->bs;
    for (p.lgbs = 0; (1 << p.lgbs) < h->bs; ++p.lgbs) {}
    p.max_blocks = h->max_blocks;
    p.num_blocks = h->num_blocks;
    p.T_max = h->T_max;
    p.P = ragged_p(h, tc5);
    p.qscale = (float)(1.4426950408889634 / sqrt((double)h->D));
    if (tc5) {
        // boxes of 64 query rows, and of as few as one token's
        CUtensorMap mq, m1;
        const int few = h->G > 16 ? h->G : 16;
        if (!kvc::make_q_tensor_map(&mq, q, N, h->H_q, h->D, q_stride, h->G, 64 / h->G) ||
            !kvc::make_q_tensor_map(&m1, q, N, h->H_q, h->D, q_stride, h->G, few / h->G))
            return KVC_ECUDA;
        const CUtensorMap* kv = h->D == 128 ? &h->tmaps[4 * (size_t)layer + 2] : &h->rmaps[2 * (size_t)layer];
        return kvc::launch_ragged_tc5(p, mq, m1, kv[0], kv[1], static_cast<cudaStream_t>(stream)) == 0 ? KVC_OK : KVC_ECUDA;
    }
    return kvc::launch_ragged_cc(h->dtype, p, static_cast<cudaStream_t>(stream)) == 0 ? KVC_OK : KVC_ECUDA;
}

}  // namespace

extern "C" {

int kvc_rope_create(kvc_rope_t* out, int rot_dim, const double* inv_freq, int layout, int n_axes, const int32_t* axis,
                    float scale) {
    if (!out) return KVC_EINVAL;
    *out = nullptr;
    if (!inv_freq || rot_dim < 2 || rot_dim % 2 != 0 || n_axes < 1 || !isfinite(scale)) return KVC_EINVAL;
    if (layout != KVC_ROPE_HALF && layout != KVC_ROPE_ADJACENT) return KVC_EINVAL;
    if (rot_dim > 256 || n_axes > 8) return KVC_EUNSUPPORTED;
    kvc_rope* r = new (std::nothrow) kvc_rope();
    if (!r) return KVC_ENOMEM;
    r->t.rot_dim = rot_dim;
    r->t.adjacent = layout == KVC_ROPE_ADJACENT;
    r->t.n_axes = n_axes;
    r->t.scale = scale;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const int a = axis ? axis[i] : 0;
        if (!isfinite(inv_freq[i]) || a < 0 || a >= n_axes) {
            delete r;
            return KVC_EINVAL;
        }
        r->t.freq[i] = kvc::rope_turns(inv_freq[i]);
        r->t.axis[i] = (uint8_t)a;
    }
    *out = r;
    return KVC_OK;
}

int kvc_rope_destroy(kvc_rope_t r) {
    delete r;
    return KVC_OK;
}

int kvc_paged_append_rope(kvc_t h, int layer, kvc_rope_t rope, const void* q, int64_t q_stride, void* q_out,
                          int64_t q_out_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* positions, int64_t pos_stride, const int32_t* block_table,
                          const int32_t* cu_seqlens, const int32_t* lens, int N, void* stream) {
    if (!h || !rope || !block_table || !cu_seqlens || !lens || N < 1) return KVC_EINVAL;
    if (!h->paged || layer < 0 || layer >= h->layers || rope->t.rot_dim > h->D) return KVC_EINVAL;
    if ((q == nullptr) != (q_out == nullptr)) return KVC_EINVAL;
    const int64_t qrow = (int64_t)h->H_q * h->D, krow = (int64_t)h->H_kv * h->D;
    if (q && (!packed_ok(q, q_stride, qrow, h->es) || !packed_ok(q_out, q_out_stride, qrow, h->es))) return KVC_EINVAL;
    if (q && q == q_out && q_stride != q_out_stride) return KVC_EINVAL;
    if (!packed_ok(k, k_stride, krow, h->es) || !packed_ok(v, v_stride, krow, h->es)) return KVC_EINVAL;
    if (positions && (!aligned(positions, 4) || (rope->t.n_axes > 1 && pos_stride < N && pos_stride != 0))) return KVC_EINVAL;
    if (!aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(lens, 4)) return KVC_EINVAL;
    const int rc = on_device(h);
    if (rc != KVC_OK) return rc;
    kvc::RopeParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.Kc = h->slab + (size_t)(2 * layer) * h->layer_bytes;
    p.Vc = h->slab + (size_t)(2 * layer + 1) * h->layer_bytes;
    p.q_ts = q_stride;
    p.qo_ts = q_out_stride;
    p.k_ts = k_stride;
    p.v_ts = v_stride;
    p.pos_ts = pos_stride;
    p.positions = positions;
    p.table = block_table;
    p.cu = cu_seqlens;
    p.lens = lens;
    p.err = h->err;
    p.B = h->B;
    p.N = N;
    p.H_q = h->H_q;
    p.H_kv = h->H_kv;
    p.D = h->D;
    p.bs = h->bs;
    p.max_blocks = h->max_blocks;
    p.num_blocks = h->num_blocks;
    p.T_max = h->T_max;
    return kvc::launch_append_rope(h->dtype, p, rope->t, h->sms, static_cast<cudaStream_t>(stream)) == 0 ? KVC_OK
                                                                                                        : KVC_ECUDA;
}

int kvc_paged_attn_workspace(kvc_t h, int N, int NG, uint64_t* bytes) {
    if (!h || !bytes || !h->paged || N < 1 || NG < 0 || NG > h->B) return KVC_EINVAL;
    // enough for either path, whatever kvc_set_math does in between
    const uint64_t a = ragged_ws(h, N, NG, true).total, b = ragged_ws(h, N, NG, false).total;
    *bytes = a > b ? a : b;
    return KVC_OK;
}

int kvc_paged_attn_ragged(kvc_t h, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride,
                          const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* lens, int N, void* ws,
                          uint64_t ws_bytes, void* stream) {
    return attn_ragged(h, layer, q, q_stride, out, out_stride, block_table, cu_seqlens, lens, N, nullptr, nullptr, 0, ws,
                       ws_bytes, stream);
}

int kvc_paged_attn_shared(kvc_t h, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride,
                          const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* lens, int N,
                          const int32_t* groups, const int32_t* prefix_lens, int NG, void* ws, uint64_t ws_bytes,
                          void* stream) {
    if (!h || !groups || !prefix_lens || NG < 1 || NG > h->B) return KVC_EINVAL;
    if (!aligned(groups, 4) || !aligned(prefix_lens, 4)) return KVC_EINVAL;
    return attn_ragged(h, layer, q, q_stride, out, out_stride, block_table, cu_seqlens, lens, N, groups, prefix_lens, NG,
                       ws, ws_bytes, stream);
}

}  // extern "C"
