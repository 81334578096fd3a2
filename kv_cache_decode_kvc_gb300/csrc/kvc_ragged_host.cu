// kvc_ragged_host.cu -- the C ABI of ragged batches over a paged cache: rotary tables, argument
// checks, scratch layout, dispatch (include/kvc.h).
#include <math.h>
#include <string.h>

#include <new>

#include "kvc_handle.cuh"
#include "kvc_q8.cuh"
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

// Which kernel attends: on CUDA cores, on the tensor cores, or on the tensor cores and an 8-bit cache's codes.
// CUDA cores take an 8-bit cache's blocks widened to its dtype.
enum class Path { CC, TC5, Q8 };
Path ragged_path(const kvc_cache* h) {
    if (h->dtype != KVC_BF16 || h->math == 1) return Path::CC;
    if (h->quant) return h->rmaps.empty() ? Path::CC : Path::Q8;
    return (h->D == 128 ? h->tc_ok : !h->rmaps.empty()) ? Path::TC5 : Path::CC;
}
// CTAs of the attention kernels at most: the tensor-core kernel fills an SM, two blocks of the
// CUDA-core kernel fit.
int ragged_p(const kvc_cache* h, Path path) {
    int rows, ctas = path == Path::TC5 ? 1 : 2;
    if (path == Path::Q8) kvc::q8_shape(h->D, h->G, &rows, &ctas);
    return h->ctas > 0 ? h->ctas : ctas * h->sms;
}
// Scratch of a path: the tensor-core kernel's CTAs hold five slots of 128 rows, the others' two of 64 (on codes:
// of a tile's rows).
kvc::RaggedScratch ragged_ws(const kvc_cache* h, int N, int NG, Path path) {
    int rows = path == Path::TC5 ? 128 : 64, ctas;
    if (path == Path::Q8) kvc::q8_shape(h->D, h->G, &rows, &ctas);
    return kvc::ragged_scratch(h->B, N, NG, h->H_q, h->D, ragged_p(h, path), path == Path::TC5 ? 5 : 2, rows);
}
// On an 8-bit cache, entries (sequences, shared prefixes) with more query rows per head than this are widened to bf16
// and attended by the kernel of plain pools: per 32 rows it takes a quarter of the time of the kernel on codes, which
// has to make up for the widening, for merging its larger pieces, and for two kernels one after the other where a batch
// has both kinds.  So what matters besides an entry's rows is whether the others go the same way, and of that the host knows
// the mean.  (24 sequences of 3000 to 6000 positions with 30 to 40, 40 to 60, 56 to 64 tokens, D = 128, 32 heads on 8: all on codes
// 258, 355, 412 us, all widened 255, 269, 273; 64 sequences of 5 tokens of 32 heads on 1 141, 145, of 7 179, 150.  D = 64, where
// the kernel on codes has one CTA an SM: 64 sequences of 1 to 5 such tokens 111 and 100, of 2 on 2 KV heads 70 and 80, 24 of 40
// to 60 tokens 393 and 176; with 20 of those 24 single tokens 124 at 256 rows, 100 at 128 and 64; 64 sequences of 20 to 80 rows 96 at
// 128, 112 at 64.  D = 128, 4 of 24 sequences with chunks of 4 x 300 rows at most: 171 at 64 to 256, 181 at 512.)
int many_rows(const kvc_cache* h, int N) {
    const int64_t mean = (int64_t)N * h->G / h->B;
    return h->D == 64 ? (mean >= 80 ? 16 : 128) : mean >= 160 ? 32 : 256;
}
// Is that worth its launches (13 to 16 us with nothing to do)?  The host knows how many rows an entry can have if every
// sequence has a token, no more (a batch whose sequences have none, against that, is attended on codes all the same), and
// how many positions it can see: where a CTA gets few tiles even then, codes are as quick.  (D = 128: up to 32, some 65 us:
// one chunk of 200 tokens of 32 heads on 8 beside 23 single ones, all of 3000 to 6000 positions, 92 us on codes, 116 widened, of 300
// 116 and 119; 64 sequences of 1 to 5 tokens on one KV head 90 and, with nothing widened, 106.)  What it knows are capacities, T_max
// and B, and these times are of tables as long as their longest sequence: with tables of 131,072 positions that chunk of 200 is
// widened all the same (116), and 24 sequences of 8 tokens take 84 us, not 72; a chunk of 1024 tokens behind 4000 positions alone among
// 1024 slots, whose others N could give a token each, stays on codes (274 us; in a batch of one, widened, 105).
bool split_rows(const kvc_cache* h, int N, int NG) {
    const int64_t most = (NG > 0 ? N : (int64_t)N - h->B + 1) * h->G;
    if (most <= 512) return false;
    int rows, ctas;
    kvc::q8_shape(h->D, h->G, &rows, &ctas);
    const int64_t tiles = (most + rows - 1) / rows * (((int64_t)h->T_max * h->D + 16383) / 16384) * h->H_kv;
    return tiles > (int64_t)(ctas == 1 ? 24 : 64) * h->sms;
}
// The parts of the scratch: the path's, that of the kernel of plain pools beside the one on codes, and the two
// widened pools.
struct Scratch {
    kvc::RaggedScratch own, many;
    uint64_t many_at, wide_at, wide_bytes, total;
    bool split;  // entries of many rows are attended apart
};
Scratch scratch_of(const kvc_cache* h, int N, int NG, Path path) {
    Scratch s{};
    s.own = ragged_ws(h, N, NG, path);
    s.split = path == Path::Q8 && split_rows(h, N, NG);
    s.many_at = s.wide_at = s.total = s.own.total;
    if (s.split) {
        s.many = ragged_ws(h, N, NG, Path::TC5);
        s.wide_at = s.total += s.many.total;
    }
    if (h->quant && (path == Path::CC || s.split)) {
        s.wide_bytes = ((uint64_t)h->layer_bytes * h->es + 255) / 256 * 256;
        s.total += 2 * s.wide_bytes;
    }
    return s;
}
void set_scratch(kvc::RaggedParams& p, char* w, const kvc::RaggedScratch& sc) {
    p.plan = reinterpret_cast<int*>(w + sc.plan);
    p.cuts = reinterpret_cast<int4*>(w + sc.cuts);
    p.row_o = reinterpret_cast<float*>(w + sc.row_o);
    p.row_ml = reinterpret_cast<float*>(w + sc.row_ml);
    p.slot_o = reinterpret_cast<float*>(w + sc.slot_o);
    p.slot_ml = reinterpret_cast<float*>(w + sc.slot_ml);
}
// The tensor-core kernel of plain pools, k / v: the pools' maps.
int launch_tc5(const kvc_cache* h, const kvc::RaggedParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
    // boxes of 64 query rows, and of as few as one token's
    CUtensorMap mq, m1;
    const int few = h->G > 16 ? h->G : 16;
    if (!kvc::make_q_tensor_map(&mq, p.q, p.N, h->H_q, h->D, p.q_ts, h->G, 64 / h->G) ||
        !kvc::make_q_tensor_map(&m1, p.q, p.N, h->H_q, h->D, p.q_ts, h->G, few / h->G))
        return KVC_ECUDA;
    return kvc::launch_ragged_tc5(p, mq, m1, k, v, st) == 0 ? KVC_OK : KVC_ECUDA;
}

int attn_ragged(kvc_t h, int layer, const void* q, int64_t q_stride, void* out, int64_t out_stride, const int32_t* table,
                const int32_t* cu, const int32_t* lens, int N, const int32_t* groups, const int32_t* prefix, int NG,
                void* ws, uint64_t ws_bytes, void* stream) {
    if (!h || !table || !cu || !lens || !ws || N < 1) return KVC_EINVAL;
    if (!h->paged || layer < 0 || layer >= h->layers) return KVC_EINVAL;
    const int64_t row = (int64_t)h->H_q * h->D;
    if (!packed_ok(q, q_stride, row, h->es) || !packed_ok(out, out_stride, row, h->es)) return KVC_EINVAL;
    if (!aligned(table, 4) || !aligned(cu, 4) || !aligned(lens, 4) || !aligned(ws, 256)) return KVC_EINVAL;
    const Path path = ragged_path(h);
    const Scratch sc = scratch_of(h, N, NG, path);
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
    set_scratch(p, w, sc.own);
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
    p.P = ragged_p(h, path);
    p.qscale = (float)(1.4426950408889634 / sqrt((double)h->D));
    p.take(0, 0);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!h->quant) {
        if (path == Path::CC) return kvc::launch_ragged_cc(h->dtype, p, st) == 0 ? KVC_OK : KVC_ECUDA;
        const CUtensorMap* kv = h->D == 128 ? &h->tmaps[4 * (size_t)layer + 2] : &h->rmaps[2 * (size_t)layer];
        return launch_tc5(h, p, kv[0], kv[1], st);
    }
    const float* Ksc = h->scales + (size_t)(2 * layer) * h->scale_stride;
    const float* Vsc = Ksc + h->scale_stride;
    kvc::RaggedParams m = p;  // the call on widened blocks
    m.K = w + sc.wide_at;
    m.V = w + sc.wide_at + sc.wide_bytes;
    m.wide = path == Path::CC ? -1 : many_rows(h, N);
    if (path == Path::CC || sc.split) {
        kvc::Q8Widen x{p, Ksc, Vsc, w + sc.wide_at, w + sc.wide_at + sc.wide_bytes};
        x.r.wide = m.wide;
        if (kvc::launch_widen(h->dtype, x, h->sms, st) != 0) return KVC_ECUDA;
    }
    if (path == Path::CC) return kvc::launch_ragged_cc(h->dtype, m, st) == 0 ? KVC_OK : KVC_ECUDA;
    if (sc.split) {
        set_scratch(m, w + sc.many_at, sc.many);
        m.row_o = p.row_o;  // (the rows of shared prefixes are merged together)
        m.row_ml = p.row_ml;
        m.P = ragged_p(h, Path::TC5);
        m.take(2, m.wide);
        p.take(1, m.wide);
        CUtensorMap mk, mv;
        const uint64_t rows = h->layer_bytes / h->D;
        const int box = h->bs < 128 ? h->bs : 128;
        if (!kvc::make_pool_tensor_map(&mk, w + sc.wide_at, rows, h->D, box) ||
            !kvc::make_pool_tensor_map(&mv, w + sc.wide_at + sc.wide_bytes, rows, h->D, box))
            return KVC_ECUDA;
        const int e = launch_tc5(h, m, mk, mv, st);
        if (e != KVC_OK) return e;
    }
    const CUtensorMap* kv = &h->rmaps[2 * (size_t)layer];
    return kvc::launch_ragged_q8(p, sc.split ? &m : nullptr, Ksc, Vsc, kv[0], kv[1], st) == 0 ? KVC_OK : KVC_ECUDA;
}

// The arguments of kvc_call, one after the other.
struct Words {
    const int64_t* w;
    bool ok = true;
    template <class T>
    T* ptr() { return reinterpret_cast<T*>((uintptr_t)*w++); }
    int64_t i64() { return *w++; }
    int i32() {
        const int64_t x = *w++;
        ok = ok && x == (int)x;
        return (int)x;
    }
    float f32() {
        double x;
        memcpy(&x, w++, 8);
        return (float)x;
    }
};

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

int kvc_paged_append_norm_rope(kvc_t h, int layer, kvc_rope_t rope, const void* q_norm, const void* k_norm, float eps,
                               const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, const int32_t* positions,
                               int64_t pos_stride, const int32_t* block_table, const int32_t* cu_seqlens,
                               const int32_t* lens, int N, void* stream) {
    if (!h || !block_table || !cu_seqlens || !lens || N < 1) return KVC_EINVAL;
    if (!h->paged || layer < 0 || layer >= h->layers || (rope && rope->t.rot_dim > h->D)) return KVC_EINVAL;
    if (!isfinite(eps) || eps < 0 || (q_norm && !q) || !aligned(q_norm, 16) || !aligned(k_norm, 16)) return KVC_EINVAL;
    static const kvc::RopeTable still{};  // no rotation: no pairs
    const kvc::RopeTable& t = rope ? rope->t : still;
    // (the 8-bit cache's kernel takes pairs in whole 16-byte vectors)
    if (h->quant && t.rot_dim % (32 / h->es) != 0) return KVC_EUNSUPPORTED;
    if ((q == nullptr) != (q_out == nullptr)) return KVC_EINVAL;
    const int64_t qrow = (int64_t)h->H_q * h->D, krow = (int64_t)h->H_kv * h->D;
    if (q && (!packed_ok(q, q_stride, qrow, h->es) || !packed_ok(q_out, q_out_stride, qrow, h->es))) return KVC_EINVAL;
    if (q && q == q_out && q_stride != q_out_stride) return KVC_EINVAL;
    if (!packed_ok(k, k_stride, krow, h->es) || !packed_ok(v, v_stride, krow, h->es)) return KVC_EINVAL;
    if (positions && (!aligned(positions, 4) || (t.n_axes > 1 && pos_stride < N && pos_stride != 0))) return KVC_EINVAL;
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
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.eps = eps;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (h->quant) {
        p.Ksc = h->scales + (size_t)(2 * layer) * h->scale_stride;
        p.Vsc = p.Ksc + h->scale_stride;
        return kvc::launch_append8(h->dtype, p, t, h->sms, s) == 0 ? KVC_OK : KVC_ECUDA;
    }
    return kvc::launch_append_rope(h->dtype, p, t, h->sms, s) == 0 ? KVC_OK : KVC_ECUDA;
}

int kvc_paged_append_rope(kvc_t h, int layer, kvc_rope_t rope, const void* q, int64_t q_stride, void* q_out,
                          int64_t q_out_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const int32_t* positions, int64_t pos_stride, const int32_t* block_table,
                          const int32_t* cu_seqlens, const int32_t* lens, int N, void* stream) {
    if (!rope) return KVC_EINVAL;
    return kvc_paged_append_norm_rope(h, layer, rope, nullptr, nullptr, 0.f, q, q_stride, q_out, q_out_stride, k, k_stride, v,
                                      v_stride, positions, pos_stride, block_table, cu_seqlens, lens, N, stream);
}

int kvc_paged_read(kvc_t h, int layer, void* k_out, int64_t k_stride, void* v_out, int64_t v_stride,
                   const int32_t* block_table, const int32_t* cu_seqlens, const int32_t* lens, int N, void* stream) {
    if (!h || !block_table || !cu_seqlens || !lens || N < 1 || (!k_out && !v_out)) return KVC_EINVAL;
    if (!h->paged || layer < 0 || layer >= h->layers) return KVC_EINVAL;
    const int64_t row = (int64_t)h->H_kv * h->D;
    if ((k_out && !packed_ok(k_out, k_stride, row, h->es)) || (v_out && !packed_ok(v_out, v_stride, row, h->es)))
        return KVC_EINVAL;
    if (!aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(lens, 4)) return KVC_EINVAL;
    // (kernels count the 16-byte pieces of a few rows in 32 bits)
    if (row * h->es >= (int64_t(1) << 30)) return KVC_EUNSUPPORTED;
    const int rc = on_device(h);
    if (rc != KVC_OK) return rc;
    kvc::Q8Read p{};
    p.Kc = h->slab + (size_t)(2 * layer) * h->layer_bytes;
    p.Vc = h->slab + (size_t)(2 * layer + 1) * h->layer_bytes;
    if (h->quant) {
        p.Ksc = h->scales + (size_t)(2 * layer) * h->scale_stride;
        p.Vsc = p.Ksc + h->scale_stride;
    }
    p.k_out = k_out;
    p.v_out = v_out;
    p.k_ts = k_stride;
    p.v_ts = v_stride;
    p.table = block_table;
    p.cu = cu_seqlens;
    p.lens = lens;
    p.err = h->err;
    p.B = h->B;
    p.N = N;
    p.H_kv = h->H_kv;
    p.D = h->D;
    p.bs = h->bs;
    p.max_blocks = h->max_blocks;
    p.num_blocks = h->num_blocks;
    p.T_max = h->T_max;
    return kvc::launch_paged_read(h->dtype, p, static_cast<cudaStream_t>(stream)) == 0 ? KVC_OK : KVC_ECUDA;
}

int kvc_paged_attn_workspace(kvc_t h, int N, int NG, uint64_t* bytes) {
    if (!h || !bytes || !h->paged || N < 1 || NG < 0 || NG > h->B) return KVC_EINVAL;
    // enough for every path, whatever kvc_set_math does in between; on an 8-bit cache for the present one (that on CUDA
    // cores holds a layer's widened pools, which a decode step on codes would never touch)
    uint64_t most = 0;
    for (const Path path : {Path::CC, Path::TC5, Path::Q8}) {
        if (h->quant ? path != ragged_path(h) : path == Path::Q8) continue;
        const uint64_t n = scratch_of(h, N, NG, path).total;
        if (n > most) most = n;
    }
    *bytes = most;
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

int kvc_call(int call, const void* args, int n) {
    if (!args || !aligned(args, 8)) return KVC_EINVAL;
    Words a{static_cast<const int64_t*>(args)};
    switch (call) {
        case KVC_CALL_PAGED_APPEND_ROPE:
        case KVC_CALL_PAGED_APPEND_NORM_ROPE: {
            const bool norm = call == KVC_CALL_PAGED_APPEND_NORM_ROPE;
            if (n != (norm ? 21 : 18)) return KVC_EINVAL;
            kvc_cache* h = a.ptr<kvc_cache>();
            const int layer = a.i32();
            kvc_rope* rope = a.ptr<kvc_rope>();
            const void *qn = nullptr, *kn = nullptr;
            float eps = 0.f;
            if (norm) {
                qn = a.ptr<const void>();
                kn = a.ptr<const void>();
                eps = a.f32();
            }
            const void* q = a.ptr<const void>();
            const int64_t qs = a.i64();
            void* qo = a.ptr<void>();
            const int64_t qos = a.i64();
            const void* k = a.ptr<const void>();
            const int64_t ks = a.i64();
            const void* v = a.ptr<const void>();
            const int64_t vs = a.i64();
            const int32_t* pos = a.ptr<const int32_t>();
            const int64_t ps = a.i64();
            const int32_t* table = a.ptr<const int32_t>();
            const int32_t* cu = a.ptr<const int32_t>();
            const int32_t* lens = a.ptr<const int32_t>();
            const int N = a.i32();
            void* stream = a.ptr<void>();
            if (!a.ok) return KVC_EINVAL;
            return norm ? kvc_paged_append_norm_rope(h, layer, rope, qn, kn, eps, q, qs, qo, qos, k, ks, v, vs, pos, ps, table,
                                                     cu, lens, N, stream)
                        : kvc_paged_append_rope(h, layer, rope, q, qs, qo, qos, k, ks, v, vs, pos, ps, table, cu, lens, N,
                                                stream);
        }
        case KVC_CALL_PAGED_READ: {
            if (n != 11) return KVC_EINVAL;
            kvc_cache* h = a.ptr<kvc_cache>();
            const int layer = a.i32();
            void* k = a.ptr<void>();
            const int64_t ks = a.i64();
            void* v = a.ptr<void>();
            const int64_t vs = a.i64();
            const int32_t* table = a.ptr<const int32_t>();
            const int32_t* cu = a.ptr<const int32_t>();
            const int32_t* lens = a.ptr<const int32_t>();
            const int N = a.i32();
            void* stream = a.ptr<void>();
            return a.ok ? kvc_paged_read(h, layer, k, ks, v, vs, table, cu, lens, N, stream) : KVC_EINVAL;
        }
        case KVC_CALL_PAGED_ATTN_RAGGED:
        case KVC_CALL_PAGED_ATTN_SHARED: {
            const bool shared = call == KVC_CALL_PAGED_ATTN_SHARED;
            if (n != (shared ? 16 : 13)) return KVC_EINVAL;
            kvc_cache* h = a.ptr<kvc_cache>();
            const int layer = a.i32();
            const void* q = a.ptr<const void>();
            const int64_t qs = a.i64();
            void* out = a.ptr<void>();
            const int64_t os = a.i64();
            const int32_t* table = a.ptr<const int32_t>();
            const int32_t* cu = a.ptr<const int32_t>();
            const int32_t* lens = a.ptr<const int32_t>();
            const int N = a.i32();
            const int32_t *groups = nullptr, *prefix = nullptr;
            int NG = 0;
            if (shared) {
                groups = a.ptr<const int32_t>();
                prefix = a.ptr<const int32_t>();
                NG = a.i32();
            }
            void* ws = a.ptr<void>();
            const uint64_t ws_bytes = (uint64_t)a.i64();
            void* stream = a.ptr<void>();
            if (!a.ok) return KVC_EINVAL;
            return shared ? kvc_paged_attn_shared(h, layer, q, qs, out, os, table, cu, lens, N, groups, prefix, NG, ws, ws_bytes,
                                                  stream)
                          : kvc_paged_attn_ragged(h, layer, q, qs, out, os, table, cu, lens, N, ws, ws_bytes, stream);
        }
    }
    return KVC_EINVAL;
}

}  // extern "C"
