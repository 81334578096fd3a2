// kvc_ragged_tc5.cu -- attention of ragged new tokens over a paged bf16 cache on the 5th-generation
// tensor cores (D = 64 or 128).
//
// The streams and their split over the CTAs are those of kvc_ragged.cuh: a tile of up to 256 query
// rows (tokens x heads of a group) against key tiles of 128.  Two sets of four softmax warps work
// on it, each with its own scores S (128 x 128 fp32, 128 columns of tensor memory), its own output O
// (128 x D fp32) and its own running state:
//   - more than 128 rows: set s takes rows [128 s, 128 s + 128); both read every K / V tile
//     from the same shared-memory copy (a K / V byte feeds 256 rows);
//   - up to 128 rows (single tokens, a small group's prefix, the last tile of a chunk): both sets
//     hold the same rows and take the key tiles in turn; their states are merged at the end of
//     the segment.  While one set does its softmax the tensor cores work for the other.
// Per tile and set: S = Q K^T (A = Q, B = K, both K-major), a thread per row loads its 128 scores,
// raises the row's reference maximum only if it grew by more than 2^8 (then O is rescaled in
// place), writes the weights as bf16 over the scores' columns, and O += P V (A = P from tensor
// memory, B = V read MN-major).  Weights as bf16: a rounding of 2^-9 per weight, at most the output's
// own rounding after the division; fp32-like weights would need a second product per tile.
// The denominator sums the unrounded weights in fp32.
//
// Warps: 0 copies (TMA), 1 issues the products, 2 walks the streams, 3 guards masked values, 4-7
// and 8-11 the two sets.  Q tiles [column block][128 rows][128 B]; K and V tiles
// [8-row group][column block][8 rows][128 B] (128-byte swizzle), one ring slot each, in the order the
// products use them.
//
// Masked values: a weight of an unseen position is 0, but 0 times an infinite or NaN value is
// NaN.  Warp 3 zeroes V rows behind the stream's end (stale or never loaded), and in the tiles of the
// causal diagonal the non-finite values of positions that some row does not see; rows that do
// see them add them at the end of the segment (a finite sum plus an infinity or NaN is that).
#include "kvc_decode_tc5.cuh"
#include "kvc_ragged_merge.cuh"

namespace kvc {

template <int D_>
struct RtCfg {
    static constexpr int D = D_;
    static constexpr int RT = 256, KT = 128;
    static constexpr int CB = D / 64;                // 128-byte column blocks of a row
    static constexpr int QTILE = 128 * D * 2;        // bytes of a Q tile (128 rows)
    static constexpr int TILE = KT * D * 2;          // bytes of a K or V tile
    static constexpr int GSTR = 1024 * CB;           // 8-row group stride of a K / V tile
    static constexpr int MISC = 3072 - 1024;         // barriers, segments, exchanged states
    static constexpr int BUDGET = 232448 - 1024;     // 227 KB less the alignment of the tiles
    static constexpr int NSLOT_A = (BUDGET - MISC - 2 * QTILE) / TILE;
    static constexpr int NSLOT = NSLOT_A > 10 ? 10 : NSLOT_A;
    static constexpr int SMEM = 2 * QTILE + NSLOT * TILE + MISC + 1024;
    static constexpr int XC = D / 2;                 // columns per exchange pass (one Q tile, fp32)
    static constexpr int THREADS = 384;
    // tensor memory columns: S of set s at 128 s, O of set s at 256 + D s
    static constexpr int TMEM_COLS = 512;
    static_assert(NSLOT >= 4, "ring too shallow");
    static_assert(NSLOT * TILE >= 2 * (MAX_B + 1) * 8, "the prefix sums lie under the ring");
};

// 32 consecutive 32-bit columns of this thread's tensor-memory lane, loaded when it returns.
__device__ __forceinline__ void tc5_ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32]; "
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 64 consecutive 32-bit columns of this thread's tensor-memory lane, loaded when it returns.
__device__ __forceinline__ void tc5_ld64(uint32_t taddr, float* v) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, "
        "%36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, "
        "%53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64]; "
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
// ... and stored (completion: tc5_wait_st).
__device__ __forceinline__ void tc5_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 "
        "[%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}; "
        :
        : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
          "r"(taddr)
        : "memory");
}

// 4-D copy of the query tile: box (64 columns, G heads, 128 / G tokens, column blocks).
__device__ __forceinline__ void tma_load_q(uint32_t dst, const CUtensorMap* map, int head, int token, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(token), "r"(0), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Item i of a segment of n key tiles, in the order the products use the tiles: true and the tile
// for V, false for K.  pair: K0 V0 K1 V1 ..; else (the sets take tiles in turn, scores two
// tiles ahead): K0 K1 V0 K2 V1 K3 .. V(n-2) V(n-1).
__device__ __forceinline__ bool ragged_item(bool pair, int n, int i, int& tile) {
    if (pair || n == 1) {
        tile = i >> 1;
        return i & 1;
    }
    if (i < 2) {
        tile = i;
        return false;
    }
    const int e = i - 2, m = 2 * (n - 2);
    if (e >= m) {
        tile = n - 2 + (e - m);
        return true;
    }
    tile = (e >> 1) + ((e & 1) ? 2 : 0);
    return !(e & 1);
}

template <int D>
struct RtMisc {
    using Seg = typename Ragged<256, 128>::Seg;
    uint64_t full[10], empty[10], vfix[10];
    uint64_t qfull, qempty, sfull[2], pfull[2], ofull[2], segfull[2], segempty[2], xch, drain;
    int64_t tmp[12];
    Seg seg[2];
    float2 xml[128];   // (m, l) of set 1's rows, for the merge of the two sets
    int nonfinite[2];  // segment parity: warp 3 took non-finite values out of V
    int abort_flag;
    uint32_t tmem;
};

template <int D>
__global__ void __launch_bounds__(384, 1)
ragged_tc5_kernel(const RaggedParams p, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV) {
    using C = RtCfg<D>;
    using R = Ragged<C::RT, C::KT>;
    using Seg = typename R::Seg;
    using Misc = RtMisc<D>;
    static_assert(sizeof(Misc) <= C::MISC, "misc area");
    extern __shared__ char rt_smem[];
    char* base = rt_smem + ((1024 - (smem_addr(rt_smem) & 1023)) & 1023);
    char* qbuf = base;
    char* ring = base + 2 * C::QTILE;
    Misc& M = *reinterpret_cast<Misc*>(ring + C::NSLOT * C::TILE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = 1 << p.lgG;
    volatile int* ab = &M.abort_flag;

    if (tid == 0) {
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&M.full[i], 1);
            mbar_init(&M.empty[i], 2);  // the products, and warp 3, which looks at every item
            mbar_init(&M.vfix[i], 1);
        }
        mbar_init(&M.qfull, 1);
        mbar_init(&M.qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&M.sfull[i], 1);
            mbar_init(&M.pfull[i], 4);
            mbar_init(&M.ofull[i], 1);
            mbar_init(&M.segfull[i], 1);
            mbar_init(&M.segempty[i], 11);  // copies, products, guard, 8 softmax warps
        }
        mbar_init(&M.xch, 8);
        mbar_init(&M.drain, 1);
        M.abort_flag = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&M.tmem)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc5_fence_before();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the split
    int64_t* gc = reinterpret_cast<int64_t*>(ring);
    int64_t* sc = gc + p.NG + 1;
    const bool valid = ragged_valid(p, tid, C::THREADS);
    int64_t x = 0, x1 = 0;
    if (valid) {
        const int64_t U = ragged_scan<C::RT, C::KT>(p, gc, sc, M.tmp, tid, C::THREADS);
        if (blockIdx.x == 0)
            for (int i = tid; i < p.NG + p.B + 2; i += C::THREADS) p.plan[i] = gc[i];
        ragged_zero_rows<__nv_bfloat16>(p, tid, C::THREADS);
        const int64_t P = ragged_ctas(U, p.P, p.min_units);
        if (blockIdx.x < P) {
            x = cta_begin(blockIdx.x, U, P);
            x1 = cta_begin(blockIdx.x + 1, U, P);
        }
    } else if (blockIdx.x == 0 && tid == 0) {
        atomicOr(p.err, DEV_BAD_SEQ);
        p.plan[p.NG] = 0;
        p.plan[p.NG + 1 + p.B] = 0;
    }
    typename R::Stream st;
    if (warp == 2 && lane == 0 && x < x1) st = R::locate(p, gc, sc, x);
    __syncthreads();  // the prefix sums are read: the ring may be filled
    tc5_fence_after();
    const uint32_t tmem = M.tmem;
    uint32_t issued = 0, qissued = 0;  // copies / products begun (copy and product threads)

    if (x < x1) {
        if (warp == 2) {
            // ================================================== streams
            if (lane == 0) {
                bool ok = true;
                for (int s = 0; ok; ++s) {
                    Seg g;
                    g.n = 0;
                    while (g.n == 0 && x < x1) {
                        g = R::segment(p, st, x, x1);
                        x = st.u0 + RAGGED_C0 + st.n;
                        if (x < x1 && !R::next(p, st)) x = x1;
                    }
                    if (s >= 2) ok = mbar_wait(&M.segempty[s & 1], ((s - 2) >> 1) & 1, ab, p.err);
                    if (!ok) break;
                    M.seg[s & 1] = g;
                    mbar_arrive(&M.segfull[s & 1]);
                    if (g.n == 0) break;
                }
            }
        } else if (warp == 0) {
            // ================================================== copies
            const uint64_t pol = policy_evict_normal();
            const int rows = p.bs < C::KT ? p.bs : C::KT;  // rows of a copied box
            const uint32_t ring_s = smem_addr(ring), q_s = smem_addr(qbuf);
            uint32_t item = 0;
            bool ok = true, last_pair = true;
            for (int s = 0; ok; ++s) {
                ok = mbar_wait(&M.segfull[s & 1], (s >> 1) & 1, ab, p.err);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                const Seg g = M.seg[s & 1];
                if (g.n == 0) break;
                const bool pair = (g.ntok << p.lgG) > 128;
                const int32_t* table = p.table + (size_t)g.seq * p.max_blocks;
                auto entry = [&](int i) {  // this lane's block of item i
                    int tile;
                    if (i >= 2 * g.n) return 0;
                    ragged_item(pair, g.n, i, tile);
                    const int t0 = g.kv0 + tile * C::KT + lane * rows;
                    return lane * rows < C::KT && t0 < g.kv_end ? __ldg(table + t0 / p.bs) : 0;
                };
                int ent = entry(0);
                if (lane == 0) {
                    // the second tile's place is also where a segment with up to 128 rows merges its sets
                    if (s > 0) ok = mbar_wait(&M.qempty, (s - 1) & 1, ab, p.err);
                    if (ok && s > 0 && pair && !last_pair)
                        ok = mbar_wait(&M.segempty[(s - 1) & 1], ((s - 1) >> 1) & 1, ab, p.err);
                    if (ok) {
                        qissued = s + 1;
                        mbar_arrive_expect_tx(&M.qfull, (pair ? 2 : 1) * C::QTILE);
                        tma_load_q(q_s, &tmQ, g.h * G, g.row0, &M.qfull);
                        if (pair) tma_load_q(q_s + C::QTILE, &tmQ, g.h * G, g.row0 + (128 >> p.lgG), &M.qfull);
                    }
                }
                last_pair = pair;
                ok = __all_sync(0xFFFFFFFFu, ok);
                for (int i = 0; ok && i < 2 * g.n; ++i, ++item) {
                    const uint32_t slot = item % C::NSLOT, use = item / C::NSLOT;
                    int tile;
                    const bool isv = ragged_item(pair, g.n, i, tile);
                    const int e0 = ent;
                    ent = entry(i + 1);
                    if (lane == 0 && use > 0) ok = mbar_wait(&M.empty[slot], (use - 1) & 1, ab, p.err);
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        ok = false;
                        break;
                    }
                    const int t0 = g.kv0 + tile * C::KT;
                    const int left = g.kv_end - t0, nbox = left >= C::KT ? C::KT / rows : (left + rows - 1) / rows;
                    if (lane == 0) mbar_arrive_expect_tx(&M.full[slot], (uint32_t)(nbox * rows * D * 2));
                    issued = item + 1;
                    __syncwarp();
                    if (lane < nbox) {
                        int e = e0;
                        if ((unsigned)e >= (unsigned)p.num_blocks) {
                            atomicOr(p.err, DEV_BAD_BLOCK);
                            e = 0;
                        }
                        const int row = (int)(((int64_t)e * p.H_kv + g.h) * p.bs + (t0 + lane * rows) % p.bs);
                        const uint32_t dst = ring_s + slot * C::TILE + lane * rows * D * 2;
                        if constexpr (D == 128) tma_load_4d(dst, isv ? &tmV : &tmK, row >> 3, rows >> 3, &M.full[slot], pol);
                        else tma_load_2d(dst, isv ? &tmV : &tmK, 0, row, &M.full[slot], pol);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&M.segempty[s & 1]);
            }
        } else if (warp == 1) {
            // ================================================== products
            if (lane == 0) {
                constexpr uint32_t ID1 = instr_desc_bf16(128, C::KT, 0, 0);
                constexpr uint32_t ID2 = instr_desc_bf16(128, D, 0, 1);
                const uint64_t dQ = smem_desc_sw128(smem_addr(qbuf), 16u, 1024u);
                const uint64_t dK = smem_desc_sw128(smem_addr(ring), 16u, C::GSTR);
                const uint64_t dV = smem_desc_sw128(smem_addr(ring), 1024u, C::GSTR);
                uint32_t item = 0, fix = 0;  // fix: parity of each slot's next guarded use
                uint32_t np[2] = {0, 0};
                bool ok = true;
                auto wait_item = [&](uint32_t it) {
                    return mbar_wait(&M.full[it % C::NSLOT], (it / C::NSLOT) & 1, ab, p.err);
                };
                auto score = [&](int set, int qt, uint32_t slot) {  // S[set] = Q tile qt . K(slot)^T
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t qo = qt * C::QTILE + (kk >> 2) * 16384 + (kk & 3) * 32;
                        const uint32_t ko = slot * C::TILE + (kk >> 2) * 1024 + (kk & 3) * 32;
                        tc5_mma(tmem + set * 128, dQ + (qo >> 4), dK + (ko >> 4), ID1, kk > 0);
                    }
                };
                auto apply = [&](int set, uint32_t slot, bool acc) {  // O[set] (+)= P[set] . V(slot)
#pragma unroll
                    for (int kk = 0; kk < C::KT / 16; ++kk) {
                        const uint32_t vo = slot * C::TILE + kk * 2 * C::GSTR;
                        tc5_mma_ta(tmem + 256 + set * D, tmem + set * 128 + kk * 8, dV + (vo >> 4), ID2,
                                   (acc || kk > 0) ? 1u : 0u);
                    }
                };
                for (int s = 0; ok; ++s) {
                    ok = mbar_wait(&M.segfull[s & 1], (s >> 1) & 1, ab, p.err);
                    if (!ok) break;
                    const Seg g = M.seg[s & 1];
                    if (g.n == 0) break;
                    const bool pair = (g.ntok << p.lgG) > 128;
                    const int n = g.n;
                    ok = mbar_wait(&M.qfull, s & 1, ab, p.err);
                    // a tile that warp 3 guards: some row does not see all of it
                    auto wait_v = [&](int tile, uint32_t it) {
                        if (!wait_item(it)) return false;
                        if (g.kv0 + (tile + 1) * C::KT > g.lim0) {
                            const uint32_t sl = it % C::NSLOT;
                            if (!mbar_wait(&M.vfix[sl], (fix >> sl) & 1, ab, p.err)) return false;
                            fix ^= 1u << sl;
                        }
                        return true;
                    };
                    auto wait_p = [&](int set) { return mbar_wait(&M.pfull[set], np[set]++ & 1, ab, p.err); };
                    issued = 1;
                    if (pair) {
                        if (!(ok = ok && wait_item(item))) break;
                        tc5_fence_after();
                        for (int set = 0; set < 2; ++set) {
                            score(set, set, item % C::NSLOT);
                            tc5_commit(&M.sfull[set]);
                        }
                        tc5_commit(&M.empty[item % C::NSLOT]);
                        ++item;
                        if (n == 1) tc5_commit(&M.qempty);
                        for (int j = 0; ok && j < n; ++j) {
                            const uint32_t vi = item, ki = item + 1;
                            if (!(ok = wait_v(j, vi))) break;
                            for (int set = 0; set < 2; ++set) {
                                if (!(ok = wait_p(set))) break;
                                tc5_fence_after();
                                apply(set, vi % C::NSLOT, j > 0);
                                if (j + 1 == n) tc5_commit(&M.ofull[set]);
                                if (set == 1) tc5_commit(&M.empty[vi % C::NSLOT]);
                                if (j + 1 < n) {
                                    if (set == 0 && !(ok = wait_item(ki))) break;
                                    tc5_fence_after();
                                    score(set, set, ki % C::NSLOT);
                                    tc5_commit(&M.sfull[set]);
                                    if (set == 1) tc5_commit(&M.empty[ki % C::NSLOT]);
                                }
                            }
                            item += j + 1 < n ? 2 : 1;
                            if (j + 2 == n) tc5_commit(&M.qempty);
                        }
                    } else {
                        for (int j = 0; ok && j < 2 && j < n; ++j, ++item) {
                            if (!(ok = wait_item(item))) break;
                            tc5_fence_after();
                            score(j, 0, item % C::NSLOT);
                            tc5_commit(&M.sfull[j]);
                            tc5_commit(&M.empty[item % C::NSLOT]);
                        }
                        if (n <= 2) tc5_commit(&M.qempty);
                        for (int j = 0; ok && j < n; ++j) {
                            const int set = j & 1;
                            if (!(ok = wait_v(j, item) && wait_p(set))) break;
                            tc5_fence_after();
                            apply(set, item % C::NSLOT, j >= 2);
                            if (j + 2 >= n) tc5_commit(&M.ofull[set]);
                            tc5_commit(&M.empty[item % C::NSLOT]);
                            ++item;
                            if (j + 2 < n) {
                                if (!(ok = wait_item(item))) break;
                                tc5_fence_after();
                                score(set, 0, item % C::NSLOT);
                                tc5_commit(&M.sfull[set]);
                                tc5_commit(&M.empty[item % C::NSLOT]);
                                ++item;
                                if (j + 3 == n) tc5_commit(&M.qempty);
                            }
                        }
                    }
                    if (ok) mbar_arrive(&M.segempty[s & 1]);
                }
            }
        } else if (warp == 3) {
            // ================================================== masked values
            uint32_t item = 0;
            bool ok = true;
            for (int s = 0; ok; ++s) {
                ok = mbar_wait(&M.segfull[s & 1], (s >> 1) & 1, ab, p.err);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                const Seg g = M.seg[s & 1];
                if (g.n == 0) break;
                const bool pair = (g.ntok << p.lgG) > 128;
                if (lane == 0) M.nonfinite[s & 1] = 0;
                __syncwarp();
                for (int i = 0; i < 2 * g.n; ++i, ++item) {
                    const uint32_t slot = item % C::NSLOT;
                    int tile;
                    const bool isv = ragged_item(pair, g.n, i, tile);
                        // every item is waited for in turn and held until it has been seen: a barrier's
                    // parity tells only neighbouring uses apart
                    ok = mbar_wait(&M.full[slot], (item / C::NSLOT) & 1, ab, p.err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const int t0 = g.kv0 + tile * C::KT;
                    if (!isv || t0 + C::KT <= g.lim0) {
                        if (lane == 0) mbar_arrive(&M.empty[slot]);
                        continue;
                    }
                    char* v = ring + slot * C::TILE;
                    const int end = g.kv_end - t0, first = g.lim0 > t0 ? g.lim0 - t0 : 0;
                    bool found = false;
                    for (int c = lane; c < (C::KT - first) * C::CB * 8; c += 32) {
                        const int r = first + c / (C::CB * 8), w = c % (C::CB * 8);
                        uint4* a = reinterpret_cast<uint4*>(v + (r >> 3) * C::GSTR + (w >> 3) * 1024 + (r & 7) * 128 +
                                                            (w & 7) * 16);
                        if (r >= end) {
                            *a = make_uint4(0, 0, 0, 0);
                        } else {
                            uint4 d = *a;
                            uint32_t* u = reinterpret_cast<uint32_t*>(&d);
                            bool hit = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((u[k] & 0x7F80u) == 0x7F80u) { u[k] &= 0xFFFF0000u; hit = true; }
                                if ((u[k] & 0x7F800000u) == 0x7F800000u) { u[k] &= 0xFFFFu; hit = true; }
                            }
                            if (hit) *a = d;
                            found |= hit;
                        }
                    }
                    if (found) M.nonfinite[s & 1] = 1;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&M.vfix[slot]);
                        mbar_arrive(&M.empty[slot]);
                    }
                }
                if (ok && lane == 0) mbar_arrive(&M.segempty[s & 1]);
            }
        } else {
            // ================================================== softmax and output
            const int set = warp >= 8 ? 1 : 0, quad = warp & 3;
            const int r128 = quad * 32 + lane;
            const uint32_t lanes = (uint32_t)(quad * 32) << 16;
            const uint32_t tS = tmem + set * 128 + lanes, tO = tmem + 256 + set * D + lanes;
            const float c = p.qscale;
            uint32_t ns = 0, no = 0, nx = 0;
            bool ok = true;
            for (int s = 0; ok; ++s) {
                ok = mbar_wait(&M.segfull[s & 1], (s >> 1) & 1, ab, p.err);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                const Seg g = M.seg[s & 1];
                if (g.n == 0) break;
                const int nrow = g.ntok << p.lgG;
                const bool pair = nrow > 128;
                const int r = (pair ? set * 128 : 0) + r128;  // row of the stream's tile
                const int rw = r - lane;                      // the warp's first row: it sees least
                const int limit = min(g.kv_end, g.lim0 + g.causal * (r >> p.lgG));
                const int limit_w = min(g.kv_end, g.lim0 + g.causal * (rw >> p.lgG));
                float m = -INFINITY, l = 0.f;  // reference maximum of the raw scores, sum of weights
                const int step = pair ? 1 : 2;
                int j0 = pair ? 0 : set;
                for (int j = j0; j < g.n; j += step) {
                    ok = mbar_wait(&M.sfull[set], ns & 1, ab, p.err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    ++ns;
                    tc5_fence_after();
                    const int t0 = g.kv0 + j * C::KT;
                    float v[128];
                    tc5_ld64(tS, v);
                    tc5_ld64(tS + 64, v + 64);
                    if (t0 + C::KT > limit_w) {
                        const int see = limit - t0;
#pragma unroll
                        for (int i = 0; i < 128; ++i) v[i] = i < see ? v[i] : -INFINITY;
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int i = 4; i < 128; i += 4) {
                        mx[0] = fmaxf(mx[0], v[i]);
                        mx[1] = fmaxf(mx[1], v[i + 1]);
                        mx[2] = fmaxf(mx[2], v[i + 2]);
                        mx[3] = fmaxf(mx[3], v[i + 3]);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // weights up to 2^8 against the reference keep their relative precision
                    const bool raise = (top - m) * c > 8.f;
                    if (__any_sync(0xFFFFFFFFu, raise)) {
                        const float mn = raise ? top : m;
                        const float f = raise ? fast_exp2((m - mn) * c) : 1.f;
                        if (j != j0) {
                            // the products into O so far are complete (S of this tile came behind them)
                            for (int d = 0; d < D; d += 32) {
                                float o[32];
                                tc5_ld32(tO + d, o);
                                uint32_t u[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
                                tc5_st32(tO + d, u);
                            }
                        }
                        l *= f;
                        m = mn;
                    }
                    const float mc = m == -INFINITY ? 0.f : -m * c;  // nothing seen yet: weights 2^-inf = 0
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 c2 = make_float2(c, c), mc2 = make_float2(mc, mc);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 a = __ffma2_rn(make_float2(v[hf * 64 + 2 * i], v[hf * 64 + 2 * i + 1]), c2, mc2);
                            const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                            sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                            w[i] = bf16x2_rn(e.x, e.y);
                        }
                        tc5_st32(tS + hf * 32, w);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tc5_wait_st();
                    tc5_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&M.pfull[set]);
                }
                if (!ok) break;
                // ---- the segment's state
                const bool mine = j0 < g.n;
                if (mine) {
                    ok = mbar_wait(&M.ofull[set], no & 1, ab, p.err);
                    ++no;
                    tc5_fence_after();
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                const bool merge = !pair && g.n > 1;  // set 1's state goes to set 0
                auto meet = [&] {  // both sets (a bounded wait: one of them may have given up)
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&M.xch);
                    ok = mbar_wait(&M.xch, nx++ & 1, ab, p.err) && ok;
                    ok = __all_sync(0xFFFFFFFFu, ok);
                };
                float f0 = 1.f, f1 = 0.f;
                float* xbuf = reinterpret_cast<float*>(qbuf + C::QTILE);
                if (merge && set == 1) M.xml[r128] = make_float2(m, l);
                const bool writes = r < nrow && (pair || set == 0);
                const int64_t row = g.row0 + (r >> p.lgG);
                const int head = g.h * G + (r & (G - 1));
                const bool nonfin = *(volatile int*)&M.nonfinite[s & 1] != 0;
#pragma unroll 1
                for (int pass = 0; pass < 2; ++pass) {
                    if (merge) {
                        if (set == 1 && ok) {
#pragma unroll 1
                            for (int d = 0; d < C::XC; d += 32) {
                                float o[32];
                                __syncwarp();
                                tc5_ld32(tO + pass * C::XC + d, o);
                                if (r < nrow)
#pragma unroll
                                    for (int i = 0; i < 32; i += 4)
                                        *reinterpret_cast<float4*>(xbuf + ((d + i) / 4 * 128 + r128) * 4) =
                                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            }
                        }
                        meet();
                        if (set == 0 && pass == 0) {
                            const float2 b = M.xml[r128];
                            const float mm = fmaxf(m, b.x), mu = mm == -INFINITY ? 0.f : mm;
                            f0 = fast_exp2((m - mu) * c);
                            f1 = b.y == 0.f ? 0.f : fast_exp2((b.x - mu) * c);
                            if (l == 0.f) f0 = 0.f;
                            l = l * f0 + b.y * f1;
                            m = mm;
                        }
                    }
                    if ((pair || set == 0) && ok) {
                        const float inv = g.dst == 0 ? 1.f / l : 1.f;
                        float *po = nullptr, *pml = nullptr;
                        if (g.dst != 0) {
                            ragged_dst(p, g, blockIdx.x, r, row, head, po, pml);
                            if (writes && pass == 0) *reinterpret_cast<float2*>(pml) = make_float2(m * c, l);
                        }
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_ts + (int64_t)head * D;
#pragma unroll 1
                        for (int d = 0; d < C::XC; d += 32) {
                            const int col = pass * C::XC + d;
                            float o[32];
                            __syncwarp();
                            tc5_ld32(tO + col, o);
                            if (writes) {
                                if (merge) {
#pragma unroll
                                    for (int i = 0; i < 32; i += 4) {
                                        const float4 b = *reinterpret_cast<const float4*>(xbuf + ((d + i) / 4 * 128 + r128) * 4);
                                        o[i] = o[i] * f0 + b.x * f1;
                                        o[i + 1] = o[i + 1] * f0 + b.y * f1;
                                        o[i + 2] = o[i + 2] * f0 + b.z * f1;
                                        o[i + 3] = o[i + 3] * f0 + b.w * f1;
                                    }
                                }
                                if (nonfin) {
                                    // the values warp 3 took out of tiles this row sees part of
                                    const int a = max(g.lim0, g.kv0), b = min(limit, g.kv0 + g.n * C::KT);
                                    for (int t = a; t < b; ++t) {
                                        const int64_t vr = cache_row_rd(p.table, p.bs, p.max_blocks, p.num_blocks, p.H_kv,
                                                                        p.T_max, g.seq, g.h, t, p.err);
                                        const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.V) + vr * D + col;
#pragma unroll
                                        for (int i = 0; i < 32; ++i) {
                                            const float x = __bfloat162float(vp[i]);
                                            if (!isfinite(x)) o[i] += x;
                                        }
                                    }
                                }
                                if (g.dst == 0) {
#pragma unroll
                                    for (int i = 0; i < 32; i += 8)
                                        *reinterpret_cast<uint4*>(out + col + i) =
                                            make_uint4(bf16x2_rn(o[i] * inv, o[i + 1] * inv), bf16x2_rn(o[i + 2] * inv, o[i + 3] * inv),
                                                       bf16x2_rn(o[i + 4] * inv, o[i + 5] * inv),
                                                       bf16x2_rn(o[i + 6] * inv, o[i + 7] * inv));
                                } else {
#pragma unroll
                                    for (int i = 0; i < 32; i += 4)
                                        *reinterpret_cast<float4*>(po + col + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                                }
                            }
                        }
                    }
                    if (merge) meet();
                }
                tc5_fence_before();
                fence_async_smem();  // the exchange area is filled by copies next
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&M.segempty[s & 1]);
            }
        }
    }
    __syncwarp();
    __syncthreads();  // every role is out of its loop (all waits are bounded)
    if (*ab) {
        // a wait timed out: let issued copies and products land, bounded
        if (tid == 0) {
            if (qissued > 0) {
                const uint64_t t = global_ns();
                while (!mbar_try_wait(&M.qfull, (qissued - 1) & 1) && global_ns() - t < WAIT_LIMIT_NS) {
                }
            }
            const uint32_t n = issued;
            for (uint32_t it = n > C::NSLOT ? n - C::NSLOT : 0; it < n; ++it) {
                const uint64_t t = global_ns();
                while (!mbar_try_wait(&M.full[it % C::NSLOT], (it / C::NSLOT) & 1) && global_ns() - t < WAIT_LIMIT_NS) {
                }
            }
        }
        if (tid == 32 && issued > 0) {
            tc5_commit(&M.drain);
            const uint64_t t = global_ns();
            while (!mbar_try_wait(&M.drain, 0) && global_ns() - t < WAIT_LIMIT_NS) {
            }
        }
    }
    tc5_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc5_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
    }
}

template <int D>
static int launch_rt(const RaggedParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    using C = RtCfg<D>;
    static PerDeviceOnce once;
    const int e0 = once.run([] {
        return (int)cudaFuncSetAttribute(ragged_tc5_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e0 != 0) return e0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)p.P);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ragged_tc5_kernel<D>, p, q, k, v);
    if (e != cudaSuccess) return (int)e;
    return launch_merge<__nv_bfloat16, C::RT, C::KT>(p, s);
}

int launch_ragged_tc5(const RaggedParams& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                      cudaStream_t s) {
    return p.D == 128 ? launch_rt<128>(p, q, k, v, s) : launch_rt<64>(p, q, k, v, s);
}

}  // namespace kvc
