// kvc_handle.cuh -- the state behind a kvc_t, shared by the host translation units of libkvc.
#pragma once

#include <vector>

#include "../../include/kvc.h"
#include "kvc_internal.cuh"

struct kvc_cache {
    int layers, B, H_q, H_kv, D, T_max, dtype, es, G;
    int device, sms;
    int ctas;          // 0 = one per SM
    int combine_mode;  // -1 = automatic
    int max_ctas;
    char* slab;        // layer l: K at (2l) * layer_bytes, V at (2l+1) * layer_bytes
    size_t layer_bytes;
    float* part_o;
    float* part_ml;
    int* counters;
    uint32_t* err;
    int math;                        // 0 automatic, 1 CUDA cores, 2 warp MMA, 3 tcgen05
    int overlap;                     // 1: early history reads before the preceding grid ends
    bool tc_ok;                      // tensor maps built (bf16 cache, rows < 2^31)
    std::vector<CUtensorMap> tmaps;  // per layer: K, V (32-row boxes), K, V (128-row boxes; 3-D
                                     // maps of whole tiles for a contiguous D = 128 cache);
                                     // paged: K, V, K, V with min(bs, 128)-row boxes
    std::vector<CUtensorMap> rmaps;  // paged bf16 pools with D = 64: per layer K, V (2-D boxes of
                                     // min(bs, 128) rows) for the ragged attention kernel
    bool paged;                      // K / V of a layer are pools [num_blocks, H_kv, bs, D]
    bool rolling;                    // T_max = window slots, position p in slot p mod T_max
    bool quant;                      // 8-bit codes + fp32 row scales (q, out, new rows in dtype)
    bool fp8;                        // the codes are E4M3 (else int8)
    float* scales;                   // int8 cache: K / V row scales of layer l at 2l, 2l + 1
    size_t scale_stride;             // floats between consecutive scale arrays (256-byte aligned)
    int bs, max_blocks, num_blocks;  // paged geometry (T_max = max_blocks * bs)
};
