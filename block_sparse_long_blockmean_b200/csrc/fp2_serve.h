// fp2_serve.h -- parameters and launchers of the serving-step kernels
// (fp2_pagemap.cu, fp2_append.cu, fp2_decode.cu, fp2_decode_tiles.cu), filled in by
// fp2_serve.cu.
#pragma once

#include "fp2_internal.h"

namespace fp2 {

// Details of device-side errors beside those of the prefill kernels.
enum : uint32_t {
    kDetFree = 6,  // the free list holds fewer pages than a step needs
    kDetRow = 7,   // slot outside the cache
};

// fp2_page_map: the step's lengths in, its map out (include/fp2.h).
struct MapParams {
    int num_seqs, total_q, page_size, page_shift, max_pages, num_pages, max_seqlen_q, max_seqlen_k;
    int num_free;
    const int32_t* prefix;
    const int32_t* fresh;      // new tokens of each sequence
    const int32_t* free_pages;
    const int32_t* free_head;
    int32_t* table;
    int32_t* cu;
    int32_t* seqlens_k;
    int32_t* positions;
    int32_t* slots;
    int32_t* free_head_out;
    uint32_t* err;
};

// fp2_append: rows of the projection in, q and the cache out (include/fp2.h).
struct AppendParams {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const float *q_weight, *k_weight, *inv_freq;
    const int32_t *positions, *slots;
    void *q_out, *k_cache, *v_cache;
    const float *q_scale, *k_scale, *v_scale;
    float eps, rope_scale;
    int total_q, Hq, Hkv, d, rot, interleaved, cache_rows, fp8;
    int chunk;                 // set by the launcher: groups of heads per warp
    uint32_t* err;
};

// fp2_decode.  p holds what the launch shares with the prefill kernels.
// Partial results: slot s = one tile's rows of hc heads [hc][rows][d] fp32 in
// part, (reference, sum) pairs [hc][rows][2] in part_ml; CTA c of the split owns
// slots 2c and 2c + 1.
struct DecodeParams {
    KParams p;
    const void *q, *k, *v;
    void* out;
    float* lse;
    float* part;
    float* part_ml;
    int4* record;              // [kDecCtas][2]: what the join kernel has to do
    float qk_scale;            // log2(e) / sqrt(d)
    // set by the launchers: KV heads of an item, those of one CTA of it, groups of
    // heads, row tiles of the longest sequence, records by item (few) or by share
    int hc, hw, groups, tiles_max, few;
    int g_shift, page_shift;   // log2 of the query heads of a KV head, of page_size
    int box;                   // rows of a copy of the tile kernel
};
constexpr int kDecHeads = 2;   // most KV heads of a CTA
constexpr int kDecCtas = 444;  // most CTAs of the split: 3 on each of 148 SMs
constexpr int kDecRows = 32;   // most packed query rows (tokens x group heads) of a tile

cudaError_t launch_page_map(const MapParams& p, cudaStream_t s);
cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t s);

}  // namespace fp2
