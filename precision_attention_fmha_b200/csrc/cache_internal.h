// cache_internal.h -- parameters of the operators over a ragged K/V cache
// (cache_attn.cu, cache_select.cu, cache_evict.cu) and their launchers.
#pragma once

#include "fmha_internal.h"

namespace fmha {

// The cache of a ragged batch. Token s of sequence b is row s of batch row b,
// or, paged, row s % page_size of page page_table[b * max_pages + s / page_size].
struct CacheView {
  int32_t B, T, Hq, Hkv, G;  // G = Hq / Hkv query heads share a KV head
  int32_t capacity;          // tokens a sequence has room for
  const int32_t* lens;       // [B] device
  const int32_t* q_lens;     // nullable [B] device: query tokens in use (<= T)
  const int32_t* page_table; // nullptr: contiguous
  int32_t num_pages, page_shift, max_pages;
  uint32_t* err;
  uint64_t wait_cycles;
};

// A call's walk over 64-key tiles (cache_tiles.cuh).
struct CacheParams {
  CacheView c;
  int32_t piece_shift;        // log2 of the rows of one TMA copy (16, 32 or 64)
  int32_t row_tiles, tile_rows;  // tiles of query rows per KV head, and rows of one
  int32_t n_ctas;             // grid
  int32_t groups, min_tiles;  // groups of CTAs that share the list of key tiles, and the least tiles a group takes
  // picked blocks: [B, T, Hkv, top], a negative id is no block; key tiles of an item, and how CTAs share them
  const int32_t* blocks;
  int32_t top, block_shift, n_blocks;
  int32_t item_tiles, n_splits, per_split;
};

struct CacheAttnParams : CacheParams {
  const uint16_t* q; int64_t q_sb, q_ss, q_sh;  // bf16 bits
  uint16_t* o; int64_t o_sb, o_ss, o_sh;
  float* lse;  // nullable [B, Hq, T]
  float scale_log2;
  const float* sf_k; int32_t sf_k_kind;
  const float* sf_v; int32_t sf_v_kind;
  // tree: byte (b, i, j) at mask[b * mask_sb + i * T + j]; nullptr: node i sees nodes 0..i
  const uint8_t* mask; int64_t mask_sb;
  float* part_o;    // [2 * n_ctas][rows per tile][D]
  float* part_lse;  // [2 * n_ctas][rows per tile], log2 units
  // tail of a packed call: its parts ([n_parts][B, T, Hq, D], and [n_parts][B, Hq, T] in part_lse, natural log)
  int32_t n_parts;
};

// Rows (query token x head of the group) that one CTA takes at once.
inline int cache_attn_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
// CTAs of an SM: with up to 8 rows three fit its registers.
constexpr int cache_attn_ctas(int rows) { return rows <= 8 ? 3 : 2; }

cudaError_t launch_cache_attn(int D, bool k8, bool v8, const CacheAttnParams& p, const CUtensorMap& tk,
                              const CUtensorMap& tv, cudaStream_t stream);
cudaError_t launch_cache_tail(const CacheAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream);
cudaError_t launch_cache_merge(int D, const CacheAttnParams& p, cudaStream_t stream);

// Attention weight that each cached key gathers over the query tokens.
struct KeyWeightsParams : CacheParams {
  const uint16_t* q; int64_t q_sb, q_ss, q_sh;
  const uint8_t* k; int64_t k_sb, k_ss, k_sh;  // strides in elements
  const float* lse;  // [B, Hq, T]
  float* weights;    // [B, Hkv, n_weights]
  int32_t n_weights, causal, accumulate;
  // prompts: query tiles of one CTA, the most runs of them a key tile has, and (several runs) their sums
  int32_t chunk, parts;
  float* part_w;     // [parts, B, Hkv, n_weights]
  uint32_t* ticket;  // next item (key tile, run)
  uint32_t n_items;
  float scale_log2;
  const float* sf_k; int32_t sf_k_kind;
};
// tq: TMA map of q (boxes of 128 tokens of one head); tk: of k (64-key ring tiles).
cudaError_t launch_key_weights_few(int D, bool k8, const KeyWeightsParams& p, const CUtensorMap& tk, cudaStream_t s);
cudaError_t launch_key_weights_many(int D, bool k8, const KeyWeightsParams& p, const CUtensorMap& tq, cudaStream_t s);
// Without query rows: weights[b, h, s] = 0 for every key s of sequence b.
cudaError_t launch_key_weights_clear(const KeyWeightsParams& p, cudaStream_t s);

// Keys that stay in a cache under a budget.
struct EvictParams {
  CacheView c;
  const float* weights; int32_t n_weights;
  int32_t budget, sinks, recent;
  int32_t* keep;    // [B, Hkv, budget]
  int32_t* counts;  // [B]
};
cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s);

// Moves the kept rows of a cache together.
struct CompactParams {
  CacheView c;
  const uint8_t *k, *v; int64_t k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;      // strides in bytes
  uint8_t *k_out, *v_out; int64_t ko_sb, ko_ss, ko_sh, vo_sb, vo_ss, vo_sh;
  const int32_t* out_table; int32_t out_pages, out_page_shift, out_max_pages, out_capacity;
  const int32_t* keep; int64_t keep_sb, keep_sh; int32_t n_keep;
  const int32_t* counts;
  const int32_t* dst_start;  // nullable: rows go to positions dst_start[b] + i
  const float* weights; float* weights_out; int32_t n_weights, n_weights_out;  // nullable
  int32_t k_bytes, v_bytes, in_place;  // bytes of a row
};
cudaError_t launch_compact(const CompactParams& p, cudaStream_t s);

// Per-block bounds of the cached keys.
struct KeyBoundsParams {
  CacheView c;
  const uint8_t* k; int64_t k_sb, k_ss, k_sh;  // strides in elements
  uint16_t* bounds;       // bf16 [B, Hkv, n_blocks, 2, D]
  const int32_t* start;   // nullable [B]: blocks that end at or before it keep their bounds
  int32_t n_blocks, block_shift;
};
cudaError_t launch_key_bounds(int D, bool k8, const KeyBoundsParams& p, cudaStream_t stream);

// Blocks picked for each query tile.
constexpr int kMaxPickBlocks = 16384;  // their 64-bit scores fit one CTA's shared memory
struct SelectParams {
  CacheView c;
  const uint16_t* q; int64_t q_sb, q_ss, q_sh;
  const uint16_t* bounds;
  int32_t n_blocks, block_shift, top, sinks, recent;
  int32_t q_tile, n_tiles;  // query tokens that share a pick; tiles of T
  int32_t cluster;          // CTAs per item
  int32_t* list;            // [B, T, Hkv, top], or
  uint8_t* mask;            // [B, Hkv, n_tiles, n_blocks]
};
cudaError_t launch_select_blocks(int D, const SelectParams& p, cudaStream_t stream);

}  // namespace fmha
