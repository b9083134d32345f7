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

struct CacheAttnParams {
  CacheView c;
  const uint16_t* q; int64_t q_sb, q_ss, q_sh;  // bf16 bits
  uint16_t* o; int64_t o_sb, o_ss, o_sh;
  float* lse;  // nullable [B, Hq, T]
  float scale_log2;
  const float* sf_k; int32_t sf_k_kind;
  const float* sf_v; int32_t sf_v_kind;
  // tree: byte (b, i, j) at mask[b * mask_sb + i * T + j]; nullptr: node i sees nodes 0..i
  const uint8_t* mask; int64_t mask_sb;
  // picked blocks (nullptr: tree mode): [B, T, Hkv, top], a negative id is no block
  const int32_t* blocks; int32_t top, block_shift, n_blocks;
  int32_t piece_shift;  // log2 of the rows of one TMA copy (16, 32 or 64)
  int32_t row_tiles;    // row tiles of 16 * WM packed rows
  int32_t n_ctas, min_tiles;  // tree: grid, and the least key tiles a CTA takes
  int32_t item_tiles, n_splits, per_split;  // picked: key tiles of an item, and how CTAs share them
  float* part_o;    // [2 * n_ctas][rows per tile][D]
  float* part_lse;  // [2 * n_ctas][rows per tile], log2 units
};

// Rows (query token x head of the group) that one CTA takes at once: 16, 32 or 64.
inline int cache_attn_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

cudaError_t launch_cache_attn(int D, bool k8, bool v8, const CacheAttnParams& p, const CUtensorMap& tk,
                              const CUtensorMap& tv, cudaStream_t stream);
cudaError_t launch_cache_merge(int D, const CacheAttnParams& p, cudaStream_t stream);

}  // namespace fmha
