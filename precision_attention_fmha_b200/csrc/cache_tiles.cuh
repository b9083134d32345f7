// cache_tiles.cuh -- what the few-row kernels over a ragged K/V cache share:
// the lengths of a sequence, and the TMA producer that gathers 64-key tiles
// from pages (or a contiguous cache) into a shared-memory ring.
#pragma once

#include "cache_internal.h"
#include "ptx_sm100.cuh"
#include "waiter.cuh"

namespace fmha {

constexpr int kTileKeys = 64;  // keys of one ring slot
constexpr int kGroups = kTileKeys / 16;

// Keys before the query tokens' own nodes (tree: the context) and query tokens in use.
struct SeqLens {
  int len, q;
};
// Lengths outside the cache are cut to it; `bad` says so.
__device__ __forceinline__ SeqLens tree_lens(const CacheView& c, int b, bool& bad) {
  int len = __ldg(c.lens + b), q = c.q_lens != nullptr ? __ldg(c.q_lens + b) : c.T;
  bad = len < 0 || q < 0 || q > c.T || len > c.capacity - q;
  len = min(max(len, 0), c.capacity);
  q = min(max(q, 0), min(c.T, c.capacity - len));
  return {len, q};
}
__device__ __forceinline__ SeqLens seq_lens(const CacheView& c, int b, bool& bad) {
  int len = __ldg(c.lens + b), q = c.q_lens != nullptr ? __ldg(c.q_lens + b) : c.T;
  bad = len < 0 || q < 0 || q > c.T || len > c.capacity;
  len = min(max(len, 0), c.capacity);
  q = min(max(q, 0), c.T);
  return {len, q};
}

// A per-tensor or per-(sequence, KV head) scale; none: 1.
__device__ __forceinline__ float sf_of(const float* sf, int kind, int64_t bh) {
  return kind == FMHA_SF_PER_TENSOR ? __ldg(sf) : kind == FMHA_SF_PER_HEAD ? __ldg(sf + bh) : 1.f;
}

// Byte layout of one tile's K (or V) in a ring slot: rows of at most 128
// bytes, swizzled as TMA writes them; a row of 256 bytes is two such columns.
template <int D, bool E8>
struct TileLayout {
  static constexpr int ROW = D * (E8 ? 1 : 2);           // bytes of one token's row
  static constexpr int SPAN = ROW >= 128 ? 128 : 64;     // swizzle span
  static constexpr int CHUNKS = ROW / SPAN;
  static constexpr int CHUNK_ELEMS = SPAN / (E8 ? 1 : 2);
  static constexpr int CHUNK_BYTES = kTileKeys * SPAN;
  static constexpr int BYTES = kTileKeys * ROW;
  // Offset of 16-byte unit u (along D) of row r.
  __device__ static __forceinline__ uint32_t at(int r, int u) {
    if constexpr (SPAN == 128) return (u >> 3) * CHUNK_BYTES + r * 128 + (((u & 7) ^ (r & 7)) << 4);
    else return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
  }
};

// Per slot, written by the producer before the slot fills: of each 16-key
// group the first key's position and how many of its keys exist.
struct TileMeta {
  int32_t pos[kGroups];
  int32_t valid[kGroups];
};

// One 16-, 32- or 64-row piece of a tile, held by one lane of the producer warp.
struct Piece {
  int pos;    // position of its first key
  int row;    // first row inside its page (contiguous: the position)
  int outer;  // page (contiguous: the sequence)
  int valid;  // keys that exist, <= 0: none
};

__device__ __forceinline__ Piece cache_piece(const CacheView& c, int b, int pos, int limit) {
  Piece e;
  e.pos = pos;
  e.valid = limit - pos;
  e.row = pos;
  e.outer = b;
  if (c.page_table != nullptr && e.valid > 0) {
    const int pg = __ldg(c.page_table + static_cast<int64_t>(b) * c.max_pages + (pos >> c.page_shift));
    const bool ok = pg >= 0 && pg < c.num_pages;
    if (!ok) atomicOr(c.err, kErrPageIndex);
    e.outer = ok ? pg : c.num_pages;  // past the pool: TMA reads zeros
    e.row = pos & ((1 << c.page_shift) - 1);
  }
  return e;
}

}  // namespace fmha
