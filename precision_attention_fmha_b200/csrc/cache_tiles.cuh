// cache_tiles.cuh -- what the few-row kernels over a ragged K/V cache share:
// the lengths of a sequence, and the TMA producer that gathers 64-key tiles
// from pages (or a contiguous cache) into a shared-memory ring.
#pragma once

#include <cuda_fp16.h>

#include "cache_internal.h"
#include "mma_sync.cuh"
#include "ptx_sm100.cuh"
#include "waiter.cuh"

namespace fmha {

constexpr uint32_t kFull = 0xffffffffu;
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

// A run of key tiles [t0, t1) of one item.
struct Seg {
  int b, t, hkv, rt;
  int t0, t1, nt;
  int ctx, nodes;  // tree: context length and nodes in use; keys: cached tokens and query tokens in use
  int first;       // position of tile 0's first key
  int limit;       // keys at or past it do not exist (picked: are hidden)
};

// The list of the sequences' key tiles, shared evenly: group i of CTAs takes
// tiles [i per, (i + 1) per), each CTA of it for one (KV head, row tile). The
// heads' rows of a token lie side by side, and the CTAs of a group read them at
// about the same time, from the same DRAM pages (48 sequences of E4M3 keys, 128-byte
// rows, 452 MB: 82 us; 99 us with each head's tiles in its own part of the list).
struct Share {
  long long total;
  int per;
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// What a walk goes over: a tree's context and nodes, the keys of picked blocks
// (a fixed number of tiles per item), all keys of a sequence, or what the
// packed kernel leaves of a tree's keys: the context past its last whole 128
// keys, and the nodes (whole items only).
enum WalkMode : int { WALK_TREE = 0, WALK_PICKED = 1, WALK_KEYS = 2, WALK_TAIL = 3 };

template <int MODE>
__device__ __forceinline__ SeqLens walk_lens(const CacheView& c, int b, bool& bad) {
  return MODE == WALK_TREE || MODE == WALK_TAIL ? tree_lens(c, b, bad) : seq_lens(c, b, bad);
}
template <int MODE>
__device__ __forceinline__ int tiles_of(const SeqLens s) {
  return (s.len + (MODE == WALK_TREE ? s.q : 0) + kTileKeys - 1) / kTileKeys;
}

// Whole warp. Tiles of sequences [0, n).
template <int MODE>
__device__ long long list_tiles(const CacheParams& p, int n, bool report) {
  long long sum = 0;
  for (int b = threadIdx.x & 31; b < n; b += 32) {
    bool bad;
    sum += tiles_of<MODE>(walk_lens<MODE>(p.c, b, bad));
    if (bad && report) atomicOr(p.c.err, kErrLength);
  }
  return warp_sum(sum);
}
template <int MODE>
__device__ Share list_share(const CacheParams& p, bool report) {
  Share s;
  s.total = list_tiles<MODE>(p, p.c.B, report);
  s.per = static_cast<int>((s.total + p.groups - 1) / p.groups);
  s.per = max(s.per, p.min_tiles);
  return s;
}

// Walks a CTA's segments; every warp keeps its own copy.
template <int MODE>
struct Walk {
  long long pos, end;    // tiles of the list; picked: items
  int b;                 // current sequence, its first tile in the list and its tiles per item
  long long base;
  int nt;
  SeqLens len;

  __device__ void start(const CacheParams& p) {
    if constexpr (MODE == WALK_PICKED) {
      pos = blockIdx.x;
      end = static_cast<long long>(p.c.B) * p.c.T * p.c.Hkv * p.row_tiles * p.n_splits;
    } else if constexpr (MODE == WALK_TAIL) {
      pos = blockIdx.x;
      end = static_cast<long long>(p.c.B) * p.c.Hkv * p.row_tiles;
    } else {
      const Share s = list_share<MODE>(p, blockIdx.x == 0);
      pos = min(s.total, static_cast<long long>(blockIdx.x / (p.c.Hkv * p.row_tiles)) * s.per);
      end = min(s.total, pos + s.per);
      b = -1;
      base = 0;
      nt = 0;
    }
  }

  __device__ bool next(const CacheParams& p, Seg& g) {
    if (pos >= end) return false;
    g.first = 0;
    if constexpr (MODE == WALK_PICKED) {
      long long item = pos / p.n_splits;
      const int j = static_cast<int>(pos - item * p.n_splits);
      pos += gridDim.x;
      g.rt = static_cast<int>(item % p.row_tiles);
      item /= p.row_tiles;
      g.hkv = static_cast<int>(item % p.c.Hkv);
      item /= p.c.Hkv;
      g.t = static_cast<int>(item % p.c.T);
      g.b = static_cast<int>(item / p.c.T);
      g.nt = p.item_tiles;
      g.t0 = min(g.nt, j * p.per_split);
      g.t1 = min(g.nt, g.t0 + p.per_split);
      bool bad;
      const SeqLens s = seq_lens(p.c, g.b, bad);
      if (bad && g.t == 0 && g.hkv == 0) atomicOr(p.c.err, kErrLength);
      g.limit = g.t < s.q ? s.len - s.q + g.t + 1 : 0;
      g.ctx = 0x7fffffff;
      g.nodes = 0;
    } else if constexpr (MODE == WALK_TAIL) {
      long long item = pos;
      pos += gridDim.x;
      g.rt = static_cast<int>(item % p.row_tiles);
      item /= p.row_tiles;
      g.hkv = static_cast<int>(item % p.c.Hkv);
      g.b = static_cast<int>(item / p.c.Hkv);
      g.t = 0;
      bool bad;
      const SeqLens s = walk_lens<MODE>(p.c, g.b, bad);
      if (bad && g.hkv == 0 && g.rt == 0) atomicOr(p.c.err, kErrLength);
      g.ctx = s.len;
      g.nodes = s.q;
      g.first = s.len & ~127;
      g.limit = s.len + s.q;
      // a row tile of padding rows alone has nothing to do
      g.nt = g.rt * p.tile_rows < s.q * p.c.G ? (g.limit - g.first + kTileKeys - 1) / kTileKeys : 0;
      g.t0 = 0;
      g.t1 = g.nt;
    } else {
      const int lane = threadIdx.x & 31;
      while (b < 0 || pos >= base + nt) {
        // 32 sequences at a time: the first whose tiles reach past pos
        if (b >= 0) base += nt;
        const int first = b + 1;
        bool bad;
        const int bb = first + lane;
        const SeqLens s = bb < p.c.B ? walk_lens<MODE>(p.c, bb, bad) : SeqLens{0, 0};
        const int n = tiles_of<MODE>(s);
        int run = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(kFull, run, o);
          if (lane >= o) run += v;
        }
        const uint32_t past = __ballot_sync(kFull, base + run > pos);
        const int k = past ? __ffs(past) - 1 : 31;
        base += __shfl_sync(kFull, run - n, k);
        nt = __shfl_sync(kFull, n, k);
        len.len = __shfl_sync(kFull, s.len, k);
        len.q = __shfl_sync(kFull, s.q, k);
        b = first + k;
        if (b >= p.c.B) return false;  // not reached: pos < total
      }
      const int hr = blockIdx.x % (p.c.Hkv * p.row_tiles);
      g.b = b;
      g.t = 0;
      g.rt = hr % p.row_tiles;
      g.hkv = hr / p.row_tiles;
      g.nt = nt;
      g.t0 = static_cast<int>(pos - base);
      g.t1 = static_cast<int>(min(static_cast<long long>(nt), g.t0 + (end - pos)));
      g.ctx = len.len;
      g.nodes = len.q;
      g.limit = MODE == WALK_TREE ? len.len + len.q : len.len;
      pos += g.t1 - g.t0;
    }
    return true;
  }
};

// ---------------------------------------------------------------- producer --
// Barriers and per-slot metadata of a ring.
template <int STAGES>
struct alignas(16) RingMisc {
  uint64_t full[STAGES], empty[STAGES];
  TileMeta meta[STAGES];
  volatile uint32_t abort;
};

// The producer warp: the tiles of the CTA's walk, in order, into the ring
// (C::HAS_V: K, then V, of a tile in one slot; else K alone).
template <class C>
__device__ void produce(const CacheParams& p, uint8_t* ring, RingMisc<C::STAGES>* misc, const CUtensorMap* tk,
                        const CUtensorMap* tv, const Waiter w) {
  using namespace ptx;
  const int lane = threadIdx.x & 31;
  const int ps = p.piece_shift, ppt = kTileKeys >> ps;  // pieces per tile
  constexpr int COPIES = C::KL::CHUNKS + (C::HAS_V ? C::VL::CHUNKS : 0);
  const int my_piece = lane / COPIES, my_copy = lane - my_piece * COPIES;
  uint32_t it = 0;
  bool ok = true;
  Walk<C::MODE> walk;
  walk.start(p);
  Seg g;
  while (ok && walk.next(p, g)) {
    // Lane l holds piece `first + l` of the item; the next 32 are fetched early.
    auto fetch = [&](int i) {
      Piece e{0, 0, 0, 0};
      if (i >= g.t1 * ppt) return e;
      if constexpr (C::MODE == WALK_PICKED) {
        const int k = p.block_shift - ps;  // pieces per block, log2
        const int slot = i >> k;
        if (slot >= p.top) return e;
        const int id = __ldg(p.blocks + ((static_cast<int64_t>(g.b) * p.c.T + g.t) * p.c.Hkv + g.hkv) * p.top + slot);
        if (id >= p.n_blocks) atomicOr(p.c.err, kErrPageIndex);
        if (id < 0 || id >= p.n_blocks) return e;
        return cache_piece(p.c, g.b, (id << p.block_shift) + ((i & ((1 << k) - 1)) << ps), g.limit);
      } else {
        return cache_piece(p.c, g.b, g.first + (i << ps), g.limit);
      }
    };
    int first = g.t0 * ppt;
    Piece cur = fetch(first + lane), nxt = fetch(first + 32 + lane);
    for (int u = g.t0; u < g.t1; ++u) {
      if (u * ppt - first >= 32) {
        first += 32;
        cur = nxt;
        nxt = fetch(first + 32 + lane);
      }
      const int at = u * ppt - first;  // lane of this tile's first piece
      const int s = it % C::STAGES;
      const uint32_t ph = (it / C::STAGES) & 1;
      if (!(ok = __all_sync(kFull, w.wait(smem_addr(&misc->empty[s]), ph ^ 1)))) break;
      ++it;
      {  // lanes 0..3: the tile's 16-key groups
        const int sub = (lane & 3) << 4;
        const int src = at + (sub >> ps);
        const int pos = __shfl_sync(kFull, cur.pos, src) + (sub & ((1 << ps) - 1));
        const int valid = __shfl_sync(kFull, cur.valid, src) - (sub & ((1 << ps) - 1));
        if (lane < kGroups) {
          misc->meta[s].pos[lane] = pos;
          misc->meta[s].valid[lane] = min(16, max(0, valid));
        }
      }
      const int src = (at + my_piece) & 31;
      const int row = __shfl_sync(kFull, cur.row, src), outer = __shfl_sync(kFull, cur.outer, src);
      const bool live = __shfl_sync(kFull, cur.valid, src) > 0 && my_piece < ppt;
      const uint32_t n = __popc(__ballot_sync(kFull, live && my_copy == 0));
      const uint32_t full = smem_addr(&misc->full[s]);
      // Lane 0's arrival publishes what all four lanes wrote to meta[s] (votes and shuffles do not order memory); a tile
      // without a live piece is full at once, so no copy's latency would cover for it.
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(full, (n << ps) * (C::KL::ROW + (C::HAS_V ? C::VL::ROW : 0)));
      __syncwarp();
      if (live) {
        const uint32_t base = smem_addr(ring + s * C::SLOT);
        if (my_copy < C::KL::CHUNKS)
          tma_load_4d(base + my_copy * C::KL::CHUNK_BYTES + (my_piece << ps) * C::KL::SPAN, tk, full,
                      my_copy * C::KL::CHUNK_ELEMS, g.hkv, row, outer);
        else
          tma_load_4d(base + C::KL::BYTES + (my_copy - C::KL::CHUNKS) * C::VL::CHUNK_BYTES +
                          (my_piece << ps) * C::VL::SPAN,
                      tv, full, (my_copy - C::KL::CHUNKS) * C::VL::CHUNK_ELEMS, g.hkv, row, outer);
      }
    }
  }
  // Every copy has landed before shared memory goes away.
  if (lane == 0)
    for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; k < it; ++k)
      w.drain(smem_addr(&misc->full[k % C::STAGES]), (k / C::STAGES) & 1u);
  __syncwarp();
}

// ---------------------------------------------------------------- clusters --
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// ------------------------------------------------------------ conversions --
// One half of a 16-bit pair (F16 or BF16) in 32 bits.
template <bool F16>
__device__ __forceinline__ float half_of(uint32_t x, int hi) {
  const uint32_t h = hi ? x >> 16 : x & 0xffffu;
  if constexpr (F16) return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
  return __uint_as_float(h << 16);
}
// Two E4M3 codes as a BF16 pair (exact: 4 significant bits, exponents -9..8).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t v) {
  const uint32_t h = ptx::e4m3x2_to_f16x2(v);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return ptx::pack_bf16x2(f.x, f.y);
}

// Row h (0: gq, 1: gq + 8) of the 16 x D query fragment of a warp, from D
// BF16 values at src (live false: zeros), and the factor that its scores take.
// For E4M3 keys the contraction runs in F16, which holds the codes exactly: the
// row is brought to [1, 2) by a power of two, so it is exact too, but for
// values 2^-14 of the row's largest and smaller, which keep an absolute error
// of 2^-25 of it; and the columns of a fragment are those whose codes one
// 32-bit word of K holds (4 j .. 4 j + 3 of each 16).
// N = 4: row h of the 16-row side; N = 2: the 8-column side (h = 0, one row per lane group).
template <bool K8, int KS, int N>
__device__ __forceinline__ void load_q(uint32_t (&qf)[KS][N], int h, float& factor, const uint16_t* src, bool live,
                                       int j) {
  if constexpr (K8) {
    uint32_t raw[KS][2];
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(src + 16 * s + 4 * j)) : make_uint2(0u, 0u);
      raw[s][0] = v.x;
      raw[s][1] = v.y;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top = fmaxf(top, fabsf(half_of<false>(raw[s][e], 0)));
        top = fmaxf(top, fabsf(half_of<false>(raw[s][e], 1)));
      }
    }
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    int ex = static_cast<int>((__float_as_uint(top) >> 23) & 0xffu);
    ex = (ex == 0 || ex == 255) ? 127 : min(ex, 253);  // zero rows and infinities as they are
    const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
    factor = __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[s][h + N / 2 * e] = ptx::pack_f16x2(half_of<false>(raw[s][e], 0) * down, half_of<false>(raw[s][e], 1) * down);
  } else {
    factor = 1.f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[s][h + N / 2 * e] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * s + 8 * e + 2 * j)) : 0u;
  }
}

// K fragments as the 16-row side (16 keys): k-steps 2 s and 2 s + 1 (E4M3), or s (BF16).
template <class C>
__device__ __forceinline__ void load_kt(uint32_t (&a)[C::K8 ? 2 : 1][4], uint32_t k_base, int key0, int s, int lane) {
  using namespace ptx;
  uint32_t r[4];
  ldsm4(r, k_base + C::KL::at(key0 + (lane & 15), 2 * s + (lane >> 4)));
  if constexpr (C::K8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[h][0] = e4m3x2_to_f16x2(r[2 * h] & 0xffffu);
      a[h][1] = e4m3x2_to_f16x2(r[2 * h + 1] & 0xffffu);
      a[h][2] = e4m3x2_to_f16x2(r[2 * h] >> 16);
      a[h][3] = e4m3x2_to_f16x2(r[2 * h + 1] >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[0][i] = r[i];
  }
}

}  // namespace fmha
