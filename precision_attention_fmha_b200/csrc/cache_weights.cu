// cache_weights.cu -- the attention weight that each cached key has gathered:
//   w[b, h, s] (+)= sum over query tokens t and heads g of KV head h of
//                   exp(scale q_tg . k_s - lse_tg),  over the (t, s) in sight.
// The log-sum-exp comes from the attention call itself, so one product with K
// and no second normalisation is left. Each key's sum is taken by one CTA in a
// fixed order: no atomics, the same bits every time.
#include <algorithm>

#include "cache_tiles.cuh"
#include "mma_sync.cuh"

namespace fmha {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_lse2(float lse) {  // -lse in log2 units; a row that sees no key weighs nothing
  return lse == -INFINITY ? -INFINITY : -lse * kLog2e;
}

// ---- few query rows: a 64-key ring, four warps of 16 keys each (K bytes bound it) ----
// S^T = K Q^T with the keys on the 16-row side, 8 query rows at a time: a
// thread's scores are two keys' (gq, gq + 8), so the sum over rows crosses only
// the four lanes of a key.
template <int D_, bool K8_>
struct KwCfg {
  static constexpr int D = D_, MODE = WALK_KEYS;
  static constexpr bool K8 = K8_, HAS_V = false;
  using KL = TileLayout<D, K8>;
  using VL = KL;
  static constexpr int SLOT = KL::BYTES;
  static constexpr int STAGES = 65536 / SLOT > 8 ? 8 : 65536 / SLOT;
  static constexpr int SMEM = STAGES * SLOT + 2048;
  static constexpr int THREADS = 160;
};

template <class C>
__device__ void weigh(const KeyWeightsParams& p, uint8_t* ring, RingMisc<C::STAGES>* misc, const Waiter w) {
  using namespace ptx;
  constexpr int D = C::D, KS = D / 16, KF = C::K8 ? KS / 2 : KS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, j = lane & 3;
  uint32_t it = 0;
  bool ok = true;
  Walk<C::MODE> walk;
  walk.start(p);
  Seg g;
  const int rows = p.c.T * p.c.G, tiles = (rows + 7) / 8;
  while (ok && walk.next(p, g)) {
    const int64_t bh = g.b * static_cast<int64_t>(p.c.Hkv) + g.hkv;
    if (g.limit > p.n_weights && threadIdx.x == 0) atomicOr(p.c.err, kErrLength);
    const float c0 = p.scale_log2 * sf_of(p.sf_k, p.sf_k_kind, bh);
    uint32_t qf[KS][2];
    float nl[2], cs[2];
    int at[2];  // position of the tokens of rows 2 j and 2 j + 1
    auto load_rows = [&](int rt) {
      const int r = rt * 8 + gq;
      const int t = r / p.c.G;
      const int head = g.hkv * p.c.G + r - t * p.c.G;
      const bool live = t < g.nodes;  // token rows in use (r < rows follows: nodes <= T)
      const float x = live ? neg_lse2(__ldg(p.lse + (static_cast<int64_t>(g.b) * p.c.Hq + head) * p.c.T + t)) : -INFINITY;
      float f;
      load_q<C::K8, KS, 2>(qf, 0, f, p.q + g.b * p.q_sb + static_cast<int64_t>(t) * p.q_ss + head * p.q_sh, live, j);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        nl[e] = __shfl_sync(kFull, x, 4 * (2 * j + e));
        cs[e] = c0 * __shfl_sync(kFull, f, 4 * (2 * j + e));
        at[e] = g.ctx - g.nodes + __shfl_sync(kFull, t, 4 * (2 * j + e));
      }
    };
    if (tiles == 1) load_rows(0);
    // The first lane of a key writes its sum; what the weights held is fetched one tile ahead (the load's latency in every
    // tile was two thirds of a decoding step's time).
    auto fetch = [&](int u, float (&x)[2]) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = u * kTileKeys + warp * 16 + gq + 8 * e;
        x[e] = p.accumulate && j == 0 && u < g.t1 && key < min(g.limit, p.n_weights) ? p.weights[bh * p.n_weights + key] : 0.f;
      }
    };
    float old[2], ahead[2];
    fetch(g.t0, ahead);
    for (int u = g.t0; u < g.t1; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) old[e] = ahead[e];
      fetch(u + 1, ahead);
      const int s = it % C::STAGES;
      ok = __all_sync(kFull, w.wait(smem_addr(&misc->full[s]), (it / C::STAGES) & 1));
      if (!ok) break;
      ++it;
      const int valid = misc->meta[s].valid[warp], pos = misc->meta[s].pos[warp];
      uint32_t kf[KF][C::K8 ? 2 : 1][4];  // the warp's 16 keys
      if (valid > 0) {
#pragma unroll
        for (int i = 0; i < KF; ++i) load_kt<C>(kf[i], smem_addr(ring + s * C::SLOT), warp * 16, i, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&misc->empty[s]));
      if (valid <= 0) continue;
      float sum[2] = {0.f, 0.f};
      for (int rt = 0; rt < tiles; ++rt) {
        if (tiles > 1) load_rows(rt);
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains
#pragma unroll
        for (int i = 0; i < KF; ++i) {
          if constexpr (C::K8) {
            mma_f16(sc[0], kf[i][0], qf[2 * i][0], qf[2 * i][1]);
            mma_f16(sc[1], kf[i][1], qf[2 * i + 1][0], qf[2 * i + 1][1]);
          } else {
            mma_bf16(sc[i & 1], kf[i][0], qf[i][0], qf[i][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // key gq + 8 (e >> 1), row 2 j + (e & 1)
          const int key = pos + gq + 8 * (e >> 1);
          const float x = ex2(fmaf(sc[0][e] + sc[1][e], cs[e & 1], nl[e & 1]));
          // hidden: later than the row's token (a key past the end holds anything, and is not written below)
          sum[e >> 1] += (p.causal && key > at[e & 1]) || nl[e & 1] == -INFINITY ? 0.f : x;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = sum[e];
        v += __shfl_xor_sync(kFull, v, 1);
        v += __shfl_xor_sync(kFull, v, 2);
        const int k = gq + 8 * e;
        if (j == 0 && k < valid && pos + k < p.n_weights) p.weights[bh * p.n_weights + pos + k] = old[e] + v;
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 3)
    key_weights_few_kernel(const __grid_constant__ KeyWeightsParams p, const __grid_constant__ CUtensorMap tk) {
  using namespace ptx;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* misc = reinterpret_cast<RingMisc<C::STAGES>*>(ring + C::STAGES * C::SLOT);
  static_assert(sizeof(RingMisc<C::STAGES>) <= 1024, "misc area");
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_addr(&misc->full[s]), 1);
      mbar_init(smem_addr(&misc->empty[s]), 4);
    }
    misc->abort = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  const Waiter w{&misc->abort, p.c.err, p.c.wait_cycles};
  if (threadIdx.x >= 128) produce<C>(p, ring, misc, &tk, &tk, w);
  else weigh<C>(p, ring, misc, w);
  __syncthreads();
}

// ---- prompts: S^T = K Q^T on the tensor cores ----
// A CTA takes 128 keys (TMEM lanes) and streams the query tiles (128 tokens of
// one head, TMEM columns) that see them: with the keys along the lanes the sum
// over queries is a sum over a thread's own columns, and no value crosses
// threads. Per tile: 4 D / 64 tensor instructions, then 128 x 128 exponentials
// by two warpgroups, 64 columns each (one warpgroup, two warps a scheduler,
// was bound by its latencies: 290 us for 6144 tokens, the pipes half idle).
// The first keys of a causal prompt are seen by all queries and the last by
// few, so a key tile's queries are cut into runs of p.chunk tiles; two CTAs
// per SM draw (key tile, run) items from a counter, the largest first, and a
// run's sums go to the workspace, where they are added in order.
// (A share of the exponentials as polynomials on the FMA pipe made it slower:
// 285 us with a quarter, 312 with half, when it took 280 without.) 6144 tokens,
// 32 heads: 255 us, the special-function pipe 69 % busy while an SM has work.
// Scores fetched 16 columns ahead, packed multiply-adds, items looked up early
// and shorter runs (280 us at 8 tiles) did not change that.
template <int D_>
struct KmCfg {
  static constexpr int D = D_;
  static constexpr int CHUNKS = D / 64;          // 128-byte swizzle columns
  static constexpr int TILE = CHUNKS * 16384;    // 128 rows
  static constexpr int STAGES = 2;
  static constexpr int SMEM = 1024 + (1 + STAGES) * TILE + 6144;
  static constexpr int SUM_THREADS = 256, THREADS = 320;
  static constexpr int MMA_WARP = 8, LOAD_WARP = 9;
  static constexpr uint32_t TMEM_COLS = 256;     // two score buffers
  static constexpr uint32_t IDESC = ptx::make_idesc(1, 1, 1, 0, 0, 128, 128);
};
struct alignas(16) KmMisc {
  uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], nl_full[8], drain;
  uint32_t tmem_base;
  volatile uint32_t abort;
  uint32_t item[2];
  uint32_t pad[2];
  // -lse of a query tile's tokens, log2 units. Written by the query producer at
  // most 2 tiles ahead of the products, which run at most 2 ahead of a warp's
  // sums: with 8 slots, and a barrier each, neither a slot nor its barrier's
  // phase can come round again before every warp has used it.
  float nl[8][128];
  double half[128];  // the second warpgroup's sums
};
static_assert(sizeof(KmMisc) <= 6144, "misc area");

// A thread's sum over 64 tokens of one score tile (columns tS ..): its key
// against tokens t0 .., of which (EDGE) those from `first` on, in use, count.
template <bool EDGE>
__device__ __forceinline__ float weigh_tile(const SeqLens s, uint32_t tS, const float4* nl, float c, uint32_t s_free,
                                            int t0, int first) {
  using namespace ptx;
  float r0 = 0.f, r1 = 0.f, r2 = 0.f, r3 = 0.f;
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t x[32];
    tmem_ld32(tS + 32 * ch, x);
    tmem_wait_ld();
    reg_fence(x);
    if (ch == 1) {  // the scores are in registers: the next product may overwrite them
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(s_free);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 n = nl[8 * ch + i];
      float e0, e1, e2, e3;
      const uint32_t* y = &x[4 * i];
      e0 = fmaf(__uint_as_float(y[0]), c, n.x);
      e1 = fmaf(__uint_as_float(y[1]), c, n.y);
      e2 = fmaf(__uint_as_float(y[2]), c, n.z);
      e3 = fmaf(__uint_as_float(y[3]), c, n.w);
      e0 = ex2(e0); e1 = ex2(e1); e2 = ex2(e2); e3 = ex2(e3);
      if constexpr (EDGE) {
        const int t = t0 + 32 * ch + 4 * i;
        e0 = t < s.q && t >= first ? e0 : 0.f;
        e1 = t + 1 < s.q && t + 1 >= first ? e1 : 0.f;
        e2 = t + 2 < s.q && t + 2 >= first ? e2 : 0.f;
        e3 = t + 3 < s.q && t + 3 >= first ? e3 : 0.f;
      }
      fadd2(r0, r1, r0, r1, e0, e1);
      fadd2(r2, r3, r2, r3, e2, e3);
    }
  }
  return (r0 + r1) + (r2 + r3);
}

template <int D, bool K8>
__global__ void __launch_bounds__(KmCfg<D>::THREADS, 2)
    key_weights_many_kernel(const __grid_constant__ KeyWeightsParams p, const __grid_constant__ CUtensorMap tq) {
  using namespace ptx;
  using C = KmCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sK = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sK + C::TILE;
  KmMisc* misc = reinterpret_cast<KmMisc*>(sQ + C::STAGES * C::TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh_n = p.c.B * p.c.Hkv;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&misc->q_full[i]), 1);
      mbar_init(smem_addr(&misc->q_empty[i]), 1);
      mbar_init(smem_addr(&misc->s_full[i]), 2);  // the product, and the log-sum-exps that the MMA warp has seen arrive
      mbar_init(smem_addr(&misc->s_free[i]), C::SUM_THREADS / 32);
    }
    for (int i = 0; i < 8; ++i) mbar_init(smem_addr(&misc->nl_full[i]), 32);
    mbar_init(smem_addr(&misc->drain), 1);
    misc->abort = 0u;
    fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_addr(&misc->tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  // An item's keys, queries and run.
  struct Item {
    int part, kt, bh, b, hkv, key0, n_keys, base, tt0, it0, n_it;
    SeqLens s;
  };
  auto decode = [&](uint32_t item) {
    Item x;
    x.part = item % p.parts;
    const int tile = item / p.parts;
    x.kt = tile / bh_n;
    x.bh = tile - x.kt * bh_n;
    x.b = x.bh / p.c.Hkv;
    x.hkv = x.bh - x.b * p.c.Hkv;
    bool bad;
    x.s = seq_lens(p.c, x.b, bad);
    if (x.kt == 0 && x.hkv == 0 && x.part == 0 && (bad || x.s.len > p.n_weights)) atomicOr(p.c.err, kErrLength);
    x.key0 = x.kt * 128;
    x.n_keys = min(128, min(x.s.len, p.n_weights) - x.key0);
    x.base = x.s.len - x.s.q;  // position of token 0
    x.tt0 = p.causal ? max(0, x.key0 - x.base) / 128 : 0;
    const int n_tt = max(0, (x.s.q + 127) / 128 - x.tt0);
    x.it0 = x.part * p.chunk;  // this run's tiles: it0 + [0, n_it) of n_tt * G
    x.n_it = min(p.chunk, n_tt * p.c.G - x.it0);
    return x;
  };
  // The next item with work, drawn by one thread (the first run of a key tile writes its zeros even without queries).
  auto draw = [&]() {
    for (;;) {
      const uint32_t item = atomicAdd(p.ticket, 1u);
      if (item >= p.n_items) return item;
      const Item x = decode(item);
      if (x.n_keys > 0 && (x.n_it > 0 || x.part == 0)) return item;
    }
  };
  if (tid == 0) misc->item[0] = draw();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  const Waiter w{&misc->abort, p.c.err, p.c.wait_cycles};
  const bool leader = warp == C::MMA_WARP && elect_one();
  int cnt = 0;     // tiles of the items before this one: slots and phases run on
  int copies = 0;  // load warp: query tiles sent

  for (int turn = 0;; ++turn) {
    // Items in order: the first keys are seen by the most queries and start first.
    const uint32_t item = misc->item[turn & 1];
    if (item >= p.n_items) break;
    const Item x = decode(item);
    const int part = x.part, bh = x.bh, b = x.b, hkv = x.hkv, key0 = x.key0, n_keys = x.n_keys, base = x.base, tt0 = x.tt0;
    const int it0 = x.it0, n_it = x.n_it;
    const SeqLens s = x.s;
    // Query tile `it`: the copy, and the log-sum-exps of its 128 tokens (four per lane, one tile ahead in registers).
    float lse4[4];
    auto fetch_lse = [&](int it) {
      const int t = (tt0 + (it0 + it) / p.c.G) * 128 + 4 * lane, head = hkv * p.c.G + (it0 + it) % p.c.G;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        lse4[e] = it < n_it && t + e < s.q ? neg_lse2(__ldg(p.lse + (static_cast<int64_t>(b) * p.c.Hq + head) * p.c.T + t + e)) : -INFINITY;
    };
    auto send_query = [&](int it) -> bool {
      const int n = cnt + it, st = n & 1;
      if (!__all_sync(kFull, w.wait(smem_addr(&misc->q_empty[st]), ((n >> 1) & 1) ^ 1))) return false;
      const uint32_t full = smem_addr(&misc->q_full[st]);
      if (lane == 0) mbar_arrive_expect_tx(full, C::TILE);
      __syncwarp();
      const int tt = tt0 + (it0 + it) / p.c.G, head = hkv * p.c.G + (it0 + it) % p.c.G;
      if (lane < C::CHUNKS) tma_load_4d(smem_addr(sQ + st * C::TILE) + lane * 16384, &tq, full, lane * 64, head, tt * 128, b);
      *reinterpret_cast<float4*>(&misc->nl[n & 7][4 * lane]) = make_float4(lse4[0], lse4[1], lse4[2], lse4[3]);
      mbar_arrive(smem_addr(&misc->nl_full[n & 7]));
      ++copies;
      fetch_lse(it + 1);
      return true;
    };
    int sent = 0;
    bool ok = true;
    if (warp == C::LOAD_WARP) {  // the first two tiles load while the keys do
      fetch_lse(0);
      for (; sent < min(2, n_it) && ok; sent += ok) ok = send_query(sent);
    } else if (warp < C::MMA_WARP) {
      // The keys, as BF16 rows in the 128-byte swizzle (E4M3 codes are BF16 values; the scale joins the score): all of a
      // thread's 16-byte units in flight at once.
      constexpr int N = 128 * (D / 8) / C::SUM_THREADS;
      uint4 v[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = tid + k * C::SUM_THREADS, r = i / (D / 8), u = i % (D / 8);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (r < n_keys) {
          const Piece e = cache_piece(p.c, b, key0 + r, s.len);
          if (p.c.page_table == nullptr || e.outer < p.c.num_pages) {  // a bad page reads zeros
            const int64_t at = e.outer * p.k_sb + e.row * p.k_ss + hkv * p.k_sh + u * 8;
            if constexpr (K8) {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(p.k + at));
              v[k].x = x.x;
              v[k].y = x.y;
            } else {
              v[k] = __ldg(reinterpret_cast<const uint4*>(p.k + at * 2));
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int i = tid + k * C::SUM_THREADS, r = i / (D / 8), u = i % (D / 8);
        if constexpr (K8)
          v[k] = make_uint4(e4m3x2_to_bf16x2(v[k].x & 0xffffu), e4m3x2_to_bf16x2(v[k].x >> 16),
                            e4m3x2_to_bf16x2(v[k].y & 0xffffu), e4m3x2_to_bf16x2(v[k].y >> 16));
        *reinterpret_cast<uint4*>(sK + (u >> 3) * 16384 + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = v[k];
      }
      fence_proxy_async_smem();  // the tensor cores read them
    }
    __syncthreads();

    if (warp == C::LOAD_WARP) {  // query tiles
      for (; sent < n_it && ok; sent += ok) ok = send_query(sent);
      if (lane == 0) misc->item[(turn + 1) & 1] = draw();  // while the last tiles are summed
    } else if (warp == C::MMA_WARP) {  // S^T = K Q^T
      auto lo = [](uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); };
      const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
      const uint32_t k_lo = lo(smem_addr(sK)), q_lo = lo(smem_addr(sQ));
      for (int it = 0; it < n_it; ++it) {
        const int n = cnt + it, st = n & 1;
        const uint32_t ph = (n >> 1) & 1;
        if (!__all_sync(kFull, w.wait(smem_addr(&misc->q_full[st]), ph)) ||
            !__all_sync(kFull, w.wait(smem_addr(&misc->nl_full[n & 7]), (n >> 3) & 1)) ||
            !__all_sync(kFull, w.wait(smem_addr(&misc->s_free[st]), ph ^ 1)))
          break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = ((i / 4) * 16384 + (i % 4) * 32) >> 4;
            const uint32_t q = q_lo + st * (C::TILE >> 4) + off;
            if (i == 0) mma_ss_f16_lean<false>(tmem + st * 128, k_lo + off, hi, q, hi, C::IDESC);
            else mma_ss_f16_lean<true>(tmem + st * 128, k_lo + off, hi, q, hi, C::IDESC);
          }
          mbar_arrive(smem_addr(&misc->s_full[st]));
          tc_commit(smem_addr(&misc->s_full[st]));
          tc_commit(smem_addr(&misc->q_empty[st]));
        }
        __syncwarp();
      }
    } else {  // one key per thread, 64 tokens of each tile
      const int row = tid & 127, side = tid >> 7, key = key0 + row;
      const float c = p.scale_log2 * sf_of(p.sf_k, p.sf_k_kind, bh);
      const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + side * 64;
      double total = 0.0;  // 32 bits inside a tile, 64 across: a prompt's sum has tens of thousands of terms
      for (int it = 0; it < n_it; ++it) {
        const int n = cnt + it, st = n & 1;
        ok = __all_sync(kFull, w.wait(smem_addr(&misc->s_full[st]), (n >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const int t0 = (tt0 + (it0 + it) / p.c.G) * 128 + side * 64;
        const bool edge = (p.causal && base + t0 < key0 + 127) || t0 + 64 > s.q;
        const float4* nl = reinterpret_cast<const float4*>(misc->nl[n & 7]) + side * 16;
        // Two copies of the pass: only tiles at the diagonal or the end test their tokens.
        total += edge ? weigh_tile<true>(s, tS + st * 128, nl, c, smem_addr(&misc->s_free[st]), t0, p.causal ? key - base : 0)
                      : weigh_tile<false>(s, tS + st * 128, nl, c, smem_addr(&misc->s_free[st]), t0, 0);
      }
      if (side == 1) misc->half[row] = total;
      named_bar_sync(1, C::SUM_THREADS);
      if (side == 0 && ok && row < n_keys) {
        total += misc->half[row];
        const int64_t at = static_cast<int64_t>(bh) * p.n_weights + key;
        if (p.parts > 1) p.part_w[static_cast<int64_t>(part) * bh_n * p.n_weights + at] = static_cast<float>(total);
        else p.weights[at] = static_cast<float>(p.accumulate ? static_cast<double>(p.weights[at]) + total : total);
      }
    }
    cnt += max(0, n_it);
    // Every product that reads the keys is done, and the next item is there. A wait that ran out ends the loop, for all
    // threads after the same turn: whoever raised the flag did so before it came here, and the barrier carries it. (Each
    // thread's own look at the flag after the barrier could see what a faster warp raised in the next turn already, and
    // the named barriers above would then wait for warps that have left.)
    if (__syncthreads_or(misc->abort != 0u)) break;
  }
  // Every copy and product issued has ended before shared and tensor memory go away (after an abort some may be in flight).
  if (warp == C::LOAD_WARP && lane == 0)
    for (int n = max(0, copies - 2); n < copies; ++n) w.drain(smem_addr(&misc->q_full[n & 1]), (n >> 1) & 1);
  if (warp == C::MMA_WARP) {
    if (leader) tc_commit(smem_addr(&misc->drain));
    __syncwarp();
    w.drain(smem_addr(&misc->drain), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Adds the runs of each key in order.
__global__ void __launch_bounds__(256) key_weights_join_kernel(const __grid_constant__ KeyWeightsParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int key = blockIdx.x * 256 + threadIdx.x, bh = blockIdx.y, b = bh / p.c.Hkv;
  bool bad;
  const SeqLens s = seq_lens(p.c, b, bad);
  if (key >= min(s.len, p.n_weights)) return;
  const int tt0 = p.causal ? max(0, key / 128 * 128 - (s.len - s.q)) / 128 : 0;
  const int n = max(1, (max(0, (s.q + 127) / 128 - tt0) * p.c.G + p.chunk - 1) / p.chunk);
  const int64_t at = static_cast<int64_t>(bh) * p.n_weights + key, stride = static_cast<int64_t>(gridDim.y) * p.n_weights;
  float sum = p.accumulate ? p.weights[at] : 0.f;
  for (int i = 0; i < n; ++i) sum += p.part_w[i * stride + at];
  p.weights[at] = sum;
}

// The sums of a call without query rows, 1024 keys of one (sequence, KV head) at a time.
constexpr int kClearKeys = 1024;
__global__ void __launch_bounds__(256) key_weights_clear_kernel(const __grid_constant__ KeyWeightsParams p, long long items) {
  const long long heads = static_cast<long long>(p.c.B) * p.c.Hkv;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const long long run = item / heads, bh = item - run * heads;
    const int b = static_cast<int>(bh / p.c.Hkv);
    bool bad;
    const SeqLens s = seq_lens(p.c, b, bad);
    if (threadIdx.x == 0 && run == 0 && bh % p.c.Hkv == 0 && (bad || s.len > p.n_weights)) atomicOr(p.c.err, kErrLength);
    const int first = static_cast<int>(run) * kClearKeys, end = min(first + kClearKeys, min(s.len, p.n_weights));
    for (int key = first + threadIdx.x; key < end; key += 256) p.weights[bh * p.n_weights + key] = 0.f;
  }
}

template <class C>
cudaError_t launch_few(const KeyWeightsParams& p, const CUtensorMap& tk, cudaStream_t s) {
  auto kern = key_weights_few_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<p.n_ctas, C::THREADS, C::SMEM, s>>>(p, tk);
  return cudaGetLastError();
}
template <int D, bool K8>
cudaError_t launch_many(const KeyWeightsParams& p, const CUtensorMap& tq, cudaStream_t s) {
  auto kern = key_weights_many_kernel<D, K8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KmCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(p.ticket, 0, sizeof(uint32_t), s);
  if (e != cudaSuccess) return e;
  kern<<<p.n_ctas, KmCfg<D>::THREADS, KmCfg<D>::SMEM, s>>>(p, tq);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.parts == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((std::min(p.c.capacity, p.n_weights) + 255) / 256, p.c.B * p.c.Hkv);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_join_kernel, p);
}

}  // namespace

cudaError_t launch_key_weights_clear(const KeyWeightsParams& p, cudaStream_t s) {
  const long long items = static_cast<long long>(p.c.B) * p.c.Hkv * ((std::min(p.c.capacity, p.n_weights) + kClearKeys - 1LL) / kClearKeys);
  key_weights_clear_kernel<<<static_cast<unsigned>(std::min(items, 1LL << 20)), 256, 0, s>>>(p, items);
  return cudaGetLastError();
}
cudaError_t launch_key_weights_few(int D, bool k8, const KeyWeightsParams& p, const CUtensorMap& tk, cudaStream_t s) {
  if (D == 64) return k8 ? launch_few<KwCfg<64, true>>(p, tk, s) : launch_few<KwCfg<64, false>>(p, tk, s);
  return k8 ? launch_few<KwCfg<128, true>>(p, tk, s) : launch_few<KwCfg<128, false>>(p, tk, s);
}
cudaError_t launch_key_weights_many(int D, bool k8, const KeyWeightsParams& p, const CUtensorMap& tq, cudaStream_t s) {
  if (D == 64) return k8 ? launch_many<64, true>(p, tq, s) : launch_many<64, false>(p, tq, s);
  return k8 ? launch_many<128, true>(p, tq, s) : launch_many<128, false>(p, tq, s);
}

}  // namespace fmha
