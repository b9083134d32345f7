// cache_weights.cu -- the attention weight that each cached key has gathered:
//   w[b, h, s] (+)= sum over query tokens t and heads g of KV head h of
//                   exp(scale q_tg . k_s - lse_tg),  over the (t, s) in sight.
// The log-sum-exp comes from the attention call itself, so one product with K
// and no second normalisation is left. Each key's sum is taken by one CTA in a
// fixed order: no atomics, the same bits every time.
#include "cache_tiles.cuh"
#include "mma_sync.cuh"

namespace fmha {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float neg_lse2(float lse) {  // -lse in log2 units; a row that sees no key weighs nothing
  return lse == -INFINITY ? -INFINITY : -lse * kLog2e;
}

// ---- few query rows: a 64-key ring, four warps of 16 keys each (K bytes bound it) ----
template <int D_, bool K8_>
struct KwCfg {
  static constexpr int D = D_, MODE = WALK_KEYS;
  static constexpr bool K8 = K8_, HAS_V = false;
  using KL = TileLayout<D, K8>;
  using VL = KL;
  static constexpr int SLOT = KL::BYTES;
  static constexpr int STAGES = 6;
  static constexpr int SMEM = STAGES * SLOT + 2048;
  static constexpr int THREADS = 160;
};

template <class C>
__device__ void weigh(const KeyWeightsParams& p, uint8_t* ring, RingMisc<C::STAGES>* misc, const Waiter w) {
  using namespace ptx;
  constexpr int D = C::D, KS = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, j = lane & 3;
  uint32_t it = 0;
  bool ok = true;
  Walk<C::MODE> walk;
  walk.start(p);
  Seg g;
  const int rows = p.c.T * p.c.G, tiles = (rows + 15) / 16;
  while (ok && walk.next(p, g)) {
    const int64_t bh = g.b * static_cast<int64_t>(p.c.Hkv) + g.hkv;
    if (g.limit > p.n_weights && threadIdx.x == 0) atomicOr(p.c.err, kErrLength);
    const float c0 = p.scale_log2 * sf_of(p.sf_k, p.sf_k_kind, bh);
    uint32_t qf[KS][4];
    float nl[2], cs[2];
    int at[2];  // position of the rows' tokens
    auto load_rows = [&](int rt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = rt * 16 + gq + 8 * h;
        const int t = r / p.c.G;
        const int head = g.hkv * p.c.G + r - t * p.c.G;
        const bool live = t < g.nodes;  // token rows in use (r < rows follows: nodes <= T)
        at[h] = g.ctx - g.nodes + t;
        nl[h] = live ? neg_lse2(__ldg(p.lse + (static_cast<int64_t>(g.b) * p.c.Hq + head) * p.c.T + t)) : -INFINITY;
        load_q<C::K8, KS, 4>(qf, h, cs[h], p.q + g.b * p.q_sb + static_cast<int64_t>(t) * p.q_ss + head * p.q_sh, live, j);
        cs[h] *= c0;
      }
    };
    if (tiles == 1) load_rows(0);
    // Lanes of the first row group hold the sums of keys 2 j, 2 j + 1, 2 j + 8, 2 j + 9; what the weights held is
    // fetched one tile ahead (the load's latency in every tile was two thirds of a decoding step's time).
    auto fetch = [&](int u, float (&x)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = u * kTileKeys + warp * 16 + 8 * (e >> 1) + 2 * j + (e & 1);
        x[e] = p.accumulate && gq == 0 && u < g.t1 && key < min(g.limit, p.n_weights) ? p.weights[bh * p.n_weights + key] : 0.f;
      }
    };
    float old[4], ahead[4];
    fetch(g.t0, ahead);
    for (int u = g.t0; u < g.t1; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) old[e] = ahead[e];
      fetch(u + 1, ahead);
      const int s = it % C::STAGES;
      ok = __all_sync(kFull, w.wait(smem_addr(&misc->full[s]), (it / C::STAGES) & 1));
      if (!ok) break;
      ++it;
      const uint32_t k_base = smem_addr(ring + s * C::SLOT);
      const int valid = misc->meta[s].valid[warp], pos = misc->meta[s].pos[warp];
      uint32_t kb[C::K8 ? KS / 2 : KS][4];  // the warp's 16 keys
      if (valid > 0) {
        const int row = warp * 16 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int i = 0; i < (C::K8 ? KS / 2 : KS); ++i) ldsm4(kb[i], k_base + C::KL::at(row, 2 * i + ((lane >> 3) & 1)));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&misc->empty[s]));
      if (valid <= 0) continue;
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      for (int rt = 0; rt < tiles; ++rt) {
        if (tiles > 1) load_rows(rt);
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if constexpr (C::K8) {
            if (i % 2 == 0) mma_k8<KS>(sc[0], sc[1], qf, i / 2, kb[i / 2]);
          } else {
            mma_bf16(sc[0], qf[i], kb[i][0], kb[i][1]);
            mma_bf16(sc[1], qf[i], kb[i][2], kb[i][3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = pos + 8 * i + 2 * j + (e & 1);
            const float x = ex2(fmaf(sc[i][e], cs[e >> 1], nl[e >> 1]));
            // hidden: later than the row's token (a key past the end holds anything, and is not written below)
            sum[i][e & 1] += (p.causal && key > at[e >> 1]) || nl[e >> 1] == -INFINITY ? 0.f : x;
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = sum[i][e];
          v += __shfl_xor_sync(kFull, v, 4);
          v += __shfl_xor_sync(kFull, v, 8);
          v += __shfl_xor_sync(kFull, v, 16);
          const int k = 8 * i + 2 * j + e;
          if (gq == 0 && k < valid && pos + k < p.n_weights) p.weights[bh * p.n_weights + pos + k] = old[2 * i + e] + v;
        }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 2)
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
// A CTA owns 128 keys (TMEM lanes) and streams the query tiles (128 tokens of
// one head, TMEM columns) that see them: with the keys along the lanes the sum
// over queries is a sum over a thread's own columns, and no value crosses
// threads. Per tile: 4 D / 64 tensor instructions, then 128 x 128 exponentials.
template <int D_>
struct KmCfg {
  static constexpr int D = D_;
  static constexpr int CHUNKS = D / 64;          // 128-byte swizzle columns
  static constexpr int TILE = CHUNKS * 16384;    // 128 rows
  static constexpr int STAGES = 2;
  static constexpr int SMEM = 1024 + (1 + STAGES) * TILE + 2048;
  static constexpr int THREADS = 192;
  static constexpr uint32_t TMEM_COLS = 256;     // two score buffers
  static constexpr uint32_t IDESC = ptx::make_idesc(1, 1, 1, 0, 0, 128, 128);
};
struct alignas(16) KmMisc {
  uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], drain;
  uint32_t tmem_base;
  volatile uint32_t abort;
  float nl[2][128];
};

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
  // Key tiles in order: the first are seen by the most queries and start first.
  const int bh_n = p.c.B * p.c.Hkv;
  const int kt = blockIdx.x / bh_n, bh = blockIdx.x - kt * bh_n;
  const int b = bh / p.c.Hkv, hkv = bh - b * p.c.Hkv;
  bool bad;
  const SeqLens s = seq_lens(p.c, b, bad);
  if (kt == 0 && hkv == 0 && tid == 0 && (bad || s.len > p.n_weights)) atomicOr(p.c.err, kErrLength);
  const int key0 = kt * 128;
  const int n_keys = min(128, min(s.len, p.n_weights) - key0);
  if (n_keys <= 0) return;
  const int base = s.len - s.q;  // position of token 0
  const int tt0 = p.causal ? max(0, key0 - base) / 128 : 0;
  const int n_tt = max(0, (s.q + 127) / 128 - tt0);
  const int n_it = n_tt * p.c.G;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&misc->q_full[i]), 1);
      mbar_init(smem_addr(&misc->q_empty[i]), 1);
      mbar_init(smem_addr(&misc->s_full[i]), 1);
      mbar_init(smem_addr(&misc->s_free[i]), 4);
    }
    mbar_init(smem_addr(&misc->drain), 1);
    misc->abort = 0u;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(smem_addr(&misc->tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  // The keys, as BF16 rows in the 128-byte swizzle (E4M3 codes are BF16 values; the scale joins the score).
  for (int i = tid; i < 128 * (D / 8); i += C::THREADS) {
    const int r = i / (D / 8), u = i % (D / 8);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < n_keys) {
      const Piece e = cache_piece(p.c, b, key0 + r, s.len);
      if (p.c.page_table == nullptr || e.outer < p.c.num_pages) {  // a bad page reads zeros
        const int64_t at = e.outer * p.k_sb + e.row * p.k_ss + hkv * p.k_sh + u * 8;
        if constexpr (K8) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(p.k + at));
          v = make_uint4(e4m3x2_to_bf16x2(x.x & 0xffffu), e4m3x2_to_bf16x2(x.x >> 16), e4m3x2_to_bf16x2(x.y & 0xffffu),
                         e4m3x2_to_bf16x2(x.y >> 16));
        } else {
          v = __ldg(reinterpret_cast<const uint4*>(p.k + at * 2));
        }
      }
    }
    *reinterpret_cast<uint4*>(sK + (u >> 3) * 16384 + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = v;
  }
  fence_proxy_async_smem();  // the tensor cores read them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  const Waiter w{&misc->abort, p.c.err, p.c.wait_cycles};

  if (warp == 5) {  // query tiles
    bool ok = true;
    int it = 0;
    for (; it < n_it && ok; ++it) {
      const int st = it & 1;
      ok = __all_sync(kFull, w.wait(smem_addr(&misc->q_empty[st]), ((it >> 1) & 1) ^ 1));
      if (!ok) break;
      const uint32_t full = smem_addr(&misc->q_full[st]);
      if (lane == 0) mbar_arrive_expect_tx(full, C::TILE);
      __syncwarp();
      const int tt = tt0 + it / p.c.G, head = hkv * p.c.G + it % p.c.G;
      if (lane < C::CHUNKS) tma_load_4d(smem_addr(sQ + st * C::TILE) + lane * 16384, &tq, full, lane * 64, head, tt * 128, b);
    }
    if (lane == 0)
      for (int k = it > 2 ? it - 2 : 0; k < it; ++k) w.drain(smem_addr(&misc->q_full[k & 1]), (k >> 1) & 1);
    __syncwarp();
  } else if (warp == 4) {  // S^T = K Q^T
    const bool leader = elect_one();
    auto lo = [](uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); };
    const uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    const uint32_t k_lo = lo(smem_addr(sK)), q_lo = lo(smem_addr(sQ));
    bool ok = true;
    for (int it = 0; it < n_it && ok; ++it) {
      const int st = it & 1;
      const uint32_t ph = (it >> 1) & 1;
      ok = __all_sync(kFull, w.wait(smem_addr(&misc->q_full[st]), ph)) &&
           __all_sync(kFull, w.wait(smem_addr(&misc->s_free[st]), ph ^ 1));
      if (!ok) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = ((i / 4) * 16384 + (i % 4) * 32) >> 4;
          const uint32_t q = q_lo + st * (C::TILE >> 4) + off;
          if (i == 0) mma_ss_f16_lean<false>(tmem + st * 128, k_lo + off, hi, q, hi, C::IDESC);
          else mma_ss_f16_lean<true>(tmem + st * 128, k_lo + off, hi, q, hi, C::IDESC);
        }
        tc_commit(smem_addr(&misc->s_full[st]));
        tc_commit(smem_addr(&misc->q_empty[st]));
      }
      __syncwarp();
    }
    if (leader) tc_commit(smem_addr(&misc->drain));
    __syncwarp();
    w.drain(smem_addr(&misc->drain), 0);
  } else {  // one key per thread
    const int key = key0 + tid;
    const float c = p.scale_log2 * sf_of(p.sf_k, p.sf_k_kind, bh);
    const uint32_t tS = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    auto lse_of = [&](int it) {
      const int t = (tt0 + it / p.c.G) * 128 + tid, head = hkv * p.c.G + it % p.c.G;
      return it < n_it && t < s.q ? neg_lse2(__ldg(p.lse + (static_cast<int64_t>(b) * p.c.Hq + head) * p.c.T + t)) : -INFINITY;
    };
    double total = 0.0;  // 32 bits inside a tile, 64 across: a prompt's sum has tens of thousands of terms
    float next = lse_of(0);
    bool ok = true;
    for (int it = 0; it < n_it; ++it) {
      const int st = it & 1;
      misc->nl[st][tid] = next;
      named_bar_sync(1, 128);
      next = lse_of(it + 1);
      if (ok) ok = __all_sync(kFull, w.wait(smem_addr(&misc->s_full[st]), (it >> 1) & 1));
      if (!ok) continue;  // an aborted CTA keeps the barrier count
      tc_fence_after();
      const int t0 = (tt0 + it / p.c.G) * 128;
      const bool edge = (p.causal && base + t0 < key0 + 127) || t0 + 128 > s.q;
      const float4* nl = reinterpret_cast<const float4*>(misc->nl[st]);
      float r0 = 0.f, r1 = 0.f, r2 = 0.f, r3 = 0.f;
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t x[32];
        tmem_ld32(tS + st * 128 + 32 * ch, x);
        tmem_wait_ld();
        reg_fence(x);
        if (ch == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&misc->s_free[st]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 n = nl[8 * ch + i];
          float e0, e1, e2, e3;
          ffma2(e0, e1, __uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]), c, c, n.x, n.y);
          ffma2(e2, e3, __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]), c, c, n.z, n.w);
          e0 = ex2(e0); e1 = ex2(e1); e2 = ex2(e2); e3 = ex2(e3);
          if (edge) {
            const int t = t0 + 32 * ch + 4 * i;  // token in use, and not before this key
            const int first = p.causal ? key - base : 0;
            e0 = t < s.q && t >= first ? e0 : 0.f;
            e1 = t + 1 < s.q && t + 1 >= first ? e1 : 0.f;
            e2 = t + 2 < s.q && t + 2 >= first ? e2 : 0.f;
            e3 = t + 3 < s.q && t + 3 >= first ? e3 : 0.f;
          }
          fadd2(r0, r1, r0, r1, e0, e1);
          fadd2(r2, r3, r2, r3, e2, e3);
        }
      }
      total += static_cast<double>((r0 + r1) + (r2 + r3));
    }
    if (ok && tid < n_keys) {
      float* dst = p.weights + static_cast<int64_t>(bh) * p.n_weights + key;
      *dst = static_cast<float>(p.accumulate ? static_cast<double>(*dst) + total : total);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
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
  kern<<<p.n_ctas, KmCfg<D>::THREADS, KmCfg<D>::SMEM, s>>>(p, tq);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights_few(int D, bool k8, const KeyWeightsParams& p, const CUtensorMap& tk, cudaStream_t s) {
  if (D == 64) return k8 ? launch_few<KwCfg<64, true>>(p, tk, s) : launch_few<KwCfg<64, false>>(p, tk, s);
  return k8 ? launch_few<KwCfg<128, true>>(p, tk, s) : launch_few<KwCfg<128, false>>(p, tk, s);
}
cudaError_t launch_key_weights_many(int D, bool k8, const KeyWeightsParams& p, const CUtensorMap& tq, cudaStream_t s) {
  if (D == 64) return k8 ? launch_many<64, true>(p, tq, s) : launch_many<64, false>(p, tq, s);
  return k8 ? launch_many<128, true>(p, tq, s) : launch_many<128, false>(p, tq, s);
}

}  // namespace fmha
