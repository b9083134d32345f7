// cache_attn.cu -- attention of a few query rows per KV head over a ragged,
// paged (or contiguous) K/V cache: a tree of drafted tokens after each
// sequence's context (one node: ordinary decoding), or the blocks of keys
// picked for each query token.
//
// O_r = sum_s p_rs V_s / l_r, p_rs = exp2(c q_r . k_s - m_r), l_r = sum_s p_rs,
// over the keys row r sees, in one pass over the keys with the running row
// maximum m. Rows are (query token, head of the KV head's group), so a K/V
// tile is read once for all query heads that share it.
//
// Work: items (sequence, [token,] KV head, row tile) x 64-key tiles. In tree
// mode the tiles of all sequences form one list that groups of CTAs (one CTA
// per KV head and row tile) share evenly, so a batch of very different lengths
// keeps every SM busy and the heads of a token are read side by side; the
// lengths are read on the device, and a launch can be captured and replayed
// with others. A CTA holds at most two partial items (its first and its last);
// their O / l and log-sum-exp go to the workspace and a second kernel merges
// them. In tail mode the whole tiles of the contexts are another kernel's: this
// one takes the rest, and joins both parts itself.
//
// 160 threads: four MMA warps and one TMA producer warp feeding a ring of
// 64-key slots.
//  - At most 16 rows (consume_t): the four warps take 16 keys of the slot each
//    (own m, l, O, joined at the item's end) and compute S^T = K Q^T and
//    O^T = V^T P^T, so the keys and the head dim fill the instructions' 16-row
//    side and 8 or 16 query rows their 8-column side.
//    Memory bounds it: 48 sequences of E4M3 keys (452 MB) 81 us.
//  - More rows (consume): a warp takes 16 rows, S = Q K^T and O = P V; with 32
//    rows two warps share the slot's keys, with 64 every warp takes all keys.
#include "cache_tiles.cuh"
#include "mma_sync.cuh"

namespace fmha {
namespace {

template <int D_, bool K8_, bool V8_, int ROWS_, int MODE_>
struct CaCfg {
  static constexpr int D = D_, ROWS = ROWS_;
  static constexpr int NT = ROWS <= 16 ? ROWS / 8 : 0;   // transposed: 8-column tiles of query rows
  static constexpr int WM = NT ? 1 : ROWS / 16, WN = 4 / WM;
  static constexpr bool K8 = K8_, V8 = V8_;
  static constexpr int MODE = MODE_;
  static constexpr bool PICKED = MODE == WALK_PICKED, TAIL = MODE == WALK_TAIL;
  static constexpr bool HAS_V = true;
  using KL = TileLayout<D, K8>;
  using VL = TileLayout<D, V8>;
  static constexpr int SLOT = KL::BYTES + VL::BYTES;
  // CTAs that share an SM, and ring slots in what shared memory each has.
  static constexpr int CTAS = cache_attn_ctas(ROWS);
  static constexpr int STAGES_FIT = ((CTAS == 3 ? 76800 : 114688) - 9216 - 2048) / SLOT;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr int RED_LD = 36;  // floats per row of the joining buffer (32 columns + padding)
  static constexpr int RED_BYTES = 4 * 16 * RED_LD * 4;
  static constexpr int SMEM = STAGES * SLOT + RED_BYTES + 2048;
  static constexpr int THREADS = 160;
  // The running maximum of the transposed arrangement moves when it is exceeded by more than 2^TAU; weights are taken
  // 2^LIFT above it. BF16 weights have the range of 32 bits. F16 weights (E4M3 values) end at 2^16, are normal down to
  // 2^-14 and zero below 2^-25: lifted to the top of that range, they are normal down to 2^-28 of the maximum (2^-29 where
  // it is exact), so a long flat tail below one dominant key keeps its share. Without, 65536 keys of 2^-27 were lost.
  static constexpr float TAU = V8 ? 1.875f : 8.f;
  static constexpr float LIFT = !V8 ? 0.f : NT ? 14.f : 15.f;
};

template <int STAGES>
struct alignas(16) CaMisc : RingMisc<STAGES> {
  float ml[4][16][2];  // (m, l) of each warp's rows
};

// --------------------------------------------------------------- MMA warps --
// A row's query token and head; token < 0: padding.
struct Row {
  int tok, head;
};
template <class C>
__device__ __forceinline__ Row row_of(const CacheAttnParams& p, const Seg& g, int r) {
  const int i = g.rt * C::ROWS + r;
  if constexpr (C::PICKED) return i < p.c.G ? Row{g.t, g.hkv * p.c.G + i} : Row{-1, 0};
  const int t = i / p.c.G;
  return t < p.c.T ? Row{t, g.hkv * p.c.G + i - t * p.c.G} : Row{-1, 0};
}

// A hidden score is -inf, which a factor of zero (a head whose scale is zero)
// would turn into a NaN: the smallest normal number gives the other scores' zeros.
__device__ __forceinline__ float score_factor(float c) { return c == 0.f ? 0x1p-126f : c; }

// Two fp32 -> the 16-bit pair the PV product takes.
template <class C>
__device__ __forceinline__ uint32_t pack_p(float a, float b) {
  return C::V8 ? ptx::pack_f16x2(a, b) : ptx::pack_bf16x2(a, b);
}

// V fragments (keys 16 x columns 32q .. 32q + 31) as four n-tiles: b0 holds
// keys 2j, 2j + 1 and b1 keys 2j + 8, 2j + 9 of a column. BF16: n-tile i is
// columns 32q + 8i ..; E4M3: lane group g's column of n-tile i is 32q + 4g + i
// (four neighbouring codes of a key come in one word), converted to F16, which
// holds every E4M3 value.
template <class C>
__device__ __forceinline__ void load_v(uint32_t (&b)[4][2], uint32_t v_base, int key0, int q, int lane) {
  using namespace ptx;
  if constexpr (C::V8) {
    const int gg = lane >> 2, j = lane & 3;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = key0 + 2 * j + (i & 1) + 8 * (i >> 1);
      w[i] = lds32(v_base + C::VL::at(r, 2 * q + (gg >> 2)) + (gg & 3) * 4);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __byte_perm(w[2 * h], w[2 * h + 1], 0x5140), hi = __byte_perm(w[2 * h], w[2 * h + 1], 0x7362);
      b[0][h] = e4m3x2_to_f16x2(lo & 0xffffu);
      b[1][h] = e4m3x2_to_f16x2(lo >> 16);
      b[2][h] = e4m3x2_to_f16x2(hi & 0xffffu);
      b[3][h] = e4m3x2_to_f16x2(hi >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t r[4];
      const int row = key0 + (lane & 7) + ((lane >> 3) & 1) * 8;
      ldsm4t(r, v_base + C::VL::at(row, 4 * q + 2 * i + (lane >> 4)));
      b[2 * i][0] = r[0];
      b[2 * i][1] = r[1];
      b[2 * i + 1][0] = r[2];
      b[2 * i + 1][1] = r[3];
    }
  }
}

// Bits 15 and 31 set where a half of a 16-bit pair is an infinity or a NaN (all exponent bits set: adding one carries).
template <bool F16>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  constexpr uint32_t E = F16 ? 0x7c007c00u : 0x7f807f80u, ONE = F16 ? 0x04000400u : 0x00800080u;
  return (x & E) + ONE;
}

// Scores of 16 queries x 16 keys, 32 columns (k-steps 2 s and 2 s + 1), from a fragment load of K's codes.
template <int KS>
__device__ __forceinline__ void mma_k8(float (&s0)[4], float (&s1)[4], const uint32_t (&qf)[KS][4], int s,
                                       const uint32_t (&r)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)  // e: which 16 columns (bit 0), which 8 keys (bit 1)
    ptx::mma_f16(e & 2 ? s1 : s0, qf[2 * s + (e & 1)], ptx::e4m3x2_to_f16x2(r[e] & 0xffffu), ptx::e4m3x2_to_f16x2(r[e] >> 16));
}

template <class C>
__device__ void consume(const CacheAttnParams& p, uint8_t* ring, float* red, CaMisc<C::STAGES>* misc, const Waiter w) {
  using namespace ptx;
  constexpr int D = C::D, KS = D / 16, NQ = D / 32;
  constexpr int GPW = kGroups / C::WN;  // 16-key groups of a slot per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp % C::WM, wn = warp / C::WM;
  const int gq = lane >> 2, j = lane & 3;
  uint32_t it = 0;
  bool ok = true;
  Walk<C::MODE> walk;
  walk.start(p);
  Seg g;
  while (walk.next(p, g)) {
    const float sfk = sf_of(p.sf_k, p.sf_k_kind, g.b * static_cast<int64_t>(p.c.Hkv) + g.hkv);
    const float sfv = sf_of(p.sf_v, p.sf_v_kind, g.b * static_cast<int64_t>(p.c.Hkv) + g.hkv);
    // Q fragments: rows gq and gq + 8 of this warp's 16.
    uint32_t qf[KS][4];
    float cs[2];
    Row rows[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rows[h] = row_of<C>(p, g, wm * 16 + gq + 8 * h);
      const uint16_t* src = p.q + g.b * p.q_sb + rows[h].tok * p.q_ss + rows[h].head * p.q_sh;
      load_q<C::K8, KS, 4>(qf, h, cs[h], src, rows[h].tok >= 0, j);
      cs[h] = score_factor(cs[h] * (p.scale_log2 * sfk));
    }
    const uint8_t* mask_row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      mask_row[h] = p.mask + (C::PICKED ? 0 : g.b * p.mask_sb + static_cast<int64_t>(max(rows[h].tok, 0)) * p.c.T);
    float acc[NQ * 4][4];
#pragma unroll
    for (int i = 0; i < NQ * 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int u = g.t0; u < g.t1 && ok; ++u) {
      const int s = it % C::STAGES;
      ok = __all_sync(kFull, w.wait(smem_addr(&misc->full[s]), (it / C::STAGES) & 1));
      if (!ok) break;
      ++it;
      const uint32_t k_base = smem_addr(ring + s * C::SLOT), v_base = k_base + C::KL::BYTES;
      int valid[GPW], pos[GPW];
      bool plain = true, any = false;  // every key of the warp's groups is seen by every row / some key exists
#pragma unroll
      for (int i = 0; i < GPW; ++i) {
        valid[i] = misc->meta[s].valid[wn * GPW + i];
        pos[i] = misc->meta[s].pos[wn * GPW + i];
        any = any || valid[i] > 0;
        plain = plain && valid[i] == 16 && pos[i] + 16 <= g.ctx;
      }
      if (any) {
        // S = Q K^T, 16 rows x 16 keys per group.
        float sc[GPW * 2][4];
#pragma unroll
        for (int i = 0; i < GPW * 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
#pragma unroll
        for (int i = 0; i < GPW; ++i) {
          const int row = (wn * GPW + i) * 16 + (lane & 7) + (lane >> 4) * 8;
          if constexpr (C::K8) {
#pragma unroll
            for (int s2 = 0; s2 < KS / 2; ++s2) {
              uint32_t r[4];
              ldsm4(r, k_base + C::KL::at(row, 2 * s2 + ((lane >> 3) & 1)));
              mma_k8<KS>(sc[2 * i], sc[2 * i + 1], qf, s2, r);
            }
          } else {
#pragma unroll
            for (int s2 = 0; s2 < KS; ++s2) {
              uint32_t r[4];
              ldsm4(r, k_base + C::KL::at(row, 2 * s2 + ((lane >> 3) & 1)));
              mma_bf16(sc[2 * i], qf[s2], r[0], r[1]);
              mma_bf16(sc[2 * i + 1], qf[s2], r[2], r[3]);
            }
          }
        }
        if (!plain) {  // hide keys: past the end, or nodes this row does not see
#pragma unroll
          for (int i = 0; i < GPW; ++i) {
            if (valid[i] == 16 && pos[i] + 16 <= g.ctx) continue;
            uint32_t show = 0xffu;  // bit 4 x + e of the group's sc[2 i + x][e]
            if constexpr (!C::PICKED) {
              const int node0 = pos[i] - g.ctx;  // node of the group's first key
              if (node0 + 16 > 0) {
                show = 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e) {  // all loads first: one latency per group, not one per key
                  const int node = node0 + (e >> 2) * 8 + 2 * j + (e & 1), tok = rows[(e >> 1) & 1].tok;
                  bool see = node < 0 || (tok >= 0 && node <= tok);
                  if (p.mask != nullptr) {
                    const uint8_t byte = __ldg(mask_row[(e >> 1) & 1] + min(max(node, 0), p.c.T - 1));
                    see = node < 0 || (tok >= 0 && byte != 0);
                  }
                  show |= see ? 1u << e : 0u;
                }
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if ((e >> 2) * 8 + 2 * j + (e & 1) >= valid[i] || !((show >> e) & 1u)) sc[2 * i + (e >> 2)][e & 3] = -INFINITY;
          }
        }
        // Running maximum, exponentials and row sums.
        float mb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < GPW * 2; ++i) mx = fmaxf(mx, fmaxf(sc[i][2 * h], sc[i][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
          const float mn = fmaxf(m[h], mx * cs[h] - C::LIFT);  // m: 2^LIFT below the maximum
          const bool up = mn > m[h];
          if (__any_sync(kFull, up)) {
            const float f = up ? ex2(m[h] - mn) : 1.f;
            m[h] = mn;
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < NQ * 4; ++i) {
              acc[i][2 * h] *= f;
              acc[i][2 * h + 1] *= f;
            }
          }
          mb[h] = m[h] == -INFINITY ? 0.f : m[h];
        }
        uint32_t pf[GPW][4];
        uint32_t seen = 0;  // not plain: bit 4 i + e of sc[i][e]
#pragma unroll
        for (int i = 0; i < GPW * 2; ++i) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!plain && GPW <= 4 && sc[i][e] != -INFINITY) seen |= 1u << (4 * i + e);
            e4[e] = ex2(fmaf(sc[i][e], cs[e >> 1], -mb[e >> 1]));
            l[e >> 1] += e4[e];
          }
          pf[i >> 1][(i & 1) * 2] = pack_p<C>(e4[0], e4[1]);
          pf[i >> 1][(i & 1) * 2 + 1] = pack_p<C>(e4[2], e4[3]);
        }
        // O += P V.
#pragma unroll
        for (int i = 0; i < GPW; ++i) {
          if (!plain && valid[i] <= 0) continue;
          const int key0 = (wn * GPW + i) * 16;
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            uint32_t b[4][2];
            load_v<C>(b, v_base, key0, q, lane);
            if (!plain && !(valid[i] == 16 && pos[i] + 16 <= g.ctx)) {
              // Rows past the end hold anything: they count as zero. A node
              // that some row does not see may hold infinities or NaN, which a
              // zero weight would not stop: such a group adds key by key.
              uint32_t keep[2];
#pragma unroll
              for (int h = 0; h < 2; ++h)
                keep[h] = (2 * j + 8 * h < valid[i] ? 0xffffu : 0u) | (2 * j + 1 + 8 * h < valid[i] ? 0xffff0000u : 0u);
              if (valid[i] < 16) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                  for (int h = 0; h < 2; ++h) b[n][h] &= keep[h];
              }
              uint32_t odd = 0u;
              if constexpr (!C::PICKED) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                  for (int h = 0; h < 2; ++h) odd |= not_finite<C::V8>(b[n][h]);
              }
              if (__any_sync(kFull, odd & 0x80008000u)) {
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                  const int from = (lane & ~3) | ((k & 7) >> 1);
                  const int bit = 4 * (2 * i + (k >> 3)) + (k & 1);
                  const uint32_t sb = __shfl_sync(kFull, seen, from);
                  // runtime-indexed registers: pick with selects
                  uint32_t w0 = 0, w1 = 0;
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint32_t a = __shfl_sync(kFull, pf[i][2 * x], from), c = __shfl_sync(kFull, pf[i][2 * x + 1], from);
                    if ((k >> 3) == x) w0 = a, w1 = c;
                  }
                  const float p0 = half_of<C::V8>(w0, k & 1), p1 = half_of<C::V8>(w1, k & 1);
                  const bool s0 = (sb >> bit) & 1u, s1 = (sb >> (bit + 2)) & 1u;
#pragma unroll
                  for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      // column 2j + e of n-tile n: its key k sits in lane (2j + e) * 4 + (k & 7) / 2
                      const uint32_t v0 = __shfl_sync(kFull, b[n][0], (2 * j + e) * 4 + ((k & 7) >> 1));
                      const uint32_t v1 = __shfl_sync(kFull, b[n][1], (2 * j + e) * 4 + ((k & 7) >> 1));
                      const float v = half_of<C::V8>(k < 8 ? v0 : v1, k & 1);
                      if (s0) acc[4 * q + n][e] = fmaf(p0, v, acc[4 * q + n][e]);
                      if (s1) acc[4 * q + n][2 + e] = fmaf(p1, v, acc[4 * q + n][2 + e]);
                    }
                }
                continue;
              }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              if constexpr (C::V8) mma_f16(acc[4 * q + n], pf[i], b[n][0], b[n][1]);
              else mma_bf16(acc[4 * q + n], pf[i], b[n][0], b[n][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&misc->empty[s]));
    }

    // Join the warps that shared the rows, and write O / l (or a partial).
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(kFull, l[h], 1);
      l[h] += __shfl_xor_sync(kFull, l[h], 2);
    }
    if (C::WN > 1) named_bar_sync(1, 128);  // the last item's (m, l) have been read
    if (j == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        misc->ml[warp][gq + 8 * h][0] = m[h];
        misc->ml[warp][gq + 8 * h][1] = l[h];
      }
    }
    if (C::WN > 1) named_bar_sync(1, 128);
    else __syncwarp();
    auto total = [&](int wmi, int r, float& M, float& L) {  // of row r of row group wmi
      M = -INFINITY;
#pragma unroll
      for (int x = 0; x < C::WN; ++x) M = fmaxf(M, misc->ml[x * C::WM + wmi][r][0]);
      const float Mb = M == -INFINITY ? 0.f : M;
      L = 0.f;
#pragma unroll
      for (int x = 0; x < C::WN; ++x) L += misc->ml[x * C::WM + wmi][r][1] * ex2(misc->ml[x * C::WM + wmi][r][0] - Mb);
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float M, L;
      total(wm, gq + 8 * h, M, L);
      f[h] = L != 0.f ? ex2(m[h] - (M == -INFINITY ? 0.f : M)) * (sfv / L) : 0.f;
    }
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    const int64_t slot = 2ll * blockIdx.x + (g.t0 == 0 ? 1 : 0);
    if constexpr (C::WN == 1) {
      if constexpr (C::TAIL) asm volatile("griddepcontrol.wait;" ::: "memory");  // the packed kernel's parts are there
      // A warp has its rows to itself and writes them from its registers, 16 bytes and more of a row at a time.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Row ro = rows[h];
        const int item_row = wm * 16 + gq + 8 * h;
        const bool mine = ro.tok >= 0 && ok;
        float M, L;
        total(wm, gq + 8 * h, M, L);
        float lse = L != 0.f ? M + __log2f(L) : -INFINITY;
        if (!C::TAIL && !whole) {
          const int64_t at = slot * C::ROWS + item_row;
          float* dst = p.part_o + at * D;
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if constexpr (C::V8) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (mine)
                  *reinterpret_cast<float4*>(dst + 32 * q + 8 * j + 4 * e) =
                      make_float4(acc[4 * q][2 * h + e] * f[h], acc[4 * q + 1][2 * h + e] * f[h],
                                  acc[4 * q + 2][2 * h + e] * f[h], acc[4 * q + 3][2 * h + e] * f[h]);
            } else {
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (mine)
                  *reinterpret_cast<float2*>(dst + 32 * q + 8 * n + 2 * j) =
                      make_float2(acc[4 * q + n][2 * h] * f[h], acc[4 * q + n][2 * h + 1] * f[h]);
            }
          }
          if (mine && j == 0) p.part_lse[at] = lse;
        } else {
          if constexpr (C::TAIL) {
            // Join the packed kernel's partial results of the context's whole 128-key tiles.
            if (mine && ro.tok < g.nodes) {
              const int64_t rows_n = static_cast<int64_t>(p.c.B) * p.c.T * p.c.Hq;
              const int64_t at_o = (static_cast<int64_t>(g.b) * p.c.T + ro.tok) * p.c.Hq + ro.head;
              const int64_t at_l = (static_cast<int64_t>(g.b) * p.c.Hq + ro.head) * p.c.T + ro.tok;
              for (int k = 0; k < p.n_parts; ++k) {
                const float x = p.part_lse[k * rows_n + at_l] * 1.4426950408889634f;
                if (x == -INFINITY) continue;  // a part without keys
                const float2* src = reinterpret_cast<const float2*>(p.part_o + (k * rows_n + at_o) * D) + j;
                float2 v[NQ * 4];
#pragma unroll
                for (int n = 0; n < NQ * 4; ++n) v[n] = src[4 * n];
                const float mn = fmaxf(M, x);
                const float fo = M == -INFINITY ? 0.f : ex2(M - mn), fx = ex2(x - mn);
                // acc f is O so far, of weight L 2^M (a NaN sum stays one)
                const float wo = L * fo, sum = wo + fx;
                const float ao = sum != 0.f ? f[h] * wo / sum : 0.f, ax = sum != 0.f ? fx / sum : 0.f;
#pragma unroll
                for (int n = 0; n < NQ * 4; ++n) {
                  acc[n][2 * h] = fmaf(v[n].x, ax, L != 0.f ? acc[n][2 * h] * ao : 0.f);
                  acc[n][2 * h + 1] = fmaf(v[n].y, ax, L != 0.f ? acc[n][2 * h + 1] * ao : 0.f);
                }
                f[h] = 1.f;
                M = mn;
                L = sum;
              }
              lse = L != 0.f ? M + __log2f(L) : -INFINITY;
            }
          }
          const bool hide = !C::PICKED && ro.tok >= g.nodes;  // a padding row: its factor may be anything
          uint16_t* dst = p.o + g.b * p.o_sb + ro.tok * p.o_ss + ro.head * p.o_sh;
          auto pair = [&](float x, float y) { return hide ? 0u : pack_bf16x2(x * f[h], y * f[h]); };
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if constexpr (C::V8) {
              if (mine)
                *reinterpret_cast<uint4*>(dst + 32 * q + 8 * j) =
                    make_uint4(pair(acc[4 * q][2 * h], acc[4 * q + 1][2 * h]), pair(acc[4 * q + 2][2 * h], acc[4 * q + 3][2 * h]),
                               pair(acc[4 * q][2 * h + 1], acc[4 * q + 1][2 * h + 1]),
                               pair(acc[4 * q + 2][2 * h + 1], acc[4 * q + 3][2 * h + 1]));
            } else {
              // Even lanes collect four columns of the first n-tile, odd lanes of the second: 32 bytes per four lanes.
#pragma unroll
              for (int n = 0; n < 4; n += 2) {
                const uint32_t x = pair(acc[4 * q + n][2 * h], acc[4 * q + n][2 * h + 1]);
                const uint32_t y = pair(acc[4 * q + n + 1][2 * h], acc[4 * q + n + 1][2 * h + 1]);
                const uint32_t other = __shfl_xor_sync(kFull, (j & 1) ? x : y, 1);
                if (mine)
                  *reinterpret_cast<uint2*>(dst + 32 * q + 8 * (n + (j & 1)) + 4 * (j >> 1)) =
                      (j & 1) ? make_uint2(other, y) : make_uint2(x, other);
              }
            }
          }
          if (mine && j == 0 && p.lse != nullptr)
            p.lse[(static_cast<int64_t>(g.b) * p.c.Hq + ro.head) * p.c.T + ro.tok] =
                hide ? -INFINITY : lse * 0.69314718055994531f;
        }
      }
      __syncwarp();  // the next item's (m, l) may be written
      continue;
    }
    // Two warps share the rows: eight lanes write a row, 16 rows a pass.
#pragma unroll 1
    for (int q = 0; q < NQ; ++q) {
      float* mine = red + warp * 16 * C::RED_LD;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = C::V8 ? 8 * j + 4 * (e & 1) + n : 8 * n + 2 * j + (e & 1);
          float v = 0.f;
#pragma unroll
          for (int qq = 0; qq < NQ; ++qq)
            if (qq == q) v = acc[4 * qq + n][e];
          mine[(gq + 8 * (e >> 1)) * C::RED_LD + col] = v * f[e >> 1];
        }
      named_bar_sync(1, 128);
#pragma unroll
      for (int ps = 0; ps < C::ROWS / 16; ++ps) {
        const int r = ps * 16 + threadIdx.x / 8, c4 = threadIdx.x % 8;
        const int wmi = r / 16, rr = r % 16;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < C::WN; ++x) {
          const float4 y =
              *reinterpret_cast<const float4*>(red + ((x * C::WM + wmi) * 16 + rr) * C::RED_LD + 4 * c4);
          v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        const int item_row = wmi * 16 + rr;
        const Row ro = row_of<C>(p, g, item_row);
        if (ro.tok < 0 || !ok) continue;
        if (!whole) {
          *reinterpret_cast<float4*>(p.part_o + (slot * C::ROWS + item_row) * D + 32 * q + 4 * c4) = v;
        } else {
          if (!C::PICKED && ro.tok >= g.nodes) v = make_float4(0.f, 0.f, 0.f, 0.f);
          uint16_t* dst = p.o + g.b * p.o_sb + ro.tok * p.o_ss + ro.head * p.o_sh + 32 * q + 4 * c4;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
        if (q == 0 && c4 == 0 && (!whole || p.lse != nullptr)) {
          float M, L;
          total(wmi, rr, M, L);
          float lse = L != 0.f ? M + __log2f(L) : -INFINITY;
          if (!whole) {
            p.part_lse[slot * C::ROWS + item_row] = lse;
          } else {
            if (!C::PICKED && ro.tok >= g.nodes) lse = -INFINITY;
            p.lse[(static_cast<int64_t>(g.b) * p.c.Hq + ro.head) * p.c.T + ro.tok] = lse * 0.69314718055994531f;
          }
        }
      }
      named_bar_sync(1, 128);
    }
  }
}

// 8x8 transpose of a 16-bit matrix across the warp: lane (g, j) holds row g, columns 2 j, 2 j + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// V^T fragments of columns 32 q .. 32 q + 31 (two 16-row tiles) x 16 keys.
// BF16: tile h is columns 32 q + 16 h ..; E4M3: rows g and g + 8 of tile h are
// columns 32 q + 4 g + 2 h and + 1 (a word holds four neighbouring columns).
template <class C>
__device__ __forceinline__ void load_vt(uint32_t (&a)[2][4], uint32_t v_base, int key0, int q, int lane) {
  using namespace ptx;
  if constexpr (C::V8) {
    const int g = lane >> 2, j = lane & 3;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = lds32(v_base + C::VL::at(key0 + 2 * j + (i & 1) + 8 * (i >> 1), 2 * q + (g >> 2)) + (g & 3) * 4);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = __byte_perm(w[2 * k], w[2 * k + 1], 0x5140), hi = __byte_perm(w[2 * k], w[2 * k + 1], 0x7362);
      a[0][2 * k] = e4m3x2_to_f16x2(lo & 0xffffu);
      a[0][2 * k + 1] = e4m3x2_to_f16x2(lo >> 16);
      a[1][2 * k] = e4m3x2_to_f16x2(hi & 0xffffu);
      a[1][2 * k + 1] = e4m3x2_to_f16x2(hi >> 16);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // matrices: keys 0-7 | 8-15 (bit 4 of the lane) x columns 0-7 | 8-15 (bit 3)
      const int row = key0 + (lane & 7) + ((lane >> 4) & 1) * 8;
      ldsm4t(a[h], v_base + C::VL::at(row, 4 * q + 2 * h + ((lane >> 3) & 1)));
    }
  }
}

template <class C>
__device__ void consume_t(const CacheAttnParams& p, uint8_t* ring, float* red, CaMisc<C::STAGES>* misc, const Waiter w) {
  using namespace ptx;
  constexpr int D = C::D, KS = D / 16, NQ = D / 32, NT = C::NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, j = lane & 3;
  uint32_t it = 0;
  bool ok = true;
  Walk<C::MODE> walk;
  walk.start(p);
  Seg g;
  while (walk.next(p, g)) {
    const int64_t bh = g.b * static_cast<int64_t>(p.c.Hkv) + g.hkv;
    const float sfk = sf_of(p.sf_k, p.sf_k_kind, bh), sfv = sf_of(p.sf_v, p.sf_v_kind, bh);
    // Q^T fragments: query row 8 n + gq of each tile; the score factors and tokens of rows 8 n + 2 j and + 1.
    uint32_t qf[NT][KS][2];
    float cs[NT][2];
    int tok[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const Row ro = row_of<C>(p, g, 8 * n + gq);
      float f;
      load_q<C::K8, KS, 2>(qf[n], 0, f, p.q + g.b * p.q_sb + ro.tok * p.q_ss + ro.head * p.q_sh, ro.tok >= 0, j);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        cs[n][e] = score_factor(p.scale_log2 * sfk * __shfl_sync(kFull, f, 4 * (2 * j + e)));
        tok[n][e] = __shfl_sync(kFull, ro.tok, 4 * (2 * j + e));
      }
    }
    float acc[NT][2 * NQ][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2 * NQ; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
    const int key0 = warp * 16;

    for (int u = g.t0; u < g.t1 && ok; ++u) {
      const int s = it % C::STAGES;
      ok = __all_sync(kFull, w.wait(smem_addr(&misc->full[s]), (it / C::STAGES) & 1));
      if (!ok) break;
      ++it;
      const uint32_t k_base = smem_addr(ring + s * C::SLOT), v_base = k_base + C::KL::BYTES;
      const int valid = misc->meta[s].valid[warp], pos = misc->meta[s].pos[warp];
      const bool plain = valid == 16 && pos + 16 <= g.ctx;
      if (valid > 0) {
        // S^T: sc[n][e] is key gq + 8 (e >> 1), query row 8 n + 2 j + (e & 1). Two chains per tile.
        float sc[NT][4], s2[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = s2[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < (C::K8 ? KS / 2 : KS); ++k) {
          uint32_t a[C::K8 ? 2 : 1][4];
          load_kt<C>(a, k_base, key0, k, lane);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (C::K8) {
              mma_f16(sc[n], a[0], qf[n][2 * k][0], qf[n][2 * k][1]);
              mma_f16(s2[n], a[1], qf[n][2 * k + 1][0], qf[n][2 * k + 1][1]);
            } else {
              mma_bf16(k & 1 ? s2[n] : sc[n], a[0], qf[n][k][0], qf[n][k][1]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] += s2[n][e];
        if (!plain) {  // hide keys: past the end, or nodes this row does not see
          uint32_t show = kFull;
          if constexpr (!C::PICKED) {
            const int node0 = pos - g.ctx;  // node of the group's first key
            if (node0 + 16 > 0) {
              show = 0u;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int node = node0 + gq + 8 * (e >> 1), t = tok[n][e & 1];
                  bool see = node < 0 || (t >= 0 && node <= t);
                  if (p.mask != nullptr) {
                    const uint8_t byte = __ldg(p.mask + g.b * p.mask_sb + static_cast<int64_t>(max(t, 0)) * p.c.T +
                                               min(max(node, 0), p.c.T - 1));
                    see = node < 0 || (t >= 0 && byte != 0);
                  }
                  show |= see ? 1u << (4 * n + e) : 0u;
                }
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (gq + 8 * (e >> 1) >= valid || !((show >> (4 * n + e)) & 1u)) sc[n][e] = -INFINITY;
        }
        // The running maximum is lazy: usually one vote says that it stays.
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) over = over || fmaxf(sc[n][e], sc[n][2 + e]) * cs[n][e] > m[n][e] + (C::TAU + C::LIFT);
        if (__any_sync(kFull, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(sc[n][e], sc[n][2 + e]) * cs[n][e];
              mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
              const float mn = fmaxf(m[n][e], mx - C::LIFT);  // m: 2^LIFT below the maximum
              const float f = mn > m[n][e] ? ex2(m[n][e] - mn) : 1.f;
              m[n][e] = mn;
              l[n][e] *= f;
#pragma unroll
              for (int i = 0; i < 2 * NQ; ++i) {
                acc[n][i][e] *= f;
                acc[n][i][2 + e] *= f;
              }
            }
        }
        uint32_t x[NT][2], pb[NT][2];
        uint32_t seen = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!plain && sc[n][e] != -INFINITY) seen |= 1u << (4 * n + e);
            e4[e] = ex2(fmaf(sc[n][e], cs[n][e & 1], m[n][e & 1] == -INFINITY ? 0.f : -m[n][e & 1]));
            l[n][e & 1] += e4[e];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            x[n][h] = pack_p<C>(e4[2 * h], e4[2 * h + 1]);
            pb[n][h] = transpose8(x[n][h]);
          }
        }
        // O^T += V^T P^T.
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          uint32_t a[2][4];
          load_vt<C>(a, v_base, key0, q, lane);
          if (!plain) {
            // Rows past the end hold anything: they count as zero. A node
            // that some row does not see may hold infinities or NaN, which a
            // zero weight would not stop: such a group adds key by key.
            uint32_t keep[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              keep[h] = (2 * j + 8 * h < valid ? 0xffffu : 0u) | (2 * j + 1 + 8 * h < valid ? 0xffff0000u : 0u);
            uint32_t odd = 0u;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a[t][i] &= keep[i >> 1];
                odd |= not_finite<C::V8>(a[t][i]);
              }
            if (__any_sync(kFull, odd & 0x80008000u)) {
#pragma unroll 1
              for (int k = 0; k < 16; ++k) {
                const int from_p = (k & 7) * 4 + j, from_v = (lane & ~3) | ((k & 7) >> 1);
                const uint32_t sb = __shfl_sync(kFull, seen, from_p) >> (2 * (k >> 3));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  const uint32_t x0 = __shfl_sync(kFull, x[n][0], from_p), x1 = __shfl_sync(kFull, x[n][1], from_p);
                  const uint32_t xk = k < 8 ? x0 : x1;
                  const float p0 = half_of<C::V8>(xk, 0), p1 = half_of<C::V8>(xk, 1);
                  const bool s0 = (sb >> (4 * n)) & 1u, s1 = (sb >> (4 * n + 1)) & 1u;
#pragma unroll
                  for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // column rows gq and gq + 8
                      const uint32_t v0 = __shfl_sync(kFull, a[t][h], from_v), v1 = __shfl_sync(kFull, a[t][2 + h], from_v);
                      const float v = half_of<C::V8>(k < 8 ? v0 : v1, k & 1);
                      if (s0) acc[n][2 * q + t][2 * h] = fmaf(p0, v, acc[n][2 * q + t][2 * h]);
                      if (s1) acc[n][2 * q + t][2 * h + 1] = fmaf(p1, v, acc[n][2 * q + t][2 * h + 1]);
                    }
                }
              }
              continue;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if constexpr (C::V8) mma_f16(acc[n][2 * q + t], a[t], pb[n][0], pb[n][1]);
              else mma_bf16(acc[n][2 * q + t], a[t], pb[n][0], pb[n][1]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&misc->empty[s]));
    }

    // Join the four warps, and write O / l (or a partial).
    named_bar_sync(1, 128);  // the last item's (m, l) have been read
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(kFull, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(kFull, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(kFull, l[n][e], 16);
        if (gq == 0) {
          misc->ml[warp][8 * n + 2 * j + e][0] = m[n][e];
          misc->ml[warp][8 * n + 2 * j + e][1] = l[n][e];
        }
      }
    named_bar_sync(1, 128);
    auto total = [&](int r, float& M, float& L) {
      M = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) M = fmaxf(M, misc->ml[x][r][0]);
      const float Mb = M == -INFINITY ? 0.f : M;
      L = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) L += misc->ml[x][r][1] * ex2(misc->ml[x][r][0] - Mb);
    };
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M, L;
        total(8 * n + 2 * j + e, M, L);
        f[n][e] = L != 0.f ? ex2(m[n][e] - (M == -INFINITY ? 0.f : M)) * (sfv / L) : 0.f;
      }
    const int r = threadIdx.x / 8, c4 = threadIdx.x % 8;  // 8 lanes per row write
    const Row ro = row_of<C>(p, g, r);
    const bool mine = r < C::ROWS && ro.tok >= 0 && ok;
    const bool whole = g.t0 == 0 && g.t1 == g.nt;
    const int64_t slot = 2ll * blockIdx.x + (g.t0 == 0 ? 1 : 0);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = C::V8 ? 4 * gq + 2 * t + (e >> 1) : 16 * t + gq + 8 * (e >> 1);
            red[(warp * 16 + 8 * n + 2 * j + (e & 1)) * C::RED_LD + col] = acc[n][2 * q + t][e] * f[n][e & 1];
          }
      named_bar_sync(1, 128);
      if (mine) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 y = *reinterpret_cast<const float4*>(red + (x * 16 + r) * C::RED_LD + 4 * c4);
          v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        if (!whole) {
          *reinterpret_cast<float4*>(p.part_o + (slot * C::ROWS + r) * D + 32 * q + 4 * c4) = v;
        } else {
          if (!C::PICKED && ro.tok >= g.nodes) v = make_float4(0.f, 0.f, 0.f, 0.f);
          uint16_t* dst = p.o + g.b * p.o_sb + ro.tok * p.o_ss + ro.head * p.o_sh + 32 * q + 4 * c4;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
      }
      named_bar_sync(1, 128);
    }
    if (mine && c4 == 0 && (!whole || p.lse != nullptr)) {
      float M, L;
      total(r, M, L);
      float lse = L != 0.f ? M + __log2f(L) : -INFINITY;
      if (!whole) {
        p.part_lse[slot * C::ROWS + r] = lse;
      } else {
        if (!C::PICKED && ro.tok >= g.nodes) lse = -INFINITY;
        p.lse[(static_cast<int64_t>(g.b) * p.c.Hq + ro.head) * p.c.T + ro.tok] = lse * 0.69314718055994531f;
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    cache_attn_kernel(const __grid_constant__ CacheAttnParams p, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv) {
  using namespace ptx;
  if constexpr (!C::TAIL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(ring + C::STAGES * C::SLOT);
  auto* misc = reinterpret_cast<CaMisc<C::STAGES>*>(ring + C::STAGES * C::SLOT + C::RED_BYTES);
  static_assert(sizeof(CaMisc<C::STAGES>) <= 1024, "misc area");
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
  if (threadIdx.x >= 128) produce<C>(p, ring, misc, &tk, &tv, w);
  else if constexpr (C::NT > 0) consume_t<C>(p, ring, red, misc, w);
  else consume<C>(p, ring, red, misc, w);
  __syncthreads();
}

// Merges the partials of items that several CTAs shared, and writes the rows
// of items without any key. One warp per row.
template <int D, bool PICKED>
__global__ void __launch_bounds__(128) cache_merge_kernel(const __grid_constant__ CacheAttnParams p, int rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5);
  long long item = blockIdx.x;
  const long long flat = item;
  const int rt = static_cast<int>(item % p.row_tiles);
  item /= p.row_tiles;
  const int hkv = static_cast<int>(item % p.c.Hkv);
  item /= p.c.Hkv;
  int tok, head, b;
  bool hidden = false;
  long long first, last;  // CTAs (tree: groups of them) that hold a partial of the item
  if constexpr (PICKED) {
    tok = static_cast<int>(item % p.c.T);
    b = static_cast<int>(item / p.c.T);
    const int i = rt * rows + row;
    if (i >= p.c.G) return;
    head = hkv * p.c.G + i;
    first = flat * p.n_splits;
    last = first + p.n_splits - 1;
  } else {
    b = static_cast<int>(item);
    const int i = rt * rows + row;
    tok = i / p.c.G;
    if (tok >= p.c.T) return;
    head = hkv * p.c.G + i - tok * p.c.G;
    bool bad;
    const SeqLens s = tree_lens(p.c, b, bad);
    const int nt = tiles_of<WALK_TREE>(s);
    hidden = tok >= s.q || nt == 0;
    const Share sh = list_share<WALK_TREE>(p, false);
    const long long t0 = list_tiles<WALK_TREE>(p, b, false);
    first = t0 / sh.per;
    last = nt > 0 ? (t0 + nt - 1) / sh.per : first;
    if (nt > 0 && first == last) return;  // written whole
  }
  uint16_t* dst = p.o + b * p.o_sb + tok * p.o_ss + head * p.o_sh;
  float* lse_out = p.lse == nullptr ? nullptr : p.lse + (static_cast<int64_t>(b) * p.c.Hq + head) * p.c.T + tok;
  constexpr int V = D / 32;  // columns per lane
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  float sum = 0.f, mx = -INFINITY;
  if (!hidden) {
    auto slot = [&](long long c) {
      const long long cta = PICKED ? c : c * p.c.Hkv * p.row_tiles + hkv * p.row_tiles + rt;
      return (2 * cta + (c == first ? 1 : 0)) * rows + row;
    };
    const int n = static_cast<int>(last - first + 1);
    for (int k = lane; k < n; k += 32) mx = fmaxf(mx, p.part_lse[slot(first + k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    // A NaN partial must reach the row: fmaxf drops it, the weights keep it.
    const float mb = mx == -INFINITY ? 0.f : mx;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const float mine = k0 + lane < n ? p.part_lse[slot(first + k0 + lane)] : -INFINITY;
      const float wgt = ptx::ex2(mine - mb);
      const int m = min(32, n - k0);
#pragma unroll 4
      for (int k = 0; k < m; ++k) {
        const float wk = __shfl_sync(kFull, wgt, k);
        const float* src = p.part_o + slot(first + k0 + k) * D + lane * V;
        sum += wk;
        if (wk == 0.f) continue;  // a partial that saw no key
        if constexpr (V == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          acc[0] = fmaf(wk, v.x, acc[0]);
          acc[1] = fmaf(wk, v.y, acc[1]);
          acc[2] = fmaf(wk, v.z, acc[2]);
          acc[3] = fmaf(wk, v.w, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          acc[0] = fmaf(wk, v.x, acc[0]);
          acc[1] = fmaf(wk, v.y, acc[1]);
        }
      }
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst + lane * 4) =
        make_uint2(ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv), ptx::pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst + lane * 2) = ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lse_out != nullptr && lane == 0)
    *lse_out = sum != 0.f ? (mx + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <class C>
cudaError_t launch_cfg(const CacheAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  auto kern = cache_attn_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<p.n_ctas, C::THREADS, C::SMEM, s>>>(p, tk, tv);
  return cudaGetLastError();
}

template <int D, bool K8, bool V8, int MODE>
cudaError_t launch_rows(const CacheAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  switch (cache_attn_rows(MODE == WALK_PICKED ? p.c.G : p.c.G * p.c.T)) {
    case 8: return launch_cfg<CaCfg<D, K8, V8, 8, MODE>>(p, tk, tv, s);
    case 16: return launch_cfg<CaCfg<D, K8, V8, 16, MODE>>(p, tk, tv, s);
    case 32: return launch_cfg<CaCfg<D, K8, V8, 32, MODE>>(p, tk, tv, s);
    default: return launch_cfg<CaCfg<D, K8, V8, 64, MODE>>(p, tk, tv, s);
  }
}

template <int D, int MODE>
cudaError_t launch_types(bool k8, bool v8, const CacheAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t s) {
  if (k8) return launch_rows<D, true, true, MODE>(p, tk, tv, s);
  return v8 ? launch_rows<D, false, true, MODE>(p, tk, tv, s) : launch_rows<D, false, false, MODE>(p, tk, tv, s);
}

}  // namespace

cudaError_t launch_cache_attn(int D, bool k8, bool v8, const CacheAttnParams& p, const CUtensorMap& tk,
                              const CUtensorMap& tv, cudaStream_t s) {
  if (p.blocks != nullptr)
    return D == 64 ? launch_types<64, WALK_PICKED>(k8, v8, p, tk, tv, s)
                   : launch_types<128, WALK_PICKED>(k8, v8, p, tk, tv, s);
  return D == 64 ? launch_types<64, WALK_TREE>(k8, v8, p, tk, tv, s)
                 : launch_types<128, WALK_TREE>(k8, v8, p, tk, tv, s);
}

cudaError_t launch_cache_tail(const CacheAttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  using C = CaCfg<128, false, false, 64, WALK_TAIL>;
  auto kern = cache_attn_kernel<C>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // Starts on the SMs that the packed kernel's last CTAs leave free, and waits for its end only to join its results.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_ctas);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, tk, tv);
}

cudaError_t launch_cache_merge(int D, const CacheAttnParams& p, cudaStream_t s) {
  const bool picked = p.blocks != nullptr;
  const int rows = cache_attn_rows(picked ? p.c.G : p.c.G * p.c.T);
  const long long items = static_cast<long long>(p.c.B) * (picked ? p.c.T : 1) * p.c.Hkv * p.row_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items), rows / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  // Set up while the attention grid still runs (the kernel waits for its end).
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (picked)
    return D == 64 ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<64, true>, p, rows)
                   : cudaLaunchKernelEx(&cfg, cache_merge_kernel<128, true>, p, rows);
  return D == 64 ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<64, false>, p, rows)
                 : cudaLaunchKernelEx(&cfg, cache_merge_kernel<128, false>, p, rows);
}

}  // namespace fmha
