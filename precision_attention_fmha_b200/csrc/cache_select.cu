// cache_select.cu -- a cheap score that picks, for each query, the blocks of
// cached keys worth attending to.
//
// Per block j and channel d the bounds are lo_jd = min and hi_jd = max over
// the block's keys. For query heads h of one KV head,
//     score_j = sum_h sum_d max(q_hd lo_jd, q_hd hi_jd)
//             = sum_d up_d hi_jd + down_d lo_jd,
//     up_d = sum_h max(q_hd, 0),  down_d = sum_h min(q_hd, 0):
// the sum over the heads of the largest product that a key inside the box
// could have, at the price of one dot product of 2 D terms per block, whatever
// the group size. The pick must not depend on the order of summation, so the
// scores are taken in 64 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "cache_tiles.cuh"

namespace fmha {
namespace {

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// One warp per (block, KV head); 16-byte loads, several rows per load. Every
// key is read once and nothing is computed twice, so the bytes bound it.
template <int D, bool E8>
__global__ void __launch_bounds__(256) key_bounds_kernel(const __grid_constant__ KeyBoundsParams p) {
  constexpr int ROW = D * (E8 ? 1 : 2), LPR = ROW / 16, RPI = 32 / LPR;
  constexpr int W = E8 ? 8 : 4;  // BF16 pairs of one 16-byte load
  const int lane = threadIdx.x & 31;
  long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int h = static_cast<int>(item % p.c.Hkv);  // neighbouring warps read neighbouring heads of the same tokens
  item /= p.c.Hkv;
  const int j = static_cast<int>(item % p.n_blocks);
  const int b = static_cast<int>(item / p.n_blocks);
  if (b >= p.c.B) return;
  int len = __ldg(p.c.lens + b);
  const int room = static_cast<int>(min(static_cast<long long>(p.c.capacity), static_cast<long long>(p.n_blocks) << p.block_shift));
  if (len < 0 || len > room) {
    if (lane == 0 && j == 0) atomicOr(p.c.err, kErrLength);
    len = min(max(len, 0), room);
  }
  const int first = j << p.block_shift;
  if (first >= len) return;  // past the sequence's end
  if (p.start != nullptr && first + (1 << p.block_shift) <= __ldg(p.start + b)) return;  // bounds still hold
  const int n = min(1 << p.block_shift, len - first);
  const int sub = lane / LPR, unit = lane % LPR;
  uint32_t lo[W], hi[W];
#pragma unroll
  for (int w = 0; w < W; ++w) lo[w] = 0x7f807f80u, hi[w] = 0xff80ff80u;  // +inf, -inf
  // Pages are at least 16 rows and a block starts on a multiple of 16: 16 rows at a time share a page.
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int pos = first + r0;
    int64_t outer = b, row = pos;
    if (p.c.page_table != nullptr) {
      const int pg = __ldg(p.c.page_table + static_cast<int64_t>(b) * p.c.max_pages + (pos >> p.c.page_shift));
      if (pg < 0 || pg >= p.c.num_pages) {
        if (lane == 0) atomicOr(p.c.err, kErrPageIndex);
        outer = -1;  // a bad page reads zeros
      } else {
        outer = pg;
      }
      row = pos & ((1 << p.c.page_shift) - 1);
    }
    const uint8_t* base = p.k + (outer * p.k_sb + row * p.k_ss + h * p.k_sh) * (E8 ? 1 : 2) + unit * 16;
    uint4 v[16 / RPI > 0 ? 16 / RPI : 1];
#pragma unroll
    for (int i = 0; i < (16 + RPI - 1) / RPI; ++i) {
      const int r = i * RPI + sub;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < 16 && r0 + r < n && outer >= 0)
        v[i] = __ldg(reinterpret_cast<const uint4*>(base + static_cast<int64_t>(r) * p.k_ss * (E8 ? 1 : 2)));
    }
#pragma unroll
    for (int i = 0; i < (16 + RPI - 1) / RPI; ++i) {
      const int r = i * RPI + sub;
      if (r >= 16 || r0 + r >= n) continue;
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (E8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t y = e4m3x2_to_bf16x2((x[w] >> (16 * e)) & 0xffffu);
            lo[2 * w + e] = min2(lo[2 * w + e], y);
            hi[2 * w + e] = max2(hi[2 * w + e], y);
          }
        } else {
          lo[w] = min2(lo[w], x[w]);
          hi[w] = max2(hi[w], x[w]);
        }
      }
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      lo[w] = min2(lo[w], __shfl_xor_sync(kFull, lo[w], o));
      hi[w] = max2(hi[w], __shfl_xor_sync(kFull, hi[w], o));
    }
  if (sub != 0) return;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.bounds) +
                  ((static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_blocks + j) * D + unit * W;  // 2 D values = D words
#pragma unroll
  for (int w = 0; w < W; w += 4) {
    *reinterpret_cast<uint4*>(dst + w) = make_uint4(lo[w], lo[w + 1], lo[w + 2], lo[w + 3]);
    *reinterpret_cast<uint4*>(dst + D / 2 + w) = make_uint4(hi[w], hi[w + 1], hi[w + 2], hi[w + 3]);
  }
}

// ------------------------------------------------------------ score and pick --
// Order like the numbers (a larger score has a larger key; -0 counts as +0).
__device__ __forceinline__ unsigned long long order_key(double x) {
  const long long v = __double_as_longlong(x + 0.0);
  return static_cast<unsigned long long>(v) ^ (v < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ uint32_t order_key(float x) {
  const int32_t v = __float_as_int(x + 0.f);
  return static_cast<uint32_t>(v) ^ (v < 0 ? ~0u : 1u << 31);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 1u << 31 : ~0u)); }

__device__ __forceinline__ float larger(float a, float b) { return b > a || b != b ? b : a; }  // a NaN stays

constexpr int kPickThreads = 256, kPickWarps = kPickThreads / 32;

struct PickMisc {
  double half64[2][128];  // down, up in 64 bits
  float half[2][128];     // and in 32
  unsigned long long ends[2][kPickWarps];
  unsigned long long prefix;
  unsigned hist[256];
  float err[8];           // each CTA's bound on the error of its scores
  int need, total;
  int warp_a[kPickWarps], warp_b[kPickWarps];
};

// The `left`-th largest of keys [0, n), eight bits a pass from the highest bit
// in which they differ. Returns the key `limit` and how many of those equal to
// it are in (`need`, the lowest first); all above it are.
template <class K>
__device__ void nth_key(const K* keys, int n, int left, PickMisc* m, K& limit, int& need) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int BITS = sizeof(K) * 8;
  K lo = static_cast<K>(~K(0)), hi = 0;
  for (int j = tid; j < n; j += kPickThreads) {
    lo = min(lo, keys[j]);
    hi = max(hi, keys[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(kFull, lo, o));
    hi = max(hi, __shfl_xor_sync(kFull, hi, o));
  }
  if (lane == 0) m->ends[0][warp] = lo, m->ends[1][warp] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) {
    lo = min(lo, static_cast<K>(m->ends[0][w]));
    hi = max(hi, static_cast<K>(m->ends[1][w]));
  }
  int shift = max(0, 56 - __clzll(static_cast<long long>(static_cast<unsigned long long>(lo ^ hi) | 1ull)));
  int from = min(BITS, shift + 8);  // keys of the current bucket agree with `prefix` in all bits from `from` up
  K prefix = from >= BITS ? K(0) : static_cast<K>(hi >> from << from);
  for (;;) {
    const unsigned digits = 1u << (from - shift);
    m->hist[tid] = 0u;
    __syncthreads();
    for (int j = tid; j < n; j += kPickThreads) {
      const K k = keys[j];
      if (from >= BITS || (k >> from) == (prefix >> from)) atomicAdd(&m->hist[static_cast<unsigned>(k >> shift) & (digits - 1u)], 1u);
    }
    __syncthreads();
    if (warp == 0) {  // lane l: digits 255 - 8 l down to 248 - 8 l
      unsigned c[8], mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine += c[e] = m->hist[255 - 8 * lane - e];
      unsigned before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(kFull, before, o);
        if (lane >= o) before += v;
      }
      before -= mine;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (before < static_cast<unsigned>(left) && before + c[e] >= static_cast<unsigned>(left)) {
          m->prefix = prefix | (static_cast<K>(255 - 8 * lane - e) << shift);
          m->need = left - static_cast<int>(before);
          m->total = static_cast<int>(c[e]);
        }
        before += c[e];
      }
    }
    __syncthreads();
    prefix = static_cast<K>(m->prefix);
    left = m->need;
    const int total = m->total;
    __syncthreads();
    if (shift == 0 || total == 1) break;  // one key left in the bucket: it is the one
    from = shift;
    shift = max(0, shift - 8);
  }
  if (shift > 0) {  // its lower bits
    for (int j = tid; j < n; j += kPickThreads)
      if ((keys[j] >> shift) == (prefix >> shift)) m->prefix = keys[j];
    __syncthreads();
    prefix = static_cast<K>(m->prefix);
  }
  limit = prefix;
  need = left;
}

// up and down of the tile's queries: thread (tid / U) sums every STEP-th row of
// the 8 channels of unit tid % U, and the STEP partial sums are added in order.
template <int D, class F>
__device__ void half_sums(const SelectParams& p, const uint16_t* q, int tokens, F (*half)[128], F* part) {
  constexpr int U = D / 8, STEP = kPickThreads / U;  // 16-byte units of a row; rows per pass
  const int tid = threadIdx.x, unit = tid % U;
  // A single token's heads are the rows; else each head's tokens are.
  const bool one = tokens == 1;
  const int rows = one ? p.c.G : tokens, outer = one ? 1 : p.c.G;
  const int64_t row_stride = one ? p.q_sh : p.q_ss;
  F up[8], down[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) up[e] = down[e] = F(0);
  for (int o = 0; o < outer; ++o)
    for (int r0 = tid / U; r0 < rows; r0 += 4 * STEP) {  // four rows' loads in flight
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k * STEP;
        v[k] = r < rows ? __ldg(reinterpret_cast<const uint4*>(q + unit * 8 + o * p.q_sh + r * row_stride)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = __uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16);
          up[e] += static_cast<F>(fmaxf(f, 0.f));
          down[e] += static_cast<F>(fminf(f, 0.f));
        }
      }
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    part[(tid / U) * 2 * D + unit * 8 + e] = down[e];
    part[(tid / U) * 2 * D + D + unit * 8 + e] = up[e];
  }
  __syncthreads();
  for (int i = tid; i < 2 * D; i += kPickThreads) {
    F sum = F(0);
    for (int r = 0; r < STEP; ++r) sum += part[r * 2 * D + i];
    half[i / D][i % D] = sum;
  }
  __syncthreads();
}

// One cluster per (sequence, query tile, KV head): every CTA scores a share of
// the blocks into CTA 0's shared memory, which picks.
//
// The scores decide in 64 bits, but 64-bit arithmetic runs at about 12 terms a
// cycle and SM here, a tenth of the bytes' pace (512 blocks of 256 terms: 19 of
// 29 us). So they are taken in 32 bits first, each with a bound E on its error:
// with T the `left`-th largest, blocks above T + 2 E are in and blocks below
// T - 2 E are out whatever the rounding was (the `left`-th largest exact score
// lies within E of T). Only what lies between, where it is not all in, is
// scored again in 64 bits; usually nothing is.
template <int D>
__global__ void __launch_bounds__(kPickThreads) select_blocks_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickMisc* m = reinterpret_cast<PickMisc*>(smem_raw);
  // 32-bit keys of all blocks (then the ids of the close ones), a verdict per block, 64-bit keys of the close ones (and
  // the partial sums of up and down).
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(PickMisc));
  uint8_t* verdict = reinterpret_cast<uint8_t*>(keys + p.pad_blocks);  // 0 out, 1 in, 2 close
  unsigned long long* keys64 = reinterpret_cast<unsigned long long*>(verdict + p.pad_blocks);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0u;
  long long item = blockIdx.x / p.cluster;
  const int h = static_cast<int>(item % p.c.Hkv);
  item /= p.c.Hkv;
  const int tile = static_cast<int>(item % p.n_tiles);
  const int b = static_cast<int>(item / p.n_tiles);
  bool bad;
  const SeqLens s = seq_lens(p.c, b, bad);
  if (bad && tid == 0) atomicOr(p.c.err, kErrLength);
  const int t0 = tile * p.q_tile, t1 = min(t0 + p.q_tile, s.q);
  // Blocks up to the position of the tile's last query token.
  const int last = s.len - s.q + t1 - 1;
  int seen = t1 > t0 && last >= 0 ? (last >> p.block_shift) + 1 : 0;
  if (seen > p.n_blocks) {
    if (tid == 0) atomicOr(p.c.err, kErrLength);
    seen = p.n_blocks;
  }
  const bool all = seen <= p.top;  // every block is picked: no scores needed
  // Blocks [f0, f1) are not forced.
  const int f0 = min(p.sinks, seen), f1 = max(f0, seen - p.recent);
  int left = p.top - (seen - (f1 - f0));
  const bool scored = !all && left > 0;
  const uint16_t* q = p.q + b * p.q_sb + static_cast<int64_t>(t0) * p.q_ss + h * p.c.G * p.q_sh;
  constexpr int LPB = D / 4, BPW = 32 / LPB;  // a block's bounds are 4 D bytes: lanes per block; blocks per warp load
  const int in = lane % LPB;
  const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_blocks * 2 * D) + in;
  if (scored) {
    half_sums<D, float>(p, q, t1 - t0, m->half, reinterpret_cast<float*>(keys64));
    if (p.cluster > 1) cluster_sync();  // every CTA of the cluster runs
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = m->half[(in * 8 + e) / D][(in * 8 + e) % D];
    const int stride = kPickWarps * p.cluster * BPW;
    const uint32_t dst = p.cluster > 1 ? in_cta(ptx::smem_addr(keys), 0) : ptx::smem_addr(keys);
    float worst = 0.f;
    for (int j = f0 + (rank * kPickWarps + warp) * BPW + lane / LPB; j - lane / LPB < f1; j += 4 * stride) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = j + i * stride < f1 ? __ldg(src + static_cast<int64_t>(j + i * stride) * LPB) : make_uint4(0u, 0u, 0u, 0u);
      float sum[4], mag[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        sum[i] = mag[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = __uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16);
          sum[i] = fmaf(w[e], f, sum[i]);
          mag[i] = fmaf(fabsf(w[e]), fabsf(f), mag[i]);
        }
      }
#pragma unroll
      for (int o = LPB / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i] += __shfl_xor_sync(kFull, sum[i], o);
          mag[i] += __shfl_xor_sync(kFull, mag[i], o);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        worst = larger(worst, mag[i]);
        if (in == i && j + i * stride < f1) {
          const uint32_t key = order_key(sum[i]);
          if (p.cluster > 1) st_cluster(dst + (j + i * stride) * 4, key);
          else keys[j + i * stride] = key;
        }
      }
    }
    // |score - exact| <= mag * 2^-24 * (additions that a term goes through: its rows' sum and 16 partial sums, 8
    // products, 6 joining steps, 2 for mag itself), one and a half times.
    const int rows = t1 - t0 == 1 ? p.c.G : ((t1 - t0 + 15) / 16) * p.c.G;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float v = __shfl_xor_sync(kFull, worst, o);
      worst = larger(worst, v);
    }
    if (lane == 0) m->warp_a[warp] = __float_as_int(worst);
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < kPickWarps; ++i) {
        worst = larger(worst, __int_as_float(m->warp_a[i]));
      }
      const float e = worst * (1.5f * 0x1p-24f) * static_cast<float>(rows + 32);
      if (p.cluster > 1) st_cluster(in_cta(ptx::smem_addr(&m->err[rank]), 0), __float_as_uint(e));
      else m->err[0] = e;
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
  }
  if (rank != 0) return;

  if (!scored) {
    // All of them, or no more than the forced ones: the lowest `top`.
    for (int j = tid; j < seen; j += kPickThreads)
      verdict[j] = all ? 1 : (j < f0 || j >= f1) && (j < f0 ? j : f0 + j - f1) < p.top;
    __syncthreads();
  } else {
    float E = 0.f;
    for (int i = 0; i < p.cluster; ++i) E = larger(E, m->err[i]);
    uint32_t limit;
    int need;
    nth_key<uint32_t>(keys + f0, f1 - f0, left, m, limit, need);
    const float T = key_value(limit), sure = T + 2.f * E, never = T - 2.f * E;
    // Verdicts; the close ones listed in ascending order (ids in their 64-bit keys' place).
    int n_in = 0, n_close = 0;
    const int run = ((seen + kPickWarps - 1) / kPickWarps + 31) & ~31;
    const int j0 = min(seen, warp * run), j1 = min(seen, j0 + run);
    for (int j = j0; j < j1; j += 32) {
      const int at = j + lane;
      uint8_t v = 0;
      if (at < j1) {
        const float x = at >= f0 && at < f1 ? key_value(keys[at]) : 0.f;
        v = at < f0 || at >= f1 ? 3 : x > sure ? 1 : x < never ? 0 : 2;
        verdict[at] = v == 3 ? 1 : v;
      }
      n_in += __popc(__ballot_sync(kFull, v == 1));
      n_close += __popc(__ballot_sync(kFull, v == 2));
    }
    if (lane == 0) m->warp_a[warp] = n_in, m->warp_b[warp] = n_close;
    __syncthreads();
    int before = 0, close = 0;
    for (int i = 0; i < kPickWarps; ++i) {
      left -= m->warp_a[i];
      if (i < warp) before += m->warp_b[i];
      close += m->warp_b[i];
    }
    __syncthreads();
    if (left < close) {  // not all of the close ones: 64 bits decide
      half_sums<D, double>(p, q, t1 - t0, m->half64, reinterpret_cast<double*>(keys64));
      uint32_t* ids = keys;  // the 32-bit keys have done their work
      for (int j = j0; j < j1; j += 32) {
        const bool c = j + lane < j1 && verdict[j + lane] == 2;
        const uint32_t bal = __ballot_sync(kFull, c);
        if (c) ids[before + __popc(bal & ((1u << lane) - 1u))] = j + lane;
        before += __popc(bal);
      }
      __syncthreads();
      for (int i = warp * BPW + lane / LPB; i - lane / LPB < close; i += kPickWarps * BPW) {
        double sum = 0.0;
        if (i < close) {
          const uint4 v = __ldg(src + static_cast<int64_t>(ids[i]) * LPB);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sum = fma(m->half64[(in * 8 + e) / D][(in * 8 + e) % D],
                      static_cast<double>(__uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16)), sum);
        }
#pragma unroll
        for (int o = LPB / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (in == 0 && i < close) keys64[i] = order_key(sum);
      }
      __syncthreads();
      unsigned long long limit64;
      nth_key<unsigned long long>(keys64, close, left, m, limit64, need);
      // The close ones above it, and the first `need` equal to it: one warp, in order.
      if (warp == 0) {
        int eq = 0;
        for (int i = 0; i < close; i += 32) {
          const unsigned long long k = i + lane < close ? keys64[i + lane] : 0ull;
          const bool e = i + lane < close && k == limit64;
          const uint32_t bal = __ballot_sync(kFull, e);
          if (i + lane < close)
            verdict[ids[i + lane]] = k > limit64 || (e && eq + __popc(bal & ((1u << lane) - 1u)) < need) ? 1 : 0;
          eq += __popc(bal);
        }
      }
    }
    __syncthreads();
  }
  // Warps take consecutive runs of blocks.
  const int run = ((seen + kPickWarps - 1) / kPickWarps + 31) & ~31;
  const int j0 = min(seen, warp * run), j1 = min(seen, j0 + run);
  if (p.mask != nullptr) {
    uint8_t* mask = p.mask + ((static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_tiles + tile) * p.n_blocks;
    for (int j = tid; j < p.n_blocks; j += kPickThreads) mask[j] = j < seen && verdict[j] != 0 ? 1 : 0;
    return;
  }
  int32_t* list = p.list + ((static_cast<int64_t>(b) * p.n_tiles + tile) * p.c.Hkv + h) * p.top;  // n_tiles = T
  int at = 0;
  for (int j = j0; j < j1; j += 32) at += __popc(__ballot_sync(kFull, j + lane < j1 && verdict[j + lane] != 0));
  if (lane == 0) m->warp_a[warp] = at;
  __syncthreads();
  at = 0;
  for (int w = 0; w < warp; ++w) at += m->warp_a[w];
  for (int j = j0; j < j1; j += 32) {
    const bool take = j + lane < j1 && verdict[j + lane] != 0;
    const uint32_t bal = __ballot_sync(kFull, take);
    if (take) list[at + __popc(bal & ((1u << lane) - 1u))] = j + lane;
    at += __popc(bal);
  }
  for (int i = min(seen, p.top) + tid; i < p.top; i += kPickThreads) list[i] = -1;
}

}  // namespace

cudaError_t launch_key_bounds(int D, bool k8, const KeyBoundsParams& p, cudaStream_t s) {
  const long long items = static_cast<long long>(p.c.B) * p.c.Hkv * p.n_blocks;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8);
  if (D == 64) {
    if (k8) key_bounds_kernel<64, true><<<grid, 256, 0, s>>>(p);
    else key_bounds_kernel<64, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (k8) key_bounds_kernel<128, true><<<grid, 256, 0, s>>>(p);
    else key_bounds_kernel<128, false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_select_blocks(int D, const SelectParams& p_in, cudaStream_t s) {
  auto kern = D == 64 ? select_blocks_kernel<64> : select_blocks_kernel<128>;
  // 13 bytes per block; the 64-bit key area also holds the partial sums of up and down (256 threads x 16 doubles).
  SelectParams p = p_in;
  p.pad_blocks = (p.n_blocks + 7) & ~7;
  const size_t smem = sizeof(PickMisc) + size_t(p.pad_blocks) * 5 + std::max<size_t>(size_t(p.pad_blocks) * 8, size_t(kPickThreads) * 16 * 8);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.c.B) * p.n_tiles * p.c.Hkv * p.cluster));
  cfg.blockDim = dim3(kPickThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fmha
