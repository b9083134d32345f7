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
// scores are taken in 64 bits (scores in 32 bits with a bound on their error
// first, and 64 only where that leaves a choice open, was no faster: 31 against
// 29 us for 256 items of 512 blocks; latencies bound it, not arithmetic).
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
// key is read once and nothing is computed twice, so the bytes bound it (4 x
// 12-16k keys on 8 heads, 120 MB: 21.8 us, 5.5 TB/s; 22.3 with CTAs of 8 warps,
// 23.4 with the pages looked up one after the other).
template <int D, bool E8>
__global__ void __launch_bounds__(128, 7) key_bounds_kernel(const __grid_constant__ KeyBoundsParams p) {
  constexpr int ROW = D * (E8 ? 1 : 2), LPR = ROW / 16, RPI = 32 / LPR;
  constexpr int W = E8 ? 8 : 4;  // BF16 pairs of one 16-byte load
  const int lane = threadIdx.x & 31;
  long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
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
  if (j >= (len + (1 << p.block_shift) - 1) >> p.block_shift) return;  // past the sequence's end
  const int first = j << p.block_shift;
  if (p.start != nullptr && first + (1 << p.block_shift) <= __ldg(p.start + b)) return;  // bounds still hold
  const int n = min(1 << p.block_shift, len - first);
  const int sub = lane / LPR, unit = lane % LPR;
  uint32_t lo[W], hi[W];
#pragma unroll
  for (int w = 0; w < W; ++w) lo[w] = 0x7f807f80u, hi[w] = 0xff80ff80u;  // +inf, -inf
  // Pages are at least 16 rows and a block starts on a multiple of 16: 16 rows at a time share a page. Lane i looks up the
  // i-th 16 rows.
  int64_t page = b;
  if (p.c.page_table != nullptr && lane * 16 < n) {
    const int pg = __ldg(p.c.page_table + static_cast<int64_t>(b) * p.c.max_pages + ((first + lane * 16) >> p.c.page_shift));
    page = pg;
    if (pg < 0 || pg >= p.c.num_pages) {
      atomicOr(p.c.err, kErrPageIndex);
      page = -1;  // a bad page reads zeros
    }
  }
  for (int r0 = 0; r0 < n; r0 += 16) {
    const int pos = first + r0;
    const int64_t outer = __shfl_sync(kFull, page, r0 >> 4);
    const int64_t row = p.c.page_table != nullptr ? pos & ((1 << p.c.page_shift) - 1) : pos;
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

// The two BF16 halves of a word as doubles. Half of the values stay off the
// conversion pipe: the high half's exponent and mantissa are moved to a
// double's places, which is the value times 2^-896 (exact, subnormals too).
__device__ __forceinline__ double bf16_low(uint32_t w) { return static_cast<double>(__uint_as_float(w << 16)); }
__device__ __forceinline__ double bf16_high(uint32_t w) {
  return __hiloint2double(static_cast<int>((w & 0x80000000u) | ((w >> 3) & 0x0fffe000u)), 0);
}

constexpr int kPickThreads = 256, kPickWarps = kPickThreads / 32;

struct PickMisc {
  double half[2][128];  // down, up
  unsigned long long ends[2][kPickWarps];
  unsigned long long prefix;
  unsigned hist[256];
  int need, total;
  int warp_in[kPickWarps], warp_eq[kPickWarps];
};

// The `left`-th largest of keys [0, n), eight bits a pass from the highest bit
// in which they differ. Returns the key `limit` and how many of those equal to
// it are in (`need`, the lowest first); all above it are.
using Key = unsigned long long;
__device__ void nth_key(const Key* keys, int n, int left, PickMisc* m, Key& limit, int& need) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Key lo = ~0ull, hi = 0ull;
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
    lo = min(lo, m->ends[0][w]);
    hi = max(hi, m->ends[1][w]);
  }
  int shift = max(0, 56 - __clzll(static_cast<long long>((lo ^ hi) | 1ull)));
  int from = min(64, shift + 8);  // keys of the current bucket agree with `prefix` in all bits from `from` up
  Key prefix = from >= 64 ? 0ull : hi >> from << from;
  for (;;) {
    const unsigned digits = 1u << (from - shift);
    m->hist[tid] = 0u;
    __syncthreads();
    for (int j = tid; j < n; j += kPickThreads) {
      const Key k = keys[j];
      if (from >= 64 || (k >> from) == (prefix >> from)) atomicAdd(&m->hist[static_cast<unsigned>(k >> shift) & (digits - 1u)], 1u);
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
          m->prefix = prefix | (static_cast<Key>(255 - 8 * lane - e) << shift);
          m->need = left - static_cast<int>(before);
          m->total = static_cast<int>(c[e]);
        }
        before += c[e];
      }
    }
    __syncthreads();
    prefix = m->prefix;
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
    prefix = m->prefix;
  }
  limit = prefix;
  need = left;
}

// up and down of the tile's queries: thread (tid / U) sums every STEP-th row of
// the 8 channels of unit tid % U, and the STEP partial sums are added in order.
// up and down are half the sum and the difference of the sums of q and of |q|.
template <int D>
__device__ void half_sums(const SelectParams& p, const uint16_t* q, int tokens, double (*half)[128], double* part) {
  constexpr int U = D / 8, STEP = kPickThreads / U;  // 16-byte units of a row; rows per pass
  const int tid = threadIdx.x, unit = tid % U;
  // A single token's heads are the rows; else each head's tokens are.
  const bool one = tokens == 1;
  const int rows = one ? p.c.G : tokens, outer = one ? 1 : p.c.G;
  const int64_t row_stride = one ? p.q_sh : p.q_ss;
  double plain[8], mag[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) plain[e] = mag[e] = 0.0;
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
          const double d = e & 1 ? bf16_high(x[e >> 1]) : bf16_low(x[e >> 1]);
          plain[e] += d;
          mag[e] += fabs(d);
        }
      }
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double f = e & 1 ? 0x1p895 : 0.5;
    part[(tid / U) * 2 * D + unit * 8 + e] = f * (plain[e] - mag[e]);
    part[(tid / U) * 2 * D + D + unit * 8 + e] = f * (plain[e] + mag[e]);
  }
  __syncthreads();
  for (int i = tid; i < 2 * D; i += kPickThreads) {
    double sum = 0.0;
    for (int r = 0; r < STEP; ++r) sum += part[r * 2 * D + i];
    half[i / D][i % D] = sum;
  }
  __syncthreads();
}

// One cluster per (sequence, query tile, KV head): every CTA scores a share of
// the blocks into CTA 0's shared memory, which picks. Four CTAs fit an SM, so
// that the grids of ordinary calls are one wave. 256 items of up to 512 blocks
// (56 MB of bounds): 25 us; 512 tiles of 128 queries x 4 heads (67 MB of q): 24 us:
// what DRAM takes of it is 9 and 10 us, the rest is the chain of loads,
// reductions, barriers and passes of the pick.
template <int D>
__global__ void __launch_bounds__(kPickThreads, 4) select_blocks_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickMisc* m = reinterpret_cast<PickMisc*>(smem_raw);
  Key* keys = reinterpret_cast<Key*>(smem_raw + sizeof(PickMisc));  // of all blocks; before them, half_sums' parts
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
  const int left = p.top - (seen - (f1 - f0));
  const bool scored = !all && left > 0;
  if (scored) {
    half_sums<D>(p, p.q + b * p.q_sb + static_cast<int64_t>(t0) * p.q_ss + h * p.c.G * p.q_sh, t1 - t0, m->half,
                 reinterpret_cast<double*>(keys));
    if (p.cluster > 1) cluster_sync();  // every CTA of the cluster runs, and CTA 0 has read its parts
    constexpr int LPB = D / 4, BPW = 32 / LPB;  // a block's bounds are 4 D bytes: lanes per block; blocks per warp load
    const int in = lane % LPB;
    const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_blocks * 2 * D) + in;
    // All scores are held times 2^-496, within a double's normal range for every q and bound: the high halves lack
    // 2^896 of it.
    double w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = m->half[(in * 8 + e) / D][(in * 8 + e) % D] * (e & 1 ? 0x1p400 : 0x1p-496);
    const int stride = kPickWarps * p.cluster * BPW;
    const uint32_t dst = p.cluster > 1 ? in_cta(ptx::smem_addr(keys), 0) : 0u;
    for (int j = f0 + (rank * kPickWarps + warp) * BPW + lane / LPB; j - lane / LPB < f1; j += 4 * stride) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = j + i * stride < f1 ? __ldg(src + static_cast<int64_t>(j + i * stride) * LPB) : make_uint4(0u, 0u, 0u, 0u);
      double sum[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        sum[i] = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[i] = fma(w[e], e & 1 ? bf16_high(x[e >> 1]) : bf16_low(x[e >> 1]), sum[i]);
      }
      // Two halving steps leave each quarter of the lanes with one of the four blocks: 6 exchanges, not 20. Every
      // block's sum is the same tree of additions, so equal bounds score equal bits.
      const bool hi2 = in & (LPB / 2), hi1 = in & (LPB / 4);
      const double a0 = (hi2 ? sum[2] : sum[0]) + __shfl_xor_sync(kFull, hi2 ? sum[0] : sum[2], LPB / 2);
      const double a1 = (hi2 ? sum[3] : sum[1]) + __shfl_xor_sync(kFull, hi2 ? sum[1] : sum[3], LPB / 2);
      double score = (hi1 ? a1 : a0) + __shfl_xor_sync(kFull, hi1 ? a0 : a1, LPB / 4);
#pragma unroll
      for (int o = LPB / 8; o > 0; o >>= 1) score += __shfl_xor_sync(kFull, score, o);
      const int at = j + (2 * hi2 + hi1) * stride;
      if (in % (LPB / 4) == 0 && at < f1) {
        if (p.cluster > 1) st_cluster64(dst + at * 8, order_key(score));
        else keys[at] = order_key(score);
      }
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
  }
  if (rank != 0) return;

  Key limit = 0ull;
  int need = 0;
  if (scored) nth_key(keys + f0, f1 - f0, left, m, limit, need);
  // 0 out, 1 in, 2 in while `need` lasts. Without scores: all blocks, or the lowest `top` of the forced ones.
  auto verdict = [&](int j) -> int {
    if (all) return 1;
    if (!scored) return (j < f0 || j >= f1) && (j < f0 ? j : f0 + j - f1) < p.top;
    if (j < f0 || j >= f1) return 1;
    return keys[j] > limit ? 1 : keys[j] == limit ? 2 : 0;
  };
  // Warps take consecutive runs of blocks.
  const int run = ((seen + kPickWarps - 1) / kPickWarps + 31) & ~31;
  const int j0 = min(seen, warp * run), j1 = min(seen, j0 + run);
  int n_in = 0, n_eq = 0;
  for (int j = j0; j < j1; j += 32) {
    const int v = j + lane < j1 ? verdict(j + lane) : 0;
    n_in += __popc(__ballot_sync(kFull, v == 1));
    n_eq += __popc(__ballot_sync(kFull, v == 2));
  }
  if (lane == 0) m->warp_in[warp] = n_in, m->warp_eq[warp] = n_eq;
  __syncthreads();
  int at = 0, eq = 0;
  for (int w = 0; w < warp; ++w) at += m->warp_in[w], eq += m->warp_eq[w];
  at += min(eq, need);
  int32_t* list = nullptr;
  uint8_t* mask = nullptr;
  if (p.mask != nullptr) mask = p.mask + ((static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_tiles + tile) * p.n_blocks;
  else list = p.list + ((static_cast<int64_t>(b) * p.n_tiles + tile) * p.c.Hkv + h) * p.top;  // n_tiles = T
  const uint32_t below = (1u << lane) - 1u;
  for (int j = j0; j < j1; j += 32) {
    const int v = j + lane < j1 ? verdict(j + lane) : 0;
    const uint32_t equal = __ballot_sync(kFull, v == 2);
    const bool take = v == 1 || (v == 2 && eq + __popc(equal & below) < need);
    eq += __popc(equal);
    if (mask != nullptr) {
      if (j + lane < j1) mask[j + lane] = take;
      continue;
    }
    const uint32_t taken = __ballot_sync(kFull, take);
    if (take) list[at + __popc(taken & below)] = j + lane;
    at += __popc(taken);
  }
  if (mask != nullptr)
    for (int j = seen + tid; j < p.n_blocks; j += kPickThreads) mask[j] = 0;
  else
    for (int i = min(seen, p.top) + tid; i < p.top; i += kPickThreads) list[i] = -1;
}

}  // namespace

cudaError_t launch_key_bounds(int D, bool k8, const KeyBoundsParams& p, cudaStream_t s) {
  const long long items = static_cast<long long>(p.c.B) * p.c.Hkv * p.n_blocks;
  const unsigned grid = static_cast<unsigned>((items + 3) / 4);
  if (D == 64) {
    if (k8) key_bounds_kernel<64, true><<<grid, 128, 0, s>>>(p);
    else key_bounds_kernel<64, false><<<grid, 128, 0, s>>>(p);
  } else {
    if (k8) key_bounds_kernel<128, true><<<grid, 128, 0, s>>>(p);
    else key_bounds_kernel<128, false><<<grid, 128, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_select_blocks(int D, const SelectParams& p, cudaStream_t s) {
  auto kern = D == 64 ? select_blocks_kernel<64> : select_blocks_kernel<128>;
  // The keys' area also holds the partial sums of up and down (256 threads x 16 doubles).
  const size_t smem = sizeof(PickMisc) + std::max(size_t(p.n_blocks), size_t(kPickThreads) * 16) * 8;
  // The limit is the kernel's, not the launch's: calls of other sizes may be under way on other threads.
  const int most = static_cast<int>(sizeof(PickMisc) + size_t(kMaxPickBlocks) * 8);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
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
