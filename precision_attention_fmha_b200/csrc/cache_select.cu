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
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory variable in CTA 0 of the cluster.
__device__ __forceinline__ uint32_t in_cta0(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Orders like the doubles: a larger score has a larger key; -0 counts as +0.
__device__ __forceinline__ unsigned long long order_key(double x) {
  const long long v = __double_as_longlong(x + 0.0);
  return static_cast<unsigned long long>(v) ^ (v < 0 ? ~0ull : 1ull << 63);
}

constexpr int kPickThreads = 256;

struct PickMisc {
  double half[2][128];     // down, up
  unsigned hist[256];
  unsigned long long prefix;
  int need, total;
  int warp_gt[kPickThreads / 32], warp_eq[kPickThreads / 32];
};

// One cluster per (sequence, query tile, KV head): every CTA scores a share of
// the blocks into CTA 0's shared memory, which then finds the `top`-th largest
// key digit by digit and writes the blocks above it in ascending order.
template <int D>
__global__ void __launch_bounds__(kPickThreads) select_blocks_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickMisc* m = reinterpret_cast<PickMisc*>(smem_raw);
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(smem_raw + sizeof(PickMisc));
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
  if (!all) {
    // up and down of this tile, in 64 bits.
    constexpr int U = D / 8, STEP = kPickThreads / U;  // 16-byte units of a row; rows per pass
    double up[8], down[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) up[e] = down[e] = 0.0;
    const int unit = tid % U, rows = (t1 - t0) * p.c.G;
    for (int r = tid / U; r < rows; r += STEP) {
      const int t = r / p.c.G, g = r - t * p.c.G;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.q + b * p.q_sb + (t0 + t) * p.q_ss +
                                                           (h * p.c.G + g) * p.q_sh + unit * 8));
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = __uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16);
        up[e] += static_cast<double>(fmaxf(f, 0.f));
        down[e] += static_cast<double>(fminf(f, 0.f));
      }
    }
    // Join the passes' partial sums through the key area (STEP x 2 x D doubles, STEP * U = 256 threads).
    double* part = reinterpret_cast<double*>(keys);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      part[(tid / U) * 2 * D + unit * 8 + e] = down[e];
      part[(tid / U) * 2 * D + D + unit * 8 + e] = up[e];
    }
    __syncthreads();
    for (int i = tid; i < 2 * D; i += kPickThreads) {
      double sum = 0.0;
      for (int r = 0; r < STEP; ++r) sum += part[r * 2 * D + i];
      m->half[i / D][i % D] = sum;
    }
    __syncthreads();
    if (p.cluster > 1) cluster_sync();  // CTA 0's key area is free
    // One block is 4 D bytes of bounds: a 16-byte unit per lane.
    constexpr int LPB = D / 4, BPW = 32 / LPB;  // lanes per block; blocks per warp load
    double w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = (&m->half[0][0])[((lane % LPB) * 8 + e) / D * 128 + ((lane % LPB) * 8 + e) % D];
    const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_blocks * 2 * D);
    const int stride = kPickThreads / 32 * p.cluster * BPW;
    const uint32_t dst = p.cluster > 1 ? in_cta0(ptx::smem_addr(keys)) : ptx::smem_addr(keys);
    for (int j0 = (rank * (kPickThreads / 32) + warp) * BPW; j0 < seen; j0 += 4 * stride) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * stride + lane / LPB;
        v[i] = j < seen ? __ldg(src + static_cast<int64_t>(j) * LPB + lane % LPB) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * stride + lane / LPB;
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        double sum = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sum = fma(w[e], static_cast<double>(__uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16)), sum);
#pragma unroll
        for (int o = LPB / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (lane % LPB == 0 && j < seen) {
          const bool forced = j < p.sinks || j >= seen - p.recent;
          const unsigned long long key = forced ? ~0ull : order_key(sum);
          if (p.cluster > 1) st_cluster(dst + j * 8, key);
          else keys[j] = key;
        }
      }
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
  }
  if (rank != 0) return;

  // The top-th largest key: eight bits a pass, from the highest.
  unsigned long long limit = 0;  // keys above `limit` are picked, and `need` of those equal to it
  int need = 0;
  if (!all) {
    int left = p.top;
    unsigned long long prefix = 0;
    int shift = 56;
    for (;; shift -= 8) {
      m->hist[tid] = 0u;
      __syncthreads();
      for (int j = tid; j < seen; j += kPickThreads) {
        const unsigned long long k = keys[j];
        if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&m->hist[(k >> shift) & 255u], 1u);
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
            m->prefix = prefix | (static_cast<unsigned long long>(255 - 8 * lane - e) << shift);
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
      if (shift == 0) {
        limit = prefix;
        need = left;
        break;
      }
      if (left == total) {  // the whole bucket is picked
        limit = prefix - 1;  // prefix > 0: a bucket of digit 0 at every level would hold all keys
        need = 0;
        break;
      }
    }
  }
  // Warps take consecutive runs of blocks; ties go to the lowest.
  const int run = ((seen + kPickThreads / 32 - 1) / (kPickThreads / 32) + 31) & ~31;
  const int j0 = warp * run, j1 = min(seen, j0 + run);
  int gt = 0, eq = 0;
  for (int j = j0; j < j1; j += 32) {
    const bool in = j + lane < j1;
    const unsigned long long k = in && !all ? keys[j + lane] : 0ull;
    gt += __popc(__ballot_sync(kFull, in && (all || k > limit)));
    eq += __popc(__ballot_sync(kFull, in && !all && k == limit));
  }
  if (lane == 0) m->warp_gt[warp] = gt, m->warp_eq[warp] = eq;
  __syncthreads();
  int gt0 = 0, eq0 = 0;
  for (int w = 0; w < warp; ++w) gt0 += m->warp_gt[w], eq0 += m->warp_eq[w];
  const int64_t row = (static_cast<int64_t>(b) * p.n_tiles + tile) * p.c.Hkv + h;  // list form: n_tiles = T
  int32_t* list = p.list + row * p.top;
  uint8_t* mask = p.mask + ((static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_tiles + tile) * p.n_blocks;
  const uint32_t below = (1u << lane) - 1u;
  for (int j = j0; j < j1; j += 32) {
    const bool in = j + lane < j1;
    const unsigned long long k = in && !all ? keys[j + lane] : 0ull;
    const bool g = in && (all || k > limit), e = in && !all && k == limit;
    const uint32_t bg = __ballot_sync(kFull, g), be = __ballot_sync(kFull, e);
    const int eqr = eq0 + __popc(be & below);
    const bool take = g || (e && eqr < need);
    if (p.mask != nullptr) {
      if (in) mask[j + lane] = take ? 1 : 0;
    } else if (take) {
      list[gt0 + __popc(bg & below) + min(eqr, need)] = j + lane;
    }
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  if (p.mask != nullptr) {
    for (int j = seen + tid; j < p.n_blocks; j += kPickThreads) mask[j] = 0;
  } else {
    for (int i = min(seen, p.top) + tid; i < p.top; i += kPickThreads) list[i] = -1;
  }
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

cudaError_t launch_select_blocks(int D, const SelectParams& p, cudaStream_t s) {
  auto kern = D == 64 ? select_blocks_kernel<64> : select_blocks_kernel<128>;
  // The key area also holds the partial sums of up and down: 256 threads x 16 doubles.
  const size_t area = std::max<size_t>(size_t(p.n_blocks) * 8, size_t(kPickThreads) * 16 * 8);
  const size_t smem = sizeof(PickMisc) + area;
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
