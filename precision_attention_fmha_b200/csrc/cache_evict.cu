// cache_evict.cu -- which keys stay in a cache under a budget, and the cache
// with the kept rows moved together.
//
// Kept of n > budget keys: the first `sinks`, the last `recent`, and of the
// others the heaviest, ties to the lowest position: the set does not depend on
// how the work is spread. n <= budget keeps everything.
#include <algorithm>

#include "cache_tiles.cuh"

namespace fmha {
namespace {

// Orders like the floats (a larger weight has a larger key; -0 counts as +0, a NaN weighs less than anything).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0u;
  const uint32_t v = __float_as_uint(w + 0.f);
  return (v & 0x80000000u) ? ~v : v | 0x80000000u;
}

constexpr int kEvictThreads = 1024, kEvictWarps = kEvictThreads / 32;

// One CTA per (sequence, KV head): the `left`-th largest weight digit by digit
// (11 + 11 + 10 bits), then the kept positions in ascending order. (Four CTAs a
// head, joining their counters over distributed shared memory, were slower for
// 64 heads of 32768 weights, 35 against 27 us: eight cluster barriers.) 20 us
// for those: a fifth of it the weights' way here, the rest the passes of one
// SM a head.
// CACHED: the keys stay in shared memory between the passes.
constexpr int kEvictCached = 49152;  // keys
template <bool CACHED>
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t cached[];
  __shared__ unsigned hist[2048];
  __shared__ unsigned sums[kEvictWarps];
  __shared__ unsigned found[3];  // digit, rank inside it, its size
  __shared__ int warp_gt[kEvictWarps], warp_eq[kEvictWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.c.Hkv, h = blockIdx.x - b * p.c.Hkv;
  int n = __ldg(p.c.lens + b);
  const int room = min(p.c.capacity, p.n_weights);
  if (n < 0 || n > room) {
    if (tid == 0) atomicOr(p.c.err, kErrLength);
    n = min(max(n, 0), room);
  }
  const float* w = p.weights + (static_cast<int64_t>(b) * p.c.Hkv + h) * p.n_weights;
  int32_t* keep = p.keep + (static_cast<int64_t>(b) * p.c.Hkv + h) * p.budget;
  const int count = min(n, p.budget);
  if (tid == 0 && h == 0) p.counts[b] = count;
  for (int i = count + tid; i < p.budget; i += kEvictThreads) keep[i] = -1;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += kEvictThreads) keep[i] = i;
    return;
  }
  const int m0 = p.sinks, m1 = n - p.recent;  // the others: m0 < m1, since sinks + recent <= budget < n
  int left = p.budget - p.sinks - p.recent;
  if constexpr (CACHED) {
    if ((reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
      const int n4 = n >> 2;
      for (int i0 = tid; i0 < n4; i0 += 8 * kEvictThreads) {  // 128 bytes per thread in flight
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * kEvictThreads < n4) x[k] = __ldg(reinterpret_cast<const float4*>(w) + i0 + k * kEvictThreads);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * kEvictThreads < n4)
            *reinterpret_cast<uint4*>(&cached[4 * (i0 + k * kEvictThreads)]) =
                make_uint4(weight_key(x[k].x), weight_key(x[k].y), weight_key(x[k].z), weight_key(x[k].w));
      }
      for (int i = 4 * n4 + tid; i < n; i += kEvictThreads) cached[i] = weight_key(__ldg(w + i));
    } else {
      for (int i0 = tid; i0 < n; i0 += 8 * kEvictThreads) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = i0 + k * kEvictThreads < n ? __ldg(w + i0 + k * kEvictThreads) : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * kEvictThreads < n) cached[i0 + k * kEvictThreads] = weight_key(x[k]);
      }
    }
    __syncthreads();
  }
  auto key_of = [&](int i) { return CACHED ? cached[i] : weight_key(__ldg(w + i)); };
  uint32_t limit = 0xfffffffeu;  // keys above it stay, and `left` of those equal to it (no weight's key is as large)
  if (left > 0) {
    uint32_t prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < 2048; i += kEvictThreads) hist[i] = 0u;
      __syncthreads();
#pragma unroll 4
      for (int i = m0 + tid; i < m1; i += kEvictThreads) {
        const uint32_t k = key_of(i);
        if (pass == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits))) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // Thread t holds the two digits 2047 - 2 t and 2046 - 2 t: a scan from the top.
      const unsigned c0 = hist[2047 - 2 * tid], c1 = hist[2046 - 2 * tid];
      unsigned run = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(kFull, run, o);
        if (lane >= o) run += v;
      }
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      unsigned before = run - c0 - c1;
      for (int i = 0; i < warp; ++i) before += sums[i];
      const unsigned want = static_cast<unsigned>(left);
      if (before < want && before + c0 >= want) found[0] = 2047 - 2 * tid, found[1] = want - before, found[2] = c0;
      before += c0;
      if (before < want && before + c1 >= want) found[0] = 2046 - 2 * tid, found[1] = want - before, found[2] = c1;
      __syncthreads();
      prefix |= found[0] << shift;
      left = static_cast<int>(found[1]);
      __syncthreads();
    }
    limit = prefix;
  }
  // Warps take consecutive runs of positions, lanes words of an odd number of them, so that the lanes are in different banks
  // (votes over neighbouring keys: 6900 clocks, not 5000, for a run of 1024).
  const int run = ((n + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int words = (run + 991) / 992, width = (run / 32 + words - 1) / words | 1, step = 32 * width;  // words of a lane
  const int j0 = min(n, warp * run), j1 = min(n, j0 + run);
  auto verdicts = [&](int at, uint32_t& gt, uint32_t& eq) {
    gt = eq = 0u;
    if (at >= j1) return;
#pragma unroll 4  // a short loop: code that runs once waits for its instructions
    for (int i = 0; i < width; ++i) {
      const uint32_t k = key_of(min(at + i, n - 1));
      gt |= (k > limit ? 1u : 0u) << i;
      eq |= (k == limit ? 1u : 0u) << i;
    }
    auto below = [&](int j) { return j <= at ? 0u : j >= at + 32 ? kFull : (1u << (j - at)) - 1u; };
    const uint32_t forced = below(m0) | ~below(m1), live = below(min(j1, at + width));
    gt = (gt | forced) & live;
    eq = eq & ~forced & live;
  };
  uint32_t gt = 0u, eq = 0u, kept[2][2] = {{0u, 0u}, {0u, 0u}};
  int gt0 = 0, eq0 = 0;
  for (int j = j0; j < j1; j += step) {
    verdicts(j + width * lane, gt, eq);
    if (j == j0) kept[0][0] = gt, kept[0][1] = eq;
    else kept[1][0] = gt, kept[1][1] = eq;
    gt0 += __reduce_add_sync(kFull, __popc(gt));
    eq0 += __reduce_add_sync(kFull, __popc(eq));
  }
  if (lane == 0) warp_gt[warp] = gt0, warp_eq[warp] = eq0;
  __syncthreads();
  gt0 = __reduce_add_sync(kFull, lane < warp ? warp_gt[lane] : 0);
  eq0 = __reduce_add_sync(kFull, lane < warp ? warp_eq[lane] : 0);
  // Cached keys have done their work: at most two words a lane hold the verdicts, and the positions are listed in the keys'
  // place and written side by side from there.
  static_assert(kEvictCached <= kEvictWarps * 2 * 32 * 31, "two words a lane");
  int32_t* list = CACHED ? reinterpret_cast<int32_t*>(cached) : keep;
  for (int j = j0; j < j1; j += step) {
    if constexpr (CACHED) gt = kept[j != j0][0], eq = kept[j != j0][1];
    else verdicts(j + width * lane, gt, eq);
    // Verdicts of the words before: two counts of at most 1024 in one word.
    const uint32_t mine = __popc(gt) | __popc(eq) << 16;
    uint32_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, before, o);
      if (lane >= o) before += v;
    }
    const uint32_t total = __shfl_sync(kFull, before, 31);
    before -= mine;
    const int eqr = eq0 + static_cast<int>(before >> 16), room_eq = max(0, left - eqr);
    if (__popc(eq) > room_eq) {  // the first of them
      uint32_t rest = eq;
      for (int i = 0; i < room_eq; ++i) rest &= rest - 1u;
      eq ^= rest;
    }
    int32_t* to = list + gt0 + static_cast<int>(before & 0xffffu) + min(eqr, left);
    for (uint32_t word = gt | eq; word != 0u; word &= word - 1u) *to++ = j + width * lane + __ffs(word) - 1;
    gt0 += static_cast<int>(total & 0xffffu);
    eq0 += static_cast<int>(total >> 16);
  }
  if constexpr (!CACHED) return;
  __syncthreads();
  for (int i = tid; i < count; i += kEvictThreads) keep[i] = list[i];
}

// ------------------------------------------------------------------ compact --
struct Place {
  int64_t outer, row;
  bool ok;
};
__device__ __forceinline__ Place place(const int32_t* table, int max_pages, int pages, int shift, int capacity, int b,
                                       int pos, uint32_t* err) {
  if (pos < 0 || pos >= capacity) {
    atomicOr(err, kErrPageIndex);
    return {0, 0, false};
  }
  if (table == nullptr) return {b, pos, true};
  const int pg = __ldg(table + static_cast<int64_t>(b) * max_pages + (pos >> shift));
  if (pg < 0 || pg >= pages) {
    atomicOr(err, kErrPageIndex);
    return {0, 0, false};
  }
  return {pg, pos & ((1 << shift) - 1), true};
}

// Kept row i of (b, h): where it comes from and where it goes.
__device__ __forceinline__ bool kept_row(const CompactParams& p, int b, int h, int i, int start, Place& src, Place& dst,
                                         int& from) {
  const int32_t* keep = p.keep + b * p.keep_sb + h * p.keep_sh;
  from = __ldg(keep + i);
  if (p.in_place && (from < start + i || (i > 0 && __ldg(keep + i - 1) >= from))) {
    atomicOr(p.c.err, kErrPageIndex);  // moving up or out of order: other rows would be overwritten first
    return false;
  }
  src = place(p.c.page_table, p.c.max_pages, p.c.num_pages, p.c.page_shift, p.c.capacity, b, from, p.c.err);
  dst = place(p.out_table, p.out_max_pages, p.out_pages, p.out_page_shift, p.out_capacity, b, start + i, p.c.err);
  return src.ok && dst.ok;
}

__device__ __forceinline__ int kept_count(const CompactParams& p, int b) {
  int n = __ldg(p.counts + b);
  if (n < 0 || n > p.n_keep) {
    atomicOr(p.c.err, kErrLength);
    n = min(max(n, 0), p.n_keep);
  }
  return n;
}

// Where the moved rows of a sequence go. No cache and no list reaches 2^30 entries: a start cut to that is as far outside,
// and its sum with a row number stays in 32 bits.
__device__ __forceinline__ int start_of(const CompactParams& p, int b) {
  return p.dst_start != nullptr ? min(max(__ldg(p.dst_start + b), -(1 << 30)), 1 << 30) : 0;
}

// Into another cache: every row on its own; positions past the kept rows clear
// their weights. A warp takes 32 rows, one lane looking up each, and moves
// them with up to eight 16-byte loads per lane in flight: the bytes bound it
// (537 MB moved in 90 us; 8 rows a warp pay for their lookups, 106 us). With
// too few rows for that to fill the SMs it takes 8 (4096 rows: 13 -> 7 us).
__host__ __device__ inline int copy_runs(const CompactParams& p, int rows) {
  const int n = p.weights_out != nullptr && p.n_weights_out > p.n_keep ? p.n_weights_out : p.n_keep;
  return (n + rows - 1) / rows;
}
template <int kCopyRows>
__global__ void __launch_bounds__(256) compact_copy_kernel(const __grid_constant__ CompactParams p) {
  const int lane = threadIdx.x & 31;
  long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int h = static_cast<int>(item % p.c.Hkv);
  item /= p.c.Hkv;
  const int runs = copy_runs(p, kCopyRows);
  const int run = static_cast<int>(item % runs);
  const int b = static_cast<int>(item / runs);
  if (b >= p.c.B) return;
  const int count = kept_count(p, b);
  const int start = start_of(p, b);
  const int i = run * kCopyRows + lane;
  Place src{0, 0, false}, dst{0, 0, false};
  int from = 0;
  bool ok = false;
  if (lane < kCopyRows && i < count) ok = kept_row(p, b, h, i, start, src, dst, from);
  const int64_t ks = src.outer * p.k_sb + src.row * p.k_ss + h * p.k_sh, vs = src.outer * p.v_sb + src.row * p.v_ss + h * p.v_sh;
  const int64_t kd = dst.outer * p.ko_sb + dst.row * p.ko_ss + h * p.ko_sh, vd = dst.outer * p.vo_sb + dst.row * p.vo_ss + h * p.vo_sh;
  if (p.weights_out != nullptr && lane < kCopyRows && start + i >= 0 && start + i < p.n_weights_out && (ok || i >= count)) {
    const int64_t bh = static_cast<int64_t>(b) * p.c.Hkv + h;
    p.weights_out[bh * p.n_weights_out + start + i] = ok && from < p.n_weights ? p.weights[bh * p.n_weights + from] : 0.f;
  }
  const uint32_t live = __ballot_sync(kFull, ok);
  if (live == 0) return;
#pragma unroll
  for (int r0 = 0; r0 < kCopyRows; r0 += 8) {
    // 8 rows at a time: at most 4 loads of K and 4 of V (256-byte rows, two per warp load).
    uint4 x[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int lpr = (t ? p.v_bytes : p.k_bytes) / 16, rpl = 32 / lpr;  // lanes per row; rows per load
      const uint8_t* from_t = (t ? p.v : p.k) + (lane % lpr) * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k * rpl + lane / lpr;
        const int64_t at = __shfl_sync(kFull, t ? vs : ks, r & 31);
        if (r < r0 + 8 && ((live >> r) & 1u)) x[t][k] = __ldg(reinterpret_cast<const uint4*>(from_t + at));
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int lpr = (t ? p.v_bytes : p.k_bytes) / 16, rpl = 32 / lpr;
      uint8_t* to_t = (t ? p.v_out : p.k_out) + (lane % lpr) * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k * rpl + lane / lpr;
        const int64_t at = __shfl_sync(kFull, t ? vd : kd, r & 31);
        if (r < r0 + 8 && ((live >> r) & 1u)) *reinterpret_cast<uint4*>(to_t + at) = x[t][k];
      }
    }
  }
}

// Inside one cache: positions never grow (from >= start + i), so rows moved in
// ascending order never overwrite one that is still to be read. A CTA owns a
// 32-byte column of the rows of one (sequence, KV head) of K, or V, or the
// weights, and takes them 512 at a time: all loads, a barrier, all stores.
constexpr int kMoveThreads = 256, kMoveUnits = 4;
__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ CompactParams p) {
  const int cols = p.k_bytes / 32, cols_v = p.v_bytes / 32;  // 32-byte columns of a row
  const int bh = blockIdx.x, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  const int what = blockIdx.y;  // columns of K, then of V, then the weights
  const int count = kept_count(p, b);
  const int start = start_of(p, b);
  const int tid = threadIdx.x;
  if (what == cols + cols_v) {
    float* w = p.weights_out + static_cast<int64_t>(bh) * p.n_weights_out;
    for (int r0 = 0; r0 < count; r0 += kMoveThreads * kMoveUnits) {
      float x[kMoveUnits];
      int to[kMoveUnits];
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u) {
        const int i = r0 + u * kMoveThreads + tid;
        to[u] = -1;
        if (i >= count) continue;
        Place src, dst;
        int from;
        if (!kept_row(p, b, h, i, start, src, dst, from)) continue;  // a row that is left out leaves its weight
        if (start + i >= p.n_weights_out) continue;
        to[u] = start + i;
        x[u] = from < p.n_weights_out ? w[from] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u)
        if (to[u] >= 0) w[to[u]] = x[u];
      __syncthreads();
    }
    for (int i = max(0, start + count) + tid; i < p.n_weights_out; i += kMoveThreads) w[i] = 0.f;
    return;
  }
  const bool is_v = what >= cols;
  const int unit = (what - (is_v ? cols : 0)) * 32 + (tid & 1) * 16;
  uint8_t* base = (is_v ? p.v_out : p.k_out) + unit;
  const int64_t sb = is_v ? p.v_sb : p.k_sb, ss = is_v ? p.v_ss : p.k_ss, sh = is_v ? p.v_sh : p.k_sh;
  constexpr int ROWS = kMoveThreads / 2;
  for (int r0 = 0; r0 < count; r0 += ROWS * kMoveUnits) {
    uint4 x[kMoveUnits];
    uint8_t* to[kMoveUnits];
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      const int i = r0 + u * ROWS + (tid >> 1);
      to[u] = nullptr;
      if (i >= count) continue;
      Place src, dst;
      int from;
      if (!kept_row(p, b, h, i, start, src, dst, from) || from == start + i) continue;
      x[u] = *reinterpret_cast<const uint4*>(base + src.outer * sb + src.row * ss + h * sh);
      to[u] = base + dst.outer * sb + dst.row * ss + h * sh;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u)
      if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = x[u];
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s) {
  const int n = std::min(p.c.capacity, p.n_weights);
  if (n <= kEvictCached) {
    const int smem = std::max(n, 1) * 4;
    // The limit is the kernel's, not the launch's: calls of other sizes may be under way on other threads.
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictCached * 4);
    if (e != cudaSuccess) return e;
    evict_select_kernel<true><<<p.c.B * p.c.Hkv, kEvictThreads, smem, s>>>(p);
  } else {
    evict_select_kernel<false><<<p.c.B * p.c.Hkv, kEvictThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t s) {
  if (p.in_place) {
    compact_move_kernel<<<dim3(p.c.B * p.c.Hkv, p.k_bytes / 32 + p.v_bytes / 32 + (p.weights_out != nullptr ? 1 : 0)), kMoveThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  const long long heads = static_cast<long long>(p.c.B) * p.c.Hkv;
  const bool wide = heads * copy_runs(p, 32) >= 4096;  // warps: about 28 per SM
  const long long items = heads * copy_runs(p, wide ? 32 : 8);
  if (items == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>((items + 7) / 8);
  if (wide) compact_copy_kernel<32><<<grid, 256, 0, s>>>(p);
  else compact_copy_kernel<8><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fmha
