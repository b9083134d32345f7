// api_cache.cu -- C ABI of the operators over a ragged K/V cache: argument
// checks, TMA descriptors and launch shapes (include/fmha.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_internal.h"
#include "host_common.h"

namespace {

using namespace fmha;
using namespace fmha::host;

constexpr int kTile = 64;  // keys of one tile of the few-row kernels

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Checks what every operator over the cache reads (need_v: V too; need_q: the
// queries), and fills the view. *k8 / *v8: E4M3 keys / values.
fmha_status check_cache(const fmha_cache_args* a, bool need_q, bool need_v, CacheView* c, bool* k8, bool* v8) {
  const int B = a->B, T = a->T, Hq = a->Hq, Hkv = a->Hkv, D = a->D;
  memset(c, 0, sizeof(*c));
  if (D != 64 && D != 128) return fail(FMHA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", D);
  if (need_q && (Hkv == 0 || Hq % Hkv != 0))
    return fail(FMHA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  *k8 = a->k.dtype == FMHA_E4M3;
  if (!*k8 && a->k.dtype != FMHA_BF16) return fail(FMHA_ERR_UNSUPPORTED, "K dtype %d unsupported", a->k.dtype);
  fmha_status st;
  if ((st = check_sf(a->sf_k, "sf_k", *k8, *k8, false, 1, false)) != FMHA_OK) return st;
  if (need_v) {
    *v8 = a->v.dtype == FMHA_E4M3;
    if (!*v8 && a->v.dtype != FMHA_BF16) return fail(FMHA_ERR_UNSUPPORTED, "V dtype %d unsupported", a->v.dtype);
    if (*k8 && !*v8) return fail(FMHA_ERR_UNSUPPORTED, "E4M3 keys need E4M3 values");
    if ((st = check_sf(a->sf_v, "sf_v", *v8, *v8, false, 1, false)) != FMHA_OK) return st;
  }
  int capacity = a->capacity;
  if (capacity < 0) return fail(FMHA_ERR_INVALID_ARG, "negative capacity");
  if (a->page_table != nullptr) {
    if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128)
      return fail(FMHA_ERR_UNSUPPORTED, "page_size %d (supported: 16, 32, 64, 128)", a->page_size);
    if (a->num_pages <= 0) return fail(FMHA_ERR_INVALID_ARG, "num_pages must be positive");
    if (a->max_pages_per_seq < 0) return fail(FMHA_ERR_INVALID_ARG, "negative max_pages_per_seq");
    if (reinterpret_cast<uintptr_t>(a->page_table) & 3u) return fail(FMHA_ERR_INVALID_ARG, "page_table misaligned");
    const int64_t room = static_cast<int64_t>(a->max_pages_per_seq) * a->page_size;
    if (room > INT32_MAX / 2) return fail(FMHA_ERR_UNSUPPORTED, "more than 2^30 tokens per sequence");
    if (capacity == 0) capacity = static_cast<int>(room);
    if (capacity > room) return fail(FMHA_ERR_INVALID_ARG, "capacity %d exceeds the page table's %d", capacity, (int)room);
  }
  if (capacity > INT32_MAX / 2) return fail(FMHA_ERR_UNSUPPORTED, "more than 2^30 tokens per sequence");
  if (a->lens == nullptr || (reinterpret_cast<uintptr_t>(a->lens) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "lens is NULL or misaligned");
  if (reinterpret_cast<uintptr_t>(a->q_lens) & 3u) return fail(FMHA_ERR_INVALID_ARG, "q_lens misaligned");
  if (reinterpret_cast<uintptr_t>(a->lse) & 3u) return fail(FMHA_ERR_INVALID_ARG, "lse misaligned");
  if (capacity > 0) {
    const int n = a->page_table != nullptr ? a->num_pages : B;
    const int s = a->page_table != nullptr ? a->page_size : capacity;
    if ((st = check_tensor(a->k, "k", n, s, Hkv, D)) != FMHA_OK) return st;
    if (need_v && (st = check_tensor(a->v, "v", n, s, Hkv, D)) != FMHA_OK) return st;
  }
  if (need_q) {
    if (a->q.dtype != FMHA_BF16) return fail(FMHA_ERR_UNSUPPORTED, "q must be BF16");
    if ((st = check_tensor(a->q, "q", B, T, Hq, D)) != FMHA_OK) return st;
    if (static_cast<int64_t>(T) * (Hq / Hkv) > INT32_MAX / 2)
      return fail(FMHA_ERR_UNSUPPORTED, "T * Hq / Hkv rows exceed 2^30");
  }
  c->B = B; c->T = T; c->Hq = Hq; c->Hkv = Hkv; c->G = need_q ? Hq / Hkv : 1;
  c->capacity = capacity;
  c->lens = a->lens;
  c->q_lens = a->q_lens;
  c->page_table = capacity > 0 ? a->page_table : nullptr;
  c->num_pages = a->num_pages;
  c->page_shift = a->page_table != nullptr ? log2_of(a->page_size) : 0;
  c->max_pages = a->max_pages_per_seq;
  return FMHA_OK;
}

// The current device's part of a view; after all argument checks.
fmha_status bind_device(CacheView* c) {
  cudaError_t e;
  c->err = device_error_word(&e);
  if (c->err == nullptr) return fail(FMHA_ERR_CUDA, "device error word: %s", cudaGetErrorString(e));
  c->wait_cycles = wait_cycles();
  return FMHA_OK;
}

// TMA map of K or V: boxes of `rows` tokens of one KV head and one swizzle column.
fmha_status cache_map(CUtensorMap* m, const fmha_cache_args* a, const CacheView& c, const fmha_tensor& t, bool e8,
                      int rows, const char* what) {
  const int eb = e8 ? 1 : 2;
  const int span = std::min(128, a->D * eb);
  const bool paged = c.page_table != nullptr;
  const uint64_t dims[4] = {uint64_t(a->D), uint64_t(a->Hkv), uint64_t(paged ? a->page_size : c.capacity),
                            uint64_t(paged ? a->num_pages : a->B)};
  const int64_t strides[3] = {t.stride_h, t.stride_s, t.stride_b};
  const uint32_t box[4] = {uint32_t(span / eb), 1, uint32_t(rows), 1};
  // L2 fetches no more than one head's row of a token: the neighbouring head's belongs to another CTA, and by the time
  // that one asks it is gone (E4M3, D = 128, 256-byte fetches: 600 MB read from DRAM for 452).
  const int row = a->D * eb;
  return make_map_n<4>(m, t.ptr, eb, dims, strides, box, what,
                       span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       row >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                  : row >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
}

// Which calls send their contexts to the packed kernel: from 128 packed rows (T * G) a whole tensor-memory tile; from 33
// where (sequence, KV head) pairs give at least half the SMs a CTA. Few-row kernel against packed, 64 rows: 16 contexts of
// 8-16k keys on 8 heads 283 against 163 us, 16 of 0.5-4k 79 against 69, 2 of 31k 106 against 118; 48 rows, 16 of 8-16k 282
// against 160, 2 of 1.2k 19 against 25; 32 rows, 16 of 8-16k 150 against 158, 16 of 0.5-4k 50 against 64.
constexpr int kPackedRows = 33, kPackedTile = 128;
constexpr int kPackedKeys = 1024;  // keys of room; below, the packed kernel would mostly start and end
constexpr int kPackedCtasPerSm = 1;

// The sizes of an attention call that do not need the device: grid and row
// tiles of the tree form.
struct TreePlan {
  int rows, row_tiles, n_ctas, groups;
  // The context's whole 128-key tiles on the decode path's packed kernel: query-tile units of a KV head, KV splits and
  // partial outputs, which the few-row kernel joins with what it takes itself. 0 parts: it takes everything.
  int units, n_splits, interleave, n_parts;
  size_t workspace_bytes;
};
constexpr int kMinTiles = 2;  // least key tiles of a group

// Groups of `heads` CTAs (one per KV head and row tile) that share the list of key tiles: as many as are resident at once,
// or, where that leaves a thin last wave, the number with the least waves times work per CTA. At most `most` have work.
int list_groups(int64_t heads, int64_t resident, int64_t most) {
  int64_t best = 1;
  double least = 1e30;
  const int64_t limit = std::max<int64_t>(1, std::min(most, heads >= resident ? int64_t(4) : resident / heads));
  for (int64_t g = heads >= resident ? 1 : limit; g <= limit; ++g) {
    const double cost = static_cast<double>((heads * g + resident - 1) / resident) / static_cast<double>(g);
    if (cost < least * 0.999) least = cost, best = g;
  }
  return static_cast<int>(best);
}

// Whether the context goes through 128-row tensor-memory tiles: many packed rows, and what that kernel is built for.
bool tree_packed(const fmha_cache_args* a, int capacity) {
  const int G = a->Hq / a->Hkv;
  const int64_t rows = static_cast<int64_t>(a->T) * G;
  return a->D == 128 && a->k.dtype == FMHA_BF16 && a->v.dtype == FMHA_BF16 && (G & (G - 1)) == 0 && G <= 128 &&
         (rows >= kPackedTile || (rows >= kPackedRows && 2 * static_cast<int64_t>(a->B) * a->Hkv >= sm_count())) &&
         capacity >= kPackedKeys && capacity <= 131072;
}

bool tree_plan(const fmha_cache_args* a, int capacity, TreePlan* t) {
  const int64_t packed = static_cast<int64_t>(a->T) * (a->Hq / a->Hkv);
  t->rows = cache_attn_rows(static_cast<int>(std::min<int64_t>(packed, 1 << 20)));
  t->row_tiles = static_cast<int>((packed + t->rows - 1) / t->rows);
  const int64_t items = static_cast<int64_t>(a->B) * a->Hkv * t->row_tiles;
  const int64_t tiles = static_cast<int64_t>(a->B) * ceil_div(std::max(capacity, 1), kTile);
  t->groups = list_groups(static_cast<int64_t>(a->Hkv) * t->row_tiles, cache_attn_ctas(t->rows) * sm_count(),
                          (tiles + kMinTiles - 1) / kMinTiles);
  if (static_cast<int64_t>(a->Hkv) * t->row_tiles * t->groups >= (int64_t(1) << 30)) return false;
  t->n_ctas = a->Hkv * t->row_tiles * t->groups;
  t->workspace_bytes = size_t(2) * t->n_ctas * t->rows * (size_t(a->D) + 1) * 4;
  t->n_parts = 0;
  if (tree_packed(a, capacity)) {
    const int tiles128 = ceil_div(static_cast<int>(packed), 128);
    t->interleave = tiles128 == 1 ? 1 : 0;
    t->units = t->interleave ? 1 : ceil_div(tiles128, 2);
    const int64_t base = static_cast<int64_t>(a->B) * a->Hkv * t->units;
    const int kv = ceil_div(capacity, 128);
    // About one CTA per SM (16 x 64 rows: 434 us; with two 469, with three 579: more partial results to join than the
    // evener lengths save); a split keeps at least 8 tiles.
    const int64_t want = (kPackedCtasPerSm * sm_count() + base - 1) / base;
    t->n_splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, kv / 8)));
    t->n_parts = t->n_splits * (t->interleave ? 2 : 1);
    t->n_ctas = static_cast<int>(std::min<int64_t>(2 * sm_count(), items));
    t->workspace_bytes = size_t(t->n_parts) * a->B * a->T * a->Hq * (size_t(a->D) + 1) * 4;
    if (base * t->n_splits >= (int64_t(1) << 31) || static_cast<int64_t>(a->B) * a->T * a->Hq >= (int64_t(1) << 32)) return false;
  }
  return items < (int64_t(1) << 31) && tiles / t->groups < (int64_t(1) << 30);
}

struct PickPlan {
  int rows, row_tiles, item_tiles, n_splits, per_split, n_ctas;
  size_t workspace_bytes;
};
bool pick_plan(const fmha_cache_args* a, int top, int block, PickPlan* t) {
  const int G = a->Hq / a->Hkv;
  t->rows = cache_attn_rows(G);
  t->row_tiles = ceil_div(G, t->rows);
  const int64_t items = static_cast<int64_t>(a->B) * a->T * a->Hkv * t->row_tiles;
  t->item_tiles = static_cast<int>((static_cast<int64_t>(top) * block + kTile - 1) / kTile);
  const int target = cache_attn_ctas(t->rows) * sm_count();
  int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(target / std::max<int64_t>(1, items), t->item_tiles)));
  t->per_split = ceil_div(t->item_tiles, splits);
  t->n_splits = ceil_div(t->item_tiles, t->per_split);
  t->n_ctas = static_cast<int>(std::min<int64_t>(items * t->n_splits, t->n_splits > 1 ? items * t->n_splits : target));
  t->workspace_bytes = t->n_splits > 1 ? size_t(2) * t->n_ctas * t->rows * (size_t(a->D) + 1) * 4 : 0;
  return items < (int64_t(1) << 31);
}

bool sizes_ok(const fmha_cache_args* a) {
  return a != nullptr && a->B >= 0 && a->T >= 0 && a->Hq >= 0 && a->Hkv >= 0 && a->D >= 0;
}
// Queries that divide over the KV heads, and rows that fit 32 bits.
bool rows_ok(const fmha_cache_args* a) {
  return sizes_ok(a) && a->B > 0 && a->T > 0 && a->Hq > 0 && a->Hkv > 0 && a->Hq % a->Hkv == 0 &&
         static_cast<int64_t>(a->T) * (a->Hq / a->Hkv) <= INT32_MAX / 2;
}
int64_t capacity_of(const fmha_cache_args* a) {
  if (a->capacity != 0 || a->page_table == nullptr) return a->capacity;
  return static_cast<int64_t>(a->max_pages_per_seq) * a->page_size;
}

fmha_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return FMHA_OK;
  if (ws == nullptr || !aligned16(ws)) return fail(FMHA_ERR_INVALID_ARG, "workspace is NULL or not 16-byte aligned");
  if (have < need) return fail(FMHA_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed", have, need);
  return FMHA_OK;
}

fmha_status check_block(int block) {
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(FMHA_ERR_UNSUPPORTED, "block %d (supported: 16, 32, 64, 128)", block);
  return FMHA_OK;
}

// Query tokens from which fmha_key_weights runs on the tensor cores' 128-token tiles.
constexpr int kManyQueries = 64;

// How a prompt's query tiles (128 tokens of one head) are cut into runs: about four per resident CTA in all, so that
// the last ones to end differ little, each of at least 8 tiles (its keys are loaded anew).
struct WeightRuns {
  int chunk, parts;
};
WeightRuns weight_runs(const fmha_cache_args* a, int capacity, int n_weights, int causal) {
  const int64_t most = static_cast<int64_t>(ceil_div(a->T, 128)) * (a->Hq / a->Hkv);  // of one key tile
  const int64_t keys = ceil_div(std::min(capacity, n_weights), 128);
  int64_t total = static_cast<int64_t>(a->B) * a->Hkv * keys * most;
  if (causal && capacity <= 2 * static_cast<int64_t>(a->T)) total /= 2;
  const int64_t chunk = std::min(most, std::max<int64_t>(8, total / (8 * sm_count())));
  return {static_cast<int>(chunk), static_cast<int>((most + chunk - 1) / chunk)};
}

// The item counter, then (several runs) their sums.
size_t weight_bytes(const fmha_cache_args* a, const WeightRuns& r, int n_weights) {
  return 16 + (r.parts > 1 ? size_t(r.parts) * a->B * a->Hkv * n_weights * 4 : 0);
}

// CTAs that score the blocks of one item: up to three per SM, while each keeps at least the 32 blocks that its warps
// load at once. 256 items of 512 blocks, with the attention after them: one CTA 66.4 us, two 64.5, four 72.4; 512 items
// of 64: one CTA 271, two 292.
int pick_cluster(int64_t items, int n_blocks) {
  int c = 1;
  while (c < 8 && items * c < 3 * sm_count() && n_blocks / (2 * c) >= 32) c *= 2;
  return c;
}

// Checks and fills what the tree and the picked form share.
fmha_status fill_attn(const fmha_cache_args* a, CacheAttnParams* p, bool* k8, bool* v8, int piece) {
  fmha_status st;
  memset(p, 0, sizeof(*p));
  if ((st = check_cache(a, true, true, &p->c, k8, v8)) != FMHA_OK) return st;
  if (a->o.dtype != FMHA_BF16) return fail(FMHA_ERR_UNSUPPORTED, "o must be BF16");
  if ((st = check_tensor(a->o, "o", a->B, a->T, a->Hq, a->D)) != FMHA_OK) return st;
  p->q = static_cast<const uint16_t*>(a->q.ptr);
  p->q_sb = a->q.stride_b; p->q_ss = a->q.stride_s; p->q_sh = a->q.stride_h;
  p->o = static_cast<uint16_t*>(a->o.ptr);
  p->o_sb = a->o.stride_b; p->o_ss = a->o.stride_s; p->o_sh = a->o.stride_h;
  p->lse = a->lse;
  const float scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(float(a->D));
  p->scale_log2 = scale * 1.4426950408889634f;
  p->sf_k = a->sf_k.ptr; p->sf_k_kind = a->sf_k.kind;
  p->sf_v = a->sf_v.ptr; p->sf_v_kind = a->sf_v.kind;
  piece = std::min(piece, kTile);
  if (p->c.page_table != nullptr) piece = std::min(piece, a->page_size);
  p->piece_shift = log2_of(piece);
  return FMHA_OK;
}

// The device's part: the error word and the TMA maps.
fmha_status bind_attn(const fmha_cache_args* a, CacheAttnParams* p, bool k8, bool v8, CUtensorMap* tk, CUtensorMap* tv) {
  fmha_status st;
  if ((st = bind_device(&p->c)) != FMHA_OK) return st;
  if (p->c.capacity == 0) {  // no key is ever loaded; any valid map will do
    const uint64_t dims[4] = {uint64_t(a->D), 1, 1, 1};
    const int64_t strides[3] = {a->D, a->D, a->D};
    const uint32_t box[4] = {64, 1, 1, 1};
    if ((st = make_map_n<4>(tk, a->q.ptr, 2, dims, strides, box, "q")) != FMHA_OK) return st;
    *tv = *tk;
    return FMHA_OK;
  }
  const int piece = 1 << p->piece_shift;
  if ((st = cache_map(tk, a, p->c, a->k, k8, piece, "k")) != FMHA_OK) return st;
  return cache_map(tv, a, p->c, a->v, v8, piece, "v");
}

// The packed kernel's parameters for the contexts' whole 128-key tiles: every row sees every key of them, and every
// tile's partial O / l and log-sum-exp go to the workspace.
fmha_status packed_params(const fmha_cache_args* a, const CacheAttnParams& c, const TreePlan& t, AttnParams* p,
                          CUtensorMap* tq, CUtensorMap* tk, CUtensorMap* tv) {
  const int G = a->Hq / a->Hkv, D = a->D;
  memset(p, 0, sizeof(*p));
  p->B = a->B; p->Hq = a->Hq; p->Hkv = a->Hkv; p->Sq = a->T; p->Skv = c.c.capacity; p->group = G;
  p->n_q_blocks = ceil_div(a->T, 128);
  p->n_kv_blocks = ceil_div(c.c.capacity, 128);
  p->scale_log2 = c.scale_log2;
  p->packed = 1;
  p->group_shift = log2_of(G);
  p->n_rows = a->T * G;
  p->n_units = t.units;
  p->n_splits = t.n_splits;
  p->split_tiles = ceil_div(p->n_kv_blocks, t.n_splits);
  p->kv_interleave = t.interleave;
  p->n_parts = t.n_parts + 1;  // more than one: every tile writes a partial, which the tail joins
  p->ctx_lens = c.c.lens;
  p->q_lens = c.c.q_lens;
  p->o_part = c.part_o;
  p->lse_part = c.part_lse;
  p->p_terms = 1;
  p->page_table = c.c.page_table; p->num_pages = a->num_pages; p->page_size = a->page_size;
  p->max_pages_per_seq = a->max_pages_per_seq;
  p->err = c.c.err;
  p->wait_cycles = c.c.wait_cycles;
  fmha_status st;
  const uint64_t dims[5] = {uint64_t(D), uint64_t(G), uint64_t(a->Hkv), uint64_t(a->T), uint64_t(a->B)};
  const int64_t str[4] = {a->q.stride_h, a->q.stride_h * G, a->q.stride_s, a->q.stride_b};
  const uint32_t box[5] = {64, uint32_t(G), 1, uint32_t(128 / G), 1};
  if ((st = make_map_n<5>(tq, a->q.ptr, 2, dims, str, box, "q")) != FMHA_OK) return st;
  const int rows = c.c.page_table != nullptr ? a->page_size : 128;
  if ((st = cache_map(tk, a, c.c, a->k, false, rows, "k")) != FMHA_OK) return st;
  return cache_map(tv, a, c.c, a->v, false, rows, "v");
}

}  // namespace

extern "C" {

size_t fmha_fwd_tree_workspace_bytes(const fmha_cache_args* a) {
  if (!rows_ok(a) || capacity_of(a) < 0 || capacity_of(a) > INT32_MAX / 2) return 0;
  TreePlan t;
  return tree_plan(a, static_cast<int>(capacity_of(a)), &t) ? t.workspace_bytes : 0;
}

fmha_status fmha_fwd_tree(const fmha_cache_args* a, const uint8_t* tree_mask, int64_t mask_stride_b, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (!sizes_ok(a)) return fail(FMHA_ERR_INVALID_ARG, "negative size");
  if (a->B == 0 || a->T == 0 || a->Hq == 0) return ok_status();  // nothing to compute
  if (mask_stride_b < 0) return fail(FMHA_ERR_INVALID_ARG, "mask stride must be >= 0");
  CacheAttnParams p;
  CUtensorMap tk, tv;
  bool k8, v8;
  fmha_status st;
  if ((st = fill_attn(a, &p, &k8, &v8, kTile)) != FMHA_OK) return st;
  TreePlan t;
  if (!tree_plan(a, p.c.capacity, &t)) return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
  if ((st = check_workspace(workspace, workspace_bytes, t.workspace_bytes)) != FMHA_OK) return st;
  if ((st = bind_attn(a, &p, k8, v8, &tk, &tv)) != FMHA_OK) return st;
  p.mask = tree_mask;
  p.mask_sb = mask_stride_b;
  p.row_tiles = t.row_tiles;
  p.tile_rows = t.rows;
  p.n_ctas = t.n_ctas;
  p.groups = t.groups;
  p.min_tiles = kMinTiles;
  p.part_o = static_cast<float*>(workspace);
  cudaError_t e;
  if (t.n_parts > 0) {
    p.part_lse = p.part_o + size_t(t.n_parts) * a->B * a->T * a->Hq * a->D;
    p.n_parts = t.n_parts;
    AttnParams ap;
    CUtensorMap tq, tkp, tvp;
    if ((st = packed_params(a, p, t, &ap, &tq, &tkp, &tvp)) != FMHA_OK) return st;
    e = launch_attention_ragged(p.c.page_table != nullptr, ap, tq, tkp, tvp, stream);
    if (e == cudaSuccess) e = launch_cache_tail(p, tk, tv, stream);
  } else {
    p.part_lse = p.part_o + size_t(2) * t.n_ctas * t.rows * a->D;
    e = launch_cache_attn(a->D, k8, v8, p, tk, tv, stream);
    if (e == cudaSuccess) e = launch_cache_merge(a->D, p, stream);
  }
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "tree attention launch: %s", cudaGetErrorString(e));
  return ok_status();
}

size_t fmha_fwd_selected_workspace_bytes(const fmha_cache_args* a, int32_t top, int32_t block) {
  if (!rows_ok(a) || top <= 0 || block <= 0 || static_cast<int64_t>(top) * block > INT32_MAX / 2) return 0;
  PickPlan t;
  return pick_plan(a, top, block, &t) ? t.workspace_bytes : 0;
}

fmha_status fmha_fwd_selected(const fmha_cache_args* a, const int32_t* blocks, int32_t top, int32_t block,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (!sizes_ok(a)) return fail(FMHA_ERR_INVALID_ARG, "negative size");
  if (a->B == 0 || a->T == 0 || a->Hq == 0) return ok_status();  // nothing to compute
  fmha_status st;
  if ((st = check_block(block)) != FMHA_OK) return st;
  if (top <= 0 || static_cast<int64_t>(top) * block > INT32_MAX / 2)
    return fail(FMHA_ERR_INVALID_ARG, "top %d out of range", top);
  if (blocks == nullptr || (reinterpret_cast<uintptr_t>(blocks) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "blocks is NULL or misaligned");
  CacheAttnParams p;
  CUtensorMap tk, tv;
  bool k8, v8;
  if ((st = fill_attn(a, &p, &k8, &v8, block)) != FMHA_OK) return st;
  PickPlan t;
  if (!pick_plan(a, top, block, &t)) return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
  if ((st = check_workspace(workspace, workspace_bytes, t.workspace_bytes)) != FMHA_OK) return st;
  if ((st = bind_attn(a, &p, k8, v8, &tk, &tv)) != FMHA_OK) return st;
  p.blocks = blocks;
  p.top = top;
  p.block_shift = log2_of(block);
  p.n_blocks = ceil_div(p.c.capacity, block);
  p.row_tiles = t.row_tiles;
  p.tile_rows = t.rows;
  p.n_ctas = t.n_ctas;
  p.item_tiles = t.item_tiles;
  p.n_splits = t.n_splits;
  p.per_split = t.per_split;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + size_t(2) * t.n_ctas * t.rows * a->D;
  cudaError_t e = launch_cache_attn(a->D, k8, v8, p, tk, tv, stream);
  if (e == cudaSuccess && t.n_splits > 1) e = launch_cache_merge(a->D, p, stream);
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "picked-block attention launch: %s", cudaGetErrorString(e));
  return ok_status();
}

fmha_status fmha_key_bounds(const fmha_cache_args* a, void* bounds, int32_t n_blocks, int32_t block,
                            const int32_t* start, cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (!sizes_ok(a) || n_blocks < 0) return fail(FMHA_ERR_INVALID_ARG, "negative size");
  if (a->B == 0 || a->Hkv == 0 || n_blocks == 0) return ok_status();
  fmha_status st;
  if ((st = check_block(block)) != FMHA_OK) return st;
  if (bounds == nullptr || !aligned16(bounds)) return fail(FMHA_ERR_INVALID_ARG, "bounds is NULL or not 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(start) & 3u) return fail(FMHA_ERR_INVALID_ARG, "start misaligned");
  KeyBoundsParams p;
  memset(&p, 0, sizeof(p));
  bool k8, v8;
  if ((st = check_cache(a, false, false, &p.c, &k8, &v8)) != FMHA_OK) return st;
  if (static_cast<int64_t>(a->B) * a->Hkv * n_blocks >= (int64_t(1) << 32))
    return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
  if ((st = bind_device(&p.c)) != FMHA_OK) return st;
  p.k = static_cast<const uint8_t*>(a->k.ptr);
  p.k_sb = a->k.stride_b; p.k_ss = a->k.stride_s; p.k_sh = a->k.stride_h;
  p.bounds = static_cast<uint16_t*>(bounds);
  p.start = start;
  p.n_blocks = n_blocks;
  p.block_shift = log2_of(block);
  cudaError_t e = launch_key_bounds(a->D, k8, p, stream);
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "key bounds launch: %s", cudaGetErrorString(e));
  return ok_status();
}

fmha_status fmha_select_blocks(const fmha_cache_args* a, const void* bounds, int32_t n_blocks, int32_t block,
                               int32_t top, int32_t sink_blocks, int32_t recent_blocks, int32_t q_tile, void* picked,
                               cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (!sizes_ok(a) || n_blocks < 0) return fail(FMHA_ERR_INVALID_ARG, "negative size");
  // Without query heads the scores are empty sums, and the ties' rule picks.
  if (a->B == 0 || a->T == 0 || (a->Hq == 0 && a->Hkv == 0)) return ok_status();
  fmha_status st;
  if ((st = check_block(block)) != FMHA_OK) return st;
  if (top <= 0) return fail(FMHA_ERR_INVALID_ARG, "top must be positive");
  if (sink_blocks < 0 || recent_blocks < 0) return fail(FMHA_ERR_INVALID_ARG, "negative sink_blocks or recent_blocks");
  if (q_tile != 1 && q_tile != 128) return fail(FMHA_ERR_UNSUPPORTED, "q_tile %d (supported: 1, 128)", q_tile);
  if (q_tile == 128 && block != 128) return fail(FMHA_ERR_UNSUPPORTED, "q_tile 128 needs blocks of 128 keys");
  if (n_blocks > kMaxPickBlocks) return fail(FMHA_ERR_UNSUPPORTED, "%d blocks (supported: up to %d)", n_blocks, kMaxPickBlocks);
  if (a->D != 64 && a->D != 128) return fail(FMHA_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", a->D);
  if (a->Hkv == 0 || a->Hq % a->Hkv != 0)
    return fail(FMHA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", a->Hq, a->Hkv);
  if (a->q.dtype != FMHA_BF16) return fail(FMHA_ERR_UNSUPPORTED, "q must be BF16");
  if (a->Hq > 0 && (st = check_tensor(a->q, "q", a->B, a->T, a->Hq, a->D)) != FMHA_OK) return st;
  if (n_blocks > 0 && (bounds == nullptr || !aligned16(bounds)))
    return fail(FMHA_ERR_INVALID_ARG, "bounds is NULL or not 16-byte aligned");
  if (q_tile == 128 && n_blocks == 0) return ok_status();  // an empty mask
  if (picked == nullptr || (q_tile == 1 && (reinterpret_cast<uintptr_t>(picked) & 3u)))
    return fail(FMHA_ERR_INVALID_ARG, "picked is NULL or misaligned");
  if (a->lens == nullptr || (reinterpret_cast<uintptr_t>(a->lens) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "lens is NULL or misaligned");
  if (reinterpret_cast<uintptr_t>(a->q_lens) & 3u) return fail(FMHA_ERR_INVALID_ARG, "q_lens misaligned");
  const int G = a->Hq / a->Hkv;
  const int n_tiles = ceil_div(a->T, q_tile);
  const int64_t items = static_cast<int64_t>(a->B) * n_tiles * a->Hkv;
  if (items >= (int64_t(1) << 27) || static_cast<int64_t>(a->T) * G > INT32_MAX / 2)
    return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
  SelectParams p;
  memset(&p, 0, sizeof(p));
  p.c.B = a->B; p.c.T = a->T; p.c.Hq = a->Hq; p.c.Hkv = a->Hkv; p.c.G = G;
  p.c.capacity = n_blocks * block;
  p.c.lens = a->lens;
  p.c.q_lens = a->q_lens;
  if ((st = bind_device(&p.c)) != FMHA_OK) return st;
  p.q = static_cast<const uint16_t*>(a->q.ptr);
  p.q_sb = a->q.stride_b; p.q_ss = a->q.stride_s; p.q_sh = a->q.stride_h;
  p.bounds = static_cast<const uint16_t*>(bounds);
  p.n_blocks = n_blocks;
  p.block_shift = log2_of(block);
  p.top = top; p.sinks = sink_blocks; p.recent = recent_blocks;
  p.q_tile = q_tile;
  p.n_tiles = n_tiles;
  p.cluster = pick_cluster(items, n_blocks);
  if (q_tile == 1) p.list = static_cast<int32_t*>(picked);
  else p.mask = static_cast<uint8_t*>(picked);
  cudaError_t e = launch_select_blocks(a->D, p, stream);
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "block selection launch: %s", cudaGetErrorString(e));
  return ok_status();
}

size_t fmha_key_weights_workspace_bytes(const fmha_cache_args* a, int32_t n_weights, int32_t causal) {
  if (!rows_ok(a) || n_weights <= 0 || capacity_of(a) <= 0 || capacity_of(a) > INT32_MAX / 2 || a->T < kManyQueries) return 0;
  const WeightRuns r = weight_runs(a, static_cast<int>(capacity_of(a)), n_weights, causal);
  return weight_bytes(a, r, n_weights);
}

fmha_status fmha_key_weights(const fmha_cache_args* a, float* weights, int32_t n_weights, int32_t causal,
                             int32_t accumulate, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (!sizes_ok(a) || n_weights < 0) return fail(FMHA_ERR_INVALID_ARG, "negative size");
  const bool no_rows = a->T == 0 || a->Hq == 0;  // every sum is empty
  if (a->B == 0 || n_weights == 0 || (no_rows && (accumulate != 0 || a->Hkv == 0))) return ok_status();
  if (weights == nullptr || (reinterpret_cast<uintptr_t>(weights) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "weights is NULL or misaligned");
  if (a->lse == nullptr && !no_rows) return fail(FMHA_ERR_INVALID_ARG, "lse is NULL");
  KeyWeightsParams p;
  memset(&p, 0, sizeof(p));
  bool k8, v8;
  fmha_status st;
  if ((st = check_cache(a, !no_rows, false, &p.c, &k8, &v8)) != FMHA_OK) return st;
  if (p.c.capacity == 0) return ok_status();  // no key
  if (no_rows) {
    if ((st = bind_device(&p.c)) != FMHA_OK) return st;
    p.weights = weights;
    p.n_weights = n_weights;
    const cudaError_t e = launch_key_weights_clear(p, stream);
    if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "key weights launch: %s", cudaGetErrorString(e));
    return ok_status();
  }
  p.q = static_cast<const uint16_t*>(a->q.ptr);
  p.q_sb = a->q.stride_b; p.q_ss = a->q.stride_s; p.q_sh = a->q.stride_h;
  p.k = static_cast<const uint8_t*>(a->k.ptr);
  p.k_sb = a->k.stride_b; p.k_ss = a->k.stride_s; p.k_sh = a->k.stride_h;
  p.lse = a->lse;
  p.weights = weights;
  p.n_weights = n_weights;
  p.causal = causal != 0;
  p.accumulate = accumulate != 0;
  const float scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.0f / std::sqrt(float(a->D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.sf_k = a->sf_k.ptr; p.sf_k_kind = a->sf_k.kind;
  const int64_t heads = static_cast<int64_t>(a->B) * a->Hkv;
  cudaError_t e;
  CUtensorMap m;
  if (a->T >= kManyQueries) {
    const WeightRuns r = weight_runs(a, p.c.capacity, n_weights, causal);
    const int64_t n = heads * ceil_div(std::min(p.c.capacity, n_weights), 128) * r.parts;
    if (n >= (int64_t(1) << 31) || heads > 65535) return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
    if ((st = check_workspace(workspace, workspace_bytes, weight_bytes(a, r, n_weights))) != FMHA_OK) return st;
    if ((st = bind_device(&p.c)) != FMHA_OK) return st;
    p.n_ctas = static_cast<int>(std::min<int64_t>(n, 2 * sm_count()));
    p.n_items = static_cast<uint32_t>(n);
    p.chunk = r.chunk;
    p.parts = r.parts;
    p.ticket = static_cast<uint32_t*>(workspace);
    p.part_w = static_cast<float*>(workspace) + 4;
    const uint64_t dims[4] = {uint64_t(a->D), uint64_t(a->Hq), uint64_t(a->T), uint64_t(a->B)};
    const int64_t strides[3] = {a->q.stride_h, a->q.stride_s, a->q.stride_b};
    const uint32_t box[4] = {64, 1, 128, 1};
    if ((st = make_map_n<4>(&m, a->q.ptr, 2, dims, strides, box, "q")) != FMHA_OK) return st;
    e = launch_key_weights_many(a->D, k8, p, m, stream);
  } else {
    const int piece = p.c.page_table != nullptr ? std::min(kTile, a->page_size) : kTile;
    if ((st = bind_device(&p.c)) != FMHA_OK) return st;
    if ((st = cache_map(&m, a, p.c, a->k, k8, piece, "k")) != FMHA_OK) return st;
    p.piece_shift = log2_of(piece);
    p.row_tiles = 1;
    p.min_tiles = 1;
    if (heads >= (int64_t(1) << 30)) return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
    p.groups = list_groups(a->Hkv, 3 * sm_count(), static_cast<int64_t>(a->B) * ceil_div(p.c.capacity, kTile));
    p.n_ctas = a->Hkv * p.groups;
    if (static_cast<int64_t>(a->B) * ceil_div(p.c.capacity, kTile) / p.groups >= (int64_t(1) << 30) ||
        static_cast<int64_t>(a->Hkv) * p.groups >= (int64_t(1) << 30))
      return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
    e = launch_key_weights_few(a->D, k8, p, m, stream);
  }
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "key weights launch: %s", cudaGetErrorString(e));
  return ok_status();
}

fmha_status fmha_evict_select(const fmha_cache_args* a, const float* weights, int32_t n_weights, int32_t budget,
                              int32_t sinks, int32_t recent, int32_t* keep, int32_t* counts, cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (a->B < 0 || a->Hkv < 0 || n_weights < 0 || a->capacity < 0) return fail(FMHA_ERR_INVALID_ARG, "negative size");
  if (budget < 1 || sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > budget)
    return fail(FMHA_ERR_INVALID_ARG, "budget %d must be positive and hold sinks %d + recent %d", budget, sinks, recent);
  if (a->B == 0 || a->Hkv == 0) return ok_status();
  if (a->lens == nullptr || (reinterpret_cast<uintptr_t>(a->lens) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "lens is NULL or misaligned");
  if (n_weights > 0 && (weights == nullptr || (reinterpret_cast<uintptr_t>(weights) & 3u)))
    return fail(FMHA_ERR_INVALID_ARG, "weights is NULL or misaligned");
  if (keep == nullptr || counts == nullptr || ((reinterpret_cast<uintptr_t>(keep) | reinterpret_cast<uintptr_t>(counts)) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "keep or counts is NULL or misaligned");
  if (static_cast<int64_t>(a->B) * a->Hkv >= (int64_t(1) << 28)) return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
  if (n_weights > INT32_MAX / 2 || budget > INT32_MAX / 2)
    return fail(FMHA_ERR_UNSUPPORTED, "more than 2^30 tokens per sequence");
  EvictParams p;
  memset(&p, 0, sizeof(p));
  p.c.B = a->B; p.c.Hkv = a->Hkv;
  p.c.capacity = a->capacity > 0 ? a->capacity : n_weights;
  p.c.lens = a->lens;
  fmha_status st;
  if ((st = bind_device(&p.c)) != FMHA_OK) return st;
  p.weights = weights;
  p.n_weights = n_weights;
  p.budget = budget; p.sinks = sinks; p.recent = recent;
  p.keep = keep;
  p.counts = counts;
  cudaError_t e = launch_evict_select(p, stream);
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "eviction launch: %s", cudaGetErrorString(e));
  return ok_status();
}

fmha_status fmha_cache_compact(const fmha_cache_args* a, const fmha_cache_args* out, const int32_t* keep,
                               int64_t keep_stride_b, int64_t keep_stride_h, int32_t n_keep, const int32_t* counts,
                               const int32_t* dst_start, const float* weights, int32_t n_weights, float* weights_out,
                               int32_t n_weights_out, cudaStream_t stream) {
  if (a == nullptr) return fail(FMHA_ERR_INVALID_ARG, "args is NULL");
  if (!sizes_ok(a) || n_keep < 0 || n_weights < 0 || n_weights_out < 0 || keep_stride_b < 0 || keep_stride_h < 0)
    return fail(FMHA_ERR_INVALID_ARG, "negative size or stride");
  if (a->B == 0 || a->Hkv == 0) return ok_status();
  if (out != nullptr && (out->B != a->B || out->Hkv != a->Hkv || out->D != a->D))
    return fail(FMHA_ERR_INVALID_ARG, "the caches differ in B, Hkv or D");
  if (n_keep > 0 && (keep == nullptr || (reinterpret_cast<uintptr_t>(keep) & 3u)))
    return fail(FMHA_ERR_INVALID_ARG, "keep is NULL or misaligned");
  if (counts == nullptr || ((reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(dst_start)) & 3u))
    return fail(FMHA_ERR_INVALID_ARG, "counts is NULL, or counts or dst_start misaligned");
  if ((weights == nullptr) != (weights_out == nullptr))
    return fail(FMHA_ERR_INVALID_ARG, "weights and weights_out go together");
  if (weights != nullptr && (out == nullptr) != (weights == weights_out))
    return fail(FMHA_ERR_INVALID_ARG, "weights_out is weights exactly when the rows move inside one cache");
  if (weights != nullptr && out == nullptr && n_weights != n_weights_out)
    return fail(FMHA_ERR_INVALID_ARG, "n_weights and n_weights_out differ");
  if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(weights_out)) & 3u)
    return fail(FMHA_ERR_INVALID_ARG, "weights misaligned");
  if (n_keep > INT32_MAX / 2 || n_weights_out > INT32_MAX / 2)
    return fail(FMHA_ERR_UNSUPPORTED, "more than 2^30 tokens per sequence");
  // The caches' own checks want lens; these calls have none.
  CompactParams p;
  memset(&p, 0, sizeof(p));
  CacheView co;
  bool k8, v8, ok8, ov8;
  fmha_status st;
  fmha_cache_args x = *a;
  memset(&x.sf_k, 0, sizeof(x.sf_k));
  memset(&x.sf_v, 0, sizeof(x.sf_v));
  x.lens = counts;
  x.q_lens = nullptr;
  x.lse = nullptr;
  if ((st = check_cache(&x, false, true, &p.c, &k8, &v8)) != FMHA_OK) return st;
  const fmha_cache_args* o = a;
  co = p.c;
  if (out != nullptr) {
    o = out;
    fmha_cache_args y = *out;
    memset(&y.sf_k, 0, sizeof(y.sf_k));
    memset(&y.sf_v, 0, sizeof(y.sf_v));
    y.lens = counts;
    y.q_lens = nullptr;
    y.lse = nullptr;
    if ((st = check_cache(&y, false, true, &co, &ok8, &ov8)) != FMHA_OK) return st;
    if (ok8 != k8 || ov8 != v8) return fail(FMHA_ERR_INVALID_ARG, "the caches differ in dtype");
  }
  const int64_t heads = static_cast<int64_t>(a->B) * a->Hkv;
  if (heads > INT32_MAX || heads * (ceil_div(std::max(n_keep, n_weights_out), 8) + 1) >= (int64_t(1) << 33))
    return fail(FMHA_ERR_UNSUPPORTED, "grid too large");
  if ((st = bind_device(&p.c)) != FMHA_OK) return st;
  const int ek = k8 ? 1 : 2, ev = v8 ? 1 : 2;
  p.k = static_cast<const uint8_t*>(a->k.ptr); p.v = static_cast<const uint8_t*>(a->v.ptr);
  p.k_sb = a->k.stride_b * ek; p.k_ss = a->k.stride_s * ek; p.k_sh = a->k.stride_h * ek;
  p.v_sb = a->v.stride_b * ev; p.v_ss = a->v.stride_s * ev; p.v_sh = a->v.stride_h * ev;
  p.k_out = static_cast<uint8_t*>(o->k.ptr); p.v_out = static_cast<uint8_t*>(o->v.ptr);
  p.ko_sb = o->k.stride_b * ek; p.ko_ss = o->k.stride_s * ek; p.ko_sh = o->k.stride_h * ek;
  p.vo_sb = o->v.stride_b * ev; p.vo_ss = o->v.stride_s * ev; p.vo_sh = o->v.stride_h * ev;
  p.out_table = co.page_table; p.out_pages = co.num_pages; p.out_page_shift = co.page_shift;
  p.out_max_pages = co.max_pages; p.out_capacity = co.capacity;
  p.keep = keep; p.keep_sb = keep_stride_b; p.keep_sh = keep_stride_h; p.n_keep = n_keep;
  p.counts = counts;
  p.dst_start = dst_start;
  p.weights = weights; p.weights_out = weights_out;
  p.n_weights = n_weights; p.n_weights_out = n_weights_out;
  p.k_bytes = a->D * ek;
  p.v_bytes = a->D * ev;
  p.in_place = out == nullptr ? 1 : 0;
  cudaError_t e = launch_compact(p, stream);
  if (e != cudaSuccess) return fail(FMHA_ERR_CUDA, "compaction launch: %s", cudaGetErrorString(e));
  return ok_status();
}

}  // extern "C"
