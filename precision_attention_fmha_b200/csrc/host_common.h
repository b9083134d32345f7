// host_common.h -- host-side helpers shared by the entry points (api.cu,
// api_cache.cu): error messages, operand checks, TMA descriptors. Defined in
// api.cu except where inline.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fmha_internal.h"

namespace fmha {
namespace host {

// Records a one-line reason (thread-local) and returns s.
fmha_status fail(fmha_status s, const char* fmt, ...);
// Clears the reason and returns FMHA_OK.
fmha_status ok_status();

// Device error word of the current device (nullptr and *err set on failure).
uint32_t* device_error_word(cudaError_t* err);
// Bound on one device-side wait for launches made now.
uint64_t wait_cycles();
int sm_count();

int elem_bytes(int dt);
// Checks a [B, S, H, D] operand: pointer, alignment, strides. Size-1 dims' strides are free.
fmha_status check_tensor(const fmha_tensor& t, const char* name, int B, int S, int H, int D);
fmha_status check_sf(const fmha_sf& sf, const char* name, bool allow_head, bool allow_tensor, bool allow_block,
                     int block_multiple, bool allow_channel);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn(cudaError_t* err);

// RANK-d map (dims innermost first, RANK = 4 or 5) with 128-byte swizzle.
// Strides in elements for dims 1..RANK-1. Size-1 dims get a packed stride so
// the descriptor stays valid whatever the caller's stride.
template <int RANK>
fmha_status make_map_n(CUtensorMap* map, void* base, int elem_bytes, const uint64_t (&dims)[RANK],
                       const int64_t (&strides_elems)[RANK - 1], const uint32_t (&box)[RANK], const char* what,
                       CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B,
                       CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  cudaError_t e;
  EncodeTiledFn fn = encode_fn(&e);
  if (fn == nullptr) return fail(FMHA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable: %s", cudaGetErrorString(e));
  cuuint64_t gdim[RANK];
  cuuint64_t gstride[RANK - 1];
  cuuint32_t ebox[RANK];
  cuuint32_t bdim[RANK];
  uint64_t packed = dims[0] * elem_bytes;
  for (int i = 0; i < RANK; ++i) {
    gdim[i] = dims[i];
    bdim[i] = box[i];
    ebox[i] = 1;
  }
  for (int i = 0; i < RANK - 1; ++i) {
    uint64_t s = static_cast<uint64_t>(strides_elems[i]) * elem_bytes;
    if (dims[i + 1] == 1) s = (packed + 15) / 16 * 16;
    gstride[i] = s;
    packed = s * dims[i + 1];
  }
  const CUtensorMapDataType dt = elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUresult r = fn(map, dt, RANK, base, gdim, gstride, bdim, ebox, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FMHA_ERR_INVALID_ARG, "TMA descriptor for %s rejected (CUresult %d)", what, (int)r);
  return FMHA_OK;
}

}  // namespace host
}  // namespace fmha
