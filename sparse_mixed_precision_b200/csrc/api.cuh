// Host helpers shared by the C entry points.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/da2.h"

namespace da2 {

// DA2_OK, or DA2_ERR_CUDA with the code kept for da2_last_cuda_error.
da2_status cuda_status(cudaError_t e);

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Longest token axis of the operators around the self-attention: lengths are rounded up to whole tiles
// (of 256 at most) in 32 bits.
constexpr int kMaxTokens = 0x7fffffff - 255;

// An NVTX range around one library call (visible in a profiler's timeline; no cost without
// an attached tool).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// One strided activation: its axes' lengths come from the call's configuration. On success
// *out holds the tensor with the strides of axes of length one set to zero (never read).
inline da2_status check_tensor(const da2_tensor* t, long B, long H, long T, int d, da2_tensor* out) {
  if (!t || !t->data) return DA2_ERR_INVALID_ARG;
  *out = *t;
  if (B == 1) out->sb = 0;
  if (H == 1) out->sh = 0;
  if (T == 1) out->st = 0;
  if ((B > 1 && t->sb < d) || (H > 1 && t->sh < d) || (T > 1 && t->st < d)) return DA2_ERR_INVALID_ARG;
  constexpr int64_t kMaxStride = int64_t(1) << 38;   // elements: byte strides stay below 2^40
  if (out->sb >= kMaxStride || out->sh >= kMaxStride || out->st >= kMaxStride) return DA2_ERR_INVALID_ARG;
  if (!aligned16(t->data) || (out->sb & 7) || (out->sh & 7) || (out->st & 7)) return DA2_ERR_ALIGNMENT;
  return DA2_OK;
}

}  // namespace da2
