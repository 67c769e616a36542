// Shared by the forward and backward kernels of the attention to an encoder's states: their
// arguments, the bounded waits of their pipelines, and tensor maps of strided activations.
#pragma once
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "tc.cuh"

namespace da2 {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One call, resolved on the host.
struct CrossArgs {
  int B, H, Hkv, group;            // group = H / Hkv query heads share a key/value head
  int Tq, Tk, d;
  float scale, scale_log2;         // softmax scale, and times log2(e)
  const int32_t* kv_len;           // null: Tk
  uint32_t* err;
  unsigned long long wait_ns;
  int stall;                       // test hook: the first load is withheld
  int sms;                         // processors of the device
  // forward
  da2_tensor out;
  float* lse;                      // null: not wanted
  int q_pairs, splits;             // 256-row query tiles per head; parts of the keys
  float *part_o, *part_lse;        // fp32 [splits][B*H*Tq][d], [splits][B*H*Tq] (log2 domain)
  // backward
  da2_tensor dout, dq, dk, dv;
  const float* lse_in;
  int q_tiles, k_tiles;            // 128-row tiles
  float *lse2, *delta;             // fp32 [B*H][128 q_tiles]: lse in the log2 domain, D
  float* part_kv;                  // fp32 [2 sms][2][d][128]: dK and dV of split sums
};

struct CrossMaps {
  CUtensorMap q, k, v, dout;
};

cudaError_t launch_cross_forward(const CrossArgs& g, const CrossMaps& m, bool bf16, cudaStream_t st);
cudaError_t launch_cross_backward(const CrossArgs& g, const CrossMaps& m, bool bf16, cudaStream_t st);

// ---------------------------------------------------------------- device helpers

// A kernel's bounded waits: a wait that runs out sets the error word and the block's abort flag;
// from then on every wait of the block returns false at once.
struct Guard {
  uint32_t* err;
  volatile uint32_t* abort;        // shared memory, starts at zero
  unsigned long long limit_ns;
};
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
static __device__ __noinline__ bool guard_wait_slow(uint64_t* bar, uint32_t parity, const Guard& gd, bool honour_abort) {
  const uint64_t t0 = global_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)
      if (tc::mbar_try_wait(bar, parity)) return true;
    if (honour_abort && *gd.abort) return false;
    if (global_ns() - t0 > gd.limit_ns) {
      set_error(gd.err, kErrWaitTimeout);
      *gd.abort = 1u;
      return false;
    }
  }
}
__device__ __forceinline__ bool guard_wait(uint64_t* bar, uint32_t parity, const Guard& gd,
                                           bool honour_abort = true) {
  if (tc::mbar_test_wait(bar, parity)) return true;
  return guard_wait_slow(bar, parity, gd, honour_abort);
}

__device__ __forceinline__ int valid_keys(const CrossArgs& g, int b) {
  if (!g.kv_len) return g.Tk;
  const int n = __ldg(g.kv_len + b);
  return n < 0 ? 0 : (n > g.Tk ? g.Tk : n);
}

// Two fp32 values rounded to the element type, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// One 128-row tile of D channels as 64-channel boxes behind each other (128-byte swizzle). Rows
// past the tensor's end are filled with zeros.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int row, int head, int b,
                                          uint64_t* bar) {
#pragma unroll
  for (int x = 0; x < D / 64; ++x) tc::tma_load_4d(dst + x * 16384, map, 64 * x, row, head, b, bar);
}

// Zeroes rows [r0, r1) of a tile in shared memory (whole rows, so the swizzle does not matter) for
// the tensor cores to read. Called by a full warp.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1, int lane) {
  for (int i = lane; i < (r1 - r0) * 8 * (D / 64); i += 32) {
    const int x = i / ((r1 - r0) * 8), o = i - x * (r1 - r0) * 8;
    *reinterpret_cast<uint4*>(tile + x * 16384 + r0 * 128 + o * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace da2
