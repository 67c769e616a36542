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
  long long wait_clocks;           // limit of every bounded device wait
  int stall;                       // test hook: the first load is withheld
  int sms;                         // processors of the device
  // forward
  da2_tensor out;
  float* lse;                      // null: not wanted
  int q_pairs, splits;             // 256-row query tiles per head; parts of the keys
  float *part_o, *part_lse;        // fp32 [splits][B*H*Tq][d], [splits][B*H*Tq] (log2 domain)
  // backward
  da2_tensor v, dout, dq, dk, dv;
  const float* lse_in;
  int q_tiles, k_tiles;            // 128-row tiles
  float *lse2, *delta;             // fp32 [B*H][128 q_tiles]: lse in the log2 domain, D
  float* part_kv;                  // fp32 [2 sms][2][d][128]: dK and dV of split sums
  int32_t* first;                  // [B + 1]: key tiles with a valid key in front of each batch entry
  float *dnorm2, *vnorm2;          // fp16: [B*H][q_tiles][4] and [B*Hkv][k_tiles], largest squared row norms
};

// Boxes of 64 channels and 128 rows (k and v of the forward pass: 64 rows).
struct CrossMaps {
  CUtensorMap q, k, v, dout, out, dq;
};

cudaError_t launch_cross_forward(const CrossArgs& g, const CrossMaps& m, bool bf16, cudaStream_t st);
cudaError_t launch_cross_backward(const CrossArgs& g, const CrossMaps& m, bool bf16, cudaStream_t st);

// ---------------------------------------------------------------- device helpers

// A kernel's bounded waits: a wait that runs out sets the error word and the block's abort flag. From
// then on a wait of the block that is not over at once ends after one suspended try (a call of 40 heads
// x 131072 queries x 4096 keys took 14 ms beyond its limits backward, 70 when every wait tried twice; a
// flag in each thread that skips the try took 5 % of the forward pass's time). Copies in flight are
// still waited for, up to the limit once more. A short inline part (one try), because the code of all of
// a kernel's waits competes with its loops for the instruction cache.
struct Guard {
  uint32_t* err;
  volatile uint32_t* abort;        // shared memory, starts at zero
  long long limit;                 // clock cycles
};
constexpr uint32_t kWaitNs = 20000;    // suspension per try
static __device__ __noinline__ bool guard_wait_slow(uint64_t* bar, uint32_t parity, uint32_t* err,
                                                    volatile uint32_t* abort, long long limit, bool honour_abort) {
  const long long t0 = clock64();
  while (!(honour_abort && *abort) && !tc::mbar_try_wait_for(bar, parity, kWaitNs)) {
    if (clock64() - t0 > limit) {
      set_error(err, kErrWaitTimeout);
      *abort = 1u;
      return false;
    }
  }
  return !(honour_abort && *abort);
}
__device__ __forceinline__ bool guard_wait(uint64_t* bar, uint32_t parity, const Guard& gd,
                                           bool honour_abort = true) {
  if (tc::mbar_try_wait_for(bar, parity, kWaitNs)) return true;
  return guard_wait_slow(bar, parity, gd.err, gd.abort, gd.limit, honour_abort);
}
// For a warp that stops when the wait fails: all lanes get the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Guard& gd) {
  return __all_sync(0xffffffffu, guard_wait(bar, parity, gd));
}
// All lanes' tensor-memory accesses before, one arrival per warp after.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  tc::fence_before_sync();
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
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

// One tile of 128 rows and D channels as 64-channel boxes behind each other (128-byte swizzle). Rows
// past the tensor's end are filled with zeros.
template <int D, int Rows = 128>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int row, int head, int b,
                                          uint64_t* bar) {
#pragma unroll
  for (int x = 0; x < D / 64; ++x) tc::tma_load_4d(dst + x * Rows * 128, map, 64 * x, row, head, b, bar);
}

// Zeroes rows [r0, r1) of such a tile in shared memory (whole rows, so the swizzle does not matter)
// for the tensor cores to read. Called by a full warp.
template <int D, int Rows = 128>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1, int lane) {
  for (int i = lane; i < (r1 - r0) * 8 * (D / 64); i += 32) {
    const int x = i / ((r1 - r0) * 8), o = i - x * (r1 - r0) * 8;
    *reinterpret_cast<uint4*>(tile + x * Rows * 128 + r0 * 128 + o * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace da2
