// RMS norm of every head of the queries and keys and the position rotation, in one pass, and
// its backward pass.
//
//   n = x / sqrt(mean(x^2) + eps),  y = n w,  (y_a, y_b) <- (y_a c - y_b s, y_a s + y_b c)
//   backward, with g the gradient rotated back by (c, -s):
//   dw = sum_rows g n,  dx = (g w - n mean(g w n)) / sqrt(mean(x^2) + eps)
//
// Memory-bound: a row is read and written once (forward) or two rows read and one written
// (backward). The tables are fp32, so that one row of cos and sin weighs as much as one row in
// and out together; each thread therefore keeps its 8 pairs' cos and sin in registers and
// walks over the heads of its token. A thread owns two 16-byte chunks of the row, d/2 apart, so
// that both members of a pair are its own in either pairing; d/16 threads share a row.
// Measured in a sequence of calls (40 heads, d = 128, bf16; copy bandwidth 6552 GB/s): forward, 32760 tokens
// token-major 240 us = 5650 GB/s, 75600 tokens head-major 535 us = 5850 GB/s; backward, 32760 tokens 409
// us = 4970 GB/s. The backward pass waits for memory: 122 registers leave two blocks per processor (24 % of
// the warps), each thread has the two rows of one head in flight, and 4.6 of 5.6 stalled cycles per
// instruction are on loads; its arithmetic would take about 150 us.
#include <cmath>

#include <cuda_fp16.h>

#include "api.cuh"
#include "common.cuh"

namespace da2 {
namespace {

constexpr int kThreads = 256;
constexpr int kNormBackBlocks = 592;   // blocks per side of the backward pass: 4 per processor

// The queries or the keys of one call.
struct NormSide {
  da2_tensor x, y, dy;   // input, output (dx in the backward pass), gradient of the output
  const float* w;
  float *dw, *part;      // weight gradient and its partial rows (null: not wanted)
  int H, chunks;         // heads and head chunks
  int blocks;            // blocks of the backward pass
  long items;            // batch entries x token blocks x head chunks
};

struct NormRopeArgs {
  NormSide side[2];
  const float *cos_t, *sin_t;
  int64_t tab_sb;        // table elements between batch entries (0: shared)
  int B, T, T_rot, d, token_blocks, head_chunk;
  float eps;
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A thread's 16 elements of a row: [8c, 8c + 8) and [d/2 + 8c, d/2 + 8c + 8).
struct Raw {
  uint4 a, b;
};
template <typename T, int D>
__device__ __forceinline__ Raw load_row(const T* row, int c) {
  Raw r;
  r.a = __ldcs(reinterpret_cast<const uint4*>(row + 8 * c));
  r.b = __ldcs(reinterpret_cast<const uint4*>(row + D / 2 + 8 * c));
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack_row(const Raw& r, float* x) {
  const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack2<T>(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T, int D>
__device__ __forceinline__ void store_row(T* row, int c, const float* x) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  __stcs(reinterpret_cast<uint4*>(row + 8 * c), make_uint4(u[0], u[1], u[2], u[3]));
  __stcs(reinterpret_cast<uint4*>(row + D / 2 + 8 * c), make_uint4(u[4], u[5], u[6], u[7]));
}
// A thread's 16 weights, laid out like its elements (16-byte aligned: a branch for other addresses took
// 5 % of the forward pass's time).
template <int D>
__device__ __forceinline__ void load_weight(const float* w, int c, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = (i & 1) * 4 + (i >> 1) * (D / 2) + 8 * c;
    const float4 v = w ? __ldg(reinterpret_cast<const float4*>(w + at)) : make_float4(1.f, 1.f, 1.f, 1.f);
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
// The 8 table entries of a thread's pairs: pairs (2i, 2i+1) lie inside its two chunks, pairs
// (i, i + d/2) across them.
template <int D, bool HALVES>
__device__ __forceinline__ void load_table(const float* row, int c, float* x) {
  const int a0 = HALVES ? 8 * c : 4 * c, a1 = HALVES ? 8 * c + 4 : D / 4 + 4 * c;
  const float4 u = __ldg(reinterpret_cast<const float4*>(row + a0));
  const float4 v = __ldg(reinterpret_cast<const float4*>(row + a1));
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}
// sgn = 1 rotates, -1 rotates back.
template <bool HALVES>
__device__ __forceinline__ void rotate(float* x, const float* cs, const float* sn, float sgn) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int ia = HALVES ? j : 2 * j, ib = HALVES ? 8 + j : 2 * j + 1;
    const float a = x[ia], b = x[ib], s = sgn * sn[j];
    x[ia] = a * cs[j] - b * s;
    x[ib] = a * s + b * cs[j];
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a block works: one batch entry, kThreads / (D/16) tokens and a chunk of the heads of
// one side (queries or keys).
template <int D>
struct Place {
  int b, t, h0, h1, c;
  bool on;
  __device__ __forceinline__ Place(const NormRopeArgs& g, const NormSide& s, long item) {
    constexpr int G = D / 16, kTok = kThreads / G;
    const long per_b = (long)g.token_blocks * s.chunks;
    b = (int)(item / per_b);
    const long rem = item - b * per_b;
    const int tb = (int)(rem / s.chunks), ch = (int)(rem - (long)tb * s.chunks);
    c = threadIdx.x % G;
    t = tb * kTok + threadIdx.x / G;
    on = t < g.T;
    if (!on) t = g.T - 1;                // reads a valid row, writes nothing
    h0 = ch * g.head_chunk;
    h1 = min(s.H, h0 + g.head_chunk);
  }
};

template <int D, bool HALVES>
__device__ __forceinline__ void token_table(const NormRopeArgs& g, const Place<D>& p, float* cs, float* sn) {
  if (p.t < g.T_rot) {
    const int64_t at = p.b * g.tab_sb + (int64_t)p.t * (D / 2);
    load_table<D, HALVES>(g.cos_t + at, p.c, cs);
    load_table<D, HALVES>(g.sin_t + at, p.c, sn);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = 1.0f, sn[j] = 0.0f;
  }
}

// kUnroll heads' loads are in flight at once per thread.
constexpr int kUnroll = 4;

template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads) k_norm_rope(NormRopeArgs g) {
  constexpr int G = D / 16;
  const bool is_k = (long)blockIdx.x >= g.side[0].items;
  const NormSide& s = g.side[is_k];
  const Place<D> p(g, s, (long)blockIdx.x - (is_k ? g.side[0].items : 0));
  float cs[8], sn[8], w[16];
  token_table<D, HALVES>(g, p, cs, sn);
  load_weight<D>(s.w, p.c, w);
  const T* in = static_cast<const T*>(s.x.data) + p.b * s.x.sb + p.t * s.x.st;
  T* out = static_cast<T*>(s.y.data) + p.b * s.y.sb + p.t * s.y.st;
  for (int h = p.h0; h < p.h1; h += kUnroll) {
    Raw raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < p.h1) raw[u] = load_row<T, D>(in + (h + u) * s.x.sh, p.c);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= p.h1) break;
      float x[16], ss = 0.0f;
      unpack_row<T>(raw[u], x);
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      const float r = rsqrtf(group_sum<G>(ss) * (1.0f / D) + g.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
      rotate<HALVES>(x, cs, sn, 1.0f);
      if (p.on) store_row<T, D>(out + (h + u) * s.y.sh, p.c, x);
    }
  }
}

// The backward pass walks a fixed number of blocks per side over the items, so that each block
// sums its rows' share of dw in registers and writes one partial row. One head at a time: with two
// in flight, whose registers leave one block per processor, the 480p layer took 532 us where it took 419,
// with four 439.
template <typename T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads) k_norm_rope_back(NormRopeArgs g) {
  constexpr int G = D / 16;
  __shared__ float red[kThreads / 32][D];
  const bool is_k = (int)blockIdx.x >= g.side[0].blocks;
  const NormSide& s = g.side[is_k];
  const int block = (int)blockIdx.x - (is_k ? g.side[0].blocks : 0);
  float w[16], dw[16];
  load_weight<D>(s.w, threadIdx.x % G, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.0f;
  for (long item = block; item < s.items; item += s.blocks) {
    const Place<D> p(g, s, item);
    float cs[8], sn[8];
    token_table<D, HALVES>(g, p, cs, sn);
    const T* in = static_cast<const T*>(s.x.data) + p.b * s.x.sb + p.t * s.x.st;
    const T* dy = static_cast<const T*>(s.dy.data) + p.b * s.dy.sb + p.t * s.dy.st;
    T* out = static_cast<T*>(s.y.data) + p.b * s.y.sb + p.t * s.y.st;
    for (int h = p.h0; h < p.h1; ++h) {
      const Raw rx = load_row<T, D>(in + h * s.x.sh, p.c), rd = load_row<T, D>(dy + h * s.dy.sh, p.c);
      float x[16], d[16], ss = 0.0f, dot = 0.0f;
      unpack_row<T>(rx, x);
      unpack_row<T>(rd, d);
      rotate<HALVES>(d, cs, sn, -1.0f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        ss = fmaf(x[i], x[i], ss);
        dot = fmaf(d[i] * w[i], x[i], dot);
      }
      const float r = rsqrtf(group_sum<G>(ss) * (1.0f / D) + g.eps);
      const float m = group_sum<G>(dot) * r * (1.0f / D);          // mean(g w n)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float n = x[i] * r;
        if (p.on) dw[i] = fmaf(d[i], n, dw[i]);
        x[i] = r * (d[i] * w[i] - n * m);
      }
      if (p.on) store_row<T, D>(out + h * s.y.sh, p.c, x);
    }
  }
  if (!s.part) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < 16; ++i) red[warp][(i >> 3) * (D / 2) + 8 * lane + (i & 7)] = dw[i];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += red[i][threadIdx.x];
    s.part[(size_t)block * D + threadIdx.x] = v;
  }
}

// dw of one side: the blocks' partial rows in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) k_norm_dw(NormRopeArgs g) {
  constexpr int kSlices = 1024 / D;
  __shared__ float red[kSlices][D];
  const NormSide& s = g.side[blockIdx.x];
  if (!s.part) return;
  const int c = threadIdx.x % D, sl = threadIdx.x / D;
  float v = 0.0f;
#pragma unroll 16                       // loads in flight; the additions keep their order
  for (int i = sl; i < s.blocks; i += kSlices) v += s.part[(size_t)i * D + c];
  red[sl][c] = v;
  __syncthreads();
  if (sl == 0) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) v += red[i][c];
    s.dw[c] = v;
  }
}

template <typename T, int D, bool HALVES>
cudaError_t launch(const NormRopeArgs& g, bool back, cudaStream_t st) {
  if (!back) {
    k_norm_rope<T, D, HALVES><<<(unsigned)(g.side[0].items + g.side[1].items), kThreads, 0, st>>>(g);
    return cudaGetLastError();
  }
  k_norm_rope_back<T, D, HALVES><<<(unsigned)(g.side[0].blocks + g.side[1].blocks), kThreads, 0, st>>>(g);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!g.side[0].part && !g.side[1].part)) return e;
  k_norm_dw<D><<<2, 1024, 0, st>>>(g);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const NormRopeArgs& g, bool halves, bool back, cudaStream_t st) {
  if (g.d == 128) return halves ? launch<T, 128, true>(g, back, st) : launch<T, 128, false>(g, back, st);
  return halves ? launch<T, 64, true>(g, back, st) : launch<T, 64, false>(g, back, st);
}

da2_status check_norm_config(const da2_norm_rope_config* c) {
  if (!c) return DA2_ERR_INVALID_ARG;
  if (c->B <= 0 || c->Hq <= 0 || c->Hk < 0 || c->T <= 0 || c->T_rot < 0 || c->T_rot > c->T)
    return DA2_ERR_INVALID_ARG;
  if (!(c->eps >= 0.0f) || std::isinf(c->eps)) return DA2_ERR_INVALID_ARG;
  if (c->dtype != DA2_DTYPE_BF16 && c->dtype != DA2_DTYPE_F16) return DA2_ERR_INVALID_ARG;
  if (c->flags & ~(DA2_ROPE_HALVES | DA2_ROPE_BATCHED)) return DA2_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return DA2_ERR_UNSUPPORTED;
  if (c->T > kMaxTokens) return DA2_ERR_UNSUPPORTED;
  // the grid holds at most one block per token block, head and batch entry
  if (((long)c->T + 31) / 32 * c->B > (1L << 30) / ((long)c->Hq + c->Hk)) return DA2_ERR_UNSUPPORTED;
  return DA2_OK;
}

// Tensors and split of the work of one call. dy is empty in the forward pass.
da2_status fill_args(const da2_norm_rope_config* c, const da2_tensor* x[2], const da2_tensor* dy[2],
                     const da2_tensor* y[2], const float* w[2], const float* cos_t, const float* sin_t,
                     NormRopeArgs* g) {
  const int H[2] = {c->Hq, c->Hk};
  if (c->T_rot > 0) {
    if (!cos_t || !sin_t) return DA2_ERR_INVALID_ARG;
    if (!aligned16(cos_t) || !aligned16(sin_t)) return DA2_ERR_ALIGNMENT;
  }
  *g = NormRopeArgs{};
  g->B = c->B; g->T = c->T; g->T_rot = c->T_rot; g->d = c->d; g->eps = c->eps;
  g->cos_t = cos_t; g->sin_t = sin_t;
  g->tab_sb = (c->flags & DA2_ROPE_BATCHED) ? (int64_t)c->T_rot * (c->d / 2) : 0;
  const int tok = kThreads / (c->d / 16);
  g->token_blocks = (c->T + tok - 1) / tok;
  // Heads per block: 16 (forward; 480p layer 239 us, 245 with 8, 313 with 20) or 8 (backward) share a
  // token's table row while that leaves two blocks for every processor (148); shorter inputs are cut
  // finer, down to one head.
  auto blocks = [&](int hc) {
    long n = 0;
    for (int s = 0; s < 2; ++s) n += (H[s] + hc - 1) / hc;
    return n * g->token_blocks * c->B;
  };
  int hc = dy ? 8 : 16;
  while (hc > 1 && blocks(hc) < 2 * 148) hc /= 2;
  g->head_chunk = hc;
  for (int s = 0; s < 2; ++s) {
    NormSide& sd = g->side[s];
    sd.H = H[s];
    sd.chunks = (H[s] + hc - 1) / hc;
    sd.items = (long)c->B * g->token_blocks * sd.chunks;
    if (H[s] == 0) continue;
    da2_status e = check_tensor(x[s], c->B, H[s], c->T, c->d, &sd.x);
    if (e == DA2_OK) e = check_tensor(y[s], c->B, H[s], c->T, c->d, &sd.y);
    if (e == DA2_OK && dy) e = check_tensor(dy[s], c->B, H[s], c->T, c->d, &sd.dy);
    if (e != DA2_OK) return e;
    if (w[s] && !aligned16(w[s])) return DA2_ERR_ALIGNMENT;
    sd.w = w[s];
  }
  return DA2_OK;
}

size_t dw_bytes(const da2_norm_rope_config* c) { return (size_t)2 * kNormBackBlocks * c->d * sizeof(float); }

}  // namespace
}  // namespace da2

using namespace da2;

extern "C" {

da2_status da2_qk_norm_rope(const da2_norm_rope_config* cfg, const da2_tensor* q, const da2_tensor* k,
                            const float* wq, const float* wk, const float* cos_t, const float* sin_t,
                            const da2_tensor* q_out, const da2_tensor* k_out, cudaStream_t stream) {
  const NvtxRange range("da2_qk_norm_rope");
  da2_status s = check_norm_config(cfg);
  if (s != DA2_OK) return s;
  const da2_tensor* x[2] = {q, k};
  const da2_tensor* y[2] = {q_out, k_out};
  const float* w[2] = {wq, wk};
  NormRopeArgs g;
  s = fill_args(cfg, x, nullptr, y, w, cos_t, sin_t, &g);
  if (s != DA2_OK) return s;
  const bool halves = (cfg->flags & DA2_ROPE_HALVES) != 0;
  return cuda_status(cfg->dtype == DA2_DTYPE_BF16 ? launch_t<__nv_bfloat16>(g, halves, false, stream)
                                                  : launch_t<__half>(g, halves, false, stream));
}

da2_status da2_qk_norm_rope_workspace_size(const da2_norm_rope_config* cfg, size_t* bytes) {
  const da2_status s = check_norm_config(cfg);
  if (s != DA2_OK) return s;
  if (!bytes) return DA2_ERR_INVALID_ARG;
  *bytes = dw_bytes(cfg);
  return DA2_OK;
}

da2_status da2_qk_norm_rope_backward(const da2_norm_rope_config* cfg, const da2_tensor* dq_out,
                                     const da2_tensor* dk_out, const da2_tensor* q, const da2_tensor* k,
                                     const float* wq, const float* wk, const float* cos_t,
                                     const float* sin_t, const da2_tensor* dq, const da2_tensor* dk,
                                     float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                     cudaStream_t stream) {
  const NvtxRange range("da2_qk_norm_rope_backward");
  da2_status s = check_norm_config(cfg);
  if (s != DA2_OK) return s;
  const da2_tensor* x[2] = {q, k};
  const da2_tensor* dy[2] = {dq_out, dk_out};
  const da2_tensor* y[2] = {dq, dk};
  const float* w[2] = {wq, wk};
  NormRopeArgs g;
  s = fill_args(cfg, x, dy, y, w, cos_t, sin_t, &g);
  if (s != DA2_OK) return s;
  float* dw[2] = {dwq, dwk};
  if (dwq || dwk) {
    if (!ws) return DA2_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
        ((reinterpret_cast<uintptr_t>(dwq) | reinterpret_cast<uintptr_t>(dwk)) & 3u) != 0)
      return DA2_ERR_ALIGNMENT;
    if (ws_bytes < dw_bytes(cfg)) return DA2_ERR_WORKSPACE;
  }
  for (int i = 0; i < 2; ++i) {
    NormSide& sd = g.side[i];
    sd.blocks = (int)(sd.items < kNormBackBlocks ? sd.items : kNormBackBlocks);
    sd.dw = sd.H > 0 ? dw[i] : nullptr;
    sd.part = sd.dw ? static_cast<float*>(ws) + (size_t)i * kNormBackBlocks * cfg->d : nullptr;
  }
  const bool halves = (cfg->flags & DA2_ROPE_HALVES) != 0;
  return cuda_status(cfg->dtype == DA2_DTYPE_BF16 ? launch_t<__nv_bfloat16>(g, halves, true, stream)
                                                  : launch_t<__half>(g, halves, true, stream));
}

}  // extern "C"
