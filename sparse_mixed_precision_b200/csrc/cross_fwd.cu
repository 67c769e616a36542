// Attention of the video tokens to an encoder's states of another length (forward).
//
//   s = q k^T scale,  p = 2^(s log2e - m),  o = (sum p v) / (sum p),  one pass over the keys with
//   the running maximum m and sum per row. m only follows the row's maximum when that has grown by
//   more than 2^8: p then stays below 2^8, the sums are exact in the same way, and the accumulator
//   is rescaled a few times at most.
//
// A work item is 256 query rows (two 128-row tiles) of one head and a run of 128-key tiles. One
// block per processor, persistent over items; neighbouring blocks work on one head, whose keys and
// values stay in L2. 384 threads:
//   warps 0-3, 4-7  softmax and epilogue of tile A, B: thread r owns query row r (TMEM lane r)
//   warp 8          issues all MMAs (one thread), owns the tensor memory
//   warp 9          loads: Q once per item, K and V tiles through a ring of stages
//   warp 10         zeroes value rows behind the length in the last tile, where the tensor holds
//                   something else there (0 times NaN would reach the sum)
// Tensor memory: S of A and B (128 columns each), O of A and B (d columns each). P overwrites its
// own S as 16-bit pairs and is the A operand of P V, so that S of the next key tile is issued
// directly behind P V, in order, with no buffer between; while one tile's softmax runs, the tensor
// cores work on the other's. In the last key tile only the 16-key groups that hold a valid key are
// multiplied.
#include <type_traits>

#include "cross.cuh"
#include "f32x2.cuh"

namespace da2 {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCleanWarp = 10;

template <int D>
struct Smem {
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kStage0 = 2 * kTile;
  static constexpr uint32_t kBars = kStage0 + kStages * kTile;
  static constexpr uint32_t kBytes = kBars + 512 + 1024;        // with room to align the base
  static_assert(kBytes <= 232448, "shared memory budget");
};
template <int D>
struct Bars {
  uint64_t kv_full[Smem<D>::kStages], kv_empty[Smem<D>::kStages];
  uint64_t s_full[2], p_full[2], q_full[2], q_empty[2], o_full[2], o_free[2];
  uint64_t v_dirty, v_clean, done;
  uint32_t tmem, abort;
};
static_assert(sizeof(Bars<64>) <= 512, "barrier area");

// tensor-memory columns of tile x
__device__ __forceinline__ constexpr uint32_t col_s(int x) { return 128u * x; }
__device__ __forceinline__ constexpr uint32_t col_o(int x) { return 256u + 128u * x; }

// Work item i: batch entry, head, 256-row query tile, and its key tiles t0 .. t0 + nt - 1.
struct Item {
  int b, h, row0, t0, nt, split, len;
  bool has_b;
  __device__ __forceinline__ Item(const CrossArgs& g, int i) {
    split = i % g.splits;
    i /= g.splits;
    const int p = i % g.q_pairs;
    i /= g.q_pairs;
    b = i / g.H;
    h = i - b * g.H;
    row0 = p * 256;
    has_b = row0 + 128 < g.Tq;
    len = valid_keys(g, b);
    const int tiles = (len + 127) >> 7;
    t0 = (int)((long)tiles * split / g.splits);
    nt = (int)((long)tiles * (split + 1) / g.splits) - t0;
  }
  __device__ __forceinline__ bool has(int x) const { return x == 0 || has_b; }
  // valid keys of this item's tile t
  __device__ __forceinline__ int keys(int t) const { return min(128, len - 128 * (t0 + t)); }
  // whether rows of the value tile must be zeroed first: the last group of 16 ends behind the length
  __device__ __forceinline__ bool dirty(const CrossArgs& g, int t) const {
    return (keys(t) & 15) != 0 && len < g.Tk;
  }
};

template <int D>
__device__ __noinline__ void rescale(uint32_t taddr, float alpha) {
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    uint32_t v[32];
    tc::tmem_ld32(taddr + c, v);
    tc::tmem_wait_ld16(v);
    tc::tmem_wait_ld16(v + 16);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
    tc::tmem_st16(taddr + c, v);
    tc::tmem_st16(taddr + c + 16, v + 16);
  }
  tc::tmem_wait_st();
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_forward(const __grid_constant__ CrossMaps maps, const __grid_constant__ CrossArgs g) {
  using S = Smem<D>;
  constexpr int kStages = S::kStages;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  Bars<D>* bars = reinterpret_cast<Bars<D>*>(sm + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = g.B * g.H * g.q_pairs * g.splits;
  const Guard gd{g.err, &bars->abort, g.wait_ns};

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(&bars->s_full[x], 1);
      tc::mbar_init(&bars->p_full[x], 128);
      tc::mbar_init(&bars->q_full[x], 1);
      tc::mbar_init(&bars->q_empty[x], 1);
      tc::mbar_init(&bars->o_full[x], 1);
      tc::mbar_init(&bars->o_free[x], 128);
    }
    tc::mbar_init(&bars->v_dirty, 1);
    tc::mbar_init(&bars->v_clean, 1);
    tc::mbar_init(&bars->done, 1);
    bars->abort = 0u;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars->tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars->tmem;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      uint32_t n = 0, q_loads[2] = {0, 0};
      bool dead = false;
      auto load = [&](const CUtensorMap* map, int row, int head, int b) {
        const uint32_t s = n % kStages;
        if (g.stall && n == 0) { ++n; return true; }
        if (!guard_wait(&bars->kv_empty[s], ((n / kStages) & 1) ^ 1, gd)) return false;
        tc::mbar_arrive_expect_tx(&bars->kv_full[s], S::kTile);
        load_tile<D>(sm + S::kStage0 + s * S::kTile, map, row, head, b, &bars->kv_full[s]);
        ++n;
        return true;
      };
      for (int i = blockIdx.x; i < items && !dead; i += gridDim.x) {
        const Item w(g, i);
        if (w.nt == 0) continue;
        for (int x = 0; x < 2 && !dead; ++x) {
          if (!w.has(x)) continue;
          if (!guard_wait(&bars->q_empty[x], (q_loads[x] & 1) ^ 1, gd)) { dead = true; break; }
          tc::mbar_arrive_expect_tx(&bars->q_full[x], S::kTile);
          load_tile<D>(sm + x * S::kTile, &maps.q, w.row0 + 128 * x, w.h, w.b, &bars->q_full[x]);
          ++q_loads[x];
        }
        for (int t = 0; t < w.nt && !dead; ++t) {
          const int row = 128 * (w.t0 + t), hk = w.h / g.group;
          dead = !load(&maps.k, row, hk, w.b);
          if (!dead) dead = !load(&maps.v, row, hk, w.b);
        }
      }
      // every copy issued above has landed before the block ends
      for (uint32_t s = 0; s < (uint32_t)kStages && s < n; ++s)
        guard_wait(&bars->kv_full[s], (((n - 1 - s) / kStages)) & 1, gd, false);
      for (int x = 0; x < 2; ++x)
        if (q_loads[x]) guard_wait(&bars->q_full[x], (q_loads[x] - 1) & 1, gd, false);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      uint32_t step = 0, q_items[2] = {0, 0}, o_items[2] = {0, 0}, p_steps[2] = {0, 0}, cleans = 0;
      // S of tile x, key tile t of an item (global step gs)
      auto issue_s = [&](const Item& w, int x, int t, uint32_t gs) -> bool {
        if (t == 0 && !guard_wait(&bars->q_full[x], q_items[x]++ & 1, gd)) return false;
        const uint32_t n = 2 * gs, s = n % kStages;
        if (!guard_wait(&bars->kv_full[s], (n / kStages) & 1, gd)) return false;
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_f16(kBf16, 128, (w.keys(t) + 15) & ~15, false);
        const uint64_t a = tc::sdesc_k(sm + x * S::kTile), b = tc::sdesc_k(sm + S::kStage0 + s * S::kTile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (k / 4) * (16384 >> 4) + (k % 4) * (32 >> 4);
          tc::mma_f16(tmem + col_s(x), a + off, b + off, id, k > 0);
        }
        tc::mma_commit(&bars->s_full[x]);
        if (x == 1 || !w.has_b) tc::mma_commit(&bars->kv_empty[s]);
        if (t == w.nt - 1) tc::mma_commit(&bars->q_empty[x]);
        return true;
      };
      auto issue_pv = [&](const Item& w, int x, int t, uint32_t gs) -> bool {
        const uint32_t n = 2 * gs + 1, s = n % kStages;
        if (!guard_wait(&bars->kv_full[s], (n / kStages) & 1, gd)) return false;
        const bool dirty = x == 0 && w.dirty(g, t);
        if (dirty) tc::mbar_arrive(&bars->v_dirty);      // cleaned while the softmax runs
        if (!guard_wait(&bars->p_full[x], p_steps[x]++ & 1, gd)) return false;
        if (dirty && !guard_wait(&bars->v_clean, cleans++ & 1, gd)) return false;
        if (t == 0) {
          if (o_items[x] > 0 && !guard_wait(&bars->o_free[x], (o_items[x] - 1) & 1, gd)) return false;
          ++o_items[x];
        }
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_f16(kBf16, 128, D, true);
        const uint64_t b = tc::sdesc_mn(sm + S::kStage0 + s * S::kTile, 16384);
        const int ks = (w.keys(t) + 15) >> 4;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < ks)
            tc::mma_f16_ta(tmem + col_o(x), tmem + col_s(x) + 8 * k, b + k * (2048 >> 4), id, (t > 0) | (k > 0));
        if (x == 1 || !w.has_b) tc::mma_commit(&bars->kv_empty[s]);
        if (t == w.nt - 1) tc::mma_commit(&bars->o_full[x]);
        return true;
      };
      int i = blockIdx.x;
      auto skip_empty = [&](int at) {
        while (at < items && Item(g, at).nt == 0) at += gridDim.x;
        return at;
      };
      bool dead = false;
      i = skip_empty(i);
      if (i < items) {
        Item w(g, i);
        for (int x = 0; x < 2 && !dead; ++x)
          if (w.has(x)) dead = !issue_s(w, x, 0, 0);
        while (!dead) {
          const int in = skip_empty(i + gridDim.x);
          const bool more = in < items;
          const Item wn(g, more ? in : i);
          for (int t = 0; t < w.nt && !dead; ++t, ++step) {
            const bool last = t == w.nt - 1;
            for (int x = 0; x < 2 && !dead; ++x) {
              if (w.has(x)) dead = !issue_pv(w, x, t, step);
              if (dead) break;
              if (!last) { if (w.has(x)) dead = !issue_s(w, x, t + 1, step + 1); }
              else if (more && wn.has(x)) dead = !issue_s(wn, x, 0, step + 1);
            }
          }
          if (!more) break;
          w = wn;
          i = in;
        }
      }
      tc::mma_commit(&bars->done);
      guard_wait(&bars->done, 0, gd, false);       // all MMAs retired before TMEM is freed
    }
  } else if (warp == kCleanWarp) {
    // The issuer names each tile to clean once it has landed: this warp, which skips all others,
    // could not tell from the stage's own barrier which of its fills that shows.
    uint32_t step = 0, cleans = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const Item w(g, i);
      if (w.nt > 0 && w.dirty(g, w.nt - 1)) {
        if (!guard_wait(&bars->v_dirty, cleans++ & 1, gd)) break;
        const int keys = w.keys(w.nt - 1);
        zero_rows<D>(sm + S::kStage0 + (2 * (step + w.nt - 1) + 1) % kStages * S::kTile, keys, (keys + 15) & ~15, lane);
        if (lane == 0) tc::mbar_arrive(&bars->v_clean);
      }
      step += w.nt;
    }
  } else if (warp < kMmaWarp) {
    const int x = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = lane_base + col_s(x), tO = lane_base + col_o(x);
    const float c = g.scale_log2;
    uint32_t step = 0, done_items = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const Item w(g, i);
      if (!w.has(x)) continue;
      const int row = w.row0 + 128 * x + r;
      const bool on = row < g.Tq;
      const size_t flat = ((size_t)w.b * g.H + w.h) * g.Tq + row;       // row of lse and the parts
      const size_t part = (size_t)w.split * g.B * g.H * g.Tq + flat;
      float m = -INFINITY, l = 0.0f;
      for (int t = 0; t < w.nt; ++t, ++step) {
        guard_wait(&bars->s_full[x], step & 1, gd);
        tc::fence_after_sync();
        const int keys = w.keys(t);
        uint32_t su[128];
        float* s = reinterpret_cast<float*>(su);
#pragma unroll
        for (int k = 0; k < 128; k += 32)
          if (k < keys) tc::tmem_ld32(tS + k, su + k);
#pragma unroll
        for (int k = 0; k < 128; k += 16) tc::tmem_wait_ld16(su + k);
        if (keys < 128) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= keys) s[k] = -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = s[q];
#pragma unroll
        for (int k = 4; k < 128; k += 8) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = k + 4 + q < 128 ? max3(mx[q], s[k + q], s[k + 4 + q]) : fmaxf(mx[q], s[k + q]);
        }
        const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        if (t == 0) {
          m = m_new;
        } else {
          const bool grow = m_new > m + 8.0f;
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? ex2(m - m_new) : 1.0f;
            rescale<D>(tO, alpha);                       // the previous P V is done: S came behind it
            l *= alpha;
            if (grow) m = m_new;
          }
        }
        const float bias = m == -INFINITY ? 0.0f : -m;   // a row of -inf scores so far: p = 0
        const f32x2 c2 = pk2(c, c), b2 = pk2(bias, bias);
        f32x2 sum[2] = {pk2(0.0f, 0.0f), pk2(0.0f, 0.0f)};
#pragma unroll
        for (int k0 = 0; k0 < 128; k0 += 32) {
          if (k0 < keys) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float a, b;
              upk2(fma2(pk2(s[k0 + k], s[k0 + k + 1]), c2, b2), a, b);
              a = ex2(a);
              b = ex2(b);
              sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pk2(a, b));
              p[k >> 1] = pack16<T>(a, b);
            }
            tc::tmem_st16(tS + k0 / 2, p);
          }
        }
        float a0, a1, b0, b1;
        upk2(sum[0], a0, a1);
        upk2(sum[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&bars->p_full[x]);
      }
      if (w.nt == 0) {                                   // no key: zero, and no weight in a join
        if (on && g.splits > 1) {
          float4* o = reinterpret_cast<float4*>(g.part_o + part * D);
          for (int k = 0; k < D / 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          g.part_lse[part] = -INFINITY;
        } else if (on) {
          uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(g.out.data) + w.b * g.out.sb + w.h * g.out.sh +
                                              row * g.out.st);
          for (int k = 0; k < D / 8; ++k) o[k] = make_uint4(0u, 0u, 0u, 0u);
          if (g.lse) g.lse[flat] = -INFINITY;
        }
        continue;
      }
      if (!guard_wait(&bars->o_full[x], done_items++ & 1, gd)) break;
      tc::fence_after_sync();
      const float inv = 1.0f / l;
      const float lse2 = m + log2f(l);
#pragma unroll
      for (int k0 = 0; k0 < D; k0 += 32) {
        uint32_t v[32];
        tc::tmem_ld32(tO + k0, v);
        tc::tmem_wait_ld16(v);
        tc::tmem_wait_ld16(v + 16);
        if (k0 + 32 == D) {                              // O is free once the last column is read
          tc::fence_before_sync();
          tc::mbar_arrive(&bars->o_free[x]);
        }
        if (!on) continue;
        if (g.splits > 1) {
          float4* o = reinterpret_cast<float4*>(g.part_o + part * D + k0);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = make_float4(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv,
                               __uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv);
        } else {
          uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(g.out.data) + w.b * g.out.sb + w.h * g.out.sh +
                                              row * g.out.st + k0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = pack16<T>(__uint_as_float(v[8 * k + 2 * e]) * inv, __uint_as_float(v[8 * k + 2 * e + 1]) * inv);
            o[k] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
      if (on) {
        if (g.splits > 1) g.part_lse[part] = lse2;
        else if (g.lse) g.lse[flat] = lse2 * kLn2;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of split keys: out = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s - max), one warp
// per row.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_cross_join(const __grid_constant__ CrossArgs g) {
  const size_t rows = (size_t)g.B * g.H * g.Tq;
  const size_t row = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float m = -INFINITY;
  for (int s = 0; s < g.splits; ++s) m = fmaxf(m, g.part_lse[s * rows + row]);
  float acc[D / 32] = {}, total = 0.0f;
  if (m != -INFINITY) {
    for (int s = 0; s < g.splits; ++s) {
      const float w = ex2(g.part_lse[s * rows + row] - m);
      total += w;
      const float* o = g.part_o + (s * rows + row) * D + lane * (D / 32);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(w, o[e], acc[e]);
    }
  }
  const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
  const size_t bh = row / g.Tq;
  const int t = (int)(row - bh * g.Tq), b = (int)(bh / g.H), h = (int)(bh - (size_t)b * g.H);
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(g.out.data) + b * g.out.sb + h * g.out.sh +
                                              t * g.out.st + lane * (D / 32));
#pragma unroll
  for (int e = 0; e < D / 64; ++e) out[e] = pack16<T>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (g.lse && lane == 0) g.lse[row] = m == -INFINITY ? -INFINITY : (m + log2f(total)) * kLn2;
}

template <typename T, int D>
cudaError_t launch(const CrossArgs& g, const CrossMaps& m, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_cross_forward<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  const int items = g.B * g.H * g.q_pairs * g.splits;
  k_cross_forward<T, D><<<items < g.sms ? items : g.sms, kThreads, Smem<D>::kBytes, st>>>(m, g);
  e = cudaGetLastError();
  if (e != cudaSuccess || g.splits == 1) return e;
  const size_t rows = (size_t)g.B * g.H * g.Tq;
  k_cross_join<T, D><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_forward(const CrossArgs& g, const CrossMaps& m, bool bf16, cudaStream_t st) {
  if (g.d == 128) return bf16 ? launch<__nv_bfloat16, 128>(g, m, st) : launch<__half, 128>(g, m, st);
  return bf16 ? launch<__nv_bfloat16, 64>(g, m, st) : launch<__half, 64>(g, m, st);
}

}  // namespace da2
