// Attention of the video tokens to an encoder's states of another length (forward).
//
//   s = q k^T scale,  p = 2^(s log2e - m),  o = (sum p v) / (sum p),  one pass over the keys with
//   the running maximum m and sum per row. m only follows the row's maximum when that has grown by
//   more than 2^8: p then stays below 2^8, the sums are exact in the same way, and the accumulator
//   is rescaled a few times at most.
//
// A work item is 256 query rows (two 128-row tiles) of one head and a run of 64-key steps. One block
// per processor, persistent over items. Neighbouring blocks work on one head, whose keys and values
// stay in L2, in either layout (40 heads token-major, the heads of the same rows on neighbouring blocks
// instead: within the noise of 2 % up to 40 MB of keys and values, 6200 us against 5700 at 160 MB). 512
// threads:
//   warps 0-3, 4-7  softmax of tile A, B: thread r owns query row r (TMEM lane r)
//   warps 8-11      epilogue of either tile: O / sum, rounded, through shared memory to a tensor-map
//                   store, while the softmax warps are on the next item
//   warps 12, 13    issue the MMAs of tile A, B; warp 12 owns the tensor memory
//   warp 14         loads K and V of the steps in turn, through a ring
//   warp 15         loads Q, once per item (and the next item's into L2 ahead)
// Tensor memory: per tile two S buffers of 64 columns and O (d columns). P overwrites its own S as
// 16-bit pairs and is the A operand of P V; S of the step after next is issued directly behind P V, so
// that a softmax warp finds its next S ready and only waits for its own arithmetic: the exponentials
// (16 per cycle and processor) bound a step at 1024 cycles for the pair of tiles, and S with 64 columns
// takes 48 cycles per MMA where 128 take 64, 1242 cycles for the pair. In the last step only the 16-key
// groups that hold a valid key are multiplied.
//
// Measured, 40 heads, d = 128, bf16, 32760 queries, in 20 calls at 1965 MHz and in a second and a half of
// calls, where the power cap leaves about 1640 MHz: 512 keys 376 us = 914 TFLOP/s and 427 us = 805, 2048
// keys 1329 us = 1034 TFLOP/s and 1498 us = 917, 64 keys 147 and 152 us (the bytes alone take 102). What
// bounds it now: instruction fetch and hand-offs, about 2000 cycles a step against 1242. Dropped, each
// slower on the 512-key case: one S
// buffer of 128 columns per tile (435 us; 510 with the row in registers), one issuing warp, MMAs issued
// from inside one lane's branch (75 cycles each to issue instead of 16 to 32), polling waits, a degree-4
// polynomial for an eighth to a half of the exponentials (no gain: they are not the bound).
#include <type_traits>

#include "cross.cuh"
#include "f32x2.cuh"

namespace da2 {
namespace {

constexpr int kThreads = 512;
constexpr int kEpiWarp = 8, kMmaWarp = 12, kLoadWarp = 14, kLoadQWarp = 15;
constexpr int kStep = 64;                                         // keys per step

template <int D>
struct Smem {
  static constexpr uint32_t kQ = 128 * D * 2;                     // per tile
  static constexpr uint32_t kHalf = kStep * D * 2;                // K or V of one step
  static constexpr uint32_t kKv = 2 * kHalf;                      // per stage: both
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kOut = 2 * kQ;                        // two 64-channel boxes of the epilogue
  static constexpr uint32_t kStage0 = kOut + 2 * 16384;
  static constexpr uint32_t kStats = kStage0 + kStages * kKv;     // [tile][row] sum and maximum
  static constexpr uint32_t kBars = kStats + 2048;
  static constexpr uint32_t kBytes = kBars + 512;
  static_assert(kBytes <= 232448, "shared memory budget");
};
template <int D>
struct Bars {
  uint64_t kv_full[Smem<D>::kStages], kv_empty[Smem<D>::kStages];
  uint64_t s_full[2][2], p_full[2][2], q_full[2], q_empty[2], pv_done[2], o_full[2], l_full[2], o_free[2];
  uint64_t done;
  uint32_t tmem, abort;
};
static_assert(sizeof(Bars<64>) <= 512, "barrier area");

// tensor-memory columns of tile x
__device__ __forceinline__ constexpr uint32_t col_s(int x, int buf) { return 128u * x + 64u * buf; }
__device__ __forceinline__ constexpr uint32_t col_o(int x) { return 256u + 128u * x; }

// Work item i: batch entry, head, 256-row query tile, and its steps t0 .. t0 + nt - 1.
struct Item {
  int b, h, row0, t0, nt, split, len;
  bool has_b;
  __device__ __forceinline__ Item(const CrossArgs& g, int i) {
    int v[7];
    decode(g, i, v);
    b = v[0], h = v[1], row0 = v[2], t0 = v[3], nt = v[4], split = v[5], len = v[6];
    has_b = row0 + 128 < g.Tq;
  }
  // not inline: its divisions in each of the kernel's roles would crowd the instruction cache
  static __device__ __noinline__ void decode(const CrossArgs& g, int i, int* v) {
    int b, h, row0, t0 = 0, split = 0;
    uint32_t u = i;
    if (g.splits > 1) {
      split = u % g.splits;
      u /= g.splits;
    }
    const uint32_t bh = u / g.q_pairs;
    row0 = (u - bh * g.q_pairs) * 256;
    b = bh / g.H;
    h = bh - b * g.H;
    const int len = valid_keys(g, b);
    int nt = (len + kStep - 1) / kStep;
    if (g.splits > 1) {
      t0 = (int)((long)nt * split / g.splits);
      nt = (int)((long)nt * (split + 1) / g.splits) - t0;
    }
    v[0] = b, v[1] = h, v[2] = row0, v[3] = t0, v[4] = nt, v[5] = split, v[6] = len;
  }
  __device__ __forceinline__ bool has(int x) const { return x == 0 || has_b; }
  // valid keys of this item's step t
  __device__ __forceinline__ int keys(int t) const { return min(kStep, len - kStep * (t0 + t)); }
  // whether rows of the value tile must be zeroed first: the last group of 16 ends behind the length
  __device__ __forceinline__ bool dirty(const CrossArgs& g, int t) const {
    return (keys(t) & 15) != 0 && len < g.Tk;
  }
};

// The scores of a chunk from `keys` on are behind the length: -inf.
__device__ __forceinline__ void mask32(float* s, int keys) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (k >= keys) s[k] = -INFINITY;
}

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

// Issues the MMAs of tile X. The whole warp runs this, one lane issues: every operand is the same in
// all lanes and stays in uniform registers (issued from inside one lane's branch, an MMA took 75
// cycles to issue, more than it runs). One warp per tile, because the waits and commits of a step take
// most of a softmax step's time. For an item without tile B, its issuer only passes the stages on.
template <typename T, int D, int X>
__device__ __forceinline__ void issue(const CrossArgs& g, uint8_t* sm, Bars<D>* bars, int items, const Guard& gd,
                                      int lane) {
  using S = Smem<D>;
  constexpr int kStages = S::kStages;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kHi = (uint32_t)(tc::kSw128 >> 32) | (1024 >> 4);     // high word of every descriptor
  constexpr uint32_t id_s = tc::idesc_f16(kBf16, 128, kStep, false), id_o = tc::idesc_f16(kBf16, 128, D, true);
  const bool lead = tc::elect_one();
  const uint32_t sm0 = tc::smem_u32(sm) >> 4;
  // A step between its S and its P V: valid keys, and flags.
  constexpr uint32_t kFirst = 1 << 7, kLast = 1 << 8;    // of the item
  constexpr uint32_t kDirty = 1 << 9;                    // value rows to zero
  constexpr uint32_t kSignal = 1 << 10;                  // P V is signalled: the next step is the last
  constexpr uint32_t kHas = 1 << 11, kAny = 1 << 12;     // the item has this tile; not an empty step
  uint32_t n_s = 0, n_pv = 0;                            // stages of K and of V
  uint32_t q_items = 0, o_items = 0, own_s = 0, own_pv = 0;      // items and steps of this tile
  auto issue_s = [&](uint32_t f) -> bool {
    const uint32_t s = n_s % kStages, parity = (n_s / kStages) & 1;
    ++n_s;
    if (!(f & kHas)) return true;
    if ((f & kFirst) && !warp_wait(&bars->q_full[X], q_items++ & 1, gd)) return false;
    if (!warp_wait(&bars->kv_full[s], parity, gd)) return false;
    tc::fence_after_sync();
    const uint32_t keys = f & 127, buf = own_s++ & 1;
    const uint32_t id = keys == kStep ? id_s : tc::idesc_f16(kBf16, 128, (keys + 15) & ~15, false);
    const uint32_t a = (sm0 + (X * S::kQ >> 4)) | 1u << 16;
    const uint32_t b = (sm0 + (S::kStage0 >> 4) + s * (S::kKv >> 4)) | 1u << 16;
    if (lead) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_f16(col_s(X, buf), tc::desc(a + (k / 4) * (16384 >> 4) + (k % 4) * (32 >> 4), kHi),
                    tc::desc(b + (k / 4) * (kStep * 128 >> 4) + (k % 4) * (32 >> 4), kHi), id, k > 0);
      tc::mma_commit(&bars->s_full[X][buf]);
      if (f & kLast) tc::mma_commit(&bars->q_empty[X]);
    }
    return true;
  };
  auto issue_pv = [&](uint32_t f) -> bool {
    const uint32_t s = n_pv % kStages, parity = (n_pv / kStages) & 1;
    ++n_pv;
    if (!(f & kHas)) {
      if (!warp_wait(&bars->kv_full[s], parity, gd)) return false;
      if (lead) tc::mbar_arrive(&bars->kv_empty[s]);
      return true;
    }
    const uint32_t keys = f & 127, buf = own_pv & 1;
    const uint32_t at = S::kStage0 + s * S::kKv + S::kHalf;
    // Value rows behind the length, up to the last group of 16, may hold anything, and 0 times NaN
    // would reach the sum: zeroed (by both issuers, with the same zeros).
    if (f & kDirty) zero_rows<D, kStep>(sm + at, keys, (keys + 15) & ~15, lane);
    if (!warp_wait(&bars->p_full[X][buf], (own_pv++ >> 1) & 1, gd)) return false;
    if ((f & kFirst) && o_items++ > 0 && !warp_wait(&bars->o_free[X], o_items & 1, gd)) return false;
    tc::fence_after_sync();
    const uint32_t b = (sm0 + (at >> 4)) | (kStep * 128 >> 4) << 16;
    if (lead) {
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        if (16 * k < keys)
          tc::mma_f16_ta(col_o(X), col_s(X, buf) + 8 * k, tc::desc(b + k * (2048 >> 4), kHi), id_o,
                         k > 0 ? 1u : !(f & kFirst));
      tc::mma_commit(&bars->kv_empty[s]);
      if (f & (kLast | kSignal)) tc::mma_commit(f & kLast ? &bars->o_full[X] : &bars->pv_done[X]);
    }
    return true;
  };
  // S runs two steps ahead of P V, over the items' ends.
  uint32_t f0 = 0, f1 = 0;
  auto step = [&](uint32_t f) -> bool {
    if ((f0 & kAny) && !issue_pv(f0)) return false;
    f0 = f1;
    f1 = f;
    return !(f & kAny) || issue_s(f);
  };
  int i = blockIdx.x, t = 0, tail = 2;                   // behind the last item two empty steps
  Item w(g, min(i, items - 1));
  while (true) {
    while (i < items && t >= w.nt) {
      i += gridDim.x;
      t = 0;
      if (i < items) w = Item(g, i);
    }
    uint32_t f = 0;
    if (i < items) {
      f = kAny | (w.has(X) ? kHas : 0u) | (t == 0 ? kFirst : 0u);
      if (t == w.nt - 1) f |= kLast | (uint32_t)w.keys(t) | (w.dirty(g, t) ? kDirty : 0u);
      else f |= kStep | (t == w.nt - 2 ? kSignal : 0u);
      ++t;
    } else if (tail-- == 0) {
      break;
    }
    if (!step(f)) break;
  }
  if (lead) tc::mma_commit(&bars->done);
  __syncwarp();
  guard_wait(&bars->done, 0, gd, false);           // all MMAs retired before TMEM is freed
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_forward(const __grid_constant__ CrossMaps maps, const __grid_constant__ CrossArgs g) {
  using S = Smem<D>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars<D>* bars = reinterpret_cast<Bars<D>*>(sm + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = g.B * g.H * g.q_pairs * g.splits;
  const Guard gd{g.err, &bars->abort, g.wait_clocks};
  if (tc::smem_u32(sm) & 1023u) {        // the swizzle needs the alignment that the declaration asks for
    if (tid == 0) set_error(g.err, kErrBadIndex);
    return;
  }

  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 2);              // both issuers
    }
    for (int x = 0; x < 2; ++x) {
      for (int k = 0; k < 2; ++k) {
        tc::mbar_init(&bars->s_full[x][k], 1);
        tc::mbar_init(&bars->p_full[x][k], 4);
      }
      tc::mbar_init(&bars->q_full[x], 1);
      tc::mbar_init(&bars->q_empty[x], 1);
      tc::mbar_init(&bars->pv_done[x], 1);
      tc::mbar_init(&bars->o_full[x], 1);
      tc::mbar_init(&bars->l_full[x], 4);
      tc::mbar_init(&bars->o_free[x], 4);
    }
    tc::mbar_init(&bars->done, 2);
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
  constexpr uint32_t tmem = 0;             // all 512 columns are this block's: the base is column 0

  if (warp < kEpiWarp) {
    const int x = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = lane_base + col_o(x);
    const float c = g.scale_log2;
    float2* stats = reinterpret_cast<float2*>(sm + S::kStats) + 128 * x + r;
    uint32_t step = 0, n_items = 0, signals = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const Item w(g, i);
      if (!w.has(x) || w.nt == 0) continue;
      float m = -INFINITY, l = 0.0f;
      for (int t = 0; t < w.nt; ++t, ++step) {
        const uint32_t buf = step & 1, tS = lane_base + col_s(x, buf);
        guard_wait(&bars->s_full[x][buf], (step >> 1) & 1, gd);
        tc::fence_after_sync();
        const int keys = w.keys(t);
        // The row is read twice, 32 columns at a time in rolled loops: the maximum, then the
        // exponentials. Unrolled with the row in registers, the loop's code does not fit the
        // instruction cache beside the other warps' and waits for instructions (2.3 of 9 stalled
        // cycles per instruction).
        const int chunks = (keys + 31) >> 5;
        float mx = -INFINITY;
#pragma unroll 1
        for (int k0 = 0; k0 < keys; k0 += 32) {
          uint32_t u[32];
          float* s = reinterpret_cast<float*>(u);
          tc::tmem_ld32(tS + k0, u);
          tc::tmem_wait_ld16(u);
          tc::tmem_wait_ld16(u + 16);
          if (k0 + 32 > keys) mask32(s, keys - k0);
          float m4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) m4[q] = max3(s[q], s[4 + q], s[8 + q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) m4[q] = max3(m4[q], s[12 + q], s[16 + q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) m4[q] = max3(m4[q], s[20 + q], s[24 + q]);
          mx = max3(mx, max3(m4[0], m4[1], s[28]), max3(max3(m4[2], m4[3], s[29]), s[30], s[31]));
        }
        const float m_new = mx * c;
        if (t == 0) {
          m = m_new;
        } else {
          const bool grow = m_new > m + 8.0f;
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? ex2(m - m_new) : 1.0f;
            // the previous step's P V is done: S of the next step was issued behind it, or, at the
            // item's end, it has a barrier of its own
            if (t < w.nt - 1) guard_wait(&bars->s_full[x][buf ^ 1], ((step + 1) >> 1) & 1, gd);
            else guard_wait(&bars->pv_done[x], signals & 1, gd);
            tc::fence_after_sync();
            rescale<D>(tO, alpha);
            l *= alpha;
            if (grow) m = m_new;
          }
        }
        const float bias = m == -INFINITY ? 0.0f : -m;   // a row of -inf scores so far: p = 0
        const f32x2 c2 = pk2(c, c), b2 = pk2(bias, bias);
        f32x2 sum[2] = {pk2(l, 0.0f), pk2(0.0f, 0.0f)};
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
          uint32_t u[32], p[16];
          float* s = reinterpret_cast<float*>(u);
          tc::tmem_ld32(tS + 32 * i, u);
          tc::tmem_wait_ld16(u);
          tc::tmem_wait_ld16(u + 16);
          if (32 * i + 32 > keys) mask32(s, keys - 32 * i);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float a, b;
            upk2(fma2(pk2(s[k], s[k + 1]), c2, b2), a, b);
            a = ex2(a);
            b = ex2(b);
            sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pk2(a, b));
            p[k >> 1] = pack16<T>(a, b);
          }
          tc::tmem_st16(tS + 16 * i, p);                 // over columns that have been read
        }
        float a0, a1, b0, b1;
        upk2(sum[0], a0, a1);
        upk2(sum[1], b0, b1);
        l = (a0 + a1) + (b0 + b1);
        tc::tmem_wait_st();
        warp_arrive(&bars->p_full[x][buf], lane);
      }
      // the epilogue has taken the previous item's statistics
      if (n_items > 0 && !warp_wait(&bars->o_free[x], (n_items - 1) & 1, gd)) break;
      signals += w.nt > 1;
      *stats = make_float2(l, m);
      warp_arrive(&bars->l_full[x], lane);
      ++n_items;
    }
  } else {
  if (warp == kLoadWarp) {
    if (lane == 0) {
      uint32_t n = 0;
      bool dead = false;
      for (int i = blockIdx.x; i < items && !dead; i += gridDim.x) {
        const Item w(g, i);
        for (int t = 0; t < w.nt; ++t, ++n) {
          const uint32_t s = n % kStages;
          if (g.stall && n == 0) continue;
          if (!guard_wait(&bars->kv_empty[s], ((n / kStages) & 1) ^ 1, gd)) { dead = true; break; }
          tc::mbar_arrive_expect_tx(&bars->kv_full[s], S::kKv);
          load_tile<D, kStep>(sm + S::kStage0 + s * S::kKv, &maps.k, kStep * (w.t0 + t), w.h / g.group, w.b, &bars->kv_full[s]);
          load_tile<D, kStep>(sm + S::kStage0 + s * S::kKv+S::kHalf, &maps.v, kStep * (w.t0 + t), w.h / g.group, w.b, &bars->kv_full[s]);
        }
      }
      // every copy issued above has landed before the block ends
#pragma unroll 1
      for (uint32_t s = 0; s < (uint32_t)kStages && s < n; ++s)
        guard_wait(&bars->kv_full[s], (((n - 1 - s) / kStages)) & 1, gd, false);
    }
  } else if (warp == kLoadQWarp) {
    if (lane == 0) {
      uint32_t q_loads[2] = {0, 0};
      bool dead = false;
      for (int i = blockIdx.x; i < items && !dead; i += gridDim.x) {
        const Item w(g, i);
        if (w.nt == 0) continue;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (dead || !w.has(x)) continue;
          if (!guard_wait(&bars->q_empty[x], (q_loads[x] & 1) ^ 1, gd)) { dead = true; continue; }
          tc::mbar_arrive_expect_tx(&bars->q_full[x], S::kQ);
          load_tile<D>(sm + x * S::kQ, &maps.q, w.row0 + 128 * x, w.h, w.b, &bars->q_full[x]);
          ++q_loads[x];
        }
        if (i + (int)gridDim.x < items) {
          const Item wn(g, i + gridDim.x);
          for (int x = 0; x < 2; ++x)
            if (wn.has(x))
              for (int c = 0; c < D; c += 64) tc::tma_prefetch_4d(&maps.q, c, wn.row0 + 128 * x, wn.h, wn.b);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (q_loads[x]) guard_wait(&bars->q_full[x], (q_loads[x] - 1) & 1, gd, false);
    }
  } else if (warp == kMmaWarp) {
    issue<T, D, 0>(g, sm, bars, items, gd, lane);
  } else if (warp == kMmaWarp + 1) {
    issue<T, D, 1>(g, sm, bars, items, gd, lane);
  } else if (warp < kMmaWarp) {
    // No wait ends this loop early: all 128 threads must meet at the named barrier. After an abort
    // every wait ends soon and what is written is undefined.
    const int r = tid & 127;
    const bool lead = tid == kEpiWarp * 32;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t n_items[2] = {0, 0}, tiles = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const Item w(g, i);
      for (int x = 0; x < 2; ++x) {
        if (!w.has(x)) continue;
        const int row = w.row0 + 128 * x + r;
        const bool on = row < g.Tq;
        const size_t flat = ((size_t)w.b * g.H + w.h) * g.Tq + row;     // row of lse and the parts
        const size_t part = (size_t)w.split * g.B * g.H * g.Tq + flat;
        if (w.nt == 0) {                                 // no key: zero, and no weight in a join
          if (on && g.splits > 1) {
            float4* o = reinterpret_cast<float4*>(g.part_o + part * D);
#pragma unroll 1
            for (int k = 0; k < D / 4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            g.part_lse[part] = -INFINITY;
          } else if (on) {
            uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(g.out.data) + w.b * g.out.sb + w.h * g.out.sh +
                                                row * g.out.st);
#pragma unroll 1
            for (int k = 0; k < D / 8; ++k) o[k] = make_uint4(0u, 0u, 0u, 0u);
            if (g.lse) g.lse[flat] = -INFINITY;
          }
          continue;
        }
        // the boxes of this tile, once the stores of their last use have read them
        uint8_t* box = sm + S::kOut + (D == 64 ? (tiles & 1) * 16384 : 0);
        if (lead) tc::bulk_wait_read<D == 64 ? 1 : 0>();
        asm volatile("bar.sync 2, 128;" ::: "memory");
        guard_wait(&bars->l_full[x], n_items[x] & 1, gd);
        const float2 lm = reinterpret_cast<const float2*>(sm + S::kStats)[128 * x + r];
        guard_wait(&bars->o_full[x], n_items[x] & 1, gd);
        ++n_items[x];
        ++tiles;
        tc::fence_after_sync();
        // a part whose scores are all -inf has no sum: no weight in the join, so its zeros must not turn NaN
        const float inv = g.splits > 1 && lm.x == 0.0f ? 0.0f : 1.0f / lm.x;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t v[32];
          tc::tmem_ld32(lane_base + col_o(x) + c0, v);
          tc::tmem_wait_ld16(v);
          tc::tmem_wait_ld16(v + 16);
          if (c0 + 32 == D) warp_arrive(&bars->o_free[x], lane);        // statistics and O are read
          if (g.splits > 1) {
            if (on) {
              float4* o = reinterpret_cast<float4*>(g.part_o + part * D + c0);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                o[k] = make_float4(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv,
                                   __uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv);
            }
            continue;
          }
          uint8_t* at = box + (c0 >> 6) * 16384 + r * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = pack16<T>(__uint_as_float(v[8 * k + 2 * e]) * inv, __uint_as_float(v[8 * k + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(at + (((k + (c0 >> 3)) ^ r) & 7) * 16) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        if (g.splits == 1) {
          tc::fence_proxy_async_smem();
          asm volatile("bar.sync 2, 128;" ::: "memory");
          if (lead) {
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 64)
              tc::tma_store_4d(&maps.out, box + (c0 >> 6) * 16384, c0, w.row0 + 128 * x, w.h, w.b);
            tc::bulk_commit();
          }
        }
        if (on) {
          const float lse2 = lm.y + log2f(lm.x);
          if (g.splits > 1) g.part_lse[part] = lse2;
          else if (g.lse) g.lse[flat] = lse2 * kLn2;
        }
      }
    }
    if (lead) tc::bulk_wait_all();
  }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bars->tmem, 512);
  }
}

// Joins the parts of split keys: out = sum_s 2^(lse_s - max) o_s / sum_s 2^(lse_s - max), one warp
// per row. No part with weight: zero without a valid key, NaN where every valid score is -inf or NaN (as
// one part alone has it).
template <typename T, int D>
__global__ void __launch_bounds__(128) k_cross_join(const __grid_constant__ CrossArgs g) {
  const size_t rows = (size_t)g.B * g.H * g.Tq;
  const size_t row = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float m = -INFINITY, none = 0.0f;                      // none: -inf, or NaN, without a part of weight
  for (int s = 0; s < g.splits; ++s) {
    const float l = g.part_lse[s * rows + row];
    m = fmaxf(m, l);
    none += l;
  }
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
  const size_t bh = row / g.Tq;
  const int t = (int)(row - bh * g.Tq), b = (int)(bh / g.H), h = (int)(bh - (size_t)b * g.H);
  const float inv = m == -INFINITY ? (valid_keys(g, b) > 0 ? NAN : 0.0f) : 1.0f / total;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(g.out.data) + b * g.out.sb + h * g.out.sh +
                                              t * g.out.st + lane * (D / 32));
#pragma unroll
  for (int e = 0; e < D / 64; ++e) out[e] = pack16<T>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (g.lse && lane == 0) g.lse[row] = m == -INFINITY ? none : (m + log2f(total)) * kLn2;
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
