// Gradients of the attention to an encoder's states.
//
//   p = 2^(s log2e - lse2),  D = sum_c dout out,  dS = p (dout v^T - D)
//   dq = scale dS k,  dk = scale dS^T q,  dv = p^T dout
//
// Two kernels without atomics, so that equal inputs give equal bits: k_cross_dq holds one query
// tile and walks the keys; k_cross_dkv holds one key tile and walks the queries. Each recomputes
// S and dP, which makes seven products of five; accumulating dq over key tiles in memory instead
// would move 8 bytes per element and key tile, more time than the two products.
// Measured (40 heads, d = 128, bf16, 32760 queries, 512 keys): 1230 us for both in 20 calls at 1965 MHz, 700
// TFLOP/s of the five products that the gradients cannot do without, 980 of the seven; 1400 us in a second
// and a half of calls, where the power cap leaves about 1570 MHz. Bound now by each step's chain of
// reading S and dP, the exponentials, and handing P and dS back to the tensor cores, and in dq by the
// change of query tiles (about 5000 cycles against 2000 a step of 1540 of MMA time).
//
// p and dS are rounded once to the 16-bit type as MMA operands (fp32 accumulators). In fp16 both
// carry a power of two, taken out of the accumulators: with many keys they fall below fp16's smallest
// normal 2^-14 otherwise. p <= 1 carries 2^6. |dS| <= |dP| + |D| <= 2 |dout row| |v row| by Cauchy and
// Schwarz, and D of a rounded out stays within 1 % of that; so dS carries 2^(13 - E), 2^E <= the bound
// |dout row| max |v row| < 2^(E+1), and stays below 33100 whatever dout's size (a fixed 2^6 overflowed at
// |dS| = 1024). In dq each query row has its own power; in dk, whose sums run over the queries, all query
// rows of a key/value head share the smallest. k_cross_vnorm leaves the value rows' largest norm of
// each key tile, k_cross_dq the dout rows' of each query tile.
#include <type_traits>

#include "cross.cuh"
#include "f32x2.cuh"

namespace da2 {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 11;             // warps 8 to 10 issue MMAs (dq), warp 8 (dk, dv)

template <typename T>
struct Scale {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr float kLog2 = kBf16 ? 0.0f : 6.0f;      // of p
  static constexpr float kInv = kBf16 ? 1.0f : 1.0f / 64.0f;
};

__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }
// Largest of a warp's squared norms: non-negative floats compare like their bits, NaN above all.
__device__ __forceinline__ float warp_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}
// The exponent of dS in fp16: 13 - E, from the squared norms of the dout row and the largest value row.
// E is kept above -40 (gradients that small are zero in fp16); an infinite or NaN norm, whose row's
// gradients are not finite, gives E = 64.
__device__ __forceinline__ int ds_exponent(float dout2, float v2) {
  const int e = (int)(__float_as_uint(dout2 * v2) >> 23 & 0xFF) - 127;
  return 13 - max(e >> 1, -40);
}
// A lane's share of the largest squared norm of a value row among the valid key tiles of one key/value
// head (warp_max joins the lanes), and the same of dout over every query tile of the query heads that
// share the head, four parts per tile.
__device__ __forceinline__ float value_norm2(const CrossArgs& g, int b, int hkv, int tiles, int lane) {
  const float* at = g.vnorm2 + ((size_t)b * g.Hkv + hkv) * g.k_tiles;
  float m = 0.0f;
#pragma unroll 1
  for (int t = lane; t < tiles; t += 32) m = fmaxf(m, at[t]);
  return m;
}
__device__ __forceinline__ float dout_norm2(const CrossArgs& g, int b, int hkv, int lane) {
  const float4* at = reinterpret_cast<const float4*>(g.dnorm2) + ((size_t)b * g.H + (size_t)hkv * g.group) * g.q_tiles;
  const int n = g.group * g.q_tiles;
  float m = 0.0f;
#pragma unroll 4
  for (int t = lane; t < n; t += 32) {
    const float4 x = at[t];
    m = fmaxf(m, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
  }
  return m;
}

// Squared norms of the value rows, the largest of each key tile's valid rows (fp16 only). D / 8 lanes
// share a row.
template <int D>
__global__ void __launch_bounds__(256) k_cross_vnorm(const __grid_constant__ CrossArgs g) {
  __shared__ float red[8];
  constexpr int G = D / 8;
  asm volatile("griddepcontrol.launch_dependents;");     // k_cross_dq may start; it waits before it reads
  const int kt = blockIdx.x % g.k_tiles, bh = blockIdx.x / g.k_tiles, b = bh / g.Hkv, hkv = bh - b * g.Hkv;
  const int end = min(valid_keys(g, b), 128 * (kt + 1)), c = threadIdx.x % G;
  const __half* v = static_cast<const __half*>(g.v.data) + b * g.v.sb + hkv * g.v.sh + 8 * c;
  float m = 0.0f;
#pragma unroll
  for (int r = 0; r < 128; r += 256 / G) {
    const int key = 128 * kt + r + threadIdx.x / G;
    float n2 = 0.0f;
    if (key < g.Tk) {                                    // before the length is known: one latency, not two
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(v + key * g.v.st));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = unpack16<__half>(w[e]);
        n2 = fmaf(x.x, x.x, fmaf(x.y, x.y, n2));
      }
    }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
    if (key < end) m = fmaxf(m, n2);
  }
  m = warp_max(m);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
    g.vnorm2[blockIdx.x] = m;
  }
}

__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t* v) {
  tc::tmem_ld32(taddr, v);
  tc::tmem_ld32(taddr + 32, v + 32);
#pragma unroll
  for (int k = 0; k < 64; k += 16) tc::tmem_wait_ld16(v + k);
}
// 32 consecutive elements of a row, rounded and stored.
template <typename T>
__device__ __forceinline__ void store32(T* dst, const uint32_t* v, float f) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[e] = pack16<T>(__uint_as_float(v[8 * k + 2 * e]) * f, __uint_as_float(v[8 * k + 2 * e + 1]) * f);
    reinterpret_cast<uint4*>(dst)[k] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// ------------------------------------------------------------------------------------ dq
// A work item is one 128-row query tile; Q and dout stay in shared memory, key and value tiles
// come through a ring. 8 softmax warps share each 128 x 128 step: thread (w, r) owns row r and the
// keys 64 w .. 64 w + 63. S and dP of the next step are multiplied as soon as this step's have been
// read into registers. D comes from dout and out, both in shared memory; when one key tile holds every
// key it is sum p dP instead, exact where a row's out is largest against its rounding, and out is not
// read. D and lse in the log2 domain are left in the workspace, padded to whole tiles, for k_cross_dkv.
// dq leaves through out's buffer and a tensor-map store.
template <int D>
struct SmemDq {
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kDo = kTile, kO = 2 * kTile, kStage0 = 3 * kTile;
  static constexpr uint32_t kExch = kStage0 + kStages * kTile;      // [D, norm][2 halves][128] fp32
  static constexpr uint32_t kBars = kExch + 2048;
  static constexpr uint32_t kBytes = kBars + 384;
  static_assert(kBytes <= 232448, "shared memory budget");
};
template <int D>
struct BarsDq {
  uint64_t kv_full[SmemDq<D>::kStages], kv_empty[SmemDq<D>::kStages];
  uint64_t q_full, q_empty, o_full, o_empty, s_full, s_free, dp_full, dp_free, ds_full[2], ds_free[2], dq_full, dq_free;
  uint64_t done;
  uint32_t tmem, abort;
};
static_assert(sizeof(BarsDq<64>) <= 384, "barrier area");

constexpr uint32_t kDqS = 0, kDqP = 128, kDqAcc = 256, kDqDs = 384;   // columns; dS: two of 64

struct ItemDq {
  int b, h, qt, nt, len;
  __device__ __forceinline__ ItemDq(const CrossArgs& g, int i) {
    int v[5];
    decode(g, i, v);
    b = v[0], h = v[1], qt = v[2], nt = v[3], len = v[4];
  }
  // not inline: its divisions in each of the kernel's roles would crowd the instruction cache
  static __device__ __noinline__ void decode(const CrossArgs& g, uint32_t u, int* v) {
    int b, h, qt;
    const uint32_t bh = u / g.q_tiles;
    qt = u - bh * g.q_tiles;
    b = bh / g.H;
    h = bh - b * g.H;
    const int len = valid_keys(g, b);
    v[0] = b, v[1] = h, v[2] = qt, v[3] = (len + 127) >> 7, v[4] = len;
  }
  __device__ __forceinline__ int keys(int t) const { return min(128, len - 128 * t); }
  __device__ __forceinline__ bool dirty(const CrossArgs& g, int t) const {
    return (keys(t) & 15) != 0 && len < g.Tk;
  }
};

// The S and dP products, each A (128 rows) x 128 rows of a tile over d channels, and the accumulating
// product of a 16-bit operand in tensor memory with a tile read by columns. Executed by one lane; the
// operands are the same in all lanes of the issuing warp and stay in uniform registers.
constexpr uint32_t kDescHi = (uint32_t)(tc::kSw128 >> 32) | (1024 >> 4);
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t acc, uint32_t a, uint32_t b, uint32_t id) {
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = (k / 4) * (16384 >> 4) + (k % 4) * (32 >> 4);
    tc::mma_f16(acc, tc::desc((a + off) | 1u << 16, kDescHi), tc::desc((b + off) | 1u << 16, kDescHi), id, k > 0);
  }
}

// Live key tiles in front of each batch entry, and their number. A full warp.
__device__ __noinline__ void count_tiles(const CrossArgs& g, int lane) {
  int before = 0;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const int b = b0 + lane, n = b < g.B ? (valid_keys(g, b) + 127) >> 7 : 0;
    int sum = n;                                         // of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (b < g.B) g.first[b] = before + sum - n;
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) g.first[g.B] = before;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_dq(const __grid_constant__ CrossMaps maps, const __grid_constant__ CrossArgs g) {
  using S = SmemDq<D>;
  constexpr int kStages = S::kStages;
  constexpr bool kBf16 = Scale<T>::kBf16;
  extern __shared__ __align__(1024) uint8_t sm[];
  BarsDq<D>* bars = reinterpret_cast<BarsDq<D>*>(sm + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = g.B * g.H * g.q_tiles;
  const Guard gd{g.err, &bars->abort, g.wait_clocks};
  if (tc::smem_u32(sm) & 1023u) {        // the swizzle needs the alignment that the declaration asks for
    if (tid == 0) set_error(g.err, kErrBadIndex);
    if (blockIdx.x == 0 && warp == 0) count_tiles(g, lane);      // k_cross_dkv indexes by it
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 1);
    }
    tc::mbar_init(&bars->q_full, 1);
    tc::mbar_init(&bars->q_empty, 2 + 8);                // S and dP, and the warps that read dout
    tc::mbar_init(&bars->o_full, 1);
    tc::mbar_init(&bars->o_empty, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->s_free, 8);
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->dp_free, 8);
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(&bars->ds_full[x], 8);
      tc::mbar_init(&bars->ds_free[x], 1);
    }
    tc::mbar_init(&bars->dq_full, 1);
    tc::mbar_init(&bars->dq_free, 8);
    tc::mbar_init(&bars->done, 3);
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

  if (warp == kLoadWarp) {
    if (lane == 0) {
      uint32_t n = 0, q_loads = 0, o_loads = 0;
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
        const ItemDq w(g, i);
        if (w.nt == 0) continue;
        if (!guard_wait(&bars->q_empty, (q_loads & 1) ^ 1, gd)) break;
        tc::mbar_arrive_expect_tx(&bars->q_full, 2 * S::kTile);
        load_tile<D>(sm, &maps.q, 128 * w.qt, w.h, w.b, &bars->q_full);
        load_tile<D>(sm + S::kDo, &maps.dout, 128 * w.qt, w.h, w.b, &bars->q_full);
        ++q_loads;
        for (int t = 0; t < w.nt && !dead; ++t) {
          dead = !load(&maps.k, 128 * t, w.h / g.group, w.b);
          if (!dead) dead = !load(&maps.v, 128 * t, w.h / g.group, w.b);
          // out, once the dq of the item before has left its buffer: behind the first step's tiles, which
          // do not wait for that
          if (t == 0 && w.nt > 1 && !dead) {
            if (q_loads > 1) dead = !guard_wait(&bars->o_empty, (q_loads - 2) & 1, gd);
            if (dead) break;
            tc::mbar_arrive_expect_tx(&bars->o_full, S::kTile);
            load_tile<D>(sm + S::kO, &maps.out, 128 * w.qt, w.h, w.b, &bars->o_full);
            ++o_loads;
          }
        }
      }
#pragma unroll 1
      for (uint32_t s = 0; s < (uint32_t)kStages && s < n; ++s)
        guard_wait(&bars->kv_full[s], ((n - 1 - s) / kStages) & 1, gd, false);
      if (q_loads) guard_wait(&bars->q_full, (q_loads - 1) & 1, gd, false);
      if (o_loads) guard_wait(&bars->o_full, (o_loads - 1) & 1, gd, false);
    }
  } else if (warp >= kMmaWarp) {
    // Three issuing warps, one per product: a warp's waits stand behind the MMAs it has issued, so that
    // one warp for all three adds their times to its own. The whole warp runs the loop, one lane issues.
    const int role = warp - kMmaWarp;      // 0: S, 1: dP, 2: dq
    const bool lead = tc::elect_one();
    const uint32_t sm0 = tc::smem_u32(sm) >> 4, stage0 = sm0 + (S::kStage0 >> 4);
    uint32_t step = 0, n_items = 0;
    bool dead = false;
    if (role == 2 && blockIdx.x == 0) count_tiles(g, lane);      // the role that waits longest at first
    for (int i = blockIdx.x; i < items && !dead; i += gridDim.x) {
      const ItemDq w(g, i);
      for (int t = 0; t < w.nt && !dead; ++t, ++step) {
        const uint32_t n = 2 * step + (role == 1 ? 1 : 0), s = n % kStages, tile = stage0 + s * (S::kTile >> 4);
        const int keys = w.keys(t);
        const bool last = t == w.nt - 1;
        dead = !warp_wait(&bars->kv_full[s], (n / kStages) & 1, gd);
        if (role < 2) {
          if (t == 0) dead = dead || !warp_wait(&bars->q_full, n_items & 1, gd);
          if (step > 0) dead = dead || !warp_wait(role ? &bars->dp_free : &bars->s_free, (step - 1) & 1, gd);
          if (dead) break;
          tc::fence_after_sync();
          const uint32_t id = tc::idesc_f16(kBf16, 128, (keys + 15) & ~15, false);
          if (lead) {
            if (role == 0) {
              mma_rows<D>(tmem + kDqS, sm0, tile, id);
              tc::mma_commit(&bars->s_full);
            } else {
              mma_rows<D>(tmem + kDqP, sm0 + (S::kDo >> 4), tile, id);
              tc::mma_commit(&bars->dp_full);
              tc::mma_commit(&bars->kv_empty[s]);
            }
            if (last) tc::mma_commit(&bars->q_empty);
          }
        } else {
          // Key rows behind the length, up to the last group of 16, may hold anything, and 0 times NaN
          // would reach the sum: zeroed (S, which may be reading them, masks its columns).
          if (last && w.dirty(g, t)) zero_rows<D>(sm + S::kStage0 + s * S::kTile, keys, (keys + 15) & ~15, lane);
          const uint32_t buf = step & 1;
          dead = dead || !warp_wait(&bars->ds_full[buf], (step >> 1) & 1, gd);
          if (t == 0 && n_items > 0) dead = dead || !warp_wait(&bars->dq_free, (n_items - 1) & 1, gd);
          if (dead) break;
          tc::fence_after_sync();
          const uint32_t b = tile | (16384 >> 4) << 16;
          constexpr uint32_t id = tc::idesc_f16(kBf16, 128, D, true);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (16 * k < keys)
                tc::mma_f16_ta(tmem + kDqAcc, tmem + kDqDs + 64 * buf + 8 * k, tc::desc(b + k * (2048 >> 4), kDescHi),
                               id, k > 0 ? 1u : t > 0);
            tc::mma_commit(&bars->kv_empty[s]);
            tc::mma_commit(&bars->ds_free[buf]);
            if (last) tc::mma_commit(&bars->dq_full);
          }
        }
        __syncwarp();
      }
      n_items += w.nt > 0;
    }
    if (lead) tc::mma_commit(&bars->done);
    __syncwarp();
    guard_wait(&bars->done, 0, gd, false);           // all issuers' MMAs retired before TMEM is freed
  } else if (warp < kMmaWarp) {
    const int half = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = g.scale_log2;
    const bool lead = tid == 0;
    uint32_t step = 0, n_items = 0, o_items = 0;
    float v2 = 0.0f;                       // the next item's value norm, read ahead
    auto ahead = [&](int i) {
      if constexpr (!kBf16) {
        if (i < items) {
          const ItemDq w(g, i);
          v2 = value_norm2(g, w.b, w.h / g.group, w.nt, lane);
        }
      }
    };
    if constexpr (!kBf16) asm volatile("griddepcontrol.wait;" ::: "memory");     // for k_cross_vnorm
    ahead(blockIdx.x);
    // no wait ends this loop early: all 256 threads must meet at the named barrier
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const ItemDq w(g, i);
      const int row = 128 * w.qt + r;
      const bool on = row < g.Tq;
      T* dq = static_cast<T*>(g.dq.data) + w.b * g.dq.sb + w.h * g.dq.sh + row * g.dq.st + half * (D / 2);
      if (w.nt == 0) {
        if (on)
          for (int k = 0; k < D / 16; ++k) reinterpret_cast<uint4*>(dq)[k] = make_uint4(0u, 0u, 0u, 0u);
        ahead(i + gridDim.x);
        continue;
      }
      const size_t bh = (size_t)w.b * g.H + w.h;
      const float lse2 = on ? g.lse_in[bh * g.Tq + row] * kLog2E : INFINITY;
      float* exch = reinterpret_cast<float*>(sm + S::kExch);
      // the two halves' parts of D, and of the norm of dout's row in fp16, meet; left for k_cross_dkv
      int ex = 0;                                        // of dS
      float n2 = 0.0f;
      auto join = [&](float part) {
        exch[half * 128 + r] = part;
        if constexpr (!kBf16) exch[256 + half * 128 + r] = n2;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float d = exch[r] + exch[128 + r];
        if (half == 0) {
          const size_t at = bh * (128 * (size_t)g.q_tiles) + row;
          g.lse2[at] = lse2;
          g.delta[at] = d;
        }
        if constexpr (!kBf16) {
          n2 = exch[256 + r] + exch[384 + r];
          ex = ds_exponent(n2, v2);
          const float tile2 = warp_max(n2);
          if (half == 0 && lane == 0) g.dnorm2[(bh * g.q_tiles + w.qt) * 4 + warp] = tile2;
        }
        return d;
      };
      // Also where the rows are not read here: q_full of this item completes only behind the item
      // before's phase of q_empty, so that no arrival below can count into that phase.
      guard_wait(&bars->q_full, n_items & 1, gd);
      float delta = 0.0f;
      if constexpr (!kBf16) {
        v2 = warp_max(v2);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int ch = half * (D / 16) + k;            // 16-byte chunk of the row, swizzled
          const uint4 u = *reinterpret_cast<const uint4*>(sm + S::kDo + (ch >> 3) * 16384 + r * 128 +
                                                          (((ch & 7) ^ (r & 7)) << 4));
          const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack16<T>(a[e]);
            n2 = fmaf(x.x, x.x, fmaf(x.y, x.y, n2));
          }
        }
      }
      if (w.nt > 1) {                                    // this thread's half of the rows of dout and out
        guard_wait(&bars->o_full, o_items++ & 1, gd);
        float part = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int ch = half * (D / 16) + k;
          const uint32_t at = (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
          const uint4 u = *reinterpret_cast<const uint4*>(sm + S::kDo + at);
          const uint4 v = *reinterpret_cast<const uint4*>(sm + S::kO + at);
          const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack16<T>(a[e]), y = unpack16<T>(b[e]);
            part = fmaf(x.x, y.x, fmaf(x.y, y.y, part));
          }
        }
        delta = join(part);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->q_empty);
      const f32x2 c2 = pk2(c, c), b2 = pk2(-lse2, -lse2);
      for (int t = 0; t < w.nt; ++t, ++step) {
        const int keys = w.keys(t) - 64 * half;          // of this thread's 64
        guard_wait(&bars->s_full, step & 1, gd);
        tc::fence_after_sync();
        uint32_t su[64], pu[64];
        float* s = reinterpret_cast<float*>(su);
        float* p = reinterpret_cast<float*>(pu);
        tmem_ld64(lane_base + kDqS + 64 * half, su);
        warp_arrive(&bars->s_free, lane);
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          float x, y;
          upk2(fma2(pk2(s[k], s[k + 1]), c2, b2), x, y);
          s[k] = ex2(x);
          s[k + 1] = ex2(y);
        }
        guard_wait(&bars->dp_full, step & 1, gd);
        tc::fence_after_sync();
        tmem_ld64(lane_base + kDqP + 64 * half, pu);
        warp_arrive(&bars->dp_free, lane);
        if (keys < 64) {                                 // also NaN from behind the length
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (k >= keys) s[k] = p[k] = 0.0f;
        }
        if (w.nt == 1) {
          f32x2 sum = pk2(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < 64; k += 2) sum = fma2(pk2(s[k], s[k + 1]), pk2(p[k], p[k + 1]), sum);
          float x, y;
          upk2(sum, x, y);
          delta = join(x + y);
        }
        const f32x2 f2 = pk2(pow2(ex), pow2(ex)), d2 = pk2(-delta * pow2(ex), -delta * pow2(ex));
        uint32_t ds[32];
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          const f32x2 dp = pk2(p[k], p[k + 1]);
          float x, y;
          upk2(mul2(kBf16 ? add2(dp, d2) : fma2(dp, f2, d2), pk2(s[k], s[k + 1])), x, y);
          ds[k >> 1] = pack16<T>(x, y);
        }
        if (step >= 2) {
          guard_wait(&bars->ds_free[step & 1], ((step >> 1) - 1) & 1, gd);
          tc::fence_after_sync();
        }
        tc::tmem_st16(lane_base + kDqDs + 64 * (step & 1) + 32 * half, ds);
        tc::tmem_st16(lane_base + kDqDs + 64 * (step & 1) + 32 * half + 16, ds + 16);
        tc::tmem_wait_st();
        warp_arrive(&bars->ds_full[step & 1], lane);
      }
      ahead(i + gridDim.x);
      guard_wait(&bars->dq_full, n_items & 1, gd);
      tc::fence_after_sync();
#pragma unroll
      for (int c0 = 0; c0 < D / 2; c0 += 32) {
        uint32_t v[32];
        tc::tmem_ld32(lane_base + kDqAcc + half * (D / 2) + c0, v);
        tc::tmem_wait_ld16(v);
        tc::tmem_wait_ld16(v + 16);
        if (c0 + 32 == D / 2) warp_arrive(&bars->dq_free, lane);
        const float f = g.scale * pow2(-ex);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int ch = half * (D / 16) + c0 / 8 + k;
          uint32_t u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            u[e] = pack16<T>(__uint_as_float(v[8 * k + 2 * e]) * f, __uint_as_float(v[8 * k + 2 * e + 1]) * f);
          *reinterpret_cast<uint4*>(sm + S::kO + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
              make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
      tc::fence_proxy_async_smem();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (lead) {
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 64)
          tc::tma_store_4d(&maps.dq, sm + S::kO + (c0 >> 6) * 16384, c0, 128 * w.qt, w.h, w.b);
        tc::bulk_commit();
        tc::bulk_wait_read<0>();
        tc::mbar_arrive(&bars->o_empty);
      }
      ++n_items;
    }
    if (lead) tc::bulk_wait_all();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bars->tmem, 512);
  }
}

// ------------------------------------------------------------------------------------ dk, dv
// A group is one key tile of one key/value head; its units are the query tiles of all query heads
// that share the head. The groups with a valid key, laid end to end, are cut into one run of units
// per block: a run that covers a group writes dk and dv, the ends of a group that blocks share go
// to the workspace as fp32 parts, two per block at most, and k_cross_dkv_join adds them in order.
// Transposed products: S^T = K Q^T and dP^T = V dout^T (key rows in the tensor-memory lanes), P^T
// and dS^T overwrite them as 16-bit A operands of dv += P^T dout and dk += dS^T Q, each next S and dP
// issued directly behind. Key rows behind the length only reach their own rows of dk and dv, which
// are written as zero.
template <int D>
struct SmemDkv {
  static constexpr uint32_t kTile = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;       // even: dout behind Q
  static constexpr uint32_t kV = kTile, kStage0 = 2 * kTile;
  static constexpr uint32_t kVec = kStage0 + kStages * kTile;       // per Q stage: lse2[128], delta[128]
  static constexpr uint32_t kBars = kVec + kStages / 2 * 1024;
  static constexpr uint32_t kBytes = kBars + 512 + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};
template <int D>
struct BarsDkv {
  uint64_t q_full[SmemDkv<D>::kStages], q_empty[SmemDkv<D>::kStages];
  uint64_t kv_full, kv_empty, s_full, p_full, dp_full, ds_full, acc_full, acc_free, done;
  uint32_t tmem, abort;
};
static_assert(sizeof(BarsDkv<64>) <= 512, "barrier area");

constexpr uint32_t kKvS = 0, kKvP = 128, kKvDv = 256, kKvDk = 384;    // columns

// The live groups, numbered by batch entry, key/value head and key tile, and how the blocks share them.
// first[b] (left by k_cross_dq) counts the live key tiles in front of batch entry b, of one head.
struct Share {
  long units;                 // of all live groups
  int n;                      // units per group
  int blocks;
  __device__ __forceinline__ Share(const CrossArgs& g) {
    n = g.group * g.q_tiles;
    units = (long)g.first[g.B] * g.Hkv * n;
    blocks = g.sms;
  }
  __device__ __forceinline__ long begin(int c) const { return units * c / blocks; }
};
// Live group i: batch entry, key/value head, key tile. The entry by bisection, so that long batches of
// short sequences do not walk the batch for every group.
struct Group {
  int b, hkv, kt, len;
  __device__ __forceinline__ Group(const CrossArgs& g, uint32_t i) {
    const int t = i / (uint32_t)g.Hkv;
    int lo = 0, hi = g.B;                                // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.first[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    const uint32_t tiles = g.first[lo + 1] - g.first[lo], rest = i - (uint32_t)g.first[lo] * g.Hkv;
    hkv = rest / tiles;
    kt = rest - hkv * tiles;
    len = valid_keys(g, b);
  }
};
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_dkv(const __grid_constant__ CrossMaps maps, const __grid_constant__ CrossArgs g) {
  using S = SmemDkv<D>;
  constexpr int kStages = S::kStages;
  constexpr bool kBf16 = Scale<T>::kBf16;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  BarsDkv<D>* bars = reinterpret_cast<BarsDkv<D>*>(sm + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Guard gd{g.err, &bars->abort, g.wait_clocks};

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->q_full[s], 1);
      tc::mbar_init(&bars->q_empty[s], 1);
    }
    tc::mbar_init(&bars->kv_full, 1);
    tc::mbar_init(&bars->kv_empty, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->p_full, 8);
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->ds_full, 8);
    tc::mbar_init(&bars->acc_full, 1);
    tc::mbar_init(&bars->acc_free, 8);
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
  constexpr uint32_t tmem = 0;             // all 512 columns are this block's: the base is column 0
  const Share sh(g);
  const long u0 = sh.begin(blockIdx.x), u1 = sh.begin(blockIdx.x + 1);

  if (warp == kLoadWarp) {
    if (lane == 0) {
      uint32_t n = 0, groups = 0;
      bool dead = false;
      for (long u = u0; u < u1 && !dead;) {
        const long gi = u / sh.n;
        const Group w(g, gi);
        const int e = (int)(min(u1, (gi + 1) * sh.n) - gi * sh.n);
        if (!guard_wait(&bars->kv_empty, (groups & 1) ^ 1, gd)) break;
        tc::mbar_arrive_expect_tx(&bars->kv_full, 2 * S::kTile);
        load_tile<D>(sm, &maps.k, 128 * w.kt, w.hkv, w.b, &bars->kv_full);
        load_tile<D>(sm + S::kV, &maps.v, 128 * w.kt, w.hkv, w.b, &bars->kv_full);
        ++groups;
        for (int i = (int)(u - gi * sh.n); i < e && !dead; ++i) {
          const int h = w.hkv * g.group + i / g.q_tiles, qt = i % g.q_tiles;
          for (int x = 0; x < 2; ++x) {                  // Q with its two vectors, then dout
            const uint32_t s = n % kStages;
            if (g.stall && n == 0) { ++n; continue; }
            if (!guard_wait(&bars->q_empty[s], ((n / kStages) & 1) ^ 1, gd)) { dead = true; break; }
            tc::mbar_arrive_expect_tx(&bars->q_full[s], S::kTile + (x == 0 ? 1024 : 0));
            load_tile<D>(sm + S::kStage0 + s * S::kTile, x == 0 ? &maps.q : &maps.dout, 128 * qt, h, w.b,
                         &bars->q_full[s]);
            if (x == 0) {
              const size_t at = (((size_t)w.b * g.H + h) * g.q_tiles + qt) * 128;
              uint8_t* vec = sm + S::kVec + s / 2 * 1024;
              tc::bulk_g2s(vec, g.lse2 + at, 512, &bars->q_full[s]);
              tc::bulk_g2s(vec + 512, g.delta + at, 512, &bars->q_full[s]);
            }
            ++n;
          }
        }
        u = gi * sh.n + e;
      }
#pragma unroll 1
      for (uint32_t s = 0; s < (uint32_t)kStages && s < n; ++s)
        guard_wait(&bars->q_full[s], ((n - 1 - s) / kStages) & 1, gd, false);
      if (groups) guard_wait(&bars->kv_full, (groups - 1) & 1, gd, false);
    }
  } else if (warp == kMmaWarp) {
    if (u0 < u1) {
      // the whole warp runs this, one lane issues
      const bool lead = tc::elect_one();
      const uint32_t sm0 = tc::smem_u32(sm) >> 4, stage0 = sm0 + (S::kStage0 >> 4);
      constexpr uint32_t id_s = tc::idesc_f16(kBf16, 128, 128, false), id_o = tc::idesc_f16(kBf16, 128, D, true);
      uint32_t groups = 0, accs = 0;
      // acc += A^T tile, A the 16-bit operand in the two 32-column halves behind col and col + 64
      auto accumulate = [&](uint32_t acc, uint32_t col, uint32_t stage, bool first) {
        const uint32_t b = (stage0 + stage * (S::kTile >> 4)) | (16384 >> 4) << 16;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc::mma_f16_ta(tmem + acc, tmem + col + 64 * (k >> 2) + 8 * (k & 3), tc::desc(b + k * (2048 >> 4), kDescHi),
                         id_o, k > 0 ? 1u : !first);
      };
      auto issue_s = [&](bool new_group, uint32_t gs) -> bool {
        if (new_group && !warp_wait(&bars->kv_full, groups++ & 1, gd)) return false;
        const uint32_t s = 2 * gs % kStages;
        if (!warp_wait(&bars->q_full[s], (2 * gs / kStages) & 1, gd)) return false;
        tc::fence_after_sync();
        if (lead) {
          mma_rows<D>(tmem + kKvS, sm0, stage0 + s * (S::kTile >> 4), id_s);
          tc::mma_commit(&bars->s_full);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](bool last_of_group, uint32_t gs) -> bool {
        const uint32_t n = 2 * gs + 1, s = n % kStages;
        if (!warp_wait(&bars->q_full[s], (n / kStages) & 1, gd)) return false;
        tc::fence_after_sync();
        if (lead) {
          mma_rows<D>(tmem + kKvP, sm0 + (S::kV >> 4), stage0 + s * (S::kTile >> 4), id_s);
          tc::mma_commit(&bars->dp_full);
          if (last_of_group) tc::mma_commit(&bars->kv_empty);
        }
        __syncwarp();
        return true;
      };
      // runs of units within a group: what is left of this run and the next
      const int n = sh.n;
      int left = (int)min((long)(n - u0 % n), u1 - u0);
      bool dead = !issue_s(true, 0) || !issue_dp(left == 1, 0);
      bool first = true;
      uint32_t step = 0;
      for (long todo = u1 - u0; todo > 0 && !dead; --todo, ++step) {
        const bool last = left == 1, more = todo > 1;
        const int left1 = last ? (int)min((long)n, todo - 1) : left - 1;      // of the next unit's run
        dead = !warp_wait(&bars->p_full, step & 1, gd);
        if (!dead && first && accs > 0) dead = !warp_wait(&bars->acc_free, (accs - 1) & 1, gd);
        if (dead) break;
        tc::fence_after_sync();
        if (lead) {
          accumulate(kKvDv, kKvS, (2 * step + 1) % kStages, first);
          tc::mma_commit(&bars->q_empty[(2 * step + 1) % kStages]);
        }
        __syncwarp();
        if (more && !issue_s(last, step + 1)) break;
        if (!warp_wait(&bars->ds_full, step & 1, gd)) break;
        tc::fence_after_sync();
        if (lead) {
          accumulate(kKvDk, kKvP, (2 * step) % kStages, first);
          tc::mma_commit(&bars->q_empty[(2 * step) % kStages]);
          if (last) tc::mma_commit(&bars->acc_full);
        }
        __syncwarp();
        accs += last;
        if (more && !issue_dp(left1 == 1, step + 1)) break;
        first = last;
        left = left1;
      }
      if (lead) tc::mma_commit(&bars->done);
      __syncwarp();
      guard_wait(&bars->done, 0, gd, false);
    }
  } else if (warp < kMmaWarp) {
    const int half = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const f32x2 c2 = pk2(g.scale_log2, g.scale_log2);
    const f32x2 k2 = pk2(Scale<T>::kLog2, Scale<T>::kLog2);
    uint32_t step = 0, accs = 0;
    bool dead = false;
    for (long u = u0; u < u1 && !dead; ++accs) {
      const long gi = u / sh.n;
      const long end = min(u1, (gi + 1) * sh.n);
      const bool whole = u == gi * sh.n && end == (gi + 1) * sh.n;
      const int slot = 2 * blockIdx.x + (u == u0 ? 0 : 1);
      int ex = 0;                                        // of dS
      if constexpr (!kBf16) {
        const Group w(g, gi);
        const float v2 = value_norm2(g, w.b, w.hkv, (w.len + 127) >> 7, lane);
        ex = ds_exponent(warp_max(dout_norm2(g, w.b, w.hkv, lane)), warp_max(v2));
      }
      // p carries 2^kLog2 already
      const f32x2 f2 = pk2(pow2(ex) * Scale<T>::kInv, pow2(ex) * Scale<T>::kInv);
      for (; u < end; ++u, ++step) {
        const uint32_t n = 2 * step, st = n % kStages;
        const float4* vec = reinterpret_cast<const float4*>(sm + S::kVec + st / 2 * 1024 + half * 256);
        guard_wait(&bars->q_full[st], (n / kStages) & 1, gd);      // the two vectors
        guard_wait(&bars->s_full, step & 1, gd);
        tc::fence_after_sync();
        uint32_t su[64];
        float* s = reinterpret_cast<float*>(su);
        tmem_ld64(lane_base + kKvS + 64 * half, su);
        uint32_t w16[32];
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          const float4 l = vec[k / 4];
          float x0, x1, x2, x3;
          upk2(fma2(pk2(s[k], s[k + 1]), c2, add2(k2, pk2(-l.x, -l.y))), x0, x1);
          upk2(fma2(pk2(s[k + 2], s[k + 3]), c2, add2(k2, pk2(-l.z, -l.w))), x2, x3);
          s[k] = ex2(x0);
          s[k + 1] = ex2(x1);
          s[k + 2] = ex2(x2);
          s[k + 3] = ex2(x3);
          w16[k / 2] = pack16<T>(s[k], s[k + 1]);
          w16[k / 2 + 1] = pack16<T>(s[k + 2], s[k + 3]);
        }
        tc::tmem_st16(lane_base + kKvS + 64 * half, w16);
        tc::tmem_st16(lane_base + kKvS + 64 * half + 16, w16 + 16);
        tc::tmem_wait_st();
        warp_arrive(&bars->p_full, lane);
        guard_wait(&bars->dp_full, step & 1, gd);
        tc::fence_after_sync();
        uint32_t pu[64];
        float* p = reinterpret_cast<float*>(pu);
        tmem_ld64(lane_base + kKvP + 64 * half, pu);
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          const float4 d = vec[32 + k / 4];
          f32x2 a = add2(pk2(p[k], p[k + 1]), pk2(-d.x, -d.y)), b = add2(pk2(p[k + 2], p[k + 3]), pk2(-d.z, -d.w));
          if constexpr (!kBf16) a = mul2(a, f2), b = mul2(b, f2);
          float x0, x1, x2, x3;
          upk2(mul2(a, pk2(s[k], s[k + 1])), x0, x1);
          upk2(mul2(b, pk2(s[k + 2], s[k + 3])), x2, x3);
          w16[k / 2] = pack16<T>(x0, x1);
          w16[k / 2 + 1] = pack16<T>(x2, x3);
        }
        tc::tmem_st16(lane_base + kKvP + 64 * half, w16);
        tc::tmem_st16(lane_base + kKvP + 64 * half + 16, w16 + 16);
        tc::tmem_wait_st();
        warp_arrive(&bars->ds_full, lane);
      }
      // the accumulators: warps 0-3 dv, warps 4-7 dk
      if (!warp_wait(&bars->acc_full, accs & 1, gd)) { dead = true; break; }
      tc::fence_after_sync();
      const Group w(g, gi);
      const int key = 128 * w.kt + r;
      const float f = half ? g.scale * pow2(-ex) : Scale<T>::kInv;
      const da2_tensor& out = half ? g.dk : g.dv;
      T* row = static_cast<T*>(out.data) + w.b * out.sb + w.hkv * out.sh + key * out.st;
      float* part = g.part_kv + ((size_t)slot * 2 + half) * D * 128 + r;
#pragma unroll
      for (int k0 = 0; k0 < D; k0 += 32) {
        uint32_t v[32];
        tc::tmem_ld32(lane_base + (half ? kKvDk : kKvDv) + k0, v);
        tc::tmem_wait_ld16(v);
        tc::tmem_wait_ld16(v + 16);
        if (k0 + 32 == D) warp_arrive(&bars->acc_free, lane);
        if (key >= w.len) {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = 0u;
        }
        if (!whole) {
#pragma unroll
          for (int k = 0; k < 32; ++k) part[(k0 + k) * 128] = __uint_as_float(v[k]) * f;
        } else if (key < g.Tk) {
          store32<T>(row + k0, v, f);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(bars->tmem, 512);
  }
}

// Adds the parts of one group's dv (y = 0) or dk (y = 1), 32 channels (z) at a time, in the order of
// the blocks; groups that one block covered are done already. Groups without a valid key are zero.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_cross_dkv_join(const __grid_constant__ CrossArgs g) {
  const int kt = blockIdx.x % g.k_tiles, bh = blockIdx.x / g.k_tiles;
  const int b = bh / g.Hkv, hkv = bh - b * g.Hkv, which = blockIdx.y, c0 = blockIdx.z * 32;
  const int key = 128 * kt + threadIdx.x;
  const int tiles = (valid_keys(g, b) + 127) >> 7;
  float acc[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) acc[k] = 0.0f;
  if (kt < tiles) {
    const Share sh(g);
    const long a = ((long)g.first[b] * g.Hkv + hkv * tiles + kt) * sh.n, e = a + sh.n;
    int c = (int)(a * sh.blocks / sh.units);             // a block at or next to the first
    while (c > 0 && sh.begin(c) > a) --c;
    while (sh.begin(c + 1) <= a) ++c;
    if (sh.begin(c + 1) >= e) return;                    // one block covered the group
    for (; sh.begin(c) < e; ++c) {
      if (sh.begin(c) == sh.begin(c + 1)) continue;
      const int slot = 2 * c + (sh.begin(c) >= a ? 0 : 1);
      const float* part = g.part_kv + ((size_t)slot * 2 + which) * D * 128 + (size_t)c0 * 128 + threadIdx.x;
#pragma unroll
      for (int k = 0; k < 32; ++k) acc[k] += part[k * 128];
      if (c + 1 >= sh.blocks) break;
    }
  }
  if (key >= g.Tk) return;
  const da2_tensor& out = which ? g.dk : g.dv;
  T* row = static_cast<T*>(out.data) + b * out.sb + hkv * out.sh + key * out.st + c0;
  store32<T>(row, reinterpret_cast<const uint32_t*>(acc), 1.0f);
}

template <typename T, int D>
cudaError_t launch(const CrossArgs& g, const CrossMaps& m, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_cross_dq<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)SmemDq<D>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cross_dkv<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)SmemDkv<D>::kBytes);
  if (e != cudaSuccess) return e;
  if constexpr (!Scale<T>::kBf16) {
    k_cross_vnorm<D><<<(unsigned)(g.B * g.Hkv * g.k_tiles), 256, 0, st>>>(g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int items = g.B * g.H * g.q_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(items < g.sms ? items : g.sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SmemDq<D>::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute early = {};                        // of k_cross_dq over k_cross_vnorm
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = Scale<T>::kBf16 ? 0 : 1;
  cudaLaunchKernelEx(&cfg, k_cross_dq<T, D>, m, g);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_cross_dkv<T, D><<<g.sms, kThreads, SmemDkv<D>::kBytes, st>>>(m, g);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_cross_dkv_join<T, D><<<dim3((unsigned)(g.B * g.Hkv * g.k_tiles), 2, D / 32), 128, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_backward(const CrossArgs& g, const CrossMaps& m, bool bf16, cudaStream_t st) {
  if (g.d == 128) return bf16 ? launch<__nv_bfloat16, 128>(g, m, st) : launch<__half, 128>(g, m, st);
  return bf16 ? launch<__nv_bfloat16, 64>(g, m, st) : launch<__half, 64>(g, m, st);
}

}  // namespace da2
