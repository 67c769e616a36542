// C entry points of the attention to an encoder's states: argument checks, workspace layout,
// tensor maps and launches.
#include <cmath>

#include "api.cuh"
#include "cross.cuh"

namespace da2 {
namespace {

constexpr size_t kErrBytes = 256;
constexpr int kSms = 148;              // B200; the workspace is sized without a device

da2_status check_cross_config(const da2_cross_config* c) {
  if (!c) return DA2_ERR_INVALID_ARG;
  if (c->B <= 0 || c->H <= 0 || c->Hkv <= 0 || c->Tq <= 0 || c->Tk <= 0 || c->H % c->Hkv != 0)
    return DA2_ERR_INVALID_ARG;
  if (!(c->sm_scale >= 0.0f) || std::isinf(c->sm_scale)) return DA2_ERR_INVALID_ARG;
  if (c->dtype != DA2_DTYPE_BF16 && c->dtype != DA2_DTYPE_F16) return DA2_ERR_INVALID_ARG;
  if (c->flags & ~DA2_FLAG_TEST_STALL) return DA2_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return DA2_ERR_UNSUPPORTED;
  if (c->Tq > kMaxTokens || c->Tk > kMaxTokens) return DA2_ERR_UNSUPPORTED;
  // work items and rows are counted in 32 bits, with room for 64 parts of the keys
  const long heads = (long)c->B * c->H;
  if (heads > (1L << 24)) return DA2_ERR_UNSUPPORTED;
  if (heads * (((long)c->Tq + 127) / 128) > (1L << 24) || heads * (((long)c->Tk + 127) / 128) > (1L << 24))
    return DA2_ERR_UNSUPPORTED;
  return DA2_OK;
}

long q_pairs(const da2_cross_config* c) { return (c->Tq + 255) / 256; }

// Parts that the keys of one query tile are split into, so that few query rows still fill the
// processors. In units of 128 keys' time: a wave of items costs its keys plus about two for filling the
// pipeline and the epilogue, and joining costs about four, plus the parts' traffic. Measured with the rule's
// parts and others (single calls, us): 40 items on 512 keys 19.5 whole, 23.6 in two parts (rule: whole); 48
// on 4096 keys 87 whole, 62 in two, 54 in three (rule); 80 on 4096 keys 66.6 whole, 60 to 62 in three
// (rule), 62.5 in eight; 120 and 147 on 4096 keys 71 and 73 whole (rule), 81 in two. From 148 items on nothing is
// split: right at 290 (128 whole, 138 in two), not just above 148 (150 items 123 whole, 105 in two, 93 in
// eight).
int choose_splits(const da2_cross_config* c) {
  const long units = (long)c->B * c->H * q_pairs(c), steps = ((long)c->Tk + 127) / 128;
  if (units >= kSms || steps < 2) return 1;
  int best = 1;
  double best_cost = (double)(steps + 2);
  const double rows = c->Tq < 256 ? c->Tq : 256;
  for (long s = 2; s <= steps && s <= 64; ++s) {
    const long waves = (units * s + kSms - 1) / kSms;
    const double cost = (double)waves * ((steps + s - 1) / s + 2 + rows / 256.0) + 4.0;
    if (cost < best_cost) best_cost = cost, best = (int)s;
  }
  return best;
}

struct FwdLayout {
  int splits;
  size_t part_o, part_lse, total;
};
FwdLayout fwd_layout(const da2_cross_config* c) {
  FwdLayout l;
  l.splits = choose_splits(c);
  const size_t rows = (size_t)c->B * c->H * c->Tq;
  l.part_o = kErrBytes;
  l.part_lse = l.part_o + (l.splits > 1 ? align256(l.splits * rows * c->d * 4) : 0);
  l.total = l.part_lse + (l.splits > 1 ? align256(l.splits * rows * 4) : 0);
  return l;
}

struct BwdLayout {
  size_t lse2, delta, part, first, dnorm2, vnorm2, total;
};
BwdLayout bwd_layout(const da2_cross_config* c) {
  BwdLayout l;
  const size_t rows = (size_t)c->B * c->H * (((size_t)c->Tq + 127) / 128 * 128);
  l.lse2 = kErrBytes;
  l.delta = l.lse2 + rows * 4;
  l.part = l.delta + rows * 4;
  l.first = l.part + (size_t)2 * kSms * 2 * c->d * 128 * 4;
  l.dnorm2 = l.first + align256(((size_t)c->B + 1) * 4);
  const bool f16 = c->dtype == DA2_DTYPE_F16;
  l.vnorm2 = l.dnorm2 + (f16 ? align256(rows / 128 * 16) : 0);
  l.total = l.vnorm2 + (f16 ? align256((size_t)c->B * c->Hkv * (((size_t)c->Tk + 127) / 128) * 4) : 0);
  return l;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library does not link the driver).
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Map of a strided activation [B][H][T][d] for boxes of `rows` tokens x 64 channels. The stride of an
// axis of length one is never used; the encoder wants a multiple of 16 bytes all the same.
cudaError_t make_map(CUtensorMap* m, const da2_tensor& t, long B, long H, long T, int d, bool bf16,
                     int rows = 128) {
  const EncodeTiled fn = encoder();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)H, (cuuint64_t)B};
  auto bytes = [&](int64_t s) { return (cuuint64_t)(s > 0 ? s : d) * 2; };
  const cuuint64_t strides[3] = {bytes(t.st), bytes(t.sh), bytes(t.sb)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, t.data,
                        dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// What both directions check and fill.
da2_status common_args(const da2_cross_config* c, const da2_tensor* q, const da2_tensor* k, const da2_tensor* v,
                       const float* lse, const int32_t* kv_len, void* ws, da2_tensor in[3], CrossArgs* g) {
  *g = CrossArgs{};
  da2_status s = check_tensor(q, c->B, c->H, c->Tq, c->d, &in[0]);
  if (s == DA2_OK) s = check_tensor(k, c->B, c->Hkv, c->Tk, c->d, &in[1]);
  if (s == DA2_OK) s = check_tensor(v, c->B, c->Hkv, c->Tk, c->d, &in[2]);
  if (s != DA2_OK) return s;
  if (!ws) return DA2_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(kv_len) & 3u) != 0)
    return DA2_ERR_ALIGNMENT;
  g->B = c->B; g->H = c->H; g->Hkv = c->Hkv; g->group = c->H / c->Hkv;
  g->Tq = c->Tq; g->Tk = c->Tk; g->d = c->d;
  g->scale = c->sm_scale > 0.0f ? c->sm_scale : 1.0f / std::sqrt((float)c->d);
  g->scale_log2 = g->scale * kLog2E;
  g->kv_len = kv_len;
  g->err = static_cast<uint32_t*>(ws);
  g->stall = (c->flags & DA2_FLAG_TEST_STALL) != 0;
  // about 2 s, longer than anything here waits; the test hook shortens it to about 50 ms
  g->wait_clocks = g->stall ? 100000000ll : 4000000000ll;
  return DA2_OK;
}

cudaError_t device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && *sms > kSms) *sms = kSms;
  return e;
}

}  // namespace
}  // namespace da2

using namespace da2;

extern "C" {

da2_status da2_cross_attention_workspace_size(const da2_cross_config* cfg, size_t* bytes) {
  const da2_status s = check_cross_config(cfg);
  if (s != DA2_OK) return s;
  if (!bytes) return DA2_ERR_INVALID_ARG;
  *bytes = fwd_layout(cfg).total;
  return DA2_OK;
}

da2_status da2_cross_attention(const da2_cross_config* cfg, const da2_tensor* q, const da2_tensor* k,
                               const da2_tensor* v, const da2_tensor* out, float* lse, const int32_t* kv_len,
                               void* ws, size_t ws_bytes, cudaStream_t stream) {
  const NvtxRange range("da2_cross_attention");
  da2_status s = check_cross_config(cfg);
  if (s != DA2_OK) return s;
  da2_tensor in[3];
  CrossArgs g;
  s = common_args(cfg, q, k, v, lse, kv_len, ws, in, &g);
  if (s == DA2_OK) s = check_tensor(out, cfg->B, cfg->H, cfg->Tq, cfg->d, &g.out);
  if (s != DA2_OK) return s;
  const FwdLayout l = fwd_layout(cfg);
  if (ws_bytes < l.total) return DA2_ERR_WORKSPACE;
  g.lse = lse;
  g.q_pairs = (int)q_pairs(cfg);
  g.splits = l.splits;
  g.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.part_o);
  g.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.part_lse);
  const bool bf16 = cfg->dtype == DA2_DTYPE_BF16;
  CrossMaps m = {};
  cudaError_t e = device_sms(&g.sms);
  if (e == cudaSuccess) e = make_map(&m.q, in[0], cfg->B, cfg->H, cfg->Tq, cfg->d, bf16);
  if (e == cudaSuccess) e = make_map(&m.k, in[1], cfg->B, cfg->Hkv, cfg->Tk, cfg->d, bf16, 64);
  if (e == cudaSuccess) e = make_map(&m.v, in[2], cfg->B, cfg->Hkv, cfg->Tk, cfg->d, bf16, 64);
  if (e == cudaSuccess) e = make_map(&m.out, g.out, cfg->B, cfg->H, cfg->Tq, cfg->d, bf16);
  if (e == cudaSuccess) e = launch_cross_forward(g, m, bf16, stream);
  return cuda_status(e);
}

da2_status da2_cross_attention_backward_workspace_size(const da2_cross_config* cfg, size_t* bytes) {
  const da2_status s = check_cross_config(cfg);
  if (s != DA2_OK) return s;
  if (!bytes) return DA2_ERR_INVALID_ARG;
  *bytes = bwd_layout(cfg).total;
  return DA2_OK;
}

da2_status da2_cross_attention_backward(const da2_cross_config* cfg, const da2_tensor* dout,
                                        const da2_tensor* q, const da2_tensor* k, const da2_tensor* v,
                                        const da2_tensor* out, const float* lse, const int32_t* kv_len,
                                        const da2_tensor* dq, const da2_tensor* dk, const da2_tensor* dv,
                                        void* ws, size_t ws_bytes, cudaStream_t stream) {
  const NvtxRange range("da2_cross_attention_backward");
  da2_status s = check_cross_config(cfg);
  if (s != DA2_OK) return s;
  da2_tensor in[3];
  CrossArgs g;
  s = common_args(cfg, q, k, v, lse, kv_len, ws, in, &g);
  if (s == DA2_OK) s = check_tensor(out, cfg->B, cfg->H, cfg->Tq, cfg->d, &g.out);
  if (s == DA2_OK) s = check_tensor(dout, cfg->B, cfg->H, cfg->Tq, cfg->d, &g.dout);
  if (s == DA2_OK) s = check_tensor(dq, cfg->B, cfg->H, cfg->Tq, cfg->d, &g.dq);
  if (s == DA2_OK) s = check_tensor(dk, cfg->B, cfg->Hkv, cfg->Tk, cfg->d, &g.dk);
  if (s == DA2_OK) s = check_tensor(dv, cfg->B, cfg->Hkv, cfg->Tk, cfg->d, &g.dv);
  if (s != DA2_OK) return s;
  if (!lse) return DA2_ERR_INVALID_ARG;
  const BwdLayout l = bwd_layout(cfg);
  if (ws_bytes < l.total) return DA2_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  g.lse_in = lse;
  g.q_tiles = (cfg->Tq + 127) / 128;
  g.k_tiles = (cfg->Tk + 127) / 128;
  g.lse2 = reinterpret_cast<float*>(base + l.lse2);
  g.delta = reinterpret_cast<float*>(base + l.delta);
  g.part_kv = reinterpret_cast<float*>(base + l.part);
  g.first = reinterpret_cast<int32_t*>(base + l.first);
  g.dnorm2 = reinterpret_cast<float*>(base + l.dnorm2);
  g.vnorm2 = reinterpret_cast<float*>(base + l.vnorm2);
  g.v = in[2];
  const bool bf16 = cfg->dtype == DA2_DTYPE_BF16;
  CrossMaps m = {};
  cudaError_t e = device_sms(&g.sms);
  if (e == cudaSuccess) e = make_map(&m.q, in[0], cfg->B, cfg->H, cfg->Tq, cfg->d, bf16);
  if (e == cudaSuccess) e = make_map(&m.k, in[1], cfg->B, cfg->Hkv, cfg->Tk, cfg->d, bf16);
  if (e == cudaSuccess) e = make_map(&m.v, in[2], cfg->B, cfg->Hkv, cfg->Tk, cfg->d, bf16);
  if (e == cudaSuccess) e = make_map(&m.dout, g.dout, cfg->B, cfg->H, cfg->Tq, cfg->d, bf16);
  if (e == cudaSuccess) e = make_map(&m.out, g.out, cfg->B, cfg->H, cfg->Tq, cfg->d, bf16);
  if (e == cudaSuccess) e = make_map(&m.dq, g.dq, cfg->B, cfg->H, cfg->Tq, cfg->d, bf16);
  if (e == cudaSuccess) e = launch_cross_backward(g, m, bf16, stream);
  return cuda_status(e);
}

da2_status da2_cross_attention_get_error(void* ws, size_t ws_bytes, cudaStream_t stream, uint32_t* word) {
  if (!ws || !word) return DA2_ERR_INVALID_ARG;
  if (ws_bytes < kErrBytes) return DA2_ERR_WORKSPACE;
  uint32_t h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, ws, 4, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0, 4, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_status(e);
  *word = h;
  return h ? DA2_ERR_TIMEOUT : DA2_OK;
}

}  // extern "C"
