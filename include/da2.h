/*
 * da2.h -- C ABI of the DraftAttention2 hot path on NVIDIA B200 (sm_100a).
 *
 * Low-resolution-guided, block-sparse, mixed-precision self-attention over
 * spatiotemporal video-DiT tokens:
 *
 *   da2_prepare       fused operand preparation: per-frame 2D average- and max-pooled
 *                     draft Q/K, window-contiguous token permutation, FP8-E4M3 and
 *                     4-bit (E2M1, one E4M3 scale per 16 elements) copies of Q/K/V.
 *   da2_draft_select  low-resolution draft attention maps (avg- and max-pooled) combined
 *                     into a block-importance score, and the shared per-(head, query
 *                     block) ranking into FP8 / FP4 / skip under the budgets.
 *   da2_attention     one attention kernel with an FP8 phase and an FP4 phase that share
 *                     the online-softmax running max / sum and the fp32 accumulator; its
 *                     epilogue writes bf16 output back in the original token order.
 *
 * Sources: "DraftAttention2: Fast Video Diffusion with Low-Resolution-Guided Mixed-
 * Precision Attention" (arXiv 2609.32628), Abstract -- pooled draft Q/K, shared ranking
 * into higher / lower precision / skip under budgets, fused operand preparation, one
 * attention kernel with precision-specific phases sharing data movement, softmax
 * statistics and output accumulation. "DraftAttention: Fast Video Diffusion via
 * Low-Resolution Attention Guidance" (arXiv 2505.14708), Abstract -- per-frame
 * downsampling into draft Q/K, reorder before and restore after the sparse attention.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Inputs q, k, v and the output are bf16 [B, H, T, d] (or [B, T, H, d] with
 *    DA2_FLAG_LAYOUT_BTHD), d contiguous, with frame-major token order
 *    t = f*Hf*Wf + y*Wf + x.
 *  - Window (ph, pw) tiles each frame; edge windows are padded. Blocks n = f*ny*nx +
 *    (y/ph)*nx + (x/pw), slot s = (y%ph)*pw + (x%pw), ny = ceil(Hf/ph), nx = ceil(Wf/pw),
 *    N = F*ny*nx blocks of bs = ph*pw slots; padded slots hold zeros and padded keys are
 *    masked out of the attention.
 *  - Budgets: the shared ranking of each query block's KV blocks is cut three times,
 *    each cut rounded half up: c8 = floor((pct_fp8*N + 50)/100), c8m = floor(((pct_fp8 +
 *    pct_mix)*N + 50)/100), ck = floor(((pct_fp8 + pct_mix + pct_fp4)*N + 50)/100). The top
 *    n8 = c8 blocks are FP8, the next nm = c8m - c8 mixed (E4M3 Q K^T, E2M1 P V), the next
 *    n4 = ck - c8m FP4; the rest are skipped.
 *  - Memory ownership: the caller allocates q, k, v, out and the workspace (device memory,
 *    size from da2_workspace_size); the library allocates no device memory and keeps no
 *    state (da2_forward_host creates and destroys three streams and a few events per call;
 *    da2_forward_noalloc uses a static device array of the library image).
 *  - Every call is asynchronous on `stream` (0 = legacy default stream) except the ones
 *    documented as synchronising. Argument errors are returned before anything is
 *    enqueued; a failed CUDA call or launch returns DA2_ERR_CUDA, and da2_last_cuda_error
 *    then gives its cudaError_t.
 *  - Supported: d in {64, 128}; any window with bs = ph*pw in {32, 64, 128}; N <= 4096;
 *    B*H <= 65535 (DA2_ERR_UNSUPPORTED otherwise); 0 <= pct_fp8, pct_mix, pct_fp4 and
 *    pct_fp8 + pct_mix + pct_fp4 <= 100 (DA2_ERR_INVALID_ARG otherwise). Tensor pointers must be 16-byte
 *    aligned and the workspace 256-byte aligned (DA2_ERR_ALIGNMENT otherwise).
 */
#ifndef DA2_H
#define DA2_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* One attention call's shape, window and budgets. */
typedef struct da2_config {
  int B, H, d;          /* batch, heads, head dim (64 or 128) */
  int F, Hf, Wf;        /* latent frames, token rows and token columns per frame */
  int ph, pw;           /* pooling window rows x columns; block size bs = ph*pw */
  int pct_fp8, pct_fp4; /* percent of KV blocks kept at FP8 / FP4; the rest is skipped */
  float sm_scale;       /* softmax scale; 0 selects 1/sqrt(d) */
  int flags;            /* DA2_FLAG_* bits */
  int pct_mix;          /* percent of KV blocks in the mixed class (E4M3 scores, E2M1 P V),
                           ranked between FP8 and FP4; 0 gives the two-class path */
  float adapt_tau;      /* > 0: error-bound-driven FP4 budget. Per query block, the KV blocks
                           ranked after the fixed budgets join FP4, in rank order, while their
                           draft score (estimated attention mass) is >= adapt_tau, up to
                           pct_fp4_max percent FP4 blocks; 0 turns it off */
  int pct_fp4_max;      /* the FP4 cap of the adaptive budget (>= pct_fp4) */
} da2_config;

enum {
  /* da2_draft_select also writes its fp32 block-importance scores to the workspace
     (scores region, [B*H][N][N]); the workspace then grows by 4*B*H*N*N bytes. */
  DA2_FLAG_EXPORT_SCORES = 1,
  /* Drop the ln(valid tokens) term of the draft logits (the maps then rank by average
     token affinity instead of block mass). */
  DA2_FLAG_NO_MASS_CORRECTION = 2,
  /* q, k, v and out are token-major, bf16 [B,T,H,d] (the heads of one token adjacent, as
     a fused QKV projection usually leaves them) instead of [B,H,T,d]; read and written in
     place, results identical. da2_forward_host then runs unpipelined. (The pages fix no
     tensor layout.) */
  DA2_FLAG_LAYOUT_BTHD = 4,
  /* Debug aid: every workspace region is followed by a 256-byte guard (the workspace grows
     accordingly; da2_workspace_size and da2_workspace_views account for it). da2_prepare
     fills the guards with 0xA5 bytes and every stage call checks them after its kernels: a
     changed guard byte sets bit 4 of the workspace error word (DA2_ERR_TIMEOUT from
     da2_get_error). Costs two small launches per stage; off in normal use. */
  DA2_FLAG_DEBUG_CANARY = 8,
  /* Test hook for the failure path, never needed in use: da2_attention's copy engine
     withholds its first K/V tile, so a bounded device wait must run out. Every bounded
     wait's limit drops from 2 s to 50 ms; the launch sets the workspace error word, stops
     issuing, waits for its copies and tensor-core work in flight, frees its tensor memory
     and ends (about 0.1 s); da2_get_error then returns DA2_ERR_TIMEOUT and the output is
     undefined. */
  DA2_FLAG_TEST_STALL = 256
};

typedef enum da2_status {
  DA2_OK = 0,
  DA2_ERR_INVALID_ARG = 1,  /* null pointer, non-positive size, budgets out of range */
  DA2_ERR_UNSUPPORTED = 2,  /* d, bs, N or B*H outside the supported set */
  DA2_ERR_ALIGNMENT = 3,    /* a pointer is not 16-byte aligned */
  DA2_ERR_WORKSPACE = 4,    /* ws_bytes smaller than da2_workspace_size */
  DA2_ERR_CUDA = 5,         /* a CUDA call or launch failed */
  DA2_ERR_TIMEOUT = 6,      /* the device error word is set (a bounded wait ran out, a bad
                               index, or an overwritten guard region) */
  DA2_ERR_SCRATCH_TOO_SMALL = 7 /* da2_forward_noalloc: the configuration's workspace does
                                   not fit the library's built-in 64 MiB device scratch */
} da2_status;

/* Byte offsets of the workspace regions (from the workspace base) and the geometry.
   Tile layouts (all per (b*H + h) then per block, each block tile contiguous):
     q8, k8   E4M3 [BH][N][tile8_qk]: bs rows (tokens) x d bytes in the tensor-core
              K-major core-matrix layout: byte (r, c) at (r/8)*(8*d) + (c/16)*128 +
              (r%8)*16 + c%16.
     q4, k4   E2M1 [BH][N][tile4_qk]: bs rows x d/2 bytes, element c in byte c/2 (even
              c in the low nibble), byte (r, b) at (r/8)*(4*d) + (b/16)*128 + (r%8)*16 +
              b%16.
     v8       E4M3 transposed [BH][N][tile8_v]: d rows (channels) x bs bytes (slots):
              byte (c, s) at (c/8)*(8*bs) + (s/16)*128 + (c%8)*16 + s%16.
     v4       E2M1 transposed [BH][N][tile4_v]: d rows x kv4/2 bytes, kv4 = max(bs, 64)
              (slots >= bs are zero codes): byte (c, b) at (c/8)*(4*kv4) + (b/16)*128 +
              (c%8)*16 + b%16.
     sfq4, sfk4  E4M3 group scales of q4/k4, [BH][N][sf_qk]: d/64 atoms of 512 bytes;
              atom kb holds rows 0..127 (rows >= bs zero) x 4 scales (channel groups
              4kb..4kb+3): byte (r, j) at kb*512 + (r%32)*16 + (r/32)*4 + j.
     sfv4     E4M3 group scales of v4, [BH][N][sf_v]: kv4/64 atoms; rows = channels
              (rows >= d zero), scales = slot groups: byte (c, j) at kb*512 + (c%32)*16 +
              (c/32)*4 + j for slot group 4kb + j (groups past bs are zero).
     sq, sk   fp32 [BH][N]   dequantisation scale of a Q / K block (block amax / 448).
     sv       fp32 [BH][d]   dequantisation scale of a V channel (channel amax / 448).
     vamax    fp32 [BH][d]   V channel amax (written by da2_prepare).
     qavg, qmax, kavg, kmax  fp32 [BH][N][d] pooled draft Q / K.
     tags     u8 [BH][N][N]  0 skip, 1 FP4, 2 FP8, 3 mixed for (query block, KV block).
     list8    i16 [BH][N][n8s], list4 i16 [BH][N][n4s], listm i16 [BH][N][nms]: kept KV
              blocks of each class per query block in ascending block order (n8s =
              max(n8,1), n4s = max(n4max,1), nms = max(nm,1)); with the adaptive budget a
              row's FP4 list holds its n4 .. n4max blocks followed by -1 entries.
     scores   fp32 [BH][N][N] (only with DA2_FLAG_EXPORT_SCORES, else size 0).
     dlog     fp32 [BH][N][2][np] the two draft logit rows (average map, max map) of every
              query block, written and read by da2_draft_select (scratch; size 0 when
              N > 1024).
     qt, kt   the pooled Q and K of qavg/qmax and kavg/kmax again, each value split into a
              tf32 high part and its fp32 remainder and laid out as the draft MMAs' operands:
              per (b, h), 128-block tile, map (average, max) and 16-channel chunk, an 8 KB hi
              part then an 8 KB lo part of 128 rows x 16 channels in the K-major core-matrix
              layout (written by da2_prepare, read by da2_draft_select; size 0 when N > 1024).
     err      u32 device error word (0 = no error): bit 1 a bounded wait ran out, bit 2 an
              index or count of the selection was out of range, bit 4 a guard region of
              DA2_FLAG_DEBUG_CANARY was overwritten.
   With DA2_FLAG_DEBUG_CANARY a 256-byte guard follows every region above.
   A DA2_DEBUG build of the library (libda2_debug.so) also checks the selection's lists
   and tags before the attention (indices in range and ascending, tags of the right class,
   counts equal to the budgets) and makes every stage call wait for its stream and return
   DA2_ERR_TIMEOUT at once when the error word is set. */
typedef struct da2_views {
  int N, bs, T, Tp, ny, nx, n8, n4, kv4;
  size_t tile8_qk, tile4_qk, tile8_v, tile4_v, sf_qk, sf_v;
  size_t q8, k8, v8, q4, k4, v4, sfq4, sfk4, sfv4;
  size_t sq, sk, sv, vamax, qavg, qmax, kavg, kmax;
  size_t tags, list8, list4, scores, err, total;
  int nm;               /* mixed KV blocks per query block */
  size_t listm;
  int n4max;            /* FP4 list length (n4 unless the adaptive budget is on) */
  size_t dlog;          /* draft logits scratch (N <= 1024), see below */
  int np;               /* its row length: N rounded up to a multiple of 4 */
  size_t qt, kt;        /* pooled Q / K split for the draft MMAs (N <= 1024), see below */
} da2_views;

/* Workspace bytes needed for `cfg` (host only, no CUDA call). */
da2_status da2_workspace_size(const da2_config* cfg, size_t* bytes);

/* Geometry and region offsets for `cfg` (host only, no CUDA call). */
da2_status da2_workspace_views(const da2_config* cfg, da2_views* views);

/* Operand preparation. q, k, v: device bf16 [B,H,T,d] ([B,T,H,d] with
   DA2_FLAG_LAYOUT_BTHD); ws: device workspace of at least
   da2_workspace_size bytes. Writes every operand, scale and pooled region of ws and
   clears its error word. Asynchronous on `stream`. */
da2_status da2_prepare(const da2_config* cfg, const void* q, const void* k, const void* v,
                       void* ws, size_t ws_bytes, cudaStream_t stream);

/* Draft maps and ranking on a prepared workspace: writes tags, list8, list4 (and scores
   with DA2_FLAG_EXPORT_SCORES). Asynchronous on `stream`. */
da2_status da2_draft_select(const da2_config* cfg, void* ws, size_t ws_bytes,
                            cudaStream_t stream);

/* Mixed-precision block-sparse attention on a prepared and selected workspace. out:
   device bf16 [B,H,T,d] ([B,T,H,d] with DA2_FLAG_LAYOUT_BTHD; every element is written). Bounded device waits that run out
   set the workspace error word (read it with da2_get_error). Asynchronous. */
da2_status da2_attention(const da2_config* cfg, void* ws, size_t ws_bytes, void* out,
                         cudaStream_t stream);

/* Debug aid (no counterpart in the paper): checks the output contract of
   da2_draft_select on a selected workspace before it reaches the attention. Per (b, h,
   query block) the FP8, mixed and FP4 lists must hold in-range, strictly ascending KV
   blocks tagged 2, 3 and 1, the FP4 list may end in -1 padding only after its last block,
   and the row must hold exactly n8 FP8 and nm mixed tags and n4..n4max FP4 tags. A
   violation sets bit 2 of the workspace error word (read it with da2_get_error). Reads
   only the workspace; asynchronous on `stream`. DA2_DEBUG builds run it inside
   da2_draft_select. */
da2_status da2_check_selection(const da2_config* cfg, void* ws, size_t ws_bytes,
                               cudaStream_t stream);

/* da2_prepare, da2_draft_select and da2_attention in order on one stream. */
da2_status da2_forward(const da2_config* cfg, const void* q, const void* k, const void* v,
                       void* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Host-buffer variant of da2_forward: copies q, k, v (host, bf16 [B,H,T,d]; pinned
   memory gives asynchronous copies) into the caller's device staging buffers dq, dk, dv,
   runs the three stages and copies the result from dout back to out_host. Heads being
   independent, it pipelines over up to 16 groups of heads: the copies in of one group and
   the copy out of another overlap the stages of a third (three internal streams, two
   sub-workspaces carved from ws, used alternately; each group's stages are exactly those
   of da2_forward on a configuration of its heads, so out_host is bit-identical to
   da2_forward's output). With fewer than 2 groups, or a workspace too small for two
   sub-workspaces, it runs everything on `stream`. Work queued on `stream` before the call
   runs first; the call synchronises `stream` before returning. Afterwards only the error
   word of ws (da2_get_error with cfg) is meaningful; the rest of ws holds the groups'
   layouts. ws_bytes must be at least da2_workspace_size(cfg). */
da2_status da2_forward_host(const da2_config* cfg, const void* q_host, const void* k_host,
                            const void* v_host, void* out_host, void* dq, void* dk,
                            void* dv, void* dout, void* ws, size_t ws_bytes,
                            cudaStream_t stream);

/* da2_forward without any device allocation, by the library or by the caller.
   No counterpart in the paper: this serves callers that cannot obtain device memory when
   they run the attention -- a plug-in inside a host framework that owns all device memory
   and exposes no allocator, or a serving loop that forbids cudaMalloc after start-up (it
   can synchronise the device and fail under fragmentation). The caller still passes q,
   k, v and out (device bf16 [B,H,T,d], 16-byte aligned); the workspace is a fixed 64 MiB
   device array inside the library, which every GPU that loads the library holds until
   the process exits. Configurations whose da2_workspace_size exceeds 64 MiB are rejected
   with DA2_ERR_SCRATCH_TOO_SMALL before anything is enqueued (the tiny workload and
   single-head 480p / 720p Wan-like layers fit; a full 40-head layer does not), and so is
   DA2_FLAG_EXPORT_SCORES (DA2_ERR_INVALID_ARG: the scores would stay in the hidden
   array). Every call looks up the array's device address on the current device
   (cudaGetSymbolAddress), so an address never outlives a device reset; the first call on
   a device also loads the library's device code there, so make it before any stream
   capture. Every call on a device shares the one array and leaves its contents behind;
   the path clears what must start at zero itself. Calls that overlap on the GPU
   (different streams, or several host threads on one device) race on the array and give
   wrong results: serialise them. Asynchronous on `stream` like da2_forward. Its device
   error word is read with da2_get_error(NULL, 0, cfg, stream, &word). */
da2_status da2_forward_noalloc(const da2_config* cfg, const void* q, const void* k,
                               const void* v, void* out, cudaStream_t stream);

/* Reads the workspace's device error word into *word and clears it (synchronises
   `stream`). Returns DA2_ERR_TIMEOUT if the word was non-zero. ws = NULL reads the word of
   the built-in array of da2_forward_noalloc (cfg as given to that call; ws_bytes is
   ignored). */
da2_status da2_get_error(void* ws, size_t ws_bytes, const da2_config* cfg,
                         cudaStream_t stream, uint32_t* word);

/* The cudaError_t of the calling host thread's most recent library call that returned
   DA2_ERR_CUDA (cudaSuccess if none). The library checks every launch with
   cudaGetLastError, which clears the runtime's own record, so this is where the code of,
   say, cudaErrorLaunchOutOfResources is kept. Host only, no CUDA call. */
int da2_last_cuda_error(void);

/* Static string naming a status. */
const char* da2_status_string(da2_status status);

/* ------------------------------------------------------------------------------------
 * Operators around the self-attention of a video-DiT block: the norm and position rotation
 * of its queries and keys in front of da2_prepare, and the attention of its tokens to an
 * encoder's states, each with its backward pass. No counterpart in the papers.
 *
 * Their tensors are given by a base pointer and element strides of batch, head and token
 * (channels are contiguous), so [B,H,T,d], [B,T,H,d] and slices of a fused projection all go
 * in as they are. Base pointers must be 16-byte aligned and strides multiples of 8 elements
 * (DA2_ERR_ALIGNMENT otherwise); the stride of an axis longer than one must be at least d
 * (DA2_ERR_INVALID_ARG otherwise: rows would overlap); the stride of an axis of length one is
 * not read. Outputs must not overlap each other or, but
 * where a call says otherwise, an input. d is 64 or 128 and the element type bf16 or fp16.
 * Every sum, norm and softmax statistic is fp32; each output is rounded once. The attention's tensor
 * cores take 16-bit operands: p (forward) and p and dS (backward) are rounded to the element type in
 * between, once each, and D is formed from the rounded out. Against 64 bits the attention's results are
 * off by 1.2 to 1.5 times what the rounding of the outputs alone makes (relative L2 0.0020 to 0.0024 instead
 * of 0.0017 in bf16, 0.0003 instead of 0.0002 in fp16).
 * da2_prepare takes bf16, and the self-attention has no backward pass: in a block of this library the
 * bf16 forms of the norm feed it, and gradients reach the norms of the attention to the encoder's states;
 * fp16 and the rotation's gradient are for a caller's own self-attention.
 * At most 2^31 - 256 tokens an axis (DA2_ERR_UNSUPPORTED otherwise).
 * The calls are asynchronous on `stream`, allocate nothing, keep nothing between calls and
 * can be captured into a CUDA graph; two calls that may overlap need workspaces of their own. */
typedef struct da2_tensor {
  void* data;           /* element (0, 0, 0, 0) */
  int64_t sb, sh, st;   /* element strides of batch, head and token */
} da2_tensor;

enum { DA2_DTYPE_BF16 = 0, DA2_DTYPE_F16 = 1 };

enum {
  /* rotate the channel pairs (c, c + d/2) instead of (2c, 2c + 1) */
  DA2_ROPE_HALVES = 1,
  /* the tables are [B][T_rot][d/2] instead of [T_rot][d/2] shared by the batch */
  DA2_ROPE_BATCHED = 2
};

/* One call of the norm and rotation. */
typedef struct da2_norm_rope_config {
  int B, Hq, Hk, T, d;  /* batch, query heads, key heads (0: no keys), tokens, head dim */
  int T_rot;            /* tokens 0 .. T_rot-1 are rotated (0: the norm alone) */
  float eps;            /* added to the mean square; finite, >= 0 */
  int dtype;            /* DA2_DTYPE_* of q, k and their outputs and gradients */
  int flags;            /* DA2_ROPE_* bits */
} da2_norm_rope_config;

/* RMS norm of each head of q and k (over its own d channels, not over all heads' together) and the
   position rotation, in one pass:
     n = x / sqrt(mean_c(x_c^2) + eps),  y = n * w,
     (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos) for channel pair i = (a, b)
   with cos, sin = row t (the token) and column i of the tables. wq, wk: fp32 [d], shared by
   the heads, 16-byte aligned; NULL means all ones. cos_t, sin_t: fp32, 16-byte aligned; not read when T_rot is
   0. q_out may be q and k_out may be k (the same pointer and strides). k and k_out are not
   read when Hk is 0 and may be NULL. A row of zeros with eps 0 gives NaN, like the formula. */
da2_status da2_qk_norm_rope(const da2_norm_rope_config* cfg, const da2_tensor* q, const da2_tensor* k,
                            const float* wq, const float* wk, const float* cos_t, const float* sin_t,
                            const da2_tensor* q_out, const da2_tensor* k_out, cudaStream_t stream);

/* Workspace bytes of da2_qk_norm_rope_backward (host only, no CUDA call). */
da2_status da2_qk_norm_rope_workspace_size(const da2_norm_rope_config* cfg, size_t* bytes);

/* Gradients of da2_qk_norm_rope: dq_out, dk_out are the gradients of its outputs, q, k its
   inputs. With g = the gradient rotated back,
     dw = sum over rows of g * n,  dx = (g w - n mean_c(g w n)) / sqrt(mean_c(x^2) + eps).
   dq may be dq_out or q, dk may be dk_out or k. dwq, dwk: fp32 [d], 4-byte aligned, overwritten (dwk is not
   written when Hk is 0); NULL skips them, and with both NULL ws is not needed. The sums run in a fixed order: equal inputs give equal bits. ws: 256-byte aligned. */
da2_status da2_qk_norm_rope_backward(const da2_norm_rope_config* cfg, const da2_tensor* dq_out,
                                     const da2_tensor* dk_out, const da2_tensor* q, const da2_tensor* k,
                                     const float* wq, const float* wk, const float* cos_t,
                                     const float* sin_t, const da2_tensor* dq, const da2_tensor* dk,
                                     float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                     cudaStream_t stream);

/* One call of the attention to an encoder's states. */
typedef struct da2_cross_config {
  int B, H, Hkv;        /* batch, query heads, key/value heads (Hkv divides H; query head h uses
                           key/value head h / (H / Hkv)) */
  int Tq, Tk, d;        /* queries, keys, head dim */
  float sm_scale;       /* softmax scale; 0 selects 1/sqrt(d) */
  int dtype;            /* DA2_DTYPE_* of every activation and gradient */
  int flags;            /* 0, or DA2_FLAG_TEST_STALL */
} da2_cross_config;

/* Workspace bytes of da2_cross_attention and of its backward pass (host only, no CUDA call). */
da2_status da2_cross_attention_workspace_size(const da2_cross_config* cfg, size_t* bytes);
da2_status da2_cross_attention_backward_workspace_size(const da2_cross_config* cfg, size_t* bytes);

/* Attention of Tq queries to Tk keys of another sequence:
     s = q k^T sm_scale,  p = softmax over keys 0 .. len[b]-1,  out = p v,
     lse = ln sum exp(s)  (fp32 [B][H][Tq]; NULL: not written).
   kv_len: device int32 [B], each taken into 0 .. Tk; NULL: Tk for every batch entry. Keys and
   values behind the length do not reach the result, whatever they hold. A batch entry of length
   0 has out = 0 and lse = -inf. Scores |s| up to 5e7: beyond, the fp32 exponent's own rounding takes p
   out of the element type's range. Within the length infinities and NaN count as the formula has it: a
   key of score -inf has no weight, and a row without any weight is NaN. Few query rows are split over their keys, the parts joined in a
   fixed order: equal inputs give equal bits.
   ws: 256-byte aligned; its first 256 bytes are the error area, to be zeroed once after the
   workspace is allocated. A bounded device wait that runs out sets a bit there
   (da2_cross_attention_get_error); nothing else in ws outlives the call. */
da2_status da2_cross_attention(const da2_cross_config* cfg, const da2_tensor* q, const da2_tensor* k,
                               const da2_tensor* v, const da2_tensor* out, float* lse, const int32_t* kv_len,
                               void* ws, size_t ws_bytes, cudaStream_t stream);

/* Gradients of da2_cross_attention; out and lse are its results, dout the gradient of out.
     D = sum_c dout out,  dS = p (dout v^T - D),
     dq = sm_scale dS k,  dk = sm_scale dS^T q,  dv = p^T dout  (dk, dv summed over the query
   heads that share a key/value head).
   Every row of dq, dk and dv is written: zero for keys behind the length and for batch entries of
   length 0. p comes from lse, whose rounding makes it relatively off by up to |lse| 2^-23. In fp16 dS
   carries powers of two from the norms of dout and v, so that any dout whose gradients fit fp16 will do. The sums run in a fixed order. ws as above, of the backward pass's own size. */
da2_status da2_cross_attention_backward(const da2_cross_config* cfg, const da2_tensor* dout,
                                        const da2_tensor* q, const da2_tensor* k, const da2_tensor* v,
                                        const da2_tensor* out, const float* lse, const int32_t* kv_len,
                                        const da2_tensor* dq, const da2_tensor* dk, const da2_tensor* dv,
                                        void* ws, size_t ws_bytes, cudaStream_t stream);

/* Reads the error word of a cross-attention workspace into *word and clears it (synchronises
   `stream`): DA2_ERR_TIMEOUT if it was non-zero. */
da2_status da2_cross_attention_get_error(void* ws, size_t ws_bytes, cudaStream_t stream, uint32_t* word);

#ifdef __cplusplus
}
#endif
#endif /* DA2_H */
