/*
 * lora_gb300.h -- C ABI for one training step of a LoRA-adapted linear layer on GB300 (sm_103a).
 *
 * The step (for each adapted linear with frozen W [out, in], adapter A [r, in], B [out, r]):
 *   forward   Y  = X W^T + s' (Xd A^T) B^T,  Xd = M * X, s' = s / (1 - p)
 *             ("8. LoRA Fundamentals", How it works: W_eff = W + s B A, s = alpha/r or alpha/sqrt(r))
 *   DoRA      Y  = (m / n) * (X W^T + s' (Xd A^T) B^T),  n_o = ||W_o + s (B A)_o||, n detached
 *             ("8. LoRA Fundamentals", How it works: canonical DoRA)
 *   backward  dY' = dY (or dY * m/n), G = dY' B, dX = dY' W + s' (G A) * M,
 *             dA += s' G^T Xd, dB += s' dY'^T (Xd A^T), dm += sum_t dY * Y / m
 *             ("Backward Bug Hunts and Vulkan Tiled GEMM", Bug #1 and Bug #2: the activation
 *             gradient through the frozen weight and the out_prod LoRA-B gradient)
 *   prepare   S = sum g^2 (double); non-finite -> reject; c = gamma * min(1, max_norm / norm)
 *             ("4.3. Training Guide", Gradient accumulation and Gradient clipping)
 *   AdamW     A-only decoupled decay from the pre-update value with the scheduled lr; LoRA+ ratio
 *             on B's lr ("4.3. Training Guide", Optimizer and Schedules)
 *   multi     token segments routed to per-slot adapters, per-slot scale/clip/Adam
 *             ("Multi-LoRA Training Example (fully-async)", Design)
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller, row-major, densely packed.
 *     Descriptor structs, group tables and slot tables are HOST pointers read during the call.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream). Every call only
 *     enqueues work on that stream and returns; nothing synchronises unless documented.
 *   - Argument errors are found on the host before any launch and return a nonzero status with
 *     nothing enqueued. A launch error returns LORA_ERR_CUDA.
 *   - The library allocates no device memory. Scratch comes from a caller workspace whose size
 *     the matching *_workspace_size call gives; a smaller workspace returns LORA_ERR_WORKSPACE.
 *   - Calls are not thread-safe on one workspace; two calls in flight need two workspaces.
 *   - Activations X, dY, Y, dX and the frozen W share one dtype (LORA_F32 or LORA_BF16;
 *     LORA_BF16_FP8 and LORA_BF16_BLK8 are bf16 with an E4M3 frozen product, see their
 *     definitions).
 *     A, B, their gradients, the Adam moments, H and the DoRA vectors are always fp32.
 *   - Shapes: 1 <= rank <= LORA_MAX_RANK and rank % 4 == 0; in and out multiples of 8;
 *     all pointers 16-byte aligned (LORA_ERR_ALIGN otherwise).
 */
#ifndef LORA_GB300_H
#define LORA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------------------------------*/
#define LORA_OK 0
#define LORA_ERR_INVALID 1      /* null pointer, negative size, bad rank, bad enum */
#define LORA_ERR_ALIGN 2        /* pointer or row stride not 16-byte aligned */
#define LORA_ERR_UNSUPPORTED 3  /* valid request this build does not serve (dtype, rank, sizes) */
#define LORA_ERR_WORKSPACE 4    /* workspace too small */
#define LORA_ERR_CUDA 5         /* a CUDA launch or runtime call failed */
#define LORA_ERR_NONFINITE 6    /* device status: a gradient element is NaN or +-Inf */
#define LORA_ERR_TIMEOUT 7      /* device status: a tensor-core pipeline wait ran out of its bound */

/* ---- enums ----------------------------------------------------------------------------------*/
/* fp32 activations and frozen W. The frozen products (forward and dX) run on bf16 tensor cores as
 * four products of a two-term bf16 split of each operand (hi = bf16(x), lo = bf16(x - hi);
 * hi*hi' + hi*lo' + lo*hi' + lo*lo'), accumulated in fp32 in periods of 256 K-elements; the
 * adapter terms and the low-rank products run in fp32. Each output of the split products is
 * within 2^-17 of sum_k |a_k w_k| of the exact product. Against a float64 reference the
 * per-tensor max relative error is shown below 1e-5 for N(0, 1)-scaled operands with
 * K <= 14336 and for heavy-tailed ones (Student-t, 3 degrees of freedom) up to K = 8192 on the
 * GPU and K = 14336 in the split arithmetic alone. */
#define LORA_F32 0
#define LORA_BF16 1
/* bf16 activations and frozen W whose frozen products (forward and dX) run on E4M3 tensor
 * cores: W quantised once by lora_prepare_weight (per output row for the forward, per input
 * column for dX), X and dY' per token inside each call, every row scaled so that its largest
 * magnitude maps to 448 (r = 448 / amax, codes = e4m3(x * r) rounded to nearest even and
 * saturated, scale = amax / 448, all in fp32; r = scale = 1 for an all-zero row). The adapter
 * branch (shrink, G, dA, dB) reads the bf16 tensors unchanged ("LoRA Training and Serving",
 * Quantized rollout: an FP8 base under a bf16-trained adapter). Single-adapter calls without
 * DoRA; in_dim and out_dim multiples of 16 and at most 16384 (LORA_ERR_UNSUPPORTED otherwise). */
#define LORA_BF16_FP8 2
/* bf16 activations over a frozen weight kept as E4M3 codes with one scale per 128 x 128 block (see
 * lora_block_product): W_prep = [W8 (out x in codes) | sw], from lora_prepare_weight (which
 * quantises a bf16 W) or filled by the caller with a checkpoint's codes and scales (the sections of
 * lora_prepared_weight_size); lora_forward does not read W, which may be NULL. X and dY' are
 * quantised per 1 x 128 block inside each call; both products read the same codes. The adapter
 * branch reads the bf16 tensors unchanged. Single-adapter calls without DoRA (LORA_ERR_UNSUPPORTED
 * otherwise); in_dim and out_dim multiples of 16 (LORA_ERR_ALIGN). */
#define LORA_BF16_BLK8 3

#define LORA_SCHED_CONSTANT 0
#define LORA_SCHED_WARMUP_COSINE 1

#define LORA_MAX_RANK 64
#define LORA_MAX_SLOTS 32
#define LORA_MAX_GROUPS 64
#define LORA_MAX_CHUNKS_PER_CALL 64

/* One adapted linear. W is [out_dim, in_dim] (nn.Linear layout). */
typedef struct lora_desc {
  int64_t in_dim;
  int64_t out_dim;
  int32_t rank;        /* r; for multi-LoRA calls: the largest slot rank (H row stride) */
  float scale;         /* s = lora_scale(alpha, rank, rslora); ignored by multi-LoRA calls */
  int32_t dtype;       /* LORA_F32 | LORA_BF16 | LORA_BF16_FP8 | LORA_BF16_BLK8 for X, W, dY, Y, dX */
  float dropout_p;     /* 0 <= p < 1; applies to the adapter branch input only */
  uint64_t seed;       /* dropout seed */
  uint32_t layer_id;   /* dropout key fields */
  uint32_t proj_id;    /* < 65536 */
  int32_t dora;        /* 1: DoRA row-magnitude mode (single-adapter calls only) */
} lora_desc;

/* Where the call's tokens sit in the optimizer step (dropout key fields). Token t of a call
 * belongs to accumulation chunk accum_ordinal + t / chunk_tokens at position t % chunk_tokens;
 * chunk_tokens == 0 means all T tokens are one chunk. At most LORA_MAX_CHUNKS_PER_CALL chunks
 * per call, and accum_ordinal + chunks <= 65536. */
typedef struct lora_ctx {
  uint64_t opt_step;
  uint32_t accum_ordinal;
  int64_t chunk_tokens;
} lora_ctx;

/* One slot of the multi-LoRA page table ("Multi-LoRA Training Example", Design: slot-keyed
 * adapter page table with per-slot rank/alpha). All pointers device, fp32. */
typedef struct lora_slot {
  const float* A;   /* [rank, in_dim] */
  const float* B;   /* [out_dim, rank] */
  float* dA;        /* [rank, in_dim], accumulated (+=) by multi_lora_backward */
  float* dB;        /* [out_dim, rank], accumulated (+=) */
  int32_t rank;     /* 1..desc.rank, multiple of 4 */
  float scale;      /* s_k = lora_scale(alpha_k, rank_k, rslora) */
} lora_slot;

/* A group of adapter parameters stored contiguously in the flat fp32 arenas (params, grads,
 * m, v share one layout): [n_a elements of kind A | n_b of kind B | n_mag DoRA magnitudes]
 * starting at `offset`. One group = one clip norm and one Adam clock: the whole model for a
 * single adapter set (global clip), or one slot for multi-LoRA. */
typedef struct lora_group {
  int64_t offset;
  int64_t n_a;
  int64_t n_b;
  int64_t n_mag;
  double grad_scale;   /* gamma: 1 / prediction tokens, or 1 / adapter_global_batch_size */
  float max_norm;      /* 0 disables clipping (normalisation by gamma still applies) */
  float lr;            /* scheduled learning rate of this update (lora_lr_at) */
  int64_t step;        /* completed updates of this group before this one (bias correction) */
} lora_group;

/* Doubles so that 1 - beta is formed on the host before rounding (0.999f would shift 1 - beta2
 * by 1.3e-5 relative). The kernels compute in fp32. */
typedef struct lora_adamw_hp {
  double beta1;         /* 0.9 */
  double beta2;         /* 0.999 */
  double eps;           /* 1e-8, added outside the square root */
  double weight_decay;  /* applied to kind A only */
  double plus_ratio;    /* LoRA+: B's lr = lr * plus_ratio */
} lora_adamw_hp;

/* ---- host helpers ---------------------------------------------------------------------------*/
/* Static string for a status code. */
const char* lora_status_string(int status);

/* s = alpha / rank, or alpha / sqrt(rank) when rslora != 0 ("8. LoRA Fundamentals", How it
 * works). Returns 0 for rank <= 0. */
float lora_scale(float alpha, int32_t rank, int32_t rslora);

/* Learning rate at optimizer-update index `step` ("4.3. Training Guide", Schedules): constant,
 * or linear warmup base*(step+1)/warmup then cosine from base to min_lr over total - warmup
 * updates (progress clamped to 1). Returns NaN for an unknown kind. */
double lora_lr_at(int32_t kind, double base, uint64_t step, uint64_t warmup, uint64_t total,
                  double min_lr);

/* Workspace bytes for lora_forward / lora_backward on T tokens. */
size_t lora_workspace_size(const lora_desc* d, int64_t T);

/* ---- frozen-weight preparation (once per frozen W, not per step) ----------------------------*/
/* Bytes of the prepared copy of W that lora_prepare_weight writes (W is frozen, so this is made
 * once and kept resident beside W):
 *   bf16: W^T [in_dim, out_dim] bf16, the K-contiguous operand of the dX product
 *         (2 * in_dim * out_dim bytes);
 *   fp32: the bf16 split of W and of W^T for the split tensor-core products, four bf16 arrays
 *         [W_hi | W_lo | W^T_hi | W^T_lo], each element x stored as x_hi = x rounded to bf16
 *         (nearest even) and x_lo = (x - x_hi) rounded to bf16 (8 * in_dim * out_dim bytes);
 *   bf16 with the E4M3 frozen product: [W8 (out x in codes) | sw (out fp32 row scales) |
 *         WT8 (in x out codes of W's columns) | swT (in fp32)], each section starting on a
 *         16-byte boundary (about 2 * in_dim * out_dim bytes);
 *   LORA_BF16_BLK8: [W8 (out x in codes, row-major) | sw (ceil(out / 128) x ceil(in / 128) fp32)],
 *         the second section from byte in_dim * out_dim (a multiple of 256).
 * Returns 0 for an invalid descriptor. */
size_t lora_prepared_weight_size(const lora_desc* d);

/* Writes the prepared copy (above) of W [out_dim, in_dim] into W_prep (16-byte aligned, at least
 * lora_prepared_weight_size bytes). */
int lora_prepare_weight(const lora_desc* d, const void* W, void* W_prep, void* stream);

/* DoRA row norm n_o = || W_o + s (B A)_o ||_2 for the current A, B (fp32 [out_dim]); call once
 * per optimizer step before the first forward ("8. LoRA Fundamentals", How it works, and its
 * norm-refresh event). For bf16 W it is evaluated on tensor cores from the expanded form
 * ||W_o||^2 + 2 s (W A^T)_o . B_o + s^2 B_o (A A^T) B_o^T (the same quantity); scratch comes from
 * ws (at least lora_dora_norm_workspace_size bytes, 16-byte aligned). */
size_t lora_dora_norm_workspace_size(const lora_desc* d);
int lora_dora_norm(const lora_desc* d, const void* W, const float* A, const float* B,
                   float* norm_out, void* ws, size_t ws_bytes, void* stream);

/* ---- forward / backward (one adapted linear, T tokens) --------------------------------------*/
/* Y [T, out] = X W^T + Hs B^T, then * (dora_m / dora_n) per column in DoRA mode.
 * W is the frozen weight and W_prep its prepared copy (lora_prepare_weight); both are required
 * (the bf16 product reads W, the fp32 product reads W_prep).
 * H_save [T, rank] fp32 receives Hs = s' (Xd A^T) (the scaled shrink), which lora_backward
 * reads. dora_m, dora_n: [out] fp32, required iff desc.dora. */
int lora_forward(const lora_desc* d, const lora_ctx* c, int64_t T, const void* X, const void* W,
                 const void* W_prep, const float* A, const float* B, const float* dora_m,
                 const float* dora_n, void* Y, float* H_save, void* ws, size_t ws_bytes,
                 void* stream);

/* dX [T, in] = dY' W + (Gs A) * M with Gs = s' dY' B (written, may be NULL to skip dX);
 * dA [r, in] += Gs^T Xd; dB [out, r] += dY'^T H_save; dm [out] += sum_t dY * Y_save / m (DoRA).
 * W_prep from lora_prepare_weight. Y_save (the forward's Y) and dm are required iff desc.dora.
 * Accumulation over chunks is the caller's sequence of calls (or one call with chunk_tokens);
 * the token sums inside one call are reduced in a fixed order, so reruns are bitwise equal. */
int lora_backward(const lora_desc* d, const lora_ctx* c, int64_t T, const void* X,
                  const void* W_prep, const float* A, const float* B, const void* dY,
                  const float* H_save, const float* dora_m, const float* dora_n,
                  const void* Y_save, void* dX, float* dA, float* dB, float* dm, void* ws,
                  size_t ws_bytes, void* stream);

/* ---- grad prepare and AdamW over flat fp32 arenas -------------------------------------------*/
/* Workspace bytes for lora_grad_prepare over these groups. */
size_t lora_grad_prepare_workspace_size(int32_t n_groups, const lora_group* groups);

/* Pass 1 of the two-pass clip for each group: S_g = sum of squares of grads[offset, offset+n)
 * accumulated beyond float precision (exact float-float per-thread partials, summed in
 * float-float within a CTA and in double across CTAs; elements above 2^40 in magnitude go to a
 * double accumulator, so no finite gradient overflows), then
 *   status[g] = LORA_ERR_NONFINITE if any element is NaN or +-Inf, else LORA_OK;
 *   scale_norm[2g]   = c = gamma * max_norm / norm if max_norm > 0 and norm > max_norm, else gamma
 *   scale_norm[2g+1] = norm = gamma * sqrt(S_g)
 * d_scale_norm [2 * n_groups] double and d_status [n_groups] int32 are device outputs.
 * 1 <= n_groups <= LORA_MAX_GROUPS. Groups must not overlap. */
int lora_grad_prepare(const float* grads, int32_t n_groups, const lora_group* groups,
                      double* d_scale_norm, int32_t* d_status, void* ws, size_t ws_bytes,
                      void* stream);

/* Allocation-free lora_grad_prepare (the paper has no counterpart; this is a deployment aid).
 * For callers that cannot allocate device memory and so cannot supply a workspace: code that
 * runs under another framework's allocator which owns the whole device pool, code that must not
 * allocate after initialisation (allocation can stall or fail mid-training), and code that
 * enqueues work while some other component is capturing a CUDA graph, where a cudaMalloc would
 * break or poison the capture. Same arguments and results as lora_grad_prepare, minus the
 * workspace: the scratch is a fixed file-scope device array of LORA_NOALLOC_PREPARE_PARTIALS
 * doubles plus a counter (about 128 KB), which every GPU that loads the library holds until
 * process exit. The call allocates nothing (no cudaMalloc, cudaFree or allocating library call).
 *   - Size limit: sum over groups of ceil(elements / 16384) must be at most
 *     LORA_NOALLOC_PREPARE_PARTIALS (one group: at most 268,435,456 elements); larger requests
 *     return LORA_ERR_UNSUPPORTED with nothing enqueued.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress) with
 *     that device current; make that first call before any stream capture on that device.
 *   - All calls share the one array: calls that overlap on the GPU (other streams, other host
 *     threads) race and give wrong results; order them on one stream. The array keeps the last
 *     call's contents; each call clears the counter it needs before use. */
#define LORA_NOALLOC_PREPARE_PARTIALS 16384
int lora_grad_prepare_noalloc(const float* grads, int32_t n_groups, const lora_group* groups,
                              double* d_scale_norm, int32_t* d_status, void* stream);

/* Pass 2 fused with the AdamW update, for every group whose device status is LORA_OK (groups
 * with another status are left untouched: params, moments and grads):
 *   g_hat = c g; m = b1 m + (1-b1) g_hat; v = b2 v + (1-b2) g_hat^2; k = step + 1;
 *   u = (m / (1 - b1^k)) / (sqrt(v / (1 - b2^k)) + eps)
 *   A:   p -= lr u + lr wd p      B: p -= lr plus_ratio u      MAG: p -= lr u
 * zero_grads != 0 also clears the group's gradients after reading them. The caller advances
 * each group's step (and re-evaluates lr) only for groups whose status was LORA_OK. */
int lora_adamw_step(float* params, float* grads, float* m, float* v, int32_t n_groups,
                    const lora_group* groups, const lora_adamw_hp* hp, const double* d_scale_norm,
                    const int32_t* d_status, int32_t zero_grads, void* stream);

/* ---- frozen product over a block-scaled E4M3 base --------------------------------------------*/
/* A frozen weight kept as E4M3 codes W8 [out_dim, in_dim] (uint8, row-major) with one fp32 scale
 * for each 128 x 128 block, sw [ceil(out_dim / 128), ceil(in_dim / 128)] (blocks at the far edges
 * are partial): W~[o, i] = sw[o / 128, i / 128] * W8[o, i] ("LoRA Training and Serving", Quantized
 * rollout: an FP8 base under a bf16-trained adapter). The activations, bf16, are quantised inside
 * each call in blocks of 1 x 128 along the contraction: x8 = e4m3(x * r), r = 448 * (1 / amax),
 * sx = amax * (1 / 448) (codes to nearest even and saturated; fp32, each operation rounded;
 * r = sx = 1 where amax is 0 or r is not finite). Then
 *   forward     (transposed = 0)  Y [T, out_dim] = X W~^T,  X [T, in_dim]
 *   input grad. (transposed != 0) Y [T, in_dim]  = X W~,    X [T, out_dim]
 *   Y[t, n] = bf16( sum over blocks kb of sx[t, kb] sw[block of (n, kb)] sum_{k in kb} x8 w8 )
 * with each block's sum in fp32 on the tensor cores and the sum over blocks in fp32 registers.
 * Both directions read the same codes, so the gradient is that of the forward's weight, and one
 * copy of the weight serves both. A row of X holding a NaN or an infinity gives a NaN row of Y
 * and touches no other row. T from 1 (one decoded token) up; in_dim and out_dim multiples of 16
 * (LORA_ERR_ALIGN), T below 2^31 - 256 and dimensions at most 2^20 (LORA_ERR_UNSUPPORTED).
 * When lora_device_check reports LORA_ERR_TIMEOUT after it, an element of Y holds its value, is NaN or is
 * as it was. */
#define LORA_SCALE_BLOCK 128
size_t lora_block_product_workspace_size(int64_t T, int64_t out_dim, int64_t in_dim,
                                         int32_t transposed);
int lora_block_product(int64_t T, int64_t out_dim, int64_t in_dim, const void* X,
                       const uint8_t* W8, const float* sw, void* Y, int32_t transposed, void* ws,
                       size_t ws_bytes, void* stream);
/* Codes and block scales of a bf16 W [out_dim, in_dim] (once per frozen weight), by the rule above
 * over 128 x 128 blocks. */
int lora_block_quantize_weight(const void* W, int64_t out_dim, int64_t in_dim, uint8_t* W8,
                               float* sw, void* stream);
/* The activations' quantisation alone: codes [rows, K] and scales [rows, ceil(K / 128)] of a bf16
 * [rows, K] matrix. K % 16 == 0. */
int lora_block_quantize(const void* src, int64_t rows, int64_t K, uint8_t* codes, float* scales,
                        void* stream);

/* ---- layer norm in front of an adapted linear -------------------------------------------------*/
/* Rows of X [T, dim], dtype LORA_F32 or LORA_BF16; gamma, beta and their gradients fp32 [dim] (they
 * may live in an arena's magnitude range: no decay, plain learning rate).
 *   LORA_NORM_LAYER: mean = sum x / dim, var = sum (x - mean)^2 / dim
 *   LORA_NORM_RMS:   mean = 0,           var = sum x^2 / dim          (beta must be NULL)
 *   rstd = 1 / sqrt(var + eps),  xhat = (x - mean) rstd
 *   forward   Y = gamma xhat + beta;  stats [T, 2] fp32 = (mean, rstd), which the backward reads
 *   backward  g = gamma dY;  dX = rstd (g - [LAYER: sum g / dim] - xhat (sum g xhat) / dim) + dX_add
 *             dgamma += sum_t dY xhat;  dbeta += sum_t dY
 * All arithmetic in fp32 from registers (the variance is of the centred values), outputs rounded
 * once. beta may be NULL (no shift); dX_add [T, dim] (the residual branch's gradient) may be NULL
 * and may be dX itself; dgamma, dbeta and dX may be NULL each (not all). The token sums are
 * reduced in a fixed order: reruns are bitwise equal. dim a multiple of 8 (LORA_ERR_ALIGN) and at
 * most LORA_NORM_MAX_DIM, T below 2^31 - 256 (LORA_ERR_UNSUPPORTED); T = 0 is a no-op.
 * When lora_device_check reports LORA_ERR_TIMEOUT after a backward pass, rows of dX may be as they were
 * and dgamma and dbeta are NaN (which lora_grad_prepare rejects), never sums that lack rows. */
#define LORA_NORM_LAYER 0
#define LORA_NORM_RMS 1
#define LORA_NORM_MAX_DIM 16384
typedef struct lora_norm_desc {
  int64_t dim;
  int32_t kind;        /* LORA_NORM_LAYER | LORA_NORM_RMS */
  int32_t dtype;       /* LORA_F32 | LORA_BF16 for X, Y, dY, dX */
  float eps;           /* >= 0 */
} lora_norm_desc;
int lora_norm_forward(const lora_norm_desc* d, int64_t T, const void* X, const float* gamma,
                      const float* beta, void* Y, float* stats, void* stream);
size_t lora_norm_backward_workspace_size(const lora_norm_desc* d, int64_t T);
int lora_norm_backward(const lora_norm_desc* d, int64_t T, const void* X, const float* gamma,
                       const void* dY, const float* stats, const void* dX_add, void* dX,
                       float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream);

/* The gradients of several projections that read the norm's output, for its backward pass:
 *   dst[i] = sum_k src[k][i], k = 0 .. n - 1 in order, in fp32, rounded once to dtype
 * (LORA_F32 or LORA_BF16). src is a host array of n device pointers, 1 <= n <= LORA_SUM_MAX
 * (LORA_ERR_UNSUPPORTED above); count elements each, a multiple of 8 (LORA_ERR_ALIGN); dst may be one
 * of them; count = 0 is a no-op. */
#define LORA_SUM_MAX 16
int lora_sum(int32_t n, const void* const* src, int64_t count, int32_t dtype, void* dst, void* stream);

/* ---- between an attention block's projections --------------------------------------------------*/
/* Norm of each query and key head and rotation by position, in one pass. For the head vector x of a
 * token at position n (pairs (a, b) of elements: LORA_ROPE_HALVES element i with i + head_dim / 2,
 * LORA_ROPE_PAIRS element 2 i with 2 i + 1; c, s = table[n, i]):
 *   r = 1 / sqrt(sum x^2 / head_dim + eps),  xhat = x r,  h = gamma xhat      (gamma NULL: h = x)
 *   forward   y: (a, b) -> (a c - b s, a s + b c) of h
 *   backward  h' = dy turned back (s -> -s);  dgamma += sum over tokens and heads of h' xhat
 *             g = gamma h';  dx = r (g - xhat (sum g xhat) / head_dim)       (gamma NULL: dx = h')
 * Q [T, q_heads, head_dim] and K [T, k_heads, head_dim] (k_heads may be 0: K and its outputs are not
 * read) with ld_q, ld_k elements from token to token, so that both may be columns of a fused
 * projection's output; dQ and dK have the same strides, YQ, YK, dYQ, dYK have ld_yq, ld_yk. A stride of
 * 0 stands for heads * head_dim. gamma_q, gamma_k and their gradients fp32 [head_dim]; gamma_q and
 * gamma_k are both given or both NULL, and without them the backward pass does not read Q and K (which
 * may be NULL) and takes no gradients of them. dgamma_q and dgamma_k may be NULL each, and the same array where
 * both norms share a weight (the queries' sum is added first). pos int32 [T] on
 * the device: a token with a negative position is padding, its rows are left as they were and it adds
 * nothing to the gradients; a position from n_pos on gives NaN. table fp32 [n_pos, head_dim / 2, 2]
 * (cosine, sine), 16-byte aligned. An output may be an input of the same strides (one decoded token in
 * place). Sums in fp32, outputs rounded once, the gradients' sums in a fixed order: reruns are bitwise
 * equal. head_dim 64, 128 or 256, at most 2^13 heads in all, T below 2^31 - 256 and n_pos at most 2^24
 * (LORA_ERR_UNSUPPORTED); strides multiples of 16 bytes (LORA_ERR_ALIGN); T = 0 is a no-op. */
#define LORA_ROPE_HALVES 0
#define LORA_ROPE_PAIRS 1
typedef struct lora_rope_desc {
  int32_t q_heads;
  int32_t k_heads;
  int32_t head_dim;
  int32_t dtype;       /* LORA_F32 | LORA_BF16 */
  int32_t layout;      /* LORA_ROPE_HALVES | LORA_ROPE_PAIRS */
  float eps;           /* >= 0 */
  int64_t ld_q, ld_k, ld_yq, ld_yk;
} lora_rope_desc;
/* table[n, i] = (cos, sin)(n inv_freq[i]) for n < n_pos, the angles in double (inv_freq: device
 * doubles [head_dim / 2], 16-byte aligned), rounded to fp32 once. */
int lora_rope_table(int64_t n_pos, int32_t head_dim, const double* inv_freq, float* table, void* stream);
int lora_rope_forward(const lora_rope_desc* d, int64_t T, const void* Q, const void* K,
                      const float* gamma_q, const float* gamma_k, const int32_t* pos,
                      const float* table, int64_t n_pos, void* YQ, void* YK, void* stream);
size_t lora_rope_backward_workspace_size(const lora_rope_desc* d, int64_t T);
int lora_rope_backward(const lora_rope_desc* d, int64_t T, const void* Q, const void* K,
                       const float* gamma_q, const float* gamma_k, const int32_t* pos,
                       const float* table, int64_t n_pos, const void* dYQ, const void* dYK, void* dQ,
                       void* dK, float* dgamma_q, float* dgamma_k, void* ws, size_t ws_bytes,
                       void* stream);

/* Causal attention over packed sequences with grouped heads. Sequence k covers tokens
 * [seq_start[k], seq_start[k + 1]); query head h reads key / value head h / (q_heads / kv_heads):
 *   S[i, j] = scale q_i . k_j for j <= i of the same sequence,  lse_i = log sum_j exp S[i, j]
 *   forward   P = exp(S - lse),  o_i = sum_j P[i, j] v_j
 *   backward  (from q, k, v, o, lse and do)  delta_i = do_i . o_i,
 *             dS[i, j] = P[i, j] (do_i . v_j - delta_i),
 *             dv_j = sum_i P[i, j] do_i,  dk_j = scale sum_i dS[i, j] q_i,  dq_i = scale sum_j dS[i, j] k_j
 *             (dk and dv summed over the query heads of their group)
 * Q, O, dO, dQ [T, q_heads, head_dim] and K, V, dK, dV [T, kv_heads, head_dim], bf16, with ld_q (Q and
 * dQ), ld_k, ld_v, ld_o (O and dO) elements from token to token (0: heads * head_dim), so that all may be
 * columns of wider buffers; lse fp32 [q_heads, T]. Tokens behind the last sequence (and between two) are
 * padding: their rows of the outputs are left as they were and no other row depends on theirs, whatever
 * they hold. A NaN or infinity within a sequence may reach any row of that sequence.
 * Products on tensor cores with fp32 sums; scores, statistics and the softmax in fp32; P and dS are
 * rounded to bf16 (2^-8 of each) as operands of the second products, everything else once at the end. No
 * atomics: reruns are bitwise equal.
 * q_heads a multiple of kv_heads, strides at least heads * head_dim (LORA_ERR_INVALID) and multiples of 8
 * elements (LORA_ERR_ALIGN); head_dim 64 or 128, dtype LORA_BF16, heads * head_dim at most 2^20 and T below
 * 2^31 - 256 (LORA_ERR_UNSUPPORTED); T = 0 is a no-op. Outputs do not overlap inputs.
 * When lora_device_check reports LORA_ERR_TIMEOUT after it, an element of an output holds its value or
 * is as it was. */
typedef struct lora_attn_desc {
  int32_t q_heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t dtype;       /* LORA_BF16 */
  float scale;         /* > 0, usually 1 / sqrt(head_dim) */
  int64_t ld_q, ld_k, ld_v, ld_o;
} lora_attn_desc;
/* The tiles of a batch, longest first, from the sequences' table (device int32 [n_seq + 1],
 * non-decreasing, within [0, T]; offsets outside are clamped, and a sequence that would begin before the
 * end of an earlier one begins there). One plan, in a caller-owned device buffer of
 * lora_attn_plan_size(T, n_seq) bytes, 16-byte aligned, serves every layer's forward and backward calls
 * over the same batch, on any streams ordered after the build; these pass the same T and n_seq (with others
 * they find no tiles and write nothing). n_seq from 1 to 2^24. One launch. */
size_t lora_attn_plan_size(int64_t T, int32_t n_seq);
int lora_attn_plan_build(int64_t T, int32_t n_seq, const int32_t* d_seq_start, void* plan,
                         size_t plan_bytes, void* stream);
int lora_attn_forward(const lora_attn_desc* d, int64_t T, int32_t n_seq, const void* plan,
                      const void* Q, const void* K, const void* V, void* O, float* lse, void* stream);
size_t lora_attn_backward_workspace_size(const lora_attn_desc* d, int64_t T);
int lora_attn_backward(const lora_attn_desc* d, int64_t T, int32_t n_seq, const void* plan,
                       const void* Q, const void* K, const void* V, const void* O, const float* lse,
                       const void* dO, void* dQ, void* dK, void* dV, void* ws, size_t ws_bytes,
                       void* stream);

/* ---- orthogonalised update (in place of lora_adamw_step for the adapter matrices) -------------*/
/* One matrix of the flat arenas, [rows, cols] row-major from element `offset` (a multiple of 4).
 * The smaller side is at most LORA_MAX_RANK and a multiple of 4. `group` indexes the call's groups
 * and the matrix lies inside that group's range; its kind decides the decay and the LoRA+ ratio. */
#define LORA_KIND_A 0
#define LORA_KIND_B 1
typedef struct lora_mat {
  int64_t offset;
  int64_t rows;
  int64_t cols;
  int32_t group;
  int32_t kind;        /* LORA_KIND_A | LORA_KIND_B */
} lora_mat;

#define LORA_MUON_ADJUST_ASPECT 0   /* s = sqrt(max(1, rows / cols)) */
#define LORA_MUON_ADJUST_RMS 1      /* s = 0.2 sqrt(max(rows, cols)): Adam's usual update RMS */
typedef struct lora_muon_hp {
  double momentum;      /* mu, 0.95 */
  double weight_decay;  /* applied to kind A only */
  double plus_ratio;    /* LoRA+: B's lr = lr * plus_ratio */
  double coef[3];       /* a, b, c of the Newton-Schulz step (3.4445, -4.7750, 2.0315) */
  int32_t steps;        /* Newton-Schulz steps, 1 .. 8 (5) */
  int32_t nesterov;     /* 1: u = c g + mu m, 0: u = m */
  int32_t adjust;       /* LORA_MUON_ADJUST_* */
} lora_muon_hp;

/* For every matrix whose group's device status is LORA_OK (others are left untouched):
 *   m = mu m + c g  (c = d_scale_norm[2 * group], from lora_grad_prepare);  u as above
 *   X = u / ||u||_F (0 where u is 0);  `steps` times: X <- (a I + b G + c G^2) X, G = X X^T over the
 *   smaller side
 *   A: p -= lr s X + lr wd p      B: p -= lr plus_ratio s X       (p before the update in the decay)
 * lr is the group's; zero_grads != 0 clears the matrices' gradients after reading them. Elements
 * of the arenas outside the matrices (DoRA magnitudes, norm weights) are not touched: give them
 * to lora_adamw_step in a group of their own. Matrices must not overlap; any number of them.
 * Precision: momentum, norms and sums in fp32. Up to a smaller side of 16 everything is fp32. Above, the
 * long products run on tensor cores: u, X between stages of at most three steps and a stage's polynomial
 * are held as two bf16 terms (16 significant bits where max |u| is at least 2^-116), the small matrices
 * are multiplied as two-term tf32 splits (about 2^-21). X is then within (2 stages + 1) 2^-16 of the
 * sequence's largest gain, in the Frobenius norm; the parameters of a rank-64 update came out 2.4e-7 off
 * in relative 2-norm, those of fp32 torch operations 6e-8.
 * When lora_device_check reports LORA_ERR_TIMEOUT after it, every element of the parameters holds its
 * update or is as it was; m (and the gradients, where they are cleared) may be those of either. */
size_t lora_muon_workspace_size(int32_t n_mats, const lora_mat* mats);
int lora_muon_step(float* params, float* grads, float* m, int32_t n_groups,
                   const lora_group* groups, int32_t n_mats, const lora_mat* mats,
                   const lora_muon_hp* hp, const double* d_scale_norm, const int32_t* d_status,
                   int32_t zero_grads, void* ws, size_t ws_bytes, void* stream);

/* ---- fused projections ----------------------------------------------------------------------*/
/* Projections that read one input (q/k/v, gate/up) run as one fused linear: one frozen product
 * over the stacked weight W_cat = [W_0; W_1; ...] ([sum out_k, in]) and one output
 * Y_cat [T, sum out_k] whose columns [off_k, off_k + out_k) (off_k = out_0 + ... + out_{k-1})
 * are projection k's, while every projection keeps its own adapter ("LoRA Training and Serving",
 * --lora-type: fused projections, and canonical adapters per q/k/v and gate/up projection):
 *   Y_k = X W_k^T + s' (Xd A_k^T) B_k^T,   dX = sum_k (dY_k W_k + s' (G_k A_k) * M),
 *   dA_k += s' G_k^T Xd,  dB_k += s' dY_k^T (Xd A_k^T),  G_k = dY_k B_k.
 * desc: in_dim, out_dim = sum out_k, the shared rank and scale, dtype LORA_BF16 or LORA_F32, no
 * DoRA; one dropout mask (desc.layer_id / proj_id) for all the projections;
 * 1 <= n_proj <= LORA_MAX_SLOTS. LORA_BF16: every out_k is a multiple of 256. LORA_F32:
 * n_proj * rank <= LORA_MAX_RANK (the group runs as one adapter of that rank whose up-projection
 * is block-diagonal). LORA_ERR_UNSUPPORTED otherwise. W_prep is lora_prepare_weight of W_cat
 * (desc above); the forward reads W (bf16) or W_prep (fp32), as lora_forward does.
 * H_save [T, n_proj * rank] fp32 holds Hs_k = s' Xd A_k^T in columns k rank .. k rank + rank - 1.
 * dX may be NULL. */
typedef struct lora_proj {
  const float* A;   /* [rank, in_dim] */
  const float* B;   /* [out_dim, rank] */
  float* dA;        /* [rank, in_dim], accumulated (+=) by lora_fused_backward */
  float* dB;        /* [out_dim, rank], accumulated (+=) */
  int64_t out_dim;  /* out_k */
} lora_proj;
size_t lora_fused_workspace_size(const lora_desc* d, int64_t T, int32_t n_proj,
                                 const lora_proj* projs);
int lora_fused_forward(const lora_desc* d, const lora_ctx* c, int64_t T, const void* X,
                       const void* W, const void* W_prep, int32_t n_proj, const lora_proj* projs,
                       void* Y, float* H_save, void* ws, size_t ws_bytes, void* stream);
int lora_fused_backward(const lora_desc* d, const lora_ctx* c, int64_t T, const void* X,
                        const void* W_prep, int32_t n_proj, const lora_proj* projs,
                        const void* dY, const float* H_save, void* dX, void* ws, size_t ws_bytes,
                        void* stream);

/* ---- adapter-state maintenance --------------------------------------------------------------*/
/* Snapshot, restore and retirement of adapter state over the groups' ranges
 * [offset, offset + n_a + n_b + n_mag) of the flat fp32 arenas ("4.3. Training Guide",
 * Validation early stopping: the best A/B are snapshotted, restored on exit, and the optimizer
 * is reset after the restore; "Multi-LoRA Training Example", a finished adapter is retired:
 * its slot cleared, its optimizer state and retained gradients zeroed, its partially
 * accumulated gradients discarded). All arrays are device fp32 with the arenas' layout and
 * 16-byte aligned; only the groups' ranges are read or written. Asynchronous on `stream`;
 * groups are checked as for lora_grad_prepare (LORA_ERR_INVALID / LORA_ERR_ALIGN before any
 * launch), a launch failure gives LORA_ERR_CUDA.
 *
 * lora_snapshot: snap = params.
 * lora_restore:  params = snap, m = v = 0, and grads = 0 when zero_grads != 0. The caller
 *                restarts each group's update count (lora_group.step = 0 on its next
 *                lora_adamw_step), which completes the optimizer reset.
 * lora_retire:   grads = m = v = 0, and params = 0 when clear_params != 0. The caller resets
 *                the slots' accumulated sample counts and update counts on the host. */
int lora_snapshot(const float* params, float* snap, int32_t n_groups, const lora_group* groups,
                  void* stream);
int lora_restore(float* params, const float* snap, float* grads, float* m, float* v,
                 int32_t n_groups, const lora_group* groups, int32_t zero_grads, void* stream);
int lora_retire(float* params, float* grads, float* m, float* v, int32_t n_groups,
                const lora_group* groups, int32_t clear_params, void* stream);

/* ---- slot-keyed multi-LoRA ------------------------------------------------------------------*/
/* Segments: segment k covers tokens [seg_start[k], seg_start[k+1]) (device int32 [n_seg + 1],
 * non-decreasing, within [0, T]) and uses slot seg_slot[k] (device int32 [n_seg]). Tokens in no
 * segment, or in a segment whose slot id is outside [0, n_slots), get no adapter (frozen output
 * only). `slots` is a host array of n_slots entries (1 <= n_slots <= LORA_MAX_SLOTS); desc.rank
 * is the largest slot rank and the row stride of H_save. desc.dora must be 0. */
size_t multi_lora_workspace_size(const lora_desc* d, int64_t T, int32_t n_seg, int32_t n_slots,
                                 const lora_slot* slots);

int multi_lora_forward(const lora_desc* d, const lora_ctx* c, int64_t T, const void* X,
                       const void* W, const void* W_prep, int32_t n_seg,
                       const int32_t* d_seg_start, const int32_t* d_seg_slot, int32_t n_slots,
                       const lora_slot* slots, void* Y, float* H_save, void* ws, size_t ws_bytes, void* stream);

/* dX may be NULL. Each slot's dA/dB accumulate that slot's tokens with weight 1; per-slot
 * 1/adapter_global_batch_size, clip and Adam are lora_grad_prepare / lora_adamw_step with one
 * group per ready slot. */
int multi_lora_backward(const lora_desc* d, const lora_ctx* c, int64_t T, const void* X,
                        const void* W_prep, int32_t n_seg, const int32_t* d_seg_start,
                        const int32_t* d_seg_slot, int32_t n_slots, const lora_slot* slots,
                        const void* dY, const float* H_save, void* dX, void* ws,
                        size_t ws_bytes, void* stream);

/* Routing plan. Every routed call over the same batch (T, segments, slots: the same token
 * routing for every projection and layer, "Multi-LoRA Training Example", Design: slot-keyed
 * page table, one routing per batch) needs the same token work tables: the row products' token
 * items, the token reductions' runs and the slot set of every 128-token tile. A plan holds them
 * in a caller-owned device buffer of multi_lora_plan_size(T, n_seg, n_slots) bytes (0 for bad
 * arguments), 16-byte aligned. multi_lora_plan_build fills it from the segment table (the same
 * rules as multi_lora_forward; three launches on `stream`); the *_planned calls take
 * (T, n_seg, plan) in place of the segment table, read the plan on their own stream and build
 * nothing, so any number of calls, on any streams ordered after the build, may share one plan.
 * A plan stays valid until the caller rewrites its buffer; its contents depend on
 * (T, n_seg, n_slots) and the segment table only, so a planned call passes the same T, n_seg and
 * n_slots as the build. Results are bit-identical to the unplanned calls. Errors: LORA_ERR_INVALID
 * (null pointers, n_seg < 1, n_slots outside 1..LORA_MAX_SLOTS), LORA_ERR_ALIGN,
 * LORA_ERR_WORKSPACE (plan_bytes too small), LORA_ERR_UNSUPPORTED (T above 2^31 - 257), then
 * the checks of multi_lora_forward / multi_lora_backward. */
size_t multi_lora_plan_size(int64_t T, int32_t n_seg, int32_t n_slots);
int multi_lora_plan_build(int64_t T, int32_t n_seg, const int32_t* d_seg_start,
                          const int32_t* d_seg_slot, int32_t n_slots, void* plan, size_t plan_bytes,
                          void* stream);
int multi_lora_forward_planned(const lora_desc* d, const lora_ctx* c, int64_t T, int32_t n_seg,
                               const void* plan, const void* X, const void* W, const void* W_prep,
                               int32_t n_slots, const lora_slot* slots, void* Y, float* H_save,
                               void* ws, size_t ws_bytes, void* stream);
int multi_lora_backward_planned(const lora_desc* d, const lora_ctx* c, int64_t T, int32_t n_seg,
                                const void* plan, const void* X, const void* W_prep,
                                int32_t n_slots, const lora_slot* slots, const void* dY,
                                const float* H_save, void* dX, void* ws, size_t ws_bytes,
                                void* stream);

/* ---- test hooks (not part of the timed path) ------------------------------------------------*/
/* Keep mask M [T, in_dim] as uint8 (1 = kept), exactly as the kernels regenerate it. */
/* Test hook: the per-row E4M3 quantisation of LORA_BF16_FP8 (see its definition) applied to a bf16
 * [rows, K] matrix: codes [rows, K] uint8 and scales [rows] fp32. K % 16 == 0, K <= 16384. */
int lora_quantize_e4m3(const void* src, int64_t rows, int64_t K, uint8_t* codes, float* scales,
                       void* stream);
int lora_dropout_mask(const lora_desc* d, const lora_ctx* c, int64_t T, uint8_t* d_mask,
                      void* stream);

/* Slot of every token (int32 [T], -1 = no adapter) under the segment rules above. */
int multi_lora_token_slots(int64_t T, int32_t n_seg, const int32_t* d_seg_start,
                           const int32_t* d_seg_slot, int32_t n_slots, int32_t* d_token_slot,
                           void* stream);

/* ---- instrumentation (benchmark and tests; not part of the method) -------------------------*/
/* Kernel classes for lora_profile_arm. */
#define LORA_PROF_NONE 0
#define LORA_PROF_FROZEN_FWD 1   /* frozen forward product with the fused up-projection */
#define LORA_PROF_FROZEN_DX 2    /* frozen dX product with the fused LoRA dX term */
#define LORA_PROF_SHRINK 3       /* Hs = s' Xd A^T */
#define LORA_PROF_G 4            /* Gs = s' dY' B */
#define LORA_PROF_RED_DB 5       /* dB token reduction */
#define LORA_PROF_RED_DA 6       /* dA token reduction */
#define LORA_PROF_PREPARE 7      /* grad-prepare pass 1 */
#define LORA_PROF_ADAMW 8        /* fused clip + AdamW */
#define LORA_PROF_RED 9          /* dB and dA token reductions in one launch */

/* Arm event brackets: the next n launches of `kernel_class` record start_events[i] before and
 * stop_events[i] after launch i on the launching stream (cudaEvent_t handles, caller-owned).
 * Re-arming replaces the previous set; n == 0 disarms. Under stream capture the records become
 * graph nodes and fire on every replay. Not thread-safe with concurrent arming. */
int lora_profile_arm(int32_t kernel_class, void* const* start_events, void* const* stop_events,
                     int32_t n);
/* How many armed brackets have been used so far. */
int32_t lora_profile_used(void);
/* Kernel launches enqueued by this library since it was loaded (all classes). */
uint64_t lora_launch_counter(void);
/* Text of the last CUDA error an entry point of this library reported as LORA_ERR_CUDA in the
 * calling thread ("no error" if none). */
const char* lora_last_cuda_error(void);
/* Error bits raised on the device by the tensor-core kernels when a pipeline wait ran out of
 * its bound (bit 0 loads, bit 1 MMA, bit 2 epilogue): the kernel then skipped its remaining
 * work, released its tensor memory and returned, so the output is invalid. Synchronous (reads
 * a device word of the current device); reset != 0 clears it. */
int lora_device_error(uint32_t* flags, int32_t reset);
/* Synchronises `stream`, then reports the device error word: LORA_ERR_TIMEOUT if any bit is set
 * (left set for lora_device_error), LORA_ERR_CUDA if the stream holds a CUDA error, else LORA_OK.
 * This is how a caller learns, after the fact, that an asynchronous call's outputs are invalid
 * because one of its kernels gave up waiting and returned early (no hang, the context stays
 * usable). The bound of each wait guards against a pipeline that can no longer make progress
 * ("4.3. Training Guide", Gradient clipping: a bad step is detected and rejected before any
 * state changes; here the same rule for a stalled kernel). */
int lora_device_check(void* stream);
/* Test hook: bound, in SM clock cycles, of the pipeline waits of the frozen-product kernels
 * (bf16 and E4M3), the norms' backward pass, the attention and the orthogonalised update launched after this call;
 * 0 restores the default (2^33 cycles, seconds).
 * Process-wide, not thread-safe with concurrent launches. A small bound makes a correct launch
 * give up: its error bits are set and its outputs are invalid. Waits that drain work already
 * issued (copies in flight, MMAs before the tensor memory is freed) keep the default bound, so
 * a kernel that gives up still leaves nothing running behind it. */
int lora_set_wait_limit(uint64_t cycles);

#ifdef __cplusplus
}
#endif

#endif /* LORA_GB300_H */
