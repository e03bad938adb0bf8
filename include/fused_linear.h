/*
 * fused_linear.h — C ABI of the B200 (sm_100a) fused linear layer
 *
 *     y = ((act(A·Wᵀ + bias)) + residual) · scale        (one kernel launch)
 *
 * Sources (web pages on GEMM epilogue fusion, cited by title and section):
 *   [epilog] "通过 cuBLASLt 的 epilog 机制实现单内核偏置融合：参数配置与性能收益"
 *            — the Matmul → plan(epilog, epilog_inputs{"bias"}) → execute → free
 *            statement of the problem; compute_type; the RELU_BIAS / GELU_BIAS /
 *            RELU_AUX_BIAS epilogs; bias shape = the result's output-feature
 *            dimension; inputs must outlive execute().
 *   [gelu]   zwxr.cn/news/294525 "Linear+GELU 算子融合" — §1/§2.1 exact GELU,
 *            §2.2.2 tanh form (0.044715), §3.1 the unfused GEMM-then-GELU design.
 *   [mlp]    "PyTorch MLP 核算子融合：從 nn.Linear 到 Fused MLP" — nn.Linear is
 *            x·Wᵀ + bias with W stored [out, in]; the GeGLU MLP gelu(g)*u.
 *   [mhc]    mhpn.cn/news/2504128 "mHC 融合" — §2.2 elementwise chain (bias,
 *            residual add, multiply by a constant), §3.3 GEMM-epilogue fusion.
 *
 * Conventions shared by every entry point
 *   - All pointers are DEVICE pointers of the current CUDA device except the
 *     out-parameter of fl_plan and the descriptor struct (host).
 *   - Matrices are row-major with an explicit leading dimension in ELEMENTS
 *     (0 = packed).  Every row pitch must be a multiple of 16 bytes and every
 *     base pointer 16-byte aligned (the tensor-memory-accelerator rule);
 *     otherwise FL_ERR_ALIGNMENT.  Logical extents may be ragged.
 *   - The caller owns every buffer and the stream.  Calls are asynchronous and
 *     stream-ordered; buffers must stay alive and unmodified until the stream
 *     has been synchronised ([epilog]: epilog inputs must outlive execute()).
 *   - Nothing aborts.  Every call returns an fl_status; on failure a message
 *     is available from fl_last_error() (thread-local, valid until the next
 *     call on that thread).  There is no CPU fallback: without a B200 the
 *     calls that launch kernels return FL_ERR_CUDA / FL_ERR_UNSUPPORTED.
 */
#ifndef FUSED_LINEAR_H_
#define FUSED_LINEAR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FL_OK = 0,
  FL_ERR_INVALID_ARG = 1,  /* null pointer, bad size, bad enum, missing operand */
  FL_ERR_UNSUPPORTED = 2,  /* combination not offered (e.g. a 16-bit accumulate) */
  FL_ERR_ALIGNMENT = 3,    /* pointer or row pitch not 16-byte aligned */
  FL_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed (message has the text) */
  FL_ERR_OOM = 5,          /* plan workspace allocation failed */
  FL_ERR_TIMEOUT = 6,      /* a bounded in-kernel wait gave up (see fl_check_status) */
  FL_ERR_DEVICE = 7        /* no usable sm_100 device */
} fl_status;

/* Storage types of operands and results. */
typedef enum { FL_F16 = 0, FL_BF16 = 1, FL_F32 = 2 } fl_dtype;

/* Compute type ([epilog] compute_type).  Accumulation is always FP32; the
 * pages warn against a 16-bit accumulate, so none is offered.
 *   FL_COMPUTE_32F        fp16/bf16 operands, fp32 accumulate (tensor cores).
 *   FL_COMPUTE_32F_3XTF32 fp32 operands, each split hi+lo into TF32 and
 *                         multiplied as hi·hi + hi·lo + lo·hi, fp32 accumulate. */
typedef enum { FL_COMPUTE_32F = 0, FL_COMPUTE_32F_3XTF32 = 1 } fl_compute;

/* Epilogue kinds ([epilog] MatmulEpilog; [gelu] exact/tanh GELU; [mlp] GeGLU).
 *   NONE            y = acc
 *   BIAS            y = acc + bias
 *   RELU_BIAS       y = max(acc + bias, 0)
 *   RELU_AUX_BIAS   as RELU_BIAS, and aux bit (m,n) = (acc + bias > 0)
 *   GELU_BIAS       y = gelu_erf(acc + bias)   = 0.5·v·(1 + erf(v/√2))
 *   GELU_TANH_BIAS  y = gelu_tanh(acc + bias)  = 0.5·v·(1 + tanh(√(2/π)(v + 0.044715 v³)))
 *   GEGLU_TANH      W is the stacked [2N, K] matrix [Wg; Wu]; y = gelu_tanh(A·Wgᵀ)·(A·Wuᵀ)
 *   GELU_SIGMOID_BIAS y = v·σ(1.702·v), the sigmoid approximation of GELU ([gelu] §2.2.2)
 *   GELU_AUX_BIAS   as GELU_BIAS, and aux = v = acc + bias stored in the output type, the
 *                   input of the GELU backward (fl_dgelu_bgrad); [epilog] keeps forward
 *                   state for the backward pass, [gelu] §2.2.1 fuses the backward too
 * Every kind up to here may add a residual and scale: y = (act(v) + residual)·scale.
 *
 * The gated feed-forward block in training ([mlp] gives its forward; no backward on the pages).
 * act is x·σ(x) (SWIGLU) or the tanh GELU (GEGLU); 16-bit operands and results:
 *   SWIGLU          W is the stacked [2N, K] matrix [Wg; Wu]; y = act(A·Wgᵀ)·(A·Wuᵀ)
 *   GEGLU_TANH_AUX, SWIGLU_AUX
 *                   the same, and aux = [A·Wgᵀ, A·Wuᵀ] stored as [M, 2N] (packed) in the output
 *                   type; N a multiple of 8
 *   DGEGLU_TANH, DSWIGLU
 *                   the backward through the gate, fused into the product that brings the
 *                   gradient: A = dy [M, K], W = the down projection's weight stored [K, N]
 *                   (b_major 1), aux = the forward's [M, 2N], read only; with dh = A·W, which is
 *                   never rounded below fp32 (and stays on the chip but for K splits, whose fp32
 *                   partial sums pass through the workspace), out [M, ldo], ldo ≥ 2N (0: 2N), is
 *                   [dh·u·act'(g), dh·act(g)]; N a multiple of 8.  out may be aux's own buffer
 *                   when ldo is 2N.  (The gradient of the block's input is then the NONE layer
 *                   out·[Wg; Wu] with b_major 1 and 2N as its K.)
 *   WGRAD           a weight gradient, y = (Aᵀ·W + residual)·scale: A stored [K, M] (lda ≥ M), W
 *                   stored [K, N] (b_major 1), K the number of tokens, any out_dtype.  The
 *                   residual (has_residual) is an earlier gradient to add to; it may be out's own
 *                   buffer, with the same type and pitch.  Sums are in fp32, in an order that
 *                   depends on the shape and the GPU alone.
 *                   The tensor cores' accumulators round towards zero, which shrinks a sum by 1e-9 of its
 *                   norm for each token.  So sums are taken in runs, and the runs rounded to nearest: of
 *                   896 tokens for fp32 results, an error of 9e-7 of the result's norm (1.1e-6 with f16
 *                   operands) whatever the tokens (random data); of 8192 for f16 and
 *                   65536 for bf16 results, shrunk by 8e-6 and 7e-5, near a twentieth of what
 *                   rounding to these types costs.
 * The sums over K of the gated kinds run in one accumulator each (several for K splits and few rows): they
 * are shrunk by 1e-9 of their norm for each k, 4e-6 at K = 4096, where rounding to f16 costs 2e-4.
 * GEGLU_TANH takes the hardware's tanh (relative error 2^-11), GEGLU_TANH_AUX and DGEGLU_TANH x·σ(y) in
 * fp32 precision, so that h may differ in its last bits between serving and training.
 * These take no bias, no unfused twin, FL_SCHED_AUTO only, and, but for WGRAD, no residual and no
 * scale. */
typedef enum {
  FL_EPI_NONE = 0,
  FL_EPI_BIAS = 1,
  FL_EPI_RELU_BIAS = 2,
  FL_EPI_RELU_AUX_BIAS = 3,
  FL_EPI_GELU_BIAS = 4,
  FL_EPI_GELU_TANH_BIAS = 5,
  FL_EPI_GEGLU_TANH = 6,
  FL_EPI_GELU_AUX_BIAS = 7,
  FL_EPI_GELU_SIGMOID_BIAS = 8,
  FL_EPI_SWIGLU = 9,
  FL_EPI_GEGLU_TANH_AUX = 10,
  FL_EPI_SWIGLU_AUX = 11,
  FL_EPI_DGEGLU_TANH = 12,
  FL_EPI_DSWIGLU = 13,
  FL_EPI_WGRAD = 14
} fl_epi_kind;

/* The "epilog" argument of fl_plan.  Zero-initialise, then set fields. */
typedef struct {
  int32_t kind;            /* fl_epi_kind */
  int32_t out_dtype;       /* fl_dtype of y */
  int32_t bias_dtype;      /* fl_dtype of bias (ignored for NONE / GEGLU_TANH) */
  int32_t residual_dtype;  /* fl_dtype of residual (when has_residual) */
  int32_t bias_axis;       /* 0: bias[n], per output column of A·Wᵀ (nn.Linear);
                              1: bias[m], per row — [epilog]'s W·x example, where the
                              output features are the result's first dimension */
  int32_t has_residual;    /* 1: add residual[m,n] after the activation */
  float scale;             /* multiply after the residual; 0 is read as 1 */
  int32_t b_major;         /* 0: W stored [N,K] (K contiguous, nn.Linear weight);
                              1: second operand stored [K,N] (N contiguous, [epilog]'s x) */
  int64_t lda, ldb, ldo, ldr; /* leading dimensions in elements, 0 = packed */
  int32_t unfused;         /* 1: bare GEMM into a plan-owned buffer, then one
                              elementwise kernel per epilogue step — the unfused
                              design of [gelu] §3.1, kept only to measure the
                              round trip that fusion removes */
  int32_t schedule;        /* fl_schedule: how CTA pairs share the output tiles */
  int32_t reserved[2];     /* must be 0 */
} fl_epilogue_desc;

/* Work schedule of the CTA-pair layouts (16-bit operands, M > 128). */
typedef enum {
  FL_SCHED_AUTO = 0,         /* the library's choice: whole tiles (stream-K measured no faster) */
  FL_SCHED_DATA_PARALLEL = 1,/* whole tiles only, each pair takes tiles p, p+pairs, ... */
  FL_SCHED_STREAM_K = 2      /* stream-K when the tiles leave pairs idle: the last partial round
                                plus one full round split over all pairs as contiguous ranges of
                                (tile, K block) units, or with at most half as many tiles as
                                pairs each tile split in two K halves; the cut tiles' fp32
                                partial sums go through the plan's workspace */
} fl_schedule;

typedef struct fl_plan_s* fl_plan_t;

/* Plan one fused linear layer of shape M×N×K ([epilog] Matmul(...).plan(epilog)).
 * Validates the combination, chooses the kernel configuration for the shape,
 * and allocates the plan's device workspace: an error word; the intermediate buffer
 * of an unfused plan; and, when the shape's tiles leave the last round of CTA pairs
 * partly idle (16-bit operands, M > 128), the stream-K workspace: one fp32 partial
 * accumulator of 32 rows x mma_n/2 columns per CTA and epilogue warp (at most
 * 148 x 8 x 16 KB = 19.4 MB on a B200) and its flags; for the kinds SWIGLU to WGRAD, when their
 * tiles would leave CTA pairs idle, the fp32 partial results of up to 32 K splits
 * (launches_per_execute of fl_plan_info is then 2).  Every execute of the plan
 * reuses this workspace, so two executes of one plan must not overlap on the GPU.
 * Needs the target device current.
 *   out     receives the plan handle (host pointer, must not be NULL)
 *   M, N, K ≥ 1 for M and N, ≥ 0 for K (K = 0 gives y = epi(0 + bias)); for
 *           GEGLU_TANH, SWIGLU and their AUX kinds, N is the width of h and W has 2N rows
 *   dtype   fl_dtype of A and W (F16/BF16 with FL_COMPUTE_32F, F32 with 3XTF32)
 * Errors: FL_ERR_INVALID_ARG, FL_ERR_UNSUPPORTED, FL_ERR_DEVICE, FL_ERR_OOM. */
fl_status fl_plan(fl_plan_t* out, int64_t M, int64_t N, int64_t K, int32_t dtype,
                  int32_t compute, const fl_epilogue_desc* epi);

/* Run the planned layer on `stream` (a cudaStream_t; NULL = legacy default stream)
 * ([epilog] execute(): one kernel launch for a fused plan; two where SWIGLU to WGRAD split K).
 *   A        [M, lda] operand
 *   W        [N, ldb] weight (b_major 0), [K, ldb] (b_major 1) or [2N, ldb] (GEGLU, SWIGLU)
 *   bias     length N (bias_axis 0) or M (bias_axis 1); required iff the kind has a bias
 *   aux      RELU_AUX_BIAS: [M, ceil(N/32)] uint32, packed rows; bit j of word w of
 *            row m is column 32w+j, least significant bit first; bits of columns ≥ N
 *            are written as 0.  GELU_AUX_BIAS: [M, ldo] in the output type (16-byte
 *            aligned), the pre-activation v.  GEGLU_TANH_AUX, SWIGLU_AUX (written) and
 *            DGEGLU_TANH, DSWIGLU (read): [M, 2N] packed, 16-byte aligned.  Null for every
 *            other kind
 *   residual [M, ldr], required iff has_residual
 *   out      [M, ldo] result
 * Errors: FL_ERR_INVALID_ARG (missing operand), FL_ERR_ALIGNMENT, FL_ERR_CUDA. */
fl_status fl_execute(fl_plan_t plan, const void* A, const void* W, const void* bias,
                     void* aux, const void* residual, void* out, void* stream);

/* Backward of RELU_AUX_BIAS: dpre[m,n] = grad[m,n] · bit(m,n), with the mask
 * written by a RELU_AUX_BIAS forward ([epilog]: the aux ReLU mask serves the
 * backward pass).  grad/dpre are [M, ld] of dtype (F16/BF16/F32); ld 0 = packed;
 * aux is [M, ceil(N/32)] packed.  dpre may alias grad.
 * Errors: FL_ERR_INVALID_ARG, FL_ERR_ALIGNMENT, FL_ERR_CUDA. */
fl_status fl_relu_backward(const void* grad, const uint32_t* aux, void* dpre, int64_t M,
                           int64_t N, int64_t ld_grad, int64_t ld_dpre, int32_t dtype,
                           void* stream);

/* Backward of the fused layer with the bias gradient fused in (no counterpart API on
 * the pages; [epilog] keeps the RELU_AUX mask for the backward pass and [gelu]
 * §2.2.1 asks that the backward of Linear+GELU be fused as well).  For y = act(v),
 * v = A·Wᵀ + bias with the bias broadcast over rows:
 *   fl_drelu_bgrad  dpre[m,n] = grad[m,n] · bit(m,n)      (mask of RELU_AUX_BIAS)
 *   fl_dgelu_bgrad  dpre[m,n] = grad[m,n] · GELU'(v[m,n])  (v of GELU_AUX_BIAS),
 *                   GELU'(v) = Φ(v) + v·φ(v), evaluated in fp32
 * and, when dbias is not null, dbias[n] = Σ_m dpre[m,n] in fp32 (of the fp32
 * products, before dpre is rounded to dtype), summed in a fixed order so that the
 * result does not depend on the schedule.
 *   grad, v, dpre  [M, ld] of dtype (F16/BF16/F32); ld 0 = packed (N)
 *   aux            [M, ceil(N/32)] uint32 packed mask (4-byte aligned)
 *   dbias          [N] fp32, or null (then no workspace is needed)
 *   workspace      fl_bias_grad_workspace_size bytes, 16-byte aligned, owned by the
 *                  caller (no initial contents needed): one row of fp32 column partial
 *                  sums per block of rows, which a second kernel adds in a fixed order.
 *                  Calls that overlap on the GPU must not share it.
 * dpre may alias grad.  Errors: FL_ERR_INVALID_ARG (null operand, negative size, ld < N,
 * workspace missing or too small), FL_ERR_ALIGNMENT, FL_ERR_CUDA. */
fl_status fl_bias_grad_workspace_size(int64_t M, int64_t N, int32_t dtype, size_t* bytes);
fl_status fl_drelu_bgrad(const void* grad, const uint32_t* aux, void* dpre, float* dbias, int64_t M,
                         int64_t N, int64_t ld_grad, int64_t ld_dpre, int32_t dtype, void* workspace,
                         size_t workspace_bytes, void* stream);
fl_status fl_dgelu_bgrad(const void* grad, const void* v, void* dpre, float* dbias, int64_t M, int64_t N,
                         int64_t ld_grad, int64_t ld_v, int64_t ld_dpre, int32_t dtype, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Failure-path self-test (no counterpart on the pages): one thread of a tiny kernel
 * waits, with the bounded wait every kernel of this library uses, on an mbarrier that
 * nothing arrives on.  The wait gives up after limit_ns (0 < limit_ns ≤ 10 s) and the
 * kernel records the timeout in a device word and returns; no trap, no fault, and the
 * context stays usable.  Synchronises `stream`.  Returns FL_ERR_TIMEOUT when the failure
 * path worked as designed, FL_ERR_CUDA otherwise, FL_ERR_INVALID_ARG for a bad limit. */
fl_status fl_wait_selftest(uint64_t limit_ns, void* stream);

/* LayerNorm of each row, the step after the residual tail ([mhc] §3.2: the row's mean
 * and variance and the normalisation in one kernel, one read and one write):
 *   z[m,n] = (x[m,n] − μ_m)/√(σ²_m + eps)·gamma[n] + beta[n],
 *   μ_m = mean of row m, σ²_m = mean of (x − μ_m)² (population variance), in fp32.
 *   x  [M, ld_x] of x_dtype; z [M, ld_z] of z_dtype.  In place: z == x with the same
 *   type and ld_z == ld_x (each row is read before it is written; other overlaps race)
 *   gamma, beta [N] of param_dtype; null gamma = 1, null beta = 0
 * Errors: FL_ERR_INVALID_ARG (null x/z, negative size, ld < N, eps < 0, M ≥ 2^31),
 * FL_ERR_ALIGNMENT, FL_ERR_CUDA. */
fl_status fl_layernorm(const void* x, const void* gamma, const void* beta, void* z, int64_t M, int64_t N,
                       int64_t ld_x, int64_t ld_z, int32_t x_dtype, int32_t z_dtype, int32_t param_dtype,
                       float eps, void* stream);

/* Dropout from a counter-based generator: no mask is stored, the backward pass draws the
 * same decisions again (no counterpart on the pages; the step between a sublayer's output
 * projection and its residual add in training).  The decision of element (m, n) of an
 * M x N matrix comes from word n mod 4 of Philox4x32-10 with key `seed` and counter
 * (m*ceil(N/4) + n/4, offset), both 64 bits with the low half first: the element is dropped
 * when the word is below floor(p*2^32), else multiplied by 1/(1-p).  It depends on M x N
 * indices only, not on pitches, types or the launch.  A dropped element gives exactly 0,
 * whatever x holds there (infinities and NaN included).  Calls with the same seed and
 * different offsets draw independent numbers. */
typedef struct {
  float p;                    /* probability of dropping an element, in [0, 1); 0: none dropped */
  int32_t reserved;           /* must be 0 */
  uint64_t seed, offset;
  const uint64_t* offset_dev; /* device pointer, 8-byte aligned, or null: added to offset (modulo
                                 2^64) when the kernel runs, so that a captured graph draws new
                                 numbers at each replay if the caller advances it in between */
} fl_dropout_desc;

/* y = residual + D(x), D the dropout above (drop null: D(x) = x).  Forward and backward in
 * one: the gradient of x is D of y's gradient with the same seed and offset, and the
 * residual's gradient is y's gradient itself.
 *   x [M, ld_x] of x_dtype; residual (or null) [M, ld_r] and y [M, ld_y] of y_dtype; ld 0 = N.
 *   y may be x's or the residual's own buffer with the same type and pitch.
 * Any alignment of the elements is accepted; rows that all start on 16 bytes run fastest.
 * M = 0 or N = 0, here and in the two below: nothing to do, and null operands are accepted (an empty
 * tensor has no address).
 * Errors: FL_ERR_INVALID_ARG (null x or y, size, ld < N, dtype, p outside [0, 1)),
 * FL_ERR_ALIGNMENT, FL_ERR_CUDA. */
fl_status fl_dropout(const void* x, const void* residual, void* y, int64_t M, int64_t N, int64_t ld_x, int64_t ld_r,
                     int64_t ld_y, int32_t x_dtype, int32_t y_dtype, const fl_dropout_desc* drop, void* stream);

/* The end of a sublayer in training, in one kernel ([mhc] §3.2 fuses the residual add and
 * the row's normalisation):
 *   s = residual + D(x),  z = (s − μ_m)·rstd_m·gamma + beta,  rstd_m = 1/√(σ²_m + eps),
 * μ_m and σ²_m the mean and the population variance of row m of s, in fp32, of s before it is
 * rounded to its type.
 *   x [M, ld_x] of x_dtype; residual (null: none) and sum (the stored s; null: not stored)
 *   [M, ld_r], [M, ld_sum] of sum_dtype; z [M, ld_z] of z_dtype; gamma, beta [N] of
 *   param_dtype (null gamma = 1, null beta = 0); mean, rstd [M] fp32, both or neither: what
 *   the backward pass reads.  drop null: no dropout.  ld 0 = N.
 *   sum and z may each be x's or the residual's own buffer with the same type and pitch (not
 *   both the same one).
 * Errors: as fl_layernorm, and FL_ERR_INVALID_ARG for p outside [0, 1). */
fl_status fl_dropout_layernorm(const void* x, const void* residual, const void* gamma, const void* beta, void* sum,
                               void* z, float* mean, float* rstd, int64_t M, int64_t N, int64_t ld_x, int64_t ld_r,
                               int64_t ld_sum, int64_t ld_z, int32_t x_dtype, int32_t sum_dtype, int32_t z_dtype,
                               int32_t param_dtype, float eps, const fl_dropout_desc* drop, void* stream);

/* Its backward pass.  With u = (s − μ)·rstd and g = dz·gamma:
 *   ds = rstd·(g − mean_n(g) − u·mean_n(g·u)) + dsum,  dres = ds,  dx = D(ds),
 *   dgamma[n] = Σ_m dz·u,  dbeta[n] = Σ_m dz  (fp32, summed in a fixed order).
 * dx is D of ds before ds is rounded to its type.
 *   dz [M, ld_dz] of z_dtype; dsum [M, ld_dsum] of sum_dtype, the gradient that reaches s by
 *   the residual stream of a pre-norm block, or null; sum [M, ld_sum] of sum_dtype, mean, rstd
 *   [M]: from the forward pass (for a plain LayerNorm, sum is its input x); gamma as there.
 *   dres [M, ld_dres] of sum_dtype, dx [M, ld_dx] of x_dtype, dgamma, dbeta [N] fp32: each may
 *   be null (not wanted), not all.  dres and dx may each be dz's, dsum's or sum's own buffer with
 *   the same type and pitch (not both the same one).  M = 0 gives dgamma = dbeta = 0, without a workspace.
 *   workspace: needed for dgamma and dbeta; fl_layernorm_grad_workspace_size bytes (for the
 *   current device; never less for more rows), 16-byte aligned, owned by the caller, no initial contents needed.  Calls
 *   that overlap on the GPU must not share it.
 * Errors: FL_ERR_INVALID_ARG (null operand, no output, size, ld < N, dtype, p, workspace),
 * FL_ERR_ALIGNMENT, FL_ERR_CUDA. */
fl_status fl_layernorm_grad_workspace_size(int64_t M, int64_t N, size_t* bytes);
fl_status fl_dropout_layernorm_backward(const void* dz, const void* dsum, const void* sum, const float* mean,
                                        const float* rstd, const void* gamma, void* dres, void* dx, float* dgamma,
                                        float* dbeta, int64_t M, int64_t N, int64_t ld_dz, int64_t ld_dsum,
                                        int64_t ld_sum, int64_t ld_dres, int64_t ld_dx, int32_t x_dtype,
                                        int32_t sum_dtype, int32_t z_dtype, int32_t param_dtype,
                                        const fl_dropout_desc* drop, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* Synchronise `stream` and read the plan's device error word.  Returns
 * FL_ERR_TIMEOUT if a bounded wait inside a kernel of this plan gave up
 * (the error word is then cleared), FL_ERR_CUDA on a CUDA error, else FL_OK. */
fl_status fl_check_status(fl_plan_t plan, void* stream);

/* Describe the configuration the plan chose (all fields are host-side ints). */
typedef struct {
  int32_t tile_m, tile_n;      /* output tile of one CTA (before split-K) */
  int32_t mma_n;               /* tensor-core N per instruction */
  int32_t swap_ab;             /* 1: W is the tensor-core A operand (small M) */
  int32_t split_k;             /* CTAs of a cluster sharing one tile along K; SWIGLU to WGRAD: splits of K */
  int32_t stages;              /* shared-memory pipeline depth */
  int32_t grid;                /* CTAs launched by the main kernel */
  int32_t smem_bytes;          /* dynamic shared memory per CTA */
  int32_t launches_per_execute;/* kernels one fl_execute launches */
  int32_t cta_pair;            /* 1: two CTAs share each 256-row tensor-core tile */
  int32_t stream_k_tiles;      /* tiles split along K over the pairs (stream-K), 0: none */
  int32_t stream_k_pairs;      /* pairs sharing those tiles' (tile, K-block) units */
  int32_t reserved[4];
} fl_plan_info;
fl_status fl_get_plan_info(fl_plan_t plan, fl_plan_info* info);

/* The configuration fl_plan would choose for these arguments on a device with
 * num_sms SMs and max_smem_per_block bytes of opt-in shared memory per block (B200:
 * 148 and 232448), computed on the host alone: the same argument checks and the same
 * choice as fl_plan, no device call, nothing allocated.  Lets a caller (or a test
 * without a GPU) inspect the layout, split-K and grid fl_plan will use.
 * Errors: those of fl_plan's argument checks; FL_ERR_INVALID_ARG for a null pointer or
 * an implausible device (num_sms outside [2, 4096], max_smem_per_block < 16384);
 * FL_ERR_UNSUPPORTED when no configuration fits. */
fl_status fl_plan_preview(int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t compute,
                          const fl_epilogue_desc* epi, int32_t num_sms, int32_t max_smem_per_block,
                          fl_plan_info* info);

/* Release a plan and its workspace ([epilog] free()).  NULL is accepted.
 * Synchronises nothing: the caller must not free a plan with work in flight. */
fl_status fl_free(fl_plan_t plan);

/* Thread-local text of the last failure on this thread ("" if none). */
const char* fl_last_error(void);

/* One fused linear layer without any device allocation (the pages have no
 * counterpart of this call).  For callers that cannot call cudaMalloc: a host
 * that owns all device memory through its own pool, or a latency-critical path
 * on which cudaMalloc/cudaFree are forbidden because they can synchronise the
 * device.  It takes fl_plan's arguments and fl_execute's operands in one call
 * and runs the same kernels; the scratch that a plan would allocate comes from
 * one fixed 32 MiB + 256 B device array inside this library (the device error
 * word, and the intermediate of an unfused call, which must fit in 32 MiB:
 * M × (N, or 2N for GEGLU_TANH, rounded up to 16 bytes) × out_dtype size;
 * larger sizes return FL_ERR_INVALID_ARG).  Every GPU that loads the library
 * holds the array until the process exits.
 *   - The first call on a device looks up the array's device address with that
 *     device current; make that first call before any stream capture.
 *   - All calls on a device share the array: calls that overlap on the GPU (on
 *     different streams, or from different threads) race on it.
 *   - The error word is cleared at each call and not read back: a bounded
 *     in-kernel wait that gives up is not reported by this entry point.
 *   - fp16/bf16 operands with FL_COMPUTE_32F only.
 *   - SWIGLU to WGRAD run without K splits, which need a workspace: slower where fl_plan would
 *     split, and their sums then run in another order than a plan's.
 * Errors: as fl_plan and fl_execute. */
fl_status fl_execute_noalloc(int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t compute,
                             const fl_epilogue_desc* epi, const void* A, const void* W,
                             const void* bias, void* aux, const void* residual, void* out,
                             void* stream);

/* Override the bound on every in-kernel wait for plans created afterwards
 * (nanoseconds; 0 restores the default of 2 s).  Test/debug use. */
fl_status fl_set_wait_limit_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif
#endif /* FUSED_LINEAR_H_ */
