/*
 * farn.h - fused rank-sum + residual add + RMSNorm on one GB300 (sm_103a).
 *
 * The operation is the contract of FlagTree pull request "[TLERaw] Add
 * NVSHMEM allreduce RMSNorm tutorial" (Summary):
 *
 *     reduced      = sum over ranks r = 0..W-1 of x[r]
 *     residual_out = reduced + residual
 *     norm_out     = RMSNorm(residual_out, weight, eps)
 *
 * with the epilogue of its Implementation section 3 (residual add, then
 * RMSNorm with FP32 accumulation) fused into the same kernel.  On one GPU
 * the W partials of the page's all-reduce are W bf16 tensors that already
 * sit in this GPU's memory; the library reads them through a pointer array,
 * so there is no collective and no cross-GPU traffic.
 *
 * Arithmetic (element (t,h); f() widens bf16 to fp32 exactly, bf16()
 * rounds fp32 to nearest even):
 *     reduced[t,h]      = bf16(f(x[0]) + f(x[1]) + ... + f(x[W-1]))   fp32, rank order
 *     residual_out[t,h] = bf16(f(reduced[t,h]) + f(residual[t,h]))
 *     rstd[t]           = 1 / sqrt(sum_h f(residual_out[t,h])^2 / H + eps)
 *     norm_out[t,h]     = bf16((f(residual_out[t,h]) * rstd[t]) * f(weight[h]))
 * reduced and residual_out are exact functions of the inputs (bit for bit
 * the same on every launch configuration); norm_out depends on the
 * summation order of the row's sum of squares and may differ by one bf16
 * ulp between launch configurations.
 *
 * Layout: every [T,H] tensor is row-major and contiguous (row t starts at
 * element t*H), bf16 (2-byte IEEE bfloat16 patterns).  weight is [H].
 * All tensor pointers are DEVICE pointers on the context's device, owned
 * by the caller; the library keeps none of them after a call returns.
 * The fast kernels need every pointer 16-byte aligned and H a multiple
 * of 8; other shapes and alignments are served by a slower kernel.
 *
 * Errors: every entry point returns FARN_OK (0) or a negative farn_status.
 * On an error nothing is launched and no output is written.
 * Launch-time CUDA errors are reported; errors of the asynchronous kernel
 * itself surface at the caller's next synchronisation, as usual in CUDA.
 */
#ifndef FARN_H_
#define FARN_H_

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of rank partials one call accepts. */
#define FARN_MAX_W 32

/* Largest number of experts of the router and of the grouped product. */
#define FARN_MAX_EXPERTS 1024

typedef enum {
    FARN_OK = 0,
    FARN_ERR_INVALID_ARG = -1,  /* null pointer, W/T/H/eps out of range     */
    FARN_ERR_UNSUPPORTED = -2,  /* shape the library cannot launch           */
    FARN_ERR_ALIAS = -3,        /* an output overlaps an input or an output  */
    FARN_ERR_CUDA = -4,         /* CUDA runtime error (launch, device query) */
    FARN_ERR_NOMEM = -5         /* host allocation of the context failed     */
} farn_status;

/* Element types of the partials (farn_forward_typed). */
typedef enum {
    FARN_BF16 = 0,   /* bfloat16, 2 bytes */
    FARN_F32 = 1     /* IEEE binary32, 4 bytes */
} farn_dtype;

/* Opaque per-device context: device properties and kernel attributes
 * queried once.  Immutable after farn_create; one context may serve any
 * number of streams and host threads at once. */
typedef struct farn_ctx farn_ctx;

/* Create a context for CUDA device `device` (this is the one-time set-up
 * that the page's host side does at initialisation, Implementation
 * section 4, "host-side C ABI"; there is no communicator to bootstrap).
 * Queries the SM count and cluster limits, sets kernel attributes and
 * allocates one 256-byte device block (the status word of the TMA-staged
 * kernel, see farn_device_status).  The caller's current device is left
 * as it was.  The environment is read here and only here: FARN_VARIANT,
 * FARN_CLUSTER, FARN_VPT, FARN_PDL, FARN_SMALL_T, FARN_BULK,
 * FARN_BULK_CTAS, FARN_STAGE, FARN_STAGE_R, FARN_STAGE_CTAS,
 * FARN_STAGE_MIN_T, FARN_STAGE_MIN_MB, FARN_TC_TILE and FARN_TC_SPLIT override
 * the kernel choice (tests and sweeps); FARN_FAULT_INJECT injects a fault for the tests: "create"
 * fails this call, "launch" makes every launch of the context fail before
 * anything is enqueued, "stall" makes CTA 0 of every TMA-staged launch
 * wait out its time limit and report it in the status word (of the
 * tensor-core products: its weights never come), "setup" makes the set-up of
 * the router and of the products' tensor-core kernels fail.  Where that set-up
 * fails the context serves the rest: farn_moe_route returns FARN_ERR_CUDA, and
 * the products take their slower kernel (see farn_plan_grouped_matmul).
 * Returns FARN_ERR_INVALID_ARG if out is NULL or device < 0 or not a device
 * of this process, FARN_ERR_CUDA if the device cannot be queried (or
 * FARN_FAULT_INJECT=create), FARN_ERR_NOMEM. */
int farn_create(farn_ctx **out, int device);

/* The fused operator on `stream` (asynchronous; the call does not wait
 * for the GPU).
 *   partials     host array of W device pointers, partials[r] -> x[r],
 *                bf16 [T,H]; the array itself is read during the call only.
 *   W            1 .. FARN_MAX_W
 *   residual     bf16 [T,H]
 *   weight       bf16 [H]
 *   eps          finite, >= 0 (fp32; added to the mean square inside sqrt)
 *   T            rows (tokens), >= 0; T == 0 returns FARN_OK and launches
 *                nothing (the tensor pointers may then be NULL, as the data
 *                pointers of empty tensors are)
 *   H            hidden size (row length), >= 1
 *   reduced_out, residual_out, norm_out   bf16 [T,H] outputs
 *   stream       CUDA stream (0 = legacy default stream)
 * Outputs may not overlap each other or any input, with one exception:
 * residual_out may be exactly residual (in-place residual update).
 * Returns FARN_ERR_INVALID_ARG (ctx or a pointer NULL, W, T, H or eps out
 * of range, T*H*2 bytes overflowing), FARN_ERR_ALIAS, FARN_ERR_UNSUPPORTED,
 * or FARN_ERR_CUDA if the launch failed. */
int farn_forward(const farn_ctx *ctx,
                 const void *const *partials, int W,
                 const void *residual, const void *weight, float eps,
                 int64_t T, int64_t H,
                 void *reduced_out, void *residual_out, void *norm_out,
                 cudaStream_t stream);

/* farn_forward with the partials in `partial_dtype` (a farn_dtype):
 * FARN_BF16 is exactly farn_forward; FARN_F32 takes fp32 partials [T,H]
 * (for example the fp32 output of a GEMM epilogue, before any rounding)
 * and sums their own fp32 values in rank order, rounding once to bf16 --
 * the "FP32 accumulation where required" of the page's Implementation
 * section 3.  residual, weight and the three outputs stay bf16; everything
 * else (layout, ownership, aliasing, errors) is as for farn_forward, with
 * each fp32 partial occupying T*H*4 bytes.  Returns FARN_ERR_INVALID_ARG
 * for an unknown dtype. */
int farn_forward_typed(const farn_ctx *ctx,
                       const void *const *partials, int partial_dtype, int W,
                       const void *residual, const void *weight, float eps,
                       int64_t T, int64_t H,
                       void *reduced_out, void *residual_out, void *norm_out,
                       cudaStream_t stream);

/* The argument checks of farn_forward alone, on the host: no CUDA call, no
 * launch, pointers are only compared, never dereferenced.  Returns what
 * farn_forward would return before launching. */
int farn_check_args(const void *const *partials, int W,
                    const void *residual, const void *weight, float eps,
                    int64_t T, int64_t H,
                    const void *reduced_out, const void *residual_out,
                    const void *norm_out);

/* Read and clear the context's device status word (blocking: waits for
 * the device).  0 means every wait of the TMA-staged kernel completed; a
 * non-zero value has one bit per kind of wait that gave up after its time
 * limit (2 s): 1 a consumer waiting for a staged segment, 2 the producer
 * waiting for a free stage, 4 a consumer in the row reduction, 8 the
 * producer draining its copies; in the products' tensor-core kernels 16 the
 * wait for operands, 32 for a free stage, 64 for a finished tile, 128 for the
 * other parts of a split row.  The kernel that gave up left its outputs
 * incomplete.  The TMA-staged kernel runs where farn_plan /
 * farn_plan_moe_combine report variant 3, and in every
 * farn_forward_noalloc call.  Returns FARN_ERR_INVALID_ARG or FARN_ERR_CUDA
 * on failure. */
int farn_device_status(const farn_ctx *ctx, int *status);

/* Release a context (NULL is accepted).  Returns FARN_OK. */
int farn_destroy(farn_ctx *ctx);

/* Text for a farn_status value (never NULL). */
const char *farn_status_string(int status);

/* Which kernel variant farn_forward would launch for this shape and these
 * pointers, without launching: 0 row (one CTA per row; decode sizes, and
 * long calls with a bf16 norm_out of W < 8 bf16 partials or of 8..11 with
 * H <= 5120, or with an FP8 / NVFP4 output of one or two partials or of
 * W < 8 with H <= 5120), 1 cluster (a cluster of CTAs splits each row; fewer than 16
 * rows), 2 generic (any H or alignment), 3 bulk (persistent CTAs whose
 * producer warp stages column segments of every input row in shared memory
 * with TMA bulk copies; rows of at most 16384 elements; calls of W >= 12
 * bf16 partials from 256 rows, long calls of 8..11 with 5120 < H < 8192,
 * or any call when enabled), 4 stage (persistent CTAs whose threads stage their own
 * vectors in shared memory with cp.async; the other long calls: 8..11
 * partials with H >= 8192, and the FP8 / NVFP4 outputs of W >= 3 partials
 * with H > 5120 or of W >= 8).
 * *cluster_size receives the CTAs per row (1 for row and generic),
 * *threads the threads per CTA.  Returns a farn_status. */
int farn_plan(const farn_ctx *ctx, int W, int64_t T, int64_t H,
              const void *const *partials, const void *residual,
              const void *weight, const void *reduced_out,
              const void *residual_out, const void *norm_out,
              int *variant, int *cluster_size, int *threads);

/* farn_forward_noalloc - the fused operator for callers that cannot
 * allocate device memory.  (No counterpart in the paper: the page's host
 * side allocates a symmetric workspace; this entry point exists for
 * callers that must not call cudaMalloc, e.g. code running inside another
 * framework's plugin or allocator interface, where every device allocation
 * has to go through that framework.)
 *
 * Same arithmetic, arguments, layout and error checks as farn_forward, but
 * without a context: `device` names the CUDA device that owns the tensors.
 * It always runs the TMA-staged kernel and allocates nothing: no
 * cudaMalloc, no cudaFree, no allocating library call.  The kernel's only
 * memory beyond the caller's tensors is a 4-byte status word kept in a
 * fixed 256-byte array that this library places in every GPU's memory for
 * the life of the process; a call needs that one word whatever T, H and W
 * are.  Every shape with 16-byte aligned tensors, H % 8 == 0 and
 * H <= 16384 is taken, for any W <= FARN_MAX_W; other shapes (tensors not
 * 16-byte aligned, H % 8 != 0, rows longer than 16384 elements) return
 * FARN_ERR_UNSUPPORTED.
 *
 * The first call on a device sets that device up (finds the array's device
 * address, reads the device limits, sets the kernels' shared-memory
 * attribute); make that first call before any stream capture.  Every call
 * clears the status word on `stream` before launching; the word is shared
 * by all calls on the device, so calls that overlap on the GPU (different
 * streams, no ordering between them) race on it.
 *
 * status_out: optional host pointer.  When non-NULL the call waits for the
 * kernel to finish and stores the status word there (0 = every wait
 * completed; bits as in farn_device_status).  When NULL the call is
 * asynchronous like farn_forward.
 * Returns FARN_OK, FARN_ERR_INVALID_ARG (as farn_forward, or device out of
 * range), FARN_ERR_ALIAS, FARN_ERR_UNSUPPORTED or FARN_ERR_CUDA. */
int farn_forward_noalloc(int device,
                         const void *const *partials, int W,
                         const void *residual, const void *weight, float eps,
                         int64_t T, int64_t H,
                         void *reduced_out, void *residual_out, void *norm_out,
                         cudaStream_t stream, int *status_out);

/* farn_forward_typed plus an FP8 copy of norm_out for the next layer's
 * GEMM.  (The page does not describe this output; it extends the fused
 * epilogue by one step.)  Per row t:
 *     amax         = max over h of |norm_out[t,h]|   (the bf16 values; NaN ignored)
 *     row_scale[t] = amax / 448, or 1 if amax is 0   (fp32; norm ~ q * scale)
 *     norm_q[t,h]  = E4M3(norm_out[t,h] * inv),  inv = 448 / amax (fp32), or 1
 * E4M3 is the OCP 8-bit float with 4 exponent and 3 fraction bits (largest
 * finite 448, no infinities); the conversion rounds to nearest even and
 * saturates larger magnitudes (and infinities) to +-448; NaN stays NaN.
 *   norm_q     uint8 [T,H] (E4M3 patterns), 16-byte aligned for the fast
 *              kernels
 *   row_scale  float [T]
 *   norm_out   bf16 [T,H], or NULL to skip writing it (it is still computed)
 * The other arguments, checks and errors are those of farn_forward_typed;
 * norm_q and row_scale take part in the aliasing checks. */
int farn_forward_quant(const farn_ctx *ctx,
                       const void *const *partials, int partial_dtype, int W,
                       const void *residual, const void *weight, float eps,
                       int64_t T, int64_t H,
                       void *reduced_out, void *residual_out, void *norm_out,
                       void *norm_q, float *row_scale,
                       cudaStream_t stream);

/* farn_forward_typed plus an NVFP4 copy of norm_out, the 4-bit input of a
 * block-scaled GEMM.  (Not described by the page either.)  Each block of 16
 * consecutive elements of a row, b = h / 16, shares one E4M3 scale under
 * the fp32 tensor scale g = tensor_scale (a calibrated input: a fused
 * kernel cannot see the whole tensor before it writes its first block):
 *     amax            = max of |norm_out| over the block (NaN ignored)
 *     block_scale[t,b] = E4M3((amax / 6) * g)            (saturating)
 *     inv             = g / value(block_scale[t,b])      (fp32 division)
 *     code[t,h]       = E2M1(norm_out[t,h] * inv)
 * E2M1 has 1 sign, 2 exponent and 1 fraction bit (magnitudes 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6); the conversion rounds to nearest even and saturates
 * larger magnitudes and infinities to +-6; a NaN element is written as +6
 * (code 7); a block whose scale is 0 gets all-zero codes.  The value a code
 * stands for is value(code) * value(block_scale) / g.
 *   norm_fp4     uint8 [T, H/2]: codes of elements 2i (low nibble) and
 *                2i+1 (high nibble) in byte i; 4-byte aligned for the
 *                fast kernels
 *   block_scale  uint8 [T, H/16] (E4M3 patterns, row-major, no swizzle)
 *   tensor_scale finite, > 0
 *   norm_out     bf16 [T,H], or NULL to skip writing it
 *   H            a multiple of 16
 * The other arguments, checks and errors are those of farn_forward_typed
 * (FARN_ERR_INVALID_ARG also for H % 16 != 0 or a bad tensor_scale);
 * norm_fp4 and block_scale take part in the aliasing checks. */
int farn_forward_nvfp4(const farn_ctx *ctx,
                       const void *const *partials, int partial_dtype, int W,
                       const void *residual, const void *weight, float eps,
                       int64_t T, int64_t H, float tensor_scale,
                       void *reduced_out, void *residual_out, void *norm_out,
                       void *norm_fp4, void *block_scale,
                       cudaStream_t stream);

/* farn_moe_combine - the MoE "local y reduce" fused with the same
 * residual add + RMSNorm.  (The page names the per-token reduction of
 * expert outputs but defines neither its weights nor its layout; this is
 * the plain reading.)  For each token t and column h:
 *     reduced[t,h] = bf16(acc),  acc = -0; for k = 0..K-1, slot s = index[t*K+k]
 *                    in [0, n_slots):  acc = acc + gates[t*K+k] * f(expert_out[s,h])
 * with the product and the sum each rounded to fp32 (no fused multiply-add),
 * k in order; slots outside [0, n_slots) (e.g. -1 for a dropped expert) are
 * skipped, and are never read.  residual_out and norm_out then follow as in
 * farn_forward.
 *   expert_out  bf16 [n_slots, H], one row per (token, expert) assignment
 *   index       int32 [T, K] (4-byte aligned), gates fp32 [T, K] (4-byte aligned)
 *   K           1 .. FARN_MAX_W
 * Other arguments, layouts, ownership, in-place residual_out and errors as
 * for farn_forward; outputs may not overlap expert_out, index or gates. */
int farn_moe_combine(const farn_ctx *ctx,
                     const void *expert_out, int64_t n_slots,
                     const int32_t *index, const float *gates, int K,
                     const void *residual, const void *weight, float eps,
                     int64_t T, int64_t H,
                     void *reduced_out, void *residual_out, void *norm_out,
                     cudaStream_t stream);

/* Which kernel farn_moe_combine would launch for this shape and these
 * pointers, without launching: 2 generic (any H or alignment), 3 bulk
 * (persistent CTAs that gather the rows into shared memory with TMA bulk
 * copies; long inputs with rows of more than 3072 elements, or 5120 below
 * 8 experts, that fit two segments of at most 512 consumer threads or more
 * segments of 256), 4 stage (persistent CTAs that gather the rows into
 * shared memory with cp.async; the other long inputs with such rows),
 * 5 combine (one CTA per row; shorter inputs and shorter rows).  *threads receives the threads per CTA (at most 544 for bulk: one
 * producer warp and the consumers; at most 512 otherwise).  Returns a farn_status (FARN_ERR_INVALID_ARG for a bad shape or a
 * NULL pointer; aliasing is not checked). */
int farn_plan_moe_combine(const farn_ctx *ctx, int K, int64_t T, int64_t H,
                          const void *expert_out, const void *residual,
                          const void *weight, const void *reduced_out,
                          const void *residual_out, const void *norm_out,
                          int *variant, int *threads);

/* farn_moe_route - the MoE router: which experts every token goes to, with
 * which gates, and where its rows lie when the (token, expert) pairs are
 * sorted by expert.  Its outputs are the inputs of farn_grouped_matmul
 * (rows, offsets) and farn_moe_combine (index, gates).
 *     experts[t,k]  the expert of the k-th largest of logits[t,:]; of equal
 *                   logits (-0 and +0 are equal) the lowest expert first.
 *                   A logit of -inf (a masked expert) or NaN is never
 *                   chosen: where fewer than K are left, -1.
 *     gates[t,k]    p(experts[t,k]) / sum of p, p(e) = exp(logits[t,e] - max)
 *                   in fp32 (1 for an infinite maximum), the sum over the
 *                   chosen experts (renormalize != 0) or over all E; 0 where
 *                   the expert is -1.
 *     offsets[e]    the first slot of expert e; offsets[E] the number of
 *                   slots in use (pairs whose expert is not -1)
 *     index[t,k]    the pair's slot, or -1: slots are sorted by expert, then
 *                   by token
 *     rows[s]       the token of slot s; -1 for slots from offsets[E] on
 * The whole numbers are exact functions of the logits.
 *   logits  bf16 or fp32 [T, E] (logits_dtype a farn_dtype)
 *   E       1 .. FARN_MAX_EXPERTS;  K  1 .. min(E, FARN_MAX_W);  T * K < 2^31
 *   experts, index  int32 [T, K];  gates  fp32 [T, K];  rows  int32 [T * K];
 *   offsets int32 [E + 1], all 4-byte aligned
 * T == 0 writes the offsets (all 0) only; the other pointers may be NULL.
 * No memory beyond the outputs is used.  Returns FARN_ERR_INVALID_ARG,
 * FARN_ERR_ALIAS (an output over another tensor) or FARN_ERR_CUDA. */
int farn_moe_route(const farn_ctx *ctx, const void *logits, int logits_dtype,
                   int64_t T, int E, int K, int renormalize,
                   int32_t *experts, float *gates, int32_t *index,
                   int32_t *rows, int32_t *offsets, cudaStream_t stream);

/* farn_grouped_matmul - the experts' products:
 *     out[s,n] = bf16( sum_h f(x[r,h]) * f(weights[e,n,h]) )
 * for every slot s of expert e, offsets[e] <= s < offsets[e+1], with r =
 * rows[s], or r = s where rows is NULL.  Products and sums in fp32 (the
 * order of the sum is the kernel's own and the same in every call with the
 * same arguments), one rounding to bf16.
 *   x        bf16 [n_rows, H]; rows NULL needs n_rows == n_slots
 *   rows     int32 [n_slots] or NULL (4-byte aligned).  A slot whose row is
 *            outside [0, n_rows) gets zeros; nothing is read for it.
 *   weights  bf16 [E, N, H], E 1 .. FARN_MAX_EXPERTS
 *   offsets  int32 [E + 1] on the device, ascending, within 0 .. n_slots.
 *            An expert may have no slots.  (Other values cannot lead outside
 *            the tensors, but the outputs are then unspecified.)
 *   out      bf16 [n_slots, N]; slots below offsets[0] and from offsets[E]
 *            on are left as they were
 *   n_slots, n_rows, N, H < 2^31; n_slots == 0 returns FARN_OK and launches
 *            nothing
 * The fast kernels need x and weights 16-byte aligned and H a multiple of 8;
 * other shapes are served by a slower kernel.  Returns FARN_ERR_INVALID_ARG,
 * FARN_ERR_ALIAS (out over an input), FARN_ERR_UNSUPPORTED (2^30 or more tiles
 * of 64 slots of one expert by 64 columns) or FARN_ERR_CUDA. */
int farn_grouped_matmul(const farn_ctx *ctx, const void *x, int64_t n_rows,
                        const int32_t *rows, int64_t n_slots,
                        const void *weights, int E, const int32_t *offsets,
                        int64_t N, int64_t H, void *out, cudaStream_t stream);

/* farn_nvfp4_quantize - NVFP4 codes and block scales of a bf16 tensor
 * x [T,H], for tensors that no norm produces (weights, expert activations):
 * the format and arithmetic of farn_forward_nvfp4's copy of norm_out, with x
 * in norm_out's place.
 *   codes        uint8 [T, H/2];  block_scale  uint8 [T, H/16]
 *   tensor_scale finite, > 0;  H a multiple of 16;  T == 0 launches nothing
 * x 16-byte and codes 8-byte aligned take the fast kernel.  Returns
 * FARN_ERR_INVALID_ARG, FARN_ERR_ALIAS, FARN_ERR_UNSUPPORTED (more than
 * 2^45 - 2^14 elements) or FARN_ERR_CUDA. */
int farn_nvfp4_quantize(const farn_ctx *ctx, const void *x, int64_t T, int64_t H,
                        float tensor_scale, void *codes, void *block_scale,
                        cudaStream_t stream);

/* farn_nvfp4_dequantize - the values that NVFP4 codes stand for, in bf16:
 *     out[t,h] = bf16( value(code) * (value(block_scale) / tensor_scale) )
 * with the quotient and the product each rounded to fp32.  Arguments and
 * errors as for farn_nvfp4_quantize; out bf16 [T,H], 16-byte aligned for the
 * fast kernel. */
int farn_nvfp4_dequantize(const farn_ctx *ctx, const void *codes,
                          const void *block_scale, int64_t T, int64_t H,
                          float tensor_scale, void *out, cudaStream_t stream);

/* farn_nvfp4_matmul - the product of two NVFP4 tensors (farn_forward_nvfp4's
 * or farn_nvfp4_quantize's outputs), for example activations by weights:
 *     out[t,n] = bf16( alpha * sum_h va[t,h] * vb[n,h] )
 *     v = value(code) * value(block_scale),  alpha = 1 / (a_tensor_scale *
 *     b_tensor_scale), rounded once to fp32
 * accumulated in fp32 (the order is the kernel's own and the same in every
 * call with the same arguments), one rounding to bf16.  A block scale of NaN
 * makes its products NaN; the sign bit of a block scale has to be 0.
 *   a_codes uint8 [T, H/2], a_scale uint8 [T, H/16]; b_codes, b_scale the
 *   same with N rows; out bf16 [T, N]
 *   H a multiple of 16; T, N, H < 2^31; T == 0 launches nothing
 * The fast kernels need the codes 16-byte aligned and H a multiple of 32 (they
 * are faster still with H a multiple of 256 and the scales 16-byte aligned);
 * other shapes are served by a slower kernel.  Returns FARN_ERR_INVALID_ARG
 * (also for an alpha that fp32 cannot hold), FARN_ERR_ALIAS,
 * FARN_ERR_UNSUPPORTED (2^30 or more tiles of 64 rows by 64 columns) or
 * FARN_ERR_CUDA. */
int farn_nvfp4_matmul(const farn_ctx *ctx, const void *a_codes,
                      const void *a_scale, float a_tensor_scale,
                      const void *b_codes, const void *b_scale,
                      float b_tensor_scale, int64_t T, int64_t N, int64_t H,
                      void *out, cudaStream_t stream);

/* Which kernel farn_grouped_matmul or farn_nvfp4_matmul would launch for these
 * sizes and pointers, without launching (only alignment and whether rows is
 * NULL matter of the pointers): 2 generic (any H or alignment), 6 tensor (the
 * tensor cores, a tile of 128 weights by 64 slots per CTA, *ctas of them
 * splitting the row), 7 pair (the tensor cores, two CTAs per tile of 256 by 256,
 * NVFP4 224, slots).  *ctas receives the CTAs per tile, *threads the threads per
 * CTA.  Returns a farn_status (FARN_ERR_INVALID_ARG for a bad or empty shape or
 * a NULL pointer, FARN_ERR_UNSUPPORTED as the call itself; aliasing is not
 * checked). */
int farn_plan_grouped_matmul(const farn_ctx *ctx, const void *x, int64_t n_rows,
                             const int32_t *rows, int64_t n_slots,
                             const void *weights, int E, int64_t N, int64_t H,
                             const void *out, int *variant, int *ctas,
                             int *threads);
int farn_plan_nvfp4_matmul(const farn_ctx *ctx, const void *a_codes,
                           const void *a_scale, const void *b_codes,
                           const void *b_scale, int64_t T, int64_t N, int64_t H,
                           const void *out, int *variant, int *ctas,
                           int *threads);

/* farn_fp8_quantize - E4M3 codes and fp32 scales of bf16 matrices x [E, T, H]
 * (E = 1: one matrix), in blocks of 128 elements of a row (block_rows 1:
 * activations) or of 128 rows by 128 columns (block_rows 128: weights); the
 * operands of the FP8 products.  Per block, the last ones of a row or matrix
 * being shorter:
 *     amax  = max |x| over the block (NaN ignored)
 *     scale = amax / 448, or 1 if amax is 0     (fp32; x ~ code * scale)
 *     code  = E4M3(x * inv),  inv = min(448 / amax, FLT_MAX) (fp32), or 1
 * with the conversion of farn_forward_quant (nearest even, saturating, NaN
 * stays NaN).  A block with an infinity has scale inf and codes 0 and NaN: its
 * values are all NaN.
 *   codes   uint8 [E, T, H]
 *   scales  fp32 [E, ceil(T / block_rows), ceil(H / 128)], 4-byte aligned
 *   E == 0 or T == 0 launches nothing
 * x 16-byte and codes 8-byte aligned with H a multiple of 8 take the fast
 * kernel (8192 rows of 5120 28 us, in blocks of 128 rows 23; of 5119 49 and 135).
 * Returns FARN_ERR_INVALID_ARG, FARN_ERR_ALIAS, FARN_ERR_UNSUPPORTED
 * (2^31 or more blocks of 128 rows, or 2^37 or more of one row) or
 * FARN_ERR_CUDA. */
int farn_fp8_quantize(const farn_ctx *ctx, const void *x, int64_t E, int64_t T,
                      int64_t H, int block_rows, void *codes, float *scales,
                      cudaStream_t stream);

/* farn_fp8_matmul - the product of two E4M3 tensors with block scales, for
 * example activations by weights:
 *     out[t,n] = bf16( sum_b s[t,n,b] * sum_{h in block b} f(a[t,h]) * f(b[n,h]) )
 *     s[t,n,b] = a_scale[t,b] * b_scale[n / 128, b],  rounded to fp32
 * over the blocks b of 128 elements of a row, every sum in fp32 (the order is
 * the kernel's own and the same in every call with the same arguments), one
 * rounding to bf16.
 *   a_codes uint8 [T, H], a_scale fp32 [T, ceil(H/128)];
 *   b_codes uint8 [N, H], b_scale fp32 [ceil(N/128), ceil(H/128)]: what
 *   farn_fp8_quantize makes with block_rows 1 and 128;  out bf16 [T, N]
 *   T, N, H < 2^31; T == 0 launches nothing
 * The fast kernels need the codes 16-byte aligned and H a multiple of 16; other
 * shapes are served by a slower kernel.  Returns FARN_ERR_INVALID_ARG,
 * FARN_ERR_ALIAS, FARN_ERR_UNSUPPORTED (2^30 or more tiles of 64 rows by 64
 * columns) or FARN_ERR_CUDA. */
int farn_fp8_matmul(const farn_ctx *ctx, const void *a_codes,
                    const float *a_scale, const void *b_codes,
                    const float *b_scale, int64_t T, int64_t N, int64_t H,
                    void *out, cudaStream_t stream);

/* farn_fp8_grouped_matmul - farn_grouped_matmul on E4M3 codes with block
 * scales: x [n_rows, H] with x_scale [n_rows, ceil(H/128)], weights [E, N, H]
 * with w_scale [E, ceil(N/128), ceil(H/128)].  Slots, rows, offsets, out and
 * errors as there; arithmetic as in farn_fp8_matmul.
 *   workspace  NULL, or workspace_bytes of device memory (16-byte aligned) that
 *              the call may overwrite, for this call alone until it has run: a
 *              long call with `rows` lays the slots' rows side by side there
 *              first and is then faster.  farn_fp8_grouped_workspace says how
 *              much such a call takes; with less, or none, the other kernel runs,
 *              whose sums are in another order: its results are the same up to the
 *              rounding of fp32 sums, not always bit for bit.  It may not overlap any
 *              tensor. */
int farn_fp8_grouped_matmul(const farn_ctx *ctx, const void *x,
                            const float *x_scale, int64_t n_rows,
                            const int32_t *rows, int64_t n_slots,
                            const void *weights, const float *w_scale, int E,
                            const int32_t *offsets, int64_t N, int64_t H,
                            void *out, void *workspace, int64_t workspace_bytes,
                            cudaStream_t stream);

/* The workspace that a farn_fp8_grouped_matmul call with `rows` and these sizes
 * uses: *bytes, 0 if none.  Returns FARN_OK or FARN_ERR_INVALID_ARG. */
int farn_fp8_grouped_workspace(const farn_ctx *ctx, int64_t n_slots, int E,
                               int64_t N, int64_t H, int64_t *bytes);

/* Which kernel farn_fp8_matmul or farn_fp8_grouped_matmul would launch for these
 * sizes and pointers, without launching: 2 generic (any H or alignment), 6 tensor
 * (the tensor cores, a tile of 128 weights by 64 slots per CTA, *ctas of them
 * splitting the row), 7 pair (the tensor cores, two CTAs per tile of 256 slots by
 * 256 weights; with `rows` only if a workspace is given, here any 16-byte aligned
 * pointer).  Otherwise as farn_plan_grouped_matmul. */
int farn_plan_fp8_matmul(const farn_ctx *ctx, const void *a_codes,
                         const void *b_codes, int64_t T, int64_t N, int64_t H,
                         const void *out, int *variant, int *ctas, int *threads);
int farn_plan_fp8_grouped_matmul(const farn_ctx *ctx, const void *x,
                                 int64_t n_rows, const int32_t *rows,
                                 int64_t n_slots, const void *weights, int E,
                                 int64_t N, int64_t H, const void *out,
                                 const void *workspace, int *variant, int *ctas,
                                 int *threads);

/* farn_qk_norm_rope - RMSNorm of every query and key head and its rotation by
 * position, in one pass.  For a head's elements x[0..D):
 *     y[i] = (x[i] * rstd) * f(weight[i]),  rstd = 1 / sqrt(mean(x^2) + eps)
 *            (y = x where the weight is NULL)
 *     for the pairs j < R/2 of the first R elements, (a, b) = (y[j], y[j + R/2]),
 *     or (y[2j], y[2j+1]) with `interleaved`:
 *            (a cos w - b sin w, b cos w + a sin w),  w = positions[axis(j), t] * freqs[j]
 *     elements from R on stay y
 * in fp32, one rounding to bf16.  The angle is exact to 2^-31 of a turn whatever
 * the position (|freqs| up to 2^8).
 *   T, D        tokens (< 2^31; 0 launches nothing), elements of a head (1 .. 1024)
 *   q           bf16 [T, q_heads, D], tokens q_stride elements apart (at least
 *               q_heads * D): heads may be read where a projection wrote them;
 *               k the same.  Either may have 0 heads (its pointers are not read).
 *   q_weight, k_weight  bf16 [D] or NULL
 *   positions   int32 [axes, T], axes 1 .. 4; freqs fp32 [R / 2], finite
 *   sections    host array [axes]: how many pairs turn by each axis, in order;
 *               their sum is R / 2
 *   R           even, 0 .. D; 0: no rotation (axes, sections, positions and freqs
 *               are not read)
 *   q_out, k_out  bf16, with strides of their own; each may be exactly its input
 *               (same address and stride), and rows of equal strides may lie
 *               between each other's
 * Fast: D a multiple of 8 up to 256, strides multiples of 4, pointers 8-byte
 * aligned, and R a multiple of 8 unless interleaved; else a slower kernel.  Returns
 * FARN_ERR_INVALID_ARG, FARN_ERR_ALIAS or FARN_ERR_CUDA. */
int farn_qk_norm_rope(const farn_ctx *ctx, int64_t T, int D, const void *q,
                      int q_heads, int64_t q_stride, const void *k, int k_heads,
                      int64_t k_stride, const void *q_weight,
                      const void *k_weight, float eps, const int32_t *positions,
                      int axes, const int *sections, const float *freqs, int R,
                      int interleaved, void *q_out, int64_t q_out_stride,
                      void *k_out, int64_t k_out_stride, cudaStream_t stream);

/* Formats of a cache of keys and values. */
#define FARN_CACHE_FP8 1    /* E4M3 codes, an fp32 scale per token and head */
#define FARN_CACHE_NVFP4 2  /* farn_nvfp4_quantize's codes and block scales */

/* A paged cache of keys and values.  Slot s of the cache, page s / page_size,
 * holds one token's `heads` rows of head_dim values, of keys and of values.
 *   codes   uint8 [n_pages, page_size, heads, head_dim] (FARN_CACHE_FP8) or
 *           [.., head_dim / 2] (FARN_CACHE_NVFP4, head_dim a multiple of 16)
 *   scale   fp32 [n_pages, page_size, heads], or uint8 [.., head_dim / 16]
 *   tensor scales: NVFP4 only, finite, > 0
 * n_pages * page_size < 2^31; head_dim 1 .. 1024.  A row in FARN_CACHE_FP8 is one
 * block of farn_fp8_quantize's arithmetic. */
typedef struct {
    int format;
    int page_size;
    int64_t n_pages;
    int heads, head_dim;
    void *k_codes, *v_codes;
    void *k_scale, *v_scale;
    float k_tensor_scale, v_tensor_scale;
} farn_kv_cache;

/* farn_qk_norm_rope with keys and values written to a cache instead: the
 * queries go to q_out, token t's keys (normed and rotated) and values (as they
 * are) to slot slots[t], quantised from fp32.  A slot outside the cache (for
 * example -1, padding) is skipped; its queries are written all the same.  The
 * slots of one call have to differ: a slot that two tokens write holds codes and
 * scales of either.  slots int32 [T]; v bf16 [T, kv_heads, D].  q_heads may be 0.
 * Fast: as farn_qk_norm_rope (v as q and k), with the cache's codes 4-byte (NVFP4:
 * 2-byte) aligned, and for an NVFP4 cache either interleaved, or R = 0, or R = D and
 * D a multiple of 32.  Every other rotation of halves into an NVFP4 cache takes the
 * slower kernel with the whole call, queries too (8192 tokens of 40 and 8 heads of
 * 128 with R = 64: 189 us, interleaved 46 us).  Returns FARN_ERR_INVALID_ARG (also
 * for a cache of other sizes), FARN_ERR_ALIAS or FARN_ERR_CUDA. */
int farn_qk_norm_rope_cache(const farn_ctx *ctx, int64_t T, int D,
                            const void *q, int q_heads, int64_t q_stride,
                            const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, int kv_heads,
                            const void *q_weight, const void *k_weight,
                            float eps, const int32_t *positions, int axes,
                            const int *sections, const float *freqs, int R,
                            int interleaved, void *q_out, int64_t q_out_stride,
                            const farn_kv_cache *cache, const int32_t *slots,
                            cudaStream_t stream);

/* farn_kv_write - keys and values bf16 [T, heads, head_dim] (token strides of
 * their own) quantised into the cache's slots, as they are.  Otherwise as
 * farn_qk_norm_rope_cache with R = 0. */
int farn_kv_write(const farn_ctx *ctx, int64_t T, const void *k,
                  int64_t k_stride, const void *v, int64_t v_stride,
                  const farn_kv_cache *cache, const int32_t *slots,
                  cudaStream_t stream);

/* farn_kv_read - the contexts of B sequences back in bf16, one after the
 * other: output token n of sequence b, offsets[b] <= n < offsets[b+1], is the
 * sequence's token i = n - offsets[b], in slot table[b, i / page_size] *
 * page_size + i % page_size:
 *     fp8    bf16(value(code) * scale)
 *     nvfp4  bf16(value(code) * (value(block scale) / tensor_scale)), as
 *            farn_nvfp4_dequantize
 *   table    int32 [B, width];  a page outside the cache, or beyond the table,
 *            reads as zeros
 *   offsets  int32 [B + 1] on the device, ascending, within 0 .. n_tokens.
 *            (Other values cannot lead outside the tensors, but the outputs
 *            are then unspecified.)
 *   k_out, v_out  bf16 [n_tokens, heads, head_dim]; tokens below offsets[0] and
 *            from offsets[B] on are left as they were
 * n_tokens == 0 or B == 0 launches nothing.  Fast: head_dim a multiple of 8,
 * codes 8-byte (NVFP4: 4-byte) and outputs 16-byte aligned.  Returns
 * FARN_ERR_INVALID_ARG, FARN_ERR_ALIAS, FARN_ERR_UNSUPPORTED (heads * head_dim
 * of 2^26 or more) or FARN_ERR_CUDA. */
int farn_kv_read(const farn_ctx *ctx, const farn_kv_cache *cache,
                 const int32_t *table, int B, int64_t width,
                 const int32_t *offsets, int64_t n_tokens, void *k_out,
                 void *v_out, cudaStream_t stream);

/* Flags of farn_plan_typed. */
#define FARN_PLAN_FP8_OUT 1   /* the call also writes the FP8 norm output */
#define FARN_PLAN_NVFP4_OUT 2 /* the call also writes the NVFP4 norm output */

/* farn_plan for partials of type `partial_dtype` (a farn_dtype), for a
 * farn_forward_typed call (flags 0), a farn_forward_quant call
 * (FARN_PLAN_FP8_OUT) or a farn_forward_nvfp4 call (FARN_PLAN_NVFP4_OUT);
 * with either flag norm_out may be NULL.  Only shape, dtype,
 * flags and pointer alignment matter; aliasing is not checked.  Returns
 * FARN_ERR_INVALID_ARG for a bad shape, dtype, flag or NULL pointer. */
int farn_plan_typed(const farn_ctx *ctx, int partial_dtype, int flags, int W,
                    int64_t T, int64_t H,
                    const void *const *partials, const void *residual,
                    const void *weight, const void *reduced_out,
                    const void *residual_out, const void *norm_out,
                    int *variant, int *cluster_size, int *threads);

#ifdef __cplusplus
}
#endif

#endif /* FARN_H_ */
