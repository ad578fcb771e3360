/*
 * linear_layer.h — C ABI of the MI355X (gfx950) GEMM / fully-connected library.
 *
 * Every entry point enqueues work on the caller's HIP stream and returns at
 * once; it never synchronises, never allocates device memory and keeps no
 * state between calls beyond a read-only cache of device properties. All
 * matrix pointers are DEVICE pointers owned by the caller. Matrices are
 * row-major: element (r, c) of a matrix with leading dimension ld is at
 * ptr[r * ld + c]. Dimensions and leading dimensions are int; offsets are
 * computed in 64 bits inside.
 *
 * Errors are never fatal: no abort, no exception crosses this boundary. Each
 * call returns one of the LL_* status codes below. Argument errors are found
 * on the host before anything is enqueued; faults during execution surface
 * on the stream like those of any other kernel.
 *
 * `stream` is a hipStream_t passed as void* (NULL = the default stream), so
 * that this header needs no HIP header.
 */
#ifndef LINEAR_LAYER_H
#define LINEAR_LAYER_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define LL_OK 0
#define LL_ERR_INVALID_VALUE 1   /* negative dimension, leading dimension too small,
                                    NULL pointer that would be dereferenced, pointer not
                                    aligned to its element size, unknown activation,
                                    an output range overlapping an input range, or an
                                    output whose tiles exceed one launch's grid (only
                                    extreme shapes: M or N within about 2^8 of 2^31
                                    with the other one small) */
#define LL_ERR_NO_DEVICE 2       /* no HIP device is current / visible */
#define LL_ERR_UNSUPPORTED_ARCH 3/* the current device is not gfx950 (MI355X class) */
#define LL_ERR_LAUNCH 4          /* the HIP runtime reported an error at launch */

/* Activations: of linear_bias_act the first two, of linear16_nt and its gradient all. */
#define LL_ACT_NONE 0
#define LL_ACT_RELU 1
#define LL_ACT_GELU 2       /* z * (1 + erf(z / sqrt(2))) / 2 */
#define LL_ACT_GELU_TANH 3  /* z * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3))) / 2 */
#define LL_ACT_SILU 4       /* z / (1 + exp(-z)) */

/*
 * gemm_f32 — C = alpha * A * B + beta * C in FP32.
 *
 * Defined on page "GEMM 优化详解" (GEMM optimisation in detail), section
 * "GEMM 基础理论 / 数学定义" (mathematical definition): the general form
 * C = alpha*A*B + beta*C with A M-by-K, B K-by-N, C M-by-N and
 * C(m,n) = sum_k A(m,k) * B(k,n). The same sum is on page "第5章-基础Kernel",
 * section 1.1.
 *
 *   M, N, K   >= 0. M == 0 or N == 0: returns LL_OK, touches nothing.
 *   A         M-by-K fp32, lda >= max(1, K). Read only if K > 0 and alpha != 0.
 *   B         K-by-N fp32, ldb >= max(1, N). Read only if K > 0 and alpha != 0.
 *   C         M-by-N fp32, ldc >= max(1, N), in/out. Read only if beta != 0, so
 *             with beta == 0 any bit pattern (NaN included) in C is ignored.
 *   alpha, beta  fp32 scalars (host values). K == 0 or alpha == 0 gives C = beta*C.
 *   stream    hipStream_t (void*), NULL for the default stream.
 *
 * Products are accumulated in FP32 on the matrix cores (MFMA), in an order of
 * the kernel's choosing. C must not overlap A or B. Pointers need only be
 * 4-byte aligned; 16-byte aligned pointers with lda, ldb, ldc, K and N all
 * multiples of 4 take the direct-to-LDS kernels; anything else the
 * register-staged kernels, which load 128-bit chunks at any alignment and
 * the chunk that crosses K or N element by element.
 */
int gemm_f32(int M, int N, int K, float alpha,
             const float *A, int lda, const float *B, int ldb,
             float beta, float *C, int ldc, void *stream);

/*
 * gemm_f16f32 — C = alpha * A * B + beta * C with IEEE binary16 A and B,
 * FP32 accumulation and FP32 C.
 *
 * The FP16-input / FP32-accumulate product of page
 * "GPU架构下的矩阵乘法深入优化" (in-depth matrix-multiply optimisation on
 * GPU architecture), section 6 (tensor-core implementation), in the general
 * form of page "GEMM 优化详解", section "GEMM 基础理论 / 数学定义".
 *
 *   A  M-by-K binary16 bit patterns (uint16_t), lda >= max(1, K).
 *   B  K-by-N binary16 bit patterns, ldb >= max(1, N).
 *   C  M-by-N fp32, ldc >= max(1, N).
 * Every other argument, rule and error as gemm_f32. Pointers to A and B need
 * only be 2-byte aligned; the direct-to-LDS kernels need 16-byte aligned
 * pointers and lda, ldb, K, N multiples of 8 (ldc a multiple of 4), other
 * operands run the register-staged kernels.
 */
int gemm_f16f32(int M, int N, int K, float alpha,
                const uint16_t *A, int lda, const uint16_t *B, int ldb,
                float beta, float *C, int ldc, void *stream);

/*
 * gemm_bf16f32 — C = alpha * A * B + beta * C with bfloat16 A and B, FP32
 * accumulation and FP32 C.
 *
 * Page "GEMM 优化详解", section "进一步优化方向" (further directions),
 * item "Tensor Core (WMMA)": the matrix units take FP16 or BF16 inputs. Same
 * product as gemm_f16f32 with the inputs in bfloat16 (1 sign, 8 exponent,
 * 7 fraction bits) instead of binary16.
 *
 *   A  M-by-K bfloat16 bit patterns (uint16_t), lda >= max(1, K).
 *   B  K-by-N bfloat16 bit patterns, ldb >= max(1, N).
 * Every other argument, rule and error as gemm_f16f32 (same kernels and tile
 * shapes, selected by LL_DTYPE_F16 below).
 */
int gemm_bf16f32(int M, int N, int K, float alpha,
                 const uint16_t *A, int lda, const uint16_t *B, int ldb,
                 float beta, float *C, int ldc, void *stream);

/*
 * linear_bias_act — Y = act(X * W + bias), the fused fully-connected layer.
 *
 * Page "GEMM 优化详解", table "为什么 GEMM 重要" (an FC layer is
 * Y = X*W + b) and section "Level 6: Kernel Fusion" (the bias, indexed by
 * output column, and then the ReLU are applied in the GEMM's write-back, so
 * the intermediate never goes to memory). The page's four flag combinations
 * map to (bias != NULL) x (act).
 *
 *   X     M-by-K fp32 (a batch of M input rows), ldx >= max(1, K).
 *   W     K-by-N fp32 weights, row-major K-by-N, ldw >= max(1, N).
 *   bias  N fp32 values, or NULL for no bias.
 *   act   LL_ACT_NONE or LL_ACT_RELU; ReLU maps y <= 0 (and NaN) to +0.0.
 *   Y     M-by-N fp32 output, ldy >= max(1, N); never read.
 * K == 0 gives Y = act(bias) (or act(0)). Y must not overlap X, W or bias.
 * Alignment rules as gemm_f32.
 */
int linear_bias_act(int M, int N, int K,
                    const float *X, int ldx, const float *W, int ldw,
                    const float *bias, int act,
                    float *Y, int ldy, void *stream);

/*
 * Transposed-B forms: B (or W) is given N-by-K, row-major, leading dimension
 * ldb >= max(1, K) (ldw for W), so that its element (k, n) is at B[n*ldb + k]:
 *
 *   gemm_f32_nt, gemm_f16f32_nt, gemm_bf16f32_nt:  C = alpha * A * B^T + beta * C
 *   linear_bias_act_nt:                            Y = act(X * W^T + bias)
 *
 * This is how a fully-connected weight is usually stored ([out][in]) and the
 * shape of products such as Q * K^T (page "GEMM 优化详解", table
 * "为什么 GEMM 重要"). B is then k-contiguous like A and the kernels stage and
 * read it exactly like A. Every other argument, rule and error is that of the
 * corresponding function above; the 128-bit kernels need ldb (ldw) to be a
 * multiple of 4 (fp32) or 8 (16-bit) instead of N.
 */
int gemm_f32_nt(int M, int N, int K, float alpha,
                const float *A, int lda, const float *B, int ldb,
                float beta, float *C, int ldc, void *stream);
int gemm_f16f32_nt(int M, int N, int K, float alpha,
                   const uint16_t *A, int lda, const uint16_t *B, int ldb,
                   float beta, float *C, int ldc, void *stream);
int gemm_bf16f32_nt(int M, int N, int K, float alpha,
                    const uint16_t *A, int lda, const uint16_t *B, int ldb,
                    float beta, float *C, int ldc, void *stream);
int linear_bias_act_nt(int M, int N, int K,
                       const float *X, int ldx, const float *W, int ldw,
                       const float *bias, int act,
                       float *Y, int ldy, void *stream);

/*
 * linear_bias_act_ws — the fused layer of linear_bias_act (w_layout
 * LL_W_K_BY_N) or linear_bias_act_nt (LL_W_N_BY_K) with a caller-provided
 * workspace, so that the bias and ReLU stay fused into the write-back of
 * every output tile (page "GEMM 优化详解", "Level 6: Kernel Fusion").
 *
 * Without a workspace, a plan that shares the K range of leftover tiles out
 * over several workgroups (stream-K; e.g. 2047 x 11008 x 4096, 88 of 344
 * tiles) adds their partial sums atomically into Y, which a pass fills with
 * the bias first and another pass finishes with the ReLU: three launches.
 * With a workspace of at least ll_linear_workspace_size bytes, the partial
 * sums go to a workspace tile and the last workgroup to contribute to a tile
 * applies bias and ReLU and writes it: one launch, no pass over Y.
 *
 *   workspace        device memory owned by the caller, 256-byte aligned, not
 *                    overlapping X, W, bias or Y; it must hold zeros before
 *                    its first use (e.g. hipMemset to 0), and every call that
 *                    completes leaves it holding zeros again. NULL (with
 *                    workspace_bytes 0) or a workspace smaller than the plan
 *                    needs: the three-launch plan runs, with the same result
 *                    up to the order of the atomic additions.
 *   workspace_bytes  its size in bytes.
 * Calls that use one workspace must not overlap in time (on one stream they
 * never do); calls with different workspaces are independent. Everything
 * else as linear_bias_act / linear_bias_act_nt; LL_ERR_INVALID_VALUE also for
 * an unknown w_layout or a misaligned or overlapping workspace.
 */
#define LL_W_K_BY_N 0
#define LL_W_N_BY_K 1
int linear_bias_act_ws(int M, int N, int K,
                       const float *X, int ldx, const float *W, int ldw, int w_layout,
                       const float *bias, int act,
                       float *Y, int ldy, void *workspace, int64_t workspace_bytes,
                       void *stream);
/* Bytes of workspace linear_bias_act_ws uses for this shape on a device with
 * num_cus compute units (num_cus <= 0: 256), assuming 128-bit-aligned
 * operands (other calls use less or none); 0 if its plan needs none; -1 for
 * a negative size or an unknown w_layout or act. Honours the overrides of
 * linear_layer_tuning.h. For 2047 x 11008 x 4096 on 256 CUs: 88 tiles of
 * 256 KiB plus counters, about 22 MiB. */
int64_t ll_linear_workspace_size(int M, int N, int K, int w_layout, int act, int num_cus);

/*
 * linear_bias_act_noalloc — linear_bias_act_ws for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): the workspace is the library's own
 * static device array of LL_NOALLOC_SCRATCH_BYTES (one per GPU, held until
 * the process ends), so the call allocates nothing and takes no workspace
 * argument. The array covers every plan on a device of up to 256 compute
 * units (a stream-K plan shares out less than one round of tiles: at most
 * 64 MiB of partial tiles plus their counters). A shape whose plan needs more
 * workspace than that (see ll_linear_workspace_size) returns
 * LL_ERR_INVALID_VALUE and runs nothing.
 * Every call on one GPU uses that GPU's single array: calls that overlap in
 * time on one GPU (other streams, other threads) race and give wrong
 * results; calls on one stream never overlap. Each call leaves the array
 * zero-filled, as the next one needs it. The array used is the current
 * device's, so `stream` must belong to the current device (else
 * LL_ERR_INVALID_VALUE). Arguments and results otherwise as
 * linear_bias_act_ws.
 */
#define LL_NOALLOC_SCRATCH_BYTES (65ll << 20)
int linear_bias_act_noalloc(int M, int N, int K,
                            const float *X, int ldx, const float *W, int ldw, int w_layout,
                            const float *bias, int act,
                            float *Y, int ldy, void *stream);

/*
 * Strided-batched products (page "GEMM 优化详解", section "矩阵大小选择策略":
 * small matrices are best run as one batched GEMM). For i in [0, batch):
 *
 *   C_i = alpha * A_i * op(B_i) + beta * C_i,   op(B) = B (trans_b 0) or B^T (trans_b 1)
 *
 * with A_i = A + i*stride_a, B_i = B + i*stride_b, C_i = C + i*stride_c
 * (strides in ELEMENTS of the operand's type). Each item follows the rules of
 * gemm_f32 / gemm_f16f32 / gemm_bf16f32 (trans_b 0: B_i K-by-N, ldb >= N;
 * trans_b 1: B_i N-by-K, ldb >= K). A stride of 0 shares one A or B among all
 * items; C items must not overlap (stride_c >= (M-1)*ldc + N when batch > 1),
 * and the address range spanned by all C items must not meet that of A's or
 * B's items. batch == 0 returns LL_OK with no launch; negative strides or
 * batch, or trans_b outside {0, 1}, give LL_ERR_INVALID_VALUE. All items run
 * in one launch (several when batch exceeds 65535), their tiles sharing the
 * CUs. The 128-bit kernels also need stride_a, stride_b (in bytes) and
 * stride_c*4 to be multiples of 16.
 */
int gemm_f32_batched(int trans_b, int M, int N, int K, float alpha,
                     const float *A, int lda, int64_t stride_a,
                     const float *B, int ldb, int64_t stride_b,
                     float beta, float *C, int ldc, int64_t stride_c,
                     int batch, void *stream);
int gemm_f16f32_batched(int trans_b, int M, int N, int K, float alpha,
                        const uint16_t *A, int lda, int64_t stride_a,
                        const uint16_t *B, int ldb, int64_t stride_b,
                        float beta, float *C, int ldc, int64_t stride_c,
                        int batch, void *stream);
int gemm_bf16f32_batched(int trans_b, int M, int N, int K, float alpha,
                         const uint16_t *A, int lda, int64_t stride_a,
                         const uint16_t *B, int ldb, int64_t stride_b,
                         float beta, float *C, int ldc, int64_t stride_c,
                         int batch, void *stream);

/*
 * Microscaled 4-bit floating point (MX4). A matrix of rows x K values is held
 * as codes and scales. Each row is cut into blocks of 32 values (the last one
 * may be shorter). A value is a 4-bit code: bit 3 the sign, bits 2..1 an
 * exponent, bit 0 a fraction, standing for 0, 0.5, 1, 1.5, 2, 3, 4 or 6. Two
 * codes share a byte, the earlier value in bits 3..0; a row has ceil(K/2)
 * bytes, and bits past its K values are written 0 and never used. A block has
 * one scale byte s, and its values are the codes' times 2^(s - 127); s = 255
 * makes all of them NaN. A row has ceil(K/32) scale bytes. This is the
 * element and scale encoding that the OCP Microscaling Formats specification
 * calls MXFP4 (E2M1 elements, E8M0 scales, blocks of 32).
 *
 * Leading dimensions of codes and scales are in BYTES; neither needs any
 * alignment.
 */

/* Element types of the microscaled formats, the residual norms and the 16-bit layer. */
#define LL_TYPE_F32 0
#define LL_TYPE_F16 1
#define LL_TYPE_BF16 2

/*
 * mx4_quantize — X (M-by-K, `type`, ldx >= max(1, K) elements) into MX4.
 * A block whose largest magnitude is t gets the scale 2^e with
 * e = floor(log2(t)) - 2, at least -127 (t = 0: -127), and each value v the
 * code nearest to v / 2^e, ties to the even code, magnitudes past 6 to 6. A
 * block that holds an infinity or a NaN gets the scale byte 255 and codes 0.
 *
 *   trans 0   codes: M rows of ceil(K/2) bytes, ldq >= max(1, that) apart;
 *             scales: M rows of ceil(K/32) bytes, lds >= max(1, that) apart.
 *   trans 1   the transposed matrix is quantised: K rows of M values, blocks
 *             along X's columns. A layer's backward products contract over
 *             other axes than its forward product and need their operands so.
 * The outputs must not overlap X or each other. M == 0 or K == 0: LL_OK,
 * touches nothing.
 */
int mx4_quantize(int M, int K, int type, const void *X, int ldx, int trans,
                 uint8_t *codes, int ldq, uint8_t *scales, int lds, void *stream);

/*
 * mx4_dequantize — Y (M-by-K, `type`, ldy >= max(1, K)) = the values that
 * codes and scales stand for. FP32 and bfloat16 hold each of them exactly, up
 * to their largest finite value; binary16 rounds those below 2^-24 steps and
 * overflows to infinity past 65504. Y must not overlap codes or scales.
 */
int mx4_dequantize(int M, int K, const uint8_t *codes, int ldq, const uint8_t *scales, int lds,
                   int type, void *Y, int ldy, void *stream);

/*
 * gemm_mx4f32_nt — C = alpha * A * B^T + beta * C with A (M-by-K) and B
 * (N-by-K, the [out][in] layout of a weight) in MX4, FP32 sums and FP32 C.
 * gemm_f16mx4f32_nt, gemm_bf16mx4f32_nt — the same with A in binary16 or
 * bfloat16 (bit patterns; lda >= max(1, K) elements) and B in MX4: every
 * decoded value of B enters its products exactly, whatever its scale (those past
 * bfloat16's range too, more slowly).
 *
 *   SA, SB    the scales of A and B; ldsa, ldsb >= max(1, ceil(K/32)) bytes.
 *   lda, ldb  bytes between rows of codes, >= max(1, ceil(K/2)).
 * Other arguments, rules and errors as gemm_f32: with beta == 0 C is not
 * read, K == 0 or alpha == 0 gives C = beta*C and reads neither operand, C
 * must not overlap an input. One launch (several where one cannot count the work
 * items: 2^27 rows of A or B and more), nothing allocated; the summation
 * order is fixed by the shape and the alignment, so equal calls give equal
 * results. Rows (of A, of B) 16 bytes aligned take direct copies into LDS when
 * the product is large; any other alignment is taken too.
 */
int gemm_mx4f32_nt(int M, int N, int K, float alpha,
                   const uint8_t *A, int lda, const uint8_t *SA, int ldsa,
                   const uint8_t *B, int ldb, const uint8_t *SB, int ldsb,
                   float beta, float *C, int ldc, void *stream);
int gemm_f16mx4f32_nt(int M, int N, int K, float alpha, const uint16_t *A, int lda,
                      const uint8_t *B, int ldb, const uint8_t *SB, int ldsb,
                      float beta, float *C, int ldc, void *stream);
int gemm_bf16mx4f32_nt(int M, int N, int K, float alpha, const uint16_t *A, int lda,
                       const uint8_t *B, int ldb, const uint8_t *SB, int ldsb,
                       float beta, float *C, int ldc, void *stream);

/*
 * The same products with a workspace. Where a product has few output tiles and a
 * long K (some ten to some hundred rows of A), K is shared out over workgroups,
 * whose sums go through the workspace and are added in order by a second launch;
 * others ignore it.
 *
 *   workspace   NULL (the plain call), or at least ll_mx4_workspace_size(M, N, K,
 *               a) bytes, 16-byte aligned, overlapping nothing; its contents need
 *               no preparation. Calls that share one must not overlap in time.
 * ll_mx4_workspace_size: bytes that help this shape on the current device, 0 if
 * none do; -1 for a negative size or an unknown `a` (LL_A_*, the form of A).
 */
#define LL_A_MX4 0
#define LL_A_F16 1
#define LL_A_BF16 2
int64_t ll_mx4_workspace_size(int M, int N, int K, int a);
int gemm_mx4f32_nt_ws(int M, int N, int K, float alpha,
                      const uint8_t *A, int lda, const uint8_t *SA, int ldsa,
                      const uint8_t *B, int ldb, const uint8_t *SB, int ldsb,
                      float beta, float *C, int ldc,
                      void *workspace, int64_t workspace_bytes, void *stream);
int gemm_f16mx4f32_nt_ws(int M, int N, int K, float alpha, const uint16_t *A, int lda,
                         const uint8_t *B, int ldb, const uint8_t *SB, int ldsb,
                         float beta, float *C, int ldc,
                         void *workspace, int64_t workspace_bytes, void *stream);
int gemm_bf16mx4f32_nt_ws(int M, int N, int K, float alpha, const uint16_t *A, int lda,
                          const uint8_t *B, int ldb, const uint8_t *SB, int ldsb,
                          float beta, float *C, int ldc,
                          void *workspace, int64_t workspace_bytes, void *stream);
/* Name of the kernel such a product takes on a device with num_cus compute units
 * (num_cus <= 0: 256), with rows of A and B on 16 bytes (`aligned`) and with a
 * workspace or not: "rows", "rows_shared", "tiny", "short", "tile_256x256",
 * "tile_128x128" or "stream_" and a tile's size; "" for a product without work or a
 * bad argument. Static string. */
const char *ll_mx4_chosen_kernel(int M, int N, int K, int a, int aligned, int workspace, int num_cus);

/*
 * rmsnorm_residual — the residual step between two blocks of a network, the
 * norm after the one and the norm before the other in one pass. For each row,
 * with r(v) = 1 / sqrt(mean(v^2) + eps):
 *
 *   x' = x + alpha * gate * (y * r(y) * w_post)
 *   h  = x' * r(x') * w_pre
 *
 *   Y       the block's output, M-by-N fp32 as every product here writes it,
 *           ldy >= max(1, N); NULL: x' = x (the norm before the first block).
 *   X       the residual stream, M-by-N of `type` (LL_TYPE_*).
 *   XO, H   x' and h, M-by-N of `type`; either may be NULL (not both). XO may
 *           be X itself (same ld); no other overlap of an output is allowed.
 *   w_post, gate, w_pre   N fp32 values each; NULL stands for ones.
 *   alpha   the residual scale; eps >= 0, finite.
 * Arithmetic is FP32; h is computed from x' before its rounding. Any ld,
 * alignment (to the element) and N. M == 0 or N == 0: LL_OK.
 */
int rmsnorm_residual(int M, int N, int type, const float *Y, int ldy,
                     const float *w_post, const float *gate, float alpha,
                     const void *X, int ldx, const float *w_pre, float eps,
                     void *XO, int ldxo, void *H, int ldh, void *stream);

/*
 * rmsnorm_residual_grad — its gradient. DXO and DH (M-by-N of `type`) are the
 * gradients that reach x' and h; either may be NULL for zero (not both). The
 * forward inputs are given again (X before any in-place update). Outputs, each
 * of which may be NULL: DY (M-by-N fp32), DX (M-by-N of `type`; may be DXO
 * itself, same ld), and the sums over rows dgate, dw_post, dw_pre (N fp32
 * values). Without Y, DY, dgate and dw_post must be NULL.
 *
 *   workspace   at least ll_rmsnorm_grad_workspace_size(M, N) bytes, 16-byte
 *               aligned, overlapping nothing; its contents need no
 *               preparation. Calls that share one must not overlap in time.
 * The order of the sums is fixed by the shape. M == 0 with N > 0 writes zeros
 * to dgate, dw_post and dw_pre.
 */
int rmsnorm_residual_grad(int M, int N, int type, const void *DXO, int lddxo, const void *DH, int lddh,
                          const float *Y, int ldy, const float *w_post, const float *gate, float alpha,
                          const void *X, int ldx, const float *w_pre, float eps,
                          float *DY, int lddy, void *DX, int lddx,
                          float *dgate, float *dw_post, float *dw_pre,
                          void *workspace, int64_t workspace_bytes, void *stream);
/* Bytes of workspace rmsnorm_residual_grad needs (at most 8 * 1024 * N for N
 * up to 8192); -1 for a negative size. */
int64_t ll_rmsnorm_grad_workspace_size(int M, int N);

/*
 * Microscaled 8-bit floating point (MX8): rows of values in blocks of 32 (the last
 * one may be shorter), a byte a value and a scale byte s a block. A byte is an
 * E4M3 number (sign, four bits of exponent with bias 7, three of fraction; up
 * to 448, no infinities, 0x7f and 0xff NaN), the block's values are the
 * numbers times 2^(s - 127), and s = 255 makes all of them NaN. A row of K values has K
 * bytes of codes and ceil(K/32) of scales. The encoding is the one that the
 * OCP Microscaling Formats specification calls MXFP8. Leading dimensions of
 * codes and scales are in bytes; neither needs any alignment.
 *
 * mx8_quantize — X (M-by-K, `type`, ldx >= max(1, K) elements) into MX8. A
 * block whose largest magnitude is t gets the smallest scale 2^e, e >= -127,
 * with t <= 448 * 2^e, so no value is clipped, and each value v the code
 * nearest to v / 2^e, ties to the even code (t = 0: e = -127). A block that holds an
 * infinity or a NaN gets the scale byte 255 and codes 0.
 * mx8_dequantize — Y (M-by-K, `type`) = the values that codes and scales
 * stand for. FP32 holds them exactly down to its smallest subnormal, bfloat16 down
 * to its own, both up to 2^128, which magnitudes from 2^128 - 2^123 on round to and
 * which is infinity in them; binary16 rounds those below 2^-14 and overflows to infinity
 * past 65504.
 * Outputs must not overlap inputs or each other. M == 0 or K == 0: LL_OK,
 * touches nothing.
 */
int mx8_quantize(int M, int K, int type, const void *X, int ldx,
                 uint8_t *codes, int ldq, uint8_t *scales, int lds, void *stream);
int mx8_dequantize(int M, int K, const uint8_t *codes, int ldq, const uint8_t *scales, int lds,
                   int type, void *Y, int ldy, void *stream);

/*
 * The 16-bit layer: a fully-connected layer with its write-back, and its gradients,
 * in binary16 or bfloat16 (`type`: LL_TYPE_F16 or LL_TYPE_BF16) with FP32 sums; dense,
 * or by groups of rows, as the experts of a mixture have them.
 *
 *   groups, offsets   NULL with groups 1: one weight for all M rows. Otherwise
 *           groups + 1 ascending row numbers in DEVICE memory (4-byte aligned):
 *           group g has the rows offsets[g] .. offsets[g+1] - 1 and a weight of its
 *           own. A group may be empty. Rows before offsets[0] and from
 *           offsets[groups] on belong to none: nothing of theirs is read or
 *           written. The numbers are read by the kernels (no copy to the host); one
 *           outside 0 .. M is taken as the nearer of the two, and one below its
 *           predecessor as that. At most LL_MAX_GROUPS groups; 0 groups: nothing happens.
 *   W       N-by-K of `type` ([out][in]), ldw >= max(1, K); group g's is stride_w * g
 *           elements after the first (0: one weight for all groups).
 * Sizes up to 2^31 - 1025 (and as many tiles as one launch takes); operands
 * need only the alignment of their elements. Where rows of X and W (of dZ and W, of dZ and X) are
 * whole multiples of 16 bytes on 16 bytes, copies go straight into LDS;
 * otherwise through registers, more slowly. Sums are taken in an order that
 * the shape, the alignment, the groups, whether there is a workspace and the GPU's number of
 * compute units fix: equal calls give equal results. Every workgroup reads all offsets, so
 * thousands of groups take time by their square (of a row each, 64 x 64 weights: 1000 groups 39 us,
 * 5000 0.55 ms, 65536 86 ms).
 *
 * linear16_nt — Z = X * W^T + bias, Y = act(Z) + R.
 *   X       M-by-K of `type`, ldx >= max(1, K).
 *   bias    groups-by-N fp32, contiguous, or NULL.
 *   act     LL_ACT_*; ReLU maps z <= 0 (and NaN) to +0.0.
 *   R, Y    M-by-N of `ytype`, which is `type` or LL_TYPE_F32. R may be NULL
 *           (nothing is added), or Y itself (same ld).
 *   Z       M-by-N of `type`, or NULL: Z as the way back needs it, and / or
 *   ZQ, ZS  the same in MX8 (M-by-N codes, M-by-ceil(N/32) scales), from its
 *           FP32 sums; both or neither.
 *   workspace   NULL, or at least ll_linear16_workspace_size(LL_L16_FORWARD, M, N,
 *           K, groups) bytes (on the current device; 0: none helps), 16-byte
 *           aligned, overlapping nothing; its contents need no preparation. With
 *           one, a product that does not fill the GPU with tiles shares K out
 *           over workgroups, whose sums a second launch adds in order, another order than
 *           without one. Calls that share one must not overlap in time.
 * Outputs must not overlap inputs or each other otherwise. K == 0: Z = bias.
 *
 * linear16_grad_act — dZ = dY * act'(Z), and dbias[g] = the sums of dZ (before its
 * rounding) over the rows of group g.
 *   DY      M-by-N of `ytype` (`type` or LL_TYPE_F32).
 *   Z, or ZQ and ZS   as linear16_nt wrote them; not read, and may all be
 *           NULL, for LL_ACT_NONE.
 *   DZ      M-by-N of `type`, or NULL. It may be DY (of that type) or Z itself, same ld.
 *   dbias   groups-by-N fp32, contiguous, or NULL; an empty group's is 0. It
 *           needs a workspace of ll_linear16_grad_act_workspace_size(M, N,
 *           groups) bytes, 16-byte aligned, overlapping nothing; its contents
 *           need no preparation. Calls that share one must not overlap in time.
 *
 * linear16_grad_input — dX (M-by-K of `xtype`: `type` or LL_TYPE_F32) = dZ
 * (M-by-N of `type`) * W. workspace as linear16_nt's, LL_L16_GRAD_INPUT.
 *
 * linear16_grad_weight — dW = dZ^T * X + beta * dW, N-by-K of `wtype` (`type` or
 * LL_TYPE_F32), lddw >= max(1, K); group g's from its own rows, stride_dw * g elements
 * after the first. With beta == 0 dW is not read; an empty group's is beta * dW.
 *   X, or XQ and XS   M-by-K of `type`, or in MX8. Values in MX8 enter their
 *           products as `type` holds them: bfloat16 exactly down to its
 *           subnormals, binary16 rounded below 2^-14 and held at +-65504.
 */
#define LL_MAX_GROUPS (1 << 20)
int linear16_nt(int M, int N, int K, int type, const uint16_t *X, int ldx,
                int groups, const int32_t *offsets,
                const uint16_t *W, int ldw, int64_t stride_w, const float *bias, int act,
                int ytype, const void *R, int ldr, void *Y, int ldy,
                uint16_t *Z, int ldz, uint8_t *ZQ, int ldzq, uint8_t *ZS, int ldzs,
                void *workspace, int64_t workspace_bytes, void *stream);
/* product: LL_L16_FORWARD or LL_L16_GRAD_INPUT; -1 for another or a negative size. */
int64_t ll_linear16_workspace_size(int product, int M, int N, int K, int groups);
/* Name of the kernel that a product without a workspace (with one that shares K out:
 * "rows" and "rows_any", else "small" and "small_any") takes on a device with num_cus
 * compute units (num_cus <= 0: 256), with rows on 16 bytes (`aligned`) or not: "rows" and
 * "rows_any" (forward, at most 64 rows a group on average), "small" and
 * "small_any" (tiles of 128 x 128), "large" (256 x 256 and pieces of them); "" for one
 * without work or a bad argument. Static string. */
#define LL_L16_FORWARD 0
#define LL_L16_GRAD_INPUT 1
#define LL_L16_GRAD_WEIGHT 2
const char *ll_linear16_chosen_kernel(int product, int M, int N, int K, int groups, int aligned, int num_cus);
int64_t ll_linear16_grad_act_workspace_size(int M, int N, int groups);
int linear16_grad_act(int M, int N, int type, int act, int ytype, const void *DY, int lddy,
                      int groups, const int32_t *offsets,
                      const uint16_t *Z, int ldz, const uint8_t *ZQ, int ldzq, const uint8_t *ZS, int ldzs,
                      uint16_t *DZ, int lddz, float *dbias,
                      void *workspace, int64_t workspace_bytes, void *stream);
int linear16_grad_input(int M, int N, int K, int type, const uint16_t *DZ, int lddz,
                        int groups, const int32_t *offsets,
                        const uint16_t *W, int ldw, int64_t stride_w,
                        int xtype, void *DX, int lddx,
                        void *workspace, int64_t workspace_bytes, void *stream);
int linear16_grad_weight(int M, int N, int K, int type, const uint16_t *DZ, int lddz,
                         int groups, const int32_t *offsets,
                         const uint16_t *X, int ldx, const uint8_t *XQ, int ldxq, const uint8_t *XS, int ldxs,
                         int wtype, float beta, void *DW, int lddw, int64_t stride_dw,
                         void *stream);

/* A static, human-readable string for a status code (never NULL). */
const char *ll_status_string(int status);

/*
 * Tile and K-split selection. Each data type has a small set of block-tile
 * shapes; by default the library picks, per call, a tile shape and a number
 * of K-splits from M, N, K and the CU count, minimising an estimate of the
 * run time: large problems get the largest tiles, and problems too small to
 * fill the device get smaller tiles or several workgroups along K (the
 * size-dependent strategy of page "GEMM 优化详解", section "矩阵大小选择策略"
 * (matrix-size strategy), re-derived for 256 CUs).
 *
 * With K-splits (split-K), each split computes alpha * A[:, Ks] * B[Ks, :]
 * for its range Ks of K and adds it into C with hardware FP32 atomics, after
 * a pass that scales C by beta (for linear_bias_act: fills Y with the bias,
 * then applies the ReLU in a pass afterwards). The result is the same sum in
 * a different, run-dependent order; it still allocates nothing.
 *
 * Some shapes split K inside the workgroup instead ("K-sliced" tiles, named
 * *_k4 and *_k2: f32_64x64_k4, f32_128x128_k2, f16_128x128_k2): the
 * workgroup's slices sum disjoint stage-aligned K ranges and add their
 * partial tiles through on-chip memory in a fixed order, so the result does
 * not depend on the run; no atomics, no extra pass. They serve problems too
 * small to fill the device (e.g. 1024^3), and the automatic choice takes them
 * only when each slice gets at least 8 stages (a forced tile is always used).
 *
 * FP32 products of at most 32 rows of A may take f32_32x128: two-wave
 * workgroups of 32x128, up to four per CU, for the rows that the 64-row
 * tiles would mostly pad.
 *
 * Single FP32 products with a few rows of A (at most 4, or at most 8 when B
 * holds at least 2^25 values) are bound by reading B from HBM, not by the
 * matrix units (page "GEMM 优化详解", table "计算复杂度分析": the intensity
 * 2MNK / (MK + KN + MN) / 4 is about M/2 FLOP per byte). They take the tile
 * f32_16x256_skinny: vector FMAs over 256 columns of C per workgroup with
 * A's rows staged in LDS, and up to 64 K-splits (added atomically, framed by
 * the same passes as above). Forced on more rows it walks them 16 at a time.
 * Single 16-bit products of one row of A with B given N-by-K and holding at
 * least 2^25 values likewise take f16_16x256_skinny_nt: dot2 instructions
 * (two 16-bit products added into an FP32 sum) over 256 columns of C per
 * workgroup, the same K-splits; forced with B given K-by-N, the 128x128 tile
 * runs in its place.
 *
 * The calls below report the choice; they touch only host memory and never
 * the GPU. (linear_layer_tuning.h declares process-wide overrides of the
 * choice for benchmarks and tests.)
 */
#define LL_DTYPE_F32 0 /* gemm_f32, linear_bias_act and their _nt forms */
#define LL_DTYPE_F16 1 /* gemm_f16f32, gemm_bf16f32 and their _nt forms */
/* Flags the ll_chosen_* queries accept OR-ed into `dtype`:
 * LL_PLAN_RELU: linear_bias_act with the ReLU, whose K-split and stream-K
 * plans pay for one more pass over Y (LL_DTYPE_F32 only);
 * LL_PLAN_B_NK: the _nt form (B given N-by-K; the FP32 skinny kernel's
 * K-split count and the 16-bit skinny kernel's choice depend on it);
 * LL_PLAN_UNALIGNED: operands that do not allow the 128-bit-load kernels
 * (a base not 16-byte aligned, or a leading dimension, K or N not a multiple
 * of 4 (fp32) or 8 (16-bit)): no stream-K, and the tiles that exist only as
 * 128-bit-load kernels (the K-sliced ones, f32_32x128 and f16_192x192_direct)
 * are not chosen automatically. */
#define LL_PLAN_RELU 0x100
#define LL_PLAN_B_NK 0x200
#define LL_PLAN_UNALIGNED 0x400

/* Number of tile shapes for a data type (0 for an unknown dtype). */
int ll_num_tiles(int dtype);
/* Name of a tile shape, e.g. "f32_256x256" ("" if out of range). Static string. */
const char *ll_tile_name(int dtype, int tile);
/* The tile / the number of K-splits the library would use for `batch`
 * M-by-N outputs (batch 1: a single product) with inner dimension K on a
 * device with num_cus compute units (num_cus <= 0: 256), honouring the
 * overrides and the LL_PLAN_* flags in dtype. -1 for an unknown dtype or
 * flag, or batch < 1. */
int ll_chosen_tile(int dtype, int M, int N, int K, int batch, int num_cus);
int ll_chosen_split_k(int dtype, int M, int N, int K, int batch, int num_cus);

/*
 * Stream-K (single products with 128-bit-aligned operands; FP32 on tiles
 * without K-slices, 16-bit on the 256x256 tile):
 * when the output tiles do not fill a whole number of rounds of the CUs, the
 * planner may run the full rounds tile by tile and share the leftover tiles'
 * K range out evenly over one round of workgroups, whose partial sums are
 * added atomically into C (prepared with beta*C, or the bias, beforehand;
 * the ReLU applied afterwards). Like a K-split, this makes the summation
 * order of those tiles run-dependent (still within the error bound; integer
 * inputs stay exact); it allocates nothing.
 *   ll_chosen_stream_k: the number of tiles the plan shares out (0: none);
 *   dtype and flags as for ll_chosen_tile; -1 for an unknown dtype or flag,
 *   or batch < 1.
 */
int ll_chosen_stream_k(int dtype, int M, int N, int K, int batch, int num_cus);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_LAYER_H */
