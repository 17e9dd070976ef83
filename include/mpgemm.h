/*
 * mpgemm.h -- mixed-precision dense matrix multiply-accumulate on AMD Instinct MI355X (gfx950).
 *
 *     D = alpha * op(A) * op(B) + beta * C
 *
 * with FP16 or BF16 inputs accumulated in FP32, or INT8 inputs accumulated in INT32.
 *
 * The call follows the GEMM statement of "Programming Tensor Cores in CUDA 9"
 * (makelele.cn/d/1827294.html), section on using Tensor Cores through cuBLAS: a handle,
 * transpose flags, m, n, k, alpha, the A, B and C matrices each with an element type and a
 * leading dimension, beta, and a compute (accumulate) type; and its section "Finishing":
 * the product is scaled by alpha and added to C scaled by beta.  The type matrix follows
 * "Mixed-Precision Programming with CUDA 8" (m.ruidan.com/infomation/detail/138780),
 * section on cuBLAS: FP32 compute on FP16 inputs with FP32 or FP16 output, and INT8 inputs
 * with integer (DP4A-style) compute.
 *
 * STORAGE IS ROW-MAJOR.  op(A) is m x k, op(B) is k x n, C and D are m x n.
 *   transa == MPGEMM_OP_N: A is stored m x k, element (i,p) at A[i*lda + p], lda >= k.
 *   transa == MPGEMM_OP_T: A is stored k x m (the buffer holds op(A)^T), element (i,p) at
 *                          A[p*lda + i], lda >= m.
 *   transb == MPGEMM_OP_N: B is stored k x n, element (p,j) at B[p*ldb + j], ldb >= n.
 *   transb == MPGEMM_OP_T: B is stored n x k ("B column-major"), element (p,j) at
 *                          B[j*ldb + p], ldb >= k.
 *   C and D: element (i,j) at [i*ldc + j], ldc >= n.  D has C's type and leading dimension.
 * A column-major caller computes D^T = op(B)^T op(A)^T: it passes (transb, transa, n, m, k,
 * B, ldb, A, lda, C, ldc), which the row-major reading turns back into its own problem.
 *
 * Supported type combinations (anything else returns MPGEMM_STATUS_NOT_SUPPORTED):
 *   a_type = b_type = MPGEMM_R_16F,  compute MPGEMM_R_32F, c_type MPGEMM_R_32F or MPGEMM_R_16F
 *   a_type = b_type = MPGEMM_R_16BF, compute MPGEMM_R_32F, c_type MPGEMM_R_32F or MPGEMM_R_16BF
 *   a_type = b_type = MPGEMM_R_8I,   compute MPGEMM_R_32I, c_type MPGEMM_R_32I
 *   a_type, b_type each MPGEMM_R_8F_E4M3 or MPGEMM_R_8F_E5M2 (either pairing; the two FP8
 *     formats of "NVIDIA Tensor Core mixed-precision computing: principles and applications",
 *     section 4.3.1), compute MPGEMM_R_32F, c_type MPGEMM_R_32F or MPGEMM_R_16BF; here
 *     "compute MPGEMM_R_32F" means an FP32 accumulator between 128-deep instructions only:
 *     the sums inside each instruction keep about 13 bits (see below), so FP8 results are
 *     not FP32-accurate sums of the products
 * FP16/BF16 outputs are rounded once from the FP32 result, to nearest with ties to even.
 * INT32 accumulation and the epilogue wrap modulo 2^32.
 *
 * FP32 result (the rounding steps, which the pages leave to the hardware): the products are
 * accumulated in k order by the matrix cores' block FMA, 8 consecutive k per block ("NVIDIA
 * Tensor Core mixed-precision computing: principles and applications", sections 2.2-2.3
 * and 4.2.1, with gfx950's parameters: products aligned to the block's largest exponent
 * with 24 fraction bits, products cut toward zero and the running sum toward minus infinity
 * below that, the block sum kept to 32 significant bits, then rounded to FP32 to nearest
 * even), starting from zero; the epilogue is alpha * acc when beta == 0, else
 * fma(alpha, acc, beta * c) in FP32.  The result is deterministic: the same inputs give the
 * same bits on every call, tile shape and launch.
 * FP8 inputs accumulate on gfx950's v_mfma_f32_16x16x128_f8f6f4, whose intermediate sums are
 * narrower (measured: groups of 8 products keep about 13 fraction bits below the group's
 * largest exponent, blocks of 16 products in k order are added to the FP32 accumulator in a
 * 24-bit window and the sum rounded to FP32 after each block); results whose partial sums stay
 * on that grid (small integers, for instance) are exact, others carry an error up to about
 * 2^-9 of sum |a b|.
 *
 * Alignment contract (there is no slower fallback path): A, B, C (when read) and D must be
 * 16-byte aligned, and lda, ldb, ldc times the element size must be multiples of 16 bytes
 * (8 elements for FP16/BF16, 16 for INT8 and FP8, 4 for FP32/INT32).  m, n and k are
 * arbitrary up to 2^31 - 1 (k up to 2^31 - 256); larger sizes return
 * MPGEMM_STATUS_NOT_SUPPORTED.
 * Operands are read in whole aligned 16-byte blocks: each row of A and B must be readable up
 * to the end of the 16-byte block holding its last element (true of any buffer whose size is
 * rows * ld elements).  Elements beyond the logical row are never used in the result.
 * The distance in bytes spanned by 256 rows of any operand (256 * ld * element size) must be
 * below 2^31; larger strides return MPGEMM_STATUS_NOT_SUPPORTED.
 *
 * Ownership and ordering: the caller allocates and owns every matrix and keeps it alive and
 * unmodified until the work queued on `stream` has finished.  mpgemm_run allocates no device
 * memory, is asynchronous, and is ordered on `stream` (a hipStream_t; NULL means the null
 * stream).  A handle is bound to the device that was current at mpgemm_create and holds only
 * host state; use one handle per host thread (a handle is not thread-safe).
 *
 * Errors are returned as status codes; nothing aborts and no exception crosses this ABI.
 * Arguments are checked on the host before any device call.  Faults that happen while the
 * queued kernel runs surface at the caller's next synchronisation of `stream`.
 */
#ifndef MPGEMM_H
#define MPGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mpgemm_handle_s *mpgemm_handle_t;

typedef enum { MPGEMM_OP_N = 0, MPGEMM_OP_T = 1 } mpgemm_op_t;

typedef enum {
    MPGEMM_R_16F = 0,   /* IEEE binary16: 1 sign, 5 exponent, 10 fraction bits */
    MPGEMM_R_16BF = 1,  /* bfloat16: upper 16 bits of an IEEE binary32 */
    MPGEMM_R_8I = 2,    /* signed 8-bit integer */
    MPGEMM_R_32F = 3,   /* IEEE binary32 */
    MPGEMM_R_32I = 4,   /* signed 32-bit integer (two's complement) */
    MPGEMM_R_8F_E4M3 = 5, /* FP8 E4M3 (OCP): 1 sign, 4 exponent (bias 7), 3 fraction bits;
                             no infinities, S.1111.111 is NaN; largest 448, smallest 2^-9 */
    MPGEMM_R_8F_E5M2 = 6  /* FP8 E5M2 (OCP): 1 sign, 5 exponent (bias 15), 2 fraction bits;
                             IEEE-style infinities and NaNs; largest 57344, smallest 2^-16 */
} mpgemm_dtype_t;

typedef enum {
    MPGEMM_STATUS_SUCCESS = 0,
    MPGEMM_STATUS_NOT_INITIALIZED = 1, /* handle not created, or already destroyed */
    MPGEMM_STATUS_INVALID_VALUE = 2,   /* null pointer, negative size, ld below its minimum */
    MPGEMM_STATUS_NOT_SUPPORTED = 3,   /* type combination, alignment or stride outside the contract */
    MPGEMM_STATUS_ALLOC_FAILED = 4,    /* host allocation of the handle failed */
    MPGEMM_STATUS_NO_DEVICE = 5,       /* no HIP device, or the current device is not gfx950 */
    MPGEMM_STATUS_LAUNCH_FAILED = 6,   /* the kernel launch was rejected by the runtime */
    MPGEMM_STATUS_INTERNAL_ERROR = 7,
    MPGEMM_STATUS_WRONG_DEVICE = 8,    /* current device differs from the handle's device */
    MPGEMM_STATUS_SCRATCH_TOO_SMALL = 9 /* mpgemm_run_bf16x3_noalloc: the split operands need
                                           more than MPGEMM_NOALLOC_SCRATCH_BYTES */
} mpgemm_status_t;

/* Size of the library's fixed scratch buffer (per device) used by mpgemm_run_bf16x3_noalloc. */
#define MPGEMM_NOALLOC_SCRATCH_BYTES (64ull << 20)

/* Create a handle bound to the current HIP device.  Returns MPGEMM_STATUS_NO_DEVICE when no
 * device is present or the device is not a gfx950, MPGEMM_STATUS_INVALID_VALUE when
 * `handle` is NULL, MPGEMM_STATUS_ALLOC_FAILED when host memory runs out.  On failure
 * *handle is set to NULL (when handle is non-NULL). */
mpgemm_status_t mpgemm_create(mpgemm_handle_t *handle);

/* Queue D = alpha * op(A) * op(B) + beta * C on `stream` (see the contract above).
 *   alpha, beta: host pointers to a float (compute MPGEMM_R_32F) or an int32_t
 *                (compute MPGEMM_R_32I), read before the call returns.
 *   C:           read only when *beta != 0; may be NULL otherwise.  D == C (in place) is
 *                allowed; any other overlap of D with A, B or C is undefined.
 *   m == 0 or n == 0 returns MPGEMM_STATUS_SUCCESS without touching the device.
 *   k == 0 gives D = beta * C (D = 0 when beta == 0); A and B may then be NULL.
 *   alpha == 0 is not special-cased: NaN or Inf in A or B still reaches D.
 * The current HIP device must be the handle's (else MPGEMM_STATUS_WRONG_DEVICE). */
mpgemm_status_t mpgemm_run(mpgemm_handle_t handle, mpgemm_op_t transa, mpgemm_op_t transb,
                           int64_t m, int64_t n, int64_t k, const void *alpha,
                           const void *A, mpgemm_dtype_t a_type, int64_t lda,
                           const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                           const void *beta, const void *C, mpgemm_dtype_t c_type, int64_t ldc,
                           void *D, mpgemm_dtype_t compute_type, void *stream);

/* FP32 GEMM from BF16 pieces (multiword emulation: "NVIDIA Tensor Core mixed-precision
 * computing: principles and applications", section 5.1, splits high-precision operands into
 * pieces the matrix cores take and sums the partial products; "The CUDA Handbook" section
 * 17.5 does FP32 GEMM on Tensor Cores by rounding inputs to TF32).  Queues on `stream`
 *
 *   D = alpha * op(A) * op(B) + beta * C        A, B, C, D, alpha, beta: FP32
 *
 * with every element x of A and B split into x_hi = RN_bf16(x) and x_lo = RN_bf16(x - x_hi)
 * (round to nearest even; x - x_hi is exact in FP32; x_lo = 0 when x_hi is Inf or NaN, so
 * Inf and NaN propagate as in an FP32 product, and finite x beyond BF16's largest value,
 * about 3.39e38, counts as infinite), and op(A) op(B) replaced by
 *
 *   A_hi B_hi + A_lo B_hi + A_hi B_lo
 *
 * computed as ONE BF16 GEMM of the kind mpgemm_run performs (FP32 accumulation, same
 * numerics and epilogue) over k3 = 3 kp, kp = k rounded up to a multiple of 8: the k index
 * runs through the three products in that order, each zero-padded from k to kp.  Per
 * element the representation error is at most about 3 * 2^-16 |a b| (A_lo B_lo and the
 * residuals are dropped), against 2^-11 for inputs rounded to TF32.
 *
 *   workspace:       device memory for the split operands, at least
 *                    mpgemm_bf16x3_workspace_size(transa, transb, m, n, k) bytes, 256-byte
 *                    aligned, not overlapping A, B, C or D; overwritten, owned by the caller,
 *                    and in use until the queued work finishes.  Layout (BF16, row-major):
 *                    A3 at offset 0: m x k3 (ld k3) for transa == N, k3 x m (ld m rounded up
 *                    to 8) for transa == T; B3 at the next 256-byte boundary: k3 x n (ld n
 *                    rounded up to 8) for transb == N, n x k3 (ld k3) for transb == T.
 *   Alignment:       A, B, C (when read), D 16-byte aligned; lda, ldb, ldc multiples of 4.
 *   Other arguments, ownership and errors as for mpgemm_run; a workspace that is NULL (with
 *   a nonzero requirement) or smaller than required returns MPGEMM_STATUS_INVALID_VALUE, a
 *   misaligned one MPGEMM_STATUS_NOT_SUPPORTED.  mpgemm_run_bf16x3 allocates nothing. */
mpgemm_status_t mpgemm_run_bf16x3(mpgemm_handle_t handle, mpgemm_op_t transa,
                                  mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                  const float *alpha, const float *A, int64_t lda,
                                  const float *B, int64_t ldb, const float *beta,
                                  const float *C, int64_t ldc, float *D, void *workspace,
                                  uint64_t workspace_bytes, void *stream);

/* mpgemm_run_bf16x3 without a workspace argument, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation and results, with the split operands kept in a fixed device array of
 * the library (MPGEMM_NOALLOC_SCRATCH_BYTES = 64 MiB per device, reserved when the library's
 * code is first loaded on a device and held until the process ends) instead of a
 * caller-provided workspace.  The call allocates nothing and frees nothing.
 *   - Problems whose workspace, mpgemm_bf16x3_workspace_size(transa, transb, m, n, k),
 *     exceeds MPGEMM_NOALLOC_SCRATCH_BYTES return MPGEMM_STATUS_SCRATCH_TOO_SMALL without
 *     launching anything (for example m x k + k x n up to about 11 million elements fits).
 *   - All calls on one device share that device's buffer, which keeps the last call's
 *     contents: calls that may overlap on one device (different streams, handles or host
 *     threads without ordering between them) race and give wrong results; calls ordered on
 *     one stream are safe.  No byte of it needs to start at zero: each call writes every
 *     byte its GEMM reads.
 *   - Other arguments, ownership and errors as for mpgemm_run_bf16x3; the handle must have
 *     been created on the current device (its creation looks the buffer's address up;
 *     MPGEMM_STATUS_INTERNAL_ERROR if that failed). */
mpgemm_status_t mpgemm_run_bf16x3_noalloc(mpgemm_handle_t handle, mpgemm_op_t transa,
                                          mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                          const float *alpha, const float *A, int64_t lda,
                                          const float *B, int64_t ldb, const float *beta,
                                          const float *C, int64_t ldc, float *D, void *stream);

/* Host-only argument check of mpgemm_run_bf16x3: returns exactly the status mpgemm_run_bf16x3
 * would return for these arguments before touching the device (the workspace's size and
 * alignment included); needs no handle and no device, and dereferences only alpha and beta. */
mpgemm_status_t mpgemm_check_bf16x3(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m,
                                    int64_t n, int64_t k, const float *alpha, const float *A,
                                    int64_t lda, const float *B, int64_t ldb, const float *beta,
                                    const float *C, int64_t ldc, const float *D,
                                    const void *workspace, uint64_t workspace_bytes);

/* GEMM with a 2:4 structured-sparse A (the page "稀疏张量核心加速模板计算的技术解析" on sparse tensor
 * cores for stencils, sections
 * 1.2.1 and 1.3.2: at most two nonzeros in every group of 4 consecutive k, stored as the kept
 * values plus 2 bits of metadata per kept value; here on gfx950's v_smfmac sparse matrix
 * cores).  Queues on `stream`
 *
 *   D = alpha * A * op(B) + beta * C,   A(i, 4q + idx(i, j)) += Ac(i, j) for j = 2q, 2q + 1
 *
 * i.e. D(i, c) = alpha * sum_j Ac(i, j) * op(B)(4 (j / 2) + idx(i, j), c) + beta * C(i, c).
 *   Ac:     the kept values, m x k/2, row-major: Ac(i, j) at Ac[i*lda + j], lda >= k/2.
 *   meta:   m rows of ld_meta bytes, ld_meta >= k/8: idx(i, j) is bits 2 (j % 4) .. +1 of byte
 *           meta[i*ld_meta + j/4] (2 bits per kept value, in k order, little-endian).  The two
 *           indices of a group are normally distinct; equal ones make both values multiply
 *           the same row of op(B).
 *   B, C, D, transb, ldb, ldc, alpha, beta: as for mpgemm_run; A is never transposed.
 *   Types:  a_type = b_type = MPGEMM_R_16F or MPGEMM_R_16BF, compute MPGEMM_R_32F, c_type
 *           MPGEMM_R_32F or a_type: numerics as for the dense FP16/BF16 GEMM, over the k/2
 *           kept products (blocks of 8 kept products, in kept order); or a_type = b_type =
 *           MPGEMM_R_8I with compute and c_type MPGEMM_R_32I: exact, wrapping INT32 arithmetic
 *           as for the dense INT8 GEMM (alpha and beta point to int32_t); or a_type and b_type
 *           each MPGEMM_R_8F_E4M3 or MPGEMM_R_8F_E5M2, compute MPGEMM_R_32F, c_type
 *           MPGEMM_R_32F or MPGEMM_R_16BF: numerics as for the dense FP8 GEMM.
 *   Sizes:  k a multiple of 128 (else MPGEMM_STATUS_NOT_SUPPORTED); m, n arbitrary.
 *   Alignment: Ac, meta, B, C (when read), D 16-byte aligned; rows of Ac and B (lda, ldb
 *           elements) and of the metadata (ld_meta bytes) multiples of 16 bytes, ldc as for
 *           mpgemm_run.
 * Ownership, ordering and errors as for mpgemm_run; nothing is allocated. */
mpgemm_status_t mpgemm_run_sp24(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t m, int64_t n,
                                int64_t k, const void *alpha, const void *Ac,
                                mpgemm_dtype_t a_type, int64_t lda, const void *meta,
                                int64_t ld_meta, const void *B, mpgemm_dtype_t b_type,
                                int64_t ldb, const void *beta, const void *C,
                                mpgemm_dtype_t c_type, int64_t ldc, void *D,
                                mpgemm_dtype_t compute_type, void *stream);

/* Host-only argument check of mpgemm_run_sp24 (as mpgemm_check is for mpgemm_run). */
mpgemm_status_t mpgemm_check_sp24(mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                  const void *alpha, const void *Ac, mpgemm_dtype_t a_type,
                                  int64_t lda, const void *meta, int64_t ld_meta, const void *B,
                                  mpgemm_dtype_t b_type, int64_t ldb, const void *beta,
                                  const void *C, mpgemm_dtype_t c_type, int64_t ldc,
                                  const void *D, mpgemm_dtype_t compute_type);

/* Workspace bytes mpgemm_run_bf16x3 needs for these sizes (0 when m, n or k is 0); 0 also
 * for negative sizes or flags outside MPGEMM_OP_N / MPGEMM_OP_T.  Host-only. */
uint64_t mpgemm_bf16x3_workspace_size(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m,
                                      int64_t n, int64_t k);

/* Host-only argument check: returns exactly the status mpgemm_run would return for these
 * arguments before touching the device (MPGEMM_STATUS_SUCCESS if it would launch).  It needs
 * no handle and no device, and dereferences only alpha and beta. */
mpgemm_status_t mpgemm_check(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m, int64_t n,
                             int64_t k, const void *alpha, const void *A, mpgemm_dtype_t a_type,
                             int64_t lda, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                             const void *beta, const void *C, mpgemm_dtype_t c_type, int64_t ldc,
                             const void *D, mpgemm_dtype_t compute_type);

/* Release a handle.  NULL or an unknown/destroyed handle returns
 * MPGEMM_STATUS_NOT_INITIALIZED.  Work already queued is not affected. */
mpgemm_status_t mpgemm_destroy(mpgemm_handle_t handle);

/* Static, NUL-terminated description of a status code (never NULL). */
const char *mpgemm_status_string(mpgemm_status_t status);

/* Tile shape (rows x columns of D per workgroup) that mpgemm_run picks for an m x n output
 * with inputs of type a_type on a device with 256 compute units (a whole MI355X; mpgemm_run
 * uses the handle's device's count), written to *tile_m and *tile_n.  Host-only; for
 * diagnostics and benchmarks.  Returns MPGEMM_STATUS_INVALID_VALUE for negative sizes or null
 * outputs. */
mpgemm_status_t mpgemm_tile_shape(int64_t m, int64_t n, mpgemm_dtype_t a_type, int *tile_m,
                                  int *tile_n);

/* ---------------------------------------------------------------------------------------
 * Products of language models: a product with its bias, activation and residual, the same for
 * rows divided among experts, and the cross entropy of a linear layer; each with its gradients.
 *
 * Types: the inputs of a product are both MPGEMM_R_16F or both MPGEMM_R_16BF, the output (and a C
 * that is read) that type or MPGEMM_R_32F, scalars are FP32.  Products are accumulated as
 * mpgemm_run's; everything after them is computed in FP32 and rounded once, to nearest even,
 * where it is stored.  Storage, alignment (16-byte pointers, row strides that are multiples of
 * 16 bytes and below the same limit), ownership, ordering and errors are mpgemm_run's; C, aux
 * and Z are, like A and B, read in whole aligned 16-byte blocks.  Sizes go up to 2^31 - 256.
 * The results of a call do not depend on other calls and are the same each time.
 * A workspace is device memory of the size that the named function gives, 256-byte aligned, owned
 * by the caller, overwritten, and in use until the queued work finishes: NULL or too small
 * returns MPGEMM_STATUS_INVALID_VALUE, misaligned MPGEMM_STATUS_NOT_SUPPORTED.  Nothing is
 * allocated and no call waits for the device, so all of them can be captured into a graph.
 * --------------------------------------------------------------------------------------- */
typedef enum {
    MPGEMM_ACT_NONE = 0,
    MPGEMM_ACT_RELU = 1,      /* max(z, 0); slope 0 at 0 */
    MPGEMM_ACT_GELU = 2,      /* z Phi(z) */
    MPGEMM_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
    MPGEMM_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} mpgemm_act_t;

typedef struct {
    int act;                  /* an mpgemm_act_t */
    const void *bias;         /* n values, added to every row; NULL: none */
    int bias_type;            /* an mpgemm_dtype_t: the inputs' type or MPGEMM_R_32F */
    int64_t bias_stride;      /* grouped products: elements between two experts' biases (0: one
                                 bias for all); otherwise ignored */
    void *aux;                /* receives Z (m x n, the inputs' type); NULL: not kept */
    int64_t ld_aux;           /* elements, >= n */
} mpgemm_epilogue_t;

/* Queue  Z = alpha * op(A) * op(B) + bias,  D = act(Z) + beta * C.
 *   C is read only when *beta != 0 and may have another type and leading dimension than D; D == C
 *   is allowed when they are alike in both.  Z, when kept, must not overlap any other argument.
 *   The activation is taken from Z before its rounding.  k == 0 gives Z = bias. */
mpgemm_status_t mpgemm_run_epilogue(mpgemm_handle_t handle, mpgemm_op_t transa, mpgemm_op_t transb,
                                    int64_t m, int64_t n, int64_t k, const float *alpha,
                                    const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                    const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                    const mpgemm_epilogue_t *epilogue, const float *beta,
                                    const void *C, mpgemm_dtype_t c_type, int64_t ldc, void *D,
                                    mpgemm_dtype_t d_type, int64_t ldd, void *stream);

/* Queue the gradient that comes through an activation:
 *   D(i, j) = alpha * (op(A) op(B))(i, j) * act'(Z(i, j)),   dbias(j) = sum over i of D(i, j)
 * with Z as mpgemm_run_epilogue kept it (the inputs' type; not read for MPGEMM_ACT_NONE), and dbias
 * n FP32 values, summed in FP32 before D's rounding in a fixed order; NULL: not computed, and
 * no workspace is needed.  m == 0 gives dbias = 0.
 *   workspace: mpgemm_epilogue_grad_workspace_size(1, m, n) bytes. */
mpgemm_status_t mpgemm_run_epilogue_grad(mpgemm_handle_t handle, mpgemm_op_t transa,
                                         mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                         const float *alpha, const void *A, mpgemm_dtype_t a_type,
                                         int64_t lda, const void *B, mpgemm_dtype_t b_type,
                                         int64_t ldb, mpgemm_act_t act, const void *Z, int64_t ldz,
                                         void *D, mpgemm_dtype_t d_type, int64_t ldd, float *dbias,
                                         void *workspace, uint64_t workspace_bytes, void *stream);

/* Queue one product for each expert's rows: row r of expert e, offsets[e] <= r < offsets[e + 1],
 *   Z(r, :) = alpha * A(r, :) * op(B_e) + bias_e,   D(r, :) = act(Z(r, :)).
 *   A: rows x k (ld lda), D: rows x n, Z (epilogue->aux): rows x n.
 *   B_e: k x n (transb == N) or n x k (transb == T) at B + e * stride_b elements; stride_b is a
 *        multiple of 8, and 0 gives all experts the same one.
 *   offsets: groups + 1 non-decreasing device integers from 0 to rows; an expert may have no
 *        rows, and rows of no expert keep what D and Z held.  They are read by the queued kernels,
 *        never by the host; values outside the contract are clamped, so that no memory outside
 *        the operands is touched, but the results are then unspecified.
 *   groups goes up to 65535. */
mpgemm_status_t mpgemm_run_grouped(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t groups,
                                   int64_t rows, int64_t n, int64_t k, const float *alpha,
                                   const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                   const int32_t *offsets, const void *B, mpgemm_dtype_t b_type,
                                   int64_t ldb, int64_t stride_b, const mpgemm_epilogue_t *epilogue,
                                   void *D, mpgemm_dtype_t d_type, int64_t ldd, void *stream);

/* mpgemm_run_epilogue_grad for experts' rows: D(r, :) = alpha * A(r, :) op(B_e) * act'(Z(r, :)),
 * dbias(e, :) = sum of expert e's rows of D (groups x n FP32 values, 0 for an expert without rows).
 *   workspace: mpgemm_epilogue_grad_workspace_size(groups, rows, n) bytes (none without dbias). */
mpgemm_status_t mpgemm_run_grouped_grad(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t groups,
                                        int64_t rows, int64_t n, int64_t k, const float *alpha,
                                        const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                        const int32_t *offsets, const void *B,
                                        mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                        mpgemm_act_t act, const void *Z, int64_t ldz, void *D,
                                        mpgemm_dtype_t d_type, int64_t ldd, float *dbias,
                                        void *workspace, uint64_t workspace_bytes, void *stream);

/* Queue the gradients of the experts' weights: for each expert
 *   D_e = alpha * A_e^T X_e + beta * D_e          (m x n at D + e * stride_d elements)
 * where A_e (rows x m as a whole, ld lda) and X_e (rows x n, ld ldx) are expert e's rows.  An
 * expert without rows gets beta * D_e.  D is read only when *beta != 0.  The experts' D must not
 * overlap: stride_d >= (m - 1) * ldd + n, a multiple of 16 bytes. */
mpgemm_status_t mpgemm_run_grouped_wgrad(mpgemm_handle_t handle, int64_t groups, int64_t rows,
                                         int64_t m, int64_t n, const float *alpha, const void *A,
                                         mpgemm_dtype_t a_type, int64_t lda, const void *X,
                                         mpgemm_dtype_t x_type, int64_t ldx, const int32_t *offsets,
                                         const float *beta, void *D, mpgemm_dtype_t d_type,
                                         int64_t ldd, int64_t stride_d, void *stream);

/* Queue the softmax cross entropy of a linear layer, without storing its logits:
 *   z(i, v) = alpha * X(i, :) . W(v, :),   lse(i) = log(sum over v of exp(z(i, v))),
 *   loss(i) = lse(i) - z(i, target(i)),  0 where the target does not count.
 *   X: m x k, W: n x k (type MPGEMM_R_16F or MPGEMM_R_16BF both), n >= 1.
 *   target: m device integers; one outside 0 .. n - 1 (-1 or -100, as a rule) does not count.
 *   loss, lse: m FP32 values each (lse of every row).
 *   workspace: mpgemm_linear_ce_workspace_size(m, n, k, type, 0) bytes. */
mpgemm_status_t mpgemm_run_linear_ce(mpgemm_handle_t handle, int64_t m, int64_t n, int64_t k,
                                     const float *alpha, const void *X, mpgemm_dtype_t type,
                                     int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                                     float *loss, float *lse, void *workspace,
                                     uint64_t workspace_bytes, void *stream);

/* Queue its gradients: with P(i, v) = (exp(z(i, v) - lse(i)) - [v == target(i)]) * grad(i), and 0 in
 * rows whose target does not count,
 *   dX = alpha * P W,   dW = alpha * P^T X      (type's; either may be NULL and is then skipped).
 *   lse: as mpgemm_run_linear_ce wrote it.  grad: m FP32 values, the gradient of each row's loss.
 *   Rows whose target does not count add nothing to dW, whatever X and grad hold there, and their
 *   dX is 0; above 128 rows they are left out of the products.
 *   P is computed in pieces of the vocabulary and rounded to the inputs' type for the products,
 *   after division by the largest |grad(i)| (FP16: and scaling by 2^13, so that small
 *   probabilities stay normal; the scale is one for the call, and an entry of P below 2^-27 of
 *   the largest |grad(i)| has fewer bits, so that rows far below the largest lose some of theirs).
 *   workspace: mpgemm_linear_ce_workspace_size(m, n, k, type, 1) bytes, which is also enough for
 *   mpgemm_run_linear_ce. */
mpgemm_status_t mpgemm_run_linear_ce_grad(mpgemm_handle_t handle, int64_t m, int64_t n, int64_t k,
                                          const float *alpha, const void *X, mpgemm_dtype_t type,
                                          int64_t ldx, const void *W, int64_t ldw,
                                          const int64_t *target, const float *lse,
                                          const float *grad, void *dX, int64_t lddx, void *dW,
                                          int64_t lddw, void *workspace, uint64_t workspace_bytes,
                                          void *stream);

/* Workspace bytes of the gradients above for dbias (groups == 1 for mpgemm_run_epilogue_grad), and
 * of the cross entropy (train != 0: of its gradients too).  0 for sizes or types outside the
 * contract and where no workspace is needed.  Host-only. */
uint64_t mpgemm_epilogue_grad_workspace_size(int64_t groups, int64_t m, int64_t n);
uint64_t mpgemm_linear_ce_workspace_size(int64_t m, int64_t n, int64_t k, mpgemm_dtype_t type,
                                         int train);

/* ---------------------------------------------------------------------------------------
 * Distillation: the loss of a linear layer's softmax against a teacher's top logits, and its
 * gradients, without storing the logits.  Types, storage and everything else are as for
 * mpgemm_run_linear_ce.
 * --------------------------------------------------------------------------------------- */
typedef struct {
    int64_t top;              /* entries of each row, 1 .. 1024 */
    const int64_t *index;     /* m x top (ld) device integers: the entries' columns; one outside
                                 0 .. n - 1 (-1, as a rule) does not count */
    const float *logit;       /* m x top (ld): the teacher's logits there */
    int64_t ld;               /* >= top; picked's too */
    float scale;              /* of the teacher's logits, -1e30 .. 1e30: 1 / its temperature, as a rule;
                                 0 gives all entries the same share */
    const float *lse;         /* m log-sum-exps of the teacher's scaled logits over all columns; NULL:
                                 over the entries that count */
} mpgemm_teacher_t;

/* Queue, with z(i, v) = alpha * X(i, :) . W(v, :) and over the entries j of row i that count,
 *   q(i, j) = exp(scale * logit(i, j) - teacher's lse(i)),     lse(i) = log(sum over v of exp(z(i, v))),
 *   loss(i) = sum over j of q(i, j) * (log q(i, j) - z(i, index(i, j)) + lse(i)).
 * A temperature of the student is part of alpha.  Without the teacher's lse the q of a row sum to 1
 * and the loss is the divergence of the student from the teacher's top entries; with it, the part of
 * that divergence that lies in them.  Entries of the same column add up as they stand.  A logit of
 * -infinity has no mass, whatever the scale; a row none of whose entries has any does not count and has loss 0.
 *   loss, lse: m FP32 values each.  picked: m x top (teacher->ld) FP32 values, z at the entries'
 *   columns (0 where an entry does not count), which the gradient takes.
 *   workspace: mpgemm_linear_distill_workspace_size(m, n, k, top, type, 0) bytes. */
mpgemm_status_t mpgemm_run_linear_distill(mpgemm_handle_t handle, int64_t m, int64_t n, int64_t k,
                                          const float *alpha, const void *X, mpgemm_dtype_t type,
                                          int64_t ldx, const void *W, int64_t ldw,
                                          const mpgemm_teacher_t *teacher, float *loss, float *lse,
                                          float *picked, void *workspace, uint64_t workspace_bytes,
                                          void *stream);

/* Queue its gradients: with Q(i) = sum over j of q(i, j) and
 *   P(i, v) = grad(i) * (Q(i) * exp(z(i, v) - lse(i)) - sum over j with index(i, j) == v of q(i, j)),
 * 0 in rows that do not count,
 *   dX = alpha * P W,   dW = alpha * P^T X      (type's; either may be NULL and is then skipped).
 *   lse, picked: as mpgemm_run_linear_distill wrote them.  grad: m FP32 values.
 *   What is said of P and of rows that do not count at mpgemm_run_linear_ce_grad holds here.  P's rounding to
 *   the inputs' type adds about as much to the error of dX and dW as their own rounding: in norm about
 *   1.4 times what dX and dW rounded from exact sums would have, more where the sums cancel.
 *   workspace: mpgemm_linear_distill_workspace_size(m, n, k, top, type, 1) bytes, which is also
 *   enough for mpgemm_run_linear_distill. */
mpgemm_status_t mpgemm_run_linear_distill_grad(mpgemm_handle_t handle, int64_t m, int64_t n, int64_t k,
                                               const float *alpha, const void *X, mpgemm_dtype_t type,
                                               int64_t ldx, const void *W, int64_t ldw,
                                               const mpgemm_teacher_t *teacher, const float *lse,
                                               const float *picked, const float *grad, void *dX,
                                               int64_t lddx, void *dW, int64_t lddw, void *workspace,
                                               uint64_t workspace_bytes, void *stream);

/* Workspace bytes of the two (train != 0: of the gradients too); 0 for sizes or types outside the
 * contract.  Host-only. */
uint64_t mpgemm_linear_distill_workspace_size(int64_t m, int64_t n, int64_t k, int64_t top,
                                              mpgemm_dtype_t type, int train);

/* Host-only argument checks (as mpgemm_check is for mpgemm_run). */
mpgemm_status_t mpgemm_check_linear_distill(int64_t m, int64_t n, int64_t k, const float *alpha,
                                            const void *X, mpgemm_dtype_t type, int64_t ldx,
                                            const void *W, int64_t ldw,
                                            const mpgemm_teacher_t *teacher, const float *loss,
                                            const float *lse, const float *picked,
                                            const void *workspace, uint64_t workspace_bytes);
mpgemm_status_t mpgemm_check_linear_distill_grad(int64_t m, int64_t n, int64_t k, const float *alpha,
                                                 const void *X, mpgemm_dtype_t type, int64_t ldx,
                                                 const void *W, int64_t ldw,
                                                 const mpgemm_teacher_t *teacher, const float *lse,
                                                 const float *picked, const float *grad,
                                                 const void *dX, int64_t lddx, const void *dW,
                                                 int64_t lddw, const void *workspace,
                                                 uint64_t workspace_bytes);

/* ---------------------------------------------------------------------------------------
 * Log probabilities of stored logits (as a product has left them), in one pass over them.
 * --------------------------------------------------------------------------------------- */

/* Queue, for each row i of z = alpha * Z (m x n, n >= 1, type MPGEMM_R_16F, MPGEMM_R_16BF or MPGEMM_R_32F,
 * read in whole aligned 16-byte blocks, 0 < alpha <= 1e30: 1 / a temperature):
 *   lse(i) = log(sum over v of exp(z(i, v))),
 *   logprob(i) = z(i, target(i)) - lse(i), 0 where the target is outside 0 .. n - 1,
 *   entropy(i) = - sum over v of p log p with p = exp(z(i, v) - lse(i)),
 *   top_index(i, j), top_logprob(i, j), j < top (0 .. 64): the columns of the row's largest logits and their
 *     log probabilities, falling, equal logits by the lower column first; past n columns -1 and -infinity.
 *   logprob (with target), lse, entropy: m FP32 values each, any NULL: not computed.  top_index: int64,
 *   top_logprob: FP32, both with rows of ld_top >= top elements; not touched for top == 0.
 *   A logit of -infinity has probability 0.  A row of nothing else has no distribution: lse, logprob and
 *   top_logprob are -infinity, the entropy 0.  A NaN or +infinity makes the row's numbers NaN (its
 *   top_index are columns in no particular order).
 *   The time depends on the values where there are many alternatives: rows that rise along the columns take up
 *   to 20 times as long as random ones (4095 x 128000 BF16 with 64: 4.1 ms and 0.22); masked and constant rows do not.
 *   ldz goes up to 2^31.  workspace: mpgemm_logprobs_workspace_size(m, n, z_type, top) bytes. */
mpgemm_status_t mpgemm_run_logprobs(mpgemm_handle_t handle, int64_t m, int64_t n, const float *alpha,
                                    const void *Z, mpgemm_dtype_t z_type, int64_t ldz,
                                    const int64_t *target, float *logprob, float *lse, float *entropy,
                                    int64_t top, int64_t *top_index, float *top_logprob,
                                    int64_t ld_top, void *workspace, uint64_t workspace_bytes,
                                    void *stream);

/* Workspace bytes (0 where none is needed, and for sizes or types outside the contract), and the
 * argument check.  Host-only. */
uint64_t mpgemm_logprobs_workspace_size(int64_t m, int64_t n, mpgemm_dtype_t z_type, int64_t top);
mpgemm_status_t mpgemm_check_logprobs(int64_t m, int64_t n, const float *alpha, const void *Z,
                                      mpgemm_dtype_t z_type, int64_t ldz, const int64_t *target,
                                      const float *logprob, const float *lse, const float *entropy,
                                      int64_t top, const int64_t *top_index, const float *top_logprob,
                                      int64_t ld_top, const void *workspace, uint64_t workspace_bytes);

/* ---------------------------------------------------------------------------------------
 * Gated products: the first half of a gated feed-forward block, both projections, the activation and
 * the product of the two in one call, and the gradient that comes back to it.  Types, storage and
 * everything else are as above; A is stored m x k.
 *
 * Pairs.  Two matrices of the same shape, type and leading dimension, the gate's and the up
 * projection's, are given by the gate's address and the elements from there to the up projection's:
 * stride_up for the weights, stride_kept for G and U, stride_d for dG and dU.  Side by side in
 * each row and one after the other are both such pairs.  Strides are multiples of 8 elements, not
 * negative; a pair that is written must not overlap itself: stride >= n and stride + n <= the leading
 * dimension, or stride >= (m - 1) * the leading dimension + n.  A pair of weights lies in one
 * allocation: the memory between the two is read too (its values have no effect), and 256 rows of
 * ldb and stride_up together span less than 2^31 bytes.
 * --------------------------------------------------------------------------------------- */
typedef struct {
    int act;                  /* an mpgemm_act_t */
    const void *bias_gate;    /* n values each, added to every row; NULL: none */
    const void *bias_up;
    int bias_type;            /* an mpgemm_dtype_t: the inputs' type or MPGEMM_R_32F */
    int64_t bias_stride;      /* grouped products: elements between two experts' biases (0: one for
                                 all); otherwise ignored */
    void *kept;               /* receives G and U (m x n each, the inputs' type); NULL: not kept */
    int64_t ld_kept;
    int64_t stride_kept;
} mpgemm_gated_t;

typedef struct {
    int act;                  /* an mpgemm_act_t */
    const void *kept;         /* G and U (m x n each, the inputs' type), as the forward call kept them */
    int64_t ld_kept;
    int64_t stride_kept;
    void *H;                  /* receives act(G) U (m x n, the inputs' type); NULL: not formed */
    int64_t ldh;
    float *dbias;             /* receives the column sums of dG (n values) and of dU (n values), for
                                 each expert; NULL: not computed */
} mpgemm_gated_grad_t;

/* Queue  G = alpha * A * op(Bg) + bias_gate,  U = alpha * A * op(Bu) + bias_up,  D = act(G) U.
 *   Bg and Bu: the pair at B (k x n for transb == N, n x k for transb == T).
 *   D is formed from G and U before their rounding.  k == 0 gives G and U their biases. */
mpgemm_status_t mpgemm_run_gated(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t m, int64_t n,
                                 int64_t k, const float *alpha, const void *A,
                                 mpgemm_dtype_t a_type, int64_t lda, const void *B,
                                 mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_up,
                                 const mpgemm_gated_t *gated, void *D, mpgemm_dtype_t d_type,
                                 int64_t ldd, void *stream);

/* Queue the gradient that comes back through a gated product: with E = alpha * A * op(B), the gradient
 * of its D (A the block's output gradient, B the down projection's weights),
 *   dG = E U act'(G),  dU = E act(G),  H = act(G) U,
 * with dG and dU the pair at D, and the column sums of both, summed in FP32 before the rounding in a
 * fixed order.  D == kept is allowed when the two pairs are alike in type, leading dimension and
 * stride: the gradients then take the factors' place.  m == 0 gives dbias = 0.
 *   workspace: mpgemm_gated_grad_workspace_size(1, m, n) bytes (none without dbias). */
mpgemm_status_t mpgemm_run_gated_grad(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t m,
                                      int64_t n, int64_t k, const float *alpha, const void *A,
                                      mpgemm_dtype_t a_type, int64_t lda, const void *B,
                                      mpgemm_dtype_t b_type, int64_t ldb,
                                      const mpgemm_gated_grad_t *grad, void *D,
                                      mpgemm_dtype_t d_type, int64_t ldd, int64_t stride_d,
                                      void *workspace, uint64_t workspace_bytes, void *stream);

/* The same for each expert's rows (see mpgemm_run_grouped for the offsets, and what becomes of rows of
 * no expert): expert e's weights are at B + e * stride_b elements, its biases at e * bias_stride, its
 * dbias at e * 2n.  workspace: mpgemm_gated_grad_workspace_size(groups, rows, n) bytes. */
mpgemm_status_t mpgemm_run_grouped_gated(mpgemm_handle_t handle, mpgemm_op_t transb, int64_t groups,
                                         int64_t rows, int64_t n, int64_t k, const float *alpha,
                                         const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                         const int32_t *offsets, const void *B,
                                         mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                         int64_t stride_up, const mpgemm_gated_t *gated, void *D,
                                         mpgemm_dtype_t d_type, int64_t ldd, void *stream);
mpgemm_status_t mpgemm_run_grouped_gated_grad(mpgemm_handle_t handle, mpgemm_op_t transb,
                                              int64_t groups, int64_t rows, int64_t n, int64_t k,
                                              const float *alpha, const void *A,
                                              mpgemm_dtype_t a_type, int64_t lda,
                                              const int32_t *offsets, const void *B,
                                              mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                              const mpgemm_gated_grad_t *grad, void *D,
                                              mpgemm_dtype_t d_type, int64_t ldd, int64_t stride_d,
                                              void *workspace, uint64_t workspace_bytes,
                                              void *stream);

/* Workspace bytes of the gradients for dbias (groups == 1 for mpgemm_run_gated_grad); 0 for sizes
 * outside the contract.  Host-only. */
uint64_t mpgemm_gated_grad_workspace_size(int64_t groups, int64_t m, int64_t n);

/* Host-only argument checks of the entry points above (as mpgemm_check is for mpgemm_run). */
mpgemm_status_t mpgemm_check_gated(mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                   const float *alpha, const void *A, mpgemm_dtype_t a_type,
                                   int64_t lda, const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                   int64_t stride_up, const mpgemm_gated_t *gated, const void *D,
                                   mpgemm_dtype_t d_type, int64_t ldd);
mpgemm_status_t mpgemm_check_gated_grad(mpgemm_op_t transb, int64_t m, int64_t n, int64_t k,
                                        const float *alpha, const void *A, mpgemm_dtype_t a_type,
                                        int64_t lda, const void *B, mpgemm_dtype_t b_type,
                                        int64_t ldb, const mpgemm_gated_grad_t *grad, const void *D,
                                        mpgemm_dtype_t d_type, int64_t ldd, int64_t stride_d,
                                        const void *workspace, uint64_t workspace_bytes);
mpgemm_status_t mpgemm_check_grouped_gated(mpgemm_op_t transb, int64_t groups, int64_t rows,
                                           int64_t n, int64_t k, const float *alpha, const void *A,
                                           mpgemm_dtype_t a_type, int64_t lda,
                                           const int32_t *offsets, const void *B,
                                           mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                           int64_t stride_up, const mpgemm_gated_t *gated,
                                           const void *D, mpgemm_dtype_t d_type, int64_t ldd);
mpgemm_status_t mpgemm_check_grouped_gated_grad(mpgemm_op_t transb, int64_t groups, int64_t rows,
                                                int64_t n, int64_t k, const float *alpha,
                                                const void *A, mpgemm_dtype_t a_type, int64_t lda,
                                                const int32_t *offsets, const void *B,
                                                mpgemm_dtype_t b_type, int64_t ldb,
                                                int64_t stride_b, const mpgemm_gated_grad_t *grad,
                                                const void *D, mpgemm_dtype_t d_type, int64_t ldd,
                                                int64_t stride_d, const void *workspace,
                                                uint64_t workspace_bytes);
mpgemm_status_t mpgemm_check_epilogue(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m, int64_t n,
                                      int64_t k, const float *alpha, const void *A,
                                      mpgemm_dtype_t a_type, int64_t lda, const void *B,
                                      mpgemm_dtype_t b_type, int64_t ldb,
                                      const mpgemm_epilogue_t *epilogue, const float *beta,
                                      const void *C, mpgemm_dtype_t c_type, int64_t ldc,
                                      const void *D, mpgemm_dtype_t d_type, int64_t ldd);
mpgemm_status_t mpgemm_check_epilogue_grad(mpgemm_op_t transa, mpgemm_op_t transb, int64_t m,
                                           int64_t n, int64_t k, const float *alpha, const void *A,
                                           mpgemm_dtype_t a_type, int64_t lda, const void *B,
                                           mpgemm_dtype_t b_type, int64_t ldb, mpgemm_act_t act,
                                           const void *Z, int64_t ldz, const void *D,
                                           mpgemm_dtype_t d_type, int64_t ldd, const float *dbias,
                                           const void *workspace, uint64_t workspace_bytes);
mpgemm_status_t mpgemm_check_grouped(mpgemm_op_t transb, int64_t groups, int64_t rows, int64_t n,
                                     int64_t k, const float *alpha, const void *A,
                                     mpgemm_dtype_t a_type, int64_t lda, const int32_t *offsets,
                                     const void *B, mpgemm_dtype_t b_type, int64_t ldb,
                                     int64_t stride_b, const mpgemm_epilogue_t *epilogue,
                                     const void *D, mpgemm_dtype_t d_type, int64_t ldd);
mpgemm_status_t mpgemm_check_grouped_grad(mpgemm_op_t transb, int64_t groups, int64_t rows,
                                          int64_t n, int64_t k, const float *alpha, const void *A,
                                          mpgemm_dtype_t a_type, int64_t lda,
                                          const int32_t *offsets, const void *B,
                                          mpgemm_dtype_t b_type, int64_t ldb, int64_t stride_b,
                                          mpgemm_act_t act, const void *Z, int64_t ldz,
                                          const void *D, mpgemm_dtype_t d_type, int64_t ldd,
                                          const float *dbias, const void *workspace,
                                          uint64_t workspace_bytes);
mpgemm_status_t mpgemm_check_grouped_wgrad(int64_t groups, int64_t rows, int64_t m, int64_t n,
                                           const float *alpha, const void *A,
                                           mpgemm_dtype_t a_type, int64_t lda, const void *X,
                                           mpgemm_dtype_t x_type, int64_t ldx,
                                           const int32_t *offsets, const float *beta,
                                           const void *D, mpgemm_dtype_t d_type, int64_t ldd,
                                           int64_t stride_d);
mpgemm_status_t mpgemm_check_linear_ce(int64_t m, int64_t n, int64_t k, const float *alpha,
                                       const void *X, mpgemm_dtype_t type, int64_t ldx,
                                       const void *W, int64_t ldw, const int64_t *target,
                                       const float *loss, const float *lse, const void *workspace,
                                       uint64_t workspace_bytes);
mpgemm_status_t mpgemm_check_linear_ce_grad(int64_t m, int64_t n, int64_t k, const float *alpha,
                                            const void *X, mpgemm_dtype_t type, int64_t ldx,
                                            const void *W, int64_t ldw, const int64_t *target,
                                            const float *lse, const float *grad, const void *dX,
                                            int64_t lddx, const void *dW, int64_t lddw,
                                            const void *workspace, uint64_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* MPGEMM_H */
