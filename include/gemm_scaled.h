/*
 * gemm_scaled.h -- C ABI of the 8-bit linear layer: products of 8-bit floating
 * point operands with a scale for each 128 elements, the quantisation that
 * makes such operands, and the root-mean-square norm that hands its rows to
 * a product in that form.
 *
 * An 8-bit operand is a matrix of e4m3 or e5m2 values q and fp32 scales s; the
 * element that it stands for is q * s.  A scale covers, of the summed dimension,
 * 128 elements (the last group may be shorter), and of the other dimension
 *
 *   GEMM_SCALE_VECTOR  one row or column.  The scales of an operand with R rows
 *                      or columns and K summed elements are ceil(K / 128) x R:
 *                      that of row r and group g at s[g * R + r].
 *   GEMM_SCALE_BLOCK   128 of them.  The scales are a matrix of blocks in the
 *                      order of the stored values: for values stored as S0 rows of
 *                      S1 contiguous elements, that of (i, j) at
 *                      s[(i / 128) * ceil(S1 / 128) + j / 128].
 *
 * A linear layer y = x * W^T (x: tokens x in, W: out x in) is
 *
 *   gemm_rms_norm (or gemm_scaled_quantize, ROWS)  x -> 8 bits
 *   gemm_scaled_quantize (BLOCKS)                  W -> 8 bits, once a step
 *   gemm_scaled_run        y = x W^T:   A = x row-major, B = W column-major
 *   gemm_scaled_quantize_both                      dy -> 8 bits, along rows and columns
 *   gemm_scaled_run        dx = dy W:   A = dy row-major, B = W row-major
 *   gemm_scaled_run        dW = dy^T x: A = dy column-major, B = x row-major, both
 *                          with vectors along the tokens (COLS)
 *
 * Conventions, beyond those of gemm.h (status codes, stream semantics and
 * dependent launches are the same):
 *  - The functions without a plan run on the current CUDA device, which must
 *    be the one that holds their operands.
 *  - Row matrices have a leading dimension in elements, at least the row
 *    length; scales, weights and sums are contiguous.  Any alignment of the
 *    element is accepted; rows at 16-byte boundaries (8-bit: 8) are faster.
 *  - Inputs and outputs must not overlap, but for the cases named below.
 *  - Results do not depend on timing (no floating-point atomics).
 *  - NaN and infinity: a NaN becomes a NaN of its own and counts for no scale;
 *    a group with an infinity has an infinite scale, so all of it stands for
 *    NaN.
 */
#ifndef PSM_GEMM_SCALED_H
#define PSM_GEMM_SCALED_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit floating point: 4 bits of exponent and 3 of mantissa (largest 448, no
 * infinity), or 5 and 2 (largest 57344). */
typedef enum { GEMM_E4M3 = 0, GEMM_E5M2 = 1 } gemm_fp8_t;
typedef enum { GEMM_SCALE_VECTOR = 0, GEMM_SCALE_BLOCK = 1 } gemm_scale_t;

/* Beside GEMM_F16 and GEMM_BF16, an output type of a scaled product. */
enum { GEMM_F32 = 2 };

/* Elements that share a scale, along the summed dimension. */
#define GEMM_SCALE_GROUP 128

/* ---------------------------------------------------------------- quantisation */

typedef enum {
    GEMM_QUANTIZE_ROWS = 0,   /* vectors along the rows: scales ceil(cols / 128) x rows */
    GEMM_QUANTIZE_COLS = 1,   /* vectors along the columns: scales ceil(rows / 128) x cols */
    GEMM_QUANTIZE_BLOCKS = 2  /* blocks: scales ceil(rows / 128) x ceil(cols / 128) */
} gemm_quantize_t;

/*
 * q, scales = x (rows x cols, 16-bit) in 8 bits.  With L the type's largest value
 * and m the largest magnitude of a group, at least 2^-100, the group's scale is
 * m / L (rounded to fp32) and q the 8-bit value nearest to x * L / m, ties to even.
 * Errors: INVALID_ARG (NULL operand, negative size, a leading dimension below
 * cols, bad enum), UNSUPPORTED (rows or cols > 2^31 - 1024, an operand not aligned
 * to its element), LAUNCH.  rows == 0 or cols == 0: nothing is written.
 */
gemm_status_t gemm_scaled_quantize(gemm_quantize_t kind, const void *x, int64_t ldx, int64_t rows,
                                   int64_t cols, gemm_dtype_t dtype, gemm_fp8_t type, void *q,
                                   int64_t ldq, float *scales, gemm_stream_t stream);

/* ROWS and COLS of one matrix, which is read once.  Errors: as above. */
gemm_status_t gemm_scaled_quantize_both(const void *x, int64_t ldx, int64_t rows, int64_t cols,
                                        gemm_dtype_t dtype, gemm_fp8_t type, void *q_rows,
                                        int64_t ldq_rows, float *scales_rows, void *q_cols,
                                        int64_t ldq_cols, float *scales_cols, gemm_stream_t stream);

/* ---------------------------------------------------------------- norm */

/*
 * Root-mean-square norm of each row, after the residual's addition:
 *
 *   s = x + residual, rounded to the 16-bit type (x where residual is NULL)
 *   rstd = 1 / sqrt(mean of s^2 + eps)
 *   y = s * rstd * weight, in fp32
 *
 * x, residual, sum, y: rows x hidden of `dtype`; weight: hidden of `dtype`.
 * Outputs, each written unless it is NULL (one of y and q at least is needed):
 * sum = s (may be x or residual, with its leading dimension); y rounded to
 * `dtype`; q and scales, y in 8 bits in vectors along the rows; rstd,
 * rows of fp32, for the gradient.  q and scales come together.
 * The 8-bit form is GEMM_QUANTIZE_ROWS's of the unrounded y: rstd cancels from y * L / m, so q
 * is the 8-bit value nearest to z * L / (the largest |z| of the group) with z = s *
 * weight, ties to even, and the scale is that largest times rstd, rounded, over L, rounded.
 * A group whose m is raised to 2^-100 has the value nearest to z * rstd * L / 2^-100, to
 * within fp32's roundings.  z is formed in fp32: it is exact from 2^-120 on, and a group in which
 * it overflows has an infinite scale.
 * Errors: INVALID_ARG (NULL x or weight, both y and q NULL, one of q and scales
 * without the other, sum without residual, negative size, negative or NaN eps, a
 * leading dimension of a given operand below hidden, bad enum), UNSUPPORTED
 * (hidden > GEMM_NORM_MAX_HIDDEN, rows > 2^31 - 1024, an operand not aligned to its
 * element), LAUNCH.  rows == 0 or hidden == 0: nothing is written.
 */
#define GEMM_NORM_MAX_HIDDEN 32768
gemm_status_t gemm_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldres,
                            const void *weight, float eps, int64_t rows, int64_t hidden,
                            gemm_dtype_t dtype, void *sum, int64_t ldsum, void *y, int64_t ldy,
                            void *q, int64_t ldq, gemm_fp8_t type, float *scales, float *rstd,
                            gemm_stream_t stream);

/* Bytes of device workspace gemm_rms_norm_grad needs (0 for rows or hidden 0).  Its contents need no
 * initialisation.  Errors: as gemm_rms_norm for the sizes, INVALID_ARG for a
 * NULL bytes. */
gemm_status_t gemm_rms_norm_grad_workspace_size(int64_t rows, int64_t hidden, size_t *bytes);

/*
 * Gradients of the norm for dy (rows x hidden), with s and rstd as the norm wrote
 * them and n = s * rstd:
 *
 *   dx = rstd * (weight * dy - n * mean(weight * dy * n)) + dsum
 *   dweight = the sum over the rows of dy * n
 *
 * dsum is the gradient that reaches s by the residual stream (NULL: none); dx,
 * rounded to `dtype`, is the gradient to x and to residual alike, and may be dy or
 * dsum, with its leading dimension.  dweight: hidden of fp32, written in full; NULL
 * where it is not wanted.
 * Errors: as gemm_rms_norm (NULL dy, s, weight, rstd or dx), WORKSPACE (NULL or
 * not 16-byte aligned while dweight is given).  rows == 0: only dweight is written,
 * as zeros.  hidden == 0: nothing is written.
 */
gemm_status_t gemm_rms_norm_grad(const void *dy, int64_t lddy, const void *s, int64_t lds,
                                 const void *weight, const float *rstd, const void *dsum,
                                 int64_t lddsum, int64_t rows, int64_t hidden, gemm_dtype_t dtype,
                                 void *dx, int64_t lddx, float *dweight, void *workspace,
                                 gemm_stream_t stream);

/* ---------------------------------------------------------------- scaled products */

typedef struct gemm_scaled_plan *gemm_scaled_plan_t;

typedef enum {
    GEMM_SCALED_STRAIGHT = 0,  /* A along the tensor memory's lanes, B along its columns */
    GEMM_SCALED_TURNED = 1,    /* B along the lanes: the rows of A cost steps of 16 */
    GEMM_SCALED_FEW = 2        /* without tensor memory, for few rows of A: A row-major and B
                                * column-major */
} gemm_scaled_form_t;

/* Options for gemm_scaled_plan_set_option (key, value). */
enum {
    /* CTAs of a scheduling unit: 1 (tiles of 128 x up to 128), or 2, a cluster
     * that runs pair MMAs (256 x 256); 0 (default) lets the plan choose. */
    GEMM_SCALED_OPT_CTAS = 1,
    /* how the product is computed, a gemm_scaled_form_t (all but STRAIGHT with one
     * CTA a unit); -1 (default) lets the plan choose. */
    GEMM_SCALED_OPT_FORM = 2,
    /* test hook: the scheduling unit with this index gives up before it writes
     * its first tile, as if a wait had run out, in every run that starts after
     * the call, replays of captured ones among them.  -1 (default) = off. */
    GEMM_SCALED_OPT_INJECT_GIVE_UP = 3
};

/* Keys for gemm_scaled_plan_get_info. */
enum {
    GEMM_SCALED_INFO_CTAS = 1,        /* CTAs of a scheduling unit (1 or 2) */
    GEMM_SCALED_INFO_FORM = 2,        /* a gemm_scaled_form_t */
    /* the rest for all forms but FEW */
    GEMM_SCALED_INFO_UNITS = 3,       /* scheduling units of a launch */
    GEMM_SCALED_INFO_TILES = 4,
    GEMM_SCALED_INFO_TILE_WIDTH = 5,  /* columns of a tile */
    GEMM_SCALED_INFO_SHARES = 6       /* parts along k of a tile that is split */
};

/*
 * Create a plan for C = A * B on the current device, where
 *
 *   C[m][n] = the sum over the groups g of k of
 *             sa(m, g) * sb(n, g) * (the sum over k in g of A[m][k] * B[k][n])
 *
 * A is M x K and B is K x N, of the 8-bit types type_a and type_b, in layout_a and
 * layout_b; each with the kind of scales given.  C is M x N row-major of out_dtype
 * (GEMM_F16, GEMM_BF16 or GEMM_F32), rounded once.  Sums are in fp32: within a
 * group by the tensor cores, over the groups in ascending order.
 * A form may multiply the two scales that meet, or a group's sum and one of them, first:
 * where one of these products is neither 0 nor a normal number of fp32, the result may be
 * less accurate, infinite or NaN.  Between operands as gemm_scaled_quantize makes them that takes
 * groups whose largest elements have a product below 2^-94 (their part of C is then
 * within 2^-111 all the same), or one above 2^128 or an element above 2^96.
 * The contiguous dimension of A and of B must be a multiple of 16.  A plan is
 * not thread-safe.
 * Errors: INVALID_ARG (NULL out, negative size, bad enum), UNSUPPORTED (a size >
 * 2^31 - 1024, a contiguous dimension that is no multiple of 16, 2^31 tiles or
 * more), NO_DEVICE, CUDA.
 */
gemm_status_t gemm_scaled_plan_create(gemm_scaled_plan_t *out, int64_t M, int64_t N, int64_t K,
                                      gemm_fp8_t type_a, gemm_fp8_t type_b, int out_dtype,
                                      gemm_layout_t layout_a, gemm_layout_t layout_b,
                                      gemm_scale_t scale_a, gemm_scale_t scale_b);

/* Same, but touches no device: for inspection only, as if the device had
 * num_sms SMs; gemm_scaled_run returns GEMM_ERR_NO_DEVICE.  Errors: as above,
 * INVALID_ARG for num_sms < 2. */
gemm_status_t gemm_scaled_plan_create_offline(gemm_scaled_plan_t *out, int64_t M, int64_t N, int64_t K,
                                              gemm_fp8_t type_a, gemm_fp8_t type_b, int out_dtype,
                                              gemm_layout_t layout_a, gemm_layout_t layout_b,
                                              gemm_scale_t scale_a, gemm_scale_t scale_b, int num_sms);

/* Set one GEMM_SCALED_OPT_* option.  On error the plan keeps its options.
 * Errors: INVALID_ARG (NULL plan, unknown key), UNSUPPORTED (value, or two options
 * that exclude each other), NO_DEVICE (offline plan) and CUDA (INJECT_GIVE_UP). */
gemm_status_t gemm_scaled_plan_set_option(gemm_scaled_plan_t plan, int key, int64_t value);

/* Read one GEMM_SCALED_INFO_* value.  Errors: INVALID_ARG. */
gemm_status_t gemm_scaled_plan_get_info(gemm_scaled_plan_t plan, int key, int64_t *value);

/* Bytes of device workspace gemm_scaled_run needs (may be 0), with the options set
 * so far.  Its contents need no
 * initialisation; two runs that share it must not overlap in time.
 * Errors: INVALID_ARG. */
gemm_status_t gemm_scaled_workspace_size(gemm_scaled_plan_t plan, size_t *bytes);

/*
 * Run the product on `stream`, asynchronously.  A and B must be 16-byte aligned;
 * C any alignment of its element (16 bytes and N a multiple of 8, 4 for fp32, are
 * faster).  K == 0: C is +0.
 * Errors: INVALID_ARG (NULL plan, or a NULL operand that is not empty),
 * UNSUPPORTED (alignment), WORKSPACE (NULL or not 16-byte aligned while one is
 * needed), NO_DEVICE (offline plan), CUDA, LAUNCH.
 */
gemm_status_t gemm_scaled_run(gemm_scaled_plan_t plan, const void *A, const float *scales_a,
                              const void *B, const float *scales_b, void *C, void *workspace,
                              gemm_stream_t stream);

/* As gemm_last_status, for a scaled plan.  After a timeout it waits for the
 * device; replays of captured runs are right again from then on, and may be
 * wrong between the timeout and this call. */
gemm_status_t gemm_scaled_last_status(gemm_scaled_plan_t plan, gemm_stream_t stream);

/* Free the plan and its words on the device: no run of it is under way, and captured ones are not
 * replayed any more.  NULL is accepted.  Always returns GEMM_OK. */
gemm_status_t gemm_scaled_plan_destroy(gemm_scaled_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* PSM_GEMM_SCALED_H */
