/*
 * gemm_moe.h -- C ABI of the mixture-of-experts operators: tokens sorted by
 * expert and back, with weights applied, and one product per expert.
 *
 * A layer of E experts gives each of T tokens to k of them.  The T * k
 * (token, choice) pairs are its slots, slot t * k + j for choice j of token t.
 * In expert order the slots of expert 0 come first, then those of expert 1,
 * and so on, in slot order within an expert; row r of that order belongs to
 * expert e when offsets[e] <= r < offsets[e + 1].  A layer is
 *
 *   gemm_moe_sort      choices -> offsets, rows (slot -> row), slots (row -> slot)
 *   gemm_moe_dispatch  token rows -> expert rows
 *   gemm_grouped_run   one product per expert (GEMM_GROUPED_ROWS), as often as
 *                      the experts have layers
 *   gemm_moe_combine   expert rows -> token rows, weighted
 *
 * and its gradient gemm_moe_combine_grad, gemm_grouped_run (ROWS with the
 * other layout of B for the rows, INNER for the experts' matrices) and
 * gemm_moe_dispatch_grad.  Group sizes stay on the device: no call reads them
 * back, so a layer can be captured into a CUDA graph.
 *
 * Conventions, beyond those of gemm.h (status codes, stream semantics and
 * dependent launches are the same):
 *  - A slot whose choice is outside [0, E) is dropped: its rows entry is -1,
 *    it takes no row, and it contributes nothing (its weight and whatever an
 *    unused row holds are not read).  Rows from offsets[E] on are unused; an
 *    operator that writes rows writes them as +0.
 *  - Row matrices have a leading dimension in elements (ldx and so on), at
 *    least the row length.  Any alignment of the 16-bit element is accepted;
 *    16-byte aligned rows are faster (of others, the whole aligned 16-byte
 *    words that hold an element of the row are read).  Offsets, rows, slots and the weights are
 *    contiguous.
 *  - Sums are in fp32, in ascending choice order, rounded once; results do
 *    not depend on timing (no floating-point atomics).
 *  - The functions without a plan run on the current CUDA device, which must
 *    be the one that holds their operands.
 *  - Inputs and outputs must not overlap.
 */
#ifndef PSM_GEMM_MOE_H
#define PSM_GEMM_MOE_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_INDEX_I32 = 0, GEMM_INDEX_I64 = 1 } gemm_index_t;

/* The most experts (groups) any call takes. */
#define GEMM_MOE_MAX_EXPERTS 1024

/*
 * Bytes of device workspace gemm_moe_sort needs for these sizes (may be 0).
 * Its contents need no initialisation.  Errors: as gemm_moe_sort for the
 * sizes, INVALID_ARG for a NULL bytes.
 */
gemm_status_t gemm_moe_sort_workspace_size(int64_t tokens, int64_t topk, int64_t experts,
                                           size_t *bytes);

/*
 * Sort the slots by expert, stably.  ids: tokens x topk choices of type
 * id_type, token t at ids + t * ld_ids.  Writes offsets (experts + 1), rows
 * (tokens * topk: the row of each slot, -1 when dropped) and slots (tokens *
 * topk: the slot of each row, -1 for unused rows), each in full.
 * tokens == 0: only offsets is written, as zeros.
 * Errors: INVALID_ARG (NULL operand, negative size, topk < 1, experts < 1,
 * ld_ids < topk, bad id_type), UNSUPPORTED (experts > GEMM_MOE_MAX_EXPERTS,
 * topk > 65535, tokens * topk > 2^31 - 1024, an operand not aligned to its
 * element),
 * WORKSPACE (NULL or not 16-byte aligned while one is needed), CUDA, LAUNCH.
 */
gemm_status_t gemm_moe_sort(const void *ids, gemm_index_t id_type, int64_t ld_ids, int64_t tokens,
                            int64_t topk, int64_t experts, int32_t *offsets, int32_t *rows,
                            int32_t *slots, void *workspace, gemm_stream_t stream);

/*
 * xs[rows[t * topk + j]] = x[t] for every slot that is kept, and +0 in the
 * unused rows.  x: tokens x hidden; xs: (tokens * topk) x hidden; rows and
 * slots as gemm_moe_sort wrote them.
 * Errors (this and the next three): INVALID_ARG (NULL operand, negative size,
 * topk < 1, a leading dimension below hidden, bad dtype), UNSUPPORTED (topk >
 * 65535, tokens * topk > 2^31 - 1024, hidden > 2^30, an operand not aligned to
 * its element), LAUNCH.  tokens == 0 or hidden == 0: an empty output is left
 * alone.
 */
gemm_status_t gemm_moe_dispatch(const void *x, int64_t ldx, const int32_t *rows,
                                const int32_t *slots, int64_t tokens, int64_t topk, int64_t hidden,
                                gemm_dtype_t dtype, void *xs, int64_t ldxs, gemm_stream_t stream);

/* Gradient of gemm_moe_dispatch: dx[t] = the sum over j of
 * dxs[rows[t * topk + j]]; +0 for a token whose slots are all dropped. */
gemm_status_t gemm_moe_dispatch_grad(const void *dxs, int64_t lddxs, const int32_t *rows,
                                     int64_t tokens, int64_t topk, int64_t hidden,
                                     gemm_dtype_t dtype, void *dx, int64_t lddx,
                                     gemm_stream_t stream);

/* y[t] = the sum over j of weights[t * topk + j] * ys[rows[t * topk + j]];
 * weights: tokens x topk fp32. */
gemm_status_t gemm_moe_combine(const void *ys, int64_t ldys, const int32_t *rows,
                               const float *weights, int64_t tokens, int64_t topk, int64_t hidden,
                               gemm_dtype_t dtype, void *y, int64_t ldy, gemm_stream_t stream);

/* Gradients of gemm_moe_combine for dy (tokens x hidden): dys[r] = weights[s]
 * * dy[s / topk] for the slot s of each row, +0 in the unused rows; dweights[s]
 * = dy[s / topk] . ys[rows[s]] in fp32, +0 for a dropped slot. */
gemm_status_t gemm_moe_combine_grad(const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                                    const int32_t *rows, const int32_t *slots,
                                    const float *weights, int64_t tokens, int64_t topk,
                                    int64_t hidden, gemm_dtype_t dtype, void *dys, int64_t lddys,
                                    float *dweights, gemm_stream_t stream);

/* ------------------------------------------------------------ grouped products */

typedef enum {
    /* C[r] = A[r] * B_g for the rows r of each group g; +0 in the unused rows. */
    GEMM_GROUPED_ROWS = 0,
    /* C_g = the sum over the rows r of group g of A[r]^T * B[r], the gradient
     * of ROWS to its B for A and the gradient of its C; +0 for an empty group. */
    GEMM_GROUPED_INNER = 1
} gemm_grouped_kind_t;

typedef struct gemm_grouped_plan *gemm_grouped_plan_t;

/* Options for gemm_grouped_plan_set_option (key, value). */
enum {
    /* CTAs of a scheduling unit: 1 (tiles of 128 x up to 128), or 2, a cluster
     * that runs pair MMAs (256 x up to 256); 0 (default) lets the plan choose. */
    GEMM_GROUPED_OPT_CTAS = 1,
    /* test hook: the scheduling unit with this index gives up before it writes
     * its first piece, as if a wait had run out, in every run that starts after
     * the call, replays of captured ones among them.  -1 (default) = off. */
    GEMM_GROUPED_OPT_INJECT_GIVE_UP = 3
};

/* Keys for gemm_grouped_plan_get_info. */
enum {
    GEMM_GROUPED_INFO_CTAS = 1,    /* CTAs of a scheduling unit (1 or 2) */
    GEMM_GROUPED_INFO_UNITS = 2,   /* scheduling units of a launch */
    GEMM_GROUPED_INFO_TILE_M = 3,  /* tile extent along C's contiguous dimension */
    GEMM_GROUPED_INFO_TILE_N = 4,  /* the largest extent along the other one */
    GEMM_GROUPED_INFO_STAGES = 5,  /* depth of the shared-memory ring */
    GEMM_GROUPED_INFO_SMEM_BYTES = 6,
    GEMM_GROUPED_INFO_GROUPS = 7
};

/*
 * Create a plan for `groups` products over `rows` rows in all, on the current
 * device.  In both kinds A is rows x K row-major.
 *   ROWS   B: groups matrices of K x N in layout_b, one after another;
 *          C: rows x N row-major.
 *   INNER  B: rows x N row-major; C: groups matrices of K x N in layout_b.
 * A, B and C have one 16-bit type; accumulation is fp32, rounded once.  The
 * sizes of the groups are given to each run, on the device.
 * K and N must be multiples of 8 and the operands 16-byte aligned, as for
 * gemm_run.  A plan is not thread-safe.
 * Errors: INVALID_ARG (NULL out, groups < 1, another negative size, bad enum),
 * UNSUPPORTED (groups > GEMM_MOE_MAX_EXPERTS, rows, N or K > 2^31 - 1024, K or
 * N not a multiple of 8, 2^31 tiles or more), NO_DEVICE, CUDA.
 */
gemm_status_t gemm_grouped_plan_create(gemm_grouped_plan_t *out, gemm_grouped_kind_t kind,
                                       int64_t groups, int64_t rows, int64_t N, int64_t K,
                                       gemm_dtype_t dtype, gemm_layout_t layout_b);

/* Same, but touches no device: for inspection only, as if the device had
 * num_sms SMs; gemm_grouped_run returns GEMM_ERR_NO_DEVICE.  Errors: as above,
 * INVALID_ARG for num_sms < 2. */
gemm_status_t gemm_grouped_plan_create_offline(gemm_grouped_plan_t *out, gemm_grouped_kind_t kind,
                                               int64_t groups, int64_t rows, int64_t N, int64_t K,
                                               gemm_dtype_t dtype, gemm_layout_t layout_b,
                                               int num_sms);

/* Set one GEMM_GROUPED_OPT_* option.  On error the plan keeps its options.
 * Errors: INVALID_ARG (NULL plan, unknown key), UNSUPPORTED (value), NO_DEVICE
 * (offline plan) and CUDA (INJECT_GIVE_UP). */
gemm_status_t gemm_grouped_plan_set_option(gemm_grouped_plan_t plan, int key, int64_t value);

/* Read one GEMM_GROUPED_INFO_* value.  Errors: INVALID_ARG. */
gemm_status_t gemm_grouped_plan_get_info(gemm_grouped_plan_t plan, int key, int64_t *value);

/*
 * Host twin of the device scheduler: the work of scheduling unit `unit` for
 * the HOST offsets given (groups + 1, ascending, at most rows), in order, 9
 * int32 each: tile (a split one as -1 - the unit of its first share), group,
 * tile along C's contiguous dimension, first row of
 * the tile (of C for ROWS, of the group's matrix along its other dimension
 * for INNER), rows stored, accumulator width, first and end k-block of 64,
 * and the tile's k-blocks.  Writes at most max_units and the full count to
 * *n_units.  Errors: INVALID_ARG.
 */
gemm_status_t gemm_grouped_plan_units(gemm_grouped_plan_t plan, const int32_t *offsets, int64_t unit,
                                      int32_t *units, int64_t max_units, int64_t *n_units);

/* Bytes of device workspace gemm_grouped_run needs (may be 0), with the options
 * set so far (GEMM_GROUPED_OPT_CTAS changes it).  Its contents need no
 * initialisation; two runs that share it must not overlap in time.
 * Errors: INVALID_ARG. */
gemm_status_t gemm_grouped_workspace_size(gemm_grouped_plan_t plan, size_t *bytes);

/*
 * Run the products on `stream`, asynchronously.  offsets: groups + 1 device
 * int32, ascending, at most `rows` (gemm_moe_sort writes such); a value out of
 * order or range is taken as the nearest one in order and range, so no
 * access leaves the operands.  The rows before offsets[0] (offsets + e of a
 * longer array runs the groups from e on) and from offsets[groups] on are
 * unused.  C is written in full.
 * Errors: INVALID_ARG (NULL plan, or a NULL operand that is not empty),
 * UNSUPPORTED (alignment), WORKSPACE (NULL or not 16-byte aligned while one is
 * needed), NO_DEVICE (offline plan), CUDA, LAUNCH.
 */
gemm_status_t gemm_grouped_run(gemm_grouped_plan_t plan, const void *A, const void *B, void *C,
                               const int32_t *offsets, void *workspace, gemm_stream_t stream);

/* As gemm_last_status, for a grouped plan.  After a timeout it waits for the
 * device; replays of captured runs are right again from then on, and may be
 * wrong between the timeout and this call. */
gemm_status_t gemm_grouped_last_status(gemm_grouped_plan_t plan, gemm_stream_t stream);

/* Free the plan.  NULL is accepted.  Always returns GEMM_OK. */
gemm_status_t gemm_grouped_plan_destroy(gemm_grouped_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* PSM_GEMM_MOE_H */
