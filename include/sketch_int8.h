/*
 * sketch_int8.h -- C ABI of the 8-bit integer linears and of their products
 * grouped by expert (MI355X, gfx950).
 *
 * They are for linears that a model does not sketch, where its weights come as
 * 8-bit integers with a scale for each output channel ("Resumen Técnico",
 * Metodología §2 and §5: layers differ in how much compression they tolerate),
 * and for mixture-of-experts prompts, whose tokens stand in groups of any size,
 * one for each expert.  Serving only: no gradients.  Sketched linears and the
 * e4m3 experts of sketch_fp8.h are not taken; the order of the terms and the
 * weighted sum by token are the caller's.  The conventions of sketch.h hold (device pointers,
 * caller-owned memory, 16-byte alignment unless said otherwise, asynchronous on
 * the caller's stream, nothing allocated, host-side checks before anything is
 * enqueued, safe under HIP graph capture).
 *
 * Format
 * ------
 * A row (a weight's output channel, a batch's token) of a matrix [M][N] has one
 * scale s = amax / 127, rounded to float32, amax the row's largest magnitude,
 * and N codes: the integer next to 127 x / amax, ties to even, exactly rounded
 * (the quotient itself is not rounded on the way).  It stands for code * s.  A
 * row of zeros has zeros for codes and scale.  A row that holds NaN or an
 * infinity has the scale NaN and zeros for codes.
 *
 * Buffer of one matrix: codes [M][ld], ld = N rounded up to 128, columns N..ld
 * zero; at byte scales_offset, M float32 scales.  `count` matrices of one shape
 * (the experts of a layer) lie `bytes` apart.  Codes and scales from elsewhere
 * may be copied into such a buffer (any code, -128 included, and any scale);
 * the products read the padding of rows, so it has to be zero.
 */
#ifndef SUB_BIT_WEIGHT_SKETCH_INT8_H
#define SUB_BIT_WEIGHT_SKETCH_INT8_H

#include "sketch.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t M, N;          /* shape of one matrix, [M][N] row-major */
    int32_t count;         /* matrices of this shape, 1..SKETCH_INT8_MAX_COUNT; 0 means 1 */
} sketch_int8_params;

typedef struct {
    int64_t ld;            /* bytes per row of codes */
    size_t scales_offset;  /* from the codes of a matrix to its scales */
    size_t bytes;          /* one matrix (a multiple of 256); the buffer has count times this */
} sketch_int8_shape;

/* x_dtype of rows that sketch_int8_encode or sketch_int8_swiglu wrote. */
#define SKETCH_INT8_ROWS 4

/* Limits (SKETCH_EINVAL beyond them).  N: 128 * 128 * N < 2^31, so that the sum
 * of any codes' products fits 32 bits. */
#define SKETCH_INT8_MAX_N 131071
#define SKETCH_INT8_MAX_M 16777216
#define SKETCH_INT8_MAX_COUNT 65536
#define SKETCH_INT8_MAX_EXPERTS 512

/*
 * sketch_int8_layout -- sizes of the buffer (host only, pure).  SKETCH_EINVAL
 * for M < 0, N < 1 or a limit passed.
 */
sketch_status sketch_int8_layout(const sketch_int8_params* p, sketch_int8_shape* shape);

/*
 * sketch_int8_encode -- W [count][M][N] of w_dtype (float32, bfloat16 or
 * binary16), its rows ldw elements apart (ldw >= N; the matrices M * ldw), into
 * `buf` (every code and scale is written, with the padding of the rows).  W need
 * only be aligned to its element.
 *   status_dev  one device int32 that the kernel ORs SKETCH_FLAG_WEIGHT_RANGE
 *               into when some element is NaN or infinite, or NULL.
 * SKETCH_EINVAL when W and buf share memory.
 */
sketch_status sketch_int8_encode(const sketch_int8_params* p, const void* W, sketch_dtype w_dtype, int64_t ldw,
                                 void* buf, int32_t* status_dev, void* stream);

/*
 * sketch_int8_swiglu -- encodes the rows of h = silu(gate) * up, silu(g) =
 * g / (1 + exp(-g)): what stands between the products of an MLP.  gate and up
 * [M][N] of `dtype`, their rows ld_gate and ld_up elements apart (two halves of
 * one product's rows, say), aligned to their element.  p->count 0 or 1.  The codes are those of
 * h before any rounding: elements whose float32 value lies too near the middle
 * of two integers are computed in float64.  An h beyond float32's range counts
 * as infinite.  status_dev and SKETCH_EINVAL as for sketch_int8_encode.
 */
sketch_status sketch_int8_swiglu(const sketch_int8_params* p, const void* gate, int64_t ld_gate, const void* up,
                                 int64_t ld_up, sketch_dtype dtype, void* buf, int32_t* status_dev, void* stream);

/*
 * sketch_int8_workspace_bytes -- device scratch sketch_int8_matmul needs for
 * `batch` rows of X on the current device (host only).  Its contents need no
 * initialisation; calls that overlap in time need separate workspaces.
 */
sketch_status sketch_int8_workspace_bytes(const sketch_int8_params* p, int64_t batch, int x_dtype, int y_dtype,
                                          size_t* bytes);

/*
 * sketch_int8_matmul -- Y[t][m] = (sum_n x8[t][n] w8[m][n]) * sx[t] * sw[m].
 *   buf      the encoded weight (count 0 or 1).
 *   X        [batch][N] of x_dtype, encoded on the way in as sketch_int8_encode
 *            does; or, with x_dtype SKETCH_INT8_ROWS, the buffer of such an
 *            encode of {batch, N, 1}, for rows that several linears share.  Both
 *            give the same bits.
 *   Y        [batch][M] of y_dtype (SKETCH_F32, SKETCH_BF16 or SKETCH_F16),
 *            overwritten.
 * The sum is exact, in 32-bit integers; it is rounded to float32, multiplied by
 * sx[t], then by sw[m], in float32, and rounded to y_dtype.  No variant of the
 * kernels gives other bits.  A row of X that holds NaN or an infinity gives a
 * row of NaN; other rows are unaffected.  batch == 0 or M == 0 is a no-op.
 * Y may share memory with X where X is encoded into the workspace first, that
 * is with more than SKETCH_INT8_TOKENS rows that are not SKETCH_INT8_ROWS; any
 * other overlap of Y or the workspace with another buffer gives SKETCH_EINVAL.
 */
#define SKETCH_INT8_TOKENS 16
sketch_status sketch_int8_matmul(const sketch_int8_params* p, const void* buf, const void* X, int x_dtype,
                                 int64_t batch, void* Y, int y_dtype, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * Terms of a product grouped by expert: pairs of a row of X and an expert, in
 * the order of the experts, counts[e] of them for expert e.
 */
typedef struct {
    int64_t terms;         /* rows of Y, up to SKETCH_INT8_MAX_M */
    const void* counts;    /* [count] integers on the device, one for each expert.  Negative ones count as 0;
                              what passes `terms` in all is cut off */
    const void* rows;      /* [terms] integers on the device: the row of X of each term; NULL: term i takes row i */
    int32_t counts_bits;   /* 32 or 64 (signed) */
    int32_t rows_bits;     /* 32 or 64 (signed); not read where rows is NULL */
} sketch_int8_groups;

sketch_status sketch_int8_group_workspace_bytes(const sketch_int8_params* p, int64_t terms, int64_t x_rows,
                                                int x_dtype, int y_dtype, size_t* bytes);

/*
 * sketch_int8_matmul_group -- Y[i][m] = (sum_n x8[r][n] w8[e][m][n]) * sx[r] *
 * sw[e][m] for term i of expert e and row r of X, rounded as in
 * sketch_int8_matmul.
 *   buf      the experts' encoded weights (count of them, up to
 *            SKETCH_INT8_MAX_EXPERTS).
 *   X        [x_rows][N] of x_dtype, or SKETCH_INT8_ROWS, as above.  A row has
 *            one set of codes, whichever terms take it.  Without g->rows,
 *            x_rows >= terms.
 *   Y        [terms][M] of y_dtype.  Rows behind the last term of the last
 *            expert are left as they were.
 * The counts are read on the device, so routing needs no wait of the host.  A
 * term whose row lies outside 0..x_rows-1 gives a row of NaN.  terms == 0 or
 * M == 0 is a no-op.  Overlap of Y or the workspace with another buffer gives
 * SKETCH_EINVAL.
 */
sketch_status sketch_int8_matmul_group(const sketch_int8_params* p, const void* buf, const void* X, int x_dtype,
                                       int64_t x_rows, const sketch_int8_groups* g, void* Y, int y_dtype,
                                       void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
