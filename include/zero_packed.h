/* zero_packed.h -- C ABI of the packed-row operators: matrices kept in 8 bits
 * with one scale for each row, on one AMD Instinct MI355X (gfx950).
 *
 * The sharded step of zero_shard.h bounds what a rank keeps of the model's
 * states; what is left are the residual states, above all the activations that
 * a layer keeps for its backward pass.  The calls here keep them in 8 bits, and
 * use them as they are: a linear layer multiplies its packed input by its packed
 * weights in 8-bit integers, the same packed input gives the weight gradient,
 * straight into the gradient buffer that the step takes in, and an activation
 * function's gradient comes from the function's packed input.
 *
 * Packed rows.  Row r of a matrix [rows][cols] is cols 8-bit integers q and one
 * fp32 scale; it stands for the values q * scale.  With top the row's largest
 * magnitude:
 *   ZERO_SCALE_POW2  scale = the smallest power of two of at least 2^-126 with
 *                    top <= 127 scale; q = x / scale, rounded to nearest even.
 *                    Every value q * scale is exact in bf16, so a packed value is
 *                    rounded once and not again where it is used.
 *   ZERO_SCALE_MAX   scale = fp32(top / 127), at least 2^-126; q = the exact
 *                    quotient x / scale, rounded to nearest even, within +-127.
 * A row of zeros has scale 0.  A row with an infinity or a NaN has scale NaN and
 * q = 0: all its values are NaN, and so are the results that they enter, down to
 * the gradient, whose step is skipped.
 * A q row takes `pitch` bytes; those from cols up to the next multiple of 16 are
 * part of it and hold zeros (zero_packed_write and zero_packed_act store them).
 *
 * Rows are tokens (activations) or output channels (weights), so the products'
 * scales are one for each token and one for each channel.  m tokens, k input
 * features, n output features; x [m][k], w [n][k], y and dy [m][n]:
 *   linear       y  = fp32(fp32(acc * x.scale) * w.scale) [+ bias], acc the exact
 *                integer sum of q products in fp32
 *   weight_grad  dw = sum over tokens of dy * x        [n][k]  [+ dw]
 *                db = sum over tokens of dy            [n]     [+ db]
 *   input_grad   dx = sum over channels of dy * w      [m][k]  [+ dx]
 * each rounded once to its result's type, to nearest even (fp16 results beyond
 * 65504 become infinite; a NaN is written to a 16-bit result as the format's
 * positive canonical quiet NaN).  The gradients' sums are fp32 sums of exact
 * products where the rows' scales are powers of two (ZERO_SCALE_POW2).  For
 * ZERO_SCALE_MAX dy * scale enters as the sum of two bf16 values, within 2^-17 of
 * itself for any fp16 dy and for bf16 dy of magnitudes from 2^-85 to 2^96: an
 * fp32 dw of 4096 normal tokens is then 2.4e-6 of its norm off, with powers of
 * two 1e-7.  Sums are formed in an order fixed by the sizes: the same inputs give
 * the same bits in every call and replay.
 *
 * Activation functions, in fp32:
 *   ZERO_ACT_GELU  f(x) = x / (1 + exp(-2 sqrt(2/pi) (x + 0.044715 x^3))), the tanh form
 *   ZERO_ACT_SILU  f(x) = x / (1 + exp(-x))
 *   y = f(x), or gated, x = [g | u] with g and u [m][n]: y = f(g) * u
 * The gradient goes by the packed values of x.
 *
 * Conventions are those of zero_shard.h (zero_status_t, zero_last_error(),
 * streams, caller-owned device memory), and:
 *   - Calls keep nothing: no handle, no state on the device.  They use the
 *     current device, which has to be the one that holds their memory.
 *   - Calls only enqueue kernels, so they can be captured into a HIP graph and
 *     replayed, at the addresses captured.
 *   - A workspace is read and written by the call's own kernels only, so calls
 *     that do not overlap in time may share one; graphs whose replays may
 *     overlap, each other or eager calls, need one each.
 *   - A result shares no element with an operand, a packed result neither, except
 *     where a call says so; column slices of one matrix are told apart by their
 *     pitch.
 *   - Matrices without rows or columns are fine; their addresses may be NULL.
 *   - A product's result of 2^22 tiles or more is refused: tiles of 256 x 256, in a
 *     linear layer of up to 64 tokens of 16 columns.
 */
#ifndef ZERO_PACKED_H
#define ZERO_PACKED_H

#include <stdint.h>

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ZERO_SCALE_POW2 = 1, ZERO_SCALE_MAX = 2 } zero_scale_t;
typedef enum { ZERO_ACT_GELU = 1, ZERO_ACT_SILU = 2 } zero_act_t;
typedef enum { ZERO_PACKED_LINEAR = 1, ZERO_PACKED_WEIGHT_GRAD = 2, ZERO_PACKED_INPUT_GRAD = 3 } zero_packed_call_t;

/* A matrix in floating point: element (r, c) is data[r * pitch + c]. */
typedef struct {
  void* data;         /* device address, aligned to the element size                  */
  int64_t rows, cols; /* each >= 0, <= 2^30                                            */
  int64_t pitch;      /* elements from row to row: >= cols and <= 2^30, or any value when rows <= 1 */
  int32_t dtype;      /* ZERO_F16, ZERO_BF16 or ZERO_F32                               */
} zero_matrix_t;

/* Packed rows.  cols <= 2^20; pitch <= 2^22. */
typedef struct {
  int8_t* q;          /* device address, 16-byte aligned                               */
  float* scale;       /* device [rows], one for each row                               */
  int64_t rows, cols; /* each >= 0; rows <= 2^30                                       */
  int64_t pitch;      /* bytes from row to row: a multiple of 16, >= cols              */
  int32_t rule;       /* zero_scale_t that the scales follow                           */
} zero_packed_t;

/* Packs x (any of the three types) into p, of the same size. */
zero_status_t zero_packed_write(const zero_matrix_t* x, const zero_packed_t* p, void* stream);

/* The values of p, rounded into out's type, of the same size. */
zero_status_t zero_packed_read(const zero_packed_t* p, const zero_matrix_t* out, void* stream);

/* Device workspace of a product call with m tokens, k input and n output
 * features; 0 where it needs none (the workspace may be NULL then).  Sizes only. */
zero_status_t zero_packed_workspace(int32_t call, int64_t m, int64_t k, int64_t n, int64_t* bytes);

/* y [m][n], of any type, from x [m][k] and w [n][k].  bias: one row of n, of any
 * type, or NULL.  k <= 131056, so that no sum leaves 32 bits.  The workspace is
 * 256-byte aligned and at least zero_packed_workspace(ZERO_PACKED_LINEAR, ...). */
zero_status_t zero_packed_linear(const zero_packed_t* x, const zero_packed_t* w, const zero_matrix_t* bias,
                                 const zero_matrix_t* y, void* workspace, int64_t workspace_capacity, void* stream);

/* dw [n][k] and, unless it is NULL, db (one row of n), each of any type, from dy
 * [m][n] (fp16 or bf16) and x [m][k].  accumulate != 0: added to what they hold. */
zero_status_t zero_packed_weight_grad(const zero_matrix_t* dy, const zero_packed_t* x, const zero_matrix_t* dw,
                                      const zero_matrix_t* db, int32_t accumulate, void* workspace,
                                      int64_t workspace_capacity, void* stream);

/* dx [m][k], of any type, from dy [m][n] (fp16 or bf16) and w [n][k].
 * accumulate != 0: added to what dx holds. */
zero_status_t zero_packed_input_grad(const zero_matrix_t* dy, const zero_packed_t* w, const zero_matrix_t* dx,
                                     int32_t accumulate, void* workspace, int64_t workspace_capacity, void* stream);

/* Activation function of x (any type) [m][n], or [m][2n] if gated != 0.  Writes
 * its packed input xp (of x's size), y [m][n] of any type and the packed result
 * yp [m][n]; each of the three may be NULL, but not all.  yp is packed from the
 * fp32 result, not from y's roundings. */
zero_status_t zero_packed_act(int32_t kind, int32_t gated, const zero_matrix_t* x, const zero_packed_t* xp,
                              const zero_matrix_t* y, const zero_packed_t* yp, void* stream);

/* dx (of xp's size) from dy [m][n], of any types, and the packed input xp.  dx
 * may be dy itself (same address, pitch and type) if gated is 0. */
zero_status_t zero_packed_act_grad(int32_t kind, int32_t gated, const zero_packed_t* xp, const zero_matrix_t* dy,
                                   const zero_matrix_t* dx, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_PACKED_H */
