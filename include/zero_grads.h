/* zero_grads.h -- C ABI of the gradient-list operators: the norm over many
 * tensors, clipping by it, and scaling into other tensors, on one AMD Instinct
 * MI355X (gfx950).
 *
 * The sharded step of zero_shard.h takes the norm of one rank's flat 16-bit
 * shard and applies the clip inside its Adam pass.  The calls here work on what
 * stands before and beside that step: the list of gradients a backward pass
 * leaves, one per parameter, in fp16, bf16 or fp32 -- its global and per-tensor
 * norms, the clipped gradients themselves, and their conversion into the flat
 * 16-bit buffer [psi] that zero_reduce_grads takes from each rank.
 *
 * With g an element (exact in fp32) and inv the call's inverse loss scale:
 *   u      = fp32(g * inv)
 *   L2:    acc = sum of u * u in fp64 (each square exact),  norm = sqrt(acc)
 *   MAX:   acc = norm = largest |u|
 *   flag   = norm not finite, which is exactly when some u is not
 *   clip:  c = max_norm / (norm + 1e-6) in fp64, rounded once to fp32, when that
 *          is below 1 and the flag is not set, else 1 (the coefficient of
 *          zero_grad_norm);  result = fp32(u * c), rounded once more, to nearest
 *          even, into the destination's type
 *   scale: result = fp32(g * factor), rounded once more into the destination's type
 * A list with an infinity or a NaN is not clipped (c = 1): its values, carried
 * over, are what makes the step that takes them in skip.  fp16 results beyond
 * 65504 become infinite; a NaN is written to a 16-bit destination as the
 * format's positive canonical quiet NaN (see zero_cast_params).
 *
 * The sums are formed in an order fixed by the list's sizes and its tensors'
 * alignment to 16 bytes: the same values there give the same bits, in every
 * call and replay and whatever else runs on the GPU.
 *
 * Conventions are those of zero_shard.h (zero_status_t, zero_last_error(),
 * streams, caller-owned device memory), and:
 *   - A handle is a plan for one list: its sizes, types and pitches.  The
 *     addresses may change from step to step (zero_grads_bind).  Calls use the
 *     device that was current at zero_grads_init.  They stand in the workspace:
 *     a call works on those of the last bind that has run before it.
 *   - One pass is zero_grads_norm -> [exchange with other ranks] ->
 *     zero_grads_clip, or both in one call, zero_grads_clip_norm; zero_grads_scale
 *     stands alone.  A zero_grads_clip without the norm of these values before
 *     it (none yet, or clipped, scaled or bound since) returns ZERO_ESTATE.
 *   - All calls but init, query and destroy only enqueue kernels, and nothing
 *     of a result is kept on the host, so they can be captured into a HIP graph
 *     and replayed.  The scalar arguments (inv, max_norm) and a bind's addresses
 *     are fixed in it.  A captured call has run when its graph is replayed and
 *     not before, and every replay counts as its calls: a clip goes by the norm
 *     that ran last, its kind and inverse scale, and every call by the addresses
 *     bound last, wherever they were captured or not.  So a graph without a bind
 *     uses whatever is bound when it is replayed, and a list bound in a graph
 *     stays bound behind it: its memory has to last until another bind has run
 *     and the graph is not replayed any more.
 *   - The host does not see replays.  Once a zero_grads_norm of the handle has
 *     been captured, or where a replay comes between a norm and its clip, the
 *     device judges: a clip that finds no norm of these values there (or, for
 *     ZERO_CLIP_EACH, none with per_tensor) writes nothing, and the
 *     zero_grads_query behind it returns ZERO_ESTATE.  A list that takes norms
 *     only (see zero_grads_plan) is not bound once a call that writes has been
 *     captured, and once one has been bound in a graph the handle does not write.
 *   - Calls on one handle must not overlap, replays of graphs captured from it
 *     included: they share its workspace.  Different handles are independent.
 */
#ifndef ZERO_GRADS_H
#define ZERO_GRADS_H

#include <stdint.h>

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zero_grads* zero_grads_t; /* opaque host handle */

typedef enum { ZERO_NORM_L2 = 1, ZERO_NORM_MAX = 2 } zero_norm_t;
typedef enum { ZERO_CLIP_GLOBAL = 1, ZERO_CLIP_EACH = 2 } zero_clip_t;

/* One tensor of a list: `rows` runs of `cols` consecutive elements, row r of the
 * source starting src_pitch * r elements after the first.  A contiguous tensor
 * is one row.  Element r * cols + c of the source is element r * cols + c of the
 * destination. */
typedef struct {
  void* src;          /* device address of the gradient, aligned to its element size; may be   */
                      /* NULL when the tensor has no elements                                  */
  void* dst;          /* where zero_grads_clip and zero_grads_scale write, or NULL: in place   */
  int64_t rows, cols; /* each >= 0; rows * cols elements                                       */
  int64_t src_pitch;  /* elements; >= cols, or any value when rows <= 1                        */
  int64_t dst_pitch;  /* the same for dst (not read when dst is NULL)                          */
  int32_t src_dtype;  /* ZERO_F16, ZERO_BF16 or ZERO_F32                                       */
  int32_t dst_dtype;  /* the same for dst (not read when dst is NULL)                          */
} zero_grads_tensor_t;

typedef struct {
  int64_t elems;           /* elements of the list                                    */
  int64_t num_chunks;      /* work items of the kernels                               */
  int64_t workspace_bytes; /* device workspace the caller allocates (256-byte aligned) */
} zero_grads_info_t;

/* Sizes only; no GPU work.  1 <= n <= 2^22 - 1 tensors, at most 2^60 elements
 * and 2^22 - 1 blocks of work (about 3.4e10 elements).
 * A destination must be its own source exactly (same address, type and pitch:
 * in place) or share no element with any source or other destination; column
 * slices of one matrix are told apart by their pitch, rows of different pitches
 * that interleave are taken to overlap.  Sources may repeat; a list whose
 * tensors without a destination overlap takes norms only, and the calls that
 * write return EINVAL.
 * EINVAL on a bad list; ENOMEM when the host tables do not fit in host memory. */
zero_status_t zero_grads_plan(const zero_grads_tensor_t* tensors, int64_t n, zero_grads_info_t* out);

/* Builds the handle and copies the work table into the workspace (device
 * memory, 256-byte aligned, kept until zero_grads_destroy).  Synchronises the
 * stream.  EINVAL on a bad list, a null or misaligned workspace or one smaller
 * than zero_grads_plan's; ENOMEM when the handle cannot be allocated. */
zero_status_t zero_grads_init(const zero_grads_tensor_t* tensors, int64_t n, void* workspace,
                              int64_t workspace_capacity, void* stream, zero_grads_t* out);

/* Sizes of an initialised handle. */
zero_status_t zero_grads_info(zero_grads_t h, zero_grads_info_t* out);

/* Gives the list's tensors new addresses, in list order (host arrays [n], read
 * during the call): src[i], and dst[i] where the list was planned with a
 * destination (dst may be NULL when no tensor was).  Sizes, types and pitches
 * stay; a tensor planned in place is bound in place, and one planned with a
 * destination is not.  Enqueues small kernels that write the work table.  EINVAL
 * on what zero_grads_plan would refuse; the handle then keeps its addresses.
 * After EHIP another bind has to come before any other call. */
zero_status_t zero_grads_bind(zero_grads_t h, void* const* src, void* const* dst, void* stream);

/* The list's norm, its flag, and with per_tensor != 0 every tensor's norm, on
 * the device.  norm is a zero_norm_t.  EINVAL on another norm or an
 * inv_loss_scale that is not finite and positive. */
zero_status_t zero_grads_norm(zero_grads_t h, int32_t norm, float inv_loss_scale, int32_t per_tensor, void* stream);

/* Device addresses, inside the workspace and fixed for the handle's lifetime.
 * acc, found_inf and tensor_acc [n] are what zero_grads_clip reads, so an
 * exchange with other ranks can happen in place between the two calls (acc and
 * tensor_acc: sum for L2, maximum for MAX; found_inf: maximum).  norm and
 * norms [n] are the norms in fp32; after a zero_grads_clip, norm is the one it
 * clipped by.  tensor_acc and norms are written by calls with per_tensor (an
 * empty tensor's are 0 in each of them).  Any output pointer may be NULL. */
zero_status_t zero_grads_device(zero_grads_t h, double** acc, int32_t** found_inf, float** norm, double** tensor_acc,
                                float** norms);

/* Writes the clipped gradients.  scope ZERO_CLIP_GLOBAL: one coefficient, from
 * the global norm; ZERO_CLIP_EACH: a coefficient for each tensor, from its own
 * norm (the norm call needs per_tensor, ESTATE otherwise).  other_ranks_found_inf
 * and other_ranks_acc (>= 0) are other ranks' flag and acc, combined by the
 * caller, for the global norm and the flag; pass 0 and 0 without other ranks or
 * after an exchange on the device.  max_norm <= 0 disables clipping; unscaling
 * and conversion remain.  In place, a call whose inv and coefficient are both 1
 * writes nothing.  EINVAL on another scope, a NaN max_norm or a negative
 * other_ranks_acc. */
zero_status_t zero_grads_clip(zero_grads_t h, int32_t scope, int32_t other_ranks_found_inf, double other_ranks_acc,
                              float max_norm, void* stream);

/* zero_grads_norm and zero_grads_clip in one call, for a list that no other rank
 * shares.  Per-tensor norms are kept if per_tensor is set or scope is
 * ZERO_CLIP_EACH.  The same results, to the bit. */
zero_status_t zero_grads_clip_norm(zero_grads_t h, int32_t norm, float inv_loss_scale, int32_t per_tensor,
                                   int32_t scope, float max_norm, void* stream);

/* Writes every element times `factor` (finite) to its destination.  In place, a
 * factor of 1 writes nothing. */
zero_status_t zero_grads_scale(zero_grads_t h, float factor, void* stream);

/* What the last zero_grads_clip (or zero_grads_clip_norm) used: the global norm,
 * whether the flag was set, and the global coefficient (1 for ZERO_CLIP_EACH).
 * Any output pointer may be NULL.  Synchronises the stream.  ESTATE before the
 * first clip has run, and when the last one found no norm. */
zero_status_t zero_grads_query(zero_grads_t h, double* norm, int32_t* found_inf, float* coef, void* stream);

/* Frees the host handle (never caller memory). */
zero_status_t zero_grads_destroy(zero_grads_t h);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_GRADS_H */
