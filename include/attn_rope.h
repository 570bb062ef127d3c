/*
 * attn_rope.h — C ABI of the heads' norm and rotation: what stands between a
 * block's projections and its attention, and its gradient.
 *
 * A part is one of a call's tensors (queries, keys, values): heads x[b, s, h, :]
 * of D channels in the layout a projection leaves them, given by its strides.
 * For each head, in this order and each where the part asks for it,
 *
 *   norm      z = weight ⊙ x / sqrt(mean(x²) + eps)
 *   rotation  pair i of `pairs` turns by the angle positions[b, s, axis[i]] ·
 *             inv_freq[i]: with a, c its two channels,
 *             (a·cos − c·sin, a·sin + c·cos).  Its channels are i and i + pairs,
 *             or 2i and 2i + 1 where `interleaved`; channels from 2·pairs on stay
 *
 * and the result goes to y[b, h, s, :], contiguous: the layout attn_fwd takes.
 * A part with neither is only laid out.  All parts of a call share the batch,
 * the tokens, D, the positions and the type, and are done in one pass.
 *
 * Several axes (time, height, width of video patches; one for text) are one
 * rotation whose pairs go by different columns of `positions`.
 *
 * Precision: x, weight and the result are rounded once, at the end; sums,
 * norms and the rotation are fp32.  An angle is found in whole turns with 64
 * bits of fraction, so that it is as exact at position 2^31 as at 1: its error
 * stays below |position| · inv_freq · 2^-52 + 2^-21 radians.
 *
 * The entry points come from the same library as attn.h's, return its status
 * codes, validate every argument before touching CUDA (but for a workspace's size,
 * which goes by the device), enqueue on the caller's stream without synchronising and
 * allocate nothing beyond the status words that attn_fwd also uses.  Make the first
 * call on a device before any stream capture.  Results do not depend on the order in
 * which the GPU ran the work.
 */
#ifndef EXACT_ATTENTION_68_ATTN_ROPE_H_
#define EXACT_ATTENTION_68_ATTN_ROPE_H_

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ROPE_MAX_PARTS 4
#define ATTN_ROPE_MAX_AXES 8

/* A rotation; the arrays are host memory, read during the call. */
typedef struct {
  const double* inv_freq; /* [pairs] radians a position; finite, |inv_freq| <= 2^20 */
  const uint8_t* axis;    /* [pairs] column of positions, < axes; NULL: all 0 */
  int64_t pairs;          /* 0 .. D/2 */
  int interleaved;        /* 0 or 1 */
} attn_rope_t;

/* Where the call's tokens stand (device memory). */
typedef struct {
  const int32_t* at;                     /* any values; 4-byte aligned */
  int64_t stride_b, stride_s, stride_a;  /* in entries, >= 0 (0: shared) */
  int64_t axes;                          /* 1 .. ATTN_ROPE_MAX_AXES */
} attn_rope_positions_t;

/* One tensor of a call. */
typedef struct {
  const void* x;        /* device, 16-bit, 16-byte aligned: x[b, s, h, d] */
  int64_t stride_b, stride_s, stride_h; /* of x in values, multiples of 8, >= 0; channels are adjacent */
  int64_t heads;        /* 1 .. 65535 */
  const void* weight;   /* device [D], 4-byte aligned: the norm's weight; NULL: no norm */
  int weight_f32;       /* 1: weight (and dweight) fp32; 0: the call's 16-bit type */
  int turn;             /* 1: rotate */
  void* y;              /* forward: device, 16-bit [B, heads, S, D] contiguous, 16-byte aligned (written).
                           backward: dy, the same layout (read) */
  void* dx;             /* backward: device, laid out by dx_stride_* (written; no two values in one place) */
  int64_t dx_stride_b, dx_stride_s, dx_stride_h;
  void* dweight;        /* backward, where weight is given: device [D], weight's type (written); NULL: not wanted */
} attn_rope_part_t;

/*
 * attn_rope_fwd — norm, rotation and layout of n parts.
 *
 *   parts      host array of n (1 .. ATTN_ROPE_MAX_PARTS); dx, its strides and
 *              dweight are ignored
 *   rope, positions   NULL where no part turns
 *   B, S       >= 1, B·S < 2^30;  D a multiple of 8, at most 256;  B·S·heads < 2^31
 *   eps        finite, >= 0
 *   dtype      ATTN_BF16 or ATTN_F16
 *
 * A y must not overlap any x, weight or other y, nor the positions.
 */
ATTN_API attn_status_t attn_rope_fwd(const attn_rope_part_t* parts, int n, const attn_rope_t* rope,
                                     const attn_rope_positions_t* positions, int64_t B, int64_t S,
                                     int64_t D, float eps, attn_dtype_t dtype, cudaStream_t stream);

/* Bytes of workspace attn_rope_bwd needs on the current device (16: none, NULL
 * will do; 0: on an argument it would refuse, or where the device cannot be asked). */
ATTN_API size_t attn_rope_bwd_workspace(const attn_rope_part_t* parts, int n, int64_t B, int64_t S,
                                        int64_t D);

/*
 * attn_rope_bwd — the gradient: from dy = ∂L/∂y of each part (in `y`), with dz
 * the rotation of dy by the negative angles and r = 1 / sqrt(mean(x²) + eps),
 *
 *   dweight = Σ_{b,s,h} dz ⊙ x·r,   dx = r·(g − x·r · mean(g ⊙ x·r)),  g = weight ⊙ dz
 *
 * or dx = dz where the part has no norm (its x is then not read and may be NULL).
 * dx may be a view of a packed gradient of the projection, in any order of its
 * dimensions, beside other parts' dx: where two dx interleave along a dimension they
 * have the same stride there and lie in the same blocks of it.  It must not overlap
 * anything read, as a range from its first value to its last.  A second launch adds up dweight, from
 * fp32 sums in the workspace (16-byte aligned, contents mean nothing before or
 * after; calls that may run at the same time need one each).
 */
ATTN_API attn_status_t attn_rope_bwd(const attn_rope_part_t* parts, int n, const attn_rope_t* rope,
                                     const attn_rope_positions_t* positions, int64_t B, int64_t S,
                                     int64_t D, float eps, attn_dtype_t dtype, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_68_ATTN_ROPE_H_ */
