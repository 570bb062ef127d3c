/*
 * attn_cross.h — C ABI of cross-attention: queries of one sequence over the keys
 * and values of another (an encoder's states, a prompt's, a memory's), and its
 * gradient.
 *
 * attn.h's attention (out = softmax(scale·q·kᵀ)·v with the row logsumexp, its
 * steps and precision) with three differences: the keys' number Sk is its own,
 * sequence b has lens[b] of them, and query heads h·G .. h·G+G-1 share key/value
 * head h, G = q_heads / heads.  No mask goes by the query's place.
 *
 * These entry points come from the same library, return attn.h's status codes,
 * record device-side findings in the status word that attn_device_status reads,
 * validate every argument before touching CUDA (but for the workspace's size, which
 * goes by the device), enqueue on the caller's stream without synchronising, and
 * allocate nothing beyond the status words that attn_fwd also uses.  Make the first call on a device before any stream capture.
 *
 * What k and v hold behind a sequence's end may be anything, NaN and infinities
 * included; it is never used.  lens is read on the device: an entry outside
 * [0, Sk] counts as the nearer end and is reported as ATTN_ERR_DEVICE_CHECK
 * (every build).
 */
#ifndef EXACT_ATTENTION_68_ATTN_CROSS_H_
#define EXACT_ATTENTION_68_ATTN_CROSS_H_

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes of a call. */
typedef struct {
  int64_t batch;    /* >= 1 */
  int64_t q_heads;  /* a multiple of heads */
  int64_t heads;    /* key/value heads, >= 1 */
  int64_t Sq;       /* >= 1; q_heads / heads · Sq < 2^31 - 128 */
  int64_t Sk;       /* >= 1; < 2^31 - 128 */
  int64_t head_dim; /* a multiple of 8, at most 256 */
} attn_cross_t;

/*
 * attn_cross_fwd_workspace — bytes of workspace that attn_cross_fwd needs on the
 * current device for these sizes (16: none, workspace may be NULL; 0: on sizes it
 * would refuse, or where the device cannot be asked).
 */
ATTN_API size_t attn_cross_fwd_workspace(const attn_cross_t* sizes);

/*
 * attn_cross_fwd — the forward.
 *
 *   q        device, 16-bit [batch, q_heads, Sq, head_dim] contiguous, 16-byte aligned
 *   k, v     device, 16-bit [batch, heads, Sk, head_dim] contiguous, 16-byte aligned
 *   lens     device int32 [batch], or NULL: all Sk
 *   out      device, 16-bit, shaped as q, 16-byte aligned (written)
 *   lse      device fp32 [batch, q_heads, Sq] (written)
 *   scale    finite, > 0
 *   dtype    ATTN_BF16 or ATTN_F16
 *   workspace, workspace_bytes   device, 16-byte aligned, at least
 *            attn_cross_fwd_workspace bytes; contents need no preparation and mean
 *            nothing afterwards.  Calls that may run at the same time (other
 *            streams, graphs that share it) need a workspace each.
 *   wait_timeout_ns  bound on each in-kernel wait (ATTN_DEFAULT_WAIT_TIMEOUT_NS)
 *
 * A query of a sequence without keys gets out = 0 and lse = -inf.  One of a sequence
 * with keys, and with a NaN score or one of +inf, gets NaN in both; with no score but
 * -inf, NaN in out and -inf in lse.  How the work is
 * cut goes by the sizes, not by lens, which is on the device.  Results do not
 * depend on the order in which the GPU ran the work.
 */
ATTN_API attn_status_t attn_cross_fwd(const attn_cross_t* sizes, const void* q, const void* k,
                                      const void* v, const int32_t* lens, void* out, float* lse,
                                      float scale, attn_dtype_t dtype, void* workspace,
                                      size_t workspace_bytes, uint64_t wait_timeout_ns,
                                      cudaStream_t stream);

/* The same for attn_cross_bwd. */
ATTN_API size_t attn_cross_bwd_workspace(const attn_cross_t* sizes);

/*
 * attn_cross_bwd — gradient of attn_cross_fwd with respect to q, k and v: attn_bwd's
 * formulas, with sums over the query heads that share a key head.
 *
 * P and dS are rounded to the 16-bit type for their products; where a call has few
 * queries (q_heads / heads · Sq <= 128, and 512 in all; or at most 64 queries and 64 keys)
 * they enter in two terms.  fp16 holds a dS below 2^-14 in steps of 2^-24, and one above
 * 65504 as an infinity, whose sums are infinite or NaN: scale the loss between the two,
 * or use bf16.
 *
 *   q, k, v, lens, out, lse   the forward's inputs and results (read)
 *   dout     device, 16-bit, shaped as q, 16-byte aligned (read)
 *   dq       device, shaped as q, 16-byte aligned (written)
 *   dk, dv   device, shaped as k, 16-byte aligned (written; 0 for keys that are not there)
 *   delta    device fp32 [batch, q_heads, Sq] (written): rowsum(dout ⊙ out)
 *   scale, dtype, workspace, wait_timeout_ns   as above
 */
ATTN_API attn_status_t attn_cross_bwd(const attn_cross_t* sizes, const void* q, const void* k,
                                      const void* v, const int32_t* lens, const void* out,
                                      const float* lse, const void* dout, void* dq, void* dk,
                                      void* dv, float* delta, float scale, attn_dtype_t dtype,
                                      void* workspace, size_t workspace_bytes,
                                      uint64_t wait_timeout_ns, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_68_ATTN_CROSS_H_ */
