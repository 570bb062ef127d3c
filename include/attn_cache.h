/*
 * attn_cache.h — C ABI of the 8-bit key/value cache and of the operators on
 * it: append, attention of new tokens over the cache, selection of pages by a
 * cheap score, and eviction by accumulated attention weight.
 *
 * These entry points extend attn.h's attention (out = softmax(scale·q·kᵀ)·v
 * with the row logsumexp) to generation: keys and values of the tokens seen so
 * far stay on the device in 8 bits, and each step's few query tokens attend
 * over them.  They come from the same shared library, return attn.h's status
 * codes, record device-side findings in the status word that
 * attn_device_status reads, validate every argument before touching CUDA,
 * enqueue on the caller's stream without synchronising, and allocate nothing
 * beyond the status words that attn_fwd also uses.  Make the first call on a
 * device before any stream capture.
 *
 * Layout.  A pool holds `pages` pages of `page` token slots (16, 32 or 64).
 * For page g, key/value head h, slot s and channel d:
 *
 *   k, v       e4m3 bytes [pages, heads, page, pitch], pitch = head_dim rounded
 *              up to a multiple of 16; channels from head_dim on are never read
 *              as values (append writes them as zero)
 *   k_scale,   fp32 [pages, heads]: the value held is code · scale.  append and
 *   v_scale    evict write powers of two from 2^-100 on; the attention takes any
 *              finite scale from 2^-100 on (less: values may count as zero)
 *   k_bounds   int8 [pages, heads, 2, pitch]: for each channel the upper, then
 *              the lower bound of the page's key codes in steps of 448/127
 *              (ceil(max·127/448), floor(min·127/448); NaN codes left out, 0 where
 *              there are no others).  An append to a page that holds tokens widens
 *              them while the scale stays, so that such a 0, or what tokens taken
 *              back since (a smaller lens) had, stays inside; where the scale
 *              grows, and in evict, they are found anew from the codes
 *
 * A power-of-two scale costs an e4m3 code no precision against any other
 * scale, and codes move to a larger power-of-two scale without a rounding
 * until they reach e4m3's subnormals.
 *
 * Sequence b holds lens[b] tokens; token j lies in page table[b, j / page],
 * slot j % page.  The last fresh[b] of them (T of them where fresh is NULL)
 * are the step's new tokens: lens already counts them when append, select and
 * fwd of the step are called, and all three take the same arrays.
 *
 * Device-side findings.  lens, fresh, table and page lists are read on the
 * device, so bad entries cannot be refused by the host.  An entry out of range
 * is never used as an address: the token, page or sequence it names is left
 * out, the rest of the call is computed, and attn_device_status reports
 * ATTN_ERR_DEVICE_CHECK (every build).  A sequence is left out when
 * fresh[b] is outside [0, T] or lens[b] outside [fresh[b], width·page].
 */
#ifndef EXACT_ATTENTION_68_ATTN_CACHE_H_
#define EXACT_ATTENTION_68_ATTN_CACHE_H_

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The most query tokens per sequence that attn_cache_fwd and
 * attn_cache_select take in one call. */
#define ATTN_CACHE_MAX_TOKENS 64

/* A pool of pages (device pointers; k, v and k_bounds 16-byte aligned, the
 * scales 4-byte). */
typedef struct {
  void* k;          /* e4m3 [pages, heads, page, pitch] */
  void* v;          /* e4m3 [pages, heads, page, pitch] */
  float* k_scale;   /* [pages, heads] */
  float* v_scale;   /* [pages, heads] */
  int8_t* k_bounds; /* [pages, heads, 2, pitch] */
  int64_t pages;    /* >= 1; pages·heads·page < 2^31 */
  int64_t heads;    /* key/value heads, 1 .. 65535 */
  int64_t head_dim; /* a multiple of 8, at most 256 */
  int64_t page;     /* token slots of a page: 16, 32 or 64 */
} attn_cache_t;

/* The sequences of a call (device pointers, 4-byte aligned). */
typedef struct {
  const int32_t* table; /* [batch, width] page numbers; entries from ceil(lens/page) on are not read */
  const int32_t* lens;  /* [batch] tokens in the cache, the new ones counted */
  const int32_t* fresh; /* [batch] new tokens of each sequence, or NULL: all T */
  int64_t batch;        /* 1 .. 65534 */
  int64_t width;        /* >= 1; width·page <= 2^30 */
} attn_cache_seqs_t;

/*
 * attn_cache_append — quantises the new tokens' keys and values into the cache.
 *
 *   k, v   device, 16-bit [batch, heads, T, head_dim] contiguous, 16-byte
 *          aligned (read); token i < fresh[b] of sequence b goes to position
 *          lens[b] - fresh[b] + i, rows from fresh[b] on are not read
 *   T      1 .. 2^30 rows per sequence
 *   dtype  ATTN_BF16 or ATTN_F16
 *
 * For each page and head touched, with a the largest finite |x| of the call's
 * tokens there: scale = 2^e, e the smallest integer >= -100 with a <= 448·2^e.
 * A page that holds earlier tokens of the sequence keeps the larger of its
 * scale and that one; where its scale grows, the earlier codes are requantised.
 * Codes are x / scale rounded to nearest even and saturated to ±448 (infinities
 * too); NaN stays NaN.  k_bounds follows as said above.  Slots behind the
 * sequence's end are left as they were.  The pages that the call writes must
 * belong to one sequence each.
 */
ATTN_API attn_status_t attn_cache_append(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                         const void* k, const void* v, int64_t T,
                                         attn_dtype_t dtype, cudaStream_t stream);

/*
 * attn_cache_fwd_workspace — bytes of workspace that attn_cache_fwd needs on
 * the current device for these sizes (0 on an argument it would refuse; 16:
 * none, workspace may be NULL).  with_mass: whether mass is passed.
 */
ATTN_API size_t attn_cache_fwd_workspace(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                         int64_t listed, int64_t q_heads, int64_t T,
                                         int with_mass);

/*
 * attn_cache_fwd — attention of the new tokens over the cache.
 *
 * Query token i of sequence b stands at position p = lens[b] - fresh[b] + i and
 * attends to the keys at positions <= p; query heads h·G .. h·G+G-1 share
 * key/value head h, G = q_heads / heads.
 *
 *   q        device, 16-bit [batch, q_heads, T, head_dim] contiguous, 16-byte aligned
 *   pages    device int32 [batch, heads, listed], or NULL: every page.  Each
 *            head reads only the pages listed for it: page indices of the
 *            sequence (columns of `table`), strictly ascending, negative
 *            entries behind the last.  Pages behind the sequence's end hold no
 *            token.  An entry not below width is left out and reported; so is
 *            one not above the entry before it or behind a negative one, and
 *            which of that list's further entries count is not specified.
 *   listed   entries per head (0 with pages = NULL)
 *   out      device, 16-bit [batch, q_heads, T, head_dim], 16-byte aligned
 *   lse      device fp32 [batch, q_heads, T]
 *   mass     device fp32 [batch, heads, width·page], or NULL: adds to position
 *            j of head h the sum over the head's queries of their attention
 *            weight on key j
 *   scale    finite, > 0
 *   workspace, workspace_bytes   device, 16-byte aligned, at least
 *            attn_cache_fwd_workspace bytes; contents need no preparation and
 *            mean nothing afterwards.  Calls that may run at the same time
 *            (other streams, graphs that share it) need a workspace each.
 *   T        1 .. ATTN_CACHE_MAX_TOKENS; q_heads a multiple of heads
 *   wait_timeout_ns  bound on each in-kernel wait (ATTN_DEFAULT_WAIT_TIMEOUT_NS)
 *
 * A query that may attend to no key gets out = 0 and lse = -inf.  One that may,
 * and has a NaN score, a score of +inf or no score but -inf, gets NaN in out and
 * lse and adds NaN to the mass of the keys it may attend to, as the formula does;
 * a NaN value code makes its channel of out NaN.
 *
 * Scores, maxima, sums and out's sums are fp32.  For the product with V the
 * weights are rounded to fp16 (half a step: 2^-11 of a weight), whatever `dtype`:
 * that is 1/8 of bf16's half step, and as much as fp16's, so that fp16 results
 * stand about a tenth further from the exact ones than with fp32 weights.  A
 * weight in mass is 2^(t - lse) of the stored lse, whose rounding adds |lse|·2^-23
 * to its relative error.  How work is cut, and the workspace, go by `width` (or
 * `listed`), not by lens, which are on the device: a table cut to the longest
 * sequence's pages saves small calls up to a half of their time.
 *
 * Rows of tokens from fresh[b] on, and sequences left out, are not written; what
 * q holds there, and slots behind a sequence's end, may be anything.  Results do
 * not depend on the order in which the GPU ran the work: every sum has a fixed
 * order.
 */
ATTN_API attn_status_t attn_cache_fwd(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                      const void* q, const int32_t* pages, int64_t listed,
                                      void* out, float* lse, float* mass, int64_t q_heads,
                                      int64_t T, float scale, attn_dtype_t dtype, void* workspace,
                                      size_t workspace_bytes, uint64_t wait_timeout_ns,
                                      cudaStream_t stream);

/*
 * attn_cache_select — the pages each sequence and key/value head should read.
 *
 * Each query row is rounded to 8 bits, qi = rint(q · (127 / a)) with a its
 * largest finite |q| (NaN as 0).  For a page, I = Σ_d max(qi_d·hi_d, qi_d·lo_d)
 * over k_bounds bounds the row's product with every key of the page; the
 * page's score is the largest (I · k_scale) · a over the head's G·fresh[b]
 * rows, two fp32 products.  I is an integer, so the score does not depend on
 * the order of summing.  The pages that hold the new tokens are always taken
 * (the latest `count` of them where they are more); the rest of `count` goes
 * to the highest scores, equal ones to the lowest page.
 *
 *   q       as for attn_cache_fwd
 *   count   >= 1 pages per head
 *   pages   device int32 [batch, heads, count]: page indices ascending, -1
 *           behind the last (all -1 for a sequence without new tokens)
 *   scores  device fp32 [batch, heads, width]: every page's score; -inf from
 *           the sequence's last page on, and for all pages of a sequence
 *           without new tokens
 */
ATTN_API attn_status_t attn_cache_select(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                         const void* q, int64_t q_heads, int64_t T,
                                         attn_dtype_t dtype, int64_t count, int32_t* pages,
                                         float* scores, cudaStream_t stream);

/* Bytes of workspace attn_cache_evict needs (0 on an argument it would refuse). */
ATTN_API size_t attn_cache_evict_workspace(const attn_cache_t* cache,
                                           const attn_cache_seqs_t* seqs, int64_t dst_width);

/*
 * attn_cache_evict — keeps the `keep` most useful tokens of each head.
 *
 * Sequence b and head h keep all tokens if lens[b] <= keep; otherwise the last
 * `recent` ones and, of the others, the keep - recent with the largest
 * mass[b, h, j] (equal ones: the lowest j; NaN counts as less than any weight).
 * They are copied in their order to positions 0, 1, ... of the pages
 * dst_table[b, :], quantised anew with scales and bounds as append makes them
 * (exact while no code becomes subnormal).  Every head keeps the same number,
 * so the sequence stays one: its table is dst_table and its length new_lens
 * from then on, and its old pages are free.
 *
 *   seqs       fresh is ignored; a sequence left out counts as empty, tokens whose
 *              table entry is out of range are moved as zeros
 *   mass       device fp32 [batch, heads, width·page] (read)
 *   dst_table  device int32 [batch, dst_width]: pages of the same pool.  The
 *              entries that are needed must differ from each other and from
 *              every page of the call's sequences; one that does not is not
 *              written and is reported.
 *   dst_width  keep <= dst_width·page <= 2^30
 *   keep       >= 1;  recent 0 .. keep
 *   kept       device int32 [batch, heads, keep]: the kept positions
 *              ascending, -1 behind the last
 *   new_lens   device int32 [batch]: min(lens, keep)
 *   mass_out   device fp32 [batch, heads, dst_width·page]: the kept tokens'
 *              weights, 0 behind the last
 *   workspace  device, 16-byte aligned, at least attn_cache_evict_workspace
 *              bytes; one per call in flight
 */
ATTN_API attn_status_t attn_cache_evict(const attn_cache_t* cache, const attn_cache_seqs_t* seqs,
                                        const float* mass, const int32_t* dst_table,
                                        int64_t dst_width, int64_t keep, int64_t recent,
                                        int32_t* kept, int32_t* new_lens, float* mass_out,
                                        void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_68_ATTN_CACHE_H_ */
