/*
 * slope_kv.h - a paged key/value cache in 16 bits and what a serving process
 * does with it:
 *
 *   slope_kv_write         keys and values of new tokens into the cache's pages
 *   slope_kv_attn          attention of each sequence's newest tokens over its
 *                          pages: one token each (a decode step), a chunk of a
 *                          prompt, or both in one call
 *   slope_kv_attn_weights  the attention weight that each cached token got from
 *                          those queries, summed over the rows and heads
 *   slope_kv_evict         keeps, of each sequence and head, the tokens with
 *                          the largest weights and moves them together
 *
 * The conventions of slope.h and slope_serving.h hold: device tensors as
 * slope_tensor, statuses, no allocation, no synchronisation, asynchronous on
 * `stream`, argument errors before any launch.  All tensors lie on the current
 * device, and outputs overlap no input but where a call says so.  Strides and
 * pointers of a tensor without rows are not looked at.  The kernels read device
 * index arrays (slots, block tables, lengths, row indices) when they run, so a
 * captured call follows them; an index out of range there is never followed,
 * as each call says.
 */
#ifndef SLOPE_KV_H
#define SLOPE_KV_H

#include "slope.h"

/* Launches of slope_kv_attn and slope_kv_attn_weights that may be queued at a time, and as many recorded into graphs. */
#define SLOPE_KV_COUNTERS 65536

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The cache of one layer: n_pages pages of page_size tokens, each with Hkv key
 * heads of dqk and value heads of dv bf16 channels.  The row of token t, head h
 * of page p starts at
 *   k + p * k_stride[0] + h * k_stride[1] + t * k_stride[2]   (elements; v alike),
 * so pages may be head-major, token-major, or slices of one buffer.
 *
 * dqk in {64, 128, 192}, dv in {64, 128} (else SLOPE_ERR_UNSUPPORTED); page_size a
 * power of two, 16 .. 1024; n_pages >= 1, n_pages * page_size < 2^31; Hkv <= 65535
 * (else SLOPE_ERR_SHAPE).  k and v are 16-byte aligned, strides positive
 * multiples of 8 elements below 2^39 (else SLOPE_ERR_STRIDE).
 */
typedef struct {
  void* k;
  void* v;
  int64_t n_pages;
  int32_t page_size;
  int32_t Hkv;
  int32_t dqk;
  int32_t dv;
  int64_t k_stride[3]; /* page, head, token */
  int64_t v_stride[3];
} slope_kv_cache;

/*
 * Which rows of q are whose, and where a sequence's keys are; for
 * slope_kv_attn and slope_kv_attn_weights.
 *
 *   B: sequences, at most 65535.
 *   cu_q: device int32 [B + 1], or NULL.  The newest tokens of sequence b are rows
 *     [cu_q[b], cu_q[b+1]) of q; bounds are taken as 0 and T at least and at
 *     most, and a range that ends before it starts as empty.  Ranges must not
 *     overlap.  Rows in no range are left as they were.
 *   q_len: without cu_q, the new tokens of every sequence, rows b * q_len on.
 *   kv_lens: device int32 [B], tokens of each sequence in the cache, the new ones
 *     included; taken as 0 if negative and as max_pages * page_size at most.
 *     Token i of n new ones has position kv_lens[b] - n + i and sees the
 *     keys at positions <= its own and, with window > 0, more than its own - window.
 *   block_table: device int32 [B, max_pages], row b's page p holds positions
 *     [p * page_size, (p+1) * page_size) of sequence b; rows lie table_stride
 *     elements apart.  Entries that no visible key needs are not used.  A page
 *     outside [0, n_pages) holds no keys.  max_pages * page_size < 2^28.
 */
typedef struct {
  int64_t B;
  const int32_t* cu_q;
  int32_t q_len;
  const int32_t* kv_lens;
  const int32_t* block_table;
  int64_t table_stride;
  int64_t max_pages;
} slope_kv_batch;

/*
 * Writes T tokens into the cache: token t goes to slot slots[t] = page *
 * page_size + index in the page.
 *   k [T, Hkv, dqk], v [T, Hkv, dv]: bf16 or fp32 (rounded to nearest even), both
 *     the same; innermost stride 1, other strides multiples of 8 elements, 16-byte
 *     aligned.
 *   slots: device int32 [T].  A token whose slot is negative or not below
 *     n_pages * page_size is skipped.  The other slots of one call have to differ
 *     from one another; a slot that occurs twice may hold a mix of its tokens.
 *   weights: NULL, or fp32 [n_pages, Hkv, page_size] (innermost stride 1): the
 *     accumulated weights of the slots written become 0.
 * Other slots keep what they hold.  T == 0 is a no-op.
 */
SLOPE_API slope_status slope_kv_write(const slope_kv_cache* cache, const slope_tensor* k, const slope_tensor* v,
                                      const int32_t* slots, slope_tensor* weights, void* stream);

/*
 * Attention of each sequence's newest tokens over its pages.
 *
 *   q bf16 [T, Hq, dqk], T < 2^28, Hq a multiple of the cache's Hkv: innermost
 *     stride 1, other strides positive multiples of 8 elements, 16-byte aligned.
 *   window, scale: as in slope.h.
 *   out bf16 or fp32 [T, Hq, dv]; lse fp32 [Hq, T] or NULL: as for
 *     slope_attn_partial (out 16-byte aligned, its strides multiples of 16
 *     bytes); a row that sees no key gets 0 and -inf, and so does one all of whose visible
 *     scores are -inf (where a softmax would be 0 / 0).
 *   workspace: device buffer of slope_kv_attn_workspace_size() bytes, 256-byte
 *     aligned; it needs no initial contents.  Calls that may overlap on the GPU
 *     need one each, captured graphs that may be replayed at the same time too.
 * B == 0 or T == 0 is a no-op.
 *
 * A launch takes a counter out of SLOPE_KV_COUNTERS on the device, another for every
 * 512 sequences after the first: keep fewer launches queued or running at a time.
 * Launches recorded into a graph take theirs out of as many others and keep them until
 * the graph and the executable graphs made of it (or updated with it) are destroyed, so
 * replays of one recording must not overlap; other calls may run beside them.  Where that
 * many are recorded in graphs that exist, a further one returns SLOPE_ERR_CUDA.
 * Softmax weights are rounded to bf16 on their way into the tensor cores; scores,
 * maxima, sums and outputs stay in fp32 until the output's rounding.  Whatever the
 * cache holds behind a sequence's last token, NaN too, reaches no row.  Among a
 * sequence's tokens a value that is not finite may also make rows NaN that the causal
 * mask or the window keeps from it, where 128 consecutive positions hold both.
 * Results do not depend on how the work was dealt to the GPU's CTAs in time: the same
 * call gives the same bits.
 */
SLOPE_API slope_status slope_kv_attn(const slope_tensor* q, const slope_kv_cache* cache, const slope_kv_batch* batch,
                                     int64_t window, float scale, slope_tensor* out, slope_tensor* lse,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes slope_kv_attn needs for T rows: of a batch without cu_q, with its q_len; of one with cu_q, whose ranges only
 * the device knows, with q_len = 0 (a workspace sized for a q_len is refused there).  0 for arguments it does not support.
 */
SLOPE_API size_t slope_kv_attn_workspace_size(int64_t T, int64_t Hq, const slope_kv_cache* cache, int32_t q_len);

/*
 * The attention weights of the cached tokens: for sequence b, key head g and token j
 *   w = sum over the query heads h of g and the new tokens i of b that see j of
 *       exp(scale * q_ih . k_jg - lse[h][i]),
 * with lse as slope_kv_attn gives it.  A row whose lse is -inf adds nothing, whatever it holds.
 *
 *   q, window, scale: as for slope_kv_attn, which rows are whose too; q may be
 *     the last rows of a chunk only.
 *   lse fp32 [Hq, T], positive strides.
 *   weights fp32 [n_pages, Hkv, page_size], innermost stride 1: the number of token
 *     j is in its page's place.  accumulate != 0 adds w to what is there (where w is 0
 *     nothing is written), else w replaces it; in both cases for positions below
 *     kv_lens[b] whose page is in range, and nowhere else.  No place of weights may
 *     be written twice in one call: not for two sequences that share a page, nor for
 *     two positions of one.
 *   workspace: slope_kv_attn_weights_workspace_size() bytes, as for slope_kv_attn.
 * B == 0 is a no-op, T == 0 a call whose sums are all 0.
 * Sums run in fp32 in an order that depends on the call's sizes and lengths alone.  A key that is not
 * finite may get a NaN whatever its scores; no other key's weight does by it.
 */
SLOPE_API slope_status slope_kv_attn_weights(const slope_tensor* q, const slope_kv_cache* cache,
                                             const slope_kv_batch* batch, const slope_tensor* lse, int64_t window,
                                             float scale, int accumulate, slope_tensor* weights, void* workspace,
                                             size_t workspace_bytes, void* stream);

SLOPE_API size_t slope_kv_attn_weights_workspace_size(int64_t T, int64_t Hq, const slope_kv_cache* cache,
                                                      int32_t q_len);

/*
 * Keeps `keep` tokens of each sequence and head, and moves them together.
 *
 * A sequence of n <= keep tokens keeps all of them.  Of a longer one each key head
 * keeps the first `first` tokens, the last `recent`, and of those between the
 * keep - first - recent with the largest weights; of equal weights the one at the lower
 * position; a NaN is below every number, and -0 equals 0.  The kept tokens go, in
 * order, to positions 0, 1, ... of the same head: key row, value row and weight.
 * Heads keep different tokens and the same number of them.
 *
 *   weights fp32 [n_pages, Hkv, page_size]: as for slope_kv_attn_weights.
 *   block_table, table_stride, max_pages, kv_lens, B: as in slope_kv_batch.  A
 *     position whose page is out of range counts as a weight below NaN; nothing is
 *     read or written there.  first and recent are kept whatever their pages.
 *   keep >= 1, first >= 0, recent >= 0, first + recent <= keep (else SLOPE_ERR_SHAPE).
 *   out_table: NULL, and the tokens move within their own pages; positions keep and
 *     after keep what they hold.  Or device int32 [B, out_pages], out_pages * page_size
 *     >= min(keep, max_pages * page_size) (else SLOPE_ERR_SHAPE), rows out_stride elements
 *     apart: the tokens are copied to the positions of these pages of the same cache,
 *     and the old ones keep what they hold.
 *     In both forms a page that one sequence's tokens go to may be no other page of the call: a
 *     prefix that sequences share is copied by each into pages of its own, not moved in place.
 *   kept: device int32 [B, Hkv, keep], dense: the old positions of the tokens kept, in order; -1 after them.
 *   out_lens: device int32 [B]: min(n, keep).  May be kv_lens itself.
 *   workspace: slope_kv_evict_workspace_size() bytes, 256-byte aligned, no initial contents, one for each
 *     call that may overlap.
 * B == 0 is a no-op.
 */
SLOPE_API slope_status slope_kv_evict(const slope_kv_cache* cache, slope_tensor* weights, int64_t B,
                                      const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                      const int32_t* kv_lens, int64_t keep, int64_t first, int64_t recent,
                                      const int32_t* out_table, int64_t out_stride, int64_t out_pages, int32_t* kept,
                                      int32_t* out_lens, void* workspace, size_t workspace_bytes, void* stream);

SLOPE_API size_t slope_kv_evict_workspace_size(int64_t B, int64_t Hkv, int64_t keep);

#ifdef __cplusplus
}
#endif

#endif /* SLOPE_KV_H */
