/*
 * slope_serving.h - the calls of libslope around the prefill attention of
 * slope.h, in the order a serving process makes them:
 *
 *   slope_qk_norm_rope   RMS norm of every query and key head and the rotation
 *                        by position, in one pass over the projections' output
 *   slope_attn_varlen    causal attention over prompts of different lengths,
 *                        packed one after another in the same tensors
 *   slope_kv4_write      keys and values into a paged cache, in 4 bits
 *   slope_kv4_read       and back: cached rows as bf16 or fp32, e.g. the prefix
 *                        that slope_attn_partial attends a new chunk to
 *   slope_kv4_attn       attention of each sequence's newest tokens over its
 *                        pages of that cache (a decode step); its out and lse
 *                        merge with other partials by slope_lse_merge
 *
 * The conventions of slope.h hold: device tensors as slope_tensor, statuses,
 * no allocation, no synchronisation, asynchronous on `stream`, argument errors
 * before any launch.  Host arrays are read during the call only.  All tensors
 * lie on the current device, and outputs overlap no input but where a call says
 * so.  Strides and pointers of a tensor without rows are not looked at.  The
 * kernels read device index arrays (positions, slots, block tables, lengths)
 * when they run; an index out of range there is never followed, as each call
 * says.
 */
#ifndef SLOPE_SERVING_H
#define SLOPE_SERVING_H

#include "slope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- positions */

/*
 * Rotation of a head's channels [begin, begin + dim) by position:
 *   (x_a, x_b) -> (x_a cos t - x_b sin t, x_b cos t + x_a sin t) * attention_factor,
 *   t = position * inv_freq[i], for pair i of dim / 2:
 *   interleaved == 0: (a, b) = (begin + i, begin + dim/2 + i)   (halves)
 *   interleaved != 0: (a, b) = (begin + 2i, begin + 2i + 1)
 * dim: a multiple of 16, 16 .. 192; begin: a multiple of 8.  inv_freq: host
 * array of dim / 2 finite radians per position (slope_rope_inv_freq makes the
 * usual ones).  The angle is reduced in 64-bit fixed point, so far positions
 * lose nothing: with frequencies up to 1 an angle is off by at most 2^-24 of a
 * turn at any position.
 */
typedef struct {
  int32_t begin;
  int32_t dim;
  int32_t interleaved;
  float attention_factor; /* finite; multiplies both cos and sin */
  const double* inv_freq; /* HOST array, dim / 2 entries */
} slope_rope;

typedef enum {
  SLOPE_ROPE_PLAIN = 0,  /* base^(-2i/dim)                                                         */
  SLOPE_ROPE_LINEAR = 1, /* every frequency divided by factor (position interpolation)              */
  SLOPE_ROPE_NTK = 2,    /* base * factor^(dim / (dim - 2)): the slowest divided by factor, the fastest kept */
  SLOPE_ROPE_BANDS = 3,  /* by wavelength: those that turn more than `fast` times in `original` positions kept,
                            those that turn less than `slow` times divided by factor, between them a ramp in the
                            number of turns                                                        */
  SLOPE_ROPE_YARN = 4    /* YaRN (Peng et al. 2023): the ramp runs over the channel index between the indices that
                            turn `fast` and `slow` times, rounded outwards; attention factor 0.1 ln(factor) + 1   */
} slope_rope_scaling;

/*
 * Host only: fills inv_freq[0 .. dim/2) and *attention_factor (1 but for
 * YARN; may be NULL).  dim even, 4 .. 512 (YARN and NTK need dim > 2), base > 1;
 * but for PLAIN factor >= 1; for BANDS and YARN original > 0 and fast > slow > 0
 * (commonly 4 and 1, or 32 and 1).  Else SLOPE_ERR_SHAPE; an unknown scaling
 * SLOPE_ERR_UNSUPPORTED.
 */
SLOPE_API slope_status slope_rope_inv_freq(int32_t dim, double base, slope_rope_scaling scaling, double factor,
                                           double original, double fast, double slow, double* inv_freq,
                                           double* attention_factor);

/*
 * One pass over queries and keys, each head of each token:
 *   y = x / sqrt(mean(x^2) + eps) * weight     (if norm != 0; a NULL weight is 1)
 *   y's channels [begin, begin + dim) rotated   (if rope != NULL)
 * in fp32, rounded once to the output's type.
 *
 *   q [T, Hq, d], k [T, Hkv, d], each bf16 or fp32 (k may be NULL, with k_out:
 *     queries alone; or q NULL, with q_out); d in {64, 128, 192}.
 *   q_weight, k_weight: fp32 or bf16, rank 2: [1, d] for every head or [H, d]; or
 *     NULL.  They need norm != 0 (else SLOPE_ERR_UNSUPPORTED).
 *   positions: device int32 [T], any values; NULL: pos0 + row, which then has to
 *     lie in [-2^31, 2^31).
 *   q_out, k_out: bf16 or fp32, the shape of q and k.  An output may be its own
 *     input (same pointer, type and strides); it may not overlap the inputs in
 *     any other way.
 * Innermost strides 1, other strides multiples of 8 elements, pointers 16-byte
 * aligned.  T == 0 is a no-op.
 */
SLOPE_API slope_status slope_qk_norm_rope(const slope_tensor* q, const slope_tensor* k, const slope_tensor* q_weight,
                                          const slope_tensor* k_weight, int norm, float eps, const slope_rope* rope,
                                          const int32_t* positions, int64_t pos0, slope_tensor* q_out,
                                          slope_tensor* k_out, void* stream);

/* ---------------------------------------------------------------- packed prompts */

/*
 * Attention over n_seqs prompts packed in one set of tensors: sequence s is
 * rows [cu_seqlens[s], cu_seqlens[s+1]), and a query sees keys of its own
 * sequence only, under the masks of slope.h (causal, window).
 *
 *   q bf16 [T, Hq, dqk], k bf16 [T, Hkv, dqk], v bf16 [T, Hkv, dv]: as for
 *     slope_attn_partial, T < 2^28.
 *   cu_seqlens: HOST array of n_seqs + 1 row indices, not descending,
 *     0 <= cu_seqlens[0], cu_seqlens[n_seqs] <= T (else SLOPE_ERR_LAYOUT).  A
 *     sequence may be empty.
 *   out bf16 or fp32 [T, Hq, dv], lse fp32 [Hq, T]: as for slope_attn_partial.
 * Rows outside [cu_seqlens[0], cu_seqlens[n_seqs]) are neither read into any
 * result nor written: whatever k and v hold there, or in another sequence, NaN
 * too, does not reach a sequence's rows.  Within a sequence a key or value that
 * is not finite may also make rows NaN that the causal mask or the window keeps
 * from it, where a 128-key tile holds both.
 * Sequences share a launch up to 128 of them, the longest first.  At dqk >= 128 a
 * launch takes one of the SLOPE_TILE_COUNTERS, as those of slope_attn_partial do.
 */
SLOPE_API slope_status slope_attn_varlen(const slope_tensor* q, const slope_tensor* k, const slope_tensor* v,
                                         const int64_t* cu_seqlens, int64_t n_seqs, int causal, int64_t window,
                                         float scale, slope_tensor* out, slope_tensor* lse, void* stream);

/* ---------------------------------------------------------------- a paged cache in 4 bits */

/*
 * The cache of one layer: n_pages pages of page_size tokens, each with Hkv key
 * heads of dqk and value heads of dv channels.
 *
 * Groups of 32 consecutive channels of a token's head share two bf16 numbers:
 *   min   = bf16(smallest channel), scale = bf16(fp32(largest - min) * fp32(1/15))
 *           (round to nearest even; a scale below 2^-126 is 0)
 *   code  = (x - min) / scale in fp64, rounded to the nearest integer, halves to
 *           even, and clamped to 0 .. 15 (0 where scale is 0)
 *   value = fma(scale, code, min) in fp32: what the cache holds.
 * A group with a NaN or an infinity, or whose range overflows fp32, has a NaN
 * min and a zero scale: it reads back as NaN.
 *
 * data: [n_pages][Hkv][page_size / 16] blocks, a block being 16 tokens of one
 * head: slope_kv4_block_bytes(dqk, dv) =
 *   16 * dqk / 2 key codes, 16 * dv / 2 value codes, then for each token
 *   dqk/32 + dv/32 words (scale << 16 | min, key groups first).
 * Codes lie in the order the attention's tensor-core operands take them.  With
 * a lane (g, q), 0 <= g < 8, 0 <= q < 4, owning 16 bytes at (chunk * 32 + 4g + q) * 16
 * of its region, and a 32-bit word holding 8 codes, the first in the low bits:
 *   key of token t, channel c: g = t % 8, q = c % 32 / 8, code c % 8 of the lane's
 *     word number t / 8 * (dqk / 32) + c / 32 (four words to a chunk);
 *   value of token t, channel c: g = c % 32 / 4, q = t % 8 / 2, chunk c / 64, word
 *     t % 2 + 2 * (t / 8), code c % 4 + 4 * (c % 64 / 32).
 *
 * dqk in {64, 128, 192}, dv in {64, 128} (else SLOPE_ERR_UNSUPPORTED); page_size a
 * power of two, 16 .. 1024; n_pages * page_size < 2^31; Hkv <= 65535 (else
 * SLOPE_ERR_SHAPE).  data is 16-byte aligned (else SLOPE_ERR_STRIDE).
 */
typedef struct {
  void* data;
  int64_t n_pages;
  int32_t page_size;
  int32_t Hkv;
  int32_t dqk;
  int32_t dv;
} slope_kv4_cache;

/* Bytes of one 16-token block of one head, and of the whole cache's data (0 for sizes that are not supported). */
SLOPE_API size_t slope_kv4_block_bytes(int32_t dqk, int32_t dv);
SLOPE_API size_t slope_kv4_cache_bytes(int64_t n_pages, int32_t page_size, int32_t Hkv, int32_t dqk, int32_t dv);

/*
 * Writes T tokens into the cache: token t goes to slot slots[t] = page *
 * page_size + index in the page.
 *   k [T, Hkv, dqk], v [T, Hkv, dv]: bf16 or fp32, both the same; innermost
 *     stride 1, other strides multiples of 8 elements, 16-byte aligned.
 *   slots: device int32 [T].  A token whose slot is negative or not below
 *     n_pages * page_size is skipped.  The other slots of one call have to differ
 *     from one another; a slot that occurs twice may hold a mix of its tokens.
 * Other slots keep what they hold.  T == 0 is a no-op.
 */
SLOPE_API slope_status slope_kv4_write(const slope_kv4_cache* cache, const slope_tensor* k, const slope_tensor* v,
                                       const int32_t* slots, void* stream);

/*
 * Reads T tokens of the cache back: row t of k [T, Hkv, dqk] and v [T, Hkv, dv]
 * (bf16 or fp32, both the same; strides as for slope_kv4_write) gets the values
 * of slot slots[t], rounded to the output's type.  Rows whose slot is out of
 * range are left as they were.  Slots may repeat.  T == 0 is a no-op.
 */
SLOPE_API slope_status slope_kv4_read(const slope_kv4_cache* cache, const int32_t* slots, slope_tensor* k,
                                      slope_tensor* v, void* stream);

/*
 * Attention of the newest q_len tokens of each of B sequences over the cache.
 *
 *   q bf16 [B * q_len, Hq, dqk]: row b * q_len + i is token i of sequence b.  It
 *     has position kv_lens[b] - q_len + i and sees the keys of its sequence at
 *     positions <= its own and, with window > 0, more than its own - window.
 *     Hq a multiple of the cache's Hkv; innermost stride 1, other strides
 *     multiples of 8 elements, 16-byte aligned.
 *   q_len: 1 .. SLOPE_KV4_MAX_Q_LEN (a longer run: read the prefix back with
 *     slope_kv4_read and use slope_attn_partial).
 *   block_table: device int32 [B, max_pages], row b's page p holds positions
 *     [p * page_size, (p+1) * page_size) of sequence b; rows lie table_stride
 *     elements apart.  Entries that no visible key needs are not used.  A page
 *     outside [0, n_pages) holds no keys.
 *   kv_lens: device int32 [B], tokens of each sequence in the cache, the newest
 *     q_len included; taken as 0 if negative and as max_pages * page_size at most.
 *   window, scale: as in slope.h (max_pages * page_size < 2^28).
 *   out bf16 or fp32 [B * q_len, Hq, dv]; lse fp32 [Hq, B * q_len] or NULL: as for
 *     slope_attn_partial; a row that sees no key gets 0 and -inf.
 *   workspace: device buffer of slope_kv4_attn_workspace_size() bytes, 256-byte
 *     aligned; it needs no initial contents.  Calls that may overlap on the GPU
 *     need one each, captured graphs that may be replayed at the same time too.
 * B == 0 is a no-op.  B <= 65535.
 *
 * Cached values are exact in the products; the softmax weights, times a group's
 * scale, are rounded to bf16 on their way into the tensor cores (as the weights
 * of slope_attn_partial are), which moves the output by at most 2^-8 of the
 * weighted mean of scale * |code - 8|; sums run in fp32.  Value scales have to lie below
 * 2^51 or the output overflows; contributions below about 2^-57 times the
 * weight are lost.  A query row's channels keep their bits down to 2^-26 of the
 * row's largest, which has to be below 2^117 (else the row is NaN); scaled scores
 * have to stay below 2^29 in magnitude, where fp32 no longer tells weights apart.
 */
#define SLOPE_KV4_MAX_Q_LEN 64
SLOPE_API slope_status slope_kv4_attn(const slope_tensor* q, const slope_kv4_cache* cache, const int32_t* block_table,
                                      int64_t table_stride, int64_t max_pages, const int32_t* kv_lens, int32_t q_len,
                                      int64_t window, float scale, slope_tensor* out, slope_tensor* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes slope_kv4_attn needs on the current device (0 for arguments it does not support). */
SLOPE_API size_t slope_kv4_attn_workspace_size(int64_t B, int64_t Hq, const slope_kv4_cache* cache, int32_t q_len);

#ifdef __cplusplus
}
#endif

#endif /* SLOPE_SERVING_H */
