/*
 * attn.h -- C ABI of the attention step of a decode over a paged cache, for
 * GB300 (sm_103a).  Same library, same conventions as moe.h: device pointers
 * owned by the caller, no state and no allocation, `stream` a cudaStream_t as
 * void*, a moe_status as the return value, device-side errors OR-ed into the
 * optional word `dev_status`.  Calls launch on the current device, which has to
 * be the one that the pointers and the stream belong to.
 *
 * The step sits between a layer's q/k/v projections and its routed-MoE part,
 * for sequences that each have some tokens in flight: one (plain decode), a
 * chain, or a tree of drafted tokens that is verified at once.
 *   attn_qk_norm_rope   normalises and rotates q and k, appends k and v
 *   attn_tree_decode    attends from the tokens in flight to the cache
 *   attn_cache_weights  adds up the softmax weight each cached slot received
 *   attn_cache_evict    keeps the slots with the most weight
 *
 * Sequences.  `lens` [batch]: committed slots of each sequence in the cache.
 * `cu` [batch + 1]: tokens cu[b] .. cu[b + 1] - 1 of the packed token arrays
 * are sequence b's tokens in flight (there may be none); cu[0] = 0, ascending,
 * cu[batch] = tokens.  Token i of sequence b belongs in slot lens[b] + i.
 * Both are device arrays.  Where they do not fit together or the cache's
 * capacity (max_pages * page_size slots), the call sets ATTN_DEV_BAD_LENGTH,
 * writes NaN to its floating outputs (at least to those of the tokens or
 * sequences concerned) and neither reads nor writes their part of the cache.
 *
 * Heads.  q_heads = G * kv_heads; query head h reads KV head h / G.  Attention
 * and weights take up to 2^31 - 2049 rows (tokens x G) in a call.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of q, k, v and the cache (all of one type in a call). */
enum { ATTN_BF16 = 0, ATTN_FP16 = 1 };

/* Bits of the device status word, beside MOE_DEV_TIMEOUT (a wait of
 * attn_tree_decode or attn_cache_weights has run out: their outputs are NaN
 * where that wait was for them). */
enum {
  ATTN_DEV_BAD_PAGE = 32,  /* a page number outside [0, pages) */
  ATTN_DEV_BAD_LENGTH = 64 /* lens or cu out of range */
};

/* A paged cache of keys and values.  Slot s of sequence b lies in page
 * page_table[b * max_pages + s / page_size], row s % page_size.  The D
 * elements of a row are contiguous; pages, heads and rows may be strided in
 * any way (strides in elements, the same for k and v), for instance
 * [pages, kv_heads, page_size, D] or [pages, page_size, kv_heads, D].  A
 * cache without paging is one page per sequence.  Page numbers of slots past
 * a sequence's end are not read.  A page that is written belongs to one
 * sequence: attn_qk_norm_rope writes the tokens' slots, and attn_cache_evict any
 * slot below the budget, in place.  Pages that sequences share (a common prefix)
 * are for calls that only read, attn_tree_decode and attn_cache_weights.
 * Supported: head_dim a multiple of 8 from 16 to 256; page_size a multiple of
 * 8 up to 2^20; strides multiples of 8 and at least head_dim; k and v 16-B
 * aligned; max_pages * page_size < 2^31 - 2048. */
typedef struct {
  void* k;
  void* v;
  long long page_stride, head_stride, row_stride;
  const int32_t* page_table; /* device, [batch x max_pages] */
  int32_t batch, max_pages;
  int32_t pages, page_size, kv_heads, head_dim;
  int32_t dtype; /* ATTN_BF16 or ATTN_FP16 */
} attn_cache;

/* Head norm, position rotation and append, in one pass over q, k and v.
 * q [tokens x q_heads x D], k, v [tokens x kv_heads x D]: heads and elements
 * contiguous, q_stride / k_stride / v_stride elements from token to token (so
 * views of one packed projection work); 16-B aligned, strides multiples of 8.
 * For each head of q and k, in FP32:
 *   y = x / sqrt(mean(x^2) + eps) * weight   (q_weight, k_weight [D] of the
 *       cache's type; both NULL: no norm, y = x)
 *   the first `rot` channels (even, 0 <= rot <= D) turn by
 *   theta_j = pos[t] * inv_freq[j], j < rot / 2: the pair (a, c) becomes
 *   magnitude * (a cos - c sin, a sin + c cos); the pair is channels
 *   (j, j + rot/2), or (2j, 2j + 1) if `interleaved`.
 * then one rounding.  inv_freq [rot / 2] is FP64 on the device and theta is
 * reduced to one turn in 64-bit fixed point: the angle is off by less than
 * (|pos| * inv_freq * 2^-54 + 2^-26) turns before its sine is taken (inv_freq
 * below 2^-9: |pos| * 2^-63 + 2^-26).  The first term is what FP64 makes of
 * inv_freq / 2 pi, the second is FP32's of the reduced angle.  Scaled
 * rotations (interpolated, stretched per frequency) are a choice of inv_freq
 * and magnitude.
 * q_out [tokens x q_heads x D] contiguous; may be q itself if q is contiguous.
 * k and v (v as it is) go to the tokens' slots of the cache.
 * slot_pos [batch x kv_heads x slot_cap] int32 or NULL: pos[t] is also
 * written to the token's slot of each head, for attn_cache_evict.
 * A bad page skips that token's append and sets ATTN_DEV_BAD_PAGE; so does a
 * slot that slot_cap does not hold, with ATTN_DEV_BAD_LENGTH. */
int attn_qk_norm_rope(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                      long long v_stride, const int32_t* pos, const int32_t* cu, const int32_t* lens, int tokens,
                      int q_heads, const void* q_weight, const void* k_weight, double eps, const double* inv_freq,
                      int rot, int interleaved, double magnitude, void* q_out, int32_t* slot_pos, int slot_cap,
                      const attn_cache* cache, int32_t* dev_status, void* stream);

/* Workspace bytes of attn_tree_decode on the current device; 0 for a cache
 * that is not supported.  It needs no initial value and may be shared by
 * calls of one stream. */
size_t attn_tree_decode_workspace(const attn_cache* cache);

/* Attention of the tokens in flight over the cache, which holds their own
 * keys and values already (attn_qk_norm_rope).  Token i of a sequence sees
 * its lens[b] committed slots and, of the tokens in flight, those whose bit
 * is set in its row of `tree`: bit j % 64 of word tree[t * tree_words + j /
 * 64] for draft j (bits past the sequence's tokens are ignored, missing words
 * are 0; there is at least one).  tree = NULL, tree_words = 0: a chain, token i
 * sees drafts 0 .. i.
 *   s_j = scale * <q, k_j>,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
 * with FP32 accumulation (1e-30 <= |scale| <= 1e30); the weights are rounded once to the cache's type
 * as operands of the second product (the sum behind lse is of the unrounded
 * ones; a weight below 2^-35 of the row's largest, or 2^-126 in BF16, may
 * become 0, and an infinite value that it meets NaN).  A token that sees nothing gets out = 0 and lse = -inf.  What a token
 * does not see has no influence on it, NaN and infinities included.
 * q [tokens x q_heads x D]: q_stride elements from token to token; out and
 * lse [tokens x q_heads] contiguous.  lse may be NULL.
 * A bad page sets ATTN_DEV_BAD_PAGE and makes the outputs of its sequence and
 * KV heads NaN.  Results are bit-identical between repeated calls. */
int attn_tree_decode(const void* q, long long q_stride, const int32_t* cu, const int32_t* lens, int tokens,
                     int q_heads, const uint64_t* tree, int tree_words, double scale, const attn_cache* cache,
                     void* out, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream);

/* The softmax weight every slot received in that step, per KV head:
 *   acc_out[b, h, j] = decay * (j < lens[b] ? acc[b, h, j] : 0)
 *                      + sum over tokens i that see j and query heads of h of exp(s_ij - lse_i)
 * for j < lens[b] + tokens in flight; later entries of acc_out are not
 * written.  q, tree and scale as for attn_tree_decode, lse as it wrote it
 * (a row with lse = -inf adds nothing, whatever its q holds; a score of -inf adds
 * 0 as any other weight of 0).  acc, acc_out [batch x kv_heads x
 * slot_cap] FP32, may be the same array.  A score's FP32 sum is cut off, not
 * rounded, by the tensor core: a weight is off by some 2^-24 times the
 * score's size, 2e-6 of the weight for scores of 40.  The sum runs over rows in
 * a fixed order: results are bit-identical between repeated calls.
 * Slots on a bad page become NaN with ATTN_DEV_BAD_PAGE. */
int attn_cache_weights(const void* q, long long q_stride, const float* lse, const int32_t* cu, const int32_t* lens,
                       int tokens, int q_heads, const uint64_t* tree, int tree_words, double scale,
                       const attn_cache* cache, const float* acc, double decay, float* acc_out, int slot_cap,
                       int32_t* dev_status, void* stream);

/* Workspace bytes of attn_cache_evict for a budget of slots.  It needs no
 * initial value and may be shared by calls of one stream. */
size_t attn_cache_evict_workspace(const attn_cache* cache, int budget);

/* Shrinks every sequence with more than `budget` slots to `budget`, for each
 * KV head on its own.  Slots are ranked: protected ones first (slot_pos <
 * sinks or slot_pos >= next_pos[b] - recent), then the larger acc (NaN counts as the
 * least), then the lower slot; the first `budget` stay (of more protected
 * slots than that, those with the larger acc).  Attention over keys
 * that are rotated already does not depend on their order, so nothing is
 * shifted: the kept slots from `budget` on move, in order, into the dropped
 * slots below `budget`, in order.  Only those rows of k and v are copied.
 * acc, slot_pos [batch x kv_heads x slot_cap] in; acc_out, slot_pos_out the
 * same for the first lens_out[b] slots (later entries are not written);
 * lens_out [batch] = min(lens, budget).  No output may be an input array.
 * next_pos [batch]: the position the sequence's next token will have.
 * A sequence of which a needed page is bad loses the rows concerned
 * (ATTN_DEV_BAD_PAGE): they are not copied, and their acc_out is NaN. */
int attn_cache_evict(const attn_cache* cache, const float* acc, const int32_t* slot_pos, int slot_cap,
                     const int32_t* lens, const int32_t* next_pos, int budget, int sinks, int recent, float* acc_out,
                     int32_t* slot_pos_out, int32_t* lens_out, void* workspace, size_t ws_bytes, int32_t* dev_status,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
