/*
 * attention.h - C ABI of attention over a paged cache of keys and values (gfx950).
 *
 * The full-attention layers that stand between the Gated DeltaNet layers of a
 * hybrid stack (a quarter of them: linlog.top article, section "Four core
 * designs", design 4).  Two entry points:
 *
 *   attn_append   norms of the query and key heads and the position rotation,
 *                 q to its own tensor, k and v into the cache; one pass
 *   attn_forward  attention of the new tokens over everything cached: single
 *                 tokens, prompts, trees of drafted tokens
 *
 * Sequences.  B sequences bring new tokens, packed one after the other: rows
 * [cu[b], cu[b + 1]) of the N rows of q, k, v and out are sequence b's, and
 * lens[b] is its number of tokens with the new ones.  New token i of the n of
 * sequence b is number lens[b] - n + i of the sequence.  A sequence may bring
 * no token.  Rows in front of cu[0] and from cu[B] on belong to no sequence:
 * outputs are left as they were there.
 *
 * Cache.  pages [n_pages][2][n_kv_heads][page_size][head_dim], the keys of a
 * page, then its values.  Number t of sequence b lies at t % page_size in page
 * table[b * max_pages + t / page_size].  Sequences may share pages that none
 * of them appends to.  A page number outside [0, n_pages) holds nothing: its
 * tokens are not appended and not seen.  cu, lens and table are read on the
 * device, so a captured graph takes their values at replay; whatever they
 * hold, no access leaves the buffers that the arguments describe.
 *
 * Conventions as in moe_layer.h: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked before anything is enqueued,
 * MOE_OK or a negative MOE_E* code with the reason in moe_last_error(),
 * deterministic results.
 */
#ifndef ATTENTION_H
#define ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ROTARY_HALF 0      /* pairs (i, i + rotary_dim / 2) */
#define ATTN_ROTARY_ADJACENT 1  /* pairs (2 i, 2 i + 1)          */

typedef struct attn_desc {
  int32_t n_q_heads;    /* a multiple of n_kv_heads, at most 256                        */
  int32_t n_kv_heads;   /* >= 1; query head h reads key head h / (n_q / n_kv)           */
  int32_t head_dim;     /* 64, 128 or 256                                               */
  int32_t dtype;        /* q, k, v, out and the cache: MOE_F32 or MOE_BF16              */
  int32_t page_size;    /* tokens a page: a power of two in [1, 1024]                   */
  int32_t max_pages;    /* row length of the page table, >= 1                           */
  int32_t rotary_dim;   /* values of a head that are rotated: even, in [0, head_dim]    */
  int32_t rotary_pairs; /* ATTN_ROTARY_HALF or ATTN_ROTARY_ADJACENT                     */
  int64_t n_pages;      /* pages of the cache, >= 1                                     */
  float scale;          /* factor on q . k (finite)                                     */
  float eps;            /* added under the square root of the norms (>= 0)              */
  float norm_offset;    /* added to the norms' weights (finite): 0, or 1 where they are held less one */
} attn_desc;

/*
 * Norms, rotation and append of N rows.  For each head x of q and of k:
 *   x <- x / sqrt(mean x^2 + eps) * (norm_offset + w)      with w = q_norm or k_norm; NULL: x stays
 *   (x_a, x_b) <- (x_a cos - x_b sin, x_b cos + x_a sin)   for the pairs of the first rotary_dim values,
 *                                                          angle positions[row] * inv_freq[pair]
 * rounded once to dtype; the angle is formed in double precision, so far
 * positions lose nothing.  v is copied.
 *   positions  [N] int32 (not the number in the sequence: drafted tokens of one depth share theirs)
 *   q          row t at q + t * q_stride elements: [n_q_heads][head_dim]; NULL (with q_out): k and v only
 *   k, v       likewise with [n_kv_heads][head_dim]
 *   q_norm, k_norm [head_dim] fp32 or NULL;  inv_freq [rotary_dim / 2] fp32 (NULL where rotary_dim is 0,
 *                                            and positions may be NULL then)
 *   q_out      [N][n_q_heads][head_dim]
 * q, k, v, q_out and pages are 16-byte aligned, strides multiples of 16 bytes.
 * Two new tokens of one place (a page twice in the table) leave one of the two.
 * B = 0 or N = 0 enqueues nothing.  B <= 2^16, N <= 2^20.  Errors: MOE_EINVAL
 * (descriptor, sizes, strides, NULL or misaligned pointers, an output that
 * overlaps another argument), MOE_EHIP if the launch fails.
 */
int attn_append(const attn_desc* d, int32_t B, int32_t N, const int32_t* cu, const int32_t* lens, const int32_t* table,
                const int32_t* positions, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, const float* q_norm, const float* k_norm, const float* inv_freq,
                void* q_out, void* pages, void* stream);

/* Bytes of workspace that attn_forward needs for these sizes (0 where it needs
 * none), or (size_t)-1 for arguments that it would refuse. */
size_t attn_workspace_bytes(const attn_desc* d, int32_t B, int32_t N, int32_t new_max, int32_t len_max);

/*
 * Attention of the new tokens over the cache, which holds theirs too:
 *   out = sum_j softmax_j(scale q . k_j) v_j
 * over the lens[b] - n tokens before the new ones and, of the new ones, those
 * up to the token itself; with a tree those whose bit is set: bit j of tree[row]
 * stands for new token j of the row's sequence (a tree brings at most 64 tokens
 * a sequence; bits past them are ignored).  A row that sees nothing is zero.
 * What a row does not see does not reach it, also where it is not finite; a
 * score of -inf counts as unseen.
 *   q, out  [N][n_q_heads][head_dim]
 *   new_max, len_max  bounds on the new tokens of a sequence and on lens, which
 *           shape the launch: rows from new_max on are left as they were,
 *           tokens from len_max on are not seen
 *   tree    [N] uint64 or NULL
 *   workspace  256-byte aligned, at least attn_workspace_bytes; its contents
 *           matter only during the call
 * B = 0, N = 0 or new_max = 0 enqueues nothing.  B <= 2^16, N <= 2^20.  Errors:
 * MOE_EINVAL as above, MOE_ENOMEM for a workspace that is too small, MOE_EHIP.
 */
int attn_forward(const attn_desc* d, int32_t B, int32_t N, int32_t new_max, int32_t len_max, const int32_t* cu,
                 const int32_t* lens, const int32_t* table, const uint64_t* tree, const void* q, const void* pages,
                 void* out, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTENTION_H */
