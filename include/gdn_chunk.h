/*
 * gdn_chunk.h - C ABI of the gated delta rule over prompts (gfx950).
 *
 * The rule of gdn_recurrence.h for many tokens at once: sequences of any
 * length, packed, 64 tokens of each at a time as matrix products instead of
 * one after the other.  Within such a chunk with incoming state S (d_v x d_k),
 * normalised keys and queries k'_i, q'_i, gates alpha_i, write strengths
 * beta_i, D_ij = alpha_{j+1} ... alpha_i and g_i = alpha_1 ... alpha_i:
 *   (I + A) U = diag(beta) (V - diag(g) K' S^T),   A_ij = beta_i D_ij k'_i . k'_j  (j < i)
 *   O = diag(g) Q' S^T + P U,                      P_ij = D_ij q'_i . k'_j         (j <= i)
 *   S <- g_C S + sum_j D_Cj u_j k'_j^T
 * which is the recurrence rearranged: the same results up to rounding, in
 * single precision or better (of the output products, where the output is
 * bf16, 16 bits).  Chunks whose keys or queries are not finite, whose gates are
 * not in [2^-20, 1] or whose write strengths are not in [0, 2] run token by
 * token, and so do the state rows whose values, or what the state predicts of
 * them, are not finite or above 2^96: what a later token holds never reaches an
 * earlier one, nor one row of a state another.
 *
 * Conventions as in moe_layer.h: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked before anything is enqueued,
 * MOE_OK or a negative MOE_E* code with the reason in moe_last_error(),
 * deterministic results.
 */
#ifndef GDN_CHUNK_H
#define GDN_CHUNK_H

#include <stddef.h>
#include <stdint.h>

#include "gdn_recurrence.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace that gdn_chunk_forward needs for B sequences of N tokens
 * together, or (size_t)-1 for arguments that it would refuse. */
size_t gdn_chunk_workspace_bytes(const gdn_desc* d, int32_t B, int32_t N);

/* Advance B independent sequences by their tokens.  Sequence b holds rows
 * [cu[b], cu[b + 1]) of N; it may hold none (its state is copied).
 *   cu         [B + 1] int32, read on the device
 *   q, k       [N][n_k_heads][d_k]   act_dtype, 16-byte aligned
 *   v          [N][n_v_heads][d_v]   act_dtype, 16-byte aligned
 *   alpha, beta [N][n_v_heads] fp32
 *   state_in   [B][n_v_heads][d_v][d_k] fp32, or NULL: zeros
 *   state_out  likewise; may be state_in itself
 *   out        [N][n_v_heads][d_v]   out_dtype
 *   T_max      bound on the tokens of a sequence; what lies behind it in a
 *              sequence is ignored
 *   workspace  256-byte aligned, at least gdn_chunk_workspace_bytes
 * Rows of no sequence are left as they were in out.  B = 0 enqueues nothing.
 * B <= 2^16, N <= 2^24.  Errors: MOE_EINVAL for a bad descriptor (as in
 * gdn_recurrence.h), sizes, a NULL or misaligned pointer, or an output that
 * overlaps another argument; MOE_ENOMEM for a workspace that is too small;
 * MOE_EHIP if a launch fails. */
int gdn_chunk_forward(const gdn_desc* d, int32_t B, int32_t N, int32_t T_max, const int32_t* cu, const void* q,
                      const void* k, const void* v, const float* alpha, const float* beta, const float* state_in,
                      float* state_out, void* out, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_CHUNK_H */
