/*
 * mxfp4.h - C ABI of microscaled 4-bit floating point (gfx950): quantisation,
 * its inverse, and products of two microscaled matrices, dense and by routed
 * expert.
 *
 * moe_layer.h's experts hold affine int4/int8 codes that every kernel turns
 * into float16 or fp32 before it multiplies.  The format here is the one that
 * the matrix units multiply as it is (the MX format of the Open Compute
 * Project with E2M1 elements and E8M0 scales): 32 consecutive values of a row
 * share one power of two.
 *
 *   m = max |x| over the 32 values,  e = max(floor(log2 m) - 2, -127)
 *   (m = 0: e = -127),  q = x / 2^e rounded to the nearest of 0, 1/2, 1, 3/2,
 *   2, 3, 4, 6 with either sign, ties to the even code, larger values to 6;
 *   the value held is q 2^e.
 *   A block with a NaN or an infinity has the scale byte 255 and holds NaN.
 *
 * Storage of a matrix [rows, cols] ("MX matrix"), Kp = cols rounded up to a
 * multiple of 256 (so that a row's codes are whole 128-byte cache lines):
 *   codes   [rows][Kp / 2] bytes, two codes a byte, the first in the low half;
 *           code = index into the list above, + 8 with a minus sign
 *   scales  [rows][Kp / 32] bytes, e + 127
 * Values past cols are zero codes; scale bytes of blocks past cols are zero.
 * Both arrays start 16-byte aligned.
 *
 * Products: y[m, n] = sum_k A[m, k] W[n, k], A and W MX matrices, the 4-bit
 * products and the sums formed by the scaled MFMA instructions in fp32.  A may
 * be given as fp32 or bf16: it is quantised by the rule above within the call.
 * With MX_ACT_SWIGLU, W holds 2 n rows, n gate rows then n up rows, and the
 * output is y[m, n] = silu(g) u, silu(g) = g / (1 + exp(-g)), in fp32 before
 * the one rounding to the output's type.
 *
 * Conventions as in moe_layer.h: device pointers owned by the caller, work
 * enqueued on `stream`, every argument checked before anything is enqueued,
 * MOE_OK or a negative MOE_E* code with the reason in moe_last_error(),
 * deterministic results (no floating-point atomics).
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stddef.h>
#include <stdint.h>

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MX_FP4 2           /* a_dtype beside MOE_F32 and MOE_BF16: A is an MX matrix */

#define MX_ACT_NONE 0
#define MX_ACT_SWIGLU 1

/* Bytes of the codes and of the scales of an MX matrix; -1 if rows or cols is
 * negative or too large (rows < 2^31, cols <= 2^20).  Pure functions. */
int64_t mx_codes_bytes(int64_t rows, int64_t cols);
int64_t mx_scales_bytes(int64_t rows, int64_t cols);

/*
 * x (dtype MOE_F32 or MOE_BF16; row r at x + r * x_stride elements, x_stride
 * >= cols) into an MX matrix, padding included; and back, exactly (every value
 * held is a bf16 and an fp32 number; NaN blocks give NaN).  The rows' starts
 * need no alignment beyond the element's.  rows = 0 or cols = 0 enqueues
 * nothing.  Errors: MOE_EINVAL (dtype, sizes, strides, NULL or misaligned
 * pointers, an output that overlaps another argument), MOE_EHIP.
 */
int mx_quantize(int32_t dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* codes, void* scales,
                void* stream);
int mx_dequantize(int32_t dtype, int64_t rows, int64_t cols, const void* codes, const void* scales, void* out,
                  int64_t out_stride, void* stream);

/*
 * Descriptor of a product.
 *   n           output columns, 1 .. 2^20
 *   k           inner length, 1 .. 2^20
 *   a_dtype     MOE_F32, MOE_BF16 or MX_FP4
 *   out_dtype   MOE_F32 or MOE_BF16 (one rounding to nearest even)
 *   act         MX_ACT_NONE or MX_ACT_SWIGLU
 * and, for mx_experts_forward only (0 otherwise):
 *   n_experts   E, 1 .. 1024
 *   top_k       k', experts per token, 1 .. 64
 *   pair_rows   0: A has one row per token; 1: one row per pair (t k' + i)
 *   codes_off,  byte offsets inside an expert's blob of the codes and scales of
 *   scales_off  its matrix (rows n, or 2 n with MX_ACT_SWIGLU; k columns);
 *               >= 0 and multiples of 16
 *   pool_bytes  size of the pool; a slot offset is usable if it is >= 0, a
 *               multiple of 256 and the blob's codes and scales end in the pool
 */
typedef struct mx_product_desc {
  int32_t n;
  int32_t k;
  int32_t a_dtype;
  int32_t out_dtype;
  int32_t act;
  int32_t n_experts;
  int32_t top_k;
  int32_t pair_rows;
  int64_t codes_off;
  int64_t scales_off;
  int64_t pool_bytes;
} mx_product_desc;

/* Workspace bytes of a product with up to T_max rows (mx_linear_forward:
 * n_experts = 0) or tokens (mx_experts_forward); 0 if the descriptor or T_max
 * is invalid.  Pure function.  A workspace is cleared once with
 * moe_workspace_init, may be used by calls of any descriptor and of
 * moe_layer.h, and must not be used by two calls that may run at once. */
size_t mx_workspace_bytes(const mx_product_desc* d, int32_t T_max);

/*
 * Dense product of M rows (0 .. 2^20; 0 enqueues nothing).
 *   a, a_scales  fp32 or bf16: a is [M, k], a_scales NULL, a aligned to its
 *                element; MX_FP4: codes and scales of an MX matrix [M, k]
 *   w_codes,     MX matrix of n (2 n with MX_ACT_SWIGLU) rows and k columns
 *   w_scales
 *   out          [M, n], out_dtype, aligned to its element
 *   workspace    ws_bytes >= mx_workspace_bytes(d, M), 256-byte aligned
 * Errors: MOE_EINVAL (also for 2^37 values of A to quantise, which a launch
 * does not hold), MOE_ENOMEM (workspace), MOE_EHIP.
 */
int mx_linear_forward(const mx_product_desc* d, int32_t M, const void* a, const void* a_scales, const void* w_codes,
                      const void* w_scales, void* out, void* workspace, size_t ws_bytes, void* stream);

/*
 * Product by routed expert: pair (t, i), t < T (0 .. 65536, with T k' < 2^22),
 * i < k', takes the matrix of expert topk_ids[t, i], whose blob starts at
 * pool_base + slot_table[expert] (the pool and table of moe_layer.h; the
 * residency manager's slots serve as they are).
 *   a, a_scales  rows as above: T of them, or T k' with pair_rows
 *   topk_ids     [T, k'] int32, as moe_router_topk and moe_router_route write them
 *   topk_w       NULL: out is [T k', n], the product of every pair.
 *                [T, k'] fp32: out is [T, n], sum_i topk_w[t, i] y[t, i], formed
 *                in fp32 in a fixed order and rounded once
 *   slot_table   [E] int64 byte offsets
 * A pair whose id is outside [0, E) or whose slot is unusable contributes
 * nothing, whatever its row of A and its weight hold (its row of the output is
 * zero), and raises MOE_ERANGE in moe_status_check(workspace).  An expert may
 * occur twice in a token's ids.  MOE_EINVAL also where a launch would need 2^32
 * threads or more (T n of 2^32 columns, 2^35 values of A to quantise, the tiles
 * of the grouped pairs: 2 n threads for each expert that has pairs and for
 * every 128 pairs, 4 n with MX_ACT_SWIGLU).  Errors as above.
 */
int mx_experts_forward(const mx_product_desc* d, int32_t T, const void* a, const void* a_scales,
                       const int32_t* topk_ids, const float* topk_w, const int64_t* slot_table, const void* pool_base,
                       void* out, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
