/*
 * tm_layer.h -- C ABI of a layer's operators beside the memory on MI355X
 * (gfx950): the norms of queries and keys for each head with their rotary
 * positions, linear attention with a decay (a memory of one matrix), and
 * products with weights held in 8-bit integers.
 *
 * They stand beside the attention window's calls (tm_attention.h), need no
 * tm_ctx, and follow the same conventions: caller-owned device memory,
 * asynchronous on `stream`, a tm_status from every call, argument checks on
 * the host before anything is launched, no state kept between calls.  Calls
 * may run at the same time with workspaces of their own.  All of them may be
 * captured into a graph.
 *
 * Tensors.  Token arrays are [batch][n_tokens][heads][dim] of bf16 or fp32
 * (tm_dtype); the last two axes are contiguous, the distances between batch
 * entries and between tokens are given in elements.  Arrays that a call
 * writes must not overlap its other arrays except where it says so.  A call
 * whose launch would have 2^32 threads or more along an axis is refused
 * (TM_ERR_INVALID).
 */
#ifndef TM_LAYER_H
#define TM_LAYER_H

#include "tm_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- norms of queries and keys for each head, with rotary positions ---- */

/* Each head vector x of the first `heads` heads (queries) and of the
 * kv_heads behind them (keys) becomes
 *   y = rotate(w * x / sqrt(mean(x^2) + eps)),
 * the mean over its head_dim elements, w = w_q or w_k (fp32 [head_dim], or
 * null: ones), the rotation that of tm_rotary (rot_dim, layout, positions,
 * freq, result_scale as there; rot_dim 0: none, positions and freq are not
 * read).  Statistics and products are fp32, y is rounded once to the dtype.
 * kv_heads may be 0 (w_k is not read).  y may be x (with the same distances).
 * Unit vectors are the case w = 1 / sqrt(head_dim).  x, y: aligned to their
 * element type, head_dim 1 .. 1024, heads + kv_heads at most 65535, eps >= 0.
 * A vector of zeros with eps = 0 gives NaN, as the formula does.  batch *
 * n_tokens == 0 is a no-op. */
tm_status tm_head_norm(const void* x, long x_batch, long x_token, void* y, long y_batch, long y_token,
                       const float* w_q, const float* w_k, double eps, const int* positions, int per_token,
                       const double* freq, double result_scale, int batch, int n_tokens, int heads, int kv_heads,
                       int head_dim, int rot_dim, tm_rope_layout layout, tm_dtype dtype, void* stream);

/* Workspace bytes of tm_head_norm_backward; 256-byte aligned, holds no data
 * between calls. */
size_t tm_head_norm_workspace_bytes(int batch, int n_tokens, int heads, int kv_heads, int head_dim);

/* The gradients of an outer loss through a tm_head_norm call of the same
 * arguments, from dy (its gradient with respect to y): dx, and dw_q, dw_k
 * (fp32 [head_dim]; null: not wanted), which are written, not added to.
 * dx may be dy or x (with the same distances).  Sums are fp32, in an order
 * that the call's sizes fix.  batch * n_tokens == 0 gives zero dw_q and dw_k. */
tm_status tm_head_norm_backward(const void* x, long x_batch, long x_token, const void* dy, long dy_batch,
                                long dy_token, void* dx, long dx_batch, long dx_token, const float* w_q,
                                const float* w_k, float* dw_q, float* dw_k, double eps, const int* positions,
                                int per_token, const double* freq, double result_scale, int batch, int n_tokens,
                                int heads, int kv_heads, int head_dim, int rot_dim, tm_rope_layout layout,
                                tm_dtype dtype, void* workspace, void* stream);

/* ---- linear attention with a decay ---- */

/* For each entry b and key head h, a state S [key_dim][value_dim] (fp32)
 * goes over the tokens t in order:
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   out_t = scale S_t^T q_t
 * for each of the heads / kv_heads query heads that share it.  g =
 * log_decay: fp32 [batch][n_tokens][kv_heads] (per_token != 0) or [kv_heads]
 * (one decay for each head); 0 keeps all, -inf drops what came before, and
 * what a token keeps below exp(-1000) counts as dropped.  Values above 0 make
 * the state grow; nothing checks them.  q [batch][n_tokens][heads][key_dim],
 * k [..][kv_heads][key_dim], v [..][kv_heads][value_dim], out contiguous
 * [batch][n_tokens][heads][value_dim].  counts: device int32 [batch], tokens
 * of each entry (clamped to 0 .. n_tokens; null: n_tokens each); rows behind
 * an entry's count are not read, and left as they were in out.  state_in,
 * state_out: fp32 [batch][kv_heads][key_dim][value_dim] contiguous, 16-byte
 * aligned; state_in null: zeros; state_out null: not wanted; state_out may be
 * state_in.  An entry without tokens keeps its state.
 * key_dim, value_dim: multiples of 8, 8 .. 256; heads a multiple of kv_heads,
 * at most 64 * kv_heads and 32768; n_tokens at most 2^30; token arrays
 * 16-byte aligned, distances multiples of 8 elements, those of tokens below
 * 2^23.
 * Products of bf16 calls are of bf16 operands with fp32 accumulation: the
 * pairs' weights within a chunk of tokens and the state before it keep 16 bits
 * (two operands each), what is added to the state 24; the outputs' own rounding
 * is coarser by 2^8.  Those of fp32 calls, and of bf16 calls of up to 5 tokens,
 * are fp32.  Decays are summed in 64 bits, the state is fp32 throughout.
 * A non-finite key or value leaves the outputs of earlier tokens as they are;
 * those of its head from its token on, and its state, are not defined.
 * batch or n_tokens 0: state_out becomes state_in (batch 0: no-op). */
tm_status tm_linear_attention(const void* q, long q_batch, long q_token, const void* k, long k_batch, long k_token,
                              const void* v, long v_batch, long v_token, const float* log_decay, int per_token,
                              const int* counts, const float* state_in, float* state_out, void* out, double scale,
                              int batch, int n_tokens, int heads, int kv_heads, int key_dim, int value_dim,
                              tm_dtype dtype, void* workspace, void* stream);

/* Workspace bytes of tm_linear_attention (backward == 0) or of its backward;
 * 256-byte aligned, holds no data between calls.  0 for calls that need none
 * (the workspace may then be null), and for sizes that the calls refuse. */
size_t tm_linear_workspace_bytes(int batch, int n_tokens, int heads, int kv_heads, int key_dim, int value_dim,
                                 int backward);

/* The gradients of an outer loss through a tm_linear_attention call of the
 * same arguments, from dout [batch][n_tokens][heads][value_dim] (distances
 * as a token array's) and dstate_out (the gradient with respect to
 * state_out; null: zeros): dq, dk, dv (contiguous, of the dtype; rows behind
 * an entry's count are left as they were), dlog_decay (fp32, of log_decay's
 * shape; per token: rows behind the count are left as they were; null: not
 * wanted) and dstate_in (fp32; null: not wanted).  dstate_in may be
 * dstate_out.  dk and dv are summed over the query heads of a key head, a
 * head's dlog_decay over batch and tokens, in an order that the call's sizes
 * fix.  The gradient of a decay of -inf, or of -1000 and below, is 0.
 * Gradients through non-finite values are not defined.  batch 0: a head's
 * dlog_decay becomes zero. */
tm_status tm_linear_attention_backward(const void* q, long q_batch, long q_token, const void* k, long k_batch,
                                       long k_token, const void* v, long v_batch, long v_token,
                                       const float* log_decay, int per_token, const int* counts,
                                       const float* state_in, const void* dout, long dout_batch, long dout_token,
                                       const float* dstate_out, void* dq, void* dk, void* dv, float* dlog_decay,
                                       float* dstate_in, double scale, int batch, int n_tokens, int heads,
                                       int kv_heads, int key_dim, int value_dim, tm_dtype dtype, void* workspace,
                                       void* stream);

/* ---- products with 8-bit integers ---- */

/* Rows of x [rows][cols] (x_row elements apart, aligned to their type) as
 * 8-bit integers with a scale each: with m = max |x| over a row,
 *   codes = (127 x) / m rounded to nearest even, scales = m / 127,
 * product and quotients in fp32 (exact for bf16: a code is off by one only
 * where an fp32 quotient stands within its rounding of a half)
 * (a row of zeros: codes and scale 0; one with a non-finite element: codes 0,
 * scale NaN).  codes: int8 [rows][code_row], 16-byte aligned, code_row a
 * multiple of 16 and at least cols; the columns behind cols become 0.
 * cols 1 .. 131072 (a row's product then fits 32 bits).  rows 0 is a no-op. */
tm_status tm_int8_quantize(const void* x, long x_row, signed char* codes, long code_row, float* scales, long rows,
                           int cols, tm_dtype dtype, void* stream);

/* y[m][n] = (sum_k a[m][k] w[n][k]) a_scales[m] w_scales[n], rounded once to
 * dtype: a [rows][code_row], w [outs][code_row] int8 in -127 .. 127 (16-byte
 * aligned, code_row a multiple of 16 and at least cols; what stands behind
 * cols must be 0 in both), y rows y_row elements apart, aligned to its type.
 * The sum is exact (32-bit integers); it takes a_scales, then w_scales, in 64
 * bits. */
tm_status tm_int8_matmul(const signed char* a, const float* a_scales, const signed char* w, const float* w_scales,
                         long code_row, void* y, long y_row, long rows, int outs, int cols, tm_dtype dtype,
                         void* stream);

/* tm_int8_quantize of x's rows and tm_int8_matmul with w in one call: the
 * same results.  code_row: cols, the next multiple of 16.  workspace: tm_int8_workspace_bytes(rows, cols), 256-byte
 * aligned, holds no data between calls. */
size_t tm_int8_workspace_bytes(long rows, int cols);
tm_status tm_int8_linear(const void* x, long x_row, const signed char* w, const float* w_scales, long code_row,
                         void* y, long y_row, long rows, int outs, int cols, tm_dtype dtype, void* workspace,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TM_LAYER_H */
