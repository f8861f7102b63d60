/*
 * wtconv_seq.h -- C ABI of the sequence operators of libwtconv.so (sm_100a):
 * the causal depthwise convolution over tokens, the selective state space
 * scan that reads it, and the norms before and after a block with its gate
 * and residual scale.  With the dense projections between them (a library's
 * matrix products) they make up a gated state space block, for training
 * (forward and gradients), for prompts and for single tokens.
 *
 * Definitions (all entry points follow them exactly, up to fp32 rounding):
 *   silu(v) = v / (1 + exp(-v));  softplus(v) = log(1 + exp(v))
 *   Causal convolution: for row b, token t, channel c, taps j = 0 .. k-1,
 *     p[b,t,c] = bias[c] + sum_j w[c][j] x[b, t-(k-1)+j, c],  y = silu(p) or p,
 *     where x at token -i (i = 1 .. k-1) is state[b][k-1-i][c], or zero.  The
 *     state after the pass holds the last k-1 inputs, oldest first.
 *   Scan: delta = softplus(dt + dt_bias) (or dt + dt_bias),
 *     h_t[c][n] = exp(delta_t[c] a[c][n]) h_{t-1}[c][n] + delta_t[c] x_t[c] b_t[g][n],
 *     y_t[c] = (sum_n c_t[g][n] h_t[c][n] + d[c] x_t[c]) silu(z_t[c]),
 *     g = c / (C / G): every C / G consecutive channels share b and c;
 *     without d or z that term or factor is left out.
 *   Norm: u = x silu(gate);  v = u w / sqrt(mean_c(u^2) + eps);
 *     res_out = res + scale v;  y = res_out w_res / sqrt(mean_c(res_out^2) + eps).
 *     Without gate u = x; without w v = u; without scale it is 1; without res
 *     y = v, and there is no res_out, scale or w_res; without w_res no y.
 *
 * Layouts: activations are rows of C contiguous channels, [B][T][C] with free
 * batch and token strides (wtconv_rows), so halves of a projection's output
 * or one request's slice of a batch need no copy.  b and c of the scan are
 * rows of G*N.  Their element type is the I/O dtype (fp32 or bf16); weights,
 * parameter gradients and the scan's state are fp32 and contiguous:
 *   w [C][k]   bias, d, dt_bias, scale, w, w_res [C]   a [C][N]
 *   scan state [B][C][N] fp32   convolution state [B][k-1][C] in the I/O dtype
 *
 * Conventions, beyond those of wtconv.h (asynchronous on `stream`, nothing
 * allocated, kept or synchronised, checks on the host before any launch,
 * gradients overwritten, fixed reduction order, capturable in CUDA graphs):
 *   - lengths (device, int32 [B], NULL = all T): row b holds min(T,
 *     lengths[b]) tokens; a length <= 0 leaves it empty.  Tokens behind are
 *     neither used (they may hold NaN) nor do they move a state; outputs and
 *     gradients there are zero.  An empty row's state comes out as it went in.
 *   - active (device, int32 [B], NULL = all) in the single-token calls: 0
 *     leaves the row's state as it is and its output zero.
 *   - Pointers need the alignment of their element type only; calls whose
 *     pointers, strides and channel counts suit wide loads use them.
 *   - Input rows may overlap or repeat (strides of 0 or more); rows of an
 *     output must not: token by token within a batch row, or batch rows
 *     within a token.  Outputs must not overlap inputs, except that a state
 *     may be updated in place (state_out == state).  Calls in which an output
 *     begins where an input does are refused where threads would read what
 *     others have written.
 *   - Workspaces hold a call's partial sums while it runs and may be reused
 *     by the next call on the same stream.
 *   - Arithmetic is fp32; the sums over a row's channels or tokens included.
 *   - WTCONV_ERR_ARG: null or negative arguments, a descriptor out of range,
 *     overlapping output rows, an output where an input begins (as above);
 *     WTCONV_ERR_ALIGN: a pointer not aligned to its
 *     elements (workspace: 16 bytes); WTCONV_ERR_WORKSPACE: workspace too
 *     small; WTCONV_ERR_UNSUPPORTED: k > 8, N > 64 or, for the norm, rows of
 *     more channels than one thread block holds (WTCONV_NORM_MAX_C).
 */
#ifndef WTCONV_SEQ_H
#define WTCONV_SEQ_H

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WTCONV_CAUSAL_MAX_K 8
#define WTCONV_SCAN_MAX_N 64
#define WTCONV_NORM_MAX_C 16384

/* Rows of an activation: channel c of token t of batch row b is
 * data[b * batch_stride + t * token_stride + c], strides in elements (the
 * token stride at most 2^31 - 1), at most 2^31 - 4096 elements a token (of the
 * scan's, with each group's rounded up to 16 bytes and to four states). */
typedef struct {
  void* data;
  long long batch_stride, token_stride;
} wtconv_rows;

/* B batch rows of T tokens (at most 2^30) of C channels, k taps, silu after it
 * or not. */
typedef struct {
  int B, T, C, k;
  wtconv_dtype io;
  int silu;
} wtconv_causal_desc;

/* N states a channel, G groups of channels that share b and c. */
typedef struct {
  int B, T, C, N, G;
  wtconv_dtype io;
  int softplus;
} wtconv_scan_desc;

/* io: type of x, gate, y and their gradients; res: of res, res_out and dres. */
typedef struct {
  int B, T, C;
  wtconv_dtype io, res;
  float eps;
} wtconv_norm_desc;

/* Causal depthwise convolution over the tokens.  bias, state, lengths and
 * state_out may be NULL.  One launch. */
wtconv_status wtconv_causal_forward(const wtconv_causal_desc* desc, const wtconv_rows* x, const float* w,
                                    const float* bias, const void* state, const int* lengths,
                                    const wtconv_rows* y, void* state_out, void* stream);

/* Gradients of <y, dy> + <state_out, dstate_out>: dx, dw [C][k], dbias [C]
 * (NULL when there is no bias) and dstate, for the state before the pass
 * (NULL when not wanted).  p is computed again from x. */
wtconv_status wtconv_causal_backward(const wtconv_causal_desc* desc, const wtconv_rows* x, const wtconv_rows* dy,
                                     const float* w, const float* bias, const void* state, const int* lengths,
                                     const void* dstate_out, const wtconv_rows* dx, float* dw, float* dbias,
                                     void* dstate, void* ws, size_t ws_bytes, void* stream);

/* One token of every row (desc->T = 1; x and y without token stride): y from
 * the state and x, and the state moved on by x, in place. */
wtconv_status wtconv_causal_step(const wtconv_causal_desc* desc, const wtconv_rows* x, const float* w,
                                 const float* bias, const int* active, const wtconv_rows* y, void* state,
                                 void* stream);

/* Bytes of workspace that wtconv_causal_backward needs (0: invalid desc). */
size_t wtconv_causal_workspace_size(const wtconv_causal_desc* desc);

/* Selective state space scan.  d, z, dt_bias, state, lengths and state_out
 * may be NULL. */
wtconv_status wtconv_scan_forward(const wtconv_scan_desc* desc, const wtconv_rows* x, const wtconv_rows* dt,
                                  const float* a, const wtconv_rows* b, const wtconv_rows* c, const float* d,
                                  const wtconv_rows* z, const float* dt_bias, const float* state,
                                  const int* lengths, const wtconv_rows* y, float* state_out, void* ws,
                                  size_t ws_bytes, void* stream);

/* Gradients of <y, dy> + <state_out, dstate_out> with respect to x, dt, a, b,
 * c, d, z, dt_bias and the state before the pass.  dd, dz, ddt_bias are
 * required exactly when d, z, dt_bias are given; dstate may be NULL.  The
 * states are computed again from the inputs. */
wtconv_status wtconv_scan_backward(const wtconv_scan_desc* desc, const wtconv_rows* x, const wtconv_rows* dt,
                                   const float* a, const wtconv_rows* b, const wtconv_rows* c, const float* d,
                                   const wtconv_rows* z, const float* dt_bias, const float* state,
                                   const int* lengths, const wtconv_rows* dy, const float* dstate_out,
                                   const wtconv_rows* dx, const wtconv_rows* ddt, float* da, const wtconv_rows* db,
                                   const wtconv_rows* dc, float* dd, const wtconv_rows* dz, float* ddt_bias,
                                   float* dstate, void* ws, size_t ws_bytes, void* stream);

/* One token of every row (desc->T = 1): y, and the state moved on in place. */
wtconv_status wtconv_scan_step(const wtconv_scan_desc* desc, const wtconv_rows* x, const wtconv_rows* dt,
                               const float* a, const wtconv_rows* b, const wtconv_rows* c, const float* d,
                               const wtconv_rows* z, const float* dt_bias, const int* active,
                               const wtconv_rows* y, float* state, void* stream);

/* Bytes of workspace of wtconv_scan_forward (backward = 0) or
 * wtconv_scan_backward (backward = 1).  0: none needed, or invalid desc. */
size_t wtconv_scan_workspace_size(const wtconv_scan_desc* desc, int backward);

/* Norms before and after a block with its gate and residual scale.  gate, w,
 * res (with scale, w_res and res_out) and lengths may be NULL; y is required
 * unless res is given without w_res, res_out when res is given. */
wtconv_status wtconv_norm_forward(const wtconv_norm_desc* desc, const wtconv_rows* x, const wtconv_rows* gate,
                                  const float* w, const wtconv_rows* res, const float* scale, const float* w_res,
                                  const int* lengths, const wtconv_rows* y, const wtconv_rows* res_out,
                                  void* stream);

/* Gradients of <y, dy> + <res_out, dres_out>: dx, dgate, dw, dres, dscale,
 * dw_res, each required exactly when its input is given.  dres_out may be
 * NULL (zero).  Everything is computed again from the inputs. */
wtconv_status wtconv_norm_backward(const wtconv_norm_desc* desc, const wtconv_rows* x, const wtconv_rows* gate,
                                   const float* w, const wtconv_rows* res, const float* scale, const float* w_res,
                                   const int* lengths, const wtconv_rows* dy, const wtconv_rows* dres_out,
                                   const wtconv_rows* dx, const wtconv_rows* dgate, float* dw,
                                   const wtconv_rows* dres, float* dscale, float* dw_res, void* ws,
                                   size_t ws_bytes, void* stream);

/* Bytes of workspace that wtconv_norm_backward needs (0: invalid desc). */
size_t wtconv_norm_workspace_size(const wtconv_norm_desc* desc);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_SEQ_H */
