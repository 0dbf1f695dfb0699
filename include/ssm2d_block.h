/*
 * ssm2d_block.h — C ABI of the operators that make a recurrent block in
 * libssm2d.so: projections with their epilogue, the norms before and after a
 * block with its gate, residual and scale, and the gated linear recurrence.
 *
 * Status codes and asynchrony are those of ssm2d.h, types, strides, outputs and
 * errors those of ssm2d_ops.h: a call checks its arguments on the host, enqueues
 * its kernels on `stream` and returns a status without waiting; it never throws
 * or aborts. All pointers are DEVICE pointers on the current HIP device, aligned
 * to their element. Strides count elements and are not negative unless said so.
 * Outputs are dense and must not alias an input unless said so. A `_bf16` entry
 * takes bfloat16 bits (uint16_t) where the plain one takes the same tensor in
 * float32; sums, statistics and states are fp32, and each bf16 output is rounded
 * once (nearest even). Sums are taken in one order whichever workgroup comes
 * first: every output is deterministic.
 *
 * Workspaces are the caller's: a call that needs one takes `workspace`
 * (16-byte aligned, at least as many bytes as the entry's _workspace function
 * says for the same shape and flags; NULL where that is 0) and uses it until
 * its work on the stream is done. The library keeps nothing between calls and
 * allocates nothing, so calls may be captured into HIP graphs in any number;
 * two graphs that may run at once need workspaces of their own.
 *   a workspace smaller than that -> SSM2D_ERR_NOMEM
 *   unknown flags or modes        -> SSM2D_ERR_BAD_FLAGS (checked first)
 * A _workspace function returns a negative status for a shape that the entry
 * refuses.
 */
#ifndef SSM2D_BLOCK_H
#define SSM2D_BLOCK_H

#include "ssm2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Linear --------------------------------------------------------------
 *
 *   z[b][r][j] = sum_i x[b][r][i] weight[j][i] + bias[j]
 *   y = act(z) + residual
 *
 * x: `rows` rows of k channels, x[b][r][i] at b * x_stride[0] + r *
 * x_stride[1] + i; or with SSM2D_LINEAR_X_MAPS channels-first maps, the scan's
 * own layout, at b * x_stride[0] + i * x_stride[1] + r. y and pre: dense
 * [batch][rows][n], or with SSM2D_LINEAR_Y_MAPS dense [batch][n][rows]; residual
 * (NULL: none) in y's layout with strides r_stride (batch; row or channel).
 * weight: [n][k] of x's type, rows w_stride apart; bias: float32 [n] (NULL: none).
 * pre (NULL: not stored): z, of y's type, what the backward of an activation
 * needs. y may be the residual's own buffer (same layout and strides, dense).
 * act: SSM2D_ACT_NONE, _RELU, _SILU (z / (1 + exp(-z))) or _GELU
 * (z (1 + erf(z / sqrt 2)) / 2).
 * bf16 products are exact and summed in fp32. float32 operands go through the
 * bf16 matrix instructions in three exact parts and six products: the three left
 * out are under 2^-21 of a term, and of its sign. GELU errs by up to 0.75e-7 |z| in
 * bf16 before its rounding (more than that rounding below z = -5.5, where GELU is under
 * 1.1e-7) and by 2^-24 |z| in float32. An operand that is Inf or NaN
 * gives Inf or NaN in the outputs that it enters (dbias too), not always the one
 * fp32 arithmetic would give.
 * Limits: rows, n, k, batch < 2^31 - 256, strides < 2^40, fewer than 2^31 tiles of
 * 64 x 64 in y, in x and in the weight, and fewer than 2^31 steps of 32 rows in the
 * batch.
 * k = 0 gives z = bias. */
#define SSM2D_ACT_NONE 0
#define SSM2D_ACT_RELU 1
#define SSM2D_ACT_SILU 2
#define SSM2D_ACT_GELU 3
#define SSM2D_LINEAR_X_MAPS 1u
#define SSM2D_LINEAR_Y_MAPS 2u

typedef struct {
    int64_t batch, rows, n, k;
    int64_t x_stride[2]; /* batch; row, or channel of maps */
    int64_t r_stride[2]; /* of the residual (forward) or dy (backward), likewise */
    int64_t w_stride;
} ssm2d_linear_shape;

int64_t ssm2d_linear_fwd_workspace(const ssm2d_linear_shape *shape, uint32_t flags);
int64_t ssm2d_linear_fwd_workspace_bf16(const ssm2d_linear_shape *shape, uint32_t flags);
int ssm2d_linear_fwd(const float *x, const float *weight, const float *bias, const float *residual, float *y, float *pre,
                     const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace, int64_t workspace_bytes,
                     void *stream);
int ssm2d_linear_fwd_bf16(const uint16_t *x, const uint16_t *weight, const float *bias, const uint16_t *residual, uint16_t *y,
                          uint16_t *pre, const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace,
                          int64_t workspace_bytes, void *stream);

/* Gradients of a loss through linear_fwd for dy = dL/dy (strides r_stride): with
 * dz = dy act'(pre),
 *   dx = dz weight,  dweight = sum dz x^T,  dbias = sum dz   over batch and rows
 * dx: dense in x's layout; dweight: dense [n][k]; dbias: float32 [n]; any of them
 * may be NULL: not computed. pre: as the forward stored it, not read without an
 * activation. The residual's gradient is dy. With an activation dz is rounded to
 * x's type for the products (dbias takes it unrounded). With rows or batch 0,
 * dweight and dbias are zeros. */
int64_t ssm2d_linear_bwd_workspace(const ssm2d_linear_shape *shape, int act, uint32_t flags);
int64_t ssm2d_linear_bwd_workspace_bf16(const ssm2d_linear_shape *shape, int act, uint32_t flags);
int ssm2d_linear_bwd(const float *x, const float *weight, const float *pre, const float *dy, float *dx, float *dweight,
                     float *dbias, const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace,
                     int64_t workspace_bytes, void *stream);
int ssm2d_linear_bwd_bf16(const uint16_t *x, const uint16_t *weight, const uint16_t *pre, const uint16_t *dy, uint16_t *dx,
                          uint16_t *dweight, float *dbias, const ssm2d_linear_shape *shape, int act, uint32_t flags,
                          void *workspace, int64_t workspace_bytes, void *stream);

/* ---- Block norm ------------------------------------------------------------
 *
 * The norm after a block with the block's gate, its scale and the residual
 * stream, and the norm before the next one. Per row of n channels, with
 * rms(v)[c] = v[c] / sqrt(mean of v^2 over c's group + eps):
 *   m = rms(x) weight act(gate),  or with SSM2D_NORM_GATE_FIRST
 *   m = rms(x act(gate)) weight
 *   out = residual + scale m
 *   y = out / sqrt(mean of out^2 over the row + eps) next_weight
 * `groups` equal groups of neighbouring channels (heads) are normed each by
 * itself. Without SSM2D_NORM_ON rms and weight are left out (the norm before a
 * block alone: out = residual + x, y its norm; dweight is zeros). gate NULL: no gate; act is SiLU,
 * or the sigmoid with SSM2D_NORM_GATE_SIGMOID. residual NULL: zeros. weight,
 * scale, next_weight: float32 [n], NULL: ones. y NULL: not computed; y comes from
 * out before it is rounded. With SSM2D_NORM_RESIDUAL_F32 residual, out, dout
 * and dresidual are float32 in the _bf16 entries too.
 * x, gate, residual, dout, dy: rows of n channels at a stride each; out and y
 * dense. out may be the residual's own buffer if that is dense.
 * Limits: n <= SSM2D_NORM_MAX_N, a multiple of groups (else SSM2D_ERR_BAD_DIM);
 * rows * n < 2^50. */
#define SSM2D_NORM_MAX_N 16384
#define SSM2D_NORM_ON 1u
#define SSM2D_NORM_GATE_SIGMOID 2u
#define SSM2D_NORM_GATE_FIRST 4u
#define SSM2D_NORM_RESIDUAL_F32 8u

typedef struct {
    int64_t rows, n, groups;
    int64_t x_stride, gate_stride, res_stride, dout_stride, dy_stride;
} ssm2d_block_norm_shape;

int ssm2d_block_norm_fwd(const float *x, const float *gate, const void *residual, const float *weight, const float *scale,
                         const float *next_weight, void *out, float *y, const ssm2d_block_norm_shape *shape, float eps,
                         uint32_t flags, void *stream);
int ssm2d_block_norm_fwd_bf16(const uint16_t *x, const uint16_t *gate, const void *residual, const float *weight,
                              const float *scale, const float *next_weight, void *out, uint16_t *y,
                              const ssm2d_block_norm_shape *shape, float eps, uint32_t flags, void *stream);

/* Gradients of block_norm_fwd for dout = dL/dout (the gradient that reaches out
 * otherwise than through y; NULL: zeros) and dy = dL/dy (NULL: zeros): dx, dgate
 * (x's type), dresidual (out's type), and dweight, dscale, dnext_weight (float32
 * [n]); any of them may be NULL: not computed. The forward is computed again from
 * x, gate and residual, in registers: nothing of it need be kept. The channel
 * sums go through per-workgroup partial sums in the workspace, added in a fixed
 * order. */
int64_t ssm2d_block_norm_bwd_workspace(const ssm2d_block_norm_shape *shape, uint32_t flags);
int ssm2d_block_norm_bwd(const float *x, const float *gate, const void *residual, const float *weight, const float *scale,
                         const float *next_weight, const void *dout, const float *dy, float *dx, float *dgate,
                         void *dresidual, float *dweight, float *dscale, float *dnext_weight,
                         const ssm2d_block_norm_shape *shape, float eps, uint32_t flags, void *workspace,
                         int64_t workspace_bytes, void *stream);
int ssm2d_block_norm_bwd_bf16(const uint16_t *x, const uint16_t *gate, const void *residual, const float *weight,
                              const float *scale, const float *next_weight, const void *dout, const uint16_t *dy,
                              uint16_t *dx, uint16_t *dgate, void *dresidual, float *dweight, float *dscale,
                              float *dnext_weight, const ssm2d_block_norm_shape *shape, float eps, uint32_t flags,
                              void *workspace, int64_t workspace_bytes, void *stream);

/* ---- Gated linear recurrence ---------------------------------------------
 *
 * Each channel by itself along the tokens, the scan's relative in one
 * dimension with the gate as input:
 *   h[t] = a[t] h[t - 1] + w[t] x[t]
 *   a = exp(g), w = 1                (g: log decay, usually <= 0; -inf clears)
 *   a = 1 / (1 + exp(-g)), w = 1 - a (SSM2D_RECUR_SIGMOID)
 * x, g: [batch][tokens][channels] at strides (batch, token) with channels
 * contiguous, or with SSM2D_RECUR_MAPS [batch][channels][tokens] at strides
 * (batch, channel) with tokens contiguous (the scan's own layout, cells as
 * tokens). h: dense in the same layout, of x's type; the state itself is fp32.
 * SSM2D_RECUR_REVERSE goes from the last token to the first (h[t - 1] is then
 * h[t + 1], "last" the first token; not with packed sequences).
 * Packed sequences (n_seq > 0, not with maps): batch = 1, cu_seqlens as in
 * ssm2d_gated_delta_fwd; else n_seq = 0, cu_seqlens is ignored and sequences =
 * batch.
 * h_init (NULL: zeros), h_last (NULL: not stored): float32
 * [sequences][channels]; h_last may be h_init. An empty sequence passes its
 * state on. One token with h_last = h_init = the state is the step of serving.
 * Growing gates (0 < g < 88): a state of 0 stays 0 until x is not. Through any run of
 * tokens that another state passes, the product of the a's has to be a float (a sum
 * of g under 88; for the gradients the flow e likewise, from the last token on):
 * tokens are joined in stretches, and where a stretch's product overflows h may be
 * Inf or NaN from there on though a[t] h[t - 1], token by token, would not be.
 * Of long rows chunks of tokens go to workgroups of their own, each of which waits
 * for the state that the one before hands on. All that it waits for runs already; a
 * wait that none the less takes more polls than ssm2d_set_spin_limit sets (seconds,
 * if it is not called) is given up: h is NaN from that chunk on, and the device's
 * next ssm2d_sync_check, of whichever stream, returns SSM2D_ERR_DEVICE_TIMEOUT.
 * Limits: batch, channels, tokens and n_seq < 2^31 - 65536, channels * batch < 2^31,
 * channels * n_seq <= 2^32 - 256, batch * tokens * channels <= 10^14. */
#define SSM2D_RECUR_SIGMOID 1u
#define SSM2D_RECUR_MAPS 2u
#define SSM2D_RECUR_REVERSE 4u

typedef struct {
    int64_t batch, tokens, channels, n_seq;
    int64_t x_stride[2], g_stride[2], dh_stride[2]; /* batch; token, or channel of maps */
} ssm2d_recurrence_shape;

int64_t ssm2d_recurrence_fwd_workspace(const ssm2d_recurrence_shape *shape, uint32_t flags);
int64_t ssm2d_recurrence_fwd_workspace_bf16(const ssm2d_recurrence_shape *shape, uint32_t flags);
int ssm2d_recurrence_fwd(const float *x, const float *g, const float *h_init, const int32_t *cu_seqlens, float *h,
                         float *h_last, const ssm2d_recurrence_shape *shape, uint32_t flags, void *workspace,
                         int64_t workspace_bytes, void *stream);
int ssm2d_recurrence_fwd_bf16(const uint16_t *x, const uint16_t *g, const float *h_init, const int32_t *cu_seqlens,
                              uint16_t *h, float *h_last, const ssm2d_recurrence_shape *shape, uint32_t flags,
                              void *workspace, int64_t workspace_bytes, void *stream);

/* Gradients of recurrence_fwd for dh = dL/dh (strides dh_stride) and dh_last =
 * dL/dh_last (NULL: zeros): with e[t] = dh[t] + a[t + 1] e[t + 1],
 *   dx = w e,   dg = a h[t - 1] e,  or  a w (h[t - 1] - x) e with the sigmoid
 * dx, dg: dense like h; dh_init (NULL: not stored): float32 [sequences][channels],
 * may be dh_last. The states are computed again in fp32. */
int64_t ssm2d_recurrence_bwd_workspace(const ssm2d_recurrence_shape *shape, uint32_t flags);
int64_t ssm2d_recurrence_bwd_workspace_bf16(const ssm2d_recurrence_shape *shape, uint32_t flags);
int ssm2d_recurrence_bwd(const float *x, const float *g, const float *h_init, const int32_t *cu_seqlens, const float *dh,
                         const float *dh_last, float *dx, float *dg, float *dh_init, const ssm2d_recurrence_shape *shape,
                         uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream);
int ssm2d_recurrence_bwd_bf16(const uint16_t *x, const uint16_t *g, const float *h_init, const int32_t *cu_seqlens,
                              const uint16_t *dh, const float *dh_last, uint16_t *dx, uint16_t *dg, float *dh_init,
                              const ssm2d_recurrence_shape *shape, uint32_t flags, void *workspace,
                              int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM2D_BLOCK_H */
