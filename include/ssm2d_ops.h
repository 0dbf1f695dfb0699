/*
 * ssm2d_ops.h — C ABI of the operators around the 2D scan in libssm2d.so:
 * layer norm, rotary positions with several axes, and the gated delta rule.
 *
 * Status codes, asynchrony, workspaces and graph capture are those of ssm2d.h:
 * a call checks its arguments on the host, enqueues its kernels on `stream`
 * (hipStream_t; NULL = the null stream) and returns a status without waiting;
 * it never throws or aborts. Workspaces belong to (device, stream), grow in
 * stream order and are freed by ssm2d_release_workspaces; once a call of the
 * same kind and size has run on a stream nothing is allocated, and the calls
 * may be captured into a HIP graph and replayed.
 * All pointers are DEVICE pointers on the current HIP device, aligned to their
 * element (wider accesses are used where the address and strides allow).
 * Strides count elements. Outputs are dense and must not alias an input
 * unless said so. A `_bf16` entry takes bfloat16 bits (uint16_t) where the
 * plain one takes the same tensor in float32; all arithmetic, statistics and
 * states are fp32, and each bf16 output is rounded once (nearest even).
 * No result depends on the order of atomics: every output is deterministic.
 *
 * Errors common to all:
 *   a negative size                                  -> SSM2D_ERR_BAD_DIM
 *   nothing to do (a zero size)                      -> SSM2D_OK (outputs that
 *                                                       sum over it are zeroed)
 *   a size beyond the limits stated at the entry     -> SSM2D_ERR_UNSUPPORTED
 *   a required pointer NULL when there is work       -> SSM2D_ERR_NULLPTR
 *   a pointer not aligned to its element             -> SSM2D_ERR_MISALIGNED
 *   workspace allocation failure                     -> SSM2D_ERR_NOMEM
 *   an error of the HIP runtime                      -> SSM2D_ERR_HIP
 * NaN and Inf inputs are not checked; they propagate.
 */
#ifndef SSM2D_OPS_H
#define SSM2D_OPS_H

#include "ssm2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Layer norm --------------------------------------------------------
 *
 *   y = (x - mean) * rstd * weight + bias,
 *   rstd = 1 / sqrt(mean((x - mean)^2) + eps)     over n channels
 *
 * x[b][c][i] lies at b * x_stride_b + c * x_stride_n + i: `batch` token rows of
 * n channels with cells = 1 and x_stride_n = 1, or channels-first maps, the
 * scan's own layout, with cells = H * W and x_stride_n = H * W. y is dense
 * [batch][n][cells]; weight, bias float32 [n] (NULL: ones, zeros); mean, rstd
 * float32 [batch][cells] (NULL: not stored). The variance is the mean of
 * squared differences from the mean, not a difference of moments. Of no channels
 * the mean is 0 and rstd 1 / sqrt(eps).
 * Limit: n <= SSM2D_LN_MAX_N. */
#define SSM2D_LN_MAX_N 16384

int ssm2d_layer_norm_fwd(const float *x, const float *weight, const float *bias, float *y, float *mean, float *rstd,
                         int64_t batch, int64_t n, int64_t cells, int64_t x_stride_b, int64_t x_stride_n, float eps,
                         void *stream);
int ssm2d_layer_norm_fwd_bf16(const uint16_t *x, const float *weight, const float *bias, uint16_t *y, float *mean,
                              float *rstd, int64_t batch, int64_t n, int64_t cells, int64_t x_stride_b,
                              int64_t x_stride_n, float eps, void *stream);

/* Gradients of the layer norm for dy = dL/dy, from x and the forward's mean
 * and rstd: with xh = (x - mean) rstd and gw = dy weight,
 *   dx = rstd (gw - mean_c(gw) - xh mean_c(gw xh)),
 *   dweight = sum dy xh,  dbias = sum dy   over batch and cells
 * (dweight, dbias: NULL = not computed). dx is dense like y, dy has strides
 * like x's. The sums go through per-workgroup partial sums in a workspace of
 * at most 4 KiB * n bytes, added in a fixed order. */
int ssm2d_layer_norm_bwd(const float *x, const float *weight, const float *mean, const float *rstd, const float *dy,
                         float *dx, float *dweight, float *dbias, int64_t batch, int64_t n, int64_t cells,
                         int64_t x_stride_b, int64_t x_stride_n, int64_t dy_stride_b, int64_t dy_stride_n, void *stream);
int ssm2d_layer_norm_bwd_bf16(const uint16_t *x, const float *weight, const float *mean, const float *rstd,
                              const uint16_t *dy, uint16_t *dx, float *dweight, float *dbias, int64_t batch, int64_t n,
                              int64_t cells, int64_t x_stride_b, int64_t x_stride_n, int64_t dy_stride_b,
                              int64_t dy_stride_n, void *stream);

/* ---- Rotary positions with several axes -----------------------------------
 *
 * Turns pairs of a head's dims by angles that belong to axes of a position:
 * rows and columns of a map, or time, height and width of a clip. The first
 * sections[0] pairs take axis 0, the next sections[1] axis 1, and so on:
 *   angle[p] = positions[axis of p][b][t] * inv_freq[p]
 *   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin)
 * Pair p is dims (p, P + p), P = the sum of the sections, or dims (2p, 2p + 1)
 * with SSM2D_ROPE_INTERLEAVED; dims from 2 P on are copied. SSM2D_ROPE_INVERSE
 * turns by -angle: the gradient of the forward with respect to q and k.
 * q: [batch][tokens][heads_q][d], k: [batch][tokens][heads_k][d] (heads_k may
 * be 0, k and k_out then NULL), inner stride 1, other strides (batch, token,
 * head) in q_stride, k_stride; q_out, k_out dense. positions: int32
 * [n_axes][batch][tokens] with strides pos_stride (axis, batch; batch stride 0
 * = shared by the batch), any sign; inv_freq: float32 [P]. sections is a HOST
 * array. The angle is formed exactly (product and its rounding error) and
 * reduced in fp32 pairs: far positions lose no digits.
 * Limits: 1 <= n_axes <= SSM2D_ROPE_MAX_AXES, d <= SSM2D_ROPE_MAX_D;
 * a section < 0 or 2 P > d -> SSM2D_ERR_BAD_DIM; unknown flags ->
 * SSM2D_ERR_BAD_FLAGS. */
#define SSM2D_ROPE_MAX_AXES 4
#define SSM2D_ROPE_MAX_D 1024
#define SSM2D_ROPE_INTERLEAVED 1u
#define SSM2D_ROPE_INVERSE 2u

typedef struct {
    int64_t batch, tokens, heads_q, heads_k, d;
    int64_t q_stride[3], k_stride[3]; /* batch, token, head */
    int64_t n_axes;
    int64_t sections[SSM2D_ROPE_MAX_AXES];
    int64_t pos_stride[2]; /* axis, batch */
} ssm2d_rope_shape;

int ssm2d_rope(const float *q, const float *k, const int32_t *positions, const float *inv_freq, float *q_out,
               float *k_out, const ssm2d_rope_shape *shape, uint32_t flags, void *stream);
int ssm2d_rope_bf16(const uint16_t *q, const uint16_t *k, const int32_t *positions, const float *inv_freq,
                    uint16_t *q_out, uint16_t *k_out, const ssm2d_rope_shape *shape, uint32_t flags, void *stream);

/* ---- Gated delta rule ------------------------------------------------------
 *
 * A linear recurrence over tokens with a matrix state S [d_k][d_v] per head,
 * the sequence relative of the 2D scan: the state decays, what it answers to
 * the key k is corrected towards v, and q reads it:
 *   S' = exp(g[t]) S;   u = beta[t] (v[t] - S'^T k[t]);   S = S' + k[t] u^T
 *   o[t] = scale S^T q[t]
 * q, k: [batch][tokens][heads_qk][d_k]; v: [batch][tokens][heads][d_v]; heads is
 * a multiple of heads_qk, head h reads query and key head h / (heads /
 * heads_qk); g (log decay, usually <= 0; -inf clears the state), beta:
 * float32 [batch][tokens][heads]; inner stride 1 except g and beta, whose
 * three strides are free. o: dense [batch][tokens][heads][d_v].
 * Packed sequences (n_seq > 0): batch = 1, and sequence s is tokens
 * cu_seqlens[s] .. cu_seqlens[s + 1] - 1 of the `tokens` ones (device int32
 * [n_seq + 1], ascending from 0 to tokens; sequences may be empty; entries
 * are clamped to 0 .. tokens, so no value makes a call read or write out of
 * range). Else n_seq = 0, cu_seqlens is ignored and sequences = batch.
 * h_init (NULL: zeros), h_last (NULL: not stored): float32
 * [sequences][heads][d_k][d_v], the state before the first and after the last
 * token; an empty sequence passes its state on. h_last may be h_init.
 * Limits: d_k <= SSM2D_DELTA_MAX_DK, d_v <= SSM2D_DELTA_MAX_DV, sequences *
 * heads < 2^24 (2^23 beyond the few tokens below), heads < 2^15, tokens < 2^31 - 64, chunks of 64 tokens < 2^22, and
 * token strides of v and dout in 0 .. 2^26 - 1.
 *
 * The forward and backward work on chunks of 64 tokens with matrix
 * instructions: products of fp32 operands split into three bf16 parts each, so
 * that states and sums keep fp32's precision, those that make a bf16 output
 * too. A NaN or Inf at a token may reach the other tokens of its chunk, but no
 * chunk before. Up to 8 tokens (bf16; 16 of float32) go through the recurrence
 * itself.
 * Heads of no keys or no values give zeros. */
#define SSM2D_DELTA_MAX_DK 128
#define SSM2D_DELTA_MAX_DV 1024

typedef struct {
    int64_t batch, tokens, n_seq;
    int64_t heads_qk, heads, d_k, d_v;
    int64_t q_stride[3], k_stride[3], v_stride[3], do_stride[3]; /* batch, token, head */
    int64_t g_stride[3], beta_stride[3];
} ssm2d_delta_shape;

int ssm2d_gated_delta_fwd(const float *q, const float *k, const float *v, const float *g, const float *beta,
                          const float *h_init, const int32_t *cu_seqlens, float *o, float *h_last,
                          const ssm2d_delta_shape *shape, float scale, void *stream);
int ssm2d_gated_delta_fwd_bf16(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *g,
                               const float *beta, const float *h_init, const int32_t *cu_seqlens, uint16_t *o,
                               float *h_last, const ssm2d_delta_shape *shape, float scale, void *stream);

/* Gradients of a loss through gated_delta_fwd, given dout = dL/do (like v,
 * strides do_stride) and dh_last = dL/dh_last (NULL: zeros): dq, dk (dense
 * [batch][tokens][heads_qk][d_k], summed over the heads that share them), dv
 * (dense like v), dg, dbeta (dense float32 [batch][tokens][heads]) and dh_init
 * (NULL: not stored; like h_init, may be dh_last). The forward's chunk states
 * are computed again. Workspaces: per head and chunk of 64 tokens, with
 * d_k' = d_k rounded up to 32, 64 or 128 and d_v' = d_v to a multiple of 32,
 * 21760 bytes for the forward and 21760 + 4 (2 d_k' + 192) d_v' for the backward,
 * and 512 d_k' per chunk and key head that several heads share (backward); packed
 * sequences count as tokens / 64 + n_seq chunks. Where few or long sequences are
 * cut into segments, per head and segment d_k' (6 d_k' + 4 d_v') bytes, twice that
 * for the backward: at most one segment for every 4 chunks and 256 in all for a
 * sequence, at most 512 for all of a packed batch. Heads are taken in passes that
 * keep all of this within 16 GiB where one key head's allows. */
int ssm2d_gated_delta_bwd(const float *q, const float *k, const float *v, const float *g, const float *beta,
                          const float *h_init, const int32_t *cu_seqlens, const float *dout, const float *dh_last,
                          float *dq, float *dk, float *dv, float *dg, float *dbeta, float *dh_init,
                          const ssm2d_delta_shape *shape, float scale, void *stream);
int ssm2d_gated_delta_bwd_bf16(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *g, const float *beta,
                               const float *h_init, const int32_t *cu_seqlens, const uint16_t *dout,
                               const float *dh_last, uint16_t *dq, uint16_t *dk, uint16_t *dv, float *dg, float *dbeta,
                               float *dh_init, const ssm2d_delta_shape *shape, float scale, void *stream);

/* The recurrence token by token, for serving: the state stays in fp32 in
 * `state` ([batch][heads][d_k][d_v], read and rewritten in place). Any number
 * of tokens; meant for one or a few. Not for packed sequences (n_seq != 0 ->
 * SSM2D_ERR_BAD_FLAGS). */
int ssm2d_gated_delta_step(const float *q, const float *k, const float *v, const float *g, const float *beta,
                           float *state, float *o, const ssm2d_delta_shape *shape, float scale, void *stream);
int ssm2d_gated_delta_step_bf16(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *g,
                                const float *beta, float *state, uint16_t *o, const ssm2d_delta_shape *shape,
                                float scale, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM2D_OPS_H */
