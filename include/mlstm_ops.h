/*
 * mlstm_ops.h -- C ABI of the operators that stand beside the mLSTM cell:
 * linear attention with a decay for each head, the gated delta rule, group norm
 * with an activation, and the norm and rotation of queries and keys.
 *
 * Linear attention keeps the mLSTM cell's matrix memory without its input
 * gate, normaliser and stabilizer; the forget gate is one constant per head.
 * With g = log_decay[h] <= 0 and s = scale:
 *
 *   S_t = e^g S_{t-1} + k_t v_t^T   [d_qk x d_v, key index first],
 *   o_t = s q_t^T S_t.
 *
 * The gated delta rule keeps the same memory and takes out of it what a key
 * already recalls before it writes; log decay g_t and strength beta_t come with
 * each token, as the cell's gates do:
 *
 *   S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,
 *   o_t = s q_t^T S_t.
 *
 * Group norm normalises the output of each head (or group of channels):
 * z = weight (x - mean) / sqrt(var + eps) + bias, y = act(z).
 *
 * The conventions of mlstm.h hold: device pointers, 16-byte aligned
 * (MLSTM_ERR_ALIGN), host-side checks before any device work, no allocation,
 * no synchronisation, work enqueued on `stream`, status codes of
 * mlstm_status_t.  io is MLSTM_F32 or MLSTM_BF16; log_decay, states,
 * statistics, weights, biases and their gradients are float32.  Results are
 * deterministic: the same call gives the same bits.
 *
 * Strides.  q, k, v, o, their gradients, x and y are four-dimensional with
 * a unit last stride and the other three strides given in elements; a NULL
 * stride array means dense, C-contiguous tensors.  Strides of linear attention
 * are multiples of 16 bytes (MLSTM_ERR_ALIGN otherwise).  They are >= 0.  Along
 * a dimension of size 1 a stride is ignored.  An input may repeat rows along
 * the first and second dimension (stride 0).  An output's elements must not
 * overlap one another, and its extent (first to last byte) must not overlap
 * the extent of any other argument (MLSTM_ERR_ALIAS); a layout whose
 * dimensions do not nest by rising stride is taken for an overlap.
 *
 * Workspaces are scratch: nothing is kept in them, and two calls that may run
 * at the same time (other streams, overlapping graphs) need separate ones.
 */
#ifndef MLSTM_OPS_H
#define MLSTM_OPS_H

#include "mlstm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element strides of the first three dimensions of a tensor whose last
 * dimension is contiguous. */
typedef struct {
    long long s0, s1, s2;
} mlstm_strides_t;

/*
 * Linear attention over whole sequences (prefill), in its chunked form.
 *
 *  q, k       [B, H, T, d_qk]  io dtype      v, o  [B, H, T, d_v]  io dtype
 *  log_decay  [H]              float32, g <= 0; -inf is a decay of 0
 *  S0         [B, H, d_qk, d_v] float32, dense, or NULL for the zero state
 *  lengths    [B] int32 on the device, or NULL.  Sequence b has
 *             min(max(lengths[b], 0), T) tokens; what its later rows of q, k
 *             and v hold (NaN included) does not matter, its later rows of o
 *             are written as zeros, and its final state is the one after its
 *             own last token (S0 itself if it has none)
 *  S_T        [B, H, d_qk, d_v] float32, dense, or NULL when not wanted; may
 *             be exactly S0 (updated in place)
 *  strides    4: of q, k, v, o over (b, h, t), or NULL.  The token stride is
 *             at least the row's length and at most 2^22 - 1.
 *  workspace  at least mlstm_linattn_fwd_workspace_size bytes (may be NULL
 *             when that is 0); contents on entry are irrelevant
 *
 * d_qk is a multiple of 16 up to 256 and d_v one up to 512, as for the cell
 * (MLSTM_ERR_UNSUPPORTED otherwise); 1 <= T <= 2^30, B, H >= 1 and
 * B * H < 2^19 (MLSTM_ERR_SHAPE).  q, k, v of a sequence's own tokens are
 * finite, and so are S0 and what they add up to, below 1e26 in magnitude (the
 * kernel holds the state scaled by up to 2^40); a NaN or an infinity reaches
 * the outputs of its own 32-token chunk and everything after it.
 *
 * Precision.  float32: float32 products and sums.  bfloat16: o is rounded once,
 * at the end; the scores and the read-out's copy of the state keep 16 bits, a
 * state that is handed out is exact to float32 sums.  (Without S_T the carried
 * state keeps 16 bits of each decayed product, so o may differ in its last bit
 * from that of a call with S_T.)
 */
mlstm_status_t mlstm_linattn_fwd_workspace_size(int B, int H, int T, int d_qk, int d_v,
                                                mlstm_dtype_t io, size_t *bytes);
mlstm_status_t mlstm_linattn_fwd(const void *q, const void *k, const void *v,
                                 const float *log_decay, const float *S0, const int *lengths,
                                 void *o, float *S_T, const mlstm_strides_t *strides, float scale,
                                 int B, int H, int T, int d_qk, int d_v, mlstm_dtype_t io,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * One token of the recurrence for B*H heads (decode).
 *
 *  q, k  [B, H, d_qk]   v, o  [B, H, d_v]  io dtype;  log_decay [H] float32
 *  S_in  [B, H, d_qk, d_v] float32, dense, or NULL for the zero state
 *  S_out same shape, required; may be exactly S_in (updated in place)
 *  strides    4: of q, k, v, o over (b, h) in s0, s1 (s2 is ignored), or NULL
 */
mlstm_status_t mlstm_linattn_step(const void *q, const void *k, const void *v,
                                  const float *log_decay, const float *S_in, void *o, float *S_out,
                                  const mlstm_strides_t *strides, float scale, int B, int H,
                                  int d_qk, int d_v, mlstm_dtype_t io, void *stream);

/*
 * Gradients of a loss with respect to q, k, v and S0 of mlstm_linattn_fwd,
 * given those with respect to o and, where the final state was used, S_T.
 * (log_decay is a constant of the model and gets none.)
 *
 *  d_o        [B, H, T, d_v] io dtype;  dS_T [B, H, d_qk, d_v] float32 or NULL (zero)
 *  dq, dk     [B, H, T, d_qk], dv [B, H, T, d_v]  io dtype, each rounded once
 *             from float32; rows behind a sequence's length are written as zeros
 *             (what d_o holds there does not matter)
 *  dS0        [B, H, d_qk, d_v] float32, or NULL when not wanted (written
 *             for a NULL S0 too: the gradient at the zero state)
 *  strides    7: of q, k, v, d_o, dq, dk, dv over (b, h, t), or NULL.  An input
 *             that repeats rows over b or h gets one gradient row for each
 *             (b, h): the caller sums them.
 * Everything else as for mlstm_linattn_fwd, the precision too.  Without dS0 what
 * is carried keeps 16 bits of each decayed product: a bfloat16 dv may differ in
 * its last bit from that of a call with dS0, and so may dq and dk where d_qk and
 * d_v are padded to the same width (64, 128, 256 or 512).
 */
mlstm_status_t mlstm_linattn_bwd_workspace_size(int B, int H, int T, int d_qk, int d_v,
                                                mlstm_dtype_t io, size_t *bytes);
mlstm_status_t mlstm_linattn_bwd(const void *q, const void *k, const void *v,
                                 const float *log_decay, const float *S0, const int *lengths,
                                 const void *d_o, const float *dS_T, void *dq, void *dk, void *dv,
                                 float *dS0, const mlstm_strides_t *strides, float scale, int B,
                                 int H, int T, int d_qk, int d_v, mlstm_dtype_t io,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * The gated delta rule over whole sequences (prefill).
 *
 *  q, k       [B, Hk, T, d_qk] io dtype      v, o  [B, H, T, d_v]  io dtype
 *             H is a multiple of Hk: head h of v reads head h / (H / Hk) of q and k
 *  log_decay  [B, H, T] float32, g <= 0; -inf forgets everything before the token
 *  beta       [B, H, T] float32
 *  S0, S_T    [B, H, d_qk, d_v] float32, dense, or NULL, as for mlstm_linattn_fwd
 *  lengths    [B] int32 or NULL, as for mlstm_linattn_fwd; the gates of later rows
 *             do not matter either
 *  strides    6: of q, k, v, log_decay, beta, o over (b, h, t), or NULL.  Those of
 *             log_decay and beta are free (0 repeats a value), and these two need
 *             4-byte alignment only.  The others are as for mlstm_linattn_fwd.
 *  workspace  at least mlstm_deltarule_fwd_workspace_size bytes
 *
 * Limits of B, H, T, d_qk and d_v are those of mlstm_linattn_fwd, 1 <= Hk <= H, and
 * the workspace below 2^40 bytes (MLSTM_ERR_SHAPE).
 * Values of a sequence's own tokens are finite but for g = -inf (a log decay
 * below -700 counts as -inf), and so is what they add up to, below 1e26 in
 * magnitude.  The recurrence itself is stable where 0 <= beta |k|^2 <= 2: keys of
 * unit length, as mlstm_qknorm_fwd makes them.  A NaN or an infinity reaches the
 * outputs of its own 32-token chunk and everything after it.
 *
 * Precision.  As for mlstm_linattn_fwd: float32 products and sums for float32;
 * for bfloat16 o is rounded once, the scores, what is written and the read-out's copy of
 * the state keep 16 bits each, and a state that is handed out is exact to float32 sums.
 */
mlstm_status_t mlstm_deltarule_fwd_workspace_size(int B, int Hk, int H, int T, int d_qk, int d_v,
                                                  mlstm_dtype_t io, size_t *bytes);
mlstm_status_t mlstm_deltarule_fwd(const void *q, const void *k, const void *v,
                                   const float *log_decay, const float *beta, const float *S0,
                                   const int *lengths, void *o, float *S_T,
                                   const mlstm_strides_t *strides, float scale, int B, int Hk, int H,
                                   int T, int d_qk, int d_v, mlstm_dtype_t io, void *workspace,
                                   size_t workspace_bytes, void *stream);

/*
 * One token of the gated delta rule for B*H heads (decode).
 *
 *  q, k  [B, Hk, d_qk]   v, o  [B, H, d_v]  io dtype;  log_decay, beta [B, H] float32
 *  S_in  [B, H, d_qk, d_v] float32, dense, or NULL for the zero state
 *  S_out same shape, required; may be exactly S_in (updated in place)
 *  strides    6: of q, k, v, log_decay, beta, o over (b, h) in s0, s1 (s2 is ignored), or NULL
 */
mlstm_status_t mlstm_deltarule_step(const void *q, const void *k, const void *v,
                                    const float *log_decay, const float *beta, const float *S_in,
                                    void *o, float *S_out, const mlstm_strides_t *strides,
                                    float scale, int B, int Hk, int H, int d_qk, int d_v,
                                    mlstm_dtype_t io, void *stream);

/*
 * Gradients of a loss with respect to every input of mlstm_deltarule_fwd, given
 * those with respect to o and, where the final state was used, S_T.
 *
 *  d_o         [B, H, T, d_v] io dtype;  dS_T [B, H, d_qk, d_v] float32 or NULL (zero)
 *  dq, dk      [B, Hk, T, d_qk], dv [B, H, T, d_v]  io dtype, each rounded once; dq
 *              and dk are summed over the heads that share a row
 *  dlog_decay, dbeta  [B, H, T] float32.  The gradient at g = -inf is 0, as the
 *              decay e^g there.  Rows of all five behind a sequence's length are
 *              written as zeros.
 *  dS0         [B, H, d_qk, d_v] float32, or NULL when not wanted (written for a
 *              NULL S0 too)
 *  strides     11: of q, k, v, log_decay, beta, d_o, dq, dk, dv, dlog_decay, dbeta
 *              over (b, h, t), or NULL
 * Everything else as for mlstm_deltarule_fwd, the precision too; dlog_decay, dbeta and dS0
 * are exact to float32 sums in bfloat16 calls as well.
 */
mlstm_status_t mlstm_deltarule_bwd_workspace_size(int B, int Hk, int H, int T, int d_qk, int d_v,
                                                  mlstm_dtype_t io, size_t *bytes);
mlstm_status_t mlstm_deltarule_bwd(const void *q, const void *k, const void *v,
                                   const float *log_decay, const float *beta, const float *S0,
                                   const int *lengths, const void *d_o, const float *dS_T, void *dq,
                                   void *dk, void *dv, float *dlog_decay, float *dbeta, float *dS0,
                                   const mlstm_strides_t *strides, float scale, int B, int Hk, int H,
                                   int T, int d_qk, int d_v, mlstm_dtype_t io, void *workspace,
                                   size_t workspace_bytes, void *stream);

typedef enum {
    MLSTM_ACT_NONE = 0,
    MLSTM_ACT_SILU = 1, /* z / (1 + e^-z) */
    MLSTM_ACT_GELU = 2  /* z Phi(z), Phi the normal distribution function */
} mlstm_act_t;

/* What one mean and variance is taken over. */
typedef enum {
    MLSTM_NORM_TOKEN = 0,   /* the D channels of a group at one position */
    MLSTM_NORM_SEQUENCE = 1 /* the D channels of a group at all S positions */
} mlstm_norm_over_t;

/*
 * Group norm with an activation, channels last: x [N, S, G, D] has N samples,
 * S positions, G groups and D channels in each group.
 *
 *  x, y          [N, S, G, D] io dtype, strides over (n, s, g): 2 (x, y) or NULL
 *  weight, bias  [G, D] float32, dense; each may be NULL (ones, zeros)
 *  mean, rstd    [N, S, G] (over tokens) or [N, G] (over sequences) float32,
 *                dense: the statistics that the backward takes.  Both NULL when
 *                not wanted, else both given (MLSTM_ERR_NULL).  The variance is the biased one.
 *  eps           > 0 (MLSTM_ERR_UNSUPPORTED otherwise)
 *  workspace     at least mlstm_groupnorm_workspace_size bytes, or NULL if that is 0
 *
 * N, S, G, D >= 1, any D; N * S, G * D and N * G below 2^30 and N * ceil(G D / 64)
 * below 2^28 (MLSTM_ERR_SHAPE).
 * D and the strides being multiples of 16 bytes makes it faster, and is not
 * required.  y may not be x.
 *
 * Precision.  float32 throughout, results rounded once.  The activations keep
 * relative precision over their whole range: SiLU's and Phi's relative errors are
 * below (8 + 1.5 |z|) 2^-24 and (16 + 1.3 z^2) 2^-24.  A group of one float32 value
 * throughout has exactly that value as its mean.
 */
mlstm_status_t mlstm_groupnorm_workspace_size(int N, int S, int G, int D, mlstm_norm_over_t over,
                                              mlstm_dtype_t io, int backward, size_t *bytes);
mlstm_status_t mlstm_groupnorm_fwd(const void *x, const float *weight, const float *bias, void *y,
                                   float *mean, float *rstd, const mlstm_strides_t *strides, int N,
                                   int S, int G, int D, mlstm_norm_over_t over, mlstm_act_t act,
                                   float eps, mlstm_dtype_t io, void *workspace,
                                   size_t workspace_bytes, void *stream);

/*
 * Gradients of mlstm_groupnorm_fwd, given dy and the forward's mean and rstd.
 *
 *  dx               [N, S, G, D] io dtype;  strides: 3, of x, dy and dx, or NULL
 *  dweight, dbias   [G, D] float32 (written, not added to); each may be NULL
 *                   when not wanted
 */
mlstm_status_t mlstm_groupnorm_bwd(const void *x, const void *dy, const float *mean,
                                   const float *rstd, const float *weight, const float *bias,
                                   void *dx, float *dweight, float *dbias,
                                   const mlstm_strides_t *strides, int N, int S, int G, int D,
                                   mlstm_norm_over_t over, mlstm_act_t act, mlstm_dtype_t io,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* What a row of queries or keys is divided by. */
typedef enum {
    MLSTM_QKNORM_NONE = 0, /* nothing */
    MLSTM_QKNORM_RMS = 1,  /* sqrt(mean x^2 + eps) */
    MLSTM_QKNORM_L2 = 2    /* sqrt(sum x^2 + eps) */
} mlstm_qknorm_t;

/* Which channels of the first 2 n make the n pairs that are rotated. */
typedef enum {
    MLSTM_ROTARY_HALF = 0, /* channels i and i + n */
    MLSTM_ROTARY_PAIRS = 1 /* channels 2 i and 2 i + 1 */
} mlstm_rotary_t;

/*
 * Norm of each head's queries and keys, and their rotation by the token's
 * position, in one pass:
 *
 *   z = weight x / norm(x),   (y_a, y_b) = A (z_a cos w - z_b sin w, z_b cos w + z_a sin w)
 *
 * with w = positions[b, t] inv_freq[i] for pair i (a, b) of the first 2 n_freq
 * channels; the other channels are z (without a norm and weights the input's own
 * bits, a NaN's aside, and so are their gradients).
 *
 *  q, yq        [B, H, T, d] io dtype;  k, yk  [B, Hk, T, d] io dtype, both NULL for
 *               queries alone (Hk is ignored then)
 *  q_weight, k_weight  [d] float32 or NULL (ones)
 *  inv_freq     [n_freq] float32, radians a position; 0 <= 2 n_freq <= d, NULL if
 *               n_freq is 0 (no rotation, A is not used either)
 *  positions    [B, T] int32, dense, or NULL for 0 ... T - 1
 *  amplitude    A
 *  strides      4: of q, k, yq, yk over (b, h, t), or NULL.  Any strides, and alignment
 *               to an element suffices; multiples of 16 bytes, d and n_freq too, are
 *               faster.  Tensors that interleave in one buffer with equal strides, as
 *               the queries and keys of a fused projection do, do not overlap here.
 *  eps          >= 0, > 0 for a norm of rows that may be zero
 *
 * 1 <= d <= 512 (MLSTM_ERR_UNSUPPORTED above); B * T * (H + Hk) below 2^31
 * (MLSTM_ERR_SHAPE).  yq may be exactly q (the same pointer and strides) and yk
 * exactly k.  Every row is computed, whatever the lengths of the sequences; a row
 * reaches no other's result.  With a norm the sum of a row's squares is finite in
 * float32, and at least 2^-100 if eps is 0; the sum of x times its gradient is finite too.
 *
 * Precision.  float32, the angle in 64 bits and reduced to a turn before its sine
 * is taken; results rounded once.
 */
mlstm_status_t mlstm_qknorm_fwd(const void *q, const void *k, const float *q_weight,
                                const float *k_weight, const float *inv_freq,
                                const int *positions, void *yq, void *yk,
                                const mlstm_strides_t *strides, int B, int H, int Hk, int T, int d,
                                int n_freq, mlstm_rotary_t layout, float amplitude,
                                mlstm_qknorm_t norm, float eps, mlstm_dtype_t io, void *stream);

/*
 * Gradients of mlstm_qknorm_fwd, given dyq and dyk.
 *
 *  dq, dk               as q and k, io dtype; dq may be exactly dyq and dk exactly dyk
 *  dq_weight, dk_weight [d] float32, written, each NULL when not wanted; summed in
 *                       an order that the sizes, strides and alignment fix
 *  strides              6: of q, k, dyq, dyk, dq, dk, or NULL
 *  workspace            at least mlstm_qknorm_bwd_workspace_size bytes, not needed if
 *                       both weight gradients are NULL
 */
mlstm_status_t mlstm_qknorm_bwd_workspace_size(int B, int H, int Hk, int T, int d, size_t *bytes);
mlstm_status_t mlstm_qknorm_bwd(const void *q, const void *k, const void *dyq, const void *dyk,
                                const float *q_weight, const float *k_weight, const float *inv_freq,
                                const int *positions, void *dq, void *dk, float *dq_weight,
                                float *dk_weight, const mlstm_strides_t *strides, int B, int H,
                                int Hk, int T, int d, int n_freq, mlstm_rotary_t layout,
                                float amplitude, mlstm_qknorm_t norm, float eps, mlstm_dtype_t io,
                                void *workspace, size_t workspace_bytes, void *stream);

/* How positions beyond the trained context are brought back into it. */
typedef enum {
    MLSTM_ROPE_PLAIN = 0,  /* not at all */
    MLSTM_ROPE_LINEAR = 1, /* every frequency divided by the factor */
    MLSTM_ROPE_BASE = 2,   /* a larger base: the slowest frequency is divided by the
                              factor, the fastest kept */
    MLSTM_ROPE_RAMP = 3    /* frequencies that make `fast` turns or more over the
                              trained context kept, those of `slow` turns or fewer
                              divided by the factor, a linear ramp over the pair
                              index between; amplitude 0.1 ln(factor) + 1 */
} mlstm_rope_scaling_t;

/*
 * The table inv_freq[i] = base^(-2 i / (2 n_freq)), scaled, and the amplitude that
 * goes with it.  On the HOST: inv_freq and amplitude are host pointers, computed in
 * 64 bits.  n_freq >= 1, base > 1, factor >= 1; MLSTM_ROPE_RAMP takes the trained
 * context's length >= 1 and fast > slow > 0 (ignored otherwise); MLSTM_ROPE_BASE
 * n_freq >= 2 (MLSTM_ERR_SHAPE; MLSTM_ERR_UNSUPPORTED for another scaling).
 */
mlstm_status_t mlstm_rope_frequencies(int n_freq, double base, mlstm_rope_scaling_t scaling,
                                      double factor, int context, double fast, double slow,
                                      float *inv_freq, float *amplitude);

#ifdef __cplusplus
}
#endif
#endif /* MLSTM_OPS_H */
