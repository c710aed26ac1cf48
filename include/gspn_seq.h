/*
 * gspn_seq.h -- token-sequence operators of libgspn (sm_100a): a short causal convolution, a
 * selective state space scan and the norms around a block. They are for sequences what the
 * propagation of gspn.h is for maps: a gated linear recurrence with learned, input-dependent
 * weights, and what a block needs beside it.
 *
 * Common rules (those of gspn.h unless said otherwise):
 *   - Sequences are B x L x C, channels side by side. Where a descriptor has strides, `*_row` and
 *     `*_tok` are the elements between rows (B) and tokens (L) of that input, so that slices of a
 *     wider projection are read in place; every other tensor is contiguous.
 *   - Packed sequences: `cu` (device, S + 1 ints, non-decreasing) gives sequence q the tokens
 *     cu[q] .. cu[q+1]-1 of the one row (B = 1); empty sequences are allowed. Without it S = 0 and
 *     the B rows are the sequences. Entries outside [0, L] are clamped. Tokens before cu[0] and
 *     from cu[S] on are not read and their outputs are left as they were.
 *   - Storage dtype GSPN_F32 or GSPN_BF16 for activations; parameters (A, D, dt_bias, w, bias, norm
 *     weights, scale), scan states and parameter gradients are fp32 for both. Arithmetic is fp32
 *     and each output is rounded once.
 *   - L and rows may be 0. Every other size is at least 1.
 *   - Outputs overlap neither inputs nor each other, except where a call says so.
 *   - B * L < 2^31 and L <= 2^30; beyond what a launch can count, GSPN_ERR_UNSUPPORTED.
 *   - Pointers must be aligned to their element; 16-byte aligned rows take the wide loads. The
 *     workspace must be 16-byte aligned. A call whose workspace size is 256 needs none of it and
 *     takes a null workspace.
 *   - Nothing is allocated, kept or synchronised; repeated calls give the same bits.
 */
#ifndef GSPN_SEQ_H
#define GSPN_SEQ_H

#include "gspn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- causal convolution
 *   u_t = bias + sum_{k<K} w[c][k] x_{t-K+1+k},   y_t = u_t or u_t sigmoid(u_t) (silu = 1).
 * What lies before a sequence is state0 (S x K-1 x C, oldest first; null: zeros). w: C x K, bias: C
 * or null. */
typedef struct {
    int B, L, C, K;          /* K = 2..4 taps */
    int S;                   /* packed sequences (0: none) */
    int dtype;               /* gspn_dtype */
    int silu;                /* 1: y = silu(u), 0: y = u */
    long long x_row, x_tok;  /* strides of x */
} gspn_conv_desc;

GSPN_API size_t gspn_conv_workspace_size(const gspn_conv_desc *desc, int for_backward);

/* y: B x L x C. state (S or B x K-1 x C, storage dtype, or null) receives the last K-1 inputs of
 * every sequence; it may be state0 itself, and must not overlap it otherwise. */
GSPN_API gspn_status gspn_conv_forward(const gspn_conv_desc *desc, const void *x, const float *w,
                                       const float *bias, const int *cu, const void *state0, void *y,
                                       void *state, void *stream);

/* Gradients of sum(dy y) + sum(dstate state): dx (B x L x C), dw (C x K), dbias (C, or null),
 * dstate0 (or null). dy: B x L x C contiguous; dstate may be null. */
GSPN_API gspn_status gspn_conv_backward(const gspn_conv_desc *desc, const void *x, const float *w,
                                        const float *bias, const int *cu, const void *state0, const void *dy,
                                        const void *dstate, void *dx, float *dw, float *dbias, void *dstate0,
                                        void *ws, size_t ws_bytes, void *stream);

/* One token for each of desc->B rows (desc->L = 1, x_tok unused): y B x C; state: slots x K-1 x C,
 * updated in place. idx (device, B ints, or null: row b has slot b) names each row's slot; a row
 * whose index is outside [0, slots) is skipped and its y left as it was. Rows that name one slot
 * take their tokens in row order. At most 65535 rows. */
GSPN_API gspn_status gspn_conv_step(const gspn_conv_desc *desc, const void *x, const float *w, const float *bias,
                                    const int *idx, int slots, void *state, void *y, void *stream);

/* ---------------------------------------------------------------- selective scan
 *   d = dt + dt_bias, through log(1 + exp(d)) if softplus = 1;
 *   h_t[c][n] = exp(d_t[c] A[c][n]) h_{t-1}[c][n] + d_t[c] x_t[c] Bm_t[g][n],  g = c / (C / G);
 *   y_t[c] = (sum_n Cm_t[g][n] h_t[c][n] + D[c] x_t[c]) * silu(z_t[c]).
 * x, dt, z: B x L x C; Bm, Cm: B x L x G x N (G x N contiguous per token); A: C x N; D, dt_bias: C.
 * z, D, dt_bias, h0 may be null. h0, h: S (or B) x C x N fp32. G divides C; 1 <= N <= 64. A row's
 * steps d should be >= 0 and A <= 0, as trained models keep them; the formula is evaluated as it
 * stands otherwise. */
typedef struct {
    int B, L, C, G, N;
    int S;                   /* packed sequences (0: none) */
    int dtype;               /* gspn_dtype */
    int softplus;            /* 1: d = log(1 + exp(dt + dt_bias)) */
    long long x_row, x_tok, dt_row, dt_tok, z_row, z_tok, b_row, b_tok, c_row, c_tok;
} gspn_ssm_desc;

GSPN_API size_t gspn_ssm_workspace_size(const gspn_ssm_desc *desc, int for_backward);

/* Bytes of the states that the training forward keeps for the backward pass (every 16th token's). */
GSPN_API size_t gspn_ssm_hsave_size(const gspn_ssm_desc *desc);

/* y: B x L x C; h (or null) receives the state behind every sequence's last token (h0, or zeros, for
 * an empty one); h may be h0. hsave (or null): gspn_ssm_hsave_size bytes for gspn_ssm_backward. */
GSPN_API gspn_status gspn_ssm_forward(const gspn_ssm_desc *desc, const void *x, const void *dt, const float *A,
                                      const void *Bm, const void *Cm, const float *D, const void *z,
                                      const float *dt_bias, const int *cu, const float *h0, void *y, float *h,
                                      float *hsave, void *ws, size_t ws_bytes, void *stream);

/* Gradients of sum(dy y) + sum(dh h). dy: B x L x C contiguous; dh may be null; hsave comes from
 * gspn_ssm_forward on the same inputs. dx, ddt, dz: B x L x C; dA: C x N; dBm, dCm: B x L x G x N;
 * dD, ddt_bias: C. dz goes with z (both or neither); dD, ddt_bias and dh0 may be null. */
GSPN_API gspn_status gspn_ssm_backward(const gspn_ssm_desc *desc, const void *x, const void *dt, const float *A,
                                       const void *Bm, const void *Cm, const float *D, const void *z,
                                       const float *dt_bias, const int *cu, const float *hsave, const void *dy,
                                       const float *dh, void *dx, void *ddt, float *dA, void *dBm, void *dCm,
                                       float *dD, void *dz, float *ddt_bias, float *dh0, void *ws,
                                       size_t ws_bytes, void *stream);

/* One token for each of desc->B rows (desc->L = 1, *_tok unused): y B x C; h: slots x C x N, updated
 * in place; idx and slots as for gspn_conv_step. C * N < 2^30. */
GSPN_API gspn_status gspn_ssm_step(const gspn_ssm_desc *desc, const void *x, const void *dt, const float *A,
                                   const void *Bm, const void *Cm, const float *D, const void *z,
                                   const float *dt_bias, const int *idx, int slots, float *h, void *y,
                                   void *stream);

/* ---------------------------------------------------------------- norms around a block
 *   v = y silu(gate);  v = norm(v) w_post + b_post;  r_out = r + scale v;  o = norm(r_out) w_pre + b_pre
 * for each of `rows` rows of C values, with norm(v) = v / sqrt(mean(v^2) + eps), of v - mean(v) if
 * center = 1. Left out where the pointer is null: gate; the norm behind the block (w_post); r;
 * scale; the norm before the next block (w_pre, then o is null too). b_post and b_pre need their
 * weight. r and r_out are of res_dtype: GSPN_F32, or dtype. o is computed from r_out before it is
 * rounded; r_out may be r itself (with r_row = C). C <= 16384. */
typedef struct {
    int rows, C;
    int dtype;               /* gspn_dtype of y, gate, o */
    int res_dtype;           /* gspn_dtype of r, r_out */
    int center;
    float eps;
    long long y_row, gate_row, r_row;   /* elements between rows of y, gate, r */
} gspn_norm_desc;

GSPN_API size_t gspn_norm_workspace_size(const gspn_norm_desc *desc, int for_backward);

GSPN_API gspn_status gspn_norm_forward(const gspn_norm_desc *desc, const void *y, const void *gate,
                                       const float *w_post, const float *b_post, const float *scale,
                                       const void *r, const float *w_pre, const float *b_pre, void *r_out,
                                       void *o, void *stream);

/* Gradients of sum(dr r_out) + sum(go o), given r_out as the forward left it (r_row is its row
 * stride): dy, dr_in (the gradient of r, res_dtype), dgate, dw_post, db_post, dscale, dw_pre, db_pre.
 * dr (or null), go: rows x C contiguous, dr of res_dtype. go and r_out go with w_pre. Each output
 * but dy may be null, and has to be where its input is null (dr_in excepted). Rows over 4096 columns have their
 * column sums in shared memory: asked for more than 200 KB of them, the call returns GSPN_ERR_UNSUPPORTED (all
 * five fit up to 10240 columns, four up to 12800, three up to 16384; the others take a second call). */
GSPN_API gspn_status gspn_norm_backward(const gspn_norm_desc *desc, const void *y, const void *gate,
                                        const float *w_post, const float *b_post, const float *scale,
                                        const void *r_out, const float *w_pre, const void *dr, const void *go,
                                        void *dy, void *dr_in, void *dgate, float *dw_post, float *db_post,
                                        float *dscale, float *dw_pre, float *db_pre, void *ws, size_t ws_bytes,
                                        void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GSPN_SEQ_H */
