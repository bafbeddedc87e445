/*
 * mgs_tokens.h -- C ABI of the operators of libmgs on the path from a token to
 * the next one, beside the layers of mgs_layers.h, for training and for serving:
 *
 *   1. the embedding lookup with scaling, and the table's gradient;
 *   2. the gated linear recurrence: a vector state, learnt decays, gates from
 *      pre-activations (forward, backward, one step at a time);
 *   3. sampling of the next token from given uniform numbers.
 *
 * Element types, strides, alignment, sizes, memory, streams, errors and empty
 * tensors are as mgs_layers.h states them: fp32 or bf16 elements, strides that
 * count elements and may be 0 but not negative, device pointers, caller-owned
 * buffers and workspaces, no allocation, arguments checked before any HIP call.
 * The workspaces carry nothing from one call to the next and need not be
 * zero-filled, but for mgs_gated_*'s.  That one has to be zero-filled once, as those of
 * mgs.h, and again after any other operator's call has had it, and before one of mgs.h has
 * it: results may be wrong otherwise, with no error to show it.
 * Calls that share a workspace must not run concurrently.  A workspace for B sequences or
 * rows, T steps or n ids serves calls of fewer too.
 */
#ifndef MGS_TOKENS_H
#define MGS_TOKENS_H

#include "mgs_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------ embedding lookup with scaling, and its gradient --- */
/*
 *     y_n = scale W[ids[n]],      dW_v = scale (sum of dy_n over n with ids[n] == v).
 *   ids  : (n), int32 (id_bits == 32) or int64 (64).  An id outside 0..vocab-1
 *          (-1, say: padding) gives a row of zeros and no gradient;
 *   W    : (vocab,d), row stride w_stride;   y : (n,d) dense out.
 */
mgs_status mgs_embed_fwd(const void *ids, int id_bits, const void *W, void *y, int64_t n, int64_t vocab,
                         int64_t d, int64_t w_stride, float scale, int dtype, void *stream);

/* Workspace bytes of mgs_embed_bwd. */
mgs_status mgs_embed_workspace_size(int64_t n, int64_t vocab, int64_t d, size_t *bytes);

/*
 *   dy : (n,d) of dtype, row stride dy_stride;
 *   dW : (vocab,d) of dw_dtype, dense.  accumulate == 0: written whole, zeros
 *        where no id points; accumulate != 0: added to, rows of no id neither
 *        read nor written.
 * Sums are fp32, in an order that the ids fix, rounded once to dw_dtype.
 */
mgs_status mgs_embed_bwd(const void *ids, int id_bits, const void *dy, void *dW, int64_t n, int64_t vocab,
                         int64_t d, int64_t dy_stride, float scale, int accumulate, int dtype, int dw_dtype,
                         void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------ gated linear recurrence --- */
/*
 * For each sequence b and channel, with gates rho = sigmoid(r), iota = sigmoid(i):
 *     log a_t = -rate softplus(lam) rho_t,      a_t = 0 where reset[b][t] != 0,
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) iota_t x_t,      y_t = h_t,   t = 1..T,
 *     h_0 = h0 (zeros if h0 == NULL).
 *   x, r, i : (B,T,D), strides x_stride, r_stride, i_stride (of b, t);
 *   lam  : (D) fp32;
 *   h0, hT : (B,D) fp32, dense; hT (the state after the last step) may be NULL;
 *   lengths : (B) int32 or NULL, as mgs_linattn_fwd's;
 *   reset : (B,T) bytes, dense, or NULL: a step with a byte that is not zero
 *          starts a document (nothing before it reaches it, finite or not);
 *   y    : (B,T,D), dense out;
 *   states : (B, ceil(T / MGS_GATED_CHUNK), D) fp32 out, or NULL: the states
 *          ahead of steps 1, MGS_GATED_CHUNK + 1, ..., which the backward reads.
 * A value that is not finite reaches its own channel only, from its step to the
 * next document (an infinity may come out as NaN).  A sigmoid or a 1 - a^2 below 2^-126
 * counts as 0.
 * The workspace is zero-filled once before its first use; it serves forward and
 * backward calls of any sizes that fit it.
 * Envelope: B ceil(D / 128) ceil(T / 64) < 2^23.
 */
enum { MGS_GATED_CHUNK = 64 };

typedef struct {
    int64_t B, T, D;
    int dtype;             /* of x, r, i, dy, y, dx, dr, di */
    float rate;            /* not negative */
    int64_t x_stride[2], r_stride[2], i_stride[2], dy_stride[2];
} mgs_gated_desc;

/* Workspace bytes of mgs_gated_fwd (backward == 0), or enough for both
 * mgs_gated_fwd and mgs_gated_bwd (backward != 0). */
mgs_status mgs_gated_workspace_size(const mgs_gated_desc *desc, int backward, size_t *bytes);

mgs_status mgs_gated_fwd(const mgs_gated_desc *desc, const void *x, const void *r, const void *i,
                         const float *lam, const float *h0, const int32_t *lengths, const uint8_t *reset,
                         void *y, float *hT, float *states, void *workspace, size_t workspace_bytes,
                         void *stream);

/*
 * Gradients of mgs_gated_fwd for L = sum_t <dy_t, y_t> + <dhT, h_T>.  With
 * G_t = dy_t + a_{t+1} G_{t+1} (dhT added at the last step), beta = sqrt(1 - a^2):
 *     dx = G beta iota,      di = G beta x iota (1 - iota),
 *     dl = G (a h_{t-1} - iota x a^2 / beta)     (of log a; 0 where a document starts;
 *                                                 without the quotient where beta == 0),
 *     dr = dl log a (1 - rho),   dlam = -rate sigmoid(lam) sum dl rho,   dh0 = a_1 G_1.
 *   dy   : (B,T,D), strides dy_stride;  dhT : (B,D) fp32 or NULL;
 *   states : the forward's;
 *   dx, dr, di : (B,T,D), dense out (zeros past a length);  dlam : (D) fp32 out,
 *          summed over sequences and steps in a fixed order (zeros where there are
 *          none);  dh0 : (B,D) fp32 out or NULL.
 */
mgs_status mgs_gated_bwd(const mgs_gated_desc *desc, const void *x, const void *r, const void *i,
                         const float *lam, const void *dy, const float *dhT, const float *states,
                         const int32_t *lengths, const uint8_t *reset, void *dx, void *dr, void *di,
                         float *dlam, float *dh0, void *workspace, size_t workspace_bytes, void *stream);

/*
 * One step for each of B sequences, on a cache of states: h[slots[b]] becomes
 * the next state, and y_b is that state.
 *   desc: T is not read; the strides of t are not read;
 *   x, r, i : (B,D);  h : (n_slots,D) fp32, dense, updated in place;
 *   slots : as mgs_linattn_step's (idle: zeros in y_b);  y : (B,D) dense out.
 */
mgs_status mgs_gated_step(const mgs_gated_desc *desc, const void *x, const void *r, const void *i,
                          const float *lam, float *h, int64_t n_slots, const int32_t *slots, void *y,
                          void *stream);

/* --------------------------------------------------- sampling of a token --- */
/*
 * For each of B rows of vocab logits x and a uniform number u:
 *     w_i = exp((x_i - max x) / temperature);
 * of the order by (w descending, index ascending)
 *     the first top_k (0 or less: all),
 *     of these the fewest that hold at least top_p of their weight (one at
 *     least; top_p >= 1: all),
 *     of these the ones with w_i >= min_p (above 1: 1);
 * the token is the first, by index, at which the running sum of the kept weights
 * exceeds u times their sum.  temperature == 0 takes the first of the largest.
 *   logits : (B,vocab), row stride logits_stride;
 *   u    : (B) fp32, taken as 0 below 0 (and where NaN) and as the float before 1
 *          from 1 on;
 *   temperature, top_p, min_p (fp32), top_k (int32): (B) each, or NULL for the
 *          desc's number.  A temperature below 0 or NaN counts as 0, a top_p or
 *          min_p that is NaN as 1 or 0;
 *   token : (B) int64 out;
 *   logp : (B) fp32 out or NULL: the log of the token's share of the kept weight.
 * -inf is a forbidden token.  A row of nothing else, or with a NaN, has token -1
 * and logp -inf; where the largest is +inf, those that are share all the weight.
 * Weights and sums are fp64, in units of the largest weight.  Those that top_p compares are
 * rounded to multiples of 2^-43, whose sums are exact; of a row's kept weights up to 4096 go
 * into the sum that u is compared with as multiples of 2^-51 (off by 2^-39 in all at most);
 * a weight below 2^-1000 counts as none.  A call's answers are the same every time; in a
 * batch of another size, or of the other type, they may differ where u times the sum is within
 * 2^-39 of a token's end.
 * Envelope: vocab <= 2^20, B < 2^22.
 */
typedef struct {
    int64_t B, vocab, logits_stride;
    int dtype;             /* of the logits */
    int top_k;
    float temperature, top_p, min_p;
} mgs_sample_desc;

mgs_status mgs_sample_workspace_size(const mgs_sample_desc *desc, size_t *bytes);

mgs_status mgs_sample(const mgs_sample_desc *desc, const void *logits, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                      void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MGS_TOKENS_H */
