/*
 * mgs_layers.h -- C ABI of the layer operators of libmgs: what a recurrent
 * language model runs around and beside the scans of mgs.h, for training and
 * for serving.
 *
 *   1. linear attention with a decay for each head: a matrix state per head,
 *      chunked for prompts and training (forward, backward), one step at a
 *      time for generation;
 *   2. the root-mean-square norm with the residual's addition: forward,
 *      forward with an 8-bit output and its scales, backward;
 *   3. the global gradient norm over many tensors, and clipping by it.
 *
 * Memory, streams, errors and empty tensors are as mgs.h states them (device
 * pointers, caller-owned buffers and workspaces, no allocation, arguments
 * checked before any HIP call), with these differences:
 *   - elements are fp32 or bf16 as the dtype argument says (MGS_F32, MGS_BF16);
 *     states, decays, scales and norms are fp32 always;
 *   - where strides are arguments they count elements, the last index is
 *     dense, and a stride may be 0 (a broadcast input) but not negative;
 *   - pointers are aligned to their element.  Inputs and outputs whose
 *     addresses and strides are multiples of 16 bytes take wide accesses, any
 *     others the same kernels with narrow ones;
 *   - a tensor may pass 2^31 elements (the limit is 2^40, and 2^31 - 65 for each
 *     size).  Grids past what one launch takes (2^32 threads) go in several; with
 *     up to 2^31 / 3 segments of sequences and heads in a whole-sequence call, and
 *     2^28 sequences times heads in a step, beyond which MGS_ERR_UNSUPPORTED.
 * The workspaces here carry nothing from one call to the next and need not be
 * zero-filled; calls that share one must not run concurrently.
 */
#ifndef MGS_LAYERS_H
#define MGS_LAYERS_H

#include "mgs.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MGS_F32 = 0, MGS_BF16 = 1 };

/* --------------------------------- linear attention with a decay per head */
/*
 * For each sequence b and head h, with a state S (dv x dk):
 *     S_t = exp(g_t) S_{t-1} + v_t k_t^T,      o_t = scale S_t q_t,   t = 1..T,
 *     S_0 = S0 (zeros if S0 == NULL).
 *   q, k : (B,T,Hk,dk), strides q_stride, k_stride (of b, t, h);  head h reads
 *          query/key head h / (H / Hk), so Hk divides H;
 *   v    : (B,T,H,dv), strides v_stride;
 *   g    : log decays, fp32: (B,T,H) with strides g_stride, or (H) dense where
 *          decay_per_head != 0.  -inf clears a finite state exactly; NaN and +inf
 *          propagate.
 *   lengths : (B) int32 or NULL: steps t > lengths[b] are not read (whatever
 *          they hold); they leave the state as it is and get zeros in every
 *          output.  Values past T mean T, values below 0 mean 0.
 *   S0, ST : (B,H,dv,dk) fp32, dense; ST (the state after the last step) may
 *          be NULL.
 *   o    : (B,T,H,dv), dense.  States are fp32; a bf16 o is rounded from a sum
 *          whose terms are good to 2^-18.
 * An element of v that is not finite makes its column of o, and its row of the
 * state, not finite from its step on (NaN also where the sum would be infinite);
 * it touches no earlier step and no other column.
 * Envelope: 1 <= dk, dv <= 128.
 */
typedef struct {
    int64_t B, T, H, Hk, dk, dv;
    int dtype;             /* of q, k, v, do_, o, dq, dk_, dv_ */
    int decay_per_head;
    float scale;
    int64_t q_stride[3], k_stride[3], v_stride[3], do_stride[3], g_stride[3];
} mgs_linattn_desc;

/* Workspace bytes of mgs_linattn_fwd (backward == 0), or enough for both
 * mgs_linattn_fwd and mgs_linattn_bwd (backward != 0); the strides and the
 * scale are not read. */
mgs_status mgs_linattn_workspace_size(const mgs_linattn_desc *desc, int backward, size_t *bytes);

mgs_status mgs_linattn_fwd(const mgs_linattn_desc *desc, const void *q, const void *k, const void *v,
                           const float *g, const float *S0, const int32_t *lengths, void *o, float *ST,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradients of mgs_linattn_fwd for L = sum_t <do_t, o_t> + <dST, S_T>.  With
 * D_T = dST + scale do_T q_T^T, D_t = exp(g_{t+1}) D_{t+1} + scale do_t q_t^T:
 *     dq_t = scale S_t^T do_t,   dk_t = D_t^T v_t,   dv_t = D_t k_t,
 *     dg_t = exp(g_t) <D_t, S_{t-1}>,   dS0 = exp(g_1) D_1.
 * dq and dk_ are summed over the heads that share a query/key head; with
 * decay_per_head, dg is (H), summed over sequences and steps: zeros where there
 * are none (T == 0, or B == 0, which needs no workspace).  All sums run in a
 * fixed order.
 * dg is formed from sums over later steps, which end at the next cleared state
 * (exp(g) == 0 in fp32, where dg is zero): no step after it, whatever it holds,
 * touches dg before it.  Up to there a non-finite v or k makes dg of up to 512
 * steps before it non-finite too.
 *   do_ : (B,T,H,dv), strides do_stride;  dST : (B,H,dv,dk) or NULL;
 *   dq, dk_ : (B,T,Hk,dk), dv_ : (B,T,H,dv), dense out;
 *   dg : fp32, (B,T,H) dense or (H), out;  dS0 : (B,H,dv,dk) out or NULL.
 */
mgs_status mgs_linattn_bwd(const mgs_linattn_desc *desc, const void *q, const void *k, const void *v,
                           const float *g, const void *do_, const float *S0, const float *dST,
                           const int32_t *lengths, void *dq, void *dk_, void *dv_, float *dg, float *dS0,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * One step for each of B sequences, on a cache of states:
 *     S[slots[b]] <- exp(g_b) S[slots[b]] + v_b k_b^T,   o_b = scale S[slots[b]] q_b.
 *   desc: T is not read; the strides of t are not read;
 *   q, k : (B,Hk,dk), v : (B,H,dv), g : (B,H) or (H);
 *   S : (n_slots,H,dv,dk) fp32 dense, updated in place;
 *   slots : (B) int32, distinct, or NULL (sequence b has slot b).  A slot
 *           outside 0..n_slots-1 (-1, say) is idle: its o_b is zeros and no
 *           state is touched;
 *   o : (B,H,dv) dense out.
 */
mgs_status mgs_linattn_step(const mgs_linattn_desc *desc, const void *q, const void *k, const void *v,
                            const float *g, float *S, int64_t n_slots, const int32_t *slots, void *o,
                            void *stream);

/* ------------------- root-mean-square norm with the residual's addition --- */
/*
 * Per row of d elements, in fp32:
 *     h = x + residual (x alone if residual == NULL),
 *     rstd = 1 / sqrt(mean(h^2) + eps),      y = h rstd w.
 *   x, residual : (rows,d), strides x_stride, r_stride of the rows;  w : (d);
 *   y, h : (rows,d) dense out;  h (rounded to dtype) may be NULL;
 *   rstd : (rows) fp32 out or NULL (the backward reads it).
 * h may be the residual's own buffer where r_stride == d, or x's where
 * x_stride == d: an update in place.
 */
mgs_status mgs_rmsnorm_fwd(const void *x, const void *residual, const void *w, void *y, void *h, float *rstd,
                           int64_t rows, int64_t d, int64_t x_stride, int64_t r_stride, float eps, int dtype,
                           void *stream);

/*
 * The same with y in 8 bits (OCP e4m3, largest value 448) and a scale for each
 * row (group == 0) or for each `group` columns of a row (group == 128; the last
 * group of a row may be narrower):
 *     scale = max(max |y| over the group, 1e-30) / 448,   y8 = round(y / scale),
 * rounded to nearest, ties to even, from the fp32 quotient of the fp32 y and
 * scale.
 *   y8 : (rows,d) bytes out;  scale : (rows, group ? ceil(d / group) : 1) fp32 out.
 */
mgs_status mgs_rmsnorm_fwd_fp8(const void *x, const void *residual, const void *w, void *y8, float *scale,
                               void *h, int64_t rows, int64_t d, int64_t x_stride, int64_t r_stride, float eps,
                               int64_t group, int dtype, void *stream);

/* Workspace bytes of mgs_rmsnorm_bwd. */
mgs_status mgs_rmsnorm_workspace_size(int64_t rows, int64_t d, size_t *bytes);

/*
 * Gradients for L = <dy, y> + <dh, h> from the forward's h and rstd:
 *     dx = rstd (dy w - h rstd^2 mean(dy w h)) + dh   (the residual's gradient is the same),
 *     dw = sum over rows of dy h rstd, in a fixed order.
 *   dy, h, dh : (rows,d) dense; dh may be NULL;  dx : (rows,d) dense out, may
 *   be dy's or dh's own buffer;  dw : (d) fp32 out.
 * w and dw have d elements whatever rows is: both are required for rows == 0
 * too, which writes zeros to dw.
 */
mgs_status mgs_rmsnorm_bwd(const void *dy, const void *h, const void *w, const float *rstd, const void *dh,
                           void *dx, float *dw, int64_t rows, int64_t d, int dtype, void *workspace,
                           size_t workspace_bytes, void *stream);

/* ------------------------------------- global gradient norm and clipping --- */
/*
 * Over n tensors, each of sizes[i] elements of dtypes[i], dense:
 *     norm = sqrt(sum of squares over all of them),
 *     out_i = in_i c,   c = min(1, max_norm / (norm + 1e-6)).
 * in, out, sizes and dtypes are host arrays, read during the call; out[i] may
 * equal in[i] (in place), and no output may overlap anything else (so a tensor
 * that is listed twice cannot be scaled in place).  Squares and their
 * sum are fp64, in a fixed order; norm is rounded to fp32 once.  Where the norm
 * is not finite (an element is not, or it would be 2^126 or more, where 1 / norm
 * is no normal fp32 number) the tensors are passed through unscaled and norm
 * says so.  With out == NULL only the norm is computed.  max_norm < 0 or NaN is
 * refused.
 *   norm : one fp32 out.
 */
mgs_status mgs_clip_norm_workspace_size(int64_t n, const int64_t *sizes, size_t *bytes);

mgs_status mgs_clip_norm(int64_t n, const void *const *in, void *const *out, const int64_t *sizes,
                         const int *dtypes, float max_norm, float *norm, void *workspace,
                         size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MGS_LAYERS_H */
