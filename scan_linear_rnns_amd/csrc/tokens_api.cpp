// tokens_api.cpp -- the C ABI declared in include/mgs_tokens.h: argument
// validation and dispatch.  As in layers_api.cpp, every refusal comes before any
// HIP call.
#include "mgs_tokens.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "api_common.hpp"
#include "tokens.hpp"

namespace {

using mgs::any_alias;
using mgs::as_stream;
using mgs::check_workspace;
using mgs::hip_status;
using mgs::Range;

constexpr int64_t kMaxElems = int64_t(1) << 40;   // of one tensor
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1 - 64;
constexpr int64_t kMaxTiles = (int64_t(1) << 23) - 1;   // workgroups of 512 threads in one launch

int64_t bounded(std::initializer_list<int64_t> dims) { return mgs::bounded_product(dims, kMaxElems, kMaxDim); }

bool aligned_to(const void *p, size_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }

bool known_dtype(int dtype) { return dtype == MGS_F32 || dtype == MGS_BF16; }

size_t size_of(int dtype) { return dtype == MGS_BF16 ? 2 : 4; }

// Bytes from the first to past the last element of B x T rows of `cols`, or -1
// where a stride is negative or the span passes the limit.
int64_t span(int64_t B, int64_t T, int64_t cols, int64_t bs, int64_t ts, size_t size)
{
    if (bs < 0 || ts < 0) return -1;
    if (B == 0 || T == 0 || cols == 0) return 0;
    const int64_t n[2] = {B - 1, T - 1}, st[2] = {bs, ts};
    int64_t total = cols;
    for (int i = 0; i < 2; ++i) {
        int64_t x;
        if (__builtin_mul_overflow(n[i], st[i], &x) || __builtin_add_overflow(total, x, &total) ||
            total > (int64_t(1) << 58))
            return -1;
    }
    return total * static_cast<int64_t>(size);
}

// ---------------------------------------------------------------- embedding

mgs_status check_embed(int64_t n, int64_t vocab, int64_t d)
{
    if (n < 0 || vocab < 0 || d <= 0) return MGS_ERR_INVALID_VALUE;
    if (bounded({n, d}) < 0 || bounded({vocab, d}) < 0) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

mgs_status check_ids(const void *ids, int id_bits, int64_t n)
{
    if (id_bits != 32 && id_bits != 64) return MGS_ERR_UNSUPPORTED;
    if ((n > 0 && !ids) || !aligned_to(ids, id_bits / 8)) return MGS_ERR_INVALID_VALUE;
    return MGS_OK;
}

// --------------------------------------------------- gated linear recurrence

mgs_status check_gated(const mgs_gated_desc *d)
{
    if (!d) return MGS_ERR_INVALID_VALUE;
    if (d->B < 0 || d->T < 0 || d->D <= 0 || !(d->rate >= 0.0f) || std::isinf(d->rate)) return MGS_ERR_INVALID_VALUE;
    if (!known_dtype(d->dtype)) return MGS_ERR_UNSUPPORTED;
    if (bounded({d->B, d->T, d->D}) < 0 || bounded({d->B, d->D}) < 0) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

bool gated_grid_fits(const mgs::GatedGeom &g)
{
    return mgs::bounded_product({g.groups, g.tiles_f}, kMaxTiles, kMaxTiles) >= 0 &&
           mgs::bounded_product({g.groups, g.tiles_b}, kMaxTiles, kMaxTiles) >= 0;
}

// The ranges of x, r, i, lam (and dy if given) into in[0..]; their count, or -1
// where one is refused.
int gated_inputs(const mgs_gated_desc &d, int64_t T, const void *x, const void *r, const void *i, const float *lam,
                 const void *dy, Range *in)
{
    const size_t size = size_of(d.dtype);
    const void *p[4] = {x, r, i, dy};
    const int64_t *st[4] = {d.x_stride, d.r_stride, d.i_stride, d.dy_stride};
    int n = 0;
    for (int k = 0; k < (dy ? 4 : 3); ++k) {
        const int64_t bytes = span(d.B, T, d.D, st[k][0], st[k][1], size);
        if (bytes < 0 || (bytes > 0 && !p[k]) || !aligned_to(p[k], size)) return -1;
        in[n++] = Range{p[k], static_cast<size_t>(bytes)};
    }
    if (!lam || !aligned_to(lam, 4)) return -1;
    in[n++] = Range{lam, static_cast<size_t>(d.D) * 4};
    return n;
}

}  // namespace

extern "C" {

mgs_status mgs_embed_fwd(const void *ids, int id_bits, const void *W, void *y, int64_t n, int64_t vocab,
                         int64_t d, int64_t w_stride, float scale, int dtype, void *stream)
{
    if (mgs_status st = check_embed(n, vocab, d)) return st;
    if (!known_dtype(dtype)) return MGS_ERR_UNSUPPORTED;
    if (mgs_status st = check_ids(ids, id_bits, n)) return st;
    const size_t size = size_of(dtype);
    const int64_t table = span(1, vocab, d, 0, w_stride, size);
    if (table < 0 || (n > 0 && table > 0 && !W) || (n > 0 && !y)) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(W, size) || !aligned_to(y, size)) return MGS_ERR_INVALID_VALUE;
    const Range in[] = {{ids, static_cast<size_t>(n) * (id_bits / 8)}, {W, static_cast<size_t>(table)}};
    const Range out[] = {{y, static_cast<size_t>(n) * d * size}};
    if (any_alias(in, 2, out, 1)) return MGS_ERR_INVALID_VALUE;
    if (n == 0) return MGS_OK;
    return hip_status(mgs::launch_embed_fwd(ids, id_bits == 64, W, y, n, vocab, d, w_stride, scale, dtype,
                                            as_stream(stream)));
}

mgs_status mgs_embed_workspace_size(int64_t n, int64_t vocab, int64_t d, size_t *bytes)
{
    if (!bytes) return MGS_ERR_INVALID_VALUE;
    if (mgs_status st = check_embed(n, vocab, d)) return st;
    *bytes = mgs::embed_geometry(n, vocab, d).bytes;
    return MGS_OK;
}

mgs_status mgs_embed_bwd(const void *ids, int id_bits, const void *dy, void *dW, int64_t n, int64_t vocab,
                         int64_t d, int64_t dy_stride, float scale, int accumulate, int dtype, int dw_dtype,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_embed(n, vocab, d)) return st;
    if (!known_dtype(dtype) || !known_dtype(dw_dtype)) return MGS_ERR_UNSUPPORTED;
    if (mgs_status st = check_ids(ids, id_bits, n)) return st;
    const size_t size = size_of(dtype), out_size = size_of(dw_dtype);
    const int64_t rows = span(1, n, d, 0, dy_stride, size);
    if (rows < 0 || (rows > 0 && !dy) || (vocab > 0 && !dW)) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(dy, size) || !aligned_to(dW, out_size)) return MGS_ERR_INVALID_VALUE;
    const Range in[] = {{ids, static_cast<size_t>(n) * (id_bits / 8)}, {dy, static_cast<size_t>(rows)}};
    const Range out[] = {{dW, static_cast<size_t>(vocab) * d * out_size}};
    if (any_alias(in, 2, out, 1)) return MGS_ERR_INVALID_VALUE;
    if (vocab == 0 || (n == 0 && accumulate)) return MGS_OK;
    const mgs::EmbedGeom g = mgs::embed_geometry(n, vocab, d);
    if (mgs_status st = check_workspace(workspace, workspace_bytes, g.bytes)) return st;
    return hip_status(mgs::launch_embed_bwd(g, ids, id_bits == 64, dy, dW, n, vocab, d, dy_stride, scale,
                                            accumulate != 0, dtype, dw_dtype, workspace, as_stream(stream)));
}

mgs_status mgs_gated_workspace_size(const mgs_gated_desc *desc, int backward, size_t *bytes)
{
    if (!bytes) return MGS_ERR_INVALID_VALUE;
    if (mgs_status st = check_gated(desc)) return st;
    const mgs::GatedGeom g = mgs::gated_geometry(*desc, backward != 0);
    if (!gated_grid_fits(g)) return MGS_ERR_UNSUPPORTED;
    *bytes = g.bytes;
    return MGS_OK;
}

mgs_status mgs_gated_fwd(const mgs_gated_desc *desc, const void *x, const void *r, const void *i,
                         const float *lam, const float *h0, const int32_t *lengths, const uint8_t *reset,
                         void *y, float *hT, float *states, void *workspace, size_t workspace_bytes,
                         void *stream)
{
    if (mgs_status st = check_gated(desc)) return st;
    const mgs_gated_desc &d = *desc;
    Range in[8];
    int n = gated_inputs(d, d.T, x, r, i, lam, nullptr, in);
    if (n < 0) return MGS_ERR_INVALID_VALUE;
    const size_t state = static_cast<size_t>(d.B) * d.D * 4, steps = static_cast<size_t>(d.B) * d.T;
    const size_t ny = steps * d.D * size_of(d.dtype);
    const size_t saved = (d.T + MGS_GATED_CHUNK - 1) / MGS_GATED_CHUNK * state;
    if (ny > 0 && !y) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(y, size_of(d.dtype)) || !aligned_to(h0, 4) || !aligned_to(lengths, 4) || !aligned_to(hT, 4) ||
        !aligned_to(states, 4))
        return MGS_ERR_INVALID_VALUE;
    in[n++] = Range{h0, state};
    in[n++] = Range{lengths, static_cast<size_t>(d.B) * 4};
    in[n++] = Range{reset, steps};
    const Range out[] = {{y, ny}, {hT, state}, {states, saved}};
    if (any_alias(in, n, out, 3)) return MGS_ERR_INVALID_VALUE;
    if (d.B == 0 || (d.T == 0 && !hT)) return MGS_OK;
    const mgs::GatedGeom g = mgs::gated_geometry(d, false);
    if (!gated_grid_fits(g)) return MGS_ERR_UNSUPPORTED;
    if (mgs_status st = check_workspace(workspace, workspace_bytes, g.bytes)) return st;
    return hip_status(mgs::launch_gated_fwd(g, d, x, r, i, lam, h0, lengths, reset, y, hT, states, workspace,
                                            as_stream(stream)));
}

mgs_status mgs_gated_bwd(const mgs_gated_desc *desc, const void *x, const void *r, const void *i,
                         const float *lam, const void *dy, const float *dhT, const float *states,
                         const int32_t *lengths, const uint8_t *reset, void *dx, void *dr, void *di,
                         float *dlam, float *dh0, void *workspace, size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_gated(desc)) return st;
    const mgs_gated_desc &d = *desc;
    const size_t size = size_of(d.dtype), steps = static_cast<size_t>(d.B) * d.T, ny = steps * d.D * size;
    if (ny > 0 && (!dy || !states || !dx || !dr || !di)) return MGS_ERR_INVALID_VALUE;
    if (!dlam) return MGS_ERR_INVALID_VALUE;   // (D), never empty
    Range in[9];
    int n = gated_inputs(d, d.T, x, r, i, lam, dy, in);
    if (n < 0) return MGS_ERR_INVALID_VALUE;
    const void *f32[] = {dhT, states, lengths, dlam, dh0}, *same[] = {dx, dr, di};
    for (const void *p : f32)
        if (!aligned_to(p, 4)) return MGS_ERR_INVALID_VALUE;
    for (const void *p : same)
        if (!aligned_to(p, size)) return MGS_ERR_INVALID_VALUE;
    const size_t state = static_cast<size_t>(d.B) * d.D * 4;
    in[n++] = Range{dhT, state};
    in[n++] = Range{states, (d.T + MGS_GATED_CHUNK - 1) / MGS_GATED_CHUNK * state};
    in[n++] = Range{lengths, static_cast<size_t>(d.B) * 4};
    in[n++] = Range{reset, steps};
    const Range out[] = {{dx, ny}, {dr, ny}, {di, ny}, {dlam, static_cast<size_t>(d.D) * 4}, {dh0, state}};
    if (any_alias(in, n, out, 5)) return MGS_ERR_INVALID_VALUE;
    const mgs::GatedGeom g = mgs::gated_geometry(d, true);
    if (!gated_grid_fits(g)) return MGS_ERR_UNSUPPORTED;
    if (d.B > 0)   // (of no sequences only dlam is left, zeros: no workspace)
        if (mgs_status st = check_workspace(workspace, workspace_bytes, g.bytes)) return st;
    return hip_status(mgs::launch_gated_bwd(g, d, x, r, i, lam, dy, dhT, states, lengths, reset, dx, dr, di, dlam,
                                            dh0, workspace, as_stream(stream)));
}

mgs_status mgs_gated_step(const mgs_gated_desc *desc, const void *x, const void *r, const void *i,
                          const float *lam, float *h, int64_t n_slots, const int32_t *slots, void *y,
                          void *stream)
{
    if (!desc) return MGS_ERR_INVALID_VALUE;
    mgs_gated_desc d = *desc;
    d.T = 1;
    d.x_stride[1] = d.r_stride[1] = d.i_stride[1] = 0;
    if (mgs_status st = check_gated(&d)) return st;
    if (n_slots < 0) return MGS_ERR_INVALID_VALUE;
    const int64_t cells = bounded({n_slots, d.D});
    if (cells < 0) return MGS_ERR_UNSUPPORTED;
    Range in[5];
    int n = gated_inputs(d, 1, x, r, i, lam, nullptr, in);
    if (n < 0) return MGS_ERR_INVALID_VALUE;
    const size_t ny = static_cast<size_t>(d.B) * d.D * size_of(d.dtype);
    if ((ny > 0 && !y) || (cells > 0 && !h) || (!slots && d.B > n_slots)) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(h, 4) || !aligned_to(slots, 4) || !aligned_to(y, size_of(d.dtype))) return MGS_ERR_INVALID_VALUE;
    in[n++] = Range{slots, static_cast<size_t>(d.B) * 4};
    const Range out[] = {{y, ny}, {h, static_cast<size_t>(cells) * 4}};
    if (any_alias(in, n, out, 2)) return MGS_ERR_INVALID_VALUE;
    if (ny == 0) return MGS_OK;
    return hip_status(mgs::launch_gated_step(d, x, r, i, lam, h, n_slots, slots, y, as_stream(stream)));
}

// ----------------------------------------------------------------- sampling

static mgs_status check_sample(const mgs_sample_desc *d)
{
    if (!d) return MGS_ERR_INVALID_VALUE;
    if (d->B < 0 || d->vocab <= 0 || d->logits_stride < 0) return MGS_ERR_INVALID_VALUE;
    if (!known_dtype(d->dtype)) return MGS_ERR_UNSUPPORTED;
    if (d->vocab > mgs::kSampleMaxVocab || bounded({d->B, d->vocab}) < 0) return MGS_ERR_UNSUPPORTED;
    if (d->B > kMaxTiles / 2) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

mgs_status mgs_sample_workspace_size(const mgs_sample_desc *desc, size_t *bytes)
{
    if (!bytes) return MGS_ERR_INVALID_VALUE;
    if (mgs_status st = check_sample(desc)) return st;
    *bytes = mgs::sample_workspace(*desc);
    return MGS_OK;
}

mgs_status mgs_sample(const mgs_sample_desc *desc, const void *logits, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                      void *workspace, size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_sample(desc)) return st;
    const mgs_sample_desc &d = *desc;
    const size_t size = size_of(d.dtype), rows = static_cast<size_t>(d.B);
    const int64_t bytes = span(1, d.B, d.vocab, 0, d.logits_stride, size);
    if (bytes < 0 || (rows > 0 && (!logits || !u || !token))) return MGS_ERR_INVALID_VALUE;
    const void *f32[] = {u, temperature, top_k, top_p, min_p, logp};
    for (const void *p : f32)
        if (!aligned_to(p, 4)) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(logits, size) || !aligned_to(token, 8)) return MGS_ERR_INVALID_VALUE;
    const Range in[] = {{logits, static_cast<size_t>(bytes)}, {u, 4 * rows}, {temperature, 4 * rows}, {top_k, 4 * rows},
                        {top_p, 4 * rows}, {min_p, 4 * rows}};
    const Range out[] = {{token, 8 * rows}, {logp, 4 * rows}};
    if (any_alias(in, 6, out, 2)) return MGS_ERR_INVALID_VALUE;
    if (rows == 0) return MGS_OK;
    if (mgs_status st = check_workspace(workspace, workspace_bytes, mgs::sample_workspace(d))) return st;
    return hip_status(mgs::launch_sample(d, logits, u, temperature, top_k, top_p, min_p, token, logp, workspace,
                                         as_stream(stream)));
}

}  // extern "C"
