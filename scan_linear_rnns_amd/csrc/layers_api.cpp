// layers_api.cpp -- the C ABI declared in include/mgs_layers.h: argument
// validation and dispatch.  As in mgs_api.cpp, every refusal comes before any
// HIP call.
#include "mgs_layers.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <memory>
#include <new>

#include "api_common.hpp"
#include "layers.hpp"

namespace {

using mgs::any_alias;
using mgs::as_stream;
using mgs::check_workspace;
using mgs::hip_status;
using mgs::Range;

constexpr int64_t kMaxElems = int64_t(1) << 40;   // of one tensor
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1 - 64;
constexpr int64_t kMaxGroups = (int64_t(1) << 31) - 1;   // workgroups numbered in 32 bits

int64_t bounded(std::initializer_list<int64_t> dims) { return mgs::bounded_product(dims, kMaxElems, kMaxDim); }

bool aligned_to(const void *p, size_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }

bool known_dtype(int dtype) { return dtype == MGS_F32 || dtype == MGS_BF16; }

size_t size_of(int dtype) { return dtype == MGS_BF16 ? 2 : 4; }

// --------------------------------------------------------- linear attention

mgs_status check_attn(const mgs_linattn_desc *d)
{
    if (!d) return MGS_ERR_INVALID_VALUE;
    if (d->B < 0 || d->T < 0 || d->H < 0 || d->Hk < 0 || d->dk <= 0 || d->dv <= 0) return MGS_ERR_INVALID_VALUE;
    if ((d->H > 0 && (d->Hk == 0 || d->H % d->Hk != 0)) || (d->H == 0 && d->Hk != 0)) return MGS_ERR_INVALID_VALUE;
    if (!known_dtype(d->dtype)) return MGS_ERR_UNSUPPORTED;
    if (d->dk > mgs::kAttnMaxDim || d->dv > mgs::kAttnMaxDim) return MGS_ERR_UNSUPPORTED;
    const int64_t big = d->dk > d->dv ? d->dk : d->dv;
    if (bounded({d->B, d->T, d->H, big}) < 0 || bounded({d->B, d->H, d->dk, d->dv}) < 0) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

// Bytes from the first to past the last element of a strided operand, or -1
// where a stride is negative or the span passes the limit.
int64_t span(int64_t B, int64_t T, int64_t H, int64_t cols, const int64_t *st, size_t size)
{
    if (st[0] < 0 || st[1] < 0 || st[2] < 0) return -1;
    if (B == 0 || T == 0 || H == 0) return 0;
    const int64_t n[3] = {B - 1, T - 1, H - 1};
    int64_t total = cols;
    for (int i = 0; i < 3; ++i) {
        int64_t x;
        if (__builtin_mul_overflow(n[i], st[i], &x) || __builtin_add_overflow(total, x, &total) ||
            total > (int64_t(1) << 58))
            return -1;
    }
    return total * static_cast<int64_t>(size);
}

// The operands' ranges (q, k, v, g and do_ if given) into in[0..]; their count,
// or -1 where one is refused.
int attn_inputs(const mgs_linattn_desc &d, int64_t T, const void *q, const void *k, const void *v, const float *g,
                const void *do_, Range *in)
{
    const size_t size = size_of(d.dtype);
    const int64_t dense_h[3] = {0, 0, 1};
    const int64_t *gst = d.decay_per_head ? dense_h : d.g_stride;
    const int64_t bytes[5] = {span(d.B, T, d.Hk, d.dk, d.q_stride, size), span(d.B, T, d.Hk, d.dk, d.k_stride, size),
                              span(d.B, T, d.H, d.dv, d.v_stride, size), span(d.B, T, d.H, 1, gst, 4),
                              do_ ? span(d.B, T, d.H, d.dv, d.do_stride, size) : 0};
    const void *p[5] = {q, k, v, g, do_};
    const int n = do_ ? 5 : 4;
    for (int i = 0; i < n; ++i) {
        if (bytes[i] < 0 || (bytes[i] > 0 && !p[i])) return -1;
        if (!aligned_to(p[i], i == 3 ? 4 : size)) return -1;
        in[i] = Range{p[i], static_cast<size_t>(bytes[i])};
    }
    return n;
}

// Workgroups of the walks, up to three a segment of a sequence and head, are
// counted in 32 bits (the other kernels' in 64)
bool attn_grids_fit(const mgs::AttnGeom &g)
{
    const int64_t items = mgs::bounded_product({g.BH, g.nSeg}, kMaxGroups, kMaxGroups);
    return items >= 0 && items <= kMaxGroups / 3 - 8;
}

}  // namespace

extern "C" {

mgs_status mgs_linattn_workspace_size(const mgs_linattn_desc *desc, int backward, size_t *bytes)
{
    if (!bytes) return MGS_ERR_INVALID_VALUE;
    if (mgs_status st = check_attn(desc)) return st;
    const mgs::AttnGeom f = mgs::attn_geometry(*desc, false), b = mgs::attn_geometry(*desc, true);
    if (!attn_grids_fit(f) || (backward && !attn_grids_fit(b))) return MGS_ERR_UNSUPPORTED;
    *bytes = backward && b.bytes > f.bytes ? b.bytes : f.bytes;
    return MGS_OK;
}

mgs_status mgs_linattn_fwd(const mgs_linattn_desc *desc, const void *q, const void *k, const void *v,
                           const float *g, const float *S0, const int32_t *lengths, void *o, float *ST,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_attn(desc)) return st;
    const mgs_linattn_desc &d = *desc;
    Range in[7];
    int n = attn_inputs(d, d.T, q, k, v, g, nullptr, in);
    if (n < 0) return MGS_ERR_INVALID_VALUE;
    const size_t states = static_cast<size_t>(d.B) * d.H * d.dk * d.dv * 4;
    const size_t rows = static_cast<size_t>(d.B) * d.T * d.H * d.dv * size_of(d.dtype);
    if (rows > 0 && !o) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(S0, 4) || !aligned_to(lengths, 4) || !aligned_to(o, size_of(d.dtype)) || !aligned_to(ST, 4))
        return MGS_ERR_INVALID_VALUE;
    in[n++] = Range{S0, states};
    in[n++] = Range{lengths, static_cast<size_t>(d.B) * 4};
    const Range out[] = {{o, rows}, {ST, states}};
    if (any_alias(in, n, out, 2)) return MGS_ERR_INVALID_VALUE;
    if (d.B == 0 || d.H == 0 || (d.T == 0 && !ST)) return MGS_OK;
    const mgs::AttnGeom geo = mgs::attn_geometry(d, false);
    if (!attn_grids_fit(geo)) return MGS_ERR_UNSUPPORTED;
    if (mgs_status st = check_workspace(workspace, workspace_bytes, geo.bytes)) return st;
    return hip_status(mgs::launch_linattn_fwd(geo, d, q, k, v, g, S0, lengths, o, ST, workspace, as_stream(stream)));
}

mgs_status mgs_linattn_bwd(const mgs_linattn_desc *desc, const void *q, const void *k, const void *v,
                           const float *g, const void *do_, const float *S0, const float *dST,
                           const int32_t *lengths, void *dq, void *dk_, void *dv_, float *dg, float *dS0,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_attn(desc)) return st;
    const mgs_linattn_desc &d = *desc;
    const size_t size = size_of(d.dtype);
    const size_t states = static_cast<size_t>(d.B) * d.H * d.dk * d.dv * 4;
    const size_t steps = static_cast<size_t>(d.B) * d.T;
    if (steps * d.H > 0 && !do_) return MGS_ERR_INVALID_VALUE;
    Range in[8];
    int n = attn_inputs(d, d.T, q, k, v, g, do_, in);
    if (n < 0) return MGS_ERR_INVALID_VALUE;
    const size_t nqk = steps * d.Hk * d.dk * size, nv = steps * d.H * d.dv * size;
    const size_t ng = (d.decay_per_head ? static_cast<size_t>(d.H) : steps * d.H) * 4;
    if (nv > 0 && (!dq || !dk_ || !dv_)) return MGS_ERR_INVALID_VALUE;
    if (ng > 0 && !dg) return MGS_ERR_INVALID_VALUE;
    const void *f32[] = {S0, dST, lengths, dg, dS0}, *same[] = {dq, dk_, dv_};
    for (const void *p : f32)
        if (!aligned_to(p, 4)) return MGS_ERR_INVALID_VALUE;
    for (const void *p : same)
        if (!aligned_to(p, size)) return MGS_ERR_INVALID_VALUE;
    in[n++] = Range{S0, states};
    in[n++] = Range{dST, states};
    in[n++] = Range{lengths, static_cast<size_t>(d.B) * 4};
    const Range out[] = {{dq, nqk}, {dk_, nqk}, {dv_, nv}, {dg, ng}, {dS0, states}};
    if (any_alias(in, n, out, 5)) return MGS_ERR_INVALID_VALUE;
    if (d.H == 0 || (d.B == 0 && !d.decay_per_head)) return MGS_OK;
    const mgs::AttnGeom geo = mgs::attn_geometry(d, true);
    if (!attn_grids_fit(geo)) return MGS_ERR_UNSUPPORTED;
    if (d.B > 0)   // (of no sequences only dg is left, (H) zeros: no workspace)
        if (mgs_status st = check_workspace(workspace, workspace_bytes, geo.bytes)) return st;
    return hip_status(mgs::launch_linattn_bwd(geo, d, q, k, v, g, do_, S0, dST, lengths, dq, dk_, dv_, dg, dS0,
                                              workspace, as_stream(stream)));
}

mgs_status mgs_linattn_step(const mgs_linattn_desc *desc, const void *q, const void *k, const void *v,
                            const float *g, float *S, int64_t n_slots, const int32_t *slots, void *o,
                            void *stream)
{
    if (!desc) return MGS_ERR_INVALID_VALUE;
    mgs_linattn_desc d = *desc;
    d.T = 1;
    d.q_stride[1] = d.k_stride[1] = d.v_stride[1] = d.g_stride[1] = 0;
    if (mgs_status st = check_attn(&d)) return st;
    if (n_slots < 0) return MGS_ERR_INVALID_VALUE;
    const int64_t cells = bounded({n_slots, d.H, d.dk, d.dv});
    if (cells < 0) return MGS_ERR_UNSUPPORTED;
    Range in[5];
    int n = attn_inputs(d, 1, q, k, v, g, nullptr, in);
    if (n < 0) return MGS_ERR_INVALID_VALUE;
    const size_t rows = static_cast<size_t>(d.B) * d.H * d.dv * size_of(d.dtype);
    if (rows > 0 && !o) return MGS_ERR_INVALID_VALUE;
    if (cells > 0 && !S) return MGS_ERR_INVALID_VALUE;
    if (!slots && d.B > n_slots) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(S, 4) || !aligned_to(slots, 4) || !aligned_to(o, size_of(d.dtype))) return MGS_ERR_INVALID_VALUE;
    in[n++] = Range{slots, static_cast<size_t>(d.B) * 4};
    const Range out[] = {{o, rows}, {S, static_cast<size_t>(cells) * 4}};
    if (any_alias(in, n, out, 2)) return MGS_ERR_INVALID_VALUE;
    if (rows == 0) return MGS_OK;
    if (d.B * d.H > kMaxGroups / 8) return MGS_ERR_UNSUPPORTED;
    return hip_status(mgs::launch_linattn_step(d, q, k, v, g, S, n_slots, slots, o, as_stream(stream)));
}

// --------------------------------------------------------------------- norm

static mgs_status check_norm(int64_t rows, int64_t d, int dtype)
{
    if (rows < 0 || d <= 0) return MGS_ERR_INVALID_VALUE;
    if (!known_dtype(dtype)) return MGS_ERR_UNSUPPORTED;
    if (d > mgs::kNormMaxDim || bounded({rows, d}) < 0) return MGS_ERR_UNSUPPORTED;
    return MGS_OK;
}

static mgs_status norm_fwd(const void *x, const void *residual, const void *w, void *y, size_t y_bytes, float *scale,
                           size_t scale_bytes, void *h, float *rstd, int64_t rows, int64_t d, int64_t x_stride,
                           int64_t r_stride, float eps, int64_t group, bool fp8, int dtype, void *stream)
{
    if (mgs_status st = check_norm(rows, d, dtype)) return st;
    if (!(eps >= 0.0f)) return MGS_ERR_INVALID_VALUE;
    const size_t size = size_of(dtype);
    const int64_t sx[3] = {0, x_stride, 0}, sr[3] = {0, r_stride, 0};
    const int64_t nx = span(1, rows, 1, d, sx, size), nr = residual ? span(1, rows, 1, d, sr, size) : 0;
    if (nx < 0 || nr < 0) return MGS_ERR_INVALID_VALUE;
    const size_t n = static_cast<size_t>(rows) * d;
    if (n > 0 && (!x || !w || !y || (fp8 && !scale))) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(x, size) || !aligned_to(residual, size) || !aligned_to(w, size) || !aligned_to(h, size) ||
        (!fp8 && !aligned_to(y, size)) || !aligned_to(scale, 4) || !aligned_to(rstd, 4))
        return MGS_ERR_INVALID_VALUE;
    // h in place of the residual or of x: the same rows at the same addresses
    const bool over_r = h && h == residual && r_stride == d, over_x = h && h == x && x_stride == d;
    const Range in[] = {{over_x ? nullptr : x, static_cast<size_t>(nx)},
                        {over_r ? nullptr : residual, static_cast<size_t>(nr)},
                        {w, static_cast<size_t>(d) * size}};
    const Range out[] = {{y, y_bytes}, {scale, scale_bytes}, {h, n * size}, {rstd, static_cast<size_t>(rows) * 4}};
    if (any_alias(in, 3, out, 4)) return MGS_ERR_INVALID_VALUE;
    if (n == 0) return MGS_OK;
    return hip_status(mgs::launch_rmsnorm_fwd(x, residual, w, y, scale, h, rstd, rows, d, x_stride, r_stride, eps,
                                              group, fp8, dtype, as_stream(stream)));
}

mgs_status mgs_rmsnorm_fwd(const void *x, const void *residual, const void *w, void *y, void *h, float *rstd,
                           int64_t rows, int64_t d, int64_t x_stride, int64_t r_stride, float eps, int dtype,
                           void *stream)
{
    if (mgs_status st = check_norm(rows, d, dtype)) return st;
    return norm_fwd(x, residual, w, y, static_cast<size_t>(rows) * d * size_of(dtype), nullptr, 0, h, rstd, rows, d,
                    x_stride, r_stride, eps, 0, false, dtype, stream);
}

mgs_status mgs_rmsnorm_fwd_fp8(const void *x, const void *residual, const void *w, void *y8, float *scale,
                               void *h, int64_t rows, int64_t d, int64_t x_stride, int64_t r_stride, float eps,
                               int64_t group, int dtype, void *stream)
{
    if (mgs_status st = check_norm(rows, d, dtype)) return st;
    if (group < 0) return MGS_ERR_INVALID_VALUE;
    if (group != 0 && group != 128) return MGS_ERR_UNSUPPORTED;
    const size_t n = static_cast<size_t>(rows) * d;
    const size_t scales = static_cast<size_t>(rows) * (group ? (d + group - 1) / group : 1) * 4;
    return norm_fwd(x, residual, w, y8, n, scale, scales, h, nullptr, rows, d, x_stride, r_stride, eps, group, true,
                    dtype, stream);
}

mgs_status mgs_rmsnorm_workspace_size(int64_t rows, int64_t d, size_t *bytes)
{
    if (!bytes) return MGS_ERR_INVALID_VALUE;
    if (mgs_status st = check_norm(rows, d, MGS_F32)) return st;
    *bytes = mgs::norm_bwd_geometry(rows, d).bytes;
    return MGS_OK;
}

mgs_status mgs_rmsnorm_bwd(const void *dy, const void *h, const void *w, const float *rstd, const void *dh,
                           void *dx, float *dw, int64_t rows, int64_t d, int dtype, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_norm(rows, d, dtype)) return st;
    const size_t size = size_of(dtype), n = static_cast<size_t>(rows) * d * size;
    if (n > 0 && (!dy || !h || !rstd || !dx)) return MGS_ERR_INVALID_VALUE;
    if (!w || !dw) return MGS_ERR_INVALID_VALUE;   // (d), never empty: read and written for rows == 0 too
    const void *same[] = {dy, h, w, dh, dx};
    for (const void *p : same)
        if (!aligned_to(p, size)) return MGS_ERR_INVALID_VALUE;
    if (!aligned_to(rstd, 4) || !aligned_to(dw, 4)) return MGS_ERR_INVALID_VALUE;
    const Range in[] = {{dx == dy ? nullptr : dy, n},
                        {h, n},
                        {w, static_cast<size_t>(d) * size},
                        {rstd, static_cast<size_t>(rows) * 4},
                        {dx == dh ? nullptr : dh, n}};
    const Range out[] = {{dx, n}, {dw, static_cast<size_t>(d) * 4}};
    if (any_alias(in, 5, out, 2)) return MGS_ERR_INVALID_VALUE;
    const mgs::NormBwdGeom g = mgs::norm_bwd_geometry(rows, d);
    if (mgs_status st = check_workspace(workspace, workspace_bytes, g.bytes)) return st;
    return hip_status(mgs::launch_rmsnorm_bwd(g, dy, h, w, rstd, dh, dx, dw, rows, d, dtype, workspace,
                                              as_stream(stream)));
}

// ----------------------------------------------------------------- clipping

static mgs_status check_clip(int64_t n, const int64_t *sizes)
{
    if (n < 0 || (n > 0 && !sizes)) return MGS_ERR_INVALID_VALUE;
    int64_t total = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (sizes[i] < 0) return MGS_ERR_INVALID_VALUE;
        if (sizes[i] > kMaxElems || (total += sizes[i]) > kMaxElems) return MGS_ERR_UNSUPPORTED;
    }
    return MGS_OK;
}

// Every output must be disjoint from every other output and from every input but
// its own: all of them in the order of their addresses, each against the furthest
// end before it.
static mgs_status check_clip_overlaps(int64_t n, const void *const *in, void *const *out, const int64_t *sizes,
                                      const int *dtypes)
{
    struct Span {
        uintptr_t begin, end;
        bool out;
    };
    std::unique_ptr<Span[]> all(new (std::nothrow) Span[2 * static_cast<size_t>(n)]);
    if (!all) return hip_status(hipErrorOutOfMemory);
    int64_t m = 0;
    for (int64_t i = 0; i < n; ++i) {
        const size_t bytes = static_cast<size_t>(sizes[i]) * size_of(dtypes[i]);
        if (bytes == 0) continue;
        const uintptr_t o = reinterpret_cast<uintptr_t>(out[i]), x = reinterpret_cast<uintptr_t>(in[i]);
        all[m++] = Span{o, o + bytes, true};
        if (x != o) all[m++] = Span{x, x + bytes, false};
    }
    std::sort(all.get(), all.get() + m, [](const Span &a, const Span &b) { return a.begin < b.begin; });
    uintptr_t end[2] = {0, 0};   // of the inputs and the outputs so far
    for (int64_t i = 0; i < m; ++i) {
        const Span &s = all[i];
        if (s.begin < end[1] || (s.out && s.begin < end[0])) return MGS_ERR_INVALID_VALUE;
        end[s.out] = std::max(end[s.out], s.end);
    }
    return MGS_OK;
}

static size_t clip_bytes(int64_t tiles) { return 256 + static_cast<size_t>(tiles) * sizeof(double); }

mgs_status mgs_clip_norm_workspace_size(int64_t n, const int64_t *sizes, size_t *bytes)
{
    if (!bytes) return MGS_ERR_INVALID_VALUE;
    if (mgs_status st = check_clip(n, sizes)) return st;
    *bytes = clip_bytes(mgs::clip_tiles(n, sizes));
    return MGS_OK;
}

mgs_status mgs_clip_norm(int64_t n, const void *const *in, void *const *out, const int64_t *sizes,
                         const int *dtypes, float max_norm, float *norm, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    if (mgs_status st = check_clip(n, sizes)) return st;
    if (!norm || !aligned_to(norm, 4) || !(max_norm >= 0.0f)) return MGS_ERR_INVALID_VALUE;
    if (n > 0 && (!in || !dtypes)) return MGS_ERR_INVALID_VALUE;
    for (int64_t i = 0; i < n; ++i) {
        if (!known_dtype(dtypes[i])) return MGS_ERR_UNSUPPORTED;
        if (sizes[i] == 0) continue;
        if (!in[i] || (out && !out[i])) return MGS_ERR_INVALID_VALUE;
        const size_t size = size_of(dtypes[i]);
        if (!aligned_to(in[i], size) || (out && !aligned_to(out[i], size))) return MGS_ERR_INVALID_VALUE;
        const Range a{in[i], sizes[i] * size}, b{out ? out[i] : nullptr, sizes[i] * size}, s{norm, 4};
        if (overlaps(a, s) || overlaps(b, s)) return MGS_ERR_INVALID_VALUE;
    }
    if (out && n > 0)
        if (mgs_status st = check_clip_overlaps(n, in, out, sizes, dtypes)) return st;
    const int64_t tiles = mgs::clip_tiles(n, sizes);
    if (mgs_status st = check_workspace(workspace, workspace_bytes, clip_bytes(tiles))) return st;
    return hip_status(mgs::launch_clip_norm(n, in, out, sizes, dtypes, max_norm, norm, workspace, tiles,
                                            as_stream(stream)));
}

}  // extern "C"
