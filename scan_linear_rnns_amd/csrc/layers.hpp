// layers.hpp -- host-side interface between layers_api.cpp and the layer
// kernels (linattn.hip, rmsnorm.hip, clip_norm.hip): geometry, workspace
// layouts and launch functions.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mgs_layers.h"

namespace mgs {

// A HIP launch has fewer than 2^32 threads along a dimension.  f(first, blocks)
// launches workgroups first .. first + blocks - 1 of `threads` threads; larger
// grids go in several launches.
template <typename F> hipError_t launch_sliced(int64_t blocks, int threads, F f)
{
    const int64_t most = ((int64_t(1) << 32) - 1) / threads / 8 * 8;   // (a multiple of the XCDs)
    for (int64_t first = 0; first < blocks; first += most) {
        f(first, static_cast<unsigned>(blocks - first < most ? blocks - first : most));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// --------------------------------------------------------- linear attention
constexpr int kAttnChunk = 64;     // steps per chunk
constexpr int kAttnMaxDim = 128;   // largest dk, dv

struct AttnGeom {
    int64_t BH;       // B * H
    int nC;           // chunks
    int segLen;       // chunks per segment
    int nSeg;         // segments per (sequence, head)
    bool grouped;     // backward: dq, dk go through fp32 partials
    // workspace byte offsets: states entering each segment from the past (and,
    // one past the last, the final one) and from the future, segment decays,
    // <q,dq> and <k,dk> per step, per-head dg partials, dq and dk partials
    size_t off_S, off_R, off_dec, off_x, off_y, off_dg, off_dq, off_dk, bytes;
};

AttnGeom attn_geometry(const mgs_linattn_desc &d, bool backward);

hipError_t launch_linattn_fwd(const AttnGeom &geo, const mgs_linattn_desc &d, const void *q, const void *k,
                              const void *v, const float *g, const float *S0, const int32_t *lengths, void *o,
                              float *ST, void *ws, hipStream_t s);
hipError_t launch_linattn_bwd(const AttnGeom &geo, const mgs_linattn_desc &d, const void *q, const void *k,
                              const void *v, const float *g, const void *do_, const float *S0, const float *dST,
                              const int32_t *lengths, void *dq, void *dk, void *dv, float *dg, float *dS0,
                              void *ws, hipStream_t s);
hipError_t launch_linattn_step(const mgs_linattn_desc &d, const void *q, const void *k, const void *v,
                               const float *g, float *S, int64_t n_slots, const int32_t *slots, void *o,
                               hipStream_t s);

// --------------------------------------------------------------------- norm
constexpr int64_t kNormMaxDim = 65536;   // a row is held by one workgroup (in registers up to 8192 columns)

struct NormBwdGeom {
    int blocks;        // workgroups, each walking rows blockIdx, blockIdx + blocks, ...
    size_t off_dw, bytes;
};

NormBwdGeom norm_bwd_geometry(int64_t rows, int64_t d);

hipError_t launch_rmsnorm_fwd(const void *x, const void *residual, const void *w, void *y, float *scale, void *h,
                              float *rstd, int64_t rows, int64_t d, int64_t x_stride, int64_t r_stride, float eps,
                              int64_t group, bool fp8, int dtype, hipStream_t s);
hipError_t launch_rmsnorm_bwd(const NormBwdGeom &geo, const void *dy, const void *h, const void *w,
                              const float *rstd, const void *dh, void *dx, float *dw, int64_t rows, int64_t d,
                              int dtype, void *ws, hipStream_t s);

// ----------------------------------------------------------------- clipping
// Elements per workgroup of the two passes, and tensors per launch (their
// addresses and sizes travel in the kernel arguments).
constexpr int64_t kClipTile = 16384;
constexpr int kClipTensors = 128;

int64_t clip_tiles(int64_t n, const int64_t *sizes);   // workgroups of a pass over all tensors

hipError_t launch_clip_norm(int64_t n, const void *const *in, void *const *out, const int64_t *sizes,
                            const int *dtypes, float max_norm, float *norm, void *ws, int64_t tiles, hipStream_t s);

}  // namespace mgs
