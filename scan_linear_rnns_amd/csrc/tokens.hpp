// tokens.hpp -- host-side interface between tokens_api.cpp and the kernels of
// the token path (embed.hip, gated.hip, sample.hip): geometry, workspace layouts
// and launch functions.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mgs_tokens.h"

namespace mgs {

// Bytes at a workspace's start that sampling and the table's gradient leave alone: the
// recurrence's launch words and the limit of its waits, were it given the same one (its
// results are wrong then, but every wait ends)
constexpr size_t kHeader = 256;

// ---------------------------------------------------------------- embedding
struct EmbedGeom {
    int bits, range;   // 2^bits sorting workgroups, ids of each
    int chunk;         // sorted places of a summing workgroup
    int64_t chunks;
    // workspace byte offsets: the number of ids inside the table, each id's first sorted
    // place, the sorted places' rows and ids, partial sums of runs of one id that cross a chunk
    size_t off_count, off_first, off_row, off_id, off_part, bytes;
};

EmbedGeom embed_geometry(int64_t n, int64_t vocab, int64_t d);

hipError_t launch_embed_fwd(const void *ids, bool wide_ids, const void *W, void *y, int64_t n, int64_t vocab,
                            int64_t d, int64_t w_stride, float scale, int dtype, hipStream_t s);
hipError_t launch_embed_bwd(const EmbedGeom &g, const void *ids, bool wide_ids, const void *dy, void *dW, int64_t n,
                            int64_t vocab, int64_t d, int64_t dy_stride, float scale, bool accumulate, int dtype,
                            int dw_dtype, void *ws, hipStream_t s);

// --------------------------------------------------- gated linear recurrence
struct GatedGeom {
    int64_t groups;       // of channels, over all sequences
    int64_t tiles_f, tiles_b;     // along T, forward and backward
    int unit;             // tiles of a look-back's unit
    size_t off_agg, off_incl, off_part, bytes;   // tagged words
};

GatedGeom gated_geometry(const mgs_gated_desc &d, bool backward);

hipError_t launch_gated_fwd(const GatedGeom &g, const mgs_gated_desc &d, const void *x, const void *r, const void *i,
                            const float *lam, const float *h0, const int32_t *lengths, const uint8_t *reset, void *y,
                            float *hT, float *states, void *ws, hipStream_t s);
hipError_t launch_gated_bwd(const GatedGeom &g, const mgs_gated_desc &d, const void *x, const void *r, const void *i,
                            const float *lam, const void *dy, const float *dhT, const float *states,
                            const int32_t *lengths, const uint8_t *reset, void *dx, void *dr, void *di, float *dlam,
                            float *dh0, void *ws, hipStream_t s);
hipError_t launch_gated_step(const mgs_gated_desc &d, const void *x, const void *r, const void *i, const float *lam,
                             float *h, int64_t n_slots, const int32_t *slots, void *y, hipStream_t s);

// ----------------------------------------------------------------- sampling
constexpr int64_t kSampleMaxVocab = int64_t(1) << 20;

size_t sample_workspace(const mgs_sample_desc &d);

hipError_t launch_sample(const mgs_sample_desc &d, const void *logits, const float *u, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                         void *ws, hipStream_t s);

}  // namespace mgs
