// clip_norm.hip -- the global norm of many tensors, and clipping by it (gfx950).
//
//     norm = sqrt(sum_i sum g_i^2),   out_i = in_i min(1, max_norm / (norm + 1e-6))
//
// Two passes over the data: one partial sum for each tile of 16384 elements,
// then the scaling.  Both are bound by HBM; what costs beside that is the
// number of launches, so a launch covers up to 128 tensors (their addresses
// and sizes travel in its arguments, nothing is copied to the device).  Squares
// are formed and added in fp64 (in fp32 they would overflow from elements of
// 2^64 on and vanish below 2^-75), in an order that depends on the sizes alone.
// Measured, 393M bf16 elements in 150 tensors (0.8 GB): the squares 161 us (4.9
// TB/s), adding up the partials 8 us, the scaling 276 us (1.6 GB, 5.8 TB/s: the
// memory-side cache still holds part of what the first pass read; in that pass's
// own order it took 70 us more).  40 tensors of up to 65536 fp32 elements: 5 and
// 7 us, less than the host's work for the call.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "layers.hpp"

namespace mgs {
namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f8v __attribute__((ext_vector_type(8), aligned(16)));

constexpr int kTile = static_cast<int>(kClipTile);
// Up to this many partials every workgroup of the scaling adds them up itself
// (four loads a thread, shorter than a launch); beyond, one workgroup does it
// first, in a launch of its own.
constexpr int64_t kClipFew = 1024;

struct ClipTable {
    const void *in[kClipTensors];
    void *out[kClipTensors];
    int64_t size[kClipTensors];
    int first[kClipTensors];   // first tile of each tensor, in this launch
    uint8_t bf16[kClipTensors], vec[kClipTensors];
    int n, at;                 // at: the launch's first tile among the table's
    int64_t base;              // the table's first tile among all
};

// The tensor that holds a tile: every lane looks at two first tiles (which are
// in rising order), so that the search is one load deep.
__device__ __forceinline__ int tensor_of(const ClipTable &t, int tile)
{
    const int lane = threadIdx.x & 63;
    const bool a = lane < t.n && t.first[lane] <= tile, b = lane + 64 < t.n && t.first[lane + 64] <= tile;
    return __builtin_amdgcn_readfirstlane(__popcll(__ballot(a)) + __popcll(__ballot(b)) - 1);
}

// over a workgroup of W waves; lds: one slot per wave
template <int W> __device__ __forceinline__ double block_sum(double v, double *lds)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += lds[w];
    return v;
}

__device__ __forceinline__ f8v widen(f8v v) { return v; }
__device__ __forceinline__ f8v widen(bf8v v) { return __builtin_convertvector(v, f8v); }

__device__ __forceinline__ double square(float x) { return static_cast<double>(x) * static_cast<double>(x); }

__device__ __forceinline__ double square8(f8v x)
{
    double s = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += square(x[e]);
    return s;
}

// n elements of a tile: whole accesses of 8, those of a full tile all in flight;
// single ones at the end, or where the address is not aligned
template <typename T, typename V> __device__ __forceinline__ double tile_squares(const T *p, int n, bool vec)
{
    double sum = 0.0;
    int done = 0;
    if (vec) {
        const V *v = reinterpret_cast<const V *>(p);
        if (n == kTile) {
#pragma unroll
            for (int i = 0; i < kTile / 2048; ++i) sum += square8(widen(v[i * 256 + threadIdx.x]));
            return sum;
        }
        done = n & ~7;
#pragma unroll 4
        for (int i = threadIdx.x; i < done / 8; i += 256) sum += square8(widen(v[i]));
    }
#pragma unroll 8
    for (int i = done + threadIdx.x; i < n; i += 256) sum += square(static_cast<float>(p[i]));
    return sum;
}

__global__ void __launch_bounds__(256) squares_kernel(ClipTable t, double *part)
{
    __shared__ double lds[4];
    const int tile = t.at + static_cast<int>(blockIdx.x), i = tensor_of(t, tile);
    const int64_t at = static_cast<int64_t>(tile - t.first[i]) * kTile;
    const int n = static_cast<int>(min(static_cast<int64_t>(kTile), t.size[i] - at));
    double s = t.bf16[i] ? tile_squares<__bf16, bf8v>(static_cast<const __bf16 *>(t.in[i]) + at, n, t.vec[i])
                         : tile_squares<float, f8v>(static_cast<const float *>(t.in[i]) + at, n, t.vec[i]);
    s = block_sum<4>(s, lds);
    if (threadIdx.x == 0) part[t.base + tile] = s;
}

// The norm from n partials, in a fixed order, by a workgroup of W waves.  From
// 2^126 on its reciprocal, and so a coefficient, is no normal fp32 number: such a
// norm counts as not finite.
template <int W> __device__ __forceinline__ float norm_of(const double *part, int64_t n, double *lds)
{
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += 64 * W) s += part[i];
    const double norm = sqrt(block_sum<W>(s, lds));
    return static_cast<float>(norm < 0x1p126 ? norm : norm * __builtin_inf());
}

__global__ void __launch_bounds__(1024) norm_kernel(const double *part, int64_t n, float *norm)
{
    __shared__ double lds[16];
    const float v = norm_of<16>(part, n, lds);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T, typename V>
__device__ __forceinline__ void tile_scale(const T *p, T *o, int n, float c, bool vec)
{
    int done = 0;
    if (vec) {
        const V *v = reinterpret_cast<const V *>(p);
        V *w = reinterpret_cast<V *>(o);
        if (n == kTile) {
            V x[kTile / 2048];
#pragma unroll
            for (int i = 0; i < kTile / 2048; ++i) x[i] = v[i * 256 + threadIdx.x];
#pragma unroll
            for (int i = 0; i < kTile / 2048; ++i) w[i * 256 + threadIdx.x] = __builtin_convertvector(widen(x[i]) * c, V);
            return;
        }
        done = n & ~7;
#pragma unroll 4
        for (int i = threadIdx.x; i < done / 8; i += 256) w[i] = __builtin_convertvector(widen(v[i]) * c, V);
    }
#pragma unroll 8
    for (int i = done + threadIdx.x; i < n; i += 256) o[i] = static_cast<T>(static_cast<float>(p[i]) * c);
}

// few != 0: the norm is added up here, and the first workgroup of the first launch
// writes it.  The tensors come in the reverse of the first pass's order, and so do
// the tiles of each: what that pass read last is still in the memory-side cache.
__global__ void __launch_bounds__(256) scale_kernel(ClipTable t, const double *part, int64_t n_part, float max_norm,
                                                    float *norm, int few)
{
    __shared__ double lds[4];
    float v;
    if (few) {
        v = norm_of<4>(part, n_part, lds);
        if (t.base + t.at + blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    } else {
        v = *norm;
    }
    float c = max_norm / (v + 1e-6f);
    if (!(c < 1.0f) || !isfinite(v)) c = 1.0f;
    const int tile = t.at + static_cast<int>(blockIdx.x), i = tensor_of(t, tile);
    if (c == 1.0f && t.in[i] == t.out[i]) return;
    const int64_t last = (t.size[i] - 1) / kTile;
    const int64_t at = (last - (tile - t.first[i])) * kTile;
    const int n = static_cast<int>(min(static_cast<int64_t>(kTile), t.size[i] - at));
    if (t.bf16[i])
        tile_scale<__bf16, bf8v>(static_cast<const __bf16 *>(t.in[i]) + at, static_cast<__bf16 *>(t.out[i]) + at, n, c, t.vec[i]);
    else
        tile_scale<float, f8v>(static_cast<const float *>(t.in[i]) + at, static_cast<float *>(t.out[i]) + at, n, c, t.vec[i]);
}

// Launches f(table, workgroups) for each group of up to kClipTensors non-empty
// tensors, from the first on, or from the last back.
template <typename F>
hipError_t each_launch(int64_t n, const void *const *in, void *const *out, const int64_t *sizes, const int *dtypes,
                       bool back, F f)
{
    ClipTable t{};
    int64_t base = 0, tiles = 0;
    auto flush = [&] {
        t.base = base;
        return launch_sliced(tiles, 256, [&](int64_t first, unsigned blocks) {
            t.at = static_cast<int>(first);
            f(t, blocks);
        });
    };
    for (int64_t j = 0; j < n; ++j) {
        const int64_t i = back ? n - 1 - j : j;
        if (sizes[i] == 0) continue;
        t.in[t.n] = in[i];
        t.out[t.n] = out ? out[i] : nullptr;
        t.size[t.n] = sizes[i];
        t.first[t.n] = static_cast<int>(tiles);
        t.bf16[t.n] = dtypes[i] == MGS_BF16 ? 1 : 0;
        t.vec[t.n] = ((reinterpret_cast<uintptr_t>(in[i]) | reinterpret_cast<uintptr_t>(t.out[t.n])) & 15u) == 0;
        ++t.n;
        tiles += (sizes[i] + kTile - 1) / kTile;
        if (t.n == kClipTensors) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
            base += tiles;
            tiles = 0;
            t.n = 0;
        }
    }
    return flush();
}

}  // namespace

int64_t clip_tiles(int64_t n, const int64_t *sizes)
{
    int64_t tiles = 0;
    for (int64_t i = 0; i < n; ++i) tiles += (sizes[i] + kTile - 1) / kTile;
    return tiles;
}

hipError_t launch_clip_norm(int64_t n, const void *const *in, void *const *out, const int64_t *sizes,
                            const int *dtypes, float max_norm, float *norm, void *ws, int64_t tiles, hipStream_t s)
{
    double *part = static_cast<double *>(ws);
    hipError_t e = each_launch(n, in, nullptr, sizes, dtypes, false, [&](const ClipTable &t, unsigned grid) {
        hipLaunchKernelGGL(squares_kernel, dim3(grid), dim3(256), 0, s, t, part);
    });
    if (e != hipSuccess) return e;
    const int few = out && tiles > 0 && tiles <= kClipFew;
    if (!few) {
        hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(1024), 0, s, part, tiles, norm);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!out) return hipSuccess;
    return each_launch(n, in, out, sizes, dtypes, true, [&](const ClipTable &t, unsigned grid) {
        hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(256), 0, s, t, part, tiles, max_norm, norm, few);
    });
}

}  // namespace mgs
