// rmsnorm.hip -- root-mean-square norm with the residual's addition, its 8-bit
// form and its gradient (gfx950).
//
//     h = x + residual,   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w
//     dx = rstd (dy w - h rstd^2 mean(dy w h)) + dh,          dw = sum_rows dy h rstd
//
// All of it is bound by HBM: a row is read once into registers (8 neighbouring
// columns per thread and turn), reduced there, and written once; the 8-bit
// form takes the maximum and rounds from the same registers, so y never goes
// to memory in a wider type.  TPR threads share a row: a wave for short rows
// (no barrier), a workgroup for long ones.
// Measured (a large copy runs at 4.7 TB/s): forward 16384 x 4096 bf16 88 us
// (538 MB, 6.1 TB/s), 8-bit forward 8191 x 5000 with a scale for each 128 columns
// 61 us (291 MB, 4.8 TB/s), gradient of 16384 x 4096 bf16 110 us (546 MB, 5.0
// TB/s) and 5 us for dw.  4095 x 1000 fp32: 13, 13 and 4 us.
// Wide rows do not fit the registers of 1024 threads: the forward spills above
// 16384 columns (2048 x 32768 bf16: 281 us, 1.9 TB/s), the gradient, which holds two
// rows, above 8192 (4096 x 16384 bf16: 248 us, 2.2 TB/s) and heavily above 16384
// (2048 x 32768 bf16: 2.1 ms, 0.25 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "layers.hpp"

namespace mgs {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;   // keeps the scale of a row of zeros invertible

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f8v __attribute__((ext_vector_type(8), aligned(16)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));

// 8 elements from p (n of them in the row), as fp32, zeros past the end
__device__ __forceinline__ f8v load8(const float *p, int n, bool vec)
{
    f8v v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (vec) {
        if (n > 0) v = *reinterpret_cast<const f8v *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] = p[i];
    }
    return v;
}

__device__ __forceinline__ f8v load8(const __bf16 *p, int n, bool vec)
{
    f8v v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (vec) {
        if (n > 0) v = __builtin_convertvector(*reinterpret_cast<const bf8v *>(p), f8v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] = static_cast<float>(p[i]);
    }
    return v;
}

__device__ __forceinline__ void store8(float *p, f8v v, int n, bool vec)
{
    if (vec) {
        if (n > 0) *reinterpret_cast<f8v *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

__device__ __forceinline__ void store8(__bf16 *p, f8v v, int n, bool vec)
{
    const bf8v b = __builtin_convertvector(v, bf8v);
    if (vec) {
        if (n > 0) *reinterpret_cast<bf8v *>(p) = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = b[i];
    }
}

// y / s rounded once: with bf16 inputs quotients do fall on ties of the 8-bit
// type, and an ulp would send them to either side.  The product with 1 / s is put
// right by its exact remainder (y - q s is a float, s being at least 2e-33 and |q|
// at most 448), three operations where a division takes ten (8191 x 5000, a pass:
// 64.3 us, divided 64.9, the product as it is 63.5).
__device__ __forceinline__ f8v quotients(f8v y, float s)
{
    const float inv = 1.0f / s;
    if (!(s < __builtin_inff())) return y / s;
    f8v q;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q0 = y[e] * inv;
        q[e] = __builtin_fmaf(__builtin_fmaf(-q0, s, y[e]), inv, q0);
    }
    return q;
}

// Over the TPR threads of a row; every thread gets the result.  lds: one slot
// per wave; a call's last reads are ordered before the next call's writes by
// the barrier at its start.
template <int TPR, bool MAX> __device__ __forceinline__ float row_reduce(float v, float *lds)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const float u = __shfl_xor(v, off, 64);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v = MAX ? fmaxf(v, lds[w]) : v + lds[w];
    }
    return v;
}

struct NormArgs {
    const void *x, *res, *w;
    void *y, *h;
    float *scale, *rstd;
    int64_t rows, xs, rs;
    int64_t first;   // this launch's first workgroup
    int d, group;
    float eps;
    int vec;
};

enum { OUT_SAME = 0, OUT_FP8_ROW = 1, OUT_FP8_GROUP = 2 };

template <typename T, int TPR, int ITER, int OUT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_fwd_kernel(NormArgs a)
{
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;   // rows per workgroup
    __shared__ float lds[16];
    const int t = threadIdx.x % TPR;
    const int64_t row = (a.first + blockIdx.x) * RPW + threadIdx.x / TPR;
    if (row >= a.rows) return;   // whole waves; with TPR > 64 whole workgroups
    const bool vec = a.vec != 0;
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    f8v h[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * TPR + t) * 8;
        h[i] = load8(x + c, a.d - c, vec);
    }
    if (a.res) {
        const T *r = static_cast<const T *>(a.res) + row * a.rs;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * TPR + t) * 8;
            h[i] += load8(r + c, a.d - c, vec);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
    if (a.h) {
        T *o = static_cast<T *>(a.h) + row * a.d;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * TPR + t) * 8;
            store8(o + c, h[i], a.d - c, vec);
        }
    }
    ss = row_reduce<TPR, false>(ss, lds);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    const T *w = static_cast<const T *>(a.w);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * TPR + t) * 8;
        h[i] *= rstd * load8(w + c, a.d - c, vec);
    }
    if constexpr (OUT == OUT_SAME) {
        T *y = static_cast<T *>(a.y) + row * a.d;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * TPR + t) * 8;
            store8(y + c, h[i], a.d - c, vec);
        }
    } else {
        float m[ITER];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            m[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m[i] = fmaxf(m[i], fabsf(h[i][e]));
        }
        if constexpr (OUT == OUT_FP8_ROW) {
#pragma unroll
            for (int i = 1; i < ITER; ++i) m[0] = fmaxf(m[0], m[i]);
            m[0] = row_reduce<TPR, true>(m[0], lds);
#pragma unroll
            for (int i = 1; i < ITER; ++i) m[i] = m[0];
        } else {   // 128 columns are 16 neighbouring lanes
#pragma unroll
            for (int off = 1; off < 16; off <<= 1)
#pragma unroll
                for (int i = 0; i < ITER; ++i) m[i] = fmaxf(m[i], __shfl_xor(m[i], off, 64));
        }
        uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.d;
        const int groups = OUT == OUT_FP8_ROW ? 1 : (a.d + 127) / 128;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * TPR + t) * 8;
            const float scale = fmaxf(m[i], kAmaxFloor) / kE4m3Max;
            const f8v q = quotients(h[i], scale);
            uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
            uint32_t hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
            if (vec) {
                if (c < a.d) *reinterpret_cast<u2v *>(y + c) = u2v{lo, hi};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < a.d) y[c + e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
            }
            if constexpr (OUT == OUT_FP8_ROW) {
                if (c == 0) a.scale[row] = scale;
            } else {
                if ((c & 127) == 0 && c < a.d) a.scale[row * groups + (c >> 7)] = scale;
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
// A workgroup walks rows blockIdx.x RPW + sub, + gridDim.x RPW, ... and keeps
// its sums of dw in registers; it writes one row of partials, which the second
// kernel adds up in order.  The next row is fetched while this one is reduced
// (16384 x 4096 bf16, forward and gradient: 255 us without that, 201 with it).
struct NormBwdArgs {
    const void *dy, *h, *w, *dh;
    const float *rstd;
    void *dx;
    float *part;
    int64_t rows;
    int d, vec;
};

// 8 elements as they are stored
template <typename T> struct Raw;
template <> struct Raw<float> { using V = f8v; };
template <> struct Raw<__bf16> { using V = bf8v; };

template <typename T> __device__ __forceinline__ typename Raw<T>::V raw8(const T *p, int n, bool vec)
{
    typename Raw<T>::V v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (vec) {
        if (n > 0) v = *reinterpret_cast<const typename Raw<T>::V *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] = p[i];
    }
    return v;
}

template <typename T, int TPR, int ITER>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_bwd_kernel(NormBwdArgs a)
{
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    using V = typename Raw<T>::V;
    __shared__ float lds[16];
    __shared__ __align__(16) float sum[RPW > 1 ? (RPW - 1) * TPR * 8 * ITER : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const bool vec = a.vec != 0, more = a.dh != nullptr;
    f8v w[ITER], dw[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * TPR + t) * 8;
        w[i] = load8(static_cast<const T *>(a.w) + c, a.d - c, vec);
        dw[i] = f8v{0, 0, 0, 0, 0, 0, 0, 0};
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * RPW;
    // the next row's elements travel while this row's are reduced
    V hn[ITER], en[ITER], dn[ITER];
    float rn = 0.0f;
    auto fetch = [&](int64_t row) {
        if (row >= a.rows) return;
        rn = a.rstd[row];
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * TPR + t) * 8;
            hn[i] = raw8(static_cast<const T *>(a.h) + row * a.d + c, a.d - c, vec);
            en[i] = raw8(static_cast<const T *>(a.dy) + row * a.d + c, a.d - c, vec);
            if (more) dn[i] = raw8(static_cast<const T *>(a.dh) + row * a.d + c, a.d - c, vec);
        }
    };
    const int64_t first = static_cast<int64_t>(blockIdx.x) * RPW + sub;
    fetch(first);
    for (int64_t row = first; row < a.rows; row += step) {
        const float rstd = rn;
        f8v hv[ITER], ev[ITER], dv[ITER];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            hv[i] = __builtin_convertvector(hn[i], f8v);
            ev[i] = __builtin_convertvector(en[i], f8v);
            if (more) dv[i] = __builtin_convertvector(dn[i], f8v);
        }
        fetch(row + step);
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            dw[i] += ev[i] * (hv[i] * rstd);
            ev[i] *= w[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(ev[i][e], hv[i][e], dot);
        }
        dot = row_reduce<TPR, false>(dot, lds);
        const float f = rstd * rstd * (dot / static_cast<float>(a.d));
        T *dx = static_cast<T *>(a.dx) + row * a.d;
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int c = (i * TPR + t) * 8;
            f8v v = rstd * (ev[i] - hv[i] * f);
            if (more) v += dv[i];
            store8(dx + c, v, a.d - c, vec);
        }
    }
    if constexpr (RPW > 1) {   // the workgroup's rows share one row of partials
        if (sub > 0)
#pragma unroll
            for (int i = 0; i < ITER; ++i) *reinterpret_cast<f8v *>(&sum[((sub - 1) * ITER + i) * TPR * 8 + t * 8]) = dw[i];
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int j = 0; j + 1 < RPW; ++j)
#pragma unroll
            for (int i = 0; i < ITER; ++i) dw[i] += *reinterpret_cast<const f8v *>(&sum[(j * ITER + i) * TPR * 8 + t * 8]);
    }
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * a.d;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int c = (i * TPR + t) * 8;
        store8(part + c, dw[i], a.d - c, vec);
    }
}

// dw: 64 columns per workgroup, each of its 16 waves a sixteenth of the partials
__global__ void __launch_bounds__(1024) dw_kernel(const float *part, float *dw, int n, int d)
{
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    const int per = (n + 15) / 16, lo = min(n, wv * per), hi = min(n, lo + per);
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (c < d) {
        const float *p = part + c;
        int r = lo;
        for (; r + 8 <= hi; r += 8)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += p[static_cast<int64_t>(r + i) * d];
        for (; r < hi; ++r) s[0] += p[static_cast<int64_t>(r) * d];
    }
    lds[wv][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (wv == 0 && c < d) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) x += lds[i][lane];
        dw[c] = x;
    }
}

bool wide(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Threads per row and turns of 8 columns: f.template operator()<TPR, ITER>()
template <typename F> hipError_t by_width(int64_t d, F f)
{
    if (d <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (d <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    if (d <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (d <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (d <= 6144) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 3>{});
    if (d <= 8192) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    if (d <= 16384) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

int rows_per_group(int64_t d) { return d <= 1024 ? 4 : 1; }

template <typename T, int OUT> hipError_t launch_fwd(NormArgs a, hipStream_t s)
{
    return by_width(a.d, [&](auto tpr, auto iter) {
        constexpr int TPR = decltype(tpr)::value, ITER = decltype(iter)::value;
        const int rpw = rows_per_group(a.d), threads = TPR < 256 ? 256 : TPR;
        return launch_sliced((a.rows + rpw - 1) / rpw, threads, [&](int64_t first, unsigned blocks) {
            a.first = first;
            hipLaunchKernelGGL((norm_fwd_kernel<T, TPR, ITER, OUT>), dim3(blocks), dim3(threads), 0, s, a);
        });
    });
}

template <typename T> hipError_t launch_fwd(const NormArgs &a, bool fp8, hipStream_t s)
{
    if (!fp8) return launch_fwd<T, OUT_SAME>(a, s);
    return a.group ? launch_fwd<T, OUT_FP8_GROUP>(a, s) : launch_fwd<T, OUT_FP8_ROW>(a, s);
}

template <typename T> hipError_t launch_bwd(const NormBwdArgs &a, int blocks, hipStream_t s)
{
    return by_width(a.d, [&](auto tpr, auto iter) {
        constexpr int TPR = decltype(tpr)::value, ITER = decltype(iter)::value;
        hipLaunchKernelGGL((norm_bwd_kernel<T, TPR, ITER>), dim3(blocks), dim3(TPR < 256 ? 256 : TPR), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const void *x, const void *residual, const void *w, void *y, float *scale, void *h,
                              float *rstd, int64_t rows, int64_t d, int64_t x_stride, int64_t r_stride, float eps,
                              int64_t group, bool fp8, int dtype, hipStream_t s)
{
    NormArgs a{};
    a.x = x, a.res = residual, a.w = w, a.y = y, a.h = h, a.scale = scale, a.rstd = rstd;
    a.rows = rows, a.xs = x_stride, a.rs = r_stride;
    a.d = static_cast<int>(d), a.group = static_cast<int>(group), a.eps = eps;
    const int64_t per16 = dtype == MGS_BF16 ? 8 : 4;
    a.vec = d % 8 == 0 && x_stride % per16 == 0 && (!residual || r_stride % per16 == 0) && wide(x) && wide(residual) &&
            wide(w) && wide(y) && wide(h);
    return dtype == MGS_BF16 ? launch_fwd<__bf16>(a, fp8, s) : launch_fwd<float>(a, fp8, s);
}

// Workgroups of the gradient: two a CU, and no more than there are rows
NormBwdGeom norm_bwd_geometry(int64_t rows, int64_t d)
{
    NormBwdGeom g{};
    const int rpw = rows_per_group(d);
    g.blocks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(512, (rows + rpw - 1) / rpw)));
    g.off_dw = 256;
    g.bytes = g.off_dw + static_cast<size_t>(g.blocks) * d * sizeof(float);
    return g;
}

hipError_t launch_rmsnorm_bwd(const NormBwdGeom &geo, const void *dy, const void *h, const void *w,
                              const float *rstd, const void *dh, void *dx, float *dw, int64_t rows, int64_t d,
                              int dtype, void *ws, hipStream_t s)
{
    NormBwdArgs a{};
    a.dy = dy, a.h = h, a.w = w, a.dh = dh, a.rstd = rstd, a.dx = dx;
    a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + geo.off_dw);
    a.rows = rows, a.d = static_cast<int>(d);
    a.vec = d % 8 == 0 && wide(dy) && wide(h) && wide(w) && wide(dh) && wide(dx);
    hipError_t e = dtype == MGS_BF16 ? launch_bwd<__bf16>(a, geo.blocks, s) : launch_bwd<float>(a, geo.blocks, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(dw_kernel, dim3(static_cast<unsigned>((d + 63) / 64)), dim3(1024), 0, s, a.part, dw,
                       geo.blocks, a.d);
    return hipGetLastError();
}

}  // namespace mgs
