// gated.hip -- the gated linear recurrence, its gradient and its single step
// (gfx950).
//
//     log a_t = -rate softplus(lam) sigmoid(r_t),   a_t = 0 where a document starts
//     h_t = a_t h_{t-1} + beta_t sigmoid(i_t) x_t,  beta_t = sqrt(1 - a_t^2)
//
// Work decomposition: a lane owns two neighbouring channels, a wave C steps of
// 128 channels in its registers, a workgroup W waves, one tile of W C steps.  Each
// wave folds its steps into a pair (A, H), h -> A h + H; the pairs meet in LDS,
// and tiles along T pass theirs by a look-back in a fixed order (below), so every
// input is read once and every output written once.  The backward is the same
// with the steps reversed, after it has formed h again from the states that the
// forward left ahead of each 64 steps.
//
// A decay that clears the state is -0, and so is the A of a pair that holds one
// (decays are not negative otherwise): nothing that comes before, finite or not, is
// multiplied by it.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "device.hpp"
#include "launch.hpp"
#include "layers.hpp"
#include "tokens.hpp"

namespace mgs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWaves = 8;                // per workgroup
constexpr int kGroup = 128;              // channels of a workgroup
constexpr int kFwdSteps = 16, kBwdSteps = 8;   // of a wave
constexpr int kUnit = 8;                 // tiles whose pairs a tile reads at most
static_assert(kUnit <= kWaves, "each wave polls one tile");
constexpr int kFwdTile = kWaves * kFwdSteps, kBwdTile = kWaves * kBwdSteps;
static_assert(kFwdTile % MGS_GATED_CHUNK == 0 && kBwdTile % MGS_GATED_CHUNK == 0, "a tile starts at a saved state");
static_assert(MGS_GATED_CHUNK % kFwdSteps == 0, "a wave saves the state ahead of it");

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ------------------------------------------------------------ two elements
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

template <typename T> struct Two;
template <> struct Two<float> { using V = f32x2; };
template <> struct Two<__bf16> { using V = bf2v; };

// Elements c and c + 1 of a row, where they exist (c < d)
template <typename T, bool PAIRS> __device__ __forceinline__ f32x2 load2(const T *row, int c, int d)
{
    if constexpr (PAIRS) {
        c = c < d ? c : d - 2;
        return __builtin_convertvector(*reinterpret_cast<const typename Two<T>::V *>(row + c), f32x2);
    } else {
        return f32x2{static_cast<float>(row[c < d ? c : d - 1]), static_cast<float>(row[c + 1 < d ? c + 1 : d - 1])};
    }
}

template <typename T, bool PAIRS> __device__ __forceinline__ void store2(T *row, int c, int d, f32x2 v)
{
    const typename Two<T>::V o = __builtin_convertvector(v, typename Two<T>::V);
    if constexpr (PAIRS) {
        if (c < d) __builtin_nontemporal_store(o, reinterpret_cast<typename Two<T>::V *>(row + c));
    } else {
        if (c < d) row[c] = o[0];
        if (c + 1 < d) row[c + 1] = o[1];
    }
}

__device__ __forceinline__ f32x2 load_f2(const float *row, int c, int d)
{
    return f32x2{row[c < d ? c : d - 1], row[c + 1 < d ? c + 1 : d - 1]};
}

__device__ __forceinline__ void store_f2(float *row, int c, int d, f32x2 v)
{
    if (c < d) row[c] = v[0];
    if (c + 1 < d) row[c + 1] = v[1];
}

// ------------------------------------------------------------------- gates
// e^-z.  For fp32 elements the exponent's rounding is made good: e is off by up to
// 2^-24 |z| otherwise.
template <typename T> __device__ __forceinline__ float exp_neg(float z)
{
    const float t = z * -kLog2e;
    const float e = ex2(t);
    if constexpr (sizeof(T) == 2) return e;
    const float lo = __builtin_fmaf(z, -kLog2e, -t) + z * -1.925963033500e-8f;   // (log2 e - its float)
    return t > 126.0f || t < -126.0f ? e : __builtin_fmaf(e, lo * 0.6931471805599453f, e);
}

// 1 - s of s = 1 / (1 + e), without cancellation; e may be infinite
__device__ __forceinline__ float shut(float e, float s) { return e > 0x1p100f ? 1.0f : e * s; }

// a = e^l and beta^2 = 1 - a^2 for l <= 0.  Near 0 both come of p = 1 - e^l by its
// series (six terms: below 2^-24 of p up to |l| = 1/4): 1 - a^2 = p (2 - p) keeps
// p's relative accuracy, where 1 - a^2 of a rounded a would lose it.
__device__ __forceinline__ void decay(float l, float &a, float &beta2)
{
    float s = __builtin_fmaf(l, 1.0f / 7.0f, 1.0f);
    s = __builtin_fmaf(l * s, 1.0f / 6.0f, 1.0f);
    s = __builtin_fmaf(l * s, 1.0f / 5.0f, 1.0f);
    s = __builtin_fmaf(l * s, 1.0f / 4.0f, 1.0f);
    s = __builtin_fmaf(l * s, 1.0f / 3.0f, 1.0f);
    s = __builtin_fmaf(l * s, 1.0f / 2.0f, 1.0f);
    const float near = -l * s;
    const bool small = l > -0.25f;
    const float e = ex2(l * kLog2e);
    const float p = small ? near : 1.0f - e;
    a = small ? 1.0f - near : e;
    beta2 = p * (1.0f + a);
}

// -rate softplus(lam)
__device__ __forceinline__ float slope(float lam, float rate)
{
    return -rate * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam))));
}

struct Gate {
    float a, b;   // h -> a h + b
};

template <typename T> __device__ __forceinline__ Gate gate(float x, float r, float i, float k, bool fresh)
{
    const float rho = rcp(1.0f + exp_neg<T>(r)), iota = rcp(1.0f + exp_neg<T>(i));
    float a, beta2;
    decay(k * rho, a, beta2);
    const float beta = fresh ? 1.0f : __builtin_amdgcn_sqrtf(beta2);
    return Gate{fresh ? -0.0f : a, beta * iota * x};
}

__device__ __forceinline__ bool clears(float A) { return __float_as_uint(A) == 0x80000000u; }
// A h + H
__device__ __forceinline__ float apply(float A, float H, float h)
{
    return clears(A) ? H : __builtin_fmaf(A, h, H);
}
// A of the first pair, then this one
__device__ __forceinline__ float chain(float A1, float A2) { return clears(A2) ? A2 : A1 * A2; }

// ------------------------------------------------------------- look-back
// Tiles of one channel group pass on their pairs in units of kUnit tiles: the
// last tile of a unit publishes the value that leaves it, the others their pair,
// and a tile reads the value that left the unit before it and the pairs of the
// tiles ahead of it in its unit, and folds them in order: results do not depend
// on which tile was early.  Wave q polls for the q-th of these, so a tile waits for
// the slowest of them once.  Words are tagged (device.hpp).  Tile indices run in the
// direction of the pass; tiles wait for smaller blockIdx only.
struct Lookback {
    WsHeader *hd;
    uint64_t *agg, *incl;     // [tile][2][group channels], [unit][group channels], per group
    uint32_t groups, tiles;   // tiles of one group
    int local;                // every partner runs on this XCD (tagged_store)
};

struct Shared {
    f32x2 A[kWaves][64], H[kWaves][64];      // the waves' pairs
    f32x2 pA[kUnit][64], pH[kUnit][64];      // the unit's tiles' pairs; pH[0]: the value that enters the unit
    uint32_t ticket[3];
};

__device__ __forceinline__ uint64_t *agg_at(const Lookback &l, int64_t tile, int64_t group)
{
    return l.agg + ((tile * l.groups + group) * 2) * kGroup;
}

__device__ __forceinline__ uint64_t *incl_at(const Lookback &l, int64_t unit, int64_t group)
{
    return l.incl + (unit * l.groups + group) * kGroup;
}

__device__ __forceinline__ void publish2(uint64_t *p, uint32_t tag, f32x2 v, int local)
{
    tagged_store(p, tag, v[0], local);
    tagged_store(p + 1, tag, v[1], local);
}

__device__ __forceinline__ f32x2 await2(const Lookback &l, const uint64_t *p, uint32_t want, uint32_t limit)
{
    for (uint32_t spin = 0;;) {
        uint64_t w0, w1;
        const bool r0 = poll(p, want, w0), r1 = poll(p + 1, want, w1);
        if (__all(r0 && r1)) return f32x2{tag_value(w0), tag_value(w1)};
        if (++spin >= limit) {
            if ((threadIdx.x & 63) == 0) raise_error(&l.hd->err, kErrSpin);
            return f32x2{0.0f, 0.0f};
        }
        backoff();
    }
}

// Whole-workgroup: the value that enters tile j, from `first` at the first one.
// sh.A, sh.H hold the waves' pairs in the order of the pass (barrier done, epoch_end
// done).  Publishes what later tiles read.
__device__ __forceinline__ f32x2 enter(const Lookback &l, Shared &sh, uint32_t j, int64_t group, f32x2 first)
{
    const int lane = threadIdx.x & 63, wv = wave();
    const uint32_t tag = sh.ticket[0], want = sh.ticket[1], limit = sh.ticket[2];
    const uint32_t unit = j / kUnit, at = j % kUnit;
    const bool closes = at == kUnit - 1;
    f32x2 TA = {1.0f, 1.0f}, TH = {0.0f, 0.0f};
    if (wv == 0) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const f32x2 A = sh.A[w][lane], H = sh.H[w][lane];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                TH[v] = apply(A[v], H[v], TH[v]);
                TA[v] = chain(TA[v], A[v]);
            }
        }
        if (!closes && j + 1 < l.tiles) {
            uint64_t *p = agg_at(l, j, group) + 2 * lane;
            publish2(p, tag, TA, l.local);
            publish2(p + kGroup, tag, TH, l.local);
        }
    }
    if (wv <= static_cast<int>(at)) {
        if (wv == 0) {
            sh.pH[0][lane] = unit == 0 ? first : await2(l, incl_at(l, unit - 1, group) + 2 * lane, want, limit);
        } else {
            const uint64_t *p = agg_at(l, static_cast<int64_t>(unit) * kUnit + wv - 1, group) + 2 * lane;
            sh.pA[wv][lane] = await2(l, p, want, limit);
            sh.pH[wv][lane] = await2(l, p + kGroup, want, limit);
        }
    }
    __syncthreads();
    f32x2 c = sh.pH[0][lane];
    for (uint32_t q = 1; q <= at; ++q) {
        const f32x2 A = sh.pA[q][lane], H = sh.pH[q][lane];
#pragma unroll
        for (int v = 0; v < 2; ++v) c[v] = apply(A[v], H[v], c[v]);
    }
    if (wv == 0 && closes && j + 1 < l.tiles) {
        f32x2 out;
#pragma unroll
        for (int v = 0; v < 2; ++v) out[v] = apply(TA[v], TH[v], c[v]);
        publish2(incl_at(l, unit, group) + 2 * lane, tag, out, l.local);
    }
    return c;
}

struct GatedArgs {
    const void *x, *r, *i, *dy;
    const float *lam, *h0, *dhT;
    const int32_t *lengths;
    const uint8_t *reset;
    float *states;        // (read by the backward)
    void *y, *dx, *dr, *di;
    float *hT, *dh0;
    uint64_t *part;       // backward: sums of dl rho, [sequence and tile][channel], tagged words
    int64_t T, D, chunks;
    uint32_t per_seq;     // groups of one sequence
    int64_t xs[2], rs[2], is[2], gs[2];
    float rate;
    Lookback l;
};

// Where a workgroup is
struct Place {
    int64_t b;
    uint32_t group, j;   // j: tile in the direction of the pass
    int c, d;          // this lane's first channel, of d
    int64_t n;         // live steps of the sequence
};

__device__ __forceinline__ Place place(const GatedArgs &a)
{
    Place p;
    p.j = blockIdx.x / a.l.groups;
    p.group = blockIdx.x - p.j * a.l.groups;
    const uint32_t b = p.group / a.per_seq;
    p.b = b;
    p.c = static_cast<int>(p.group - b * a.per_seq) * kGroup + 2 * (threadIdx.x & 63);
    p.d = static_cast<int>(a.D);
    p.n = a.T;
    if (a.lengths) {
        const int64_t n = a.lengths[p.b];
        p.n = n < 0 ? 0 : n < a.T ? n : a.T;
    }
    return p;
}

// Which of the wave's N steps from t0 on start a document
template <int N> __device__ __forceinline__ uint64_t resets(const GatedArgs &a, const Place &p, int64_t t0)
{
    if (!a.reset) return 0;
    const int lane = threadIdx.x & 63;
    const bool in = lane < N && t0 + lane < p.n;
    return __ballot(in && a.reset[p.b * a.T + t0 + lane] != 0);
}

template <typename T, bool PAIRS, bool MULTI>
__global__ void __launch_bounds__(64 * kWaves) gated_fwd_kernel(GatedArgs a)
{
    constexpr int C = kFwdSteps;
    __shared__ Shared sh;
    const int lane = threadIdx.x & 63, wv = wave();
    const Place p = place(a);
    const int64_t t0 = static_cast<int64_t>(p.j) * kFwdTile + wv * C;
    const T *x = static_cast<const T *>(a.x) + p.b * a.xs[0];
    const T *r = static_cast<const T *>(a.r) + p.b * a.rs[0];
    const T *in = static_cast<const T *>(a.i) + p.b * a.is[0];

    // steps past the length read the last live row again (nothing, where there is none)
    f32x2 rx[C], rr[C], ri[C];
    if (t0 < p.n) {
#pragma unroll
        for (int s = 0; s < C; ++s) {
            const int64_t t = t0 + s < p.n ? t0 + s : p.n - 1;
            rx[s] = load2<T, PAIRS>(x + t * a.xs[1], p.c, p.d);
            rr[s] = load2<T, PAIRS>(r + t * a.rs[1], p.c, p.d);
            ri[s] = load2<T, PAIRS>(in + t * a.is[1], p.c, p.d);
        }
    } else {
#pragma unroll
        for (int s = 0; s < C; ++s) rx[s] = rr[s] = ri[s] = f32x2{0.0f, 0.0f};
    }
    Launch ep{0, 0};
    if constexpr (MULTI) ep = epoch_begin(a.l.hd);
    f32x2 k = load_f2(a.lam, p.c, p.d), first = {0.0f, 0.0f};
    if (a.h0) first = load_f2(a.h0 + p.b * a.D, p.c, p.d);
#pragma unroll
    for (int v = 0; v < 2; ++v) k[v] = slope(k[v], a.rate);
    const uint64_t fresh = resets<C>(a, p, t0);

    f32x2 ga[C], gb[C], A = {1.0f, 1.0f}, H = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < C; ++s) {
        const bool live = t0 + s < p.n;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const Gate g = gate<T>(rx[s][v], rr[s][v], ri[s][v], k[v], (fresh >> s) & 1);
            ga[s][v] = live ? g.a : 1.0f;
            gb[s][v] = live ? g.b : 0.0f;
            H[v] = apply(ga[s][v], gb[s][v], H[v]);
            A[v] = chain(A[v], ga[s][v]);
        }
    }
    sh.A[wv][lane] = A;
    sh.H[wv][lane] = H;
    if (MULTI && threadIdx.x == 0) epoch_end(a.l.hd, ep, a.l.tiles * a.l.groups, sh.ticket);
    __syncthreads();
    f32x2 h = first;
    if constexpr (MULTI) h = enter(a.l, sh, p.j, p.group, first);
    for (int w = 0; w < wv; ++w) {
        const f32x2 wA = sh.A[w][lane], wH = sh.H[w][lane];
#pragma unroll
        for (int v = 0; v < 2; ++v) h[v] = apply(wA[v], wH[v], h[v]);
    }
    if (a.states && t0 % MGS_GATED_CHUNK == 0 && t0 < a.T)
        store_f2(a.states + (p.b * a.chunks + t0 / MGS_GATED_CHUNK) * a.D, p.c, p.d, h);
    T *y = static_cast<T *>(a.y) + p.b * a.T * a.D;
#pragma unroll
    for (int s = 0; s < C; ++s) {
#pragma unroll
        for (int v = 0; v < 2; ++v) h[v] = apply(ga[s][v], gb[s][v], h[v]);
        if (t0 + s < a.T)
            store2<T, PAIRS>(y + (t0 + s) * a.D, p.c, p.d, t0 + s < p.n ? h : f32x2{0.0f, 0.0f});
    }
    if (a.hT && p.j + 1 == a.l.tiles && wv == kWaves - 1) store_f2(a.hT + p.b * a.D, p.c, p.d, h);
}

template <typename T, bool PAIRS, bool MULTI>
__global__ void __launch_bounds__(64 * kWaves) gated_bwd_kernel(GatedArgs a)
{
    constexpr int C = kBwdSteps;
    __shared__ Shared sh;
    __shared__ f32x2 sF[2][kWaves][64];   // the waves' pairs of the forward; later their sums of dl rho
    const int lane = threadIdx.x & 63;
    const int pass = wave(), wv = kWaves - 1 - pass;   // in the order of the pass, and of the steps
    const Place p = place(a);
    const int64_t tile = static_cast<int64_t>(a.l.tiles) - 1 - p.j;
    const int64_t t0 = tile * kBwdTile + wv * C;
    const T *x = static_cast<const T *>(a.x) + p.b * a.xs[0];
    const T *r = static_cast<const T *>(a.r) + p.b * a.rs[0];
    const T *in = static_cast<const T *>(a.i) + p.b * a.is[0];
    const T *dy = static_cast<const T *>(a.dy) + p.b * a.gs[0];

    f32x2 rx[C], rr[C], ri[C], g[C];
    if (t0 < p.n) {
#pragma unroll
        for (int s = 0; s < C; ++s) {
            const int64_t t = t0 + s < p.n ? t0 + s : p.n - 1;
            rx[s] = load2<T, PAIRS>(x + t * a.xs[1], p.c, p.d);
            rr[s] = load2<T, PAIRS>(r + t * a.rs[1], p.c, p.d);
            ri[s] = load2<T, PAIRS>(in + t * a.is[1], p.c, p.d);
            g[s] = load2<T, PAIRS>(dy + t * a.gs[1], p.c, p.d);
        }
    } else {
#pragma unroll
        for (int s = 0; s < C; ++s) rx[s] = rr[s] = ri[s] = g[s] = f32x2{0.0f, 0.0f};
    }
    Launch ep{0, 0};
    if constexpr (MULTI) ep = epoch_begin(a.l.hd);
    f32x2 k = load_f2(a.lam, p.c, p.d), first = {0.0f, 0.0f}, h = {0.0f, 0.0f};
    if (a.dhT) first = load_f2(a.dhT + p.b * a.D, p.c, p.d);
    if (tile * kBwdTile < a.T)
        h = load_f2(a.states + (p.b * a.chunks + tile * (kBwdTile / MGS_GATED_CHUNK)) * a.D, p.c, p.d);
#pragma unroll
    for (int v = 0; v < 2; ++v) k[v] = slope(k[v], a.rate);
    const uint64_t fresh = resets<C>(a, p, t0);

    // Per step: the decay, and what G multiplies: m1 -> dx, m2 -> di, and for dl rho
    // first iota x a^2 / beta, then (a h_{t-1} - that) rho
    f32x2 ga[C], gb[C], m1[C], m2[C], w[C], rho[C], late[C];
    f32x2 A = {1.0f, 1.0f}, H = {0.0f, 0.0f}, K = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < C; ++s) {
        const bool live = t0 + s < p.n, fr = (fresh >> s) & 1;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float er = exp_neg<T>(rr[s][v]), ei = exp_neg<T>(ri[s][v]);
            const float rh = rcp(1.0f + er), io = rcp(1.0f + ei);
            float da, beta2;
            decay(k[v] * rh, da, beta2);
            const float beta = fr ? 1.0f : __builtin_amdgcn_sqrtf(beta2);
            const float ix = io * rx[s][v];
            const float b = beta * ix;
            ga[s][v] = live ? (fr ? -0.0f : da) : 1.0f;
            gb[s][v] = live ? b : 0.0f;
            m1[s][v] = beta * io;
            m2[s][v] = b * shut(ei, io);
            w[s][v] = fr || beta == 0.0f ? 0.0f : ix * (da * da) * rcp(beta);
            rho[s][v] = rh;
            late[s][v] = shut(er, rh);
            if (!live) g[s][v] = 0.0f;
            H[v] = apply(ga[s][v], gb[s][v], H[v]);
            A[v] = chain(A[v], ga[s][v]);
        }
    }
    sF[0][wv][lane] = A;
    sF[1][wv][lane] = H;
#pragma unroll
    for (int s = C - 1; s >= 0; --s)
#pragma unroll
        for (int v = 0; v < 2; ++v) K[v] = clears(ga[s][v]) ? 0.0f : ga[s][v] * (g[s][v] + K[v]);
    sh.A[pass][lane] = A;
    sh.H[pass][lane] = K;
    if (MULTI && threadIdx.x == 0) epoch_end(a.l.hd, ep, a.l.tiles * a.l.groups, sh.ticket);
    __syncthreads();
    for (int q = 0; q < wv; ++q) {
        const f32x2 wA = sF[0][q][lane], wH = sF[1][q][lane];
#pragma unroll
        for (int v = 0; v < 2; ++v) h[v] = apply(wA[v], wH[v], h[v]);
    }
#pragma unroll
    for (int s = 0; s < C; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const bool clear = clears(ga[s][v]);
            const float ah = clear ? 0.0f : ga[s][v] * h[v];
            w[s][v] = clear ? 0.0f : (ah - w[s][v]) * rho[s][v];
            h[v] = ah + gb[s][v];
        }
    K = first;
    if constexpr (MULTI) K = enter(a.l, sh, p.j, p.group, first);
    for (int q = 0; q < pass; ++q) {
        const f32x2 wA = sh.A[q][lane], wK = sh.H[q][lane];
#pragma unroll
        for (int v = 0; v < 2; ++v) K[v] = apply(wA[v], wK[v], K[v]);
    }
    T *dx = static_cast<T *>(a.dx) + p.b * a.T * a.D, *dr = static_cast<T *>(a.dr) + p.b * a.T * a.D;
    T *di = static_cast<T *>(a.di) + p.b * a.T * a.D;
    f32x2 sum = {0.0f, 0.0f};
#pragma unroll
    for (int s = C - 1; s >= 0; --s) {
        f32x2 ox, orr, oi;
        const bool live = t0 + s < p.n;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float G = g[s][v] + K[v];
            const float dl = G * w[s][v];
            ox[v] = live ? G * m1[s][v] : 0.0f;
            oi[v] = live ? G * m2[s][v] : 0.0f;
            orr[v] = live ? dl * k[v] * late[s][v] : 0.0f;
            sum[v] += live ? dl : 0.0f;
            K[v] = clears(ga[s][v]) ? 0.0f : ga[s][v] * G;
        }
        if (t0 + s < a.T) {
            store2<T, PAIRS>(dx + (t0 + s) * a.D, p.c, p.d, ox);
            store2<T, PAIRS>(dr + (t0 + s) * a.D, p.c, p.d, orr);
            store2<T, PAIRS>(di + (t0 + s) * a.D, p.c, p.d, oi);
        }
    }
    if (a.dh0 && tile == 0 && wv == 0) store_f2(a.dh0 + p.b * a.D, p.c, p.d, K);
    __syncthreads();
    sF[0][wv][lane] = sum;
    __syncthreads();
    if (wv == 0) {
        for (int q = 1; q < kWaves; ++q) sum += sF[0][q][lane];
        uint64_t *o = a.part + (p.b * a.l.tiles + tile) * a.D;
        const uint32_t tag = MULTI ? sh.ticket[0] : 0;   // (never the tag of a later launch)
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (p.c + v < p.d)
                o[p.c + v] = (static_cast<uint64_t>(tag) << 32) | __float_as_uint(sum[v]);
    }
}

// dlam: the partial sums of a channel in order, in fp64, over 16 waves' shares
__global__ void __launch_bounds__(1024) gated_dlam_kernel(const uint64_t *part, const float *lam, float *dlam,
                                                         int64_t first, int64_t rows, int64_t D, float rate)
{
    __shared__ double s[16][64];
    const int lane = threadIdx.x & 63, wv = wave();
    const int64_t c = (first + blockIdx.x) * 64 + lane, cc = c < D ? c : D - 1;
    const int64_t share = (rows + 15) / 16;
    double sum = 0.0;
    for (int64_t i = wv * share; i < (wv + 1) * share && i < rows; ++i)
        sum += static_cast<double>(tag_value(part[i * D + cc]));
    s[wv][lane] = sum;
    __syncthreads();
    if (wv != 0 || c >= D) return;
    for (int q = 1; q < 16; ++q) sum += s[q][lane];
    const float z = lam[c];
    dlam[c] = rows == 0 ? 0.0f : static_cast<float>(sum * (-static_cast<double>(rate) / (1.0 + exp(-static_cast<double>(z)))));
}

struct StepArgs {
    const void *x, *r, *i;
    const float *lam;
    float *h;
    const int32_t *slots;
    void *y;
    int64_t first, blocks_per_row, xs, rs, is, D, n_slots;
    float rate;
};

// One workgroup: up to 512 channels of a sequence
template <typename T, bool PAIRS> __global__ void __launch_bounds__(256) gated_step_kernel(StepArgs a)
{
    const int64_t at = a.first + blockIdx.x, b = at / a.blocks_per_row;
    const int c = static_cast<int>(at - b * a.blocks_per_row) * 512 + 2 * threadIdx.x, d = static_cast<int>(a.D);
    if (c >= d) return;
    const int64_t slot = a.slots ? a.slots[b] : b;
    T *y = static_cast<T *>(a.y) + b * a.D;
    if (slot < 0 || slot >= a.n_slots) {
        store2<T, PAIRS>(y, c, d, f32x2{0.0f, 0.0f});
        return;
    }
    const f32x2 x = load2<T, PAIRS>(static_cast<const T *>(a.x) + b * a.xs, c, d);
    const f32x2 r = load2<T, PAIRS>(static_cast<const T *>(a.r) + b * a.rs, c, d);
    const f32x2 i = load2<T, PAIRS>(static_cast<const T *>(a.i) + b * a.is, c, d);
    const f32x2 lam = load_f2(a.lam, c, d);
    float *row = a.h + slot * a.D;
    f32x2 h = load_f2(row, c, d);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const Gate g = gate<T>(x[v], r[v], i[v], slope(lam[v], a.rate), false);
        h[v] = __builtin_fmaf(g.a, h[v], g.b);
    }
    store_f2(row, c, d, h);
    store2<T, PAIRS>(y, c, d, h);
}

bool even(const int64_t *st, int n)
{
    for (int i = 0; i < n; ++i)
        if (st[i] & 1) return false;
    return true;
}

// whether two neighbouring elements can be moved at once everywhere
bool pairs(const mgs_gated_desc &d, int strides, std::initializer_list<const void *> ptrs)
{
    const uintptr_t mask = (d.dtype == MGS_BF16 ? 4 : 8) - 1;
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & mask) return false;
    return (d.D & 1) == 0 && even(d.x_stride, strides) && even(d.r_stride, strides) && even(d.i_stride, strides);
}

GatedArgs arguments(const GatedGeom &g, const mgs_gated_desc &d, int64_t tiles, void *ws)
{
    GatedArgs a{};
    char *w = static_cast<char *>(ws);
    a.T = d.T;
    a.D = d.D;
    a.chunks = (d.T + MGS_GATED_CHUNK - 1) / MGS_GATED_CHUNK;
    a.per_seq = static_cast<uint32_t>((d.D + kGroup - 1) / kGroup);
    for (int i = 0; i < 2; ++i) {
        a.xs[i] = d.x_stride[i];
        a.rs[i] = d.r_stride[i];
        a.is[i] = d.i_stride[i];
        a.gs[i] = d.dy_stride[i];
    }
    a.rate = d.rate;
    a.l.hd = reinterpret_cast<WsHeader *>(w);
    a.l.agg = reinterpret_cast<uint64_t *>(w + g.off_agg);
    a.l.incl = reinterpret_cast<uint64_t *>(w + g.off_incl);
    a.part = reinterpret_cast<uint64_t *>(w + g.off_part);
    a.l.groups = static_cast<uint32_t>(g.groups);
    a.l.tiles = static_cast<uint32_t>(tiles);
    const int xcds = xcd_count();
    a.l.local = xcds > 0 && g.groups % xcds == 0;
    return a;
}

template <typename T> hipError_t run_fwd(const GatedArgs &a, bool two, hipStream_t s)
{
    const dim3 grid(a.l.groups * a.l.tiles), block(64 * kWaves);
    if (a.l.tiles > 1) {
        if (two) gated_fwd_kernel<T, true, true><<<grid, block, 0, s>>>(a);
        else gated_fwd_kernel<T, false, true><<<grid, block, 0, s>>>(a);
    } else {
        if (two) gated_fwd_kernel<T, true, false><<<grid, block, 0, s>>>(a);
        else gated_fwd_kernel<T, false, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename T> hipError_t run_bwd(const GatedArgs &a, bool two, hipStream_t s)
{
    const dim3 grid(a.l.groups * a.l.tiles), block(64 * kWaves);
    if (a.l.tiles > 1) {
        if (two) gated_bwd_kernel<T, true, true><<<grid, block, 0, s>>>(a);
        else gated_bwd_kernel<T, false, true><<<grid, block, 0, s>>>(a);
    } else {
        if (two) gated_bwd_kernel<T, true, false><<<grid, block, 0, s>>>(a);
        else gated_bwd_kernel<T, false, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

GatedGeom gated_geometry(const mgs_gated_desc &d, bool backward)
{
    GatedGeom g{};
    g.groups = d.B * ((d.D + kGroup - 1) / kGroup);
    // (no steps: one tile, which hands the state on)
    g.tiles_f = std::max<int64_t>(1, (d.T + kFwdTile - 1) / kFwdTile);
    g.tiles_b = std::max<int64_t>(1, (d.T + kBwdTile - 1) / kBwdTile);
    const int64_t tiles = backward ? std::max(g.tiles_f, g.tiles_b) : g.tiles_f;
    // every word behind the header is a tagged one, whatever call it is written by,
    // so that a call of other sizes takes none of them for its own
    size_t off = sizeof(WsHeader);
    g.off_agg = off;
    if (tiles > 1) off = align256(off + static_cast<size_t>(tiles) * g.groups * 2 * kGroup * 8);
    g.off_incl = off;
    if (tiles > 1) off = align256(off + static_cast<size_t>(tiles / kUnit) * g.groups * kGroup * 8);
    g.off_part = off;
    if (backward) off = align256(off + static_cast<size_t>(g.tiles_b) * d.B * d.D * 8);
    g.bytes = off;
    return g;
}

hipError_t launch_gated_fwd(const GatedGeom &g, const mgs_gated_desc &d, const void *x, const void *r, const void *i,
                            const float *lam, const float *h0, const int32_t *lengths, const uint8_t *reset, void *y,
                            float *hT, float *states, void *ws, hipStream_t s)
{
    GatedArgs a = arguments(g, d, g.tiles_f, ws);
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.h0 = h0; a.lengths = lengths; a.reset = reset;
    a.y = y; a.hT = hT; a.states = states;
    const bool two = pairs(d, 2, {x, r, i, y});
    return d.dtype == MGS_BF16 ? run_fwd<__bf16>(a, two, s) : run_fwd<float>(a, two, s);
}

hipError_t launch_gated_bwd(const GatedGeom &g, const mgs_gated_desc &d, const void *x, const void *r, const void *i,
                            const float *lam, const void *dy, const float *dhT, const float *states,
                            const int32_t *lengths, const uint8_t *reset, void *dx, void *dr, void *di, float *dlam,
                            float *dh0, void *ws, hipStream_t s)
{
    GatedArgs a = arguments(g, d, g.tiles_b, ws);
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.dy = dy; a.dhT = dhT; a.lengths = lengths; a.reset = reset;
    a.states = const_cast<float *>(states);
    a.dx = dx; a.dr = dr; a.di = di; a.dh0 = dh0;
    int64_t rows = 0;
    if (d.B > 0) {
        const bool two = pairs(d, 2, {x, r, i, dy, dx, dr, di}) && even(d.dy_stride, 2);
        const hipError_t e = d.dtype == MGS_BF16 ? run_bwd<__bf16>(a, two, s) : run_bwd<float>(a, two, s);
        if (e != hipSuccess) return e;
        rows = d.T > 0 ? d.B * g.tiles_b : 0;
    }
    return launch_sliced((d.D + 63) / 64, 1024, [&](int64_t first, unsigned blocks) {
        gated_dlam_kernel<<<dim3(blocks), dim3(1024), 0, s>>>(a.part, lam, dlam, first, rows, d.D, d.rate);
    });
}

hipError_t launch_gated_step(const mgs_gated_desc &d, const void *x, const void *r, const void *i, const float *lam,
                             float *h, int64_t n_slots, const int32_t *slots, void *y, hipStream_t s)
{
    StepArgs a{x, r, i, lam, h, slots, y, 0, (d.D + 511) / 512, d.x_stride[0], d.r_stride[0], d.i_stride[0], d.D,
               n_slots, d.rate};
    const bool two = pairs(d, 1, {x, r, i, y});
    return launch_sliced(d.B * a.blocks_per_row, 256, [&](int64_t first, unsigned blocks) {
        a.first = first;
        const dim3 grid(blocks), block(256);
        if (d.dtype == MGS_BF16) {
            if (two) gated_step_kernel<__bf16, true><<<grid, block, 0, s>>>(a);
            else gated_step_kernel<__bf16, false><<<grid, block, 0, s>>>(a);
        } else {
            if (two) gated_step_kernel<float, true><<<grid, block, 0, s>>>(a);
            else gated_step_kernel<float, false><<<grid, block, 0, s>>>(a);
        }
    });
}

}  // namespace mgs
