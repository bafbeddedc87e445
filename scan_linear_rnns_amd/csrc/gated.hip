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
//
// What bounds it: HBM, and in the bf16 backward the gates' operations beside it (35 an
// element forward, 77 backward, the reciprocals, exponentials and roots among them a
// quarter as fast as the others).  Medians of kernels: 1 x 65536 x 1024, bf16: 118 us, 4.7
// TB/s (a copy: 5.0); 4 x 4096 x 4096, bf16: 117 and 231 + 6 for dlam, 4.7 and 4.5 TB/s, the
// VALU 60 and 69 % busy (the shortest 111 and 213); 16 x 1024 x 1000, fp32: 59 and 113 + 5, 5.1
// and 4.6 TB/s.  A step of 256 x 4096: 7.5 us, of it 3 for the launch and 3.3 for the bytes.
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
constexpr int kGroup = 128;              // channels of a workgroup
constexpr int kPollers = 7;              // waves of a workgroup that read other tiles' pairs
// Waves of a workgroup, steps of a wave, and how many waves share a SIMD
template <int WAVES, int STEPS, int OCCUPANCY> struct Shape {
    static constexpr int W = WAVES, C = STEPS, occupancy = OCCUPANCY, tile = W * C;
    static constexpr bool several = W > kPollers;   // serves several tiles along T
    static_assert(!several || tile % MGS_GATED_CHUNK == 0, "a tile starts at a saved state");
    static_assert(MGS_GATED_CHUNK % C == 0, "a wave saves the state ahead of it");
};
// Measured (us at 4 x 4096 x 4096, bf16, and 16 x 1024 x 1000, fp32).  Forward 8 waves
// of 16 steps: 118 and 60; of 8 steps: 130 and 59 (and 74 against 57 on a ragged prompt);
// 16 waves of 8: 162 and 74.  Backward 8 waves of 8 steps, 128 registers (the fp32 one
// would spill, and takes 157, two waves a SIMD): 237 and 131; fp32 with 128: 141; bf16 with
// 133: 314; 16 waves of 4 steps: 315 and 137; of 8: 281 and 165.  (All with look-back
// units of 22 tiles; with those below the ones taken need 111 and 58, 219 and 112.)
template <typename T> struct Fwd : Shape<8, 16, 4> {};
template <typename T> struct Bwd : Shape<8, 8, 2> {};
template <> struct Bwd<__bf16> : Shape<8, 8, 4> {};

// Sequences of up to 16 steps (64 of 4 x 4096, bf16: 11 and 17 us, with the shapes above 27
// and 36).  Shorter ones load and evaluate 16 too, the last live one again.
constexpr int kShort = 16;
struct FwdShort : Shape<1, kShort, 4> {};
struct BwdShort : Shape<2, kShort / 2, 2> {};

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }

__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ------------------------------------------------------------ two elements
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

template <typename T> struct Two;
template <> struct Two<float> { using V = f32x2; };
template <> struct Two<__bf16> { using V = bf2v; };

// A lane's two channels, c and c + 1 of the d that its workgroup has: byte offsets from
// the first of them, past the last channel the last one's (those results are not
// stored).
template <typename T, bool PAIRS> struct Lane {
    uint32_t at, next;
    bool in, both;
    __device__ __forceinline__ Lane(int c, int d) : in(c < d), both(c + 1 < d)
    {
        const int size = sizeof(T);
        if constexpr (PAIRS) {
            at = static_cast<uint32_t>((in ? c : d - 2) * size);
            next = at + size;
        } else {
            at = static_cast<uint32_t>((in ? c : d - 1) * size);
            next = static_cast<uint32_t>((both ? c + 1 : d - 1) * size);
        }
    }
    __device__ __forceinline__ typename Two<T>::V load(const char *row) const
    {
        if constexpr (PAIRS)
            return *reinterpret_cast<const typename Two<T>::V *>(row + at);
        else
            return typename Two<T>::V{*reinterpret_cast<const T *>(row + at), *reinterpret_cast<const T *>(row + next)};
    }
    // (in a lane that is `in`)
    __device__ __forceinline__ void store(char *row, f32x2 v) const
    {
        const typename Two<T>::V o = __builtin_convertvector(v, typename Two<T>::V);
        if constexpr (PAIRS) {
            __builtin_nontemporal_store(o, reinterpret_cast<typename Two<T>::V *>(row + at));
        } else {
            *reinterpret_cast<T *>(row + at) = o[0];
            if (both) *reinterpret_cast<T *>(row + next) = o[1];
        }
    }
};

template <typename V> __device__ __forceinline__ f32x2 wide(V v) { return __builtin_convertvector(v, f32x2); }

// Holds the compiler to computing v here: it would put off what is needed only behind
// the barriers, and keep the operands, which are more
__device__ __forceinline__ void settle(f32x2 &v)
{
    float x = v[0], y = v[1];
    asm volatile("" : "+v"(x), "+v"(y));
    v = f32x2{x, y};
}

// wide(v), later: hides that things of v have been computed before, which would be kept
// all the while
template <typename V> __device__ __forceinline__ f32x2 again(V v)
{
    if constexpr (sizeof(V) == 4) {
        uint32_t u = __builtin_bit_cast(uint32_t, v);
        asm volatile("" : "+v"(u));
        return wide(__builtin_bit_cast(V, u));
    } else {
        asm volatile("" : "+v"(v));
        return v;
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

// a = 2^l and beta^2 = 1 - a^2 for l <= 0 (log2 a; -inf where a document starts).  1 - a loses
// what a rounds away where a is near 1: 2^-20.4 of it at |l| = 1/16 with an a that is rounded
// once, 2^-19.4 with one that is an ulp off.  Below that the series of 1 - 2^l takes its place,
// four terms, off by 2^-22.5 at most.
__device__ __forceinline__ void decay(float l, float &a, float &beta2)
{
    a = ex2(l);
    float s = __builtin_fmaf(l, -9.618129107628477e-3f, -5.550410866482158e-2f);
    s = __builtin_fmaf(l, s, -2.402265069591007e-1f);
    s = __builtin_fmaf(l, s, -6.931471805599453e-1f);
    const float p = l > -0.0625f ? l * s : 1.0f - a;
    beta2 = __builtin_fmaf(p, a, p);
}

// -rate softplus(lam), and that in base 2
__device__ __forceinline__ float slope(float lam, float rate)
{
    return -rate * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam))));
}
__device__ __forceinline__ float slope2(float lam, float rate) { return slope(lam, rate) * kLog2e; }

struct Gate {
    float a, b;   // h -> a h + b
};

// k: slope2; start: -inf where a document starts, 0 elsewhere
template <typename T> __device__ __forceinline__ Gate gate(float x, float r, float i, float k, float start)
{
    const float rho = rcp(1.0f + exp_neg<T>(r)), iota = rcp(1.0f + exp_neg<T>(i));
    float a, beta2;
    decay(__builtin_fmaf(k, rho, start), a, beta2);
    return Gate{a, __builtin_amdgcn_sqrtf(beta2) * iota * x};
}

__device__ __forceinline__ bool clears(float A) { return __float_as_uint(A) == 0x80000000u; }
// A h + H
__device__ __forceinline__ float apply(float A, float H, float h)
{
    return clears(A) ? H : __builtin_fmaf(A, h, H);
}
// A of the first pair, then this one
__device__ __forceinline__ float chain(float A1, float A2) { return clears(A2) ? A2 : A1 * A2; }
// The pair (A, H), then (A2, H2)
__device__ __forceinline__ void append(f32x2 &A, f32x2 &H, f32x2 A2, f32x2 H2)
{
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        H[v] = apply(A2[v], H2[v], H[v]);
        A[v] = chain(A[v], A2[v]);
    }
}
__device__ __forceinline__ f32x2 apply2(f32x2 A, f32x2 H, f32x2 h)
{
    return f32x2{apply(A[0], H[0], h[0]), apply(A[1], H[1], h[1])};
}

// ------------------------------------------------------------- look-back
// Tiles of one channel group pass on their pairs in units of l.unit tiles: the last
// tile of a unit publishes the value that leaves it, the others their pair, and a tile
// reads the value that left the unit before it and the pairs of the tiles ahead of it in
// its unit, and folds them in order: results do not depend on which tile was early.
// Wave 0 polls for the first, the others for l.per pairs each, so a tile waits for the
// slowest of them once.  Words are tagged (device.hpp).  Tile indices run in the
// direction of the pass; tiles wait for smaller blockIdx only.
struct Lookback {
    WsHeader *hd;
    uint64_t *agg, *incl;     // [tile][2][group channels], [unit][group channels], per group
    uint32_t groups, tiles;   // tiles of one group
    uint32_t unit, per;
    int local;                // every partner runs on this XCD (tagged_store)
};

template <int W> struct Shared {
    f32x2 A[W][64], H[W][64];      // the waves' pairs; then those of all waves ahead of each
    f32x2 pA[kPollers + 1][64], pH[kPollers + 1][64];   // the unit's pairs, each of l.per tiles; pH[0]: what enters it
    float k[kGroup];                         // slope2
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

// Whole-workgroup: the value that enters wave `pass` of tile j, from `first` at the
// first one.  sh.A, sh.H hold the waves' pairs in the order of the pass (barrier and, with
// MULTI, epoch_end done).  Publishes what later tiles read.
template <bool MULTI, int W>
__device__ __forceinline__ f32x2 enter(const Lookback &l, Shared<W> &sh, uint32_t j, uint32_t group, int pass, f32x2 first)
{
    const int lane = threadIdx.x & 63;
    const uint32_t tag = sh.ticket[0], want = sh.ticket[1], limit = sh.ticket[2];
    const uint32_t unit = MULTI ? j / l.unit : 0, at = j - unit * l.unit;
    const bool closes = at == l.unit - 1;
    f32x2 TA = {1.0f, 1.0f}, TH = {0.0f, 0.0f};
    if (pass == 0) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const f32x2 A = sh.A[w][lane], H = sh.H[w][lane];
            sh.A[w][lane] = TA;
            sh.H[w][lane] = TH;
            append(TA, TH, A, H);
        }
        if (MULTI && !closes && j + 1 < l.tiles) {
            uint64_t *p = agg_at(l, j, group) + 2 * lane;
            publish2(p, tag, TA, l.local);
            publish2(p + kGroup, tag, TH, l.local);
        }
    }
    if constexpr (MULTI) {
        if (pass == 0) {
            sh.pH[0][lane] = unit == 0 ? first : await2(l, incl_at(l, unit - 1, group) + 2 * lane, want, limit);
        } else if (pass <= kPollers) {
            const uint32_t end = pass * l.per < at ? pass * l.per : at;
            uint32_t q = (pass - 1) * l.per;
            f32x2 A = {1.0f, 1.0f}, H = {0.0f, 0.0f};
            const bool any = q < end;
            for (; q < end; ++q) {
                const uint64_t *p = agg_at(l, static_cast<int64_t>(unit) * l.unit + q, group) + 2 * lane;
                const f32x2 A2 = await2(l, p, want, limit), H2 = await2(l, p + kGroup, want, limit);
                append(A, H, A2, H2);
            }
            if (any) {
                sh.pA[pass][lane] = A;
                sh.pH[pass][lane] = H;
            }
        }
    }
    __syncthreads();
    f32x2 c = first;
    if constexpr (MULTI) {
        c = sh.pH[0][lane];
        for (uint32_t q = 1; (q - 1) * l.per < at; ++q) c = apply2(sh.pA[q][lane], sh.pH[q][lane], c);
        if (pass == 0 && closes && j + 1 < l.tiles)
            publish2(incl_at(l, unit, group) + 2 * lane, tag, apply2(TA, TH, c), l.local);
    }
    return apply2(sh.A[pass][lane], sh.H[pass][lane], c);
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
    int64_t at;        // the workgroup's first channel
    int c, d;          // of its d channels, this lane's first
    int64_t n;         // live steps of the sequence
};

__device__ __forceinline__ Place place(const GatedArgs &a)
{
    Place p;
    p.j = blockIdx.x / a.l.groups;
    p.group = blockIdx.x - p.j * a.l.groups;
    const uint32_t b = p.group / a.per_seq;
    p.b = b;
    p.at = static_cast<int64_t>(p.group - b * a.per_seq) * kGroup;
    p.c = 2 * (threadIdx.x & 63);
    p.d = static_cast<int>(a.D - p.at < kGroup ? a.D - p.at : kGroup);
    p.n = a.T;
    if (a.lengths) {
        const int64_t n = a.lengths[p.b];
        p.n = n < 0 ? 0 : n < a.T ? n : a.T;
    }
    return p;
}

// A wave's steps
struct Steps {
    int64_t t0;
    int all, live;     // of its N: inside T, inside the length
    uint32_t fresh;    // the ones that start a document
};

template <int N> __device__ __forceinline__ Steps steps(const GatedArgs &a, const Place &p, int64_t t0)
{
    static_assert(N <= 32, "a bit for each");
    Steps w;
    w.t0 = t0;
    w.all = static_cast<int>(a.T - t0 < 0 ? 0 : a.T - t0 < N ? a.T - t0 : N);
    w.live = static_cast<int>(p.n - t0 < 0 ? 0 : p.n - t0 < N ? p.n - t0 : N);
    w.fresh = 0;
    if (a.reset) {
        const int lane = threadIdx.x & 63;
        const uint8_t *from = a.reset + p.b * a.T + t0;
        w.fresh = static_cast<uint32_t>(__ballot(lane < w.live && from[lane < w.live ? lane : 0] != 0));
    }
    return w;
}

// Whether all N steps of a tile from t on are live and none starts a document: a
// workgroup takes one of two bodies by this
template <int N> __device__ __forceinline__ bool plain_tile(const GatedArgs &a, const Place &p, int64_t t)
{
    if (t + N > p.n) return false;
    if (!a.reset) return true;
    const uint8_t *from = a.reset + p.b * a.T + t;
    int any = 0;
#pragma unroll
    for (int i = 0; i < N; i += 64) any |= from[(i + (threadIdx.x & 63)) % N];
    return __ballot(any != 0) == 0;
}

// The wave's N rows of a (B,T,...) tensor; past the last live one, that one again
// (there is one)
template <typename T, int N, bool PLAIN, typename L>
__device__ __forceinline__ void rows(const void *base, const int64_t *stride, const Place &p, const Steps &w, const L &lane,
                                     typename Two<T>::V *out)
{
    const int64_t step = stride[1] * static_cast<int64_t>(sizeof(T));
    const char *row = static_cast<const char *>(base) + (p.b * stride[0] + p.at) * static_cast<int64_t>(sizeof(T)) + w.t0 * step;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        out[s] = lane.load(row);
        row += PLAIN || s + 1 < w.live ? step : 0;
    }
}

// The wave's rows of a dense output: f(step) of the live ones, zeros of the others
template <typename T, int N, bool PLAIN, typename L, typename F>
__device__ __forceinline__ void put_rows(void *base, const GatedArgs &a, const Place &p, const Steps &w, const L &lane, F f)
{
    const int64_t step = a.D * static_cast<int64_t>(sizeof(T));
    char *row = static_cast<char *>(base) + (p.b * a.T + w.t0) * step + p.at * static_cast<int64_t>(sizeof(T));
    if (!lane.in) return;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if constexpr (PLAIN)
            lane.store(row, f(s));
        else if (s < w.all)
            lane.store(row, s < w.live ? f(s) : f32x2{0.0f, 0.0f});
        row += step;
    }
}

// The channels' slope2 into LDS (a logarithm and two exponentials each: once per
// workgroup, not once per wave)
template <int W> __device__ __forceinline__ void fill_slopes(const GatedArgs &a, const Place &p, Shared<W> &sh)
{
    for (int i = threadIdx.x; i < kGroup; i += 64 * W) {
        const int64_t c = p.at + i;
        sh.k[i] = slope2(a.lam[c < a.D ? c : a.D - 1], a.rate);
    }
}

// A tile that lies past its sequence's length: hands on what enters it, `from` (or
// zeros) at the first one, and returns it
template <bool MULTI, int W>
__device__ __forceinline__ f32x2 pass_on(const GatedArgs &a, const Place &p, Shared<W> &sh, int pass, const float *from)
{
    const int lane = threadIdx.x & 63;
    Launch ep{0, 0};
    if constexpr (MULTI) ep = epoch_begin(a.l.hd);
    f32x2 first = {0.0f, 0.0f};
    if (from) first = load_f2(from + p.b * a.D + p.at, p.c, p.d);
    sh.A[pass][lane] = f32x2{1.0f, 1.0f};
    sh.H[pass][lane] = f32x2{0.0f, 0.0f};
    if (MULTI && threadIdx.x == 0) epoch_end(a.l.hd, ep, a.l.tiles * a.l.groups, sh.ticket);
    __syncthreads();
    return enter<MULTI>(a.l, sh, p.j, p.group, pass, first);
}

// The pair of a wave's steps.  Steps past the length become the identity, the decays of
// those that start a document -0.
template <int N, bool PLAIN> __device__ __forceinline__ void fold(const Steps &w, f32x2 *ga, f32x2 *gb, f32x2 &A, f32x2 &H)
{
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if constexpr (PLAIN) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                H[v] = __builtin_fmaf(ga[s][v], H[v], gb[s][v]);
                A[v] *= ga[s][v];
            }
            continue;
        }
        const bool live = s < w.live, fresh = (w.fresh >> s) & 1;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            ga[s][v] = live ? (fresh ? -0.0f : ga[s][v]) : 1.0f;
            gb[s][v] = live ? gb[s][v] : 0.0f;
        }
        append(A, H, ga[s], gb[s]);
    }
}

template <typename T, typename S, bool PAIRS, bool MULTI, bool PLAIN>
__device__ __forceinline__ void fwd_tile(const GatedArgs &a, const Place &p, Shared<S::W> &sh)
{
    constexpr int C = S::C, W = S::W;
    const int lane = threadIdx.x & 63, wv = wave();
    const Lane<T, PAIRS> two(p.c, p.d);
    const Steps w = steps<C>(a, p, static_cast<int64_t>(p.j) * S::tile + wv * C);
    f32x2 h, ga[C], gb[C];
    if (!PLAIN && static_cast<int64_t>(p.j) * S::tile >= p.n) {   // no step of the tile is live
        h = pass_on<MULTI>(a, p, sh, wv, a.h0);
#pragma unroll
        for (int s = 0; s < C; ++s) {
            ga[s] = f32x2{1.0f, 1.0f};
            gb[s] = f32x2{0.0f, 0.0f};
        }
    } else {
        typename Two<T>::V rx[C], rr[C], ri[C];
        if (PLAIN || w.live > 0) {
            rows<T, C, PLAIN>(a.x, a.xs, p, w, two, rx);
            rows<T, C, PLAIN>(a.r, a.rs, p, w, two, rr);
            rows<T, C, PLAIN>(a.i, a.is, p, w, two, ri);
        }
        Launch ep{0, 0};
        if constexpr (MULTI) ep = epoch_begin(a.l.hd);
        f32x2 first = {0.0f, 0.0f};
        if (a.h0) first = load_f2(a.h0 + p.b * a.D + p.at, p.c, p.d);
        fill_slopes(a, p, sh);
        __syncthreads();
        const f32x2 k = {sh.k[2 * lane], sh.k[2 * lane + 1]};
        f32x2 A = {1.0f, 1.0f}, H = {0.0f, 0.0f};
        if (!PLAIN && w.live == 0) {   // (a short sequence: most of the tile's waves)
#pragma unroll
            for (int s = 0; s < C; ++s) {
                ga[s] = f32x2{1.0f, 1.0f};
                gb[s] = f32x2{0.0f, 0.0f};
            }
        } else {
#pragma unroll
            for (int s = 0; s < C; ++s) {
                const f32x2 x = wide(rx[s]), r = wide(rr[s]), i = wide(ri[s]);
                const float start = !PLAIN && (w.fresh >> s) & 1 ? -__builtin_inff() : 0.0f;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const Gate g = gate<T>(x[v], r[v], i[v], k[v], start);
                    ga[s][v] = g.a;
                    gb[s][v] = g.b;
                }
                settle(ga[s]);
                settle(gb[s]);
            }
            fold<C, PLAIN>(w, ga, gb, A, H);
        }
        sh.A[wv][lane] = A;
        sh.H[wv][lane] = H;
        if (MULTI && threadIdx.x == 0) epoch_end(a.l.hd, ep, a.l.tiles * a.l.groups, sh.ticket);
        __syncthreads();
        h = enter<MULTI>(a.l, sh, p.j, p.group, wv, first);
    }
    if (a.states && w.t0 % MGS_GATED_CHUNK == 0 && (PLAIN || w.t0 < a.T))
        store_f2(a.states + (p.b * a.chunks + w.t0 / MGS_GATED_CHUNK) * a.D + p.at, p.c, p.d, h);
    put_rows<T, C, PLAIN>(a.y, a, p, w, two, [&](int s) {
        if constexpr (PLAIN) {
#pragma unroll
            for (int v = 0; v < 2; ++v) h[v] = __builtin_fmaf(ga[s][v], h[v], gb[s][v]);
        } else {
            h = apply2(ga[s], gb[s], h);
        }
        return h;
    });
    // (steps past the length leave it as it is)
    if (a.hT && p.j + 1 == a.l.tiles && wv == W - 1) store_f2(a.hT + p.b * a.D + p.at, p.c, p.d, h);
}

template <typename T, typename S, bool PAIRS, bool MULTI>
__global__ void __launch_bounds__(64 * S::W, S::occupancy) gated_fwd_kernel(GatedArgs a)
{
    __shared__ Shared<S::W> sh;
    const Place p = place(a);
    static_assert(S::several || !MULTI, "enough waves to wait for other tiles");
    if (plain_tile<S::tile>(a, p, static_cast<int64_t>(p.j) * S::tile))
        fwd_tile<T, S, PAIRS, MULTI, true>(a, p, sh);
    else
        fwd_tile<T, S, PAIRS, MULTI, false>(a, p, sh);
}

// One step of the backward from its inputs
struct Slopes {
    float a, b;
    float x, i;    // d b / d x, d b / d i
    float l;       // -d b / d log a: iota x a^2 / beta
};

template <typename T> __device__ __forceinline__ Slopes slopes(float x, float r, float i, float k, float start)
{
    const float rho = rcp(1.0f + exp_neg<T>(r)), ei = exp_neg<T>(i), iota = rcp(1.0f + ei);
    Slopes o;
    float beta2;
    decay(__builtin_fmaf(k, rho, start), o.a, beta2);
    // 1 / beta; 1 - a^2 below the smallest normal number counts as 0
    const float inv = beta2 < 0x1p-126f ? 0.0f : __builtin_amdgcn_rsqf(beta2), ix = iota * x;
    o.x = beta2 * inv * iota;
    o.b = o.x * x;
    o.i = o.b * shut(ei, iota);
    o.l = ix * (o.a * o.a) * inv;
    return o;
}

// A tile's sums of dl rho, for dlam
__device__ __forceinline__ void put_part(const GatedArgs &a, const Place &p, int64_t tile, uint32_t tag, f32x2 sum)
{
    uint64_t *o = a.part + (p.b * a.l.tiles + tile) * a.D + p.at;
#pragma unroll
    for (int v = 0; v < 2; ++v)
        if (p.c + v < p.d) o[p.c + v] = (static_cast<uint64_t>(tag) << 32) | __float_as_uint(sum[v]);
}

template <int W> struct BwdShared {
    Shared<W> s;
    f32x2 F[2][W][64];   // the waves' pairs of the forward; then (second) the state ahead of each
    f32x2 sum[W][64];
};

template <typename T, typename S, bool PAIRS, bool MULTI, bool PLAIN>
__device__ __forceinline__ void bwd_tile(const GatedArgs &a, const Place &p, int64_t tile, BwdShared<S::W> &sh)
{
    constexpr int C = S::C, W = S::W;
    const int lane = threadIdx.x & 63;
    const int pass = wave(), wv = W - 1 - pass;   // in the order of the pass, and of the steps
    const Lane<T, PAIRS> two(p.c, p.d);
    const Steps w = steps<C>(a, p, tile * S::tile + wv * C);
    if (!PLAIN && tile * S::tile >= p.n) {   // no step of the tile is live
        const f32x2 K = pass_on<MULTI>(a, p, sh.s, pass, a.dhT);
        for (void *o : {a.dx, a.dr, a.di})
            put_rows<T, C, false>(o, a, p, w, two, [](int) { return f32x2{0.0f, 0.0f}; });
        if (a.dh0 && tile == 0 && wv == 0) store_f2(a.dh0 + p.b * a.D + p.at, p.c, p.d, K);
        if (wv == 0) put_part(a, p, tile, MULTI ? sh.s.ticket[0] : 0, f32x2{0.0f, 0.0f});
        return;
    }
    typename Two<T>::V rx[C], rr[C], ri[C], rg[C];
    if (PLAIN || w.live > 0) {
        rows<T, C, PLAIN>(a.x, a.xs, p, w, two, rx);
        rows<T, C, PLAIN>(a.r, a.rs, p, w, two, rr);
        rows<T, C, PLAIN>(a.i, a.is, p, w, two, ri);
        rows<T, C, PLAIN>(a.dy, a.gs, p, w, two, rg);
    }
    Launch ep{0, 0};
    if constexpr (MULTI) ep = epoch_begin(a.l.hd);
    f32x2 first = {0.0f, 0.0f}, state = {0.0f, 0.0f};
    if (a.dhT) first = load_f2(a.dhT + p.b * a.D + p.at, p.c, p.d);
    if (pass == 1)
        state = load_f2(a.states + (p.b * a.chunks + tile * S::tile / MGS_GATED_CHUNK) * a.D + p.at, p.c, p.d);
    fill_slopes(a, p, sh.s);
    __syncthreads();
    const f32x2 k = {sh.s.k[2 * lane], sh.s.k[2 * lane + 1]};

    // Per step: the decay, and what G multiplies: m1 -> dx, m2 -> di, m3 -> dl (first
    // what is subtracted there).  b = m1 x
    f32x2 ga[C], m1[C], m2[C], m3[C], A = {1.0f, 1.0f}, H = {0.0f, 0.0f}, K = {0.0f, 0.0f};
    if (!PLAIN && w.live == 0) {   // (a short sequence: most of the tile's waves)
#pragma unroll
        for (int s = 0; s < C; ++s) {
            ga[s] = f32x2{1.0f, 1.0f};
            m1[s] = m2[s] = m3[s] = f32x2{0.0f, 0.0f};
        }
    } else {
#pragma unroll
        for (int s = 0; s < C; ++s) {
            const f32x2 x = wide(rx[s]), r = wide(rr[s]), i = wide(ri[s]);
            const bool live = PLAIN || s < w.live, fresh = !PLAIN && (w.fresh >> s) & 1;
            const float start = fresh ? -__builtin_inff() : 0.0f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const Slopes o = slopes<T>(x[v], r[v], i[v], k[v], start);
                ga[s][v] = !live ? 1.0f : fresh ? -0.0f : o.a;
                m1[s][v] = o.x;
                m2[s][v] = o.i;
                m3[s][v] = o.l;
                const float b = live ? o.b : 0.0f;
                H[v] = PLAIN ? __builtin_fmaf(ga[s][v], H[v], b) : apply(ga[s][v], b, H[v]);
                A[v] = PLAIN ? A[v] * ga[s][v] : chain(A[v], ga[s][v]);
            }
            settle(ga[s]);
            settle(m1[s]);
            settle(m2[s]);
            settle(m3[s]);
        }
    }
    // G times the decay, or nothing where that clears
    auto back = [&](float decay, float G) { return !PLAIN && clears(decay) ? 0.0f : decay * G; };
#pragma unroll
    for (int s = C - 1; s >= 0; --s) {
        const f32x2 g = again(rg[s]);
#pragma unroll
        for (int v = 0; v < 2; ++v) K[v] = back(ga[s][v], (PLAIN || s < w.live ? g[v] : 0.0f) + K[v]);
    }
    sh.F[0][wv][lane] = A;
    sh.F[1][wv][lane] = H;
    sh.s.A[pass][lane] = A;
    sh.s.H[pass][lane] = K;
    if (MULTI && threadIdx.x == 0) epoch_end(a.l.hd, ep, a.l.tiles * a.l.groups, sh.s.ticket);
    __syncthreads();
    if (pass == 1) {
#pragma unroll
        for (int q = 0; q < W; ++q) {
            const f32x2 fA = sh.F[0][q][lane], fH = sh.F[1][q][lane];
            sh.F[1][q][lane] = state;
            state = apply2(fA, fH, state);
        }
    }
    K = enter<MULTI>(a.l, sh.s, p.j, p.group, pass, first);
    f32x2 h = sh.F[1][wv][lane], sum = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < C; ++s) {
        const f32x2 x = again(rx[s]);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float b = PLAIN || s < w.live ? m1[s][v] * x[v] : 0.0f;
            if constexpr (PLAIN) {
                m3[s][v] = __builtin_fmaf(ga[s][v], h[v], -m3[s][v]);
                h[v] = __builtin_fmaf(ga[s][v], h[v], b);
            } else {
                const float ah = back(ga[s][v], h[v]);
                m3[s][v] = ah - m3[s][v];
                h[v] = ah + b;
            }
        }
    }
    const f32x2 kn = k * 0.6931471805599453f;   // log a = kn rho
#pragma unroll
    for (int s = C - 1; s >= 0; --s) {
        const f32x2 g = again(rg[s]), r = again(rr[s]);
        const bool live = PLAIN || s < w.live;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const bool clear = !PLAIN && clears(ga[s][v]);
            const float er = exp_neg<T>(r[v]), rho = rcp(1.0f + er);
            const float G = (live ? g[v] : 0.0f) + K[v], dl = clear ? 0.0f : G * m3[s][v] * rho;   // (dl rho)
            m1[s][v] *= G;
            m2[s][v] *= G;
            m3[s][v] = clear ? 0.0f : dl * kn[v] * shut(er, rho);
            sum[v] += live ? dl : 0.0f;
            K[v] = back(ga[s][v], G);
        }
    }
    put_rows<T, C, PLAIN>(a.dx, a, p, w, two, [&](int s) { return m1[s]; });
    put_rows<T, C, PLAIN>(a.dr, a, p, w, two, [&](int s) { return m3[s]; });
    put_rows<T, C, PLAIN>(a.di, a, p, w, two, [&](int s) { return m2[s]; });
    if (a.dh0 && tile == 0 && wv == 0) store_f2(a.dh0 + p.b * a.D + p.at, p.c, p.d, K);
    sh.sum[wv][lane] = sum;
    __syncthreads();
    if (wv == 0) {
        for (int q = 1; q < W; ++q) sum += sh.sum[q][lane];
        put_part(a, p, tile, MULTI ? sh.s.ticket[0] : 0, sum);   // (0: never the tag of a later launch)
    }
}

template <typename T, typename S, bool PAIRS, bool MULTI>
__global__ void __launch_bounds__(64 * S::W, S::occupancy) gated_bwd_kernel(GatedArgs a)
{
    __shared__ BwdShared<S::W> sh;
    const Place p = place(a);
    const int64_t tile = static_cast<int64_t>(a.l.tiles) - 1 - p.j;
    static_assert(S::several || !MULTI, "enough waves to wait for other tiles");
    if (plain_tile<S::tile>(a, p, tile * S::tile))
        bwd_tile<T, S, PAIRS, MULTI, true>(a, p, tile, sh);
    else
        bwd_tile<T, S, PAIRS, MULTI, false>(a, p, tile, sh);
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
    const int64_t end = (wv + 1) * share < rows ? (wv + 1) * share : rows;
    constexpr int U = 16;   // loads in flight
    for (int64_t i = wv * share; i < end; i += U) {
        float v[U];
#pragma unroll
        for (int e = 0; e < U; ++e) v[e] = tag_value(part[(i + e < end ? i + e : end - 1) * D + cc]);
#pragma unroll
        for (int e = 0; e < U; ++e) sum += i + e < end ? static_cast<double>(v[e]) : 0.0;
    }
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
    const int64_t from = (at - b * a.blocks_per_row) * 512;   // this workgroup's first channel
    const int c = 2 * threadIdx.x, d = static_cast<int>(a.D - from < 512 ? a.D - from : 512);
    if (c >= d) return;
    const Lane<T, PAIRS> two(c, d);
    const int64_t slot = a.slots ? a.slots[b] : b;
    char *y = static_cast<char *>(a.y) + (b * a.D + from) * static_cast<int64_t>(sizeof(T));
    if (slot < 0 || slot >= a.n_slots) {
        two.store(y, f32x2{0.0f, 0.0f});
        return;
    }
    auto row = [&](const void *p, int64_t stride) {
        return wide(two.load(static_cast<const char *>(p) + (b * stride + from) * static_cast<int64_t>(sizeof(T))));
    };
    const f32x2 x = row(a.x, a.xs), r = row(a.r, a.rs), i = row(a.i, a.is);
    const f32x2 lam = load_f2(a.lam + from, c, d);
    float *state = a.h + slot * a.D + from;
    f32x2 h = load_f2(state, c, d);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const Gate g = gate<T>(x[v], r[v], i[v], slope2(lam[v], a.rate), 0.0f);
        h[v] = __builtin_fmaf(g.a, h[v], g.b);
    }
    store_f2(state, c, d, h);
    two.store(y, h);
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
    a.l.unit = static_cast<uint32_t>(g.unit);
    a.l.per = static_cast<uint32_t>((g.unit - 1 + kPollers - 1) / kPollers + (g.unit == 1));
    a.l.tiles = static_cast<uint32_t>(tiles);
    const int xcds = xcd_count();
    a.l.local = xcds > 0 && g.groups % xcds == 0;
    return a;
}

template <typename T, typename S, bool MULTI> hipError_t run_fwd_as(const GatedArgs &a, bool two, hipStream_t s)
{
    const dim3 grid(a.l.groups * a.l.tiles), block(64 * S::W);
    if (two) gated_fwd_kernel<T, S, true, MULTI><<<grid, block, 0, s>>>(a);
    else gated_fwd_kernel<T, S, false, MULTI><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T> hipError_t run_fwd(const GatedArgs &a, bool two, hipStream_t s)
{
    if (a.T <= kShort) return run_fwd_as<T, FwdShort, false>(a, two, s);
    return a.l.tiles > 1 ? run_fwd_as<T, Fwd<T>, true>(a, two, s) : run_fwd_as<T, Fwd<T>, false>(a, two, s);
}

template <typename T, typename S, bool MULTI> hipError_t run_bwd_as(const GatedArgs &a, bool two, hipStream_t s)
{
    const dim3 grid(a.l.groups * a.l.tiles), block(64 * S::W);
    if (two) gated_bwd_kernel<T, S, true, MULTI><<<grid, block, 0, s>>>(a);
    else gated_bwd_kernel<T, S, false, MULTI><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T> hipError_t run_bwd(const GatedArgs &a, bool two, hipStream_t s)
{
    if (a.T <= kShort) return run_bwd_as<T, BwdShort, false>(a, two, s);
    return a.l.tiles > 1 ? run_bwd_as<T, Bwd<T>, true>(a, two, s) : run_bwd_as<T, Bwd<T>, false>(a, two, s);
}

}  // namespace

GatedGeom gated_geometry(const mgs_gated_desc &d, bool backward)
{
    GatedGeom g{};
    g.groups = d.B * ((d.D + kGroup - 1) / kGroup);
    // (no steps: one tile, which hands the state on)
    const bool half = d.dtype == MGS_BF16;
    const int64_t tf = half ? Fwd<__bf16>::tile : Fwd<float>::tile, tb = half ? Bwd<__bf16>::tile : Bwd<float>::tile;
    g.tiles_f = std::max<int64_t>(1, (d.T + tf - 1) / tf);
    g.tiles_b = std::max<int64_t>(1, (d.T + tb - 1) / tb);
    // A unit is one hop of 1.2 us along a sequence: enough tiles that the hops do not take
    // longer than the data, and no more, for a tile reads half a unit's pairs.  Measured on
    // 4096 forward tiles in all, us forward / backward, bf16, with units of 1, 2, 4, 8, 22, 36,
    // 64 tiles (not on few tiles, where the hops are most of the time: 2048 steps of 20 groups
    // are five of them, 18 / 31 with 8.4 / 15 of bytes):
    //   128 groups (4 x 4096 steps)  112/220 114/232 117/233 118/237 129/256 139/266 145/300
    //   16 (2 x 32768)               144/327 113/251 116/252 120/256 130/275 135/297 147/329
    //   8 (65536)                    240/514 160/358 113/270 116/260 127/286 135/309 149/346
    //   2 (262144)                   1440/3063 801/1725 497/1092 322/732 161/425 157/416 171/442
    //   1 (1048576)                  5686/12184 3107/6731 1774/3962 1201/2808 490/1394 328/1084 291/1031
    g.unit = static_cast<int>(std::max<int64_t>(1, 64 / std::max<int64_t>(1, g.groups)));
    const int64_t tiles = backward ? std::max(g.tiles_f, g.tiles_b) : g.tiles_f;
    // every word behind the header is a tagged one, whatever call it is written by,
    // so that a call of other sizes takes none of them for its own
    size_t off = sizeof(WsHeader);
    g.off_agg = off;
    if (tiles > 1 && g.unit > 1) off = align256(off + static_cast<size_t>(tiles) * g.groups * 2 * kGroup * 8);
    g.off_incl = off;
    // (32 groups need 2 1/2 words a tile and channel, their units being of two tiles; more
    // groups with units of one have room for a call of those too)
    const int64_t lines = g.unit > 1 ? tiles / g.unit * g.groups : tiles * std::max<int64_t>(g.groups, 80);
    if (tiles > 1) off = align256(off + static_cast<size_t>(lines) * kGroup * 8);
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
