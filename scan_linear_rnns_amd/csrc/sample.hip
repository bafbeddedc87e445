// sample.hip -- sampling of the next token with temperature, top-k, top-p and
// min-p (gfx950).
//
// The filters keep a prefix of the order by (logit descending, index ascending), so
// what is kept is an edge: everything above its value, and its equals up to an index.
// A row goes through
//   1. its largest logit;
//   2. a histogram over (largest - x) / temperature, in steps of 1/64 to e^-16, wider ones
//      to where no weight is left: of the counts for top-k, of the weights, as multiples of
//      2^-43, for top-p (integers: their sums do not depend on the order of the atomics);
//   3. the few that lie in the bin where the filter ends (for top-k, all up to there),
//      gathered and sorted, and the sums of the weights ahead of that bin, a sum for
//      each wave's share of the row;
//   4. the edge, from the sorted ones; the share in which the running sum passes u
//      times the total; the token in that share.
// A row without top-k and top-p needs 1, the sums of 3, and 4; without min-p too, 1 and 3
// are one pass.  Where a bin holds too many to sort (equal logits by the thousand), its
// values are split again, one histogram after another, by the row's workgroup alone.
// Large batches take a workgroup a row for all of it; for small ones a long row is cut into
// slices, each step a launch.  Rows of bf16 logits that need 2 are counted by value instead
// (below).
//
// What bounds it: for few rows the chain of barriers and launches (1 row of 32000, bf16,
// all filters 21 us, of them 3 for the launch; 37 of 50001, fp32, no filter 8.7 + 9.2, with
// 1.5 us of bytes).  256 rows of 128000, bf16, mixed settings, are 65.5 MB, 13 us at a copy's
// rate: 46 counted, 26 until all is counted, 10 for the ends and sums, 11 for the token.
// Without the additions to LDS the first takes as long: a wave reads its share in four rounds
// and waits for each (56 % of the waves' cycles), the VALU is busy half of the time, the
// LDS a fifth.  The same in fp32, 26 us of bytes, goes by weights' fp64 operations: by top-p
// 110 to 115 (26 the largest, 46 histogram, 29 gathering, 6 the edge, 8 the token), without
// filters 52, mixed 133.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "launch.hpp"
#include "layers.hpp"
#include "tokens.hpp"

namespace mgs {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
// half of the bins are of 1/64, half of 43/64: to e^-704, less than 2^-1000
constexpr float kPerUnit = 64.0f, kFar = 43.0f;
constexpr int kList = 4096;         // candidates that are sorted
constexpr int kCounted = 256;       // up to here sorting counts the smaller ones
constexpr int kMaxSlices = 64;
constexpr int kWorkgroups = 256;    // that rows are cut into: one for each CU
constexpr float kInf = __builtin_inff(), kMax = 3.4028234663852886e38f;

struct SampleArgs {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *token;
    float *logp;
    int64_t stride;
    char *ws;
    size_t slot;     // workspace bytes of a row
    int vocab, slices, share, k0;
    float t0, p0, m0;
    bool vec, plain;     // plain: no row has a filter
};

__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Unsigned numbers in the order of the floats (no NaN; -0 counts as 0), never 0
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// The larger of two, NaN if one is
__device__ __forceinline__ float larger(float x, float y)
{
    return x != x || y != y ? __builtin_nanf("") : fmaxf(x, y);
}

// ---------------------------------------------------------- a row's settings
enum { DONE = 0, GREEDY = 1, PLAIN = 2, TOP_K = 3, TOP_P = 4 };

struct Row {
    int kind;
    int top_k;           // 0: off
    float max, top;      // the largest logit; the same, the largest number where it is infinite
    float half;          // of top
    float least;         // no smaller one passes min-p (the floor without it)
    float floor;         // what is below has no weight: -inf, or all but +inf
    float nothing;       // what is below has a weight of less than 2^-1000, or is below the floor
    float inv;           // 1 / temperature
    double scale;        // log2 e / temperature
    double top_p, min_p;
    float u;
};

__device__ __forceinline__ Row settings(const SampleArgs &a, int64_t b, float top)
{
    Row r;
    float tau = a.temperature ? a.temperature[b] : a.t0, p = a.top_p ? a.top_p[b] : a.p0;
    float m = a.min_p ? a.min_p[b] : a.m0;
    const int k = a.top_k ? a.top_k[b] : a.k0;
    const float u = a.u[b];
    r.u = u > 0.0f ? (u < 1.0f ? u : 0.99999994f) : 0.0f;
    r.max = top;
    r.top = fminf(top, kMax);
    r.half = 0.5f * r.top;
    r.floor = top == kInf ? kInf : -kMax;
    r.inv = 1.0f / tau;
    r.scale = 1.4426950408889634 / static_cast<double>(tau);
    // (rounded up: were it down, a value between could have a weight below 2^-1022)
    const double end = static_cast<double>(r.top) - 693.1471805599453 * static_cast<double>(tau);
    const float near = static_cast<float>(end);
    r.nothing = fmaxf(r.floor, static_cast<double>(near) < end ? of_key(key_of(near) + 1) : near);
    r.top_k = k > 0 && k < a.vocab ? k : 0;
    r.top_p = p < 1.0f ? (p > 0.0f ? p : 0.0f) : 1.0;
    r.min_p = m > 0.0f ? (m < 1.0f ? m : 1.0f) : 0.0f;
    r.least = r.floor;
    if (r.min_p > 0.0) {   // a little lower: the weight itself decides
        const double x = r.top + static_cast<double>(tau) * log(r.min_p);
        r.least = fmaxf(r.floor, static_cast<float>(x - 1e-6 * (fabs(x) + fabs(static_cast<double>(r.top)))));
    }
    r.kind = !(top > -kInf) ? DONE : !(tau > 0.0f) ? GREEDY : r.top_k ? TOP_K : r.top_p < 1.0 ? TOP_P : PLAIN;
    return r;
}

// ------------------------------------------------------------------ weights
constexpr int kRoots = 256;

// 2^(j/256), for the function below
__device__ __forceinline__ void fill_roots(double *roots)
{
    if (threadIdx.x < kRoots) roots[threadIdx.x] = exp2(static_cast<double>(threadIdx.x) / kRoots);
}

// e^((x - top) / temperature) in fp64, x not above the largest: y = n + j/256 + s,
// |s| <= 1/512, 2^s by its series to s^4 (the next term is below 2^-54).  What is below
// r.nothing is nothing.  No branches: neighbouring values' chains run side by side (with a
// branch for that, 256 rows of 128000 without filters took 64 us, now 52; the fp64
// operations, eight cycles each, are two thirds of it).
__device__ __forceinline__ double weight(float x, const Row &r, const double *roots)
{
    constexpr double kShift = 1.5 * 17592186044416.0;   // 2^44: adding it rounds to 1/256
    const bool some = x >= r.nothing;
    const float v = some ? fminf(x, kMax) : r.top;
    const double y = (static_cast<double>(v) - static_cast<double>(r.top)) * r.scale;
    const double z = y + kShift, s = y - (z - kShift);
    const int k = __double2loint(z);
    double q = __builtin_fma(9.6181291076284772e-3, s, 5.5504108664821580e-2);
    q = __builtin_fma(q, s, 2.4022650695910071e-1);
    q = __builtin_fma(q, s, 6.9314718055994531e-1);
    const double root = roots[k & (kRoots - 1)], w = __builtin_fma(q * s, root, root);
    const int hi = __double2hiint(w) + ((k >> 8) << 20), lo = __double2loint(w);
    return __hiloint2double(some ? hi : 0, some ? lo : 0);
}

// w <= 1 as a multiple of 2^-43 (rounded: 2^20 of them fit 64 bits, and are off by 2^-24 in
// sum at the very most, a number u's own step)
__device__ __forceinline__ uint64_t fixed(double w)
{
    constexpr double kOne = 768.0;   // 1.5 * 2^(52 - 43)
    return __double_as_longlong(w + kOne) - __double_as_longlong(kOne);
}

// The weight that top-p asks for, of `all`, in these steps: of the order, the ones with less
// ahead of them stay (so the first does)
__device__ __forceinline__ uint64_t needed(const Row &r, uint64_t all)
{
    const double want = ceil(r.top_p * static_cast<double>(all));
    return want > 1.0 ? static_cast<uint64_t>(want) : 1;
}

// The bin of x, kBins past the last one and below the floor; falls with x.  (Of half the
// distance, which is finite: a temperature may be as large.)
__device__ __forceinline__ int bin_of(float x, const Row &r)
{
    constexpr float kBend = kBins / 2 - kBins / 2 / kFar;
    const float d = __builtin_fmaf(-0.5f, fminf(x, kMax), r.half), far = d * r.inv * (2.0f * kPerUnit);
    const float t = fminf(far, __builtin_fmaf(far, 1.0f / kFar, kBend));
    const int bin = t < static_cast<float>(kBins) ? static_cast<int>(t) : kBins;
    return x >= r.floor ? (d == 0.0f ? 0 : bin) : kBins;   // (0 times an infinite inv is no number)
}

// The least x whose bin is `bin` or less (bin < kBins), by the whole wave: 64 keys at a
// time
__device__ __forceinline__ float bin_floor(int bin, const Row &r)
{
    const uint32_t lane = threadIdx.x & 63;
    uint32_t lo = key_of(r.floor), hi = key_of(r.floor == kInf ? kInf : r.top);   // hi's bin is 0
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 64 + 1, at = hi - lo > lane * step ? lo + lane * step : hi;
        const uint64_t in = __ballot(bin_of(of_key(at), r) <= bin);   // the lanes from some one on
        if (in == 0) {
            lo = __builtin_amdgcn_readlane(at, 63) + 1;
            continue;
        }
        const int first = __builtin_ctzll(in);
        hi = __builtin_amdgcn_readlane(at, first);
        lo = first == 0 ? hi : __builtin_amdgcn_readlane(at, first - 1) + 1;
    }
    return of_key(hi);
}

// ------------------------------------------------------------ walking a row
template <typename T> struct Wide;
template <> struct Wide<float> {
    typedef float V __attribute__((ext_vector_type(4)));
    static constexpr int N = 4;
};
template <> struct Wide<__bf16> {
    typedef __bf16 V __attribute__((ext_vector_type(8)));
    static constexpr int N = 8;
};

// What a wave reads at once from place `base` of a row on, before hi: four times N
// neighbours a lane; -inf stands for places from hi on
constexpr int kLoads = 4;

template <typename T>
__device__ __forceinline__ void load_some(const T *x, int base, int hi, bool vec, float (&v)[kLoads][Wide<T>::N])
{
    constexpr int N = Wide<T>::N;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int i = base + (j * 64 + lane) * N;
        if (vec && i + N <= hi) {
            const typename Wide<T>::V w = *reinterpret_cast<const typename Wide<T>::V *>(x + i);
#pragma unroll
            for (int e = 0; e < N; ++e) v[j][e] = static_cast<float>(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) v[j][e] = i + e < hi ? static_cast<float>(x[i + e]) : -kInf;
        }
    }
}

// f(values, index of the first) for the places lo..hi-1, hi <= V, of a row, four
// neighbours a lane at a time; lo is a multiple of what a wave reads at once.  -inf stands
// for places past hi.  The wave stays whole.
template <typename T, typename F> __device__ __forceinline__ void walk4(const T *x, int lo, int hi, bool vec, F f)
{
    constexpr int N = Wide<T>::N;
    const int lane = threadIdx.x & 63;
    for (int base = lo; base < hi; base += 64 * N * kLoads) {
        float v[kLoads][N];
        load_some(x, base, hi, vec, v);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (base + j * 64 * N >= hi) break;
#pragma unroll
            for (int e = 0; e < N; e += 4) f(&v[j][e], base + (j * 64 + lane) * N + e);
        }
    }
}

// The same one by one: f(value, index)
template <typename T, typename F> __device__ __forceinline__ void walk(const T *x, int lo, int hi, bool vec, F f)
{
    walk4(x, lo, hi, vec, [&](const float *v, int i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f(v[e], i + e);
    });
}

// What a wave's lanes have written to LDS is there for its others (its LDS accesses run
// in order: this holds the compiler to that)
__device__ __forceinline__ void wave_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Values of a wave's lanes that wait until there are 64 of them, so that what is done
// with few of a row's values is done with whole waves.  Four a lane are taken in at once.
constexpr int kQueue = 63 + 4 * 64;

struct Queue {
    float *held;   // kQueue of the wave's own, in LDS
    int n = 0;

    template <typename P, typename F> __device__ __forceinline__ void push4(const float *v, P in, F f)
    {
        uint64_t who[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) who[e] = __ballot(in(v[e]));
        if ((who[0] | who[1] | who[2] | who[3]) == 0) return;
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(who[e] >> 32),
                                                         __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(who[e]), 0));
            if (in(v[e])) held[n + before] = v[e];
            n += __popcll(who[e]);
        }
        wave_order();
        for (; n >= 64;) {
            n -= 64;
            f(held[n + lane]);
        }
        wave_order();
    }
    template <typename F> __device__ __forceinline__ void rest(F f)
    {
        wave_order();
        const int lane = threadIdx.x & 63;
        if (lane < n) f(held[lane]);
    }
};

// ------------------------------------------------------------ workgroup sums
template <typename V> __device__ __forceinline__ V wave_sum(V v)
{
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// The sum over the threads before this one, and over all of them
template <typename V> __device__ __forceinline__ V scan_block(V v, V *lds, V &all)
{
    const int lane = threadIdx.x & 63, wv = wave();
    V up = v;
    for (int off = 1; off < 64; off <<= 1) {
        const V o = __shfl_up(up, off, 64);
        if (lane >= off) up += o;
    }
    __syncthreads();
    if (lane == 63) lds[wv] = up;
    __syncthreads();
    V before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wv) before += lds[w];
        all += lds[w];
    }
    const V prev = __shfl_up(up, 1, 64);
    return lane ? before + prev : before;
}

// Sorts n entries, all different but for ~0, n a power of two from 64 on.  Few: each
// entry's place is the number of smaller ones, counted by kThreads / n threads (two
// barriers, where sorting in steps takes some thirty; the reads grow with n^2: at 512
// a row's last step took 61 us, in steps 36); many: in steps.
__device__ __forceinline__ void sort_list(uint64_t *list, int n)
{
    __syncthreads();
    if (n <= kCounted) {
        const int each = kThreads / n, e = threadIdx.x / each, part = threadIdx.x % each;
        const uint64_t own = list[e];
        const int per = n / each;
        int smaller = 0;
#pragma unroll 8
        for (int i = 0; i < per; ++i) {
            const int at = part * per + i;
            const uint64_t o = list[at];
            smaller += o < own || (o == own && at < e);
        }
        for (int off = 1; off < each; off <<= 1) smaller += __shfl_xor(smaller, off, 64);
        __syncthreads();
        if (part == 0) list[smaller] = own;
        __syncthreads();
        return;
    }
    for (int size = 2; size <= n; size *= 2)
        for (int step = size / 2; step; step /= 2) {
            for (int p = threadIdx.x; p < n / 2; p += kThreads) {
                const int i = (p / step) * 2 * step + p % step, j = i + step;
                const uint64_t x = list[i], y = list[j];
                if ((x > y) == ((i & size) == 0)) {
                    list[i] = y;
                    list[j] = x;
                }
            }
            __syncthreads();
        }
}

// ------------------------------------------------------------- steps 1 to 3
struct Shared {
    uint64_t mass[kBins];
    uint32_t count[kBins];
    uint64_t list[kList];
    double sub[kMaxSlices * kWaves];
    double roots[kRoots];
    double wd[kWaves];
    uint64_t wu[kWaves];
    float top[kWaves];
    uint32_t n;
    int bin, at, last;
    uint64_t ahead;
    double w_at;
};

// Workspace of a row that is cut into slices
struct Slot {
    float *top;        // of each slice; NaN where the slice has one
    uint32_t *n;       // candidates
    uint32_t *count;
    uint64_t *mass, *list;
    float *maxima;     // kGroups of each slice
    double *sub;
};

constexpr int kGroups = 64;   // of 16 threads
constexpr size_t kSlotMass = 512, kSlotCount = kSlotMass + 8 * kBins, kSlotList = kSlotCount + 4 * kBins,
                 kSlotMaxima = kSlotList + 8 * kList, kSlotSub = kSlotMaxima + 4 * kGroups * kMaxSlices;

__device__ __forceinline__ Slot slot_of(const SampleArgs &a, int64_t b)
{
    char *w = a.ws + kHeader + b * a.slot;
    return Slot{reinterpret_cast<float *>(w), reinterpret_cast<uint32_t *>(w + 256),
                reinterpret_cast<uint32_t *>(w + kSlotCount), reinterpret_cast<uint64_t *>(w + kSlotMass),
                reinterpret_cast<uint64_t *>(w + kSlotList), reinterpret_cast<float *>(w + kSlotMaxima),
                reinterpret_cast<double *>(w + kSlotSub)};
}

// 1: the largest of a slice, NaN if it holds one, known to every thread; `own`: of the
// values that this thread has read
template <typename T>
__device__ __forceinline__ float slice_top(const SampleArgs &a, const T *x, int lo, int hi, Shared &sh, float &own)
{
    float top = -kInf;
    bool nan = false;
    walk(x, lo, hi, a.vec, [&](float v, int) {
        top = fmaxf(top, v);
        nan |= v != v;
    });
    own = top;
    if (nan) top = __builtin_nanf("");
    for (int off = 32; off; off >>= 1) {
        const float o = __shfl_xor(top, off, 64);
        top = larger(top, o);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.top[wave()] = top;
    __syncthreads();
    top = sh.top[0];
    for (int w = 1; w < kWaves; ++w) top = larger(top, sh.top[w]);
    return top;
}

// 2: the histogram of a wave's share into LDS
template <typename T>
__device__ __forceinline__ void histogram(const SampleArgs &a, const Row &r, const T *x, int lo, int hi, Shared &sh)
{
    if (r.kind == TOP_K)
        walk(x, lo, hi, a.vec, [&](float v, int) {
            const int bin = bin_of(v, r);
            if (bin < kBins) atomicAdd(&sh.count[bin], 1u);
        });
    else
        walk4(x, lo, hi, a.vec, [&](const float *v, int) {
            // all four chains side by side, ahead of the branches
            int bin[4];
            uint64_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bin[e] = bin_of(v[e], r);
                w[e] = fixed(weight(v[e], r, sh.roots));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (bin[e] < kBins) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[bin[e]]), w[e]);
        });
}

// Whole workgroup: the bin in which the filter ends, from the row's histogram: the first
// at whose end there are top_k, or top_p of the weight.  -> sh.bin, what is ahead of
// it -> sh.ahead.  kBins where all are kept.  How many, or how much, are wanted.
__device__ __forceinline__ uint64_t end_bin(const Row &r, const uint32_t *count, const uint64_t *mass, Shared &sh)
{
    const int b = 2 * threadIdx.x;
    uint64_t v0, v1, all;
    if (r.kind == TOP_K) {
        v0 = count[b];
        v1 = count[b + 1];
    } else {
        v0 = mass[b];
        v1 = mass[b + 1];
    }
    if (threadIdx.x == 0) sh.bin = kBins;
    const uint64_t before = scan_block(v0 + v1, sh.wu, all);
    const uint64_t want = r.kind == TOP_K ? static_cast<uint64_t>(r.top_k) : needed(r, all);
    const bool e0 = before < want && before + v0 >= want;
    const bool e1 = before + v0 < want && before + v0 + v1 >= want;
    if (e0 || e1) {
        sh.bin = e0 ? b : b + 1;
        sh.ahead = e0 ? before : before + v0;
    }
    __syncthreads();
    return want;
}

// 3: candidates into the list (`n` and `list` in LDS or the workspace), and the sum of
// the weights ahead of them in this wave's share (top-p; of all of it without filters).
// More than kList candidates are counted but not kept.
template <typename T>
__device__ __forceinline__ double gather(const SampleArgs &a, const Row &r, const T *x, int lo, int hi, int end, Shared &sh,
                                         uint32_t *n, uint64_t *list)
{
    double sum = 0.0;
    const int lane = threadIdx.x & 63;
    auto add = [&](float v) {
        const double w = weight(v, r, sh.roots);
        sum += w >= r.min_p ? w : 0.0;
    };
    // (the histogram has been read)
    static_assert(sizeof(sh.mass) + sizeof(sh.count) >= sizeof(float) * kQueue * kWaves, "room for the queues");
    Queue queue{reinterpret_cast<float *>(sh.mass) + wave() * kQueue};
    if (r.kind == PLAIN) {
        if (r.min_p > 0.0)   // few pass it, as a rule: their weights are taken 64 at a time
            walk4(x, lo, hi, a.vec, [&](const float *v, int) {
                queue.push4(v, [&](float y) { return y >= r.least; }, add);
            });
        else
            walk(x, lo, hi, a.vec, [&](float v, int) {
                const double w = weight(v, r, sh.roots);
                sum += v >= r.floor ? w : 0.0;
            });
        queue.rest(add);
        return wave_sum(sum);
    }
    const bool share = r.kind == TOP_P && end > 0;
    const float from = bin_floor(end < kBins ? end : kBins - 1, r);
    const float past = share ? bin_floor(end - 1, r) : 0.0f, least = fmaxf(past, r.least);
    auto candidate = [&](float y) { return y >= from && !(share && y >= past); };
    walk4(x, lo, hi, a.vec, [&](const float *v, int i) {
        if (share) queue.push4(v, [&](float y) { return y >= least; }, add);
        if (__ballot(candidate(v[0]) || candidate(v[1]) || candidate(v[2]) || candidate(v[3])) == 0) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t who = __ballot(candidate(v[e]));
            if (!who) continue;
            uint32_t at = 0;
            if (lane == __builtin_ctzll(who)) at = atomicAdd(n, static_cast<uint32_t>(__popcll(who)));
            at = __builtin_amdgcn_readlane(at, __builtin_ctzll(who)) + __popcll(who & ((1ull << lane) - 1));
            if (candidate(v[e]) && at < kList)
                list[at] = (static_cast<uint64_t>(~key_of(v[e])) << 32) | static_cast<uint32_t>(i + e);
        }
    });
    queue.rest(add);
    return wave_sum(sum);
}

// -------------------------------------------------------------------- step 4
struct Edge {
    uint32_t key;   // kept: keys above this one, and its equals
    int limit;      // up to this index
};

__device__ __forceinline__ bool kept(float v, int i, const Edge &e)
{
    const uint32_t k = key_of(v);
    return k > e.key || (k == e.key && i <= e.limit);
}

__device__ __forceinline__ void emit(const SampleArgs &a, int64_t b, int64_t token, float logp)
{
    a.token[b] = token;
    if (a.logp) a.logp[b] = logp;
}

// The token of a row whose shares' kept weights are sh.sub[0..subs)
template <typename T>
__device__ __forceinline__ void pick(const SampleArgs &a, const Row &r, int64_t b, const T *x, int subs, const Edge &e,
                                     Shared &sh)
{
    double all, total;
    const double mine = threadIdx.x < static_cast<unsigned>(subs) ? sh.sub[threadIdx.x] : 0.0;
    const double before = scan_block(mine, sh.wd, total);
    const double target = static_cast<double>(r.u) * total;
    if (threadIdx.x == 0) sh.at = subs;
    __syncthreads();
    if (mine > 0.0 && before + mine > target) atomicMin(&sh.at, static_cast<int>(threadIdx.x));
    __syncthreads();
    // (a target that rounding puts past the last share's end: the last one)
    const int j = sh.at;
    if (threadIdx.x == 0) sh.last = -1;
    __syncthreads();
    if (j == subs && mine > 0.0) atomicMax(&sh.last, static_cast<int>(threadIdx.x));
    __syncthreads();
    const int sub = j < subs ? j : sh.last;
    if (threadIdx.x == static_cast<unsigned>(sub)) sh.w_at = before;
    __syncthreads();
    const double start = sh.w_at;
    const int lo = sub * a.share, hi = lo + a.share < a.vocab ? lo + a.share : a.vocab;
    // each thread takes neighbouring places
    const int per = (a.share + kThreads - 1) / kThreads;
    const int i0 = lo + static_cast<int>(threadIdx.x) * per, i1 = i0 + per < hi ? i0 + per : hi;
    auto weight_at = [&](int i) {
        const float v = static_cast<float>(x[i]);
        if (!(v >= r.floor) || !kept(v, i, e)) return 0.0;
        const double w = weight(v, r, sh.roots);
        return w >= r.min_p ? w : 0.0;
    };
    double own = 0.0;
    for (int i = i0; i < i1; ++i) own += weight_at(i);
    const double ahead = start + scan_block(own, sh.wd, all);
    if (threadIdx.x == 0) {
        sh.at = kThreads;
        sh.last = -1;
    }
    __syncthreads();
    const int me = static_cast<int>(threadIdx.x);
    if (own > 0.0) {
        if (ahead + own > target) atomicMin(&sh.at, me);
        atomicMax(&sh.last, me);
    }
    __syncthreads();
    // the first thread whose places pass the target (the last with any, where rounding has
    // put it past all of them) finds the place: its last one, if none passes it
    if (me != (sh.at < kThreads ? sh.at : sh.last)) return;
    int at = -1;
    double run = ahead, w_at = 0.0;
    for (int i = i0; i < i1; ++i) {
        const double w = weight_at(i);
        if (!(w > 0.0)) continue;
        run += w;
        at = i;
        w_at = w;
        if (run > target) break;
    }
    emit(a, b, at, static_cast<float>(log(w_at / total)));
}

// The first of the largest, which is among the places from..to-1
template <typename T>
__device__ __forceinline__ void pick_first(const SampleArgs &a, const Row &r, int64_t b, const T *x, int from, int to, int &at)
{
    if (threadIdx.x == 0) at = to;
    __syncthreads();
    const int per = (to - from + kWaves * 512 - 1) / (kWaves * 512) * 512;
    const int lo = from + wave() * per, hi = lo + per < to ? lo + per : to;
    int first = to;
    walk(x, lo, hi, a.vec, [&](float v, int i) {
        if (v == r.max && i < first) first = i;
    });
    if (first < to) atomicMin(&at, first);
    __syncthreads();
    if (threadIdx.x == 0) emit(a, b, at, 0.0f);
}

// Sorted candidates' weights: a thread holds four neighbours
struct Four {
    double w[4];
};

__device__ __forceinline__ Four weights4(const Row &r, const uint64_t *list, int n, Shared &sh, bool by_index)
{
    Four f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * threadIdx.x + e;
        const uint64_t c = list[i < n ? i : 0];
        const uint32_t key = by_index ? ~static_cast<uint32_t>(c) : ~static_cast<uint32_t>(c >> 32);
        f.w[e] = i < n && c != ~0ull ? weight(of_key(key), r, sh.roots) : 0.0;
    }
    return f;
}

// Of the weights as top-p compares them, those of the threads before this one, and all
__device__ __forceinline__ uint64_t ahead4(const Four &f, Shared &sh, uint64_t &all)
{
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += fixed(f.w[e]);
    return scan_block(sum, sh.wu, all);
}

__device__ __forceinline__ int pad_list(uint64_t *list, int n)
{
    int size = 64;
    while (size < n) size *= 2;
    __syncthreads();
    for (int i = n + threadIdx.x; i < size; i += kThreads) list[i] = ~0ull;
    return size;
}

// How many of the n sorted candidates stay: those with less than `want` of the weight
// ahead of them, `run` of it ahead of this thread's
__device__ __forceinline__ int cut(const Four &f, int n, uint64_t run, uint64_t want, Shared &sh)
{
    __syncthreads();
    if (threadIdx.x == 0) sh.at = 0;
    __syncthreads();
    int most = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * threadIdx.x + e;
        if (i < n && run < want) most = i + 1;
        run += fixed(f.w[e]);
    }
    if (most) atomicMax(&sh.at, most);
    __syncthreads();
    return sh.at;
}

// The edge of top-p among the n candidates, unsorted: the last that is entered with less
// than `want` of the weight ahead of it (of them: `ahead`, which is less, and the ones
// before).  Histograms over their order narrow it to a few, which are sorted.
__device__ __forceinline__ Edge select(const Row &r, int n, uint64_t ahead, uint64_t want, Shared &sh)
{
    __syncthreads();   // (the histogram has been read)
    uint64_t lo = 0, hi = ~0ull;   // the ones in question
    uint64_t *few = sh.mass;
    int left = n;
    while (left > kCounted) {
        uint64_t least = ~0ull, most = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t c = sh.list[i];
            if (c < lo || c > hi) continue;
            least = c < least ? c : least;
            most = c > most ? c : most;
        }
        for (int off = 32; off; off >>= 1) {
            const uint64_t o = __shfl_xor(least, off, 64), p = __shfl_xor(most, off, 64);
            least = o < least ? o : least;
            most = p > most ? p : most;
        }
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            sh.wu[wave()] = least;
            sh.wd[wave()] = __longlong_as_double(static_cast<long long>(most));
        }
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            sh.count[i] = 0;
            sh.mass[i] = 0;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint64_t o = sh.wu[w], p = static_cast<uint64_t>(__double_as_longlong(sh.wd[w]));
            least = o < least ? o : least;
            most = p > most ? p : most;
        }
        const int bits = 64 - __builtin_clzll((most - least) | 1), shift = bits > kBinBits ? bits - kBinBits : 0;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t c = sh.list[i];
            if (c < lo || c > hi) continue;
            const int bin = static_cast<int>((c - least) >> shift);
            atomicAdd(&sh.count[bin], 1u);
            atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[bin]),
                      fixed(weight(of_key(~static_cast<uint32_t>(c >> 32)), r, sh.roots)));
        }
        if (threadIdx.x == 0) sh.bin = 0;   // (the least is in it)
        __syncthreads();
        const int b = 2 * threadIdx.x;
        const uint64_t v0 = sh.mass[b], v1 = sh.mass[b + 1];
        const uint32_t c0 = sh.count[b], c1 = sh.count[b + 1];
        uint64_t all;
        const uint64_t sum = scan_block(v0 + v1, sh.wu, all);
        if (c1 && ahead + sum + v0 < want) atomicMax(&sh.bin, b + 1);
        else if (c0 && ahead + sum < want) atomicMax(&sh.bin, b);
        __syncthreads();
        const int bin = sh.bin;
        if (b == (bin & ~1)) sh.ahead = bin & 1 ? sum + v0 : sum;
        __syncthreads();
        ahead += sh.ahead;
        lo = least + (static_cast<uint64_t>(bin) << shift);
        hi = lo + ((1ull << shift) - 1);
        left = static_cast<int>(sh.count[bin]);
        __syncthreads();   // (the next histogram, or the few, take its place)
    }
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t c = sh.list[i];
        if (c >= lo && c <= hi) few[atomicAdd(&sh.n, 1u)] = c;
    }
    sort_list(few, pad_list(few, left));
    uint64_t all;
    const Four f = weights4(r, few, left, sh, false);
    const int m = cut(f, left, ahead + ahead4(f, sh, all), want, sh);
    const uint64_t c = few[m > 1 ? m - 1 : 0];
    return Edge{~static_cast<uint32_t>(c >> 32), static_cast<int>(static_cast<uint32_t>(c))};
}

// Top-k: the list holds all candidates, n of them; top-p, min-p and the draw are done on it
__device__ __forceinline__ void finish_list(const SampleArgs &a, const Row &r, int64_t b, int n, Shared &sh)
{
    sort_list(sh.list, pad_list(sh.list, n));
    n = n < r.top_k ? n : r.top_k;
    Four f = weights4(r, sh.list, n, sh, false);
    if (r.top_p < 1.0) {
        uint64_t mass;
        const uint64_t ahead = ahead4(f, sh, mass);
        n = cut(f, n, ahead, needed(r, mass), sh);
    }
    __syncthreads();
    // by index; what min-p drops goes to the end
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = 4 * threadIdx.x + e;
        if (i < n) {
            const uint64_t c = sh.list[i];
            sh.list[i] = f.w[e] >= r.min_p ? (c << 32) | (c >> 32) : ~0ull;
        }
    }
    sort_list(sh.list, pad_list(sh.list, n));
    f = weights4(r, sh.list, n, sh, true);   // (none of the dropped ones)
    double all, run = scan_block(((f.w[0] + f.w[1]) + f.w[2]) + f.w[3], sh.wd, all);
    const double target = static_cast<double>(r.u) * all;
    if (threadIdx.x == 0) sh.at = n;
    __syncthreads();
    int at = -1, last = -1;
    double w_at = 0.0, w_last = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        run += f.w[e];
        if (f.w[e] > 0.0) {
            last = 4 * threadIdx.x + e;
            w_last = f.w[e];
            if (at < 0 && run > target) {
                at = last;
                w_at = w_last;
            }
        }
    }
    if (threadIdx.x == 0) sh.last = -1;
    __syncthreads();
    if (at >= 0) atomicMin(&sh.at, at);
    if (last >= 0) atomicMax(&sh.last, last);
    __syncthreads();
    const int found = sh.at;
    if (at >= 0 && at == found) emit(a, b, static_cast<int64_t>(sh.list[at] >> 32), static_cast<float>(log(w_at / all)));
    if (found == n && last >= 0 && last == sh.last)
        emit(a, b, static_cast<int64_t>(sh.list[last] >> 32), static_cast<float>(log(w_last / all)));
}

// ---------------------------------------------- rows with too many candidates
// The edge of a filter over what `before` keeps, by the row's workgroup alone: want
// (a count, or a weight) is reached within the keys lo..hi, with `ahead`, which is less,
// above hi.  The range is split by histograms until it is short enough to sort or one value.
template <typename T, bool MASS>
__device__ __forceinline__ Edge narrow(const SampleArgs &a, const Row &r, const T *x, uint32_t lo, uint32_t hi, uint64_t ahead,
                                       uint64_t want, const Edge &before, Shared &sh)
{
    const int per = (a.vocab + kWaves * 512 - 1) / (kWaves * 512) * 512;
    const int i0 = wave() * per, i1 = i0 + per < a.vocab ? i0 + per : a.vocab;
    for (;;) {
        // histogram of lo..hi, largest first
        const int bits = 32 - __builtin_clz((hi - lo) | 1), shift = bits > kBinBits ? bits - kBinBits : 0;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            sh.count[i] = 0;
            sh.mass[i] = 0;
        }
        __syncthreads();
        walk(x, i0, i1, a.vec, [&](float v, int i) {
            const uint32_t k = key_of(v);
            if (!(v >= r.floor) || k < lo || k > hi || !kept(v, i, before)) return;
            // (many are equal here: one addition for the lanes with the first one's value)
            const uint64_t same = __ballot(k == __builtin_amdgcn_readfirstlane(k));
            const bool mine = k == __builtin_amdgcn_readfirstlane(k);
            if (mine && (threadIdx.x & 63) != __builtin_ctzll(same)) return;
            const uint32_t many = mine ? __popcll(same) : 1;
            const int bin = (hi - k) >> shift;
            atomicAdd(&sh.count[bin], many);
            if constexpr (MASS)
                atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[bin]), fixed(weight(v, r, sh.roots)) * many);
        });
        __syncthreads();
        const int b = 2 * threadIdx.x;
        const uint64_t v0 = MASS ? sh.mass[b] : sh.count[b], v1 = MASS ? sh.mass[b + 1] : sh.count[b + 1];
        uint64_t all;
        const uint64_t sum = scan_block(v0 + v1, sh.wu, all);
        if (threadIdx.x == 0) {
            sh.bin = 0;
            sh.last = -1;
        }
        __syncthreads();
        // the last bin that is entered with less than `want` ahead, and is not empty (the
        // first that is not empty is such a one)
        const uint32_t c0 = sh.count[b], c1 = sh.count[b + 1];
        if (c1 && ahead + sum + v0 < want) atomicMax(&sh.bin, b + 1);
        else if (c0 && ahead + sum < want) atomicMax(&sh.bin, b);
        __syncthreads();
        const int bin = sh.bin;
        if (b == (bin & ~1)) sh.ahead = bin & 1 ? sum + v0 : sum;
        __syncthreads();
        ahead += sh.ahead;
        const uint32_t top = hi - (static_cast<uint32_t>(bin) << shift);
        const uint32_t span = (1u << shift) - 1;
        lo = top - lo > span ? top - span : lo;
        hi = top;
        const int n = sh.count[bin];
        if (n <= kList) {
            // few: sort them
            __syncthreads();
            if (threadIdx.x == 0) sh.n = 0;
            __syncthreads();
            walk(x, i0, i1, a.vec, [&](float v, int i) {
                const uint32_t k = key_of(v);
                if (!(v >= r.floor) || k < lo || k > hi || !kept(v, i, before)) return;
                sh.list[atomicAdd(&sh.n, 1u)] = (static_cast<uint64_t>(~k) << 32) | static_cast<uint32_t>(i);
            });
            sort_list(sh.list, pad_list(sh.list, n));
            int m;
            if constexpr (MASS) {
                uint64_t in;
                const Four f = weights4(r, sh.list, n, sh, false);
                m = cut(f, n, ahead + ahead4(f, sh, in), want, sh);
            } else {
                m = want - ahead < static_cast<uint64_t>(n) ? static_cast<int>(want - ahead) : n;
            }
            const uint64_t c = sh.list[m - 1];
            __syncthreads();
            return Edge{~static_cast<uint32_t>(c >> 32), static_cast<int>(static_cast<uint32_t>(c))};
        }
        if (lo == hi) {
            // one value: the first few of its places
            int m = n;
            uint64_t places = want - ahead;
            if constexpr (MASS) {
                const uint64_t w = fixed(weight(of_key(lo), r, sh.roots));
                places = w ? (places - 1) / w + 1 : n;
            }
            if (places < static_cast<uint64_t>(n)) m = static_cast<int>(places);
            // the index of the m-th: counted by threads' neighbouring places
            const int each = (a.vocab + kThreads - 1) / kThreads;
            const int j0 = threadIdx.x * each, j1 = j0 + each < a.vocab ? j0 + each : a.vocab;
            uint64_t own = 0, total;
            auto same = [&](int i) {
                const float v = static_cast<float>(x[i]);
                return key_of(v) == lo && kept(v, i, before);
            };
            for (int i = j0; i < j1; ++i) own += same(i);
            uint64_t seen = scan_block(own, sh.wu, total);
            if (seen < static_cast<uint64_t>(m) && seen + own >= static_cast<uint64_t>(m))
                for (int i = j0; i < j1; ++i)
                    if (same(i) && ++seen == static_cast<uint64_t>(m)) sh.last = i;
            __syncthreads();
            const int limit = sh.last;
            __syncthreads();
            return Edge{lo, limit};
        }
    }
}

// Kept weights of all of a row, into the shares' sums
template <typename T>
__device__ __forceinline__ void kept_sums(const SampleArgs &a, const Row &r, const T *x, int subs, const Edge &e, Shared &sh)
{
    for (int s = wave(); s < subs; s += kWaves) {
        double sum = 0.0;
        const int lo = s * a.share, hi = lo + a.share < a.vocab ? lo + a.share : a.vocab;
        walk(x, lo, hi, a.vec, [&](float v, int i) {
            if (!(v >= r.floor) || !kept(v, i, e)) return;
            const double w = weight(v, r, sh.roots);
            sum += w >= r.min_p ? w : 0.0;
        });
        sum = wave_sum(sum);
        if ((threadIdx.x & 63) == 0) sh.sub[s] = sum;
    }
    __syncthreads();
}

// The weight that the edge keeps, as top-p compares it
template <typename T>
__device__ __forceinline__ uint64_t kept_mass(const SampleArgs &a, const Row &r, const T *x, const Edge &e, Shared &sh)
{
    const int per = (a.vocab + kWaves * 512 - 1) / (kWaves * 512) * 512;
    const int i0 = wave() * per, i1 = i0 + per < a.vocab ? i0 + per : a.vocab;
    uint64_t sum = 0, all;
    walk(x, i0, i1, a.vec, [&](float v, int i) {
        if (v >= r.floor && kept(v, i, e)) sum += fixed(weight(v, r, sh.roots));
    });
    scan_block(sum, sh.wu, all);
    return all;
}

template <typename T>
__device__ __forceinline__ void solve_alone(const SampleArgs &a, const Row &r, int64_t b, const T *x, int subs, Shared &sh)
{
    Edge e{0, a.vocab};
    const uint32_t top = key_of(r.max);
    if (r.top_k) e = narrow<T, false>(a, r, x, 1, top, 0, static_cast<uint64_t>(r.top_k), e, sh);
    if (r.top_p < 1.0) e = narrow<T, true>(a, r, x, 1, top, 0, needed(r, kept_mass(a, r, x, e, sh)), e, sh);
    kept_sums(a, r, x, subs, e, sh);
    pick(a, r, b, x, subs, e, sh);
}

// The last step of a row: thresholds and candidates are known (in LDS: sh.bin, sh.ahead,
// sh.list with `n` found in all, sh.sub)
template <typename T>
__device__ __forceinline__ void finish(const SampleArgs &a, const Row &r, int64_t b, const T *x, int subs, int n,
                                       uint64_t want, Shared &sh)
{
    if (r.kind == PLAIN) {
        pick(a, r, b, x, subs, Edge{0, a.vocab}, sh);
        return;
    }
    if (n > kList && r.kind == TOP_P) {
        // the end's bin is known, and the weight ahead of it
        const int end = sh.bin;
        const uint64_t ahead = sh.ahead;
        const uint32_t lo = key_of(bin_floor(end, r));
        const uint32_t hi = end > 0 ? key_of(bin_floor(end - 1, r)) - 1 : key_of(r.max);
        const Edge e = narrow<T, true>(a, r, x, lo, hi, ahead, want, Edge{0, a.vocab}, sh);
        kept_sums(a, r, x, subs, e, sh);
        pick(a, r, b, x, subs, e, sh);
        return;
    }
    if (n > kList) {
        solve_alone(a, r, b, x, subs, sh);
        return;
    }
    if (r.kind == TOP_K) {
        finish_list(a, r, b, n, sh);
        return;
    }
    const Edge e = select(r, n, sh.ahead, want, sh);
    // the weights of the kept ones into the sums of their shares: up to 2^12 multiples
    // of 2^-51, rounded down, whose sum no order changes (each is 2^-44 or more, so that a
    // share with a kept one has a sum)
    uint64_t *more = reinterpret_cast<uint64_t *>(sh.count);
    static_assert(sizeof(sh.count) >= sizeof(uint64_t) * kMaxSlices * kWaves, "one for each share");
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(subs)) more[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t c = sh.list[i];
        const float v = of_key(~static_cast<uint32_t>(c >> 32));
        const int at = static_cast<int>(static_cast<uint32_t>(c));
        const double w = weight(v, r, sh.roots);
        if (kept(v, at, e) && w >= r.min_p)
            atomicAdd(reinterpret_cast<unsigned long long *>(&more[at / a.share]),
                      static_cast<unsigned long long>(w * 0x1p51));
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(subs)) sh.sub[threadIdx.x] += static_cast<double>(more[threadIdx.x]) * 0x1p-51;
    __syncthreads();
    pick(a, r, b, x, subs, e, sh);
}

__device__ __forceinline__ void clear_histogram(Shared &sh)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        sh.count[i] = 0;
        sh.mass[i] = 0;
    }
    if (threadIdx.x == 0) sh.n = 0;
}

// Whole workgroup: a bin up to which there are top_k logits at least: that many of the
// threads' largest ones (`own`) are.  About as many logits are, where top_k is half of the
// threads or less and they lie anywhere.  Whether there is such a bin.
__device__ __forceinline__ bool end_of_maxima(const Row &r, float own, Shared &sh)
{
    const int bin = bin_of(own, r);
    if (bin < kBins) atomicAdd(&sh.count[bin], 1u);
    __syncthreads();
    end_bin(r, sh.count, sh.mass, sh);
    return sh.bin < kBins;
}

// Without filters, 1 and 3 at once: the sum of the weights of a wave's share, as parts of
// the share's own largest (`top`; NaN if it holds one), which is 1 of them
template <typename T>
__device__ __forceinline__ double share_sum(const SampleArgs &a, int64_t b, const T *x, int lo, int hi, const double *roots,
                                            float &top)
{
    constexpr int N = Wide<T>::N;
    double sum = 0.0;
    bool nan = false;
    Row r{};
    top = -kInf;
    for (int base = lo; base < hi; base += 64 * N * kLoads) {
        float v[kLoads][N], most = -kInf;
        load_some(x, base, hi, a.vec, v);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                most = fmaxf(most, v[j][e]);
                nan |= v[j][e] != v[j][e];
            }
        for (int off = 32; off; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
        if (most > top) {
            r = settings(a, b, most);
            if (r.kind == PLAIN) sum *= weight(top, r, roots);
            top = most;
        }
        if (!(top > -kInf) || r.kind != PLAIN) continue;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (base + j * 64 * N >= hi) break;
#pragma unroll
            for (int e = 0; e < N; ++e) sum += weight(v[j][e], r, roots);
        }
    }
    if (__ballot(nan)) top = __builtin_nanf("");
    return wave_sum(sum);
}

// The shares' sums as parts of the row's largest.  (One of a share whose own largest has no
// weight is nothing: its token could not be found.)
__device__ __forceinline__ void scale_sums(const Row &r, int subs, const double *sums, const float *tops, int stride, Shared &sh)
{
    for (int i = threadIdx.x; i < subs; i += kThreads)
        sh.sub[i] = sums[i] * weight(tops[i / kWaves * stride + i % kWaves], r, sh.roots);
    __syncthreads();
}

// A row from its logits
template <typename T> __device__ __forceinline__ void by_sorting(const SampleArgs &a, int64_t b, const T *x, Shared &sh)
{
    const int lo = wave() * a.share < a.vocab ? wave() * a.share : a.vocab;
    const int hi = lo + a.share < a.vocab ? lo + a.share : a.vocab;
    fill_roots(sh.roots);
    clear_histogram(sh);
    float own;
    const Row r = settings(a, b, slice_top(a, x, lo, hi, sh, own));
    if (r.kind == DONE) {
        if (threadIdx.x == 0) emit(a, b, -1, -kInf);
        return;
    }
    if (r.kind == GREEDY) {
        pick_first(a, r, b, x, 0, a.vocab, sh.at);
        return;
    }
    uint64_t want = 0;
    bool known = r.kind == PLAIN;
    if (r.kind == TOP_K && r.top_k <= kThreads / 2) {
        known = end_of_maxima(r, own, sh);
        if (!known) clear_histogram(sh);
        __syncthreads();
    }
    if (!known) {
        histogram(a, r, x, lo, hi, sh);
        __syncthreads();
        want = end_bin(r, sh.count, sh.mass, sh);
    }
    const double sum = gather(a, r, x, lo, hi, sh.bin, sh, &sh.n, sh.list);
    if ((threadIdx.x & 63) == 0) sh.sub[wave()] = sum;
    __syncthreads();
    finish(a, r, b, x, kWaves, static_cast<int>(sh.n), want, sh);
}

template <typename T> __global__ void __launch_bounds__(kThreads) sample_row_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    const int64_t b = blockIdx.x;
    by_sorting(a, b, static_cast<const T *>(a.logits) + b * a.stride, sh);
}

template <typename T> __global__ void __launch_bounds__(kThreads) sample_plain_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    const int64_t b = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + b * a.stride;
    const int lo = wave() * a.share < a.vocab ? wave() * a.share : a.vocab;
    fill_roots(sh.roots);
    __syncthreads();
    float top;
    const double sum = share_sum(a, b, x, lo, lo + a.share < a.vocab ? lo + a.share : a.vocab, sh.roots, top);
    if ((threadIdx.x & 63) == 0) {
        sh.top[wave()] = top;
        sh.wd[wave()] = sum;
    }
    __syncthreads();
    top = sh.top[0];
    for (int w = 1; w < kWaves; ++w) top = larger(top, sh.top[w]);
    const Row r = settings(a, b, top);
    if (r.kind == DONE) {
        if (threadIdx.x == 0) emit(a, b, -1, -kInf);
        return;
    }
    if (r.kind == GREEDY) {
        pick_first(a, r, b, x, 0, a.vocab, sh.at);
        return;
    }
    scale_sums(r, kWaves, sh.wd, sh.top, kWaves, sh);
    pick(a, r, b, x, kWaves, Edge{0, a.vocab}, sh);
}

// ------------------------------------------------ rows counted by their values
// bf16 has so few values between 2^-13 and 2^10 that a workgroup counts each, for a share
// of the row and another: one pass over the row, then all filters end at a value and a
// number of its equals, the shares' sums are products of counts and weights, and the
// token's share alone is read again.  Values nearer to 0, but not 0, are listed, their weights
// taken one by one; a row where a filter ends among them, or with values past 2^10 that
// matter, goes by sorting.
constexpr int kTallies = 4;                       // shares
constexpr int kFirstMag = 114 << 7, kSide = 23 << 7;   // 2^-13 as bits; values of a sign
constexpr int kMiddle = kSide, kValues = 2 * kSide + 1;   // from the largest to the smallest; 0 is the middle
constexpr int kOutside = kValues + 1;                     // of no weight
constexpr int kEach = (kValues + kThreads - 1) / kThreads;
constexpr int kOthers = 512;
constexpr uint32_t kStop = 1, kLow = 2;           // a value that counting does not serve; one of -2^10 or less

struct Tally {
    alignas(16) uint32_t count[kTallies][kEach * kThreads];
    double w[kEach * kThreads];         // of the values ahead of the edge; 0 for the others
    double roots[kRoots];
    uint32_t others[kOthers];   // bits, share << 16
    uint64_t wu[kWaves], mid, mid_sum[kTallies];
    double wd[kWaves], part[kTallies][kWaves], w_edge;
    uint32_t eq[kWaves];
    uint32_t n, flags, m;
    int top, edge, at;
};

__device__ __forceinline__ float value_of(int pos)
{
    const int c = pos < kMiddle ? kMiddle - pos : pos - kMiddle;
    const float v = __uint_as_float(static_cast<uint32_t>(kFirstMag - 1 + c) << 16 | (pos < kMiddle ? 0u : 0x80000000u));
    return c == 0 ? 0.0f : v;
}

// Whether a value, the one with these bits, is listed
__device__ __forceinline__ bool listed(uint32_t bits) { return (bits & 0x7FFFu) - 1u < kFirstMag - 1u; }

// How far it is from the middle, if it is not: above kSide outside
__device__ __forceinline__ int distance(uint32_t bits)
{
    const int over = static_cast<int>(bits & 0x7FFFu) - (kFirstMag - 1);
    return over > 0 ? over : 0;
}

__device__ __forceinline__ int place_of(uint32_t bits, int distance)
{
    return kMiddle + (bits & 0x8000u ? distance : -distance);
}

typedef uint32_t Bits8 __attribute__((ext_vector_type(4)));

// Eight values from place i on; -inf stands for places from hi on
__device__ __forceinline__ Bits8 load_bits(const __bf16 *x, int i, int hi, bool vec)
{
    const uint16_t *bits = reinterpret_cast<const uint16_t *>(x);
    if (vec && i + 8 <= hi) return *reinterpret_cast<const Bits8 *>(bits + i);
    Bits8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t low = i + 2 * e < hi ? bits[i + 2 * e] : 0xFF80u;
        v[e] = low | static_cast<uint32_t>(i + 2 * e + 1 < hi ? bits[i + 2 * e + 1] : 0xFF80u) << 16;
    }
    return v;
}

__device__ __forceinline__ uint32_t bits_of(const Bits8 &v, int e) { return e & 1 ? v[e / 2] >> 16 : v[e / 2] & 0xFFFFu; }

// f(eight values) for the places lo..hi-1 of a row, a wave's
template <typename F> __device__ __forceinline__ void walk_bits(const __bf16 *x, int lo, int hi, bool vec, F f)
{
    constexpr int U = 4;
    const int lane = threadIdx.x & 63;
    for (int base = lo; base < hi; base += 512 * U) {
        Bits8 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] = load_bits(x, base + (j * 64 + lane) * 8, hi, vec);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (base + j * 512 >= hi) break;
            f(v[j]);
        }
    }
}

// The kept weight of a value, but for the edge's; `middle`: whether there are listed ones that
// stay
__device__ __forceinline__ double weight_of(uint32_t bits, bool middle, const Row &r, const Tally &t, int &pos)
{
    const int c = distance(bits);
    pos = c <= kSide && !listed(bits) ? place_of(bits, c) : kOutside;
    double w = t.w[pos];
    if (middle && listed(bits)) {
        w = weight(__uint_as_float(bits << 16), r, t.roots);
        w = w >= r.min_p ? w : 0.0;
    }
    return w;
}

// The token, when all is counted: it is in share s, with `ahead` of the kept weight ahead
// of it, and the share's first m values equal to the edge stay
__device__ __forceinline__ void pick_in(const SampleArgs &a, const Row &r, int64_t b, const __bf16 *x, int s, double ahead,
                                        double total, double target, int edge, uint32_t m, Tally &t)
{
    const int whole = a.share * (kWaves / kTallies), sub = a.share / kTallies, lane = threadIdx.x & 63;
    const int from = s * whole, to = from + whole < a.vocab ? from + whole : a.vocab;
    const bool middle = edge > kMiddle && t.n > 0;
    const double each = t.w_edge;
    // each wave's part of the share
    const int own = from + wave() * sub;
    double sum = 0.0;
    uint32_t equal = 0;
    walk_bits(x, own < to ? own : to, own + sub < to ? own + sub : to, a.vec, [&](const Bits8 &v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int pos;
            sum += weight_of(bits_of(v, e), middle, r, t, pos);
            equal += pos == edge;
        }
    });
    sum = wave_sum(sum);
    equal = wave_sum(equal);
    if (lane == 0) {
        t.wd[wave()] = sum;
        t.eq[wave()] = equal;
    }
    __syncthreads();
    int part = 0;   // (the last with any weight, where rounding has put the target past all)
    double run = ahead, start = ahead;
    uint32_t rest = m, left = m;
    bool found = false;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t stay = t.eq[w] < rest ? t.eq[w] : rest;
        const double mine = t.wd[w] + stay * each;
        if (mine > 0.0 && !found) {
            part = w;
            start = run;
            left = rest;
            found = run + mine > target;
        }
        run += mine;
        rest -= stay;
    }
    if (wave() != part) return;
    // its wave finds the place
    run = start;
    int last = -1;
    double w_last = 0.0;
    const int lo = from + part * sub, hi = lo + sub < to ? lo + sub : to;
    for (int base = lo; base < hi; base += 512) {
        const int i = base + lane * 8;
        const Bits8 v = load_bits(x, i, hi, a.vec);
        double w[8], mine = 0.0;
        bool same[8];
        uint32_t equals = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int pos;
            w[e] = weight_of(bits_of(v, e), middle, r, t, pos);
            same[e] = pos == edge;
            equals += same[e];
        }
        if (__ballot(equals != 0) && left) {
            uint32_t up = equals;
            for (int off = 1; off < 64; off <<= 1) {
                const uint32_t o = __shfl_up(up, off, 64);
                if (lane >= off) up += o;
            }
            uint32_t before = up - equals;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (same[e] && before < left) w[e] = each;
                before += same[e];
            }
            const uint32_t seen = __builtin_amdgcn_readlane(up, 63);
            left -= seen < left ? seen : left;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mine += w[e];
            if (w[e] > 0.0) {
                last = i + e;
                w_last = w[e];
            }
        }
        double up = mine;
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(up, off, 64);
            if (lane >= off) up += o;
        }
        const uint64_t past = __ballot(mine > 0.0 && run + up > target);
        if (past) {
            if (lane != __builtin_ctzll(past)) return;
            double at = run + (up - mine), w_at = 0.0;
            int chosen = -1;
            bool over = false;   // (the last one, if rounding leaves none)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (w[e] > 0.0 && !over) {
                    chosen = i + e;
                    w_at = w[e];
                }
                at += w[e];
                over |= at > target;
            }
            emit(a, b, chosen, static_cast<float>(log(w_at / total)));
            return;
        }
        run += __shfl(up, 63, 64);
    }
    int most = last;
    for (int off = 32; off; off >>= 1) {
        const int o = __shfl_xor(most, off, 64);
        most = o > most ? o : most;
    }
    if (last == most && last >= 0) emit(a, b, last, static_cast<float>(log(w_last / total)));
}

// A row by counting; false (for the whole workgroup) where that does not serve it
__device__ __forceinline__ bool by_counting(const SampleArgs &a, int64_t b, const __bf16 *x, Tally &t)
{
    const int s_own = wave() / (kWaves / kTallies), me = static_cast<int>(threadIdx.x);
    fill_roots(t.roots);
    for (int i = me; i < static_cast<int>(sizeof(t.count) / 16); i += kThreads)
        reinterpret_cast<f32x4 *>(&t.count[0][0])[i] = f32x4{0, 0, 0, 0};
    if (me < kTallies) t.mid_sum[me] = 0;
    if (me == 0) {
        t.mid = 0;
        t.w_edge = 0.0;
        t.n = t.flags = t.m = 0;
        t.top = kValues;
        t.edge = -1;
    }
    __syncthreads();
    {
        const int lo = wave() * a.share < a.vocab ? wave() * a.share : a.vocab;
        const int hi = lo + a.share < a.vocab ? lo + a.share : a.vocab;
        uint32_t *count = t.count[s_own], flags = 0, seen = 0;
        walk_bits(x, lo, hi, a.vec, [&](const Bits8 &v) {
            if (seen > kOthers) return;   // (it goes by sorting)
            uint32_t least = ~0u;
            int most = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t o = bits_of(v, e), m = (o & 0x7FFFu) - 1u;
                const int c = distance(o);
                least = m < least ? m : least;
                most = c > most ? c : most;
                if (c <= kSide) atomicAdd(&count[place_of(o, c)], 1u);   // (what is listed is taken back)
            }
            if (__ballot(least < kFirstMag - 1u || most > kSide) == 0) return;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t o = bits_of(v, e);
                const int c = distance(o);
                if (c > kSide && o != 0xFF80u) flags |= o > 0x8000u && o < 0xFF80u ? kLow : kStop;
                const uint64_t who = __ballot(listed(o));
                if (!who) continue;
                uint32_t at = 0;
                const uint32_t many = static_cast<uint32_t>(__popcll(who));
                if ((me & 63) == __builtin_ctzll(who)) {
                    at = atomicAdd(&t.n, many);
                    atomicSub(&count[kMiddle], many);
                }
                at = __builtin_amdgcn_readlane(at, __builtin_ctzll(who)) + __popcll(who & ((1ull << (me & 63)) - 1));
                if (listed(o) && at < kOthers) t.others[at] = o | static_cast<uint32_t>(s_own) << 16;
                seen += many;
            }
        });
        if (flags) atomicOr(&t.flags, flags);
    }
    __syncthreads();
    if ((t.flags & kStop) || t.n > kOthers) return false;

    // this thread's neighbouring values
    uint32_t n[kEach];
    int first = kValues;
#pragma unroll
    for (int e = kEach - 1; e >= 0; --e) {
        const int pos = me * kEach + e;
        n[e] = 0;
#pragma unroll
        for (int s = 0; s < kTallies; ++s) n[e] += t.count[s][pos];
        if (n[e]) first = pos;
    }
    if (first < kValues) atomicMin(&t.top, first);
    __syncthreads();
    const int top = t.top;
    const uint32_t others = t.n;
    if (top == kValues || (top >= kMiddle && others)) return false;
    const Row r = settings(a, b, value_of(top));
    if (r.kind == GREEDY) {
        int s = 0;
        while (t.count[s][top] == 0) ++s;
        const int whole = a.share * (kWaves / kTallies), from = s * whole;
        pick_first(a, r, b, x, from, from + whole < a.vocab ? from + whole : a.vocab, t.at);
        return true;
    }
    if ((t.flags & kLow) && !(r.nothing > -1024.0f)) return false;
    double w[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int pos = me * kEach + e;
        // (not of one above the largest: none has it, and none times a weight past the numbers is NaN)
        w[e] = weight(fminf(value_of(pos < kValues ? pos : kValues - 1), r.top), r, t.roots);
    }
    for (int i = me; i < static_cast<int>(others); i += kThreads) {
        const double o = weight(__uint_as_float(t.others[i] << 16), r, t.roots);
        atomicAdd(reinterpret_cast<unsigned long long *>(&t.mid), static_cast<unsigned long long>(fixed(o)));
        // (one step at least: a share with a token in it has a sum)
        const unsigned long long steps = o * 0x1p51 > 1.0 ? static_cast<unsigned long long>(o * 0x1p51) : o > 0.0;
        if (o >= r.min_p)
            atomicAdd(reinterpret_cast<unsigned long long *>(&t.mid_sum[t.others[i] >> 16]), steps);
    }
    // how many of each value stay, and the last of them (what is listed goes with 0)
    if (me == kMiddle / kEach) n[kMiddle % kEach] += others;
    uint64_t all;
    bool stop = false;
    int last = -1;
    if (r.top_k) {
        uint64_t sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) sum += n[e];
        uint64_t before = scan_block(sum, t.wu, all);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const uint64_t k = static_cast<uint64_t>(r.top_k), room = before < k ? k - before : 0;
            before += n[e];
            stop |= me * kEach + e == kMiddle && others && room > 0 && room < n[e];
            n[e] = n[e] < room ? n[e] : static_cast<uint32_t>(room);
        }
    }
    __syncthreads();
    if (r.top_p < 1.0) {
        uint64_t q[kEach], sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            q[e] = fixed(w[e]) * n[e];
            if (me * kEach + e == kMiddle && others && n[e]) q[e] += t.mid - fixed(w[e]) * others;
            sum += q[e];
        }
        uint64_t before = scan_block(sum, t.wu, all);
        const uint64_t want = needed(r, all);
        uint64_t left = 0, one = 0;
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            if (n[e] && before < want) {
                last = me * kEach + e;
                left = want - 1 - before;
                one = fixed(w[e]);
                most = n[e];
            }
            before += q[e];
        }
        if (last >= 0) atomicMax(&t.edge, last);
        __syncthreads();
        if (last >= 0 && last == t.edge) t.m = one && left / one < most ? static_cast<uint32_t>(left / one) + 1 : most;
    } else if (r.top_k) {
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            if (n[e]) {
                last = me * kEach + e;
                most = n[e];
            }
        if (last >= 0) atomicMax(&t.edge, last);
        __syncthreads();
        if (last >= 0 && last == t.edge) t.m = most;
    }
    if (stop) atomicOr(&t.flags, kStop);
    __syncthreads();
    const int edge = t.edge < 0 ? kValues : t.edge;
    if ((edge == kMiddle && others) || (t.flags & kStop)) return false;
    const uint32_t m = t.m;
    // the shares' kept weights
    double sums[kTallies] = {};
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int pos = me * kEach + e;
        uint32_t rest = pos < edge ? 0xFFFFFFFFu : pos == edge ? m : 0;
        const double each = w[e] >= r.min_p ? w[e] : 0.0;
        t.w[pos] = pos < edge ? each : 0.0;
        if (pos == edge) t.w_edge = each;
#pragma unroll
        for (int s = 0; s < kTallies; ++s) {
            const uint32_t c = t.count[s][pos], stay = c < rest ? c : rest;
            rest -= stay;
            sums[s] += stay * each;
        }
    }
    // (a quarter of the lanes for each share)
    const int lane = me & 63, quarter = lane >> 4;
    static_assert(kTallies == 4 && kWaves == 16, "a lane for each share's wave");
    auto halves = [&](double low, double high, int bit) {   // of the other lanes too: low where the bit is not set
        return (lane & bit ? high : low) + __shfl_xor(lane & bit ? low : high, bit, 64);
    };
    auto within = [&](double v) {
        for (int off = 8; off; off >>= 1) v += __shfl_xor(v, off, 64);
        return v;
    };
    const double wave_part = within(halves(halves(sums[0], sums[2], 32), halves(sums[1], sums[3], 32), 16));
    if ((lane & 15) == 0) t.part[quarter][wave()] = wave_part;
    __syncthreads();
    const double share_sum = within(t.part[quarter][lane & 15]);
    double total = 0.0;
#pragma unroll
    for (int s = 0; s < kTallies; ++s) {
        sums[s] = __shfl(share_sum, 16 * s, 64) + (edge > kMiddle ? static_cast<double>(t.mid_sum[s]) * 0x1p-51 : 0.0);
        total += sums[s];
    }
    const double target = static_cast<double>(r.u) * total;
    int in = 0;
    double ahead = 0.0, run = 0.0;
    bool found = false;
#pragma unroll
    for (int s = 0; s < kTallies; ++s) {   // (the last one, where rounding has put the target past all)
        if (sums[s] > 0.0 && !found) {
            in = s;
            ahead = run;
            found = run + sums[s] > target;
        }
        run += sums[s];
    }
    uint32_t left = m;
    if (edge < kValues)
        for (int s = 0; s < in; ++s) left -= t.count[s][edge] < left ? t.count[s][edge] : left;
    pick_in(a, r, b, x, in, ahead, total, target, edge, left, t);
    return true;
}

__global__ void __launch_bounds__(kThreads) sample_count_kernel(SampleArgs a)
{
    __shared__ union Either {
        Shared sh;
        Tally t;
    } u;
    const int64_t b = blockIdx.x;
    const __bf16 *x = static_cast<const __bf16 *>(a.logits) + b * a.stride;
    if (by_counting(a, b, x, u.t)) return;
    __syncthreads();
    by_sorting(a, b, x, u.sh);
}

// ------------------------------------------------------ rows cut into slices
// Workgroup: blockIdx.x / slices is the row
struct Piece {
    int64_t b;
    int slice, lo, hi;   // this wave's share
};

__device__ __forceinline__ Piece piece(const SampleArgs &a)
{
    Piece p;
    const int64_t row = blockIdx.x / a.slices;
    p.b = row;
    p.slice = static_cast<int>(blockIdx.x - row * a.slices);
    const int64_t lo = static_cast<int64_t>(p.slice * kWaves + wave()) * a.share;
    p.lo = static_cast<int>(lo < a.vocab ? lo : a.vocab);
    p.hi = p.lo + a.share < a.vocab ? p.lo + a.share : a.vocab;
    return p;
}

__device__ __forceinline__ float row_top(const SampleArgs &a, const Slot &s)
{
    static_assert(kMaxSlices <= 64, "a lane for each");
    const int lane = threadIdx.x & 63;
    float top = lane < a.slices ? s.top[lane] : -kInf;
    for (int off = 32; off; off >>= 1) top = larger(top, __shfl_xor(top, off, 64));
    return top;
}

// Whether top_k's end comes of the groups' largest logits (as end_of_maxima says), and not
// of a histogram of all
__device__ __forceinline__ bool by_maxima(const SampleArgs &a, const Row &r) { return r.top_k <= kGroups / 2 * a.slices; }

template <typename T> __global__ void __launch_bounds__(kThreads) sample_top_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    const Piece p = piece(a);
    const Slot s = slot_of(a, p.b);
    const T *x = static_cast<const T *>(a.logits) + p.b * a.stride;
    if (a.plain) {
        fill_roots(sh.roots);
        __syncthreads();
        float most;
        const double sum = share_sum(a, p.b, x, p.lo, p.hi, sh.roots, most);
        if ((threadIdx.x & 63) == 0) {
            s.sub[p.slice * kWaves + wave()] = sum;
            s.maxima[p.slice * kGroups + wave()] = sh.top[wave()] = most;
        }
        __syncthreads();
        if (threadIdx.x != 0) return;
        for (int w = 0; w < kWaves; ++w) most = larger(most, sh.top[w]);
        s.top[p.slice] = most;
        return;
    }
    float own;
    const float top = slice_top(a, x, p.lo, p.hi, sh, own);
    if (threadIdx.x == 0) s.top[p.slice] = top;
    for (int off = 1; off < kThreads / kGroups; off <<= 1) own = fmaxf(own, __shfl_xor(own, off, 64));
    if (threadIdx.x % (kThreads / kGroups) == 0) s.maxima[p.slice * kGroups + threadIdx.x / (kThreads / kGroups)] = own;
    for (int i = p.slice * kThreads + threadIdx.x; i < kBins; i += a.slices * kThreads) {
        s.count[i] = 0;
        s.mass[i] = 0;
    }
    if (p.slice == 0 && threadIdx.x == 0) *s.n = 0;
}

template <typename T> __global__ void __launch_bounds__(kThreads) sample_bins_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    const Piece p = piece(a);
    const Slot s = slot_of(a, p.b);
    const Row r = settings(a, p.b, row_top(a, s));
    if ((r.kind != TOP_K || by_maxima(a, r)) && r.kind != TOP_P) return;
    fill_roots(sh.roots);
    clear_histogram(sh);
    __syncthreads();
    histogram(a, r, static_cast<const T *>(a.logits) + p.b * a.stride, p.lo, p.hi, sh);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        if (r.kind == TOP_K && sh.count[i]) atomicAdd(&s.count[i], sh.count[i]);
        if (r.kind == TOP_P && sh.mass[i]) atomicAdd(reinterpret_cast<unsigned long long *>(&s.mass[i]), sh.mass[i]);
    }
}

template <typename T> __global__ void __launch_bounds__(kThreads) sample_gather_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    const Piece p = piece(a);
    const Slot s = slot_of(a, p.b);
    const Row r = settings(a, p.b, row_top(a, s));
    if (r.kind == DONE || r.kind == GREEDY) return;
    fill_roots(sh.roots);
    if (r.kind == TOP_K && by_maxima(a, r)) {
        clear_histogram(sh);
        __syncthreads();
        for (int i = threadIdx.x; i < kGroups * a.slices; i += kThreads) {
            const int bin = bin_of(s.maxima[i], r);
            if (bin < kBins) atomicAdd(&sh.count[bin], 1u);
        }
        __syncthreads();
        end_bin(r, sh.count, sh.mass, sh);
    } else if (r.kind != PLAIN) {
        end_bin(r, s.count, s.mass, sh);
    }
    __syncthreads();
    const double sum = gather(a, r, static_cast<const T *>(a.logits) + p.b * a.stride, p.lo, p.hi, sh.bin, sh, s.n, s.list);
    if ((threadIdx.x & 63) == 0) s.sub[p.slice * kWaves + wave()] = sum;
}

template <typename T> __global__ void __launch_bounds__(kThreads) sample_pick_kernel(SampleArgs a)
{
    __shared__ Shared sh;
    const int64_t b = blockIdx.x;
    const Slot s = slot_of(a, b);
    const T *x = static_cast<const T *>(a.logits) + b * a.stride;
    const Row r = settings(a, b, row_top(a, s));
    if (r.kind == DONE) {
        if (threadIdx.x == 0) emit(a, b, -1, -kInf);
        return;
    }
    if (r.kind == GREEDY) {
        pick_first(a, r, b, x, 0, a.vocab, sh.at);
        return;
    }
    fill_roots(sh.roots);
    const int subs = a.slices * kWaves;
    if (a.plain) {
        __syncthreads();
        scale_sums(r, subs, s.sub, s.maxima, kGroups, sh);
        pick(a, r, b, x, subs, Edge{0, a.vocab}, sh);
        return;
    }
    const int n = static_cast<int>(*s.n);
    for (int i = threadIdx.x; i < subs; i += kThreads) sh.sub[i] = s.sub[i];
    uint64_t want = 0;
    if (r.kind != PLAIN) {
        for (int i = threadIdx.x; i < n && i < kList; i += kThreads) sh.list[i] = s.list[i];
        __syncthreads();
        if (r.kind == TOP_P) want = end_bin(r, s.count, s.mass, sh);
    }
    __syncthreads();
    finish(a, r, b, x, subs, n, want, sh);
}

struct SampleGeom {
    int slices, share;
    size_t slot;
};

constexpr int kShort = 4 * kWaves;   // what waves read at once, of a row that is not cut

int64_t wave_steps(const mgs_sample_desc &d)
{
    const int64_t step = 64 * (d.dtype == MGS_BF16 ? 8 : 4);
    return (d.vocab + step - 1) / step;
}

// cut: whether rows may be cut at all
SampleGeom sample_geometry(const mgs_sample_desc &d, bool cut)
{
    SampleGeom g{};
    const int64_t step = 64 * (d.dtype == MGS_BF16 ? 8 : 4), steps = wave_steps(d);
    // Workgroups for every CU, no more than there are waves' steps.  Rows of up to four
    // steps a wave stay with one (32000, bf16, by sorting, all filters: 1 row 21 us, cut in four
    // 26; 128 rows of mixed settings 44, in two 55); longer ones are cut (8 rows of 128000: 52, whole
    // or in four 72 and 57).
    int64_t s = !cut || steps <= kShort || d.B <= 0 ? 1 : std::min<int64_t>((steps + kWaves - 1) / kWaves, kWorkgroups / d.B);
    s = std::max<int64_t>(1, std::min<int64_t>(s, kMaxSlices));
    g.slices = static_cast<int>(s);
    g.share = static_cast<int>((steps + s * kWaves - 1) / (s * kWaves) * step);
    g.slot = s > 1 ? align256(kSlotSub + sizeof(double) * kWaves * s) : 0;
    return g;
}

// Whether some row's filter ends where only a histogram tells; one top_k for all rows that
// the threads' largest logits serve needs none
bool histograms(const SampleArgs &a)
{
    if (a.top_k) return true;
    if (a.k0 > 0 && a.k0 < a.vocab) return a.k0 > (a.slices > 1 ? kGroups / 2 * a.slices : kThreads / 2);
    return a.top_p || a.p0 < 1.0f;
}

// Whether bf16 rows are counted.  Measured, us, counted / otherwise.  With a histogram, by
// top-p: 1 and 256 rows of 32000 21/37 and 23/43, 1 and 8 of 131072 40/39 and 41/45, 256 of
// 128000 with mixed settings 45/120; of 262144 8 rows 66/56, 32 69/70, 64 70/92; 64 and 128 of
// 2^20 237/231 and 245/417.  Without one: 1 row of 32000 18/17, 256 of 50001 37/34, of 128000
// 40/46; 1 of 128000 36/15; by top-k 256 of 128000 41/38, by min-p 40/33.
bool counted(const mgs_sample_desc &d, const SampleArgs &a)
{
    if (d.dtype != MGS_BF16) return false;
    const int64_t steps = wave_steps(d);
    if (histograms(a)) return a.slices <= 4 || steps <= 4 * kShort;
    return a.plain && a.slices == 1 && steps > 2 * kShort;
}

template <typename T> hipError_t run(const SampleArgs &a, unsigned rows, hipStream_t s)
{
    if (a.slices == 1) {
        if (a.plain) sample_plain_kernel<T><<<dim3(rows), dim3(kThreads), 0, s>>>(a);
        else sample_row_kernel<T><<<dim3(rows), dim3(kThreads), 0, s>>>(a);
        return hipGetLastError();
    }
    const dim3 grid(rows * a.slices), block(kThreads);
    sample_top_kernel<T><<<grid, block, 0, s>>>(a);
    if (histograms(a)) sample_bins_kernel<T><<<grid, block, 0, s>>>(a);
    if (!a.plain) sample_gather_kernel<T><<<grid, block, 0, s>>>(a);
    sample_pick_kernel<T><<<dim3(rows), block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t sample_workspace(const mgs_sample_desc &d)
{
    // (more rows than this are not cut; the bytes of fewer grow with their number)
    mgs_sample_desc cut = d;
    cut.B = std::min<int64_t>(d.B, kWorkgroups / 2);
    return kHeader + sample_geometry(cut, true).slot * static_cast<size_t>(cut.B);
}

hipError_t launch_sample(const mgs_sample_desc &d, const void *logits, const float *u, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                         void *ws, hipStream_t s)
{
    SampleGeom g = sample_geometry(d, true);
    const int size = d.dtype == MGS_BF16 ? 2 : 4;
    const bool vec = (reinterpret_cast<uintptr_t>(logits) & 15) == 0 && (d.B == 1 || (d.logits_stride * size) % 16 == 0);
    SampleArgs a{logits, u, temperature, top_p, min_p, top_k, token, logp, d.logits_stride,
                       static_cast<char *>(ws), g.slot, static_cast<int>(d.vocab), g.slices, g.share, d.top_k,
                       d.temperature, d.top_p, d.min_p, vec, false};
    a.plain = !histograms(a) && !(a.k0 > 0 && a.k0 < a.vocab) && !a.min_p && !(a.m0 > 0.0f);
    const unsigned rows = static_cast<unsigned>(d.B);
    if (counted(d, a)) {
        g = sample_geometry(d, false);
        a.slices = g.slices;
        a.share = g.share;
        sample_count_kernel<<<dim3(rows), dim3(kThreads), 0, s>>>(a);
        return hipGetLastError();
    }
    return d.dtype == MGS_BF16 ? run<__bf16>(a, rows, s) : run<float>(a, rows, s);
}

}  // namespace mgs
