// sample.hip -- sampling of the next token with temperature, top-k, top-p and
// min-p (gfx950).
//
// All three filters keep a prefix of the order by (logit descending, index
// ascending), so what is kept is a threshold: everything above a value, and of its
// equals the first few by index.
#include <hip/hip_runtime.h>

#include "device.hpp"
#include "layers.hpp"
#include "tokens.hpp"

namespace mgs {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

struct SampleArgs {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *token;
    float *logp;
    int64_t vocab, stride;
    int k0;
    float t0, p0, m0;
};

// Unsigned numbers in the order of the floats (NaN apart; -0 counts as 0)
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ double weight(float x, float top, double inv)
{
    if (x == top) return 1.0;
    if (x == -__builtin_inff() || top == __builtin_inff()) return 0.0;
    return exp((static_cast<double>(x) - static_cast<double>(top)) * inv);
}

template <typename V> __device__ __forceinline__ V block_sum(V v, V *lds)
{
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
    for (int w = 1; w < kWaves; ++w) v += lds[w];
    return v;
}

// sum over the threads before this one
template <typename V> __device__ __forceinline__ V block_before(V v, V *lds)
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    V up = v;
    for (int off = 1; off < 64; off <<= 1) {
        const V o = __shfl_up(up, off, 64);
        if (lane >= off) up += o;
    }
    __syncthreads();
    if (lane == 63) lds[wv] = up;
    __syncthreads();
    V sum = 0;
    for (int w = 0; w < wv; ++w) sum += lds[w];
    const V prev = __shfl_up(up, 1, 64);
    return lane ? sum + prev : sum;
}

// A workgroup for each row
template <typename T> __global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a)
{
    __shared__ double sd[kWaves];
    __shared__ uint64_t su[kWaves];
    __shared__ int found;
    const int64_t b = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + b * a.stride;
    const int V = static_cast<int>(a.vocab), tid = threadIdx.x;
    float tau = a.temperature ? a.temperature[b] : a.t0, top_p = a.top_p ? a.top_p[b] : a.p0;
    float min_p = a.min_p ? a.min_p[b] : a.m0, u = a.u[b];
    const int top_k = a.top_k ? a.top_k[b] : a.k0;
    if (!(tau > 0.0f)) tau = 0.0f;
    min_p = min_p > 0.0f ? (min_p < 1.0f ? min_p : 1.0f) : 0.0f;
    u = u > 0.0f ? (u < 1.0f ? u : 0.99999994f) : 0.0f;

    // the largest, its first place; whether there is a NaN
    uint64_t best = 0;   // (key, places from the end)
    bool nan = false;
    for (int i = tid; i < V; i += kThreads) {
        const float v = static_cast<float>(x[i]);
        nan |= v != v;
        const uint64_t c = (static_cast<uint64_t>(key_of(v)) << 32) | static_cast<uint32_t>(~i);
        best = c > best ? c : best;
    }
    for (int off = 32; off; off >>= 1) {
        const uint64_t o = __shfl_xor(best, off, 64);
        best = o > best ? o : best;
    }
    if ((tid & 63) == 0) su[tid >> 6] = best;
    nan = __syncthreads_or(nan);
    for (int w = 0; w < kWaves; ++w) best = su[w] > best ? su[w] : best;
    const uint32_t top_key = static_cast<uint32_t>(best >> 32);
    const float top = of_key(top_key);
    const float inf = __builtin_inff();
    if (nan || top == -inf || V == 0) {
        if (tid == 0) {
            a.token[b] = -1;
            if (a.logp) a.logp[b] = -inf;
        }
        return;
    }
    if (tau == 0.0f) {
        if (tid == 0) {
            a.token[b] = static_cast<int64_t>(~static_cast<uint32_t>(best));
            if (a.logp) a.logp[b] = 0.0f;
        }
        return;
    }
    const double inv = 1.0 / static_cast<double>(tau);

    // kept: keys above `edge`, and the first `ties` of its equals
    uint32_t edge = 0;
    int64_t ties = V;
    __syncthreads();
    auto count_over = [&](uint32_t k) {   // keys above k
        uint64_t n = 0;
        for (int i = tid; i < V; i += kThreads) n += key_of(static_cast<float>(x[i])) > k;
        return static_cast<int64_t>(block_sum(n, su));
    };
    auto mass_over = [&](uint32_t k, uint32_t floor, int64_t equal) {   // of keys above k, and `equal` of floor's
        double m = 0.0;
        for (int i = tid; i < V; i += kThreads) {
            const float v = static_cast<float>(x[i]);
            const uint32_t c = key_of(v);
            if (c > k && c > floor) m += weight(v, top, inv);
        }
        m = block_sum(m, sd);
        if (floor > k) m += static_cast<double>(equal) * weight(of_key(floor), top, inv);
        return m;
    };
    if (top_k > 0 && top_k < V) {
        // the smallest key with fewer than top_k above it
        uint32_t lo = 0, hi = 0xFFFFFFFFu;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (count_over(mid) < top_k) hi = mid;
            else lo = mid + 1;
        }
        edge = lo;
        ties = top_k - count_over(lo);
    }
    if (top_p < 1.0f) {
        int64_t equal = count_over(edge - 1) - count_over(edge);
        if (edge == 0) equal = 0;
        equal = equal < ties ? equal : ties;
        const double want = static_cast<double>(top_p) * mass_over(0, edge, equal);
        uint32_t lo = edge, hi = top_key;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (mass_over(mid, edge, equal) < want) hi = mid;
            else lo = mid + 1;
        }
        // of the equals of lo, those with less than `want` ahead of them
        const double ahead = mass_over(lo, edge, equal), w = weight(of_key(lo), top, inv);
        const int64_t same = lo == edge ? equal : count_over(lo - 1) - count_over(lo);
        int64_t n = 0, most = same;
        while (n < most) {
            const int64_t mid = (n + most) / 2;
            if (ahead + static_cast<double>(mid) * w < want) n = mid + 1;
            else most = mid;
        }
        edge = lo;
        ties = lo == top_key && n == 0 ? 1 : n;
    }
    // kept weights of each thread's neighbouring places, equals of the edge counted from the first
    const int per = (V + kThreads - 1) / kThreads;
    const int i0 = tid * per, i1 = i0 + per < V ? i0 + per : V;
    int64_t equals = 0;
    for (int i = i0; i < i1; ++i) equals += key_of(static_cast<float>(x[i])) == edge;
    int64_t seen = static_cast<int64_t>(block_before(static_cast<uint64_t>(equals), su));
    auto kept = [&](int i, int64_t &rank) {
        const float v = static_cast<float>(x[i]);
        const uint32_t c = key_of(v);
        if (c < edge || (c == edge && rank++ >= ties)) return 0.0;
        const double w = weight(v, top, inv);
        return w >= static_cast<double>(min_p) ? w : 0.0;
    };
    double mine = 0.0;
    int64_t rank = seen;
    for (int i = i0; i < i1; ++i) mine += kept(i, rank);
    const double before = block_before(mine, sd), total = block_sum(mine, sd);
    const double target = static_cast<double>(u) * total;
    if (tid == 0) found = V;
    __syncthreads();
    int at = V;
    double w_at = 0.0, run = before;
    rank = seen;
    if (before + mine > target)
        for (int i = i0; i < i1; ++i) {
            const double w = kept(i, rank);
            run += w;
            if (run > target && w > 0.0) {
                at = i;
                w_at = w;
                break;
            }
        }
    if (at < V) atomicMin(&found, at);
    __syncthreads();
    if (at < V && at == found) {
        a.token[b] = at;
        if (a.logp) a.logp[b] = static_cast<float>(log(w_at / total));
    }
}

}  // namespace

size_t sample_workspace(const mgs_sample_desc &) { return 256; }

hipError_t launch_sample(const mgs_sample_desc &d, const void *logits, const float *u, const float *temperature,
                         const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                         void *, hipStream_t s)
{
    SampleArgs a{logits, u, temperature, top_p, min_p, top_k, token, logp, d.vocab, d.logits_stride, d.top_k,
                 d.temperature, d.top_p, d.min_p};
    const dim3 grid(static_cast<unsigned>(d.B)), block(kThreads);
    if (d.dtype == MGS_BF16) sample_kernel<__bf16><<<grid, block, 0, s>>>(a);
    else sample_kernel<float><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mgs
