// embed.hip -- the embedding lookup with scaling, and the table's gradient by
// sorted ids (gfx950).
//
//     y_n = scale W[id_n],      dW_v = scale sum over n with id_n = v of dy_n
//
// Gradient: three kernels.  The first sorts the places n by their ids (equal ones next to
// each other; the order of the ids does not matter): of 2^b workgroups each serves the
// ids of one remainder, so that the low ids, which are most of a text in many
// vocabularies, are spread over all of them (in ranges of ids, one workgroup had half
// of the places: 32768 of them 243 us).  It reads all ids (they stay in L2) and places its
// own by counting, without a word to any other workgroup.  The second walks the sorted
// places in chunks of equal length, so that an id that makes up half of a text costs
// no workgroup more than the others, adds the rows up in fp32 and writes each sum that
// lies inside a chunk, while workgroups behind these write the zeros of the rows that no
// id points to, most of the traffic of a large table; the third joins the sums that cross
// chunks.  All orders are fixed by the ids.
//
// What bounds it: bytes, where there are many.  32768 rows of 2048 of 128000, bf16: lookup
// 40 us (220 MB reach HBM: 5.5 TB/s), the gradient 12.7 + 135 + 6.6, where 667 MB of rows and
// table move at 4.9 TB/s; added to the table 59 in all (11766 rows occur).  4095 rows of 1000 of
// 5003, fp32: 8.2, and 5.8 + 9.6 + 4.8, of it some 3 a launch; added 18.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "launch.hpp"
#include "layers.hpp"
#include "tokens.hpp"

namespace mgs {
namespace {

constexpr int kMaxChunk = 32;     // sorted places of a workgroup (one more lane looks behind them)
constexpr int kSortWaves = 16;
constexpr int kMaxRange = 512;    // ids of a sorting workgroup
constexpr int kHeld = 256;        // places of its ids that a sorting wave remembers

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f8v __attribute__((ext_vector_type(8), aligned(16)));

template <typename T> struct Raw;
template <> struct Raw<float> { using V = f8v; };
template <> struct Raw<__bf16> { using V = bf8v; };

__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// elements c .. c + 7 of a row of d, zeros past its end
template <typename T> __device__ __forceinline__ f8v load8(const T *row, int64_t c, int64_t d, bool vec)
{
    f8v v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (vec) {
        if (c < d) v = __builtin_convertvector(*reinterpret_cast<const typename Raw<T>::V *>(row + c), f8v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < d) v[i] = static_cast<float>(row[c + i]);
    }
    return v;
}

template <typename T> __device__ __forceinline__ void store8(T *row, int64_t c, int64_t d, bool vec, f8v v)
{
    const typename Raw<T>::V o = __builtin_convertvector(v, typename Raw<T>::V);
    if (vec) {
        if (c < d) *reinterpret_cast<typename Raw<T>::V *>(row + c) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < d) row[c + i] = o[i];
    }
}

__device__ __forceinline__ int64_t id_at(const void *ids, bool wide, int64_t n)
{
    return wide ? static_cast<const int64_t *>(ids)[n] : static_cast<const int32_t *>(ids)[n];
}

// ------------------------------------------------------------------ lookup
struct LookupArgs {
    const void *ids, *W;
    void *y;
    int64_t first, n, vocab, d, ws;
    int slabs;         // pieces of 8 columns of a row, rounded up to a power of two, at most 256
    float scale;
    bool wide_ids, vec;
};

// `slabs` threads share a row, and take kRows of them, their loads in flight together
// (32768 rows of 2048, bf16: one row each 45 us)
constexpr int kRows = 4;

template <typename T> __global__ void __launch_bounds__(256) lookup_kernel(LookupArgs a)
{
    const int per = 256 / a.slabs, sub = threadIdx.x / a.slabs, t = threadIdx.x % a.slabs;
    const int64_t n0 = (a.first + blockIdx.x) * (per * kRows) + sub;
    int64_t id[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t n = n0 + k * per;
        id[k] = n < a.n ? id_at(a.ids, a.wide_ids, n) : -1;
    }
    for (int64_t c = 8 * t; c < a.d; c += 8 * a.slabs) {
        f8v v[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            v[k] = f8v{0, 0, 0, 0, 0, 0, 0, 0};
            if (id[k] >= 0 && id[k] < a.vocab)
                v[k] = load8(static_cast<const T *>(a.W) + id[k] * a.ws, c, a.d, a.vec);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t n = n0 + k * per;
            if (n < a.n) store8(static_cast<T *>(a.y) + n * a.d, c, a.d, a.vec, a.scale * v[k]);
        }
    }
}

// -------------------------------------------------------------------- sort
// Where an id stands in the order: by its remainder, then its quotient
__device__ __forceinline__ int64_t order_of(int32_t id, int bits, int range)
{
    return static_cast<int64_t>(id & ((1 << bits) - 1)) * range + (id >> bits);
}

struct SortArgs {
    const void *ids;
    int64_t block, n, vocab, d;
    int bits, range;    // 2^bits workgroups, ids of each
    int64_t *count;     // ids inside the table
    int32_t *first;     // the first place of each id, in their order, and one past the last
    int32_t *row, *id;  // sorted
};

// f(id, place) for the wave's places n0..n1-1, lane by lane, several loads in flight.  Ids
// outside the table are -1, and so are places past the end (the wave stays whole)
template <typename I, typename F> __device__ __forceinline__ void each_id(const SortArgs &a, uint32_t n0, uint32_t n1, F f)
{
    constexpr int kBatch = 4;
    const I *ids = static_cast<const I *>(a.ids);
    const I vocab = static_cast<I>(a.vocab);   // (unsigned: what is negative is past it)
    for (uint32_t n = n0 + (threadIdx.x & 63); n - (threadIdx.x & 63) < n1; n += 64 * kBatch) {
        I id[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) id[k] = ids[n + 64 * k < n1 ? n + 64 * k : n1 - 1];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            f(id[k] < vocab && n + 64 * k < n1 ? static_cast<int32_t>(id[k]) : -1, n + 64 * k);
    }
}

// Each wave takes an equal share of the places and counts its ids of the range in a
// row of its own, so that it places them in order without a barrier afterwards: from
// what it remembers of them, or, if they are more, by reading its share again (32768
// ids, all read twice: 22 us).
template <typename I> __global__ void __launch_bounds__(64 * kSortWaves) sort_kernel(SortArgs a)
{
    __shared__ int32_t at[kSortWaves * kMaxRange];   // [wave][local id]: counts, then next places
    __shared__ int32_t below[kSortWaves];
    __shared__ int32_t scan[kSortWaves];
    __shared__ int2 held[kSortWaves][kHeld];         // id, place
    const int lane = threadIdx.x & 63, wv = wave();
    const int32_t mask = (1 << a.bits) - 1, own = static_cast<int32_t>(a.block + blockIdx.x);
    const int ids = a.range;   // (the last one may lie past the table)
    for (int i = threadIdx.x; i < kSortWaves * a.range; i += 64 * kSortWaves) at[i] = 0;
    __syncthreads();
    const uint32_t count = static_cast<uint32_t>(a.n), share = (count + kSortWaves - 1) / kSortWaves;
    const uint32_t n0 = wv * share < count ? wv * share : count, n1 = share < count - n0 ? n0 + share : count;
    int32_t *mine = at + wv * a.range;
    int32_t smaller = 0;
    int many = 0;
    each_id<I>(a, n0, n1, [&](int32_t id, uint32_t n) {
        const int32_t rest = id >= 0 ? id & mask : mask + 1;
        smaller += rest < own;
        const bool hit = rest == own;
        const uint64_t who = __ballot(hit);
        if (!who) return;
        if (hit) {
            atomicAdd(&at[wv * a.range + (id >> a.bits)], 1);
            const int i = many + __popcll(who & ((1ull << lane) - 1));
            if (i < kHeld) held[wv][i] = int2{id, static_cast<int32_t>(n)};
        }
        many += __popcll(who);
    });
    for (int off = 32; off; off >>= 1) smaller += __shfl_xor(smaller, off, 64);
    if (lane == 0) below[wv] = smaller;
    __syncthreads();
    int32_t base = 0;
    for (int w = 0; w < kSortWaves; ++w) base += below[w];
    // exclusive sums over (id, wave): a thread for each id
    static_assert(kMaxRange <= 64 * kSortWaves, "a thread for each id");
    const int i = threadIdx.x;
    int32_t sum = 0;
    if (i < ids)
        for (int w = 0; w < kSortWaves; ++w) sum += at[w * a.range + i];
    int32_t before = sum;   // of the threads up to this one
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t u = __shfl_up(before, off, 64);
        if (lane >= off) before += u;
    }
    if (lane == 63) scan[wv] = before;
    before -= sum;
    __syncthreads();
    for (int w = 0; w < wv; ++w) before += scan[w];
    if (i < ids) {
        int32_t next = base + before;
        a.first[static_cast<int64_t>(own) * a.range + i] = next;
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = at[w * a.range + i];
            at[w * a.range + i] = next;
            next += c;
        }
        if (own == mask && i == ids - 1) {
            a.first[static_cast<int64_t>(own + 1) * a.range] = next;
            *a.count = next;
        }
    }
    __syncthreads();
    auto put = [&](int32_t id, uint32_t n) {
        const int local = id >= 0 && (id & mask) == own ? id >> a.bits : -1;
        // one round for each id among the lanes: its lanes in order
        for (uint64_t left = __ballot(local >= 0); left;) {
            const int now = __builtin_amdgcn_readlane(local, __builtin_ctzll(left));
            const uint64_t same = __ballot(local == now);
            const int32_t start = mine[now];
            if (local == now) {
                const int32_t place = start + __popcll(same & ((1ull << lane) - 1));
                a.row[place] = static_cast<int32_t>(n);
                a.id[place] = id;
            }
            if (lane == 0) mine[now] = start + __popcll(same);
            // (a wave's LDS accesses run in order: this holds the compiler to that)
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            left &= ~same;
        }
    };
    if (many > kHeld) {
        each_id<I>(a, n0, n1, put);
        return;
    }
    for (int i = 0; i < many; i += 64) {
        const int2 h = held[wv][i + lane];   // (a multiple of 64 has room)
        put(i + lane < many ? h.x : -1, h.y);
    }
}

// -------------------------------------------------------------------- sums
struct SumArgs {
    const int64_t *count;
    const int32_t *first, *row, *id;
    float *part;       // [chunk][2][d]: of the run that enters the chunk, of the one that leaves it
    const void *dy;
    void *dW;
    int64_t block, d, gs;
    int64_t blocks;    // that add up; the ones behind them clear rows
    int64_t vocab, row_bytes;
    int bits, range, slabs, chunk;
    float scale;
    bool add, vec_in, vec_out;
};

template <typename D> __device__ __forceinline__ void put(const SumArgs &a, int64_t id, int64_t c, f8v sum)
{
    D *o = static_cast<D *>(a.dW) + id * a.d;
    sum *= a.scale;
    if (a.add) sum += load8(o, c, a.d, a.vec_out);
    store8(o, c, a.d, a.vec_out, sum);
}

__device__ __forceinline__ f8v *partial(const SumArgs &a, int64_t chunk, int which, int64_t c)
{
    const int64_t width = (a.d + 7) / 8 * 8;
    return reinterpret_cast<f8v *>(a.part + (chunk * 2 + which) * width + c);
}

// Eight elements as they are stored
template <typename T> struct Raw8 {
    typename Raw<T>::V v;
    __device__ __forceinline__ void load(const T *row, int64_t c, int64_t d, bool vec)
    {
        v = typename Raw<T>::V{0, 0, 0, 0, 0, 0, 0, 0};
        if (vec) {
            if (c < d) v = *reinterpret_cast<const typename Raw<T>::V *>(row + c);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < d) v[i] = row[c + i];
        }
    }
};

// Zeros for the rows of no id among kClear ids of a wave
constexpr int kClear = 16;

__device__ __forceinline__ void clear_rows(const SumArgs &a, int64_t block)
{
    const int lane = threadIdx.x & 63;
    const int64_t id0 = (block * 4 + wave()) * kClear, mine = id0 + lane;
    bool empty = false;
    if (lane < kClear && mine < a.vocab) {
        const int64_t o = order_of(static_cast<int32_t>(mine), a.bits, a.range);
        empty = a.first[o] == a.first[o + 1];
    }
    for (uint64_t left = __ballot(empty); left; left &= left - 1) {
        char *row = static_cast<char *>(a.dW) + (id0 + __builtin_ctzll(left)) * a.row_bytes;
        const int64_t head = (16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15;
        const int64_t wide = head < a.row_bytes ? (a.row_bytes - head) / 16 : 0;
        for (int64_t o = lane; o < wide; o += 64) {
            const f32x4 z = {0, 0, 0, 0};
            __builtin_nontemporal_store(z, reinterpret_cast<f32x4 *>(row + head) + o);
        }
        if (head == 0 && 16 * wide == a.row_bytes) continue;
        // the ends, in halves: an element is two or four bytes
        for (int64_t o = 2 * lane; o < a.row_bytes; o += 128)
            if (o < head || o >= head + 16 * wide) *reinterpret_cast<uint16_t *>(row + o) = 0;
    }
}

// `slabs` threads walk a chunk, 8 columns each, kAhead rows in flight and as many on
// their way.  WAVES: whole waves share a chunk, so that its places are scalars.
template <typename T, typename D, bool WAVES> __global__ void __launch_bounds__(256) sum_kernel(SumArgs a)
{
    constexpr int kAhead = sizeof(T) == 2 ? 8 : 4;
    if (a.block + blockIdx.x >= a.blocks) {
        if (blockIdx.y == 0) clear_rows(a, a.block + blockIdx.x - a.blocks);
        return;
    }
    int sub = threadIdx.x / a.slabs;
    if constexpr (WAVES) sub = __builtin_amdgcn_readfirstlane(sub);
    const int t = threadIdx.x % a.slabs;
    const int64_t chunk = (a.block + blockIdx.x) * (256 / a.slabs) + sub, total = *a.count;
    const int64_t k0 = chunk * a.chunk, k1 = k0 + a.chunk < total ? k0 + a.chunk : total;
    if (k0 >= k1) return;
    const int32_t *ids = a.id + k0, *rows = a.row + k0;
    const int n = static_cast<int>(k1 - k0);
    // lane k of each wave: the k-th place's row and id, lane n: the id behind the chunk, the
    // one ahead of it
    const int lane = threadIdx.x & 63;
    int32_t lane_id = -1, lane_row = 0, ahead = -1;
    if (WAVES) {
        if (lane <= n && k0 + lane < total) lane_id = ids[lane];
        if (lane < n) lane_row = rows[lane];
        if (k0 > 0) ahead = ids[-1];
    } else if (k0 > 0) {
        ahead = ids[-1];
    }
    auto id_of = [&](int k) -> int32_t {   // k <= n; -1 past the last place
        if constexpr (WAVES) return __builtin_amdgcn_readlane(lane_id, k);
        return k0 + k < total ? ids[k] : -1;
    };
    auto row_of = [&](int k) -> int64_t {
        if constexpr (WAVES) return __builtin_amdgcn_readlane(lane_row, k);
        return rows[k];
    };
    const bool entered = ahead == id_of(0);
    for (int64_t c = 8 * (t + static_cast<int64_t>(blockIdx.y) * a.slabs); c < a.d;
         c += 8 * static_cast<int64_t>(a.slabs) * gridDim.y) {
        Raw8<T> v[2][kAhead];
        auto fetch = [&](int k, Raw8<T> *to) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                to[j].load(static_cast<const T *>(a.dy) + row_of(k + j < n ? k + j : n - 1) * a.gs, c, a.d, a.vec_in);
        };
        f8v sum = {0, 0, 0, 0, 0, 0, 0, 0};
        bool inside = entered;   // in the run that enters the chunk
        auto add = [&](int k, const Raw8<T> *from) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (k + j >= n) break;
                sum += __builtin_convertvector(from[j].v, f8v);
                const int32_t id = id_of(k + j);
                const bool last = k + j + 1 == n, ends = id_of(k + j + 1) != id;
                if (!ends && !last) continue;
                if (inside)
                    *partial(a, chunk, 0, c) = sum;
                else if (ends)
                    put<D>(a, id, c, sum);
                else
                    *partial(a, chunk, 1, c) = sum;
                inside = false;
                sum = f8v{0, 0, 0, 0, 0, 0, 0, 0};
            }
        };
        fetch(0, v[0]);
        for (int k = 0; k < n; k += 2 * kAhead) {
            if (k + kAhead < n) fetch(k + kAhead, v[1]);
            add(k, v[0]);
            if (k + 2 * kAhead < n) fetch(k + 2 * kAhead, v[0]);
            add(k + kAhead, v[1]);
        }
    }
}

// Runs that leave the chunk they start in: its partial sum, and those of the chunks
// that they enter, shared among four waves and added in order
template <typename D> __global__ void __launch_bounds__(256) join_kernel(SumArgs a)
{
    __shared__ f8v s[4][64];
    const int64_t chunk = a.block + blockIdx.x, total = *a.count;
    const int64_t k0 = chunk * a.chunk, k1 = k0 + a.chunk;
    if (k1 >= total) return;
    const int32_t id = a.id[k1 - 1];
    const int64_t order = order_of(id, a.bits, a.range);
    if (a.id[k1] != id || a.first[order] < k0) return;
    const int64_t last = (a.first[order + 1] - 1) / a.chunk, many = last - chunk;   // chunks that it enters
    const int lane = threadIdx.x & 63, wv = wave();
    const int64_t share = (many + 3) / 4;
    const int64_t q0 = chunk + 1 + wv * share, q1 = q0 + share < last + 1 ? q0 + share : last + 1;
    for (int64_t c0 = 512 * static_cast<int64_t>(blockIdx.y); c0 < a.d; c0 += 512 * static_cast<int64_t>(gridDim.y)) {
        const int64_t c = c0 + 8 * lane;
        f8v sum = {0, 0, 0, 0, 0, 0, 0, 0};
        if (c < a.d) {
            if (wv == 0) sum = *partial(a, chunk, 1, c);
            for (int64_t q = q0; q < q1; q += 4) {
                f8v v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = *partial(a, q + k < q1 ? q + k : q1 - 1, 0, c);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (q + k < q1) sum += v[k];
            }
        }
        s[wv][lane] = sum;
        __syncthreads();
        if (wv == 0 && c < a.d) put<D>(a, id, c, ((sum + s[1][lane]) + s[2][lane]) + s[3][lane]);
        __syncthreads();
    }
}

int slabs_of(int64_t d)
{
    int s = 1;
    while (s < 256 && s * 8 < d) s *= 2;
    return s;
}

// whether rows of d elements, `stride` apart, can be moved eight elements at once
bool whole8(const void *p, int64_t d, int64_t stride, int size)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && d % 8 == 0 && (stride * size) % 16 == 0;
}

template <typename T, typename D>
hipError_t sums(SumArgs a, const EmbedGeom &g, hipStream_t s)
{
    const unsigned cols = static_cast<unsigned>(std::min<int64_t>((a.d + 8 * a.slabs - 1) / (8 * a.slabs), 64));
    const int per = 256 / a.slabs;
    a.blocks = (g.chunks + per - 1) / per;
    const int64_t clearing = a.add ? 0 : (a.vocab + 4 * kClear - 1) / (4 * kClear);
    hipError_t e = launch_sliced(a.blocks + clearing, 256, [&](int64_t first, unsigned blocks) {
        a.block = first;
        if (a.slabs >= 64) sum_kernel<T, D, true><<<dim3(blocks, cols), dim3(256), 0, s>>>(a);
        else sum_kernel<T, D, false><<<dim3(blocks, cols), dim3(256), 0, s>>>(a);
    });
    if (e != hipSuccess || g.chunks < 2) return e;
    return launch_sliced(g.chunks - 1, 256, [&](int64_t first, unsigned blocks) {
        a.block = first;
        join_kernel<D><<<dim3(blocks, static_cast<unsigned>(std::min<int64_t>((a.d + 511) / 512, 64))), dim3(256), 0, s>>>(a);
    });
}

}  // namespace

EmbedGeom embed_geometry(int64_t n, int64_t vocab, int64_t d)
{
    EmbedGeom g{};
    // a workgroup for each of the 256 CUs, or for 16 ids where there are few
    while (g.bits < 8 && (int64_t(16) << g.bits) < vocab) ++g.bits;
    while ((int64_t(kMaxRange) << g.bits) < vocab) ++g.bits;
    g.range = static_cast<int>((vocab + (int64_t(1) << g.bits) - 1) >> g.bits);
    g.chunk = n <= 8192 ? 8 : n <= 16384 ? 16 : kMaxChunk;
    g.chunks = (n + g.chunk - 1) / g.chunk;
    size_t off = kHeader;
    g.off_count = off; off += 256;
    g.off_first = off; off = align256(off + ((static_cast<size_t>(g.range) << g.bits) + 1) * 4);
    g.off_row = off;   off = align256(off + static_cast<size_t>(n) * 4);
    g.off_id = off;    off = align256(off + static_cast<size_t>(n) * 4);
    g.off_part = off;
    // (fewer ids, in shorter chunks, may have more of them: room for these too)
    const int64_t room = std::max(g.chunks, std::min<int64_t>((n + 7) / 8, 1024));
    off = align256(off + static_cast<size_t>(room) * 2 * ((d + 7) / 8 * 8) * 4);
    g.bytes = off;
    return g;
}

hipError_t launch_embed_fwd(const void *ids, bool wide_ids, const void *W, void *y, int64_t n, int64_t vocab,
                            int64_t d, int64_t w_stride, float scale, int dtype, hipStream_t s)
{
    const int size = dtype == MGS_BF16 ? 2 : 4;
    LookupArgs a{ids, W, y, 0, n, vocab, d, w_stride, slabs_of(d), scale, wide_ids,
                 whole8(W, d, w_stride, size) && whole8(y, d, d, size)};
    const int per = 256 / a.slabs * kRows;
    return launch_sliced((n + per - 1) / per, 256, [&](int64_t first, unsigned blocks) {
        a.first = first;
        if (dtype == MGS_BF16) lookup_kernel<__bf16><<<dim3(blocks), dim3(256), 0, s>>>(a);
        else lookup_kernel<float><<<dim3(blocks), dim3(256), 0, s>>>(a);
    });
}

hipError_t launch_embed_bwd(const EmbedGeom &g, const void *ids, bool wide_ids, const void *dy, void *dW, int64_t n,
                            int64_t vocab, int64_t d, int64_t dy_stride, float scale, bool accumulate, int dtype,
                            int dw_dtype, void *ws, hipStream_t s)
{
    char *w = static_cast<char *>(ws);
    const int out = dw_dtype == MGS_BF16 ? 2 : 4, size = dtype == MGS_BF16 ? 2 : 4;
    SortArgs a{};
    a.ids = ids;
    a.n = n;
    a.vocab = vocab;
    a.d = d;
    a.bits = g.bits;
    a.range = g.range;
    a.count = reinterpret_cast<int64_t *>(w + g.off_count);
    a.first = reinterpret_cast<int32_t *>(w + g.off_first);
    a.row = reinterpret_cast<int32_t *>(w + g.off_row);
    a.id = reinterpret_cast<int32_t *>(w + g.off_id);
    const hipError_t e = launch_sliced(int64_t(1) << g.bits, 64 * kSortWaves, [&](int64_t first, unsigned blocks) {
        a.block = first;
        if (wide_ids) sort_kernel<uint64_t><<<dim3(blocks), dim3(64 * kSortWaves), 0, s>>>(a);
        else sort_kernel<uint32_t><<<dim3(blocks), dim3(64 * kSortWaves), 0, s>>>(a);
    });
    if (e != hipSuccess) return e;
    SumArgs b{};
    b.count = a.count;
    b.first = a.first;
    b.row = a.row;
    b.id = a.id;
    b.part = reinterpret_cast<float *>(w + g.off_part);
    b.dy = dy;
    b.dW = dW;
    b.d = d;
    b.vocab = vocab;
    b.row_bytes = d * out;
    b.gs = dy_stride;
    b.bits = g.bits;
    b.range = g.range;
    b.slabs = slabs_of(d);
    b.chunk = g.chunk;
    b.scale = scale;
    b.add = accumulate;
    b.vec_in = whole8(dy, d, dy_stride, size);
    b.vec_out = whole8(dW, d, d, out);
    if (dtype == MGS_BF16)
        return dw_dtype == MGS_BF16 ? sums<__bf16, __bf16>(b, g, s) : sums<__bf16, float>(b, g, s);
    return dw_dtype == MGS_BF16 ? sums<float, __bf16>(b, g, s) : sums<float, float>(b, g, s);
}

}  // namespace mgs
