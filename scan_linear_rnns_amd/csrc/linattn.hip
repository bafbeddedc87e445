// linattn.hip -- linear attention with a decay for each head (gfx950).
//
//     S_t = a_t S_{t-1} + v_t k_t^T,   o_t = s S_t q_t,   a_t = exp(g_t),
// S (dv x dk) per sequence and head.  Within a chunk of C = 64 steps entered
// with state S, and G_i the sum of the chunk's g up to step i,
//     o_i = s [ e^{G_i} S q_i + sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j ],
//     S  <- e^{G_C} S + sum_j e^{G_C - G_j} v_j k_j^T:
// matrix products over the chunk.  All exponents are differences of sums of
// the same chunk, kept in base 2 as two floats (a double rounded to head and
// tail), so a difference is good to 2^-24 of itself however large the sums that it
// comes of, and e^{-inf} (a cleared state) is an exact zero.
//
// The three gradients are the same walk with other operands.  With do in the
// query's place, v in the key's and k in the value's, the walk's output is dq
// (its state is S transposed).  Backwards in time, with each step's decay
// applied one step later, (k; q, do) gives dv from the state
// R_t = a_{t+1} D_{t+1} (D = dL/dS) and (v; do, q) gives dk from R transposed.
// One kernel serves all four.
//
// Along the steps a sequence is cut into segments when there are too few
// (sequence, head) pairs to fill the chip: a first pass forms each segment's
// own contribution to the state, a second chains them (elementwise), and the
// walks start from the chained states.
//
// The gradient of g: with x_t = q_t . dq_t and y_t = k_t . dk_t, scaling all
// decays from step t on shows
//     dg_t = sum_{s=t}^{e} (x_s - y_s) + <R_e, S_e>
// for any e >= t.  e is the step ahead of the next one whose decay is zero, where
// <R_e, S_e> = dg_{e+1} = 0, or else the end of t's segment (at most 512 steps):
// rounding in the sum grows with its length, and nothing of what follows a
// cleared state reaches the steps before it.
//
// MFMA layout: lane l supplies row (or column) l % 16 of an operand; its
// elements of a 16-wide reduction block are 4 (l / 16) .. + 3, and register r
// of a result is row 4 (l / 16) + r, column l % 16.  A result tile is thus an
// operand of the next product as it stands.  bf16 takes two blocks per
// v_mfma_f32_16x16x32_bf16, fp32 four v_mfma_f32_16x16x4f32 per block.
// Where an fp32 value (a decayed score, a state, a weighted value) meets bf16
// inputs it is split into three bf16 terms, head, middle and tail, which hold
// its 24 bits: the states and dg keep fp32 accuracy.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.hpp"
#include "layers.hpp"

namespace mgs {
namespace {

constexpr int kC = kAttnChunk;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eTail = static_cast<float>(1.44269504088896340736 - static_cast<double>(kLog2e));

typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f8v __attribute__((ext_vector_type(8), aligned(16)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));

template <typename T> struct Num;

template <> struct Num<float> {
    using Frag = f4v;                    // 4 elements of a reduction block
    static constexpr int NS = 1;         // terms an fp32 value is split into
    static constexpr int PADQ = 4, PADK = 4, PADV = 8;
    using Vec8 = f8v;
};
template <> struct Num<__bf16> {
    using Frag = bf4;
    static constexpr int NS = 3;
    static constexpr int PADQ = 4, PADK = 8, PADV = 16;
    using Vec8 = bf8;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return static_cast<float>(x); }

// reduction blocks 2m, 2m + 1 of D += A B
__device__ __forceinline__ f4v mma2(f4v a0, f4v a1, f4v b0, f4v b1, f4v c)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[j], b0[j], c, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[j], b1[j], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ f4v mma2(bf4 a0, bf4 a1, bf4 b0, bf4 b1, f4v c)
{
    const bf8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    const bf8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// an fp32 fragment as fragments of T that sum to it, or to its first 16 bits (two of bf16)
__device__ __forceinline__ void split(f4v x, f4v (&out)[1]) { out[0] = x; }

// two floats rounded to bf16, the first in the low half
__device__ __forceinline__ uint32_t pack(float x, float y)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2v{x, y}), bf2));
}

template <int N> __device__ __forceinline__ void split(f4v x, bf4 (&out)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u2v p = {pack(x[0], x[1]), pack(x[2], x[3])};
        // (opaque: the compiler would round each element again for its remainder)
        asm volatile("" : "+v"(p));
        out[i] = __builtin_bit_cast(bf4, p);
        if (i + 1 < N)
            x -= f4v{__uint_as_float(p[0] << 16), __uint_as_float(p[0] & 0xffff0000u), __uint_as_float(p[1] << 16),
                     __uint_as_float(p[1] & 0xffff0000u)};
    }
}

// 4 contiguous elements in LDS (aligned to the fragment)
template <typename T> __device__ __forceinline__ typename Num<T>::Frag frag(const T *p)
{
    return *reinterpret_cast<const typename Num<T>::Frag *>(p);
}

// A tile of 64 rows of D elements in LDS, LD apart, read as fragments of rows (li
// = row, block b of 16 columns) and of columns (rows row0 + 4 lq + r of column
// 16 t + li).  For 16-bit elements a column fragment is one transposing read:
// each of 16 lanes addresses 4 elements of a row, and lane i gets column i of the
// 4 x 16 block.  16 lanes read 128 bytes in one go if they touch each of 32 banks
// once: of bf16 rows LD = 4 (mod 64) elements apart for rows, 16 for columns; 8
// costs both a second go, more seldom for columns.  q is read by rows, v by
// columns, k by both, mostly columns.
template <typename T, int D, int PAD> struct Tile {
    using N = Num<T>;
    static constexpr int LD = D + PAD, SIZE = kC * LD;
    static __device__ __forceinline__ void store8(T *m, int r, int c, typename N::Vec8 x)
    {
        if constexpr (LD % 8 == 0) {
            *reinterpret_cast<typename N::Vec8 *>(m + r * LD + c) = x;
        } else {
            *reinterpret_cast<typename N::Frag *>(m + r * LD + c) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
            *reinterpret_cast<typename N::Frag *>(m + r * LD + c + 4) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
        }
    }
    static __device__ __forceinline__ typename N::Frag row(const T *m, int row0, int b, int li, int lq)
    {
        return frag(m + (row0 + li) * LD + 16 * b + 4 * lq);
    }
    static __device__ __forceinline__ typename N::Frag col(const T *m, int row0, int t, int li, int lq)
    {
        if constexpr (sizeof(T) == 4) {
            const T *p = m + (row0 + 4 * lq) * LD + 16 * t + li;
            return f4v{p[0], p[LD], p[2 * LD], p[3 * LD]};
        } else {
            typedef __attribute__((address_space(3))) s4v *lds_ptr;
            const T *p = m + (row0 + 4 * lq + (li >> 2)) * LD + 16 * t + 4 * (li & 3);
            return __builtin_bit_cast(typename N::Frag, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p)));
        }
    }
};

// ------------------------------------------------------------------- walks

struct Operand {
    const void *p;           // element (b, t, h, c) at b sb + t st + (h / div) sh + c
    int64_t sb, st, sh;
    int div, cols;
};

struct Role {
    Operand q, k, v;
    Operand dot;             // dots of the output rows with this, or p == NULL
    void *out;               // (B,T,H,v.cols) dense: T, or fp32 with out_f32
    float *xdot;             // (B,H,T)
    const float *state;      // entering states, or NULL (zeros): + bh st_bh + seg st_seg
    float *final;            // state after the walk (+ bh * sc-by-sk elements), or NULL
    float *local;            // state-only pass: segment contributions, like `state`
    int64_t st_bh, st_seg;
    int sc, sk;              // element strides of the state's output column and reduction index
    float intra, inter, src; // factors of the chunk's own part, the state's part, the sources
    int rev, out_f32;
};

struct WalkArgs {
    Role role[3];
    const float *g;
    int64_t gb, gt, gh;
    const int32_t *lengths;
    float *dec;              // state-only pass: decay over each segment (bh, seg), by the forward role
    uint32_t items;          // (b, h, segment) triples
    uint32_t first;          // this launch's first workgroup
    int nRoles, T, H, nC, nSeg, segLen, vec;
};

// Cuts a workgroup-uniform value off from how it was computed.  Without it the
// compiler keeps whole argument structures in scalar registers through the walk,
// and the lane masks and products made from them, and spills.
__device__ __forceinline__ int keep(int x)
{
    x = __builtin_amdgcn_readfirstlane(x);
    asm volatile("" : "+s"(x));
    return x;
}
__device__ __forceinline__ float keep(float x) { return __int_as_float(keep(__float_as_int(x))); }
__device__ __forceinline__ int64_t keep(int64_t x)
{
    const int lo = keep(static_cast<int>(x)), hi = keep(static_cast<int>(x >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo));
}
// addresses: plain numbers, turned into global pointers where they are used
__device__ __forceinline__ int64_t keep(const void *p) { return keep(static_cast<int64_t>(reinterpret_cast<uintptr_t>(p))); }

template <typename V> using Global = __attribute__((address_space(1))) V;

// Buffer accesses, at a workgroup-uniform address plus a lane offset: a lane
// whose offset is kNowhere reads zeros and writes nothing, with no branch, so
// the number of accesses in flight is known and waiting for one does not mean
// waiting for all (loads and stores share a counter).
constexpr uint32_t kReach = 1u << 30, kNowhere = 1u << 31;

struct Buffer {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit Buffer(int64_t base)
        : r(__builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(base), 0, kReach, 0x00027000))
    {
    }
    template <typename V> __device__ __forceinline__ V load(uint32_t off) const
    {
        if constexpr (sizeof(V) == 32) {
            struct { u4v a, b; } x{__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0),
                                   __builtin_amdgcn_raw_buffer_load_b128(r, off, 16, 0)};
            return __builtin_bit_cast(V, x);
        } else if constexpr (sizeof(V) == 16) {
            return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
        } else if constexpr (sizeof(V) == 8) {
            return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
        } else {
            static_assert(sizeof(V) == 4, "size");
            return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
        }
    }
    template <typename V> __device__ __forceinline__ void store(uint32_t off, V v) const
    {
        if constexpr (sizeof(V) == 16) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4v, v), r, off, 0, 0);
        } else {
            static_assert(sizeof(V) == 8, "size");
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2v, v), r, off, 0, 0);
        }
    }
};

// Where a chunk lies: rows [lo, hi) of it are live (inside the sequence and its
// length), row r is step tb + r, or tb + 63 - r backwards (tb may then lie
// ahead of the sequence: only live rows are addressed).
struct Chunk {
    int64_t tb;
    int lo, hi, rows;
};

__device__ __forceinline__ Chunk chunk_at(int ch, int T, int len, int rev)
{
    const int t0 = ch * kC, t1 = min(T, t0 + kC);
    Chunk c;
    c.rows = t1 - t0;
    c.tb = rev ? t1 - kC : t0;
    c.lo = rev ? min(c.rows, max(0, t1 - len)) : 0;
    c.hi = rev ? c.rows : max(0, min(c.rows, len - t0));
    return c;
}

// One 64-row tile on its way from global memory to LDS: DIM columns, 8 per
// thread and turn.  Rows that are not live are zeros and are not read.  A wide
// access is a workgroup-uniform chunk address plus a 32-bit lane offset that
// stays the same from chunk to chunk.
template <typename T, int DIM, int THREADS, bool VEC> struct Stage {
    static constexpr int PER = kC * DIM / 8 / THREADS;
    static constexpr int TURN = THREADS / (DIM / 8);   // rows per turn
    using Vec8 = typename Num<T>::Vec8;
    Vec8 x[PER];
    int64_t base;      // address of (b, 0, h, 0)
    int64_t st;        // bytes from step to step
    uint32_t off;      // bytes from the chunk's first step, first turn
    uint32_t turn;     // bytes from turn to turn
    int vrow;          // row of the first turn; of columns past the end, out of any chunk
    int cols, rev;

    __device__ __forceinline__ void init(const Operand &o, int64_t b, int h, int rev_)
    {
        base = keep(static_cast<const T *>(o.p) + b * o.sb + (h / o.div) * o.sh);
        st = keep(o.st * static_cast<int64_t>(sizeof(T)));
        cols = keep(o.cols);
        rev = rev_;
        turn = static_cast<uint32_t>(st) * static_cast<uint32_t>(TURN);
        if (rev) turn = 0u - turn;
        const int r = row(0);
        vrow = col() < cols ? r : kC;
        off = (rev ? kC - 1 - r : r) * static_cast<uint32_t>(st) + static_cast<uint32_t>(col() * sizeof(T));
    }
    __device__ __forceinline__ int row(int i) const { return threadIdx.x / (DIM / 8) + TURN * i; }
    __device__ __forceinline__ int col() const { return threadIdx.x % (DIM / 8) * 8; }

    __device__ __forceinline__ void load(const Chunk &ck)
    {
        if constexpr (VEC) {
            const Buffer p(base + ck.tb * st);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const bool live = static_cast<uint32_t>(vrow + TURN * i - ck.lo) < static_cast<uint32_t>(ck.hi - ck.lo);
                x[i] = p.template load<Vec8>(live ? off + i * turn : kNowhere);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                x[i] = Vec8(0);
                const int r = row(i);
                const Global<const T> *p = reinterpret_cast<const Global<const T> *>(base + (ck.tb + (rev ? kC - 1 - r : r)) * st);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r >= ck.lo && r < ck.hi && col() + j < cols) x[i][j] = p[col() + j];
            }
        }
    }
    template <typename Tile> __device__ __forceinline__ void store(T *lds) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) Tile::store8(lds, row(i), col(), x[i]);
    }
};

// The chunk's decay sums in base 2, by one wave, lane = row.  Forward G_r
// includes row r's own decay, backward (rows in reverse order) it does not.
// A decay below 2^-20000 clears the state as -inf does (the clamp keeps the
// differences finite); NaN passes the comparison and propagates.
struct Decays {
    float hi[kC], lo[kC];    // G
    float src[kC];           // factor of source j: e^{total - G_j}, times the role's
    float total;             // e^{total}
    float log2_total;
};

// x of the lane `ctrl` (a DPP lane shift) points at, 0 where there is none
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp(double x)
{
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(x), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(x), CTRL, ROWS, 0xf, false);
    return __hiloint2double(hi, lo);
}

__device__ __forceinline__ void chunk_decays(float g, float src, int rev, Decays &d)
{
    const int r = threadIdx.x & 63;
    double x = static_cast<double>(g) * 1.4426950408889634074;
    if (x < -20000.0) x = -20000.0;
    double G = x;   // inclusive sums: within 16 lanes, then over the rows of 16
    G += dpp<0x111, 0xf>(G);
    G += dpp<0x112, 0xf>(G);
    G += dpp<0x114, 0xf>(G);
    G += dpp<0x118, 0xf>(G);
    G += dpp<0x142, 0xa>(G);
    G += dpp<0x143, 0xc>(G);
    const double total = __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(G), 63),
                                          __builtin_amdgcn_readlane(__double2loint(G), 63));
    if (rev) G = dpp<0x138, 0xf>(G);   // one lane up: row r without its own
    const float hi = static_cast<float>(G);
    d.hi[r] = hi;
    d.lo[r] = static_cast<float>(G - static_cast<double>(hi));
    d.src[r] = src * __builtin_amdgcn_exp2f(static_cast<float>(total - G));
    if (r == 0) {
        d.total = __builtin_amdgcn_exp2f(static_cast<float>(total));
        d.log2_total = static_cast<float>(total);
    }
}

// Workgroup barrier that waits for this wave's LDS operations only: loads from
// global memory (the next chunk's) stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Zeros in place of the non-finite elements of a wave's value fragments (rows
// 16 jb + 4 lq + r, column li), and NaN in the output tiles (row 16 i + li,
// columns 4 lq + r) from their rows on.
template <typename T>
__device__ __forceinline__ void drop_non_finite(typename Num<T>::Frag (&vf)[4], f4v (&O)[4], int li, int lq)
{
    int first = kC;   // of column li
#pragma unroll
    for (int jb = 3; jb >= 0; --jb)
#pragma unroll
        for (int r = 3; r >= 0; --r)
            if (!isfinite(to_f32(vf[jb][r]))) {
                first = 16 * jb + 4 * lq + r;
                vf[jb][r] = static_cast<T>(0.0f);
            }
    first = min(first, __shfl_xor(first, 16, 64));
    first = min(first, __shfl_xor(first, 32, 64));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int f = __shfl(first, 4 * lq + r, 64);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (16 * i + li >= f) O[i][r] = __builtin_nanf("");
    }
}

// The ten 16 x 16 score tiles on or below the diagonal, tile = 4 i + j, one per
// nibble, and the two above it that are read as zeros.
constexpr uint64_t kScoreTiles = 0xB1FEDCA98540ull;

// KD, VD: the reduction dimension and the output columns, padded.  Each of the
// VD / 16 waves owns 16 output columns: of the state it keeps S^T tiles
// (reduction index x column) in accumulators, and it forms the same columns of
// the output, transposed, so that a lane holds 4 neighbouring columns of a row.
// The scores are formed once per workgroup and shared through LDS.  (With 32
// columns a wave, half as many waves read LDS half as often, but their registers
// leave two waves a SIMD, and waits and vector arithmetic then show.)
//
// What bounds it: nothing alone.  Measured on B=4, T=4096, 16 heads of 128 x 128,
// bf16 (67 MB a tensor; a large copy runs at 4.7 TB/s): STATE 47 us (169 MB of k,
// v and states, 3.6 TB/s), OUT 88 us (306 MB, 3.5 TB/s; 75 us, 4.1 TB/s, on one
// sequence of 32768 steps x 8 heads), the two DOTS roles 233 us (726 MB, 3.1
// TB/s; matrix cores busy 27% of the time, vector ALUs 46%).  A chunk is a chain
// of LDS tile, products, splits into bf16 terms and two barriers; two workgroups
// a CU fill each other's waits in part.  (At 128 x 128 in bf16 2 to 4 vector
// registers spill in OUT and DOTS.)  fp32, B=16, T=1024, one head of 64 x 64 (256
// walks of one chunk a role): STATE 8, OUT 10, the three gradients in one launch
// 19 us: the latency of a launch and of one chunk's loads, barriers and products
// (an fp32 product of 64 x 64 x 64 keeps a CU's matrix cores 1 us), not the 4 MB a
// tensor.  A chunk past a sequence's length reads nothing, but is walked as any
// other.
// MODE: STATE, the walk from a zero state without outputs; OUT, outputs rounded
// to T; DOTS, outputs in T or fp32 (partials of shared heads), and, of the roles
// that ask for them, the dots of their rows for dg.
// bf16 terms: the weighted values of the state's update take three, so a state is
// fp32 whether it leaves the kernel or not, and what else a call asks for does not
// change its outputs (two where only outputs come of it would save 2 to 3%).
// States and scores on their way into an output take three in DOTS, whose outputs
// make dg, and two in OUT, whose outputs are rounded to bf16: 2^-18 of each term
// ahead of 2^-9 of the sum (three: prompts and training 3 to 6% longer).
enum { STATE, OUT, DOTS };

// Waves a SIMD that the registers are cut for: as many as LDS lets in, or one more
// (bf16 64 x 64 with dots gets two, fp32 of 128 by 64 one).
template <typename T> constexpr int walk_waves(int KD, int VD, int mode)
{
    if (sizeof(T) == 4) return (mode == STATE && KD + VD <= 192) || KD + VD == 128 ? 3 : 2;
    return VD == 128 ? 4 : mode == STATE ? 4 : KD == 64 ? 3 : 2;
}

template <typename T, int KD, int VD, int MODE, bool VEC>
__global__ void __launch_bounds__(4 * VD, walk_waves<T>(KD, VD, MODE)) walk_kernel(WalkArgs a)
{
    using N = Num<T>;
    using Frag = typename N::Frag;
    constexpr bool STATE_ONLY = MODE == STATE;
    constexpr int NS = N::NS;                                 // terms of the weighted values
    constexpr int NO = N::NS == 3 && MODE != DOTS ? 2 : N::NS;   // of states and scores
    constexpr int kThreads = 4 * VD, NW = VD / 16;
    constexpr int NKB = KD / 16;       // reduction blocks
    using TQ = Tile<T, KD, N::PADQ>;
    using TK = Tile<T, KD, N::PADK>;
    using TV = Tile<T, VD, sizeof(T) == 4 ? NW : N::PADV>;
    constexpr int LA = kC + 4;
    __shared__ __align__(16) T sQ[STATE_ONLY ? 8 : TQ::SIZE - N::PADQ];
    __shared__ __align__(16) T sK[TK::SIZE - N::PADK];
    __shared__ __align__(16) T sV[TV::SIZE];
    // fp32 scores take the place of q, which is done with by then, and the last rows
    // of q and k have no padding: 42 blocks of 1280 bytes at 64 x 64, so three
    // workgroups fit a CU (training B=16, T=1024, one head: 58.1 us, with two 62.2)
    constexpr bool OVER = sizeof(T) == 4 && !STATE_ONLY;
    static_assert(TQ::LD >= LA);
    __shared__ __align__(16) T sA_own[STATE_ONLY || OVER ? 8 : NO * kC * LA];
    T *const sA = OVER ? sQ : sA_own;
    __shared__ __align__(16) Decays sDecays[2];

    // the waves' partial dots of row r: in the 32 bytes after row r of the value tile
    auto partial = [&](int w, int r) -> float & { return reinterpret_cast<float *>(sV + r * TV::LD + VD)[w]; };

    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int li = lane & 15, lq = lane >> 4;
    // the roles of 8 neighbouring items run side by side, an item's on one XCD:
    // they read the same rows
    const uint32_t group = a.first + blockIdx.x, rest = group >> 3;
    const uint32_t item = (rest / a.nRoles) * 8 + (group & 7);
    if (item >= a.items) return;
    const Role &ro = a.role[rest % a.nRoles];
    const int seg = static_cast<int>(item % a.nSeg);
    const uint32_t bh = item / a.nSeg;
    const int64_t b = bh / a.H;
    const int h = static_cast<int>(bh % a.H);
    int len = a.T;
    if (a.lengths) len = max(0, min(a.T, a.lengths[b]));
    len = keep(len);
    const int c_lo = seg * a.segLen, chunks = min(a.nC, c_lo + a.segLen) - c_lo;
    const int rev = keep(ro.rev), cols = keep(ro.v.cols), kcols = keep(ro.k.cols);
    const int T_ = keep(a.T), H_ = keep(a.H);

    const int col0 = wv * 16;   // this wave's first column
    f4v S[NKB];
    const float *state = STATE_ONLY ? nullptr : ro.state;
    const int sc = keep(ro.sc), sk = keep(ro.sk);
    if (state) {
        // all loads in flight at once: out-of-range elements read the last one and
        // are zeroed after
        state += static_cast<int64_t>(bh) * ro.st_bh + seg * ro.st_seg;
        const int c = col0 + li;
        const float *p = state + min(c, cols - 1) * sc;
        if (VEC && sk == 1) {
#pragma unroll
            for (int t = 0; t < NKB; ++t)
                S[t] = *reinterpret_cast<const f4v *>(p + min(16 * t + 4 * lq, kcols - 4));
        } else {
#pragma unroll
            for (int t = 0; t < NKB; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] = p[min(16 * t + 4 * lq + r, kcols - 1) * sk];
        }
        if (cols < VD || kcols < KD) {
#pragma unroll
            for (int t = 0; t < NKB; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[t][r] = col0 + li < cols && 16 * t + 4 * lq + r < kcols ? S[t][r] : 0.0f;
        }
    } else {
#pragma unroll
        for (int t = 0; t < NKB; ++t)
            S[t] = f4v{0, 0, 0, 0};
    }
    if constexpr (!STATE_ONLY && !OVER) {   // the tiles above the diagonal stay zero
        for (int i = tid; i < NO * kC * LA; i += kThreads) sA[i] = static_cast<T>(0.0f);
    }

    Stage<T, KD, kThreads, VEC> q, k;
    Stage<T, VD, kThreads, VEC> v;
    k.init(ro.k, b, h, rev);
    v.init(ro.v, b, h, rev);
    if constexpr (!STATE_ONLY) q.init(ro.q, b, h, rev);
    const int64_t gp = keep(a.g + b * a.gb + h * a.gh);
    const int64_t gt = keep(a.gt * 4);
    const float intra = keep(ro.intra), inter = keep(ro.inter), src_f = keep(ro.src);

    // rows of the output and of what they are dotted with: lane offsets of row li
    // (rows 16 i + li lie 16 i rows further on, or back), columns 4 lq
    const int out_f32 = keep(MODE == DOTS && ro.out_f32 ? 1 : 0);
    const int dots_on = keep(MODE == DOTS && ro.dot.p ? 1 : 0);
    const int o_size = out_f32 ? 4 : static_cast<int>(sizeof(T));
    const int64_t o_st = static_cast<int64_t>(H_) * cols * o_size, d_st = keep(ro.dot.st * static_cast<int64_t>(sizeof(T)));
    const int o_step = rev ? -16 : 16;
    const int64_t o_base = keep(static_cast<char *>(ro.out) + (b * T_ * H_ + h) * cols * o_size);
    const int64_t d_base = keep(static_cast<const T *>(ro.dot.p) + b * ro.dot.sb + (dots_on ? h / ro.dot.div : 0) * ro.dot.sh);
    const int finals = keep(ro.final ? 1 : 0);
    const int64_t xdot = keep(ro.xdot + static_cast<int64_t>(bh) * T_);
    // The rows of the next chunk travel while this one is worked on; its decay sums
    // are formed by the last wave, which has the fewest score tiles, meanwhile.
    float g = 0.0f;
    auto place = [&](int n) {
        Chunk ck = chunk_at(rev ? c_lo + chunks - 1 - n : c_lo + n, T_, len, rev);
        if (n >= chunks) ck.lo = ck.hi = 0;   // nothing to read
        return ck;
    };
    auto load_g = [&](int n) {
        const Chunk ck = place(n);
        g = 0.0f;
        if (lane >= ck.lo && lane < ck.hi)
            g = *reinterpret_cast<const Global<const float> *>(gp + (ck.tb + (rev ? kC - 1 - lane : lane)) * gt);
    };
    auto load = [&](int n) {
        const Chunk ck = place(n);
        k.load(ck);
        v.load(ck);
        if constexpr (!STATE_ONLY) q.load(ck);
    };
    const bool sums = wv == NW - 1;
    if (sums) load_g(0);
    load(0);
    if (sums) {
        chunk_decays(g, src_f, rev, sDecays[0]);
        load_g(1);
    }

    float seg_log2 = 0.0f;
    for (int n = 0; n < chunks; ++n) {
        // (opaque: addresses made of them are cheaper to form again than to keep)
        asm volatile("" : "+v"(li), "+v"(lq));
        [[maybe_unused]] const int orow = rev ? kC - 1 - li : li, c = col0 + 4 * lq;
        const Decays &sD = sDecays[n & 1];
        k.template store<TK>(sK);
        v.template store<TV>(sV);
        if constexpr (!STATE_ONLY) q.template store<TQ>(sQ);
        lds_barrier();
        const Chunk ck = place(n);

        if constexpr (STATE_ONLY) load(n + 1);
        if (sums) {
            chunk_decays(g, src_f, rev, sDecays[(n + 1) & 1]);
            load_g(n + 2);
        }

        if constexpr (!STATE_ONLY) {
            // scores: tile (i, j) with rows of q as columns, so that a lane holds
            // 4 neighbouring sources of one row
            [[maybe_unused]] f4v held[(12 + NW - 1) / NW];
#pragma unroll
            for (int it = 0; it < (10 + NW - 1) / NW; ++it) {
                const int slot = wv + NW * it;
                if (slot < 10) {
                    const int tile = static_cast<int>((kScoreTiles >> (4 * slot)) & 15);
                    const int i = tile >> 2, j = tile & 3;
                    f4v p = {0, 0, 0, 0};
#pragma unroll
                    for (int m = 0; m < NKB / 2; ++m)
                        p = mma2(TK::row(sK, 16 * j, 2 * m, li, lq), TK::row(sK, 16 * j, 2 * m + 1, li, lq),
                                 TQ::row(sQ, 16 * i, 2 * m, li, lq), TQ::row(sQ, 16 * i, 2 * m + 1, li, lq), p);
                    const int row = 16 * i + li, src = 16 * j + 4 * lq;
                    const float gh = sD.hi[row], gl = sD.lo[row];
                    const f4v sh = *reinterpret_cast<const f4v *>(&sD.hi[src]), sl = *reinterpret_cast<const f4v *>(&sD.lo[src]);
                    f4v w;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float e = intra * __builtin_amdgcn_exp2f((gh - sh[r]) + (gl - sl[r])) * p[r];
                        asm volatile("" : "+v"(e));   // (computed for every lane: a branch costs more)
                        w[r] = src + r <= row ? e : 0.0f;
                    }
                    if constexpr (OVER) {
                        held[it] = w;
                    } else {
                        Frag ws[NO];
                        split(w, ws);
#pragma unroll
                        for (int s = 0; s < NO; ++s)
                            *reinterpret_cast<Frag *>(&sA[s * kC * LA + row * LA + src]) = ws[s];
                    }
                }
            }
            // the state's part of the output (which needs no one's scores), then the
            // chunk's own
            f4v O[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) O[i] = f4v{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < NKB / 2; ++m) {
                Frag q0[4], q1[4], s0[NO], s1[NO];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q0[i] = TQ::row(sQ, 16 * i, 2 * m, li, lq);
                    q1[i] = TQ::row(sQ, 16 * i, 2 * m + 1, li, lq);
                }
                split(S[2 * m], s0);
                split(S[2 * m + 1], s1);
#pragma unroll
                for (int s = 0; s < NO; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[i] = mma2(s0[s], s1[s], q0[i], q1[i], O[i]);
            }
            load(n + 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = inter * __builtin_amdgcn_exp2f(sD.hi[16 * i + li]);
                O[i] *= w;
            }
            if constexpr (OVER) {
                lds_barrier();
#pragma unroll
                for (int it = 0; it < (12 + NW - 1) / NW; ++it) {
                    const int slot = wv + NW * it;
                    if (slot < 12) {   // the last two are the zeros above the diagonal that are read
                        const int tile = static_cast<int>((kScoreTiles >> (4 * slot)) & 15);
                        const int row = 16 * (tile >> 2) + li, src = 16 * (tile & 3) + 4 * lq;
                        *reinterpret_cast<f4v *>(&sA[row * LA + src]) = slot < 10 ? held[it] : f4v{0, 0, 0, 0};
                    }
                }
            }
            lds_barrier();
            Frag vf[4];
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) vf[jb] = TV::col(sV, 16 * jb, wv, li, lq);
            // A product with a zero weight would carry a non-finite value to rows ahead
            // of its own: such values are taken out, and from their row on their
            // column is NaN.  A product with zeros finds them.
            {
                f4v probe = {0, 0, 0, 0};
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int jb = 0; jb < 4; ++jb) probe += vf[jb] * 0.0f;
                } else {   // (by a matrix product with zeros)
                    const Frag z = __builtin_bit_cast(Frag, uint64_t(0));
                    probe = mma2(vf[0], vf[1], z, z, probe);
                    probe = mma2(vf[2], vf[3], z, z, probe);
                }
                if (__any((probe[0] + probe[1]) + (probe[2] + probe[3]) != 0.0f)) drop_non_finite<T>(vf, O, li, lq);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int s = 0; s < NO; ++s) {
                    Frag a0[4], a1[4];
#pragma unroll
                    for (int i = 2 * m; i < 4; ++i) {
                        const T *ar = &sA[s * kC * LA + (16 * i + li) * LA + 32 * m + 4 * lq];
                        a0[i] = frag(ar);
                        a1[i] = frag(ar + 16);
                    }
#pragma unroll
                    for (int i = 2 * m; i < 4; ++i) O[i] = mma2(vf[2 * m], vf[2 * m + 1], a0[i], a1[i], O[i]);
                }

            [[maybe_unused]] Frag dots[MODE == DOTS ? 4 : 1];
            if constexpr (MODE == DOTS) {
                [[maybe_unused]] const int64_t p = d_base + ck.tb * d_st;
                const Buffer buf(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * i + li;
                    const bool live = r >= ck.lo && r < ck.hi && dots_on;
                    if constexpr (VEC) {
                        const uint32_t at = (orow + o_step * i) * static_cast<uint32_t>(d_st) + c * static_cast<uint32_t>(sizeof(T));
                        dots[i] = buf.template load<Frag>(live && c < cols ? at : kNowhere);
                    } else {
                        const Global<const T> *x = reinterpret_cast<const Global<const T> *>(p + (orow + o_step * i) * d_st) + c;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            dots[i][e] = static_cast<T>(0.0f);
                            if (live && c + e < cols) dots[i][e] = x[e];
                        }
                    }
                }
            }
            // rows of the output (zeros past the sequence's length) and their dots
            if (ck.hi - ck.lo < kC) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (16 * i + li < ck.lo || 16 * i + li >= ck.hi) O[i] = f4v{0, 0, 0, 0};
            }
            const int64_t op = o_base + ck.tb * o_st;
            const Buffer out(op);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = orow + o_step * i;
                const f4v y = O[i];
                const Frag z = __builtin_convertvector(y, Frag);
                if constexpr (VEC) {
                    uint32_t at = static_cast<uint32_t>(rr) * static_cast<uint32_t>(o_st) + c * static_cast<uint32_t>(o_size);
                    if (16 * i + li >= ck.rows || c >= cols) at = kNowhere;
                    if (MODE == DOTS && out_f32) out.store(at, y);
                    else out.store(at, z);
                } else if (16 * i + li < ck.rows) {
                    const int64_t at = op + rr * o_st + c * o_size;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < cols) {
                            if (out_f32) reinterpret_cast<Global<float> *>(at)[e] = y[e];
                            else reinterpret_cast<Global<T> *>(at)[e] = z[e];
                        }
                }
            }
            if constexpr (MODE == DOTS) {
                // columns past the end have zero dots, rows that are not live zero outputs
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f4v x = __builtin_convertvector(dots[i], f4v) * O[i];
                    float dot = (x[0] + x[1]) + (x[2] + x[3]);
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (lq == 0) partial(wv, 16 * i + li) = dot;
                }
            }
        }

        // S <- e^{total} S + sum over the chunk of weighted sources (which nothing reads
        // after the last chunk, unless the state leaves the kernel)
        if (STATE_ONLY || n + 1 < chunks || finals) {
            const float dec = sD.total;
#pragma unroll
            for (int t = 0; t < NKB; ++t) S[t] *= dec;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                Frag v0[NS], v1[NS];
                const Frag x0 = TV::col(sV, 32 * m, wv, li, lq), x1 = TV::col(sV, 32 * m + 16, wv, li, lq);
                const f4v w0 = *reinterpret_cast<const f4v *>(&sD.src[32 * m + 4 * lq]);
                const f4v w1 = *reinterpret_cast<const f4v *>(&sD.src[32 * m + 16 + 4 * lq]);
#pragma unroll
                for (int t0 = 0; t0 < NKB; t0 += 4) {
                    Frag k0[4], k1[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        k0[t] = TK::col(sK, 32 * m, t0 + t, li, lq);
                        k1[t] = TK::col(sK, 32 * m + 16, t0 + t, li, lq);
                    }
                    if (t0 == 0) {
                        split(__builtin_convertvector(x0, f4v) * w0, v0);
                        split(__builtin_convertvector(x1, f4v) * w1, v1);
                    }
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int t = 0; t < 4; ++t) S[t0 + t] = mma2(k0[t], k1[t], v0[s], v1[s], S[t0 + t]);
                }
            }
        }
        if constexpr (STATE_ONLY) seg_log2 += sD.log2_total;
        lds_barrier();
        if constexpr (MODE == DOTS) {
            if (dots_on && tid < ck.rows) {
                float x = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) x += partial(w, tid);
                reinterpret_cast<Global<float> *>(xdot)[ck.tb + (rev ? kC - 1 - tid : tid)] = x;
            }
        }
    }

    float *fin = STATE_ONLY ? ro.local : ro.final;
    if (fin) {
        fin += static_cast<int64_t>(bh) * ro.st_bh + (STATE_ONLY ? seg * ro.st_seg : 0);
        const int c = col0 + li;
        float *p = fin + c * sc;
        if (VEC && sk == 1) {
#pragma unroll
            for (int t = 0; t < NKB; ++t)
                if (c < cols && 16 * t + 4 * lq < kcols) *reinterpret_cast<f4v *>(p + 16 * t + 4 * lq) = S[t];
        } else {
#pragma unroll
            for (int t = 0; t < NKB; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (c < cols && 16 * t + 4 * lq + r < kcols) p[(16 * t + 4 * lq + r) * sk] = S[t][r];
        }
    }
    if (STATE_ONLY && !rev && tid == 0) a.dec[static_cast<int64_t>(bh) * a.nSeg + seg] = __builtin_amdgcn_exp2f(seg_log2);
}

// ---------------------------------------------------- chaining the segments
// Forward (blockIdx.y == 0): slot n of S gets the state entering segment n,
// slot nSeg and ST the last one.  Backward: slot n of R gets the state entering
// segment n from the future, dS0 the one left at the start.  One thread per
// state element; 8 segments of loads in flight.  Bound by its traffic: 512
// segments of 128 x 128 states, 70 MB, in 13 to 15 us (5 TB/s); both directions
// 25 us.
struct ChainArgs {
    float *S, *R;
    const float *dec, *S0, *dST;
    float *ST, *dS0;
    int64_t BH, first;       // first: this launch's first workgroup
    int nSeg, E;             // E = dv dk
};

__global__ void __launch_bounds__(256) chain_kernel(ChainArgs a)
{
    const int64_t at = (a.first + blockIdx.x) * 256 + threadIdx.x;
    if (at >= a.BH * a.E) return;
    const int64_t bh = at / a.E;
    const int e = static_cast<int>(at - bh * a.E);
    const bool rev = blockIdx.y != 0;
    const int stride = rev ? -a.E : a.E;
    const float *first = rev ? a.dST : a.S0;
    float s = first ? first[at] : 0.0f;
    float *p = rev ? a.R + (bh * a.nSeg + a.nSeg - 1) * a.E + e : a.S + bh * (a.nSeg + 1) * a.E + e;
    const float *dec = a.dec + bh * a.nSeg + (rev ? a.nSeg - 1 : 0);
    const int dd = rev ? -1 : 1;
    for (int n0 = 0; n0 < a.nSeg; n0 += 8) {
        float u[8], w[8];
        const int m = min(8, a.nSeg - n0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = min(i, m - 1);   // past the end: the last one again, unused
            u[i] = p[static_cast<int64_t>(n0 + j) * stride];
            w[i] = dec[(n0 + j) * dd];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < m) {
                p[static_cast<int64_t>(n0 + i) * stride] = s;
                s = __builtin_fmaf(w[i], s, u[i]);
            }
    }
    if (!rev) {
        a.S[(bh * (a.nSeg + 1) + a.nSeg) * a.E + e] = s;
        if (a.ST) a.ST[at] = s;
    } else if (a.dS0) {
        a.dS0[at] = s;
    }
}

// --------------------------------------------------------------- dg and sums
// dg of one (sequence, head, segment): the suffix sums of x - y from the
// segment's end and <R, S> there, in double.  A step whose decay is zero has no
// gradient (dg = a_t <D_t, S_{t-1}>), and the sums of the steps before it start
// anew, from zero: a segmented scan, the flags of 64 steps as one lane mask.
// Bound by reading the states: 512 segments of 128 x 128, 70 MB, in 19 us (3.7
// TB/s).
struct DgArgs {
    const float *x, *y, *S, *R;   // S: entering states, segment n's end is slot n + 1; R may be NULL
    const float *g;
    int64_t gb, gt, gh;
    const int32_t *lengths;
    float *dg;                    // (B,T,H), or per-head partials (B,H,nSeg)
    int64_t s_bh, s_seg, r_bh, r_seg;   // strides of S (from slot 1 on) and R
    int64_t first;                // this launch's first workgroup
    int T, H, nSeg, segLen, E, per_head, vec;   // vec: E is a multiple of 8, S and R are 16-byte aligned
};

__device__ __forceinline__ double block_sum(double v, double *lds)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ void __launch_bounds__(256) dg_kernel(DgArgs a)
{
    __shared__ double red[4];
    __shared__ int restarts[4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t item = a.first + blockIdx.x;
    const int seg = static_cast<int>(item % a.nSeg);
    const int64_t bh = item / a.nSeg, b = bh / a.H;
    const int h = static_cast<int>(bh - b * a.H);
    const int t_lo = seg * a.segLen * kC, t_hi = min(a.T, t_lo + a.segLen * kC);
    int len = a.T;
    if (a.lengths) len = max(0, min(a.T, a.lengths[b]));

    double flux = 0.0;
    if (a.R) {
        const float *S = a.S + bh * a.s_bh + seg * a.s_seg, *R = a.R + bh * a.r_bh + seg * a.r_seg;
        if (a.vec) {   // four wide loads of each in flight
            double part[4] = {0.0, 0.0, 0.0, 0.0};
            int e = 4 * tid;
            for (; e + 3 * 1024 < a.E; e += 4 * 1024) {
                f4v x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = *reinterpret_cast<const f4v *>(S + e + 1024 * i);
                    y[i] = *reinterpret_cast<const f4v *>(R + e + 1024 * i);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i] += static_cast<double>(x[i][j]) * static_cast<double>(y[i][j]);
            }
            for (; e < a.E; e += 1024) {
                const f4v x = *reinterpret_cast<const f4v *>(S + e), y = *reinterpret_cast<const f4v *>(R + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) part[j] += static_cast<double>(x[j]) * static_cast<double>(y[j]);
            }
            flux = (part[0] + part[1]) + (part[2] + part[3]);
        } else {
            for (int e = tid; e < a.E; e += 256) flux += static_cast<double>(S[e]) * static_cast<double>(R[e]);
        }
    }
    flux = block_sum(flux, red);

    // 256 steps at a time, the latest first; thread i holds step hi - 1 - i.  flux is
    // the sum carried in from the later steps; a clearing step (and what is carried
    // to it) counts nothing for the steps before it.
    double sum = 0.0;
    for (int hi = t_hi; hi > t_lo; hi -= 256) {
        const int t = hi - 1 - tid;
        const bool live = t >= t_lo && t < len;
        const bool clears = live && a.g[b * a.gb + t * a.gt + h * a.gh] < -104.0f;
        double v = 0.0;
        if (live && !clears) v = static_cast<double>(a.x[bh * a.T + t]) - static_cast<double>(a.y[bh * a.T + t]);
        // lanes up to this one that clear; the sum starts after the last of them
        const uint64_t upto = __ballot(clears) & (~uint64_t(0) >> (63 - lane));
        const int from = upto ? 63 - __builtin_clzll(upto) : -1;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double u = __shfl_up(v, off, 64);
            if (lane - off >= max(from, 0)) v += u;
        }
        __syncthreads();
        if (lane == 63) {
            red[tid >> 6] = v;
            restarts[tid >> 6] = from >= 0;
        }
        __syncthreads();
        double mine = flux;   // carried in to this wave's first step
        for (int w = 0; w < 4; ++w) {
            if (w == (tid >> 6)) mine = flux;
            flux = restarts[w] ? red[w] : flux + red[w];
        }
        const double val = live && !clears ? (from >= 0 ? v : v + mine) : 0.0;
        if (t >= t_lo) {
            if (!a.per_head) a.dg[(b * a.T + t) * a.H + h] = static_cast<float>(val);
            else sum += val;
        }
    }
    if (a.per_head) {
        sum = block_sum(sum, red);
        if (tid == 0) a.dg[item] = static_cast<float>(sum);
    }
}

// dg of a decay per head: the partials of all sequences and segments, in order
__global__ void __launch_bounds__(256) dg_head_kernel(const float *part, float *dg, int64_t B, int H, int nSeg,
                                                      int first)
{
    __shared__ double red[4];
    const int h = first + static_cast<int>(blockIdx.x);
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < B * nSeg; i += 256) s += part[((i / nSeg) * H + h) * nSeg + i % nSeg];
    s = block_sum(s, red);
    if (threadIdx.x == 0) dg[h] = static_cast<float>(s);
}

// dq, dk of a query/key head: its value heads' fp32 partials (B T,H,d) summed in order
template <typename T>
__global__ void __launch_bounds__(256) group_sum_kernel(const float *p0, const float *p1, T *o0, T *o1, int64_t n, int H,
                                                        int Hk, int d, int64_t first)
{
    const int64_t at = (first + blockIdx.x) * 256 + threadIdx.x;   // of (B T,Hk,d)
    if (at >= n) return;
    const float *p = blockIdx.y ? p1 : p0;
    const int per = H / Hk;
    const int64_t row = at / (static_cast<int64_t>(Hk) * d);
    const int rest = static_cast<int>(at - row * Hk * d), hk = rest / d, c = rest - hk * d;
    p += (row * H + static_cast<int64_t>(hk) * per) * d + c;
    float s = 0.0f;
    for (int i = 0; i < per; ++i) s += p[static_cast<int64_t>(i) * d];
    (blockIdx.y ? o1 : o0)[at] = static_cast<T>(s);
}

// -------------------------------------------------------------------- a step
// One workgroup per (sequence, head, 16 R rows of the state): 16 lanes a row,
// each 4 (dk <= 64) or 2 x 4 neighbouring elements of R rows.  The state is
// read and written once; everything else is small.  Bound by HBM: 256 sequences
// x 16 heads of 128 x 128, 541 MB, in 104 us (5.2 TB/s); one sequence x 16 heads
// of 64 x 64 in 3 us, less than its launch.
struct StepArgs {
    const void *q, *k, *v;
    const float *g;
    float *S;
    void *o;
    const int32_t *slots;
    int64_t qb, qh, kb, kh, vb, vh, gb, gh;
    int64_t n_slots;
    uint32_t first;          // this launch's first workgroup
    int H, div, dk, dv, tiles, vec;
    float scale;
};

template <typename T, int NV, int R, bool VEC>
__global__ void __launch_bounds__(256) step_kernel(StepArgs a)
{
    using Frag = typename Num<T>::Frag;
    const int li = threadIdx.x & 15, row = threadIdx.x >> 4;
    const uint32_t group = a.first + blockIdx.x, bh = group / a.tiles;
    const int r0 = static_cast<int>(group - bh * a.tiles) * (16 * R) + row;
    const int64_t b = bh / a.H;
    const int h = static_cast<int>(bh % a.H);
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool live = slot >= 0 && slot < a.n_slots;
    T *o = static_cast<T *>(a.o) + static_cast<int64_t>(bh) * a.dv;
    if (!live) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (li == 0 && r0 + 16 * j < a.dv) o[r0 + 16 * j] = static_cast<T>(0.0f);
        return;
    }
    float *S = a.S + (slot * a.H + h) * static_cast<int64_t>(a.dv) * a.dk;
    // the state first: all its loads in flight before anything waits
    f4v s[R][NV];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int r = r0 + 16 * j, c = 64 * n + 4 * li;
            s[j][n] = f4v{0, 0, 0, 0};
            if constexpr (VEC) {
                if (r < a.dv && c < a.dk) s[j][n] = __builtin_nontemporal_load(reinterpret_cast<const f4v *>(S + r * a.dk + c));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r < a.dv && c + e < a.dk) s[j][n][e] = S[r * a.dk + c + e];
            }
        }
    const T *q = static_cast<const T *>(a.q) + b * a.qb + (h / a.div) * a.qh;
    const T *k = static_cast<const T *>(a.k) + b * a.kb + (h / a.div) * a.kh;
    const T *v = static_cast<const T *>(a.v) + b * a.vb + h * a.vh;
    f4v qf[NV], kf[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = 64 * n + 4 * li;
        qf[n] = kf[n] = f4v{0, 0, 0, 0};
        if constexpr (VEC) {
            if (c < a.dk) {
                qf[n] = __builtin_convertvector(*reinterpret_cast<const Frag *>(q + c), f4v);
                kf[n] = __builtin_convertvector(*reinterpret_cast<const Frag *>(k + c), f4v);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < a.dk) {
                    qf[n][e] = to_f32(q[c + e]);
                    kf[n][e] = to_f32(k[c + e]);
                }
        }
    }
    // e^g with the product's rounding made up for (of an exponent of 100 it is 2^-18)
    const float g = a.g[b * a.gb + h * a.gh], e = g * kLog2e;
    const float tail = __builtin_fmaf(g, kLog2eTail, __builtin_fmaf(g, kLog2e, -e));
    const float near = __builtin_amdgcn_exp2f(e);
    const float dec = near > 0.0f && near < __builtin_inff() ? __builtin_fmaf(near, tail * 0.693147180559945309417f, near) : near;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const int r = r0 + 16 * j;
        const float vr = r < a.dv ? to_f32(v[r]) : 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = 64 * n + 4 * li;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[j][n][e] = __builtin_fmaf(vr, kf[n][e], dec * s[j][n][e]);
                if (c + e < a.dk) dot = __builtin_fmaf(s[j][n][e], qf[n][e], dot);
            }
            if constexpr (VEC) {
                if (r < a.dv && c < a.dk) __builtin_nontemporal_store(s[j][n], reinterpret_cast<f4v *>(S + r * a.dk + c));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r < a.dv && c + e < a.dk) S[r * a.dk + c + e] = s[j][n][e];
            }
        }
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) dot += __shfl_xor(dot, off, 64);
        if (li == 0 && r < a.dv) o[r] = static_cast<T>(a.scale * dot);
    }
}

// --------------------------------------------------------------------- host

// Whether rows at p, with strides of (b, t, h), take 16-byte accesses and 64 of
// them lie within a buffer access's reach
bool wide(const void *p, const int64_t *st, int n, size_t size)
{
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    for (int i = 0; i < n; ++i)
        if ((static_cast<size_t>(st[i]) * size) & 15u) return false;
    return n < 3 || st[1] < (int64_t(1) << 21);
}

template <typename T, int MODE, bool VEC>
hipError_t launch_walk(WalkArgs a, int kdim, int vdim, hipStream_t s)
{
    const int threads = vdim <= 64 ? 256 : 512;
    const int64_t groups = (static_cast<int64_t>(a.items) + 7) / 8 * 8 * a.nRoles;
    return launch_sliced(groups, threads, [&](int64_t first, unsigned blocks) {
        const dim3 grid(blocks), block(threads);
        a.first = static_cast<uint32_t>(first);
        if (kdim <= 64 && vdim <= 64) hipLaunchKernelGGL((walk_kernel<T, 64, 64, MODE, VEC>), grid, block, 0, s, a);
        else if (kdim <= 64) hipLaunchKernelGGL((walk_kernel<T, 64, 128, MODE, VEC>), grid, block, 0, s, a);
        else if (vdim <= 64) hipLaunchKernelGGL((walk_kernel<T, 128, 64, MODE, VEC>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((walk_kernel<T, 128, 128, MODE, VEC>), grid, block, 0, s, a);
    });
}

template <int MODE> hipError_t launch_walk(int dtype, const WalkArgs &a, int kdim, int vdim, hipStream_t s)
{
    if (dtype == MGS_BF16)
        return a.vec ? launch_walk<__bf16, MODE, true>(a, kdim, vdim, s) : launch_walk<__bf16, MODE, false>(a, kdim, vdim, s);
    return a.vec ? launch_walk<float, MODE, true>(a, kdim, vdim, s) : launch_walk<float, MODE, false>(a, kdim, vdim, s);
}

template <typename T, int NV, int R> hipError_t launch_step(StepArgs a, int64_t heads, hipStream_t s)
{
    return launch_sliced(heads * a.tiles, 256, [&](int64_t first, unsigned blocks) {
        const dim3 grid(blocks), block(256);
        a.first = static_cast<uint32_t>(first);
        if (a.vec) hipLaunchKernelGGL((step_kernel<T, NV, R, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((step_kernel<T, NV, R, false>), grid, block, 0, s, a);
    });
}

template <typename T> hipError_t launch_step(const StepArgs &a, int64_t heads, int rows, hipStream_t s)
{
    if (a.dk <= 64) return rows == 4 ? launch_step<T, 1, 4>(a, heads, s) : launch_step<T, 1, 1>(a, heads, s);
    return rows == 4 ? launch_step<T, 2, 4>(a, heads, s) : launch_step<T, 2, 1>(a, heads, s);
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

// Segments: a walk takes one workgroup through its chunks in order, and of those
// with outputs LDS lets 512 of 8 waves (fp32: 256) or 768 of 4 (64 x 64; bf16 with
// dots: 512) on the chip.  A long sequence of few heads is cut until there are 512
// walks, or 1024 of 64 x 64 (512 of either kind are left whole: cutting costs two
// more launches and reads k and v twice).  No one target is best: half of it, it
// and twice it take 95, 85, 95 us for ragged prompts of 8 x 1999 steps x 16 heads
// of 64 x 128, but 126, 132, 152 for one of 32768 steps x 8 heads of 128 x 128, and
// for 4 x 4096 steps x 8 heads 39, 42, 55 (bf16, 64 x 64), 68, 75, 96 (128 x 128), 67,
// 69, 78 and 168, 176, 200 (the same in fp32).
// The backward also bounds a segment to 8 chunks, which bounds the rounding of
// dg's sums.
AttnGeom attn_geometry(const mgs_linattn_desc &d, bool backward)
{
    AttnGeom g{};
    g.BH = d.B * d.H;
    g.nC = static_cast<int>((d.T + kC - 1) / kC);
    const int64_t walks = std::max<int64_t>(1, g.BH * (backward ? 3 : 1));
    const int64_t want = d.dk <= 64 && d.dv <= 64 ? 1024 : 512;
    const int64_t seg = walks >= 512 ? 1 : (want + walks - 1) / walks;
    int64_t len = std::max<int64_t>(1, (g.nC + seg - 1) / seg);
    if (backward) len = std::min<int64_t>(len, 8);
    g.segLen = static_cast<int>(len);
    g.nSeg = static_cast<int>(std::max<int64_t>(1, (g.nC + len - 1) / len));
    g.grouped = backward && d.H != d.Hk;
    const size_t E = static_cast<size_t>(d.dk) * d.dv * 4, BH = static_cast<size_t>(g.BH);
    const size_t steps = static_cast<size_t>(d.B) * d.T * d.H;
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t off = at;
        at += align_up(bytes);
        return off;
    };
    if (g.nSeg > 1) {
        g.off_S = take(BH * (g.nSeg + 1) * E);
        if (backward) g.off_R = take(BH * g.nSeg * E);
        g.off_dec = take(BH * g.nSeg * 4);
    } else if (backward) {
        g.off_S = take(BH * E);   // the final state
    }
    if (backward) {
        g.off_x = take(steps * 4);
        g.off_y = take(steps * 4);
        g.off_dg = take(BH * g.nSeg * 4);
        if (g.grouped) {
            g.off_dq = take(steps * d.dk * 4);
            g.off_dk = take(steps * d.dk * 4);
        }
    }
    g.bytes = at;
    return g;
}

namespace {

Operand operand(const void *p, const int64_t *st, int64_t heads, int64_t H, int64_t cols)
{
    return Operand{p, st[0], st[1], st[2], static_cast<int>(H / heads), static_cast<int>(cols)};
}

WalkArgs walk_args(const AttnGeom &geo, const mgs_linattn_desc &d, const float *g, const int32_t *lengths, bool vec)
{
    WalkArgs a{};
    a.g = g;
    a.gb = d.decay_per_head ? 0 : d.g_stride[0];
    a.gt = d.decay_per_head ? 0 : d.g_stride[1];
    a.gh = d.decay_per_head ? 1 : d.g_stride[2];
    a.lengths = lengths;
    a.items = static_cast<uint32_t>(geo.BH * geo.nSeg);
    a.T = static_cast<int>(d.T);
    a.H = static_cast<int>(d.H);
    a.nC = geo.nC;
    a.nSeg = geo.nSeg;
    a.segLen = geo.segLen;
    a.vec = vec;
    return a;
}

hipError_t launch_chain(const AttnGeom &geo, ChainArgs c, int directions, hipStream_t s)
{
    return launch_sliced((geo.BH * c.E + 255) / 256, 256, [&](int64_t first, unsigned blocks) {
        c.first = first;
        hipLaunchKernelGGL(chain_kernel, dim3(blocks, directions), dim3(256), 0, s, c);
    });
}

hipError_t copy_state(const float *from, float *to, int64_t n, hipStream_t s);

__global__ void __launch_bounds__(256) copy_state_kernel(const float *from, float *to, int64_t n, int64_t first)
{
    const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.0f;
}

// `to` <- `from`, or zeros: states and gradients of empty sequences
hipError_t copy_state(const float *from, float *to, int64_t n, hipStream_t s)
{
    if (!to || n == 0) return hipSuccess;
    return launch_sliced((n + 255) / 256, 256, [&](int64_t first, unsigned blocks) {
        hipLaunchKernelGGL(copy_state_kernel, dim3(blocks), dim3(256), 0, s, from, to, n, first);
    });
}

}  // namespace

hipError_t launch_linattn_fwd(const AttnGeom &geo, const mgs_linattn_desc &d, const void *q, const void *k,
                              const void *v, const float *g, const float *S0, const int32_t *lengths, void *o,
                              float *ST, void *ws, hipStream_t s)
{
    const int dk = static_cast<int>(d.dk), dv = static_cast<int>(d.dv), E = dk * dv;
    if (geo.nC == 0) return copy_state(S0, ST, geo.BH * E, s);
    const size_t size = d.dtype == MGS_BF16 ? 2 : 4;
    const bool vec = dk % 8 == 0 && dv % 8 == 0 && d.H < (1 << 14) && wide(q, d.q_stride, 3, size) && wide(k, d.k_stride, 3, size) &&
                     wide(v, d.v_stride, 3, size) && wide(o, nullptr, 0, size) && wide(S0, nullptr, 0, 4) &&
                     wide(ST, nullptr, 0, 4);
    WalkArgs a = walk_args(geo, d, g, lengths, vec);
    a.nRoles = 1;
    Role &r = a.role[0];
    r.q = operand(q, d.q_stride, d.Hk, d.H, dk);
    r.k = operand(k, d.k_stride, d.Hk, d.H, dk);
    r.v = operand(v, d.v_stride, d.H, d.H, dv);
    r.out = o;
    r.sc = dk;
    r.sk = 1;
    r.intra = r.inter = d.scale;
    r.src = 1.0f;
    if (geo.nSeg == 1) {
        r.state = S0;
        r.final = ST;
        r.st_bh = E;
        return launch_walk<OUT>(d.dtype, a, dk, dv, s);
    }
    char *w = static_cast<char *>(ws);
    float *S = reinterpret_cast<float *>(w + geo.off_S);
    r.st_bh = static_cast<int64_t>(geo.nSeg + 1) * E;
    r.st_seg = E;
    r.local = S;
    a.dec = reinterpret_cast<float *>(w + geo.off_dec);
    hipError_t e = launch_walk<STATE>(d.dtype, a, dk, dv, s);
    if (e != hipSuccess) return e;
    ChainArgs c{};
    c.S = S;
    c.dec = a.dec;
    c.S0 = S0;
    c.ST = ST;
    c.BH = geo.BH;
    c.nSeg = geo.nSeg;
    c.E = E;
    e = launch_chain(geo, c, 1, s);
    if (e != hipSuccess) return e;
    r.state = S;
    return launch_walk<OUT>(d.dtype, a, dk, dv, s);
}

hipError_t launch_linattn_bwd(const AttnGeom &geo, const mgs_linattn_desc &d, const void *q, const void *k,
                              const void *v, const float *g, const void *do_, const float *S0, const float *dST,
                              const int32_t *lengths, void *dq, void *dk_, void *dv_, float *dg, float *dS0,
                              void *ws, hipStream_t s)
{
    const int dk = static_cast<int>(d.dk), dv = static_cast<int>(d.dv), E = dk * dv, H = static_cast<int>(d.H);
    hipError_t e;
    if (geo.nC == 0 || geo.BH == 0) {   // nothing to walk: sums over no steps, gradients that pass through
        if (d.decay_per_head && (e = copy_state(nullptr, dg, d.H, s)) != hipSuccess) return e;
        return copy_state(dST, dS0, geo.BH * E, s);
    }
    char *w = static_cast<char *>(ws);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(w + off); };
    float *S = at(geo.off_S), *R = geo.nSeg > 1 ? at(geo.off_R) : nullptr;
    float *x = at(geo.off_x), *y = at(geo.off_y);
    const size_t size = d.dtype == MGS_BF16 ? 2 : 4;
    const bool vec = dk % 8 == 0 && dv % 8 == 0 && d.H < (1 << 14) && wide(q, d.q_stride, 3, size) && wide(k, d.k_stride, 3, size) &&
                     wide(v, d.v_stride, 3, size) && wide(do_, d.do_stride, 3, size) && wide(dq, nullptr, 0, size) &&
                     wide(dk_, nullptr, 0, size) && wide(dv_, nullptr, 0, size) && wide(S0, nullptr, 0, 4) &&
                     wide(dST, nullptr, 0, 4) && wide(dS0, nullptr, 0, 4);
    WalkArgs a = walk_args(geo, d, g, lengths, vec);
    const Operand oq = operand(q, d.q_stride, d.Hk, d.H, dk), ok = operand(k, d.k_stride, d.Hk, d.H, dk);
    const Operand ov = operand(v, d.v_stride, d.H, d.H, dv), oo = operand(do_, d.do_stride, d.H, d.H, dv);
    const int64_t S_bh = static_cast<int64_t>(geo.nSeg > 1 ? geo.nSeg + 1 : 1) * E;
    const int64_t R_bh = static_cast<int64_t>(geo.nSeg) * E;

    Role rq{}, rk{}, rv{};   // of dq, dk, dv
    rq.q = oo, rq.k = ov, rq.v = ok, rq.dot = oq;
    rq.sc = 1, rq.sk = dk, rq.st_bh = S_bh, rq.st_seg = E;
    rq.intra = rq.inter = d.scale, rq.src = 1.0f;
    rq.xdot = x;
    rk.q = ov, rk.k = oo, rk.v = oq, rk.dot = ok;
    rk.sc = 1, rk.sk = dk;
    rk.xdot = y;
    rv.q = ok, rv.k = oq, rv.v = oo;
    rv.sc = dk, rv.sk = 1;
    for (Role *r : {&rk, &rv}) {
        r->st_bh = R_bh, r->st_seg = E;
        r->intra = r->src = d.scale, r->inter = 1.0f;
        r->rev = 1;
    }
    rq.out = geo.grouped ? static_cast<void *>(at(geo.off_dq)) : dq;
    rk.out = geo.grouped ? static_cast<void *>(at(geo.off_dk)) : dk_;
    rq.out_f32 = rk.out_f32 = geo.grouped;
    rv.out = dv_;

    if (geo.nSeg > 1) {
        // contributions of the segments to S (k, v) and R (q, do)
        WalkArgs l = a;
        l.nRoles = 2;
        l.dec = at(geo.off_dec);
        l.role[0].k = ok, l.role[0].v = ov, l.role[0].sc = dk, l.role[0].sk = 1, l.role[0].src = 1.0f;
        l.role[0].local = S, l.role[0].st_bh = S_bh, l.role[0].st_seg = E;
        l.role[1] = rv;
        l.role[1].local = R;
        if ((e = launch_walk<STATE>(d.dtype, l, dk, dv, s)) != hipSuccess) return e;
        ChainArgs c{};
        c.S = S, c.R = R, c.dec = l.dec, c.S0 = S0, c.dST = dST, c.dS0 = dS0;
        c.BH = geo.BH, c.nSeg = geo.nSeg, c.E = E;
        if ((e = launch_chain(geo, c, 2, s)) != hipSuccess) return e;
        rq.state = S;
        rk.state = rv.state = R;
    } else {
        rq.state = S0;
        rq.final = S;
        rk.state = rv.state = dST;
        rv.final = dS0;
    }
    // the dq and dk walks reduce over dv, the dv walk over dk
    // Few walks go in one launch: of one chunk, fp32 64 x 64, 64 walks a role 15 us
    // against 24 in two, 256: 22 against 29; bf16 128 x 128, 17 against 25 and 32
    // against 31.  Of many, dv's take the kernel without dots, which makes little
    // difference: 4 x 4096 x 16 heads in bf16, 128 x 128: 393 us so and 383 in one
    // (510 and 511 with the forward); 64 x 64: 171 and 174.
    const bool together = a.items <= 256 && (dk <= 64) == (dv <= 64);
    a.role[0] = rq, a.role[1] = rk, a.role[2] = rv;
    a.nRoles = together ? 3 : 2;
    if ((e = launch_walk<DOTS>(d.dtype, a, dv, dk, s)) != hipSuccess) return e;
    if (!together) {
        a.role[0] = rv;
        a.nRoles = 1;
        if ((e = launch_walk<OUT>(d.dtype, a, dk, dv, s)) != hipSuccess) return e;
    }

    DgArgs m{};
    m.x = x, m.y = y;
    m.S = geo.nSeg > 1 ? S + E : S;
    m.R = geo.nSeg > 1 ? R : dST;
    m.s_bh = S_bh, m.s_seg = E, m.r_bh = R_bh, m.r_seg = E;
    m.g = g, m.gb = a.gb, m.gt = a.gt, m.gh = a.gh;
    m.lengths = lengths;
    m.dg = d.decay_per_head ? at(geo.off_dg) : dg;
    m.T = a.T, m.H = H, m.nSeg = geo.nSeg, m.segLen = geo.segLen, m.E = E;
    m.per_head = d.decay_per_head != 0;
    m.vec = E % 8 == 0 && wide(dST, nullptr, 0, 4);
    e = launch_sliced(a.items, 256, [&](int64_t first, unsigned blocks) {
        m.first = first;
        hipLaunchKernelGGL(dg_kernel, dim3(blocks), dim3(256), 0, s, m);
    });
    if (e != hipSuccess) return e;
    if (d.decay_per_head) {
        e = launch_sliced(H, 256, [&](int64_t first, unsigned blocks) {
            hipLaunchKernelGGL(dg_head_kernel, dim3(blocks), dim3(256), 0, s, m.dg, dg, d.B, H, geo.nSeg,
                               static_cast<int>(first));
        });
        if (e != hipSuccess) return e;
    }
    if (geo.grouped) {
        const int64_t n = d.B * d.T * d.Hk * d.dk;
        const int Hk = static_cast<int>(d.Hk);
        e = launch_sliced((n + 255) / 256, 256, [&](int64_t first, unsigned blocks) {
            const dim3 grid(blocks, 2);
            if (d.dtype == MGS_BF16)
                hipLaunchKernelGGL(group_sum_kernel<__bf16>, grid, dim3(256), 0, s, at(geo.off_dq), at(geo.off_dk),
                                   static_cast<__bf16 *>(dq), static_cast<__bf16 *>(dk_), n, H, Hk, dk, first);
            else
                hipLaunchKernelGGL(group_sum_kernel<float>, grid, dim3(256), 0, s, at(geo.off_dq), at(geo.off_dk),
                                   static_cast<float *>(dq), static_cast<float *>(dk_), n, H, Hk, dk, first);
        });
    }
    return e;
}

hipError_t launch_linattn_step(const mgs_linattn_desc &d, const void *q, const void *k, const void *v,
                               const float *g, float *S, int64_t n_slots, const int32_t *slots, void *o,
                               hipStream_t s)
{
    StepArgs a{};
    a.q = q, a.k = k, a.v = v, a.g = g, a.S = S, a.o = o, a.slots = slots, a.n_slots = n_slots;
    a.qb = d.q_stride[0], a.qh = d.q_stride[2], a.kb = d.k_stride[0], a.kh = d.k_stride[2];
    a.vb = d.v_stride[0], a.vh = d.v_stride[2];
    a.gb = d.decay_per_head ? 0 : d.g_stride[0];
    a.gh = d.decay_per_head ? 1 : d.g_stride[2];
    a.H = static_cast<int>(d.H), a.div = static_cast<int>(d.H / d.Hk);
    a.dk = static_cast<int>(d.dk), a.dv = static_cast<int>(d.dv);
    // 4 rows a thread keep more of the state in flight, 1 spreads a small batch over
    // more of the chip.  By row tiles of 16, one row and four: 128 x 128, 512: 3.8
    // and 4.8 us, 2048: 7.2 and 7.3, 4096: 14.0 and 12.4, 16384: 48.9 and 48.9, 32768:
    // 97 and 103; 64 x 64, 1024: 3.9 and 5.8, 4096: 8.9 and 8.2, 8192: 15.7 and 13.4.
    const int rows = d.B * d.H * ((a.dv + 15) / 16) >= 4096 ? 4 : 1;
    a.tiles = (a.dv + 16 * rows - 1) / (16 * rows);
    const size_t size = d.dtype == MGS_BF16 ? 2 : 4;
    const int64_t sq[2] = {a.qb, a.qh}, sk[2] = {a.kb, a.kh};
    a.vec = a.dk % 8 == 0 && wide(S, nullptr, 0, 4) && wide(q, sq, 2, size) && wide(k, sk, 2, size);
    a.scale = d.scale;
    if (d.dtype == MGS_BF16) return launch_step<__bf16>(a, d.B * d.H, rows, s);
    return launch_step<float>(a, d.B * d.H, rows, s);
}

}  // namespace mgs
