// Layer norm over rows, forward and backward (waste_train.h).
//
// Both are one pass over the rows, whose floor is memory: 16384 x 7168 bf16 is 470 MB forward and 705 MB backward, 70 and
// 104 us at the 6.75 TB/s of a plain copy.  The mean comes first and the squares are taken about it (two sums over
// the row as it is held, no cancellation).
//   forward_stream_kernel  many rows: 92 us = 5.1 TB/s (rows of 7167 values, which begin anywhere: 124 us)
//   forward_few_kernel     up to 4 rows an SM: one row 3 us and the launch
//   backward_held_kernel   140 us = 5.0 TB/s (rows of 7167: 270 us; fp32 233 and 282, floor 209), with the partial sums of dw and db; reduce_kernel
//                          adds those up: one row of them a CTA, 152 at most
//   forward_kernel, dx_kernel, columns_kernel  rows past 8192 values: read two or three times, from L2 as far as it holds
//                          (4096 x 16384 bf16: 82 us forward, 175 backward, floors 40 and 60; of 16391 values 205 and 499)
// Short rows cost their steps: 65536 x 256 bf16 31 us forward and 47 backward, floors 10 and 15 (16384 x 1000: 23 and 35, 10
// and 15).
// What bounds the forward is the chain of steps of a row (wait, sum, squares, write) on the warps an SM holds; the backward's
// lanes also hold the sums of their columns, so a row takes 14 of its 16 warps, and two rows are in work at once (of 16 bits;
// of fp32, two in work leave too few on their way: 292 us against 233).
// Rows that begin anywhere: results go out in whole 16-byte pieces, and what does not lie in the same pieces is moved by
// words and half words in registers (single values through shared memory: 215 and 460 us).  The sums of dw and db are tied
// to columns, so the backward moves both operands there: that is what it costs.
// Spilled registers cost more than elsewhere: the rows on their way leave the L1 cache 28 KB, and what does not fit
// there goes to L2 (1024 threads with 52 bytes spilled 110 us, 896 with 24 bytes 98, 768 with none 92).
#include <type_traits>

#include "train.cuh"

namespace wm {
namespace train {

namespace {

constexpr int kThreads = 512;

__device__ uint32_t g_norm_timeout;

template <class T> __device__ __forceinline__ float widen(T v) { return (float)v; }
template <class T> __device__ __forceinline__ T round_to(float v);
template <> __device__ __forceinline__ float round_to<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }

// V consecutive values: whole 16-byte pieces where V is 8.
template <class T, int V> struct alignas(V == 8 ? 16 : sizeof(T)) Piece {
    T v[V];
};
template <class T, int V> __device__ __forceinline__ Piece<T, V> load(const T *p) {
    return *reinterpret_cast<const Piece<T, V> *>(p);
}
// All warps of group g, 16 groups at most.
__device__ __forceinline__ void group_meet(int gw, int g) {
    if (gw == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(g), "r"(gw * 32) : "memory");
}

// Sum over the warps of a group (gw of them, 16 at most; group `g` of the CTA), in every thread.  slot alternates
// between two halves of part (32 floats each), so one barrier a sum is enough.
__device__ __forceinline__ float group_sum(float v, int gw, int g, float *part, int &slot) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (gw == 1) return v;
    const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - g * gw;
    float *p = part + slot * 32 + g * gw;
    slot ^= 1;
    if (lane == 0) p[warp] = v;
    group_meet(gw, g);
    v = (lane & 15) < gw ? p[lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// n sums at once (1, 2 or 4), in every thread; part: 64 n floats.  The lanes share the values out between them in the first
// steps, so that 2 sums take 5 + 4 exchanges instead of 18, and 4 take 6 + 3 instead of 36.
template <int n> __device__ __forceinline__ void group_sums(float (&v)[n], int gw, int g, float *part, int &slot) {
    static_assert(n == 1 || n == 2 || n == 4, "a warp, its halves or quarters");
    if constexpr (n == 1) {
        v[0] = group_sum(v[0], gw, g, part, slot);
        return;
    }
    constexpr int kLanes = 32 / n;
    const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - g * gw, mine = lane / kLanes;
    float k = 0.f;
    if constexpr (n == 2) {
        const bool up = lane & 16;
        k = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    } else if constexpr (n == 4) {
        const bool up = lane & 16, odd = lane & 8;
        const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
        const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
        k = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    if (gw > 1) {
        float *p = part + slot * 32 * n + mine * 32 + g * gw;
        slot ^= 1;
        const int i = lane % kLanes;
        if (i == 0) p[warp] = k;
        group_meet(gw, g);
        k = i < gw ? p[i] : 0.f;
        if (kLanes < 16 && i + kLanes < gw) k += p[i + kLanes];
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    }
#pragma unroll
    for (int j = 0; j < n; ++j) v[j] = __shfl_sync(0xffffffffu, k, j * kLanes);
}

// The kernels that read a row once hold it in registers or in shared memory.  Rows come by bulk copies, one instruction
// each, some ahead; values are computed in pairs (one instruction for both); w and b stand in shared memory in fp32.
// kHeld: values a lane where a row is spread over up to 16 warps.
constexpr int kHeld = 16;
// Rows of a group in work at once in the backward: two of 16 bits, where two more fit on their way behind them.
template <class X, class Y, int V> constexpr int kRowsAtOnce = V == 8 && sizeof(X) + sizeof(Y) == 4 ? 2 : 1;
constexpr int kHeldThreads = 512;
constexpr int kHeldMost = kHeld * kHeldThreads;
constexpr int kHeldSmem = 220 << 10;
constexpr int kDeepMost = 8;

// Two values at a time.
__device__ __forceinline__ uint64_t bits(float2 v) { return *reinterpret_cast<uint64_t *>(&v); }
__device__ __forceinline__ float2 pair(uint64_t v) { return *reinterpret_cast<float2 *>(&v); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return pair(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return pair(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(d);
}
__device__ __forceinline__ float2 widen2(const float *p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 widen2(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 widen2(const __half *p) { return __half22float2(*reinterpret_cast<const __half2 *>(p)); }
__device__ __forceinline__ void round2(float *p, float2 v) { p[0] = v.x, p[1] = v.y; }
__device__ __forceinline__ void round2(__nv_bfloat16 *p, float2 v) { *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y); }
__device__ __forceinline__ void round2(__half *p, float2 v) { *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(v.x, v.y); }

// V values of w or b from column c on.
template <class T, int V> __device__ __forceinline__ void widen_all(const void *p, int c, float (&o)[V]) {
    const Piece<T, V> q = load<T, V>(static_cast<const T *>(p) + c);
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = widen(q.v[k]);
}
template <int V> __device__ __forceinline__ void widen_params(const void *p, int dtype, int c, float none, float (&o)[V]) {
    if (!p) {
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = none;
    } else if (dtype == WASTE_ACT_F32) {
        widen_all<float>(p, c, o);
    } else if (dtype == WASTE_ACT_BF16) {
        widen_all<__nv_bfloat16>(p, c, o);
    } else {
        widen_all<__half>(p, c, o);
    }
}
// A lane's values of a row, in kHeld / V pieces a group's width apart: whole pieces from a copy of the row in shared
// memory, single values straight from memory.  kFull: the row fills all lanes.
template <class X, int V, bool kFull> struct Lane {
    enum { H = kHeld, kPieces = H / V };
    int t, gt, d;
    __device__ __forceinline__ int column(int i) const { return (i * gt + t) * V; }
    __device__ __forceinline__ bool in(int i) const { return kFull || column(i) < d; }
    // zeros past the row's end
    __device__ __forceinline__ void take(const X *row, float2 (&x)[H / 2]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (V == 8) {
                Piece<X, V> q = {};
                if (in(i)) q = load<X, V>(row + column(i));
#pragma unroll
                for (int k = 0; k < V / 2; ++k) x[V / 2 * i + k] = widen2(&q.v[2 * k]);
            } else {
                const float v = in(i) ? widen(row[column(i)]) : 0.f;
                if (i & 1)
                    x[i / 2].y = v;
                else
                    x[i / 2].x = v;
            }
        }
    }
    // rounded to their places
    template <class Y> __device__ __forceinline__ void give(Y *row, const float2 (&y)[H / 2]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if (!in(i)) continue;
            if constexpr (V == 8) {
                Piece<Y, V> o;
#pragma unroll
                for (int k = 0; k < V / 2; ++k) round2(&o.v[2 * k], y[V / 2 * i + k]);
                *reinterpret_cast<Piece<Y, V> *>(row + column(i)) = o;
            } else {
                row[column(i)] = round_to<Y>(i & 1 ? y[i / 2].y : y[i / 2].x);
            }
        }
    }
    // w or b at the same places, `none` past the row's end
    __device__ __forceinline__ void params(const void *p, int dtype, float none, float2 (&o)[H / 2]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = none;
            if (in(i)) widen_params<V>(p, dtype, column(i), none, v);
#pragma unroll
            for (int k = 0; k < V; ++k) ((V * i + k) & 1 ? o[(V * i + k) / 2].y : o[(V * i + k) / 2].x) = v[k];
        }
    }
    // Whether the two values of pair j are the row's.
    __device__ __forceinline__ bool first(int j) const { return in(2 * j / V); }
    __device__ __forceinline__ bool second(int j) const { return in((2 * j + 1) / V); }
};
// Values of w (and b) in shared memory, in fp32, filled by all threads.
// Whole rows: of every eight the first four in one half and the last four in the other, so that the lanes of a
// warp, eight columns apart, read neighbouring 16 bytes.
__device__ __forceinline__ void stage(float *to, const void *p, int dtype, int d, float none) {
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
        float v[1];
        widen_params<1>(p, dtype, i, none, v);
        to[(i & 4 ? d / 2 : 0) + (i >> 3) * 4 + (i & 3)] = v[0];
    }
}
// Any rows: columns of the same remainder by eight stand together, so that lanes eight columns apart read neighbours
// wherever they begin, -7 to d + 7 (zeros past d); n of them beside each other (w alone; w and b).
__host__ __device__ constexpr int eighths(int d) { return (d + 15) / 8; }
template <int n> __device__ __forceinline__ void stage_any(float *to, const void *w, const void *b, int dtype, int d) {
    for (int i = threadIdx.x; i < 8 * eighths(d); i += blockDim.x) {
        float v[1] = {0.f}, u[1] = {0.f};
        if (i < d) {
            widen_params<1>(w, dtype, i, 1.f, v);
            if (n == 2) widen_params<1>(b, dtype, i, 0.f, u);
        }
        const int at = n * ((i & 7) * eighths(d) + (i >> 3));
        to[at] = v[0];
        if (n == 2) to[at + 1] = u[0];
    }
}
// Byte of column c there.
template <int n> __device__ __forceinline__ uint32_t place_any(int d, int c) { return 4 * n * ((c & 7) * eighths(d) + (c >> 3)); }
// A piece in shared memory, said to be there (an address that the compiler has lost track of goes the long way).
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
    return u;
}
__device__ __forceinline__ float shared_float(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float2 shared_float2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
template <class X> __device__ __forceinline__ Piece<X, 8> load_shared(uint32_t at) {
    Piece<X, 8> q;
    reinterpret_cast<uint4 *>(&q)[0] = shared16(at);
    if constexpr (sizeof(X) == 4) reinterpret_cast<uint4 *>(&q)[1] = shared16(at + 16);
    return q;
}

// Eight values that begin anywhere: the 16-byte pieces around them, moved by words and by half a word.  Reads up to 14
// bytes before and 30 behind what is asked for.
template <class X> __device__ __forceinline__ Piece<X, 8> load_any(uint32_t at) {
    constexpr int W = 2 * sizeof(X); // words
    if ((at & 15) == 0) return load_shared<X>(at);
    Piece<X, 8> q;
    uint32_t u[W + 4], v[W + 2], w[W + 1];
#pragma unroll
    for (int i = 0; i < W + 4; i += 4) {
        const uint4 s = shared16((at & ~15u) + 4 * i);
        u[i] = s.x, u[i + 1] = s.y, u[i + 2] = s.z, u[i + 3] = s.w;
    }
#pragma unroll
    for (int i = 0; i < W + 2; ++i) v[i] = at & 8 ? u[i + 2] : u[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) w[i] = at & 4 ? v[i + 1] : v[i];
#pragma unroll
    for (int i = 0; i < W; ++i)
        reinterpret_cast<uint32_t *>(&q)[i] = sizeof(X) == 2 ? __funnelshift_r(w[i], w[i + 1], (at & 2) * 8) : w[i];
    return q;
}
// Zeros in those of eight values from column c on that are not the row's.
__device__ __forceinline__ void trim(float2 *x, int c, int d) {
    if (c >= 0 && c + 8 <= d) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (c + 2 * k < 0 || c + 2 * k >= d) x[k].x = 0.f;
        if (c + 2 * k + 1 < 0 || c + 2 * k + 1 >= d) x[k].y = 0.f;
    }
}
// Eight results to column c on, of which those outside the row are left out; the first on 16 bytes.
template <class Y> __device__ __forceinline__ void give_any(Y *row, int c, int d, const Piece<Y, 8> &o) {
    if (c >= 0 && c + 8 <= d) {
        *reinterpret_cast<Piece<Y, 8> *>(row + c) = o;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k >= 0 && c + k < d) row[c + k] = o.v[k];
    }
}
// Values between a 16-byte boundary and p.
template <class Y> __device__ __forceinline__ int before16(const Y *p) { return (int)(((uintptr_t)p & 15) / sizeof(Y)); }

// Four of them from column c on (a multiple of 4).
__device__ __forceinline__ void four(uint32_t p, int d, int c, float2 &a, float2 &b) {
    const uint4 q = shared16(p + ((c & 4 ? d / 2 : 0) + (c >> 3) * 4) * 4);
    a = make_float2(__uint_as_float(q.x), __uint_as_float(q.y)), b = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
}

// Beside rows that begin anywhere there is room for what load_any reads around them, from column -7 to d + 7.
constexpr uint32_t kRingFront = 32, kRingBack = 64; // the shift, and 48
// The rows of one operand on their way to a group of warps: places in shared memory, filled in order by bulk
// copies of one thread.  A place is free again once the group has met (in a sum) behind its reading.  Copies take whole
// 16-byte pieces: of a row that begins or ends inside one, its neighbours in that piece come too (nothing lies
// between them and the row that could be out of memory: allocations begin and end on such pieces), and are not used.
template <class X, bool kWhole> struct Ring {
    const X *p;
    int64_t ld;
    int d;
    uint32_t at, pitch; // this group's places
    enum { kFront = kWhole ? 0 : kRingFront };
    __device__ __forceinline__ const X *row_at(int64_t row) const { return p + row * ld; }
    // bytes between the place's start and the row's
    __device__ __forceinline__ uint32_t shift(int64_t row) const { return kWhole ? 0 : (uint32_t)(uintptr_t)row_at(row) & 15u; }
    __device__ __forceinline__ uint32_t bytes(int64_t row) const { return (shift(row) + d * (uint32_t)sizeof(X) + 15) & ~15u; }
    __device__ __forceinline__ uint32_t place(int64_t row, uint32_t i) const { return at + i * pitch + kFront + shift(row); }
    __device__ __forceinline__ void copy(int64_t row, uint32_t i, uint32_t bar) const {
        tc::bulk_g2s(at + i * pitch + kFront, reinterpret_cast<const uint8_t *>(row_at(row)) - shift(row), bytes(row), bar);
    }
};
__host__ __device__ constexpr uint32_t ring_pitch(int d, uint32_t size, bool whole) {
    return (d * size + 15) / 16 * 16 + (whole ? 0 : kRingFront + kRingBack);
}
// Few rows: a row a group, straight from memory, w and b held too, for all loads to be on their way at once.
template <class X, class Y, int V>
__global__ void __launch_bounds__(kHeldThreads) forward_few_kernel(const NormFwd P, int gw) {
    using L = Lane<X, V, false>;
    constexpr int N = kHeld / 2;
    __shared__ float part[64];
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    const L lane{t, gt, P.d};
    int slot = 0;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < P.T; row += (int64_t)gridDim.x * groups) {
        float2 x[N], w[N], b[N], s = both(0.f);
        lane.take(static_cast<const X *>(P.x.p) + row * P.x.ld, x);
        lane.params(P.w, P.w_dtype, 1.f, w);
        lane.params(P.b, P.w_dtype, 0.f, b);
#pragma unroll
        for (int i = 0; i < N; ++i) s = add2(s, x[i]);
        const float mu = group_sum(s.x + s.y, gw, g, part, slot) * inv;
        s = both(0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = add2(x[i], both(-mu));
            if (!lane.first(i)) x[i].x = 0.f;
            if (!lane.second(i)) x[i].y = 0.f;
            s = fma2(x[i], x[i], s);
        }
        const float r = 1.f / sqrtf(group_sum(s.x + s.y, gw, g, part, slot) * inv + P.eps);
        if (P.mean && t == 0) {
            P.mean[row] = mu;
            P.rstd[row] = r;
        }
        Y *y = static_cast<Y *>(P.y.p) + row * P.y.ld;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fma2(mul2(x[i], both(r)), w[i], b[i]);
        lane.give(y, x);
    }
}

// Many rows: kStreamHeld values a lane, so that a row takes eight warps at most and an SM works on four rows or more at
// once, each group at a step of its own.
// Rows that begin anywhere (V = 1): a lane's eight columns are those of a whole 16-byte piece of y.
constexpr int kStreamHeld = 32, kStreamThreads = 768;
template <class X, class Y, int V>
__global__ void __launch_bounds__(kStreamThreads) forward_stream_kernel(const NormFwd P, int gw, int deep) {
    constexpr int kPieces = kStreamHeld / 8, kSize = sizeof(X);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[64];
    __shared__ __align__(8) uint64_t bars[kStreamThreads / 32 * kDeepMost];
    __shared__ uint32_t gave_up;
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    const int step = gridDim.x * groups, row0 = blockIdx.x * groups + g; // rows are 2^30 at most
    const uint32_t pitch = ring_pitch(P.d, kSize, V == 8), bar0 = tc::smem_u32(bars + g * deep);
    const Ring<X, V == 8> ring{static_cast<const X *>(P.x.p), P.x.ld, P.d, tc::smem_u32(smem) + g * deep * pitch, pitch};
    float *w = reinterpret_cast<float *>(smem + (size_t)groups * deep * pitch), *b = w + P.d;
    const uint32_t w_at = tc::smem_u32(w), b_at = tc::smem_u32(b);
    const auto ask = [&](int row, uint32_t i) {
        tc::mbar_arrive_expect_tx(bar0 + 8 * i, ring.bytes(row));
        ring.copy(row, i, bar0 + 8 * i);
    };
    if (threadIdx.x == 0) gave_up = 0;
    if (t == 0) {
        for (int i = 0; i < deep; ++i) tc::mbar_init(bar0 + 8 * i, 1);
        tc::mbar_init_fence();
        for (int i = 0; i < deep && row0 + i * step < P.T; ++i) ask(row0 + i * step, i);
    }
    if constexpr (V == 8) {
        stage(w, P.w, P.w_dtype, P.d, 1.f);
        stage(b, P.b, P.w_dtype, P.d, 0.f);
    } else {
        stage_any<2>(w, P.w, P.b, P.w_dtype, P.d);
    }
    __syncthreads();
    int slot = 0;
    uint32_t turn = 0, phase = 0;
    for (int row = row0; row < P.T; row += step) {
        float2 x[kStreamHeld / 2], s = both(0.f);
        const int before = V == 8 ? 0 : before16(static_cast<Y *>(P.y.p) + (int64_t)row * P.y.ld);
        const auto column = [&](int i) { return (i * gt + t) * 8 - before; };
        wait_row(bar0 + 8 * turn, phase, &gave_up, &g_norm_timeout);
        const uint32_t from = ring.place(row, turn);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const bool in = column(i) < P.d;
            if constexpr (V == 8) {
                if (in) {
                    const Piece<X, 8> q = load_shared<X>(from + column(i) * kSize);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[4 * i + k] = widen2(&q.v[2 * k]);
                        s = add2(s, x[4 * i + k]);
                    }
                }
            } else if (in) {
                const Piece<X, 8> q = load_any<X>(from + column(i) * kSize);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[4 * i + k] = widen2(&q.v[2 * k]);
                trim(x + 4 * i, column(i), P.d);
#pragma unroll
                for (int k = 0; k < 4; ++k) s = add2(s, x[4 * i + k]);
            }
        }
        const float mu = group_sum(s.x + s.y, gw, g, part, slot) * inv;
        if (t == 0 && row + deep * step < P.T) ask(row + deep * step, turn); // the group has read this one
        if (++turn == (uint32_t)deep) turn = 0, phase ^= 1;
        s = both(0.f);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const bool in = column(i) < P.d;
            if constexpr (V == 8) {
                if (in) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[4 * i + k] = add2(x[4 * i + k], both(-mu));
                        s = fma2(x[4 * i + k], x[4 * i + k], s);
                    }
                }
            } else if (in) {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[4 * i + k] = add2(x[4 * i + k], both(-mu));
                trim(x + 4 * i, column(i), P.d);
#pragma unroll
                for (int k = 0; k < 4; ++k) s = fma2(x[4 * i + k], x[4 * i + k], s);
            }
        }
        const float r = 1.f / sqrtf(group_sum(s.x + s.y, gw, g, part, slot) * inv + P.eps);
        if (P.mean && t == 0) {
            P.mean[row] = mu;
            P.rstd[row] = r;
        }
        Y *y = static_cast<Y *>(P.y.p) + (int64_t)row * P.y.ld;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (column(i) < P.d) {
                Piece<Y, 8> o;
                if constexpr (V == 8) {
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        float2 w0, w1, b0, b1;
                        four(w_at, P.d, column(i) + k, w0, w1);
                        four(b_at, P.d, column(i) + k, b0, b1);
                        round2(&o.v[k], fma2(mul2(x[4 * i + k / 2], both(r)), w0, b0));
                        round2(&o.v[k + 2], fma2(mul2(x[4 * i + k / 2 + 1], both(r)), w1, b1));
                    }
                    *reinterpret_cast<Piece<Y, 8> *>(y + column(i)) = o;
                } else {
                    const int c = column(i);
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 u = shared_float2(w_at + place_any<2>(P.d, c + k)), v = shared_float2(w_at + place_any<2>(P.d, c + k + 1));
                        round2(&o.v[k], fma2(mul2(x[4 * i + k / 2], both(r)), make_float2(u.x, v.x), make_float2(u.y, v.y)));
                    }
                    give_any(y, c, P.d, o);
                }
            }
    }
    settle(&gave_up);
}

// dx, and a CTA's share of dw and db, in one pass.
template <class X, class Y, int V, bool kFull>
__global__ void __launch_bounds__(kHeldThreads) backward_held_kernel(const NormBwd P, int gw, int deep) {
    using L = Lane<X, 8, kFull>; // its columns, for dw and db
    constexpr int N = kHeld / 2, R = kRowsAtOnce<X, Y, V>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[128 * R];
    __shared__ __align__(8) uint64_t bars[kHeldThreads / 32 * kDeepMost];
    __shared__ uint32_t gave_up;
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    const int64_t step = (int64_t)gridDim.x * groups, row0 = (int64_t)blockIdx.x * groups + g;
    const L lx{t, gt, P.d};
    // x and dy of a row stand behind each other and share a barrier
    const uint32_t xp = ring_pitch(P.d, sizeof(X), V == 8), pitch = xp + ring_pitch(P.d, sizeof(Y), V == 8);
    const uint32_t bar0 = tc::smem_u32(bars + g * deep), mine = tc::smem_u32(smem) + g * deep * pitch;
    const Ring<X, V == 8> rx{static_cast<const X *>(P.x.p), P.x.ld, P.d, mine, pitch};
    const Ring<Y, V == 8> ry{static_cast<const Y *>(P.dy.p), P.dy.ld, P.d, mine + xp, pitch};
    float *w = reinterpret_cast<float *>(smem + (size_t)groups * deep * pitch);
    const uint32_t w_at = tc::smem_u32(w);
    const auto ask = [&](int64_t row, uint32_t i) {
        tc::mbar_arrive_expect_tx(bar0 + 8 * i, rx.bytes(row) + ry.bytes(row));
        rx.copy(row, i, bar0 + 8 * i);
        ry.copy(row, i, bar0 + 8 * i);
    };
    if (threadIdx.x == 0) gave_up = 0;
    if (t == 0) {
        for (int i = 0; i < deep; ++i) tc::mbar_init(bar0 + 8 * i, 1);
        tc::mbar_init_fence();
        for (int i = 0; i < deep && row0 + i * step < P.T; ++i) ask(row0 + i * step, i);
    }
    if constexpr (V == 8)
        stage(w, P.w, P.w_dtype, P.d, 1.f);
    else
        stage_any<1>(w, P.w, nullptr, P.w_dtype, P.d);
    __syncthreads();
    float2 dw[N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = db[i] = both(0.f);
    float mu_next[R], r_next[R];
    const auto stats = [&](int64_t row) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const bool in = row + q * step < P.T;
            mu_next[q] = in ? P.mean[row + q * step] : 0.f;
            r_next[q] = in ? P.rstd[row + q * step] : 0.f;
        }
    };
    stats(row0);
    int slot = 0;
    uint32_t turn = 0, phase = 0;
    for (int64_t row = row0; row < P.T; row += R * step) {
        float mu[R], r[R];
#pragma unroll
        for (int q = 0; q < R; ++q) mu[q] = mu_next[q], r[q] = r_next[q];
        stats(row + R * step);
        const uint32_t first = turn;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (row + q * step < P.T) wait_row(bar0 + 8 * turn, phase, &gave_up, &g_norm_timeout);
            if (++turn == (uint32_t)deep) turn = 0, phase ^= 1;
        }
        // x - mu and dy of row q, eight columns from col on, zeros past the row's ends
        const auto piece = [&](int q, int col, float2(&c)[4], float2(&e)[4]) {
            uint32_t at = first + q;
            if (at >= (uint32_t)deep) at -= deep;
            const int64_t from = row + q * step;
            const bool there = (kFull || col < P.d) && from < P.T;
            Piece<X, 8> u = {};
            Piece<Y, 8> v = {};
            if (there) {
                const uint32_t ux = rx.place(from, at) + col * (int)sizeof(X), vy = ry.place(from, at) + col * (int)sizeof(Y);
                u = V == 8 ? load_shared<X>(ux) : load_any<X>(ux);
                v = V == 8 ? load_shared<Y>(vy) : load_any<Y>(vy);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c[k] = add2(widen2(&u.v[2 * k]), both(-mu[q]));
                e[k] = widen2(&v.v[2 * k]);
            }
            if (V != 8) {
                trim(c, col, P.d);
                trim(e, col, P.d);
            }
        };
        const auto weights = [&](int col, float2(&o)[4]) {
            if (!kFull && col >= P.d) {
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = both(0.f);
                return;
            }
            if constexpr (V == 8) {
                four(w_at, P.d, col, o[0], o[1]);
                four(w_at, P.d, col + 4, o[2], o[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) (k & 1 ? o[k / 2].y : o[k / 2].x) = shared_float(w_at + place_any<1>(P.d, col + k));
            }
        };
        float2 s1[R], s2[R];
#pragma unroll
        for (int q = 0; q < R; ++q) s1[q] = s2[q] = both(0.f);
#pragma unroll
        for (int i = 0; i < kHeld / 8; ++i) { // past the row's end dy is zero, so all of these are
            float2 wv[4];
            weights(lx.column(i), wv);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                float2 c[4], e[4];
                piece(q, lx.column(i), c, e);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 xh = mul2(c[k], both(r[q])), gv = mul2(e[k], wv[k]);
                    dw[4 * i + k] = fma2(e[k], xh, dw[4 * i + k]);
                    db[4 * i + k] = add2(db[4 * i + k], e[k]);
                    s1[q] = add2(s1[q], gv);
                    s2[q] = fma2(gv, xh, s2[q]);
                }
            }
        }
        float s[2 * R];
#pragma unroll
        for (int q = 0; q < R; ++q) s[2 * q] = s1[q].x + s1[q].y, s[2 * q + 1] = s2[q].x + s2[q].y;
        group_sums(s, gw, g, part, slot);
        if (t == 0 && row > row0) // the rows before these have been read by all: into their places
            for (int q = 0; q < R; ++q)
                if (row + (q + deep - R) * step < P.T) ask(row + (q + deep - R) * step, (first + deep - R + q) % deep);
#pragma unroll
        for (int i = 0; i < kHeld / 8 && P.dx.p; ++i) {
            float2 wv[4];
            if (V == 8) weights(lx.column(i), wv);
#pragma unroll
            for (int q = 0; q < R; ++q) {
                X *dx = static_cast<X *>(P.dx.p) + (row + q * step) * P.dx.ld;
                const int col = lx.column(i) - (V == 8 ? 0 : before16(dx)); // whole 16-byte pieces of dx
                if (V != 8) weights(col, wv);
                float2 c[4], e[4];
                piece(q, col, c, e);
                // r (g - m1 - (x - mu) r m2), its factors of the row put together first
                const float2 rr = both(r[q]), c1 = both(-r[q] * (s[2 * q] * inv)), c2 = both(-r[q] * (r[q] * (s[2 * q + 1] * inv)));
                Piece<X, 8> o;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    round2(&o.v[2 * k], fma2(mul2(e[k], wv[k]), rr, fma2(c[k], c2, c1)));
                if (row + q * step >= P.T || (!kFull && col >= P.d)) continue;
                if constexpr (V == 8)
                    *reinterpret_cast<Piece<X, 8> *>(dx + col) = o;
                else
                    give_any(dx, col, P.d, o);
            }
        }
    }
    settle(&gave_up);
    if (!P.dw && !P.db) return;
    // the groups' sums, added up in their order (barrier 0 is the first group's own until here)
    asm volatile("bar.sync 15;" ::: "memory");
    float *sum = reinterpret_cast<float *>(smem) + (size_t)g * 2 * P.d, *out = P.parts + (size_t)blockIdx.x * 2 * P.d;
    if (groups == 1) sum = out;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int c = lx.column(i / 8) + i % 8;
        if (!kFull && c >= P.d) continue;
        sum[c] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
        sum[P.d + c] = i & 1 ? db[i / 2].y : db[i / 2].x;
    }
    if (groups == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * P.d; c += blockDim.x) {
        float v = 0.f;
        for (int j = 0; j < groups; ++j) v += reinterpret_cast<const float *>(smem)[(size_t)j * 2 * P.d + c];
        out[c] = v;
    }
}

// Rows longer than that: read again for each step.
template <class X, class Y, int V>
__global__ void __launch_bounds__(kThreads) forward_kernel(const NormFwd P, int gw) {
    __shared__ float part[64];
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    int slot = 0;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < P.T; row += (int64_t)gridDim.x * groups) {
        const X *x = static_cast<const X *>(P.x.p) + row * P.x.ld;
        Y *y = static_cast<Y *>(P.y.p) + row * P.y.ld;
        float s = 0.f;
        for (int c = t * V; c < P.d; c += gt * V) {
            const auto q = load<X, V>(x + c);
#pragma unroll
            for (int i = 0; i < V; ++i) s += widen(q.v[i]);
        }
        const float mu = group_sum(s, gw, g, part, slot) * inv;
        s = 0.f;
        for (int c = t * V; c < P.d; c += gt * V) {
            const auto q = load<X, V>(x + c);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = widen(q.v[i]) - mu;
                s = fmaf(v, v, s);
            }
        }
        const float r = 1.f / sqrtf(group_sum(s, gw, g, part, slot) * inv + P.eps);
        for (int c = t * V; c < P.d; c += gt * V) {
            const auto q = load<X, V>(x + c);
            Piece<Y, V> o;
            float w[V], b[V];
            widen_params<V>(P.w, P.w_dtype, c, 1.f, w);
            widen_params<V>(P.b, P.w_dtype, c, 0.f, b);
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = round_to<Y>(fmaf((widen(q.v[i]) - mu) * r, w[i], b[i]));
            *reinterpret_cast<Piece<Y, V> *>(y + c) = o;
        }
        if (P.mean && t == 0) {
            P.mean[row] = mu;
            P.rstd[row] = r;
        }
    }
}

template <class X, class Y, int V>
__global__ void __launch_bounds__(kThreads) dx_kernel(const NormBwd P, int gw) {
    __shared__ float part[64];
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    int slot = 0;
    for (int64_t row = (int64_t)blockIdx.x * groups + g; row < P.T; row += (int64_t)gridDim.x * groups) {
        const X *x = static_cast<const X *>(P.x.p) + row * P.x.ld;
        const Y *dy = static_cast<const Y *>(P.dy.p) + row * P.dy.ld;
        X *dx = static_cast<X *>(P.dx.p) + row * P.dx.ld;
        const float mu = P.mean[row], r = P.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        for (int c = t * V; c < P.d; c += gt * V) {
            const auto q = load<X, V>(x + c);
            const auto e = load<Y, V>(dy + c);
            float w[V];
            widen_params<V>(P.w, P.w_dtype, c, 1.f, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gv = widen(e.v[i]) * w[i];
                s1 += gv;
                s2 = fmaf(gv, (widen(q.v[i]) - mu) * r, s2);
            }
        }
        s1 = group_sum(s1, gw, g, part, slot) * inv;
        s2 = group_sum(s2, gw, g, part, slot) * inv;
        for (int c = t * V; c < P.d; c += gt * V) {
            const auto q = load<X, V>(x + c);
            const auto e = load<Y, V>(dy + c);
            Piece<X, V> o;
            float w[V];
            widen_params<V>(P.w, P.w_dtype, c, 1.f, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (widen(q.v[i]) - mu) * r, gv = widen(e.v[i]) * w[i];
                o.v[i] = round_to<X>(r * (gv - s1 - xh * s2));
            }
            *reinterpret_cast<Piece<X, V> *>(dx + c) = o;
        }
    }
}

// Sums of dy xh and of dy over a share of the rows: a lane holds V columns, a CTA's 16 warps take its rows in turn.
template <class X, class Y, int V>
__global__ void __launch_bounds__(kThreads) columns_kernel(const NormBwd P) {
    __shared__ float part[2][kThreads * V];
    tc::grid_wait_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * V;
    float dw[V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.f;
    const int64_t r0 = (int64_t)P.T * blockIdx.y / gridDim.y, r1 = (int64_t)P.T * (blockIdx.y + 1) / gridDim.y;
    if (c < P.d)
        for (int64_t row = r0 + warp; row < r1; row += kThreads / 32) {
            const auto q = load<X, V>(static_cast<const X *>(P.x.p) + row * P.x.ld + c);
            const auto e = load<Y, V>(static_cast<const Y *>(P.dy.p) + row * P.dy.ld + c);
            const float mu = P.mean[row], r = P.rstd[row];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dw[i] = fmaf(widen(e.v[i]), (widen(q.v[i]) - mu) * r, dw[i]);
                db[i] += widen(e.v[i]);
            }
        }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        part[0][(warp * 32 + lane) * V + i] = dw[i];
        part[1][(warp * 32 + lane) * V + i] = db[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * 32 * V; i += kThreads) {
        const int which = i / (32 * V), j = i % (32 * V);
        const int64_t col = (int64_t)blockIdx.x * 32 * V + j;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += part[which][w * 32 * V + j];
        if (col < P.d) P.parts[((size_t)blockIdx.y * 2 + which) * P.d + col] = s;
    }
}

template <class O> __device__ __forceinline__ void put(void *p, int64_t i, float v, int add) {
    O *o = static_cast<O *>(p) + i;
    *o = round_to<O>(add ? (float)*o + v : v);
}
// dw and db from n rows of partial sums: a warp's lanes take 32 columns, the CTA's 8 warps each a share of the rows.
__global__ void __launch_bounds__(256) reduce_kernel(const NormBwd P, int n) {
    __shared__ float part[8][32];
    tc::grid_wait_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, all = 2ll * P.d;
    float s = 0.f;
    if (i < all)
#pragma unroll 8
        for (int j = n * warp / 8; j < n * (warp + 1) / 8; ++j) s += P.parts[(size_t)j * all + i];
    part[warp][lane] = s;
    __syncthreads();
    if (warp || i >= all) return;
    const int which = i >= P.d;
    const int64_t c = which ? i - P.d : i;
    void *out = which ? P.db : P.dw;
    if (!out) return;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w][lane];
    if (P.grad_dtype == WASTE_ACT_F32)
        put<float>(out, c, s, P.accumulate);
    else if (P.grad_dtype == WASTE_ACT_BF16)
        put<__nv_bfloat16>(out, c, s, P.accumulate);
    else
        put<__half>(out, c, s, P.accumulate);
}

// f with the two types and the values of a piece as arguments.
template <class F> cudaError_t by_types(int x, int y, bool whole, F f) {
    const auto inner = [&](auto tx) {
        const auto last = [&](auto ty) {
            return whole ? f(tx, ty, std::integral_constant<int, 8>()) : f(tx, ty, std::integral_constant<int, 1>());
        };
        return y == WASTE_ACT_F32 ? last(float()) : y == WASTE_ACT_BF16 ? last(__nv_bfloat16()) : last(__half());
    };
    return x == WASTE_ACT_F32 ? inner(float()) : x == WASTE_ACT_BF16 ? inner(__nv_bfloat16()) : inner(__half());
}
bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
bool whole_rows(const Rows &r, int dtype, int T) {
    return aligned16(r.p) && (T < 2 || r.ld * (int64_t)dense::type_size(dtype) % 16 == 0);
}

// Rows of `bytes` a group keeps on their way beside `rest` bytes in shared memory, those in work among them.  In the backward
// twice kRowsAtOnce and more, which the order of its places needs (fp32: rows of x and dy are 64 KB for 16 warps, beside 32 KB
// of w).  In the forward one and more, read to registers before its place takes the next (fp32: 24 warps' rows are up to
// 96 KB beside up to 64 KB of w and b, so rows of 4024 to 4096, 5640 to 6144 and 7048 values on have none ahead).
int rows_ahead(size_t bytes, size_t rest, int groups) {
    const size_t n = (kHeldSmem - rest) / (bytes * groups);
    return n > kDeepMost ? kDeepMost : (int)n;
}
// Pieces of eight columns of a row, as many as there are where they begin anywhere; whether all lanes hold them.
int eights(int d, bool whole) { return whole ? d / 8 : (d + 14) / 8; }
bool at_once(int d, bool whole) { return eights(d, whole) * 8 <= kHeldMost; }
constexpr int kFewRows = 4; // an SM
// Warps of a group for a row of `pieces` pieces.
int group_warps(int pieces, int per_lane) { return (pieces + 32 * per_lane - 1) / (32 * per_lane); }
cudaError_t reduce(const NormBwd &P, int n, cudaStream_t s) {
    return launch_behind(reduce_kernel, dim3((unsigned)((2ll * P.d + 31) / 32)), dim3(256), 0, s, P, n);
}

} // namespace

cudaError_t launch_norm_forward(const NormFwd &P, cudaStream_t s) {
    const bool whole = P.d % 8 == 0 && aligned16(P.w) && aligned16(P.b) && whole_rows(P.x, P.x_dtype, P.T) &&
                       whole_rows(P.y, P.y_dtype, P.T);
    return by_types(P.x_dtype, P.y_dtype, whole, [&](auto x, auto y, auto v) {
        using X = decltype(x);
        using Y = decltype(y);
        constexpr int V = decltype(v)::value;
        const int pieces = P.d / V + (P.d % V != 0), sms = device_sm_count();
        if (P.d <= kHeldMost) {
            if (P.T > kFewRows * sms && at_once(P.d, V == 8)) {
                static SmemAttr attr;
                const auto kernel = forward_stream_kernel<X, Y, V>;
                const int gw = group_warps(eights(P.d, V == 8), kStreamHeld / 8);
                const int groups = kStreamThreads / 32 / gw; // 12 at most where a group has barriers
                const size_t row = ring_pitch(P.d, sizeof(X), V == 8), rest = V == 8 ? (size_t)P.d * 8 : (size_t)eighths(P.d) * 64;
                const int deep = rows_ahead(row, rest, groups), smem = (int)(deep * groups * row + rest);
                const cudaError_t e = ensure_smem(attr, reinterpret_cast<const void *>(kernel), smem);
                if (e != cudaSuccess) return e;
                const int blocks = (P.T + groups - 1) / groups;
                return launch_behind(kernel, dim3(blocks < sms ? blocks : sms), dim3(groups * gw * 32), smem, s, P, gw, deep);
            }
            const int gw = group_warps(pieces, kHeld / V), most = kHeldThreads / 32 / gw;
            int groups = (P.T + sms - 1) / sms; // as many CTAs as there are SMs before several groups a CTA
            if (groups > most) groups = most;
            const int blocks = (P.T + groups - 1) / groups;
            return launch_behind(forward_few_kernel<X, Y, V>, dim3(blocks < 4 * sms ? blocks : 4 * sms), dim3(groups * gw * 32), 0, s, P, gw);
        }
        return launch_behind(forward_kernel<X, Y, V>, dim3(P.T < 4 * sms ? P.T : 4 * sms), dim3(kThreads), 0, s, P, kThreads / 32);
    });
}

cudaError_t launch_norm_backward(const NormBwd &P, cudaStream_t s) {
    const bool whole = P.d % 8 == 0 && aligned16(P.w) && whole_rows(P.x, P.x_dtype, P.T) && whole_rows(P.dy, P.y_dtype, P.T) &&
                       (!P.dx.p || whole_rows(P.dx, P.x_dtype, P.T));
    return by_types(P.x_dtype, P.y_dtype, whole, [&](auto x, auto y, auto v) {
        using X = decltype(x);
        using Y = decltype(y);
        constexpr int V = decltype(v)::value;
        const int pieces = P.d / V + (P.d % V != 0), sms = device_sm_count();
        const bool sums = P.dw || P.db;
        cudaError_t e = cudaSuccess;
        if (at_once(P.d, V == 8)) {
            const int gw = group_warps(eights(P.d, V == 8), kHeld / 8);
            int groups = kHeldThreads / 32 / gw, need = (P.T + sms - 1) / sms;
            if (groups > need) groups = need; // 8 at most where a group has barriers
            const int threads = groups * gw * 32, most = sms < kNormParts ? sms : kNormParts, all = (P.T + groups - 1) / groups;
            const int blocks = all < most ? all : most;
            const auto launch = [&](auto full) {
                constexpr bool kFull = decltype(full)::value;
                static SmemAttr attr;
                const auto kernel = backward_held_kernel<X, Y, V, kFull>;
                const size_t row = ring_pitch(P.d, sizeof(X), V == 8) + ring_pitch(P.d, sizeof(Y), V == 8), rest = V == 8 ? (size_t)P.d * 4 : (size_t)eighths(P.d) * 32;
                const int deep = rows_ahead(row, rest, groups), last = groups > 1 ? groups * P.d * 8 : 0;
                const int ring = (int)(deep * groups * row + rest), smem = ring > last ? ring : last;
                const cudaError_t f = ensure_smem(attr, reinterpret_cast<const void *>(kernel), smem);
                return f == cudaSuccess ? launch_behind(kernel, dim3(blocks), dim3(threads), smem, s, P, gw, deep) : f;
            };
            if (V == 8 && P.d == gw * 32 * kHeld) {
                if constexpr (V == 8) e = launch(std::true_type());
            } else {
                e = launch(std::false_type());
            }
            return e == cudaSuccess && sums ? reduce(P, blocks, s) : e;
        }
        if (sums) { // before dx, which may take dy's place
            const int across = (pieces + 31) / 32;
            int down = (4 * sms + across - 1) / across, most = (P.T + 15) / 16;
            if (most > kNormParts) most = kNormParts;
            if (down > most) down = most;
            e = launch_behind(columns_kernel<X, Y, V>, dim3(across, down), dim3(kThreads), 0, s, P);
            if (e == cudaSuccess) e = reduce(P, down, s);
        }
        if (e != cudaSuccess || !P.dx.p) return e;
        return launch_behind(dx_kernel<X, Y, V>, dim3(P.T < 4 * sms ? P.T : 4 * sms), dim3(kThreads), 0, s, P, kThreads / 32);
    });
}

cudaError_t norm_word(uint32_t **word) { return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_norm_timeout); }
cudaError_t norm_timeout(uint32_t *out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_timeout, sizeof v);
    const uint32_t zero = 0;
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_norm_timeout, &zero, sizeof zero);
    *out |= v;
    return e;
}

} // namespace train
} // namespace wm
