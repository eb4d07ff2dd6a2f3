// Layer norm over rows, forward and backward (waste_train.h).
#include <type_traits>

#include "train.cuh"

namespace wm {
namespace train {

namespace {

constexpr int kThreads = 512;

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
// Sum over the warps of a group (gw of them, group `g` of the CTA), in every thread.  slot alternates between
// two halves of part, so one barrier a sum is enough.
__device__ __forceinline__ float group_sum(float v, int gw, int g, float *part, int &slot) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (gw == 1) return v;
    const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - g * gw;
    float *p = part + slot * 16 + g * gw;
    slot ^= 1;
    if (lane == 0) p[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(gw * 32) : "memory");
    v = lane < gw ? p[lane] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
}

// Two sums at once; part: 64 floats.
__device__ __forceinline__ void group_sum2(float &a, float &b, int gw, int g, float *part, int &slot) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (gw == 1) return;
    const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - g * gw;
    float *p = part + slot * 32 + g * gw;
    slot ^= 1;
    if (lane == 0) p[warp] = a, p[16 + warp] = b;
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(gw * 32) : "memory");
    a = lane < gw ? p[lane] : 0.f;
    b = lane < gw ? p[16 + lane] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    a = __shfl_sync(0xffffffffu, a, 0);
    b = __shfl_sync(0xffffffffu, b, 0);
}

// The kernels that read a row once hold it in registers: so many values a lane, of rows up to kHeldMost.  The work is
// bound by the instructions per value before memory is (29 of them took 126 us for 16384 x 7168 bf16, where memory
// needs 70), so values are held and computed in pairs (one instruction for both), a reduction is spread over many
// values a lane, and rows that fill all lanes go without masks.
constexpr int kFwdHeld = 32, kFwdThreads = 256;
constexpr int kBwdHeld = 16, kBwdThreads = 512;
constexpr int kHeldMost = 8192;
static_assert(kFwdHeld * kFwdThreads == kHeldMost && kBwdHeld * kBwdThreads == kHeldMost, "one row a CTA at most");

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

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void close_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_left() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A lane's H values of a row, in H / V pieces a group's width apart.  Whole pieces come through shared memory, each
// lane's own (asynchronous copies need no registers while they are on their way, and no barrier: nobody else
// reads them); single values straight from memory.  kFull: the row fills all lanes.
template <class X, int V, int H, bool kFull> struct Lane {
    static constexpr int kPieces = H / V, kParts = V == 8 ? V * (int)sizeof(X) / 16 : 0;
    static constexpr uint32_t kSlot = kPieces * kParts * 16; // bytes a lane and row
    int t, gt, d;
    uint32_t ring, wide; // this lane's, and 16 bytes for every thread of the CTA
    __device__ Lane(int t_, int gt_, int d_, uint32_t smem) : t(t_), gt(gt_), d(d_), ring(smem + threadIdx.x * 16), wide(blockDim.x * 16) {}
    __device__ __forceinline__ int column(int i) const { return (i * gt + t) * V; }
    __device__ __forceinline__ bool in(int i) const { return kFull || column(i) < d; }
    __device__ __forceinline__ void ask(const X *row, int slot) const {
        if constexpr (V == 8) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if (in(i))
#pragma unroll
                    for (int j = 0; j < kParts; ++j)
                        copy16(ring + ((slot * kPieces + i) * kParts + j) * wide,
                               reinterpret_cast<const char *>(row + column(i)) + 16 * j);
        }
    }
    // zeros past the row's end
    __device__ __forceinline__ void take(const X *row, int slot, float2 (&x)[H / 2]) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (V == 8) {
                Piece<X, V> q;
#pragma unroll
                for (int j = 0; j < kParts; ++j) {
                    uint4 u = {};
                    if (in(i))
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                                     : "r"(ring + ((slot * kPieces + i) * kParts + j) * wide)
                                     : "memory");
                    reinterpret_cast<uint4 *>(&q)[j] = u;
                }
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
    // Whether the two values of pair j are the row's.
    __device__ __forceinline__ bool first(int j) const { return in(2 * j / V); }
    __device__ __forceinline__ bool second(int j) const { return in((2 * j + 1) / V); }
};
// V values of w or b from column c on.
template <class T, int V> __device__ __forceinline__ void widen_all(const void *p, int c, float (&o)[V]) {
    const Piece<T, V> q = load<T, V>(static_cast<const T *>(p) + c);
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = widen(q.v[k]);
}
template <int V> __device__ __forceinline__ void params(const void *p, int dtype, int c, float none, float (&o)[V]) {
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
// A lane's values of w or b, `none` past the row's end too.
template <class T, class L, int H> __device__ __forceinline__ void widen_row(const L &l, const void *p, float none, float2 (&o)[H]) {
    constexpr int n = L::kPieces, V = 2 * H / n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
        if constexpr (V == 8) {
            if (l.in(i)) {
                const Piece<T, V> q = load<T, V>(static_cast<const T *>(p) + l.column(i));
#pragma unroll
                for (int k = 0; k < V / 2; ++k) o[V / 2 * i + k] = widen2(&q.v[2 * k]);
            } else {
#pragma unroll
                for (int k = 0; k < V / 2; ++k) o[V / 2 * i + k] = both(none);
            }
        } else {
            const float v = l.in(i) ? widen(static_cast<const T *>(p)[l.column(i)]) : none;
            if (i & 1)
                o[i / 2].y = v;
            else
                o[i / 2].x = v;
        }
    }
}
template <class L, int H> __device__ __forceinline__ void param_row(const L &l, const void *p, int dtype, float none, float2 (&o)[H]) {
    if (!p) {
#pragma unroll
        for (int k = 0; k < H; ++k) o[k] = both(none);
    } else if (dtype == WASTE_ACT_F32) {
        widen_row<float>(l, p, none, o);
    } else if (dtype == WASTE_ACT_BF16) {
        widen_row<__nv_bfloat16>(l, p, none, o);
    } else {
        widen_row<__half>(l, p, none, o);
    }
}

// Rows on their way to a CTA whose lanes hold so many bytes of one: as many as shared memory has room for.
constexpr int deep(uint32_t bytes, uint32_t most) { return bytes * 4 <= most ? 4 : 3; }
template <class L> constexpr int forward_deep() { return deep(L::kSlot * kFwdThreads, 72 << 10); } // three CTAs an SM, or two
template <class LX, class LY> constexpr int backward_deep() { return deep((LX::kSlot + LY::kSlot) * kBwdThreads, 200 << 10); }

// One pass: a group holds its row in registers, the next rows are on their way.
template <class X, class Y, int V, bool kFull>
__global__ void __launch_bounds__(kFwdThreads, 3) forward_held_kernel(const NormFwd P, int gw) {
    using L = Lane<X, V, kFwdHeld, kFull>;
    constexpr int kDeep = forward_deep<L>(), N = kFwdHeld / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[32];
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    const int64_t step = (int64_t)gridDim.x * groups, row0 = (int64_t)blockIdx.x * groups + g;
    const L lane(t, gt, P.d, tc::smem_u32(smem));
    const auto x_at = [&](int64_t row) { return static_cast<const X *>(P.x.p) + row * P.x.ld; };
#pragma unroll
    for (int i = 0; i < kDeep - 1; ++i) {
        if (row0 + i * step < P.T) lane.ask(x_at(row0 + i * step), i);
        close_copies();
    }
    int slot = 0, turn = 0;
    for (int64_t row = row0; row < P.T; row += step) {
        const int last = turn == 0 ? kDeep - 1 : turn - 1;
        if (row + (kDeep - 1) * step < P.T) lane.ask(x_at(row + (kDeep - 1) * step), last);
        close_copies();
        copies_left<kDeep - 1>();
        float2 x[N], s = both(0.f);
        lane.take(x_at(row), turn, x);
        turn = turn + 1 == kDeep ? 0 : turn + 1;
#pragma unroll
        for (int i = 0; i < N; ++i) s = add2(s, x[i]);
        const float mu = group_sum(s.x + s.y, gw, g, part, slot) * inv;
        s = both(0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = add2(x[i], both(-mu));
            if (!kFull && !lane.first(i)) x[i].x = 0.f;
            if (!kFull && !lane.second(i)) x[i].y = 0.f;
            s = fma2(x[i], x[i], s);
        }
        const float r = 1.f / sqrtf(group_sum(s.x + s.y, gw, g, part, slot) * inv + P.eps);
        Y *y = static_cast<Y *>(P.y.p) + row * P.y.ld;
#pragma unroll
        for (int i = 0; i < L::kPieces; ++i) { // w and b piece by piece: they would not fit beside the row
            if (!lane.in(i)) continue;
            const int c = lane.column(i);
            float w[V], b[V];
            params<V>(P.w, P.w_dtype, c, 1.f, w);
            params<V>(P.b, P.w_dtype, c, 0.f, b);
            if constexpr (V == 8) {
                Piece<Y, V> o;
#pragma unroll
                for (int k = 0; k < V; k += 2)
                    round2(&o.v[k], fma2(mul2(x[(V * i + k) / 2], both(r)), make_float2(w[k], w[k + 1]), make_float2(b[k], b[k + 1])));
                *reinterpret_cast<Piece<Y, V> *>(y + c) = o;
            } else {
                y[c] = round_to<Y>(fmaf((i & 1 ? x[i / 2].y : x[i / 2].x) * r, w[0], b[0]));
            }
        }
        if (P.mean && t == 0) {
            P.mean[row] = mu;
            P.rstd[row] = r;
        }
    }
}

// dx, and a CTA's share of dw and db, in one pass.
template <class X, class Y, int V, bool kFull>
__global__ void __launch_bounds__(kBwdThreads) backward_held_kernel(const NormBwd P, int gw) {
    using LX = Lane<X, V, kBwdHeld, kFull>;
    using LY = Lane<Y, V, kBwdHeld, kFull>;
    constexpr int kDeep = backward_deep<LX, LY>(), N = kBwdHeld / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[64];
    tc::grid_wait_release();
    const int gt = gw * 32, g = threadIdx.x / gt, t = threadIdx.x % gt, groups = blockDim.x / gt;
    const float inv = 1.f / (float)P.d;
    const int64_t step = (int64_t)gridDim.x * groups, row0 = (int64_t)blockIdx.x * groups + g;
    const LX lx(t, gt, P.d, tc::smem_u32(smem));
    const LY ly(t, gt, P.d, tc::smem_u32(smem) + kDeep * LX::kSlot * blockDim.x);
    const auto x_at = [&](int64_t row) { return static_cast<const X *>(P.x.p) + row * P.x.ld; };
    const auto y_at = [&](int64_t row) { return static_cast<const Y *>(P.dy.p) + row * P.dy.ld; };
    const auto ask = [&](int64_t row, int slot) {
        if (row < P.T) {
            lx.ask(x_at(row), slot);
            ly.ask(y_at(row), slot);
        }
        close_copies();
    };
    float2 dw[N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = db[i] = both(0.f);
#pragma unroll
    for (int i = 0; i < kDeep - 1; ++i) ask(row0 + i * step, i);
    float mu_next = 0.f, r_next = 0.f;
    if (row0 < P.T) mu_next = P.mean[row0], r_next = P.rstd[row0];
    int slot = 0, turn = 0;
    for (int64_t row = row0; row < P.T; row += step) {
        const float mu = mu_next, r = r_next;
        if (row + step < P.T) mu_next = P.mean[row + step], r_next = P.rstd[row + step];
        ask(row + (kDeep - 1) * step, turn == 0 ? kDeep - 1 : turn - 1);
        copies_left<kDeep - 1>();
        float2 x[N], e[N], w[N], s1 = both(0.f), s2 = both(0.f);
        param_row(lx, P.w, P.w_dtype, 0.f, w);
        lx.take(x_at(row), turn, x);
        ly.take(y_at(row), turn, e);
        turn = turn + 1 == kDeep ? 0 : turn + 1;
#pragma unroll
        for (int i = 0; i < N; ++i) { // past the row's end dy is zero, so all of these are
            x[i] = mul2(add2(x[i], both(-mu)), both(r));
            dw[i] = fma2(e[i], x[i], dw[i]);
            db[i] = add2(db[i], e[i]);
            if (P.w) e[i] = mul2(e[i], w[i]);
            s1 = add2(s1, e[i]);
            s2 = fma2(e[i], x[i], s2);
        }
        if (P.dx.p) {
            float a = s1.x + s1.y, b = s2.x + s2.y;
            group_sum2(a, b, gw, g, part, slot);
            const float2 c1 = both(-a * inv), c2 = both(-b * inv), rr = both(r);
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = mul2(fma2(x[i], c2, add2(e[i], c1)), rr);
            lx.give(static_cast<X *>(P.dx.p) + row * P.dx.ld, e);
        }
    }
    if (!P.dw && !P.db) return;
    // the groups' sums, one behind another
    copies_left<0>();
    __syncthreads();
    float *sum = reinterpret_cast<float *>(smem);
    for (int j = 0; j < groups; ++j) {
        if (g == j)
#pragma unroll
            for (int i = 0; i < kBwdHeld; ++i) {
                const int c = lx.column(i / V) + i % V;
                if (lx.in(i / V)) {
                    float &vw = i & 1 ? dw[i / 2].y : dw[i / 2].x, &vb = i & 1 ? db[i / 2].y : db[i / 2].x;
                    vw += j ? sum[c] : 0.f;
                    vb += j ? sum[P.d + c] : 0.f;
                    if (j + 1 < groups) {
                        sum[c] = vw;
                        sum[P.d + c] = vb;
                    } else {
                        P.parts[(size_t)blockIdx.x * 2 * P.d + c] = vw;
                        P.parts[((size_t)blockIdx.x * 2 + 1) * P.d + c] = vb;
                    }
                }
            }
        __syncthreads();
    }
}

// Rows longer than that: read again for each step.
template <class X, class Y, int V>
__global__ void __launch_bounds__(kThreads) forward_kernel(const NormFwd P, int gw) {
    __shared__ float part[32];
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
            params<V>(P.w, P.w_dtype, c, 1.f, w);
            params<V>(P.b, P.w_dtype, c, 0.f, b);
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
    __shared__ float part[32];
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
            params<V>(P.w, P.w_dtype, c, 1.f, w);
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
            params<V>(P.w, P.w_dtype, c, 1.f, w);
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

// Warps of a group for a row of `pieces` pieces.
int group_warps(int pieces, int per_lane) { return (pieces + 32 * per_lane - 1) / (32 * per_lane); }
// CTAs of the forward an SM holds, by shared memory.
int held_ctas(int smem) { return smem > 75 << 10 ? 2 : 3; }
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
            const int gw = group_warps(pieces, kFwdHeld / V), groups = kFwdThreads / 32 / gw, threads = groups * gw * 32;
            const auto launch = [&](auto full) {
                using L = Lane<X, V, kFwdHeld, decltype(full)::value>;
                static SmemAttr attr;
                const auto kernel = forward_held_kernel<X, Y, V, decltype(full)::value>;
                const int blocks = (P.T + groups - 1) / groups, smem = forward_deep<L>() * L::kSlot * threads;
                cudaError_t e = ensure_smem(attr, reinterpret_cast<const void *>(kernel), smem);
                if (e != cudaSuccess) return e;
                const int most = held_ctas(smem) * sms;
                return launch_behind(kernel, dim3(blocks < most ? blocks : most), dim3(threads), smem, s, P, gw);
            };
            if constexpr (V == 8)
                if (P.d == gw * 32 * kFwdHeld) return launch(std::true_type());
            return launch(std::false_type());
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
        if (P.d <= kHeldMost) {
            const int gw = group_warps(pieces, kBwdHeld / V), groups = kBwdThreads / 32 / gw, threads = groups * gw * 32;
            const int most = sms < kNormParts ? sms : kNormParts, need = (P.T + groups - 1) / groups;
            const int blocks = need < most ? need : most;
            const auto launch = [&](auto full) {
                constexpr bool kFull = decltype(full)::value;
                using LX = Lane<X, V, kBwdHeld, kFull>;
                using LY = Lane<Y, V, kBwdHeld, kFull>;
                static SmemAttr attr;
                const auto kernel = backward_held_kernel<X, Y, V, kFull>;
                const int ring = backward_deep<LX, LY>() * (LX::kSlot + LY::kSlot) * threads, last = groups > 1 ? P.d * 8 : 0;
                const int smem = ring > last ? ring : last;
                const cudaError_t f = ensure_smem(attr, reinterpret_cast<const void *>(kernel), smem);
                return f == cudaSuccess ? launch_behind(kernel, dim3(blocks), dim3(threads), smem, s, P, gw) : f;
            };
            if (V == 8 && P.d == gw * 32 * kBwdHeld) {
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

} // namespace train
} // namespace wm
