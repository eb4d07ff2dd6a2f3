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
// Value i of w or b (a uniform switch over the type), `none` where there is none.
__device__ __forceinline__ float param(const void *p, int dtype, int i, float none) {
    if (!p) return none;
    if (dtype == WASTE_ACT_F32) return static_cast<const float *>(p)[i];
    if (dtype == WASTE_ACT_BF16) return (float)static_cast<const __nv_bfloat16 *>(p)[i];
    return (float)static_cast<const __half *>(p)[i];
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
#pragma unroll
            for (int i = 0; i < V; ++i)
                o.v[i] = round_to<Y>(fmaf((widen(q.v[i]) - mu) * r, param(P.w, P.w_dtype, c + i, 1.f),
                                          param(P.b, P.w_dtype, c + i, 0.f)));
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
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gv = widen(e.v[i]) * param(P.w, P.w_dtype, c + i, 1.f);
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
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (widen(q.v[i]) - mu) * r, gv = widen(e.v[i]) * param(P.w, P.w_dtype, c + i, 1.f);
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
// dw and db from n rows of partial sums, in their order.
__global__ void __launch_bounds__(256) reduce_kernel(const NormBwd P, int n) {
    tc::grid_wait_release();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= 2ll * P.d) return;
    const int which = i >= P.d;
    const int64_t c = which ? i - P.d : i;
    void *out = which ? P.db : P.dw;
    if (!out) return;
    float s = 0.f;
    for (int j = 0; j < n; ++j) s += P.parts[(size_t)j * 2 * P.d + i];
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
bool whole_rows(const Rows &r, int dtype, int T) {
    return ((uintptr_t)r.p & 15) == 0 && (T < 2 || r.ld * (int64_t)dense::type_size(dtype) % 16 == 0);
}

} // namespace

cudaError_t launch_norm_forward(const NormFwd &P, cudaStream_t s) {
    const bool whole = P.d % 8 == 0 && whole_rows(P.x, P.x_dtype, P.T) && whole_rows(P.y, P.y_dtype, P.T);
    return by_types(P.x_dtype, P.y_dtype, whole, [&](auto x, auto y, auto v) {
        constexpr int V = decltype(v)::value;
        const int pieces = P.d / V + (P.d % V != 0);
        int gw = 1;
        while (gw < kThreads / 32 && gw * 64 < pieces) gw *= 2;
        const int groups = kThreads / 32 / gw, blocks = (P.T + groups - 1) / groups, most = 4 * device_sm_count();
        return launch_behind(forward_kernel<decltype(x), decltype(y), V>, dim3(blocks < most ? blocks : most), dim3(kThreads), 0,
                             s, P, gw);
    });
}

cudaError_t launch_norm_backward(const NormBwd &P, cudaStream_t s) {
    const bool whole = P.d % 8 == 0 && whole_rows(P.x, P.x_dtype, P.T) && whole_rows(P.dy, P.y_dtype, P.T) &&
                       (!P.dx.p || whole_rows(P.dx, P.x_dtype, P.T));
    return by_types(P.x_dtype, P.y_dtype, whole, [&](auto x, auto y, auto v) {
        constexpr int V = decltype(v)::value;
        const int pieces = P.d / V + (P.d % V != 0), sms = device_sm_count();
        cudaError_t e = cudaSuccess;
        if (P.dw || P.db) { // before dx, which may take dy's place
            const int across = (pieces + 31) / 32;
            int down = (4 * sms + across - 1) / across, most = (P.T + 15) / 16;
            if (most > kNormParts) most = kNormParts;
            if (down > most) down = most;
            e = launch_behind(columns_kernel<decltype(x), decltype(y), V>, dim3(across, down), dim3(kThreads), 0, s, P);
            if (e == cudaSuccess) e = launch_behind(reduce_kernel, dim3((unsigned)((2ll * P.d + 255) / 256)), dim3(256), 0, s, P, down);
        }
        if (e != cudaSuccess || !P.dx.p) return e;
        int gw = 1;
        while (gw < kThreads / 32 && gw * 64 < pieces) gw *= 2;
        const int groups = kThreads / 32 / gw, blocks = (P.T + groups - 1) / groups, most = 4 * sms;
        return launch_behind(dx_kernel<decltype(x), decltype(y), V>, dim3(blocks < most ? blocks : most), dim3(kThreads), 0, s, P,
                             gw);
    });
}

} // namespace train
} // namespace wm
