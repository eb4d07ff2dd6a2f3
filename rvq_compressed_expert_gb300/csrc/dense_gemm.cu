// Products of the dense operators: D[m][n] = sum_k A[m][k] B[n][k], fp32 sums.
//
// One kernel for all of them: operands are read through accessors (16-bit matrices in either
// order, microscaled 4-bit matrices), one or two products share the A operand (gate and up), and
// what becomes of the sums is an epilogue functor.  64 x 64 tiles, 16 deep, staged in shared
// memory as fp32; 4 x 4 sums a thread.
#include "dense.cuh"

namespace wm {
namespace dense {

namespace {

constexpr int kTile = 64, kDeep = 16;

template <class T> __device__ __forceinline__ T to_type(float v);
template <> __device__ __forceinline__ float to_type<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half to_type<__half>(float v) { return __float2half_rn(v); }

// Element (row, k) of a matrix stored [rows][K] (kT = false) or [K][rows] (kT = true).
template <class T, bool kT> struct Half {
    const T *p;
    size_t ld;
    int rows;
    __device__ float at(int r, int k) const { return (float)(kT ? p[(size_t)k * ld + r] : p[(size_t)r * ld + k]); }
};
struct Mx4 {
    const uint8_t *codes, *scales;
    int rows, cols, kb;
    __device__ float at(int r, int k) const {
        const uint32_t c = codes[(size_t)r * (cols / 2) + (k >> 1)] >> (4 * (k & 1));
        return mx_value(c) * mx_scale(scales[mx_scale_at(r, k / kMxBlock, kb)]);
    }
};

// kPair: two products with the same A (epilogue gets both sums); kSum: two products added.
enum { kOne, kPair, kSum };

template <int kForm, class A, class B, class E>
__global__ void __launch_bounds__(256) product_kernel(int M, int N, int K, A a, B b, A a2, B b2, E epi) {
    __shared__ float sa[2][kDeep][kTile + 1], sb[2][kDeep][kTile + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    for (int m0 = blockIdx.y * kTile; m0 < M; m0 += gridDim.y * kTile) {
        const int n0 = blockIdx.x * kTile;
        float c[2][4][4] = {};
        for (int k0 = 0; k0 < K; k0 += kDeep) {
            for (int i = tid; i < kTile * kDeep; i += 256) {
                const int k = i % kDeep, r = i / kDeep;
                const bool ka = k0 + k < K, ma = ka && m0 + r < M, na = ka && n0 + r < N;
                sa[0][k][r] = ma ? a.at(m0 + r, k0 + k) : 0.f;
                sb[0][k][r] = na ? b.at(n0 + r, k0 + k) : 0.f;
                if (kForm == kSum) sa[1][k][r] = ma ? a2.at(m0 + r, k0 + k) : 0.f;
                if (kForm != kOne) sb[1][k][r] = na ? b2.at(n0 + r, k0 + k) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kDeep; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        c[0][i][j] = fmaf(sa[0][k][ty + 16 * i], sb[0][k][tx + 16 * j], c[0][i][j]);
                        if (kForm == kPair) c[1][i][j] = fmaf(sa[0][k][ty + 16 * i], sb[1][k][tx + 16 * j], c[1][i][j]);
                        if (kForm == kSum) c[0][i][j] = fmaf(sa[1][k][ty + 16 * i], sb[1][k][tx + 16 * j], c[0][i][j]);
                    }
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m < M && n < N) epi(m, n, c[0][i][j], c[1][i][j]);
            }
    }
}

template <int kForm, class A, class B, class E>
cudaError_t product(int M, int N, int K, A a, B b, A a2, B b2, E epi, cudaStream_t s) {
    const int gy = (M + kTile - 1) / kTile;
    product_kernel<kForm><<<dim3((N + kTile - 1) / kTile, gy < 65535 ? gy : 65535), 256, 0, s>>>(M, N, K, a, b, a2, b2,
                                                                                               epi);
    return cudaGetLastError();
}

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + __expf(-g)); }

template <class O> struct Store {
    O *out;
    size_t ld;
    int add;
    __device__ void operator()(int m, int n, float c, float) const {
        O &o = out[(size_t)m * ld + n];
        o = to_type<O>(add ? (float)o + c : c);
    }
};
// a = silu(g) u; g and u kept if asked for
template <class T, class O> struct Gated {
    O *a;
    T *g, *u;
    size_t ld;
    __device__ void operator()(int m, int n, float cg, float cu) const {
        const size_t i = (size_t)m * ld + n;
        a[i] = to_type<O>(cg * sigmoid(cg) * cu);
        if (g) {
            g[i] = to_type<T>(cg);
            u[i] = to_type<T>(cu);
        }
    }
};
// da -> a, dg, du from the kept g and u
template <class T> struct GatedGrad {
    const T *g, *u;
    T *a, *dg, *du;
    size_t ld;
    __device__ void operator()(int m, int n, float da, float) const {
        const size_t i = (size_t)m * ld + n;
        const float gv = (float)g[i], uv = (float)u[i], s = sigmoid(gv);
        a[i] = to_type<T>(gv * s * uv);
        du[i] = to_type<T>(da * gv * s);
        dg[i] = to_type<T>(da * uv * s * (1.f + gv * (1.f - s)));
    }
};

template <class T, bool kT> Half<T, kT> mat(const void *p, int ld) { return {static_cast<const T *>(p), (size_t)ld, 0}; }

template <class A, class B>
cudaError_t store(int M, int N, int K, A a, B b, void *out, int dtype, int add, cudaStream_t s) {
    if (dtype == WASTE_ACT_F32)
        return product<kOne>(M, N, K, a, b, a, b, Store<float>{static_cast<float *>(out), (size_t)N, add}, s);
    if (dtype == WASTE_ACT_BF16)
        return product<kOne>(M, N, K, a, b, a, b, Store<__nv_bfloat16>{static_cast<__nv_bfloat16 *>(out), (size_t)N, add}, s);
    return product<kOne>(M, N, K, a, b, a, b, Store<__half>{static_cast<__half *>(out), (size_t)N, add}, s);
}

template <class T> cudaError_t forward(const FfnFwd &P, cudaStream_t s) {
    const auto x = mat<T, false>(P.x, P.d);
    cudaError_t e = product<kPair>(P.T, P.f, P.d, x, mat<T, false>(P.wg, P.d), x, mat<T, false>(P.wu, P.d),
                                   Gated<T, T>{static_cast<T *>(P.a), static_cast<T *>(P.g), static_cast<T *>(P.u),
                                               (size_t)P.f}, s);
    if (e != cudaSuccess) return e;
    return store(P.T, P.d, P.f, mat<T, false>(P.a, P.f), mat<T, false>(P.wd, P.f), P.out, P.out_dtype, P.mode, s);
}

template <class T> cudaError_t backward(const FfnBwd &P, cudaStream_t s) {
    const auto dy = mat<T, false>(P.dy, P.d);
    const auto wd = mat<T, true>(P.wd, P.f);
    cudaError_t e = product<kOne>(P.T, P.f, P.d, dy, wd, dy, wd,
                                  GatedGrad<T>{static_cast<const T *>(P.g), static_cast<const T *>(P.u),
                                               static_cast<T *>(P.a), static_cast<T *>(P.dg), static_cast<T *>(P.du),
                                               (size_t)P.f}, s);
    if (e == cudaSuccess && P.dx)
        e = product<kSum>(P.T, P.d, P.f, mat<T, false>(P.dg, P.f), mat<T, true>(P.wg, P.d), mat<T, false>(P.du, P.f),
                          mat<T, true>(P.wu, P.d), Store<T>{static_cast<T *>(P.dx), (size_t)P.d, 0}, s);
    if (!P.dwg) return e;
    const auto xt = mat<T, true>(P.x, P.d);
    if (e == cudaSuccess)
        e = store(P.f, P.d, P.T, mat<T, true>(P.dg, P.f), xt, P.dwg, P.grad_dtype, P.accumulate, s);
    if (e == cudaSuccess)
        e = store(P.f, P.d, P.T, mat<T, true>(P.du, P.f), xt, P.dwu, P.grad_dtype, P.accumulate, s);
    if (e == cudaSuccess)
        e = store(P.d, P.f, P.T, mat<T, true>(P.dy, P.d), mat<T, true>(P.a, P.f), P.dwd, P.grad_dtype, P.accumulate, s);
    return e;
}

Mx4 mx(const Mx4Mat &m) { return {m.codes, m.scales, m.rows, m.cols, (m.cols + 127) / 128}; }

} // namespace

cudaError_t launch_ffn_forward(const FfnFwd &P, cudaStream_t s) {
    return P.dtype == WASTE_ACT_BF16 ? forward<__nv_bfloat16>(P, s) : forward<__half>(P, s);
}

cudaError_t launch_ffn_backward(const FfnBwd &P, cudaStream_t s) {
    return P.dtype == WASTE_ACT_BF16 ? backward<__nv_bfloat16>(P, s) : backward<__half>(P, s);
}

cudaError_t launch_mx4_matmul(const Mx4Mat &a, const Mx4Mat &b, void *out, int out_dtype, int mode, cudaStream_t s) {
    return store(a.rows, b.rows, a.cols, mx(a), mx(b), out, out_dtype, mode, s);
}

size_t mx4_gated_scratch(int T, int f) { return (size_t)T * f * 4; }

cudaError_t launch_mx4_gated(const Mx4Mat &x, const Mx4Mat &gate, const Mx4Mat &up, uint8_t *codes, uint8_t *scales,
                             void *scratch, cudaStream_t s) {
    const int f = gate.rows;
    cudaError_t e = product<kPair>(x.rows, f, x.cols, mx(x), mx(gate), mx(x), mx(up),
                                   Gated<float, float>{static_cast<float *>(scratch), nullptr, nullptr, (size_t)f}, s);
    if (e != cudaSuccess) return e;
    return launch_mx4_quantize(scratch, WASTE_ACT_F32, x.rows, f, f, codes, scales, s);
}

} // namespace dense
} // namespace wm
