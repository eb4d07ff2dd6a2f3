// Microscaled 4-bit matrices: quantisation and its inverse.
#include "dense.cuh"

namespace wm {
namespace dense {

namespace {

template <class T> __device__ __forceinline__ float to_f(T v) { return (float)v; }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// One thread per block of 32 values; scale tiles are written whole, zero past the end.
template <class T>
__global__ void __launch_bounds__(256) quantize_kernel(const T *__restrict__ x, int rows, int cols, int64_t ld,
                                                       uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const int kb = (cols + 127) / 128, nb = cols / kMxBlock;
    const size_t total = (size_t)((rows + 127) / 128) * 128 * kb * 4;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
        const int row = (int)(i / (kb * 4)), b = (int)(i % (kb * 4));
        uint8_t *sp = scales + mx_scale_at(row, b, kb);
        if (row >= rows || b >= nb) {
            *sp = 0;
            continue;
        }
        const T *p = x + (size_t)row * ld + (size_t)b * kMxBlock;
        float v[kMxBlock];
#pragma unroll
        for (int j = 0; j < kMxBlock; ++j) v[j] = to_f(p[j]);
        uint32_t w[4];
        *sp = mx_quantize(v, w);
        *reinterpret_cast<uint4 *>(codes + (size_t)row * (cols / 2) + b * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <class T>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales, int rows, int cols,
                                                         T *__restrict__ out, int64_t ld) {
    const int kb = (cols + 127) / 128, nb = cols / kMxBlock;
    const size_t total = (size_t)rows * nb;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
        const int row = (int)(i / nb), b = (int)(i % nb);
        const float s = mx_scale(scales[mx_scale_at(row, b, kb)]);
        const uint4 c = *reinterpret_cast<const uint4 *>(codes + (size_t)row * (cols / 2) + b * 16);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        T *p = out + (size_t)row * ld + (size_t)b * kMxBlock;
#pragma unroll
        for (int j = 0; j < kMxBlock; ++j) p[j] = from_f<T>(mx_value(w[j >> 3] >> (4 * (j & 7))) * s);
    }
}

int grid_for(size_t n) {
    const size_t g = (n + 255) / 256, most = (size_t)device_sm_count() * 16;
    return (int)(g < most ? g : most);
}

} // namespace

cudaError_t launch_mx4_quantize(const void *x, int dtype, int rows, int cols, int64_t ld, uint8_t *codes,
                                uint8_t *scales, cudaStream_t s) {
    const int g = grid_for((size_t)((rows + 127) / 128) * 128 * ((cols + 127) / 128) * 4);
    if (dtype == WASTE_ACT_F32)
        quantize_kernel<<<g, 256, 0, s>>>(static_cast<const float *>(x), rows, cols, ld, codes, scales);
    else if (dtype == WASTE_ACT_BF16)
        quantize_kernel<<<g, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(x), rows, cols, ld, codes, scales);
    else
        quantize_kernel<<<g, 256, 0, s>>>(static_cast<const __half *>(x), rows, cols, ld, codes, scales);
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const Mx4Mat &m, void *out, int dtype, int64_t ld, cudaStream_t s) {
    const int g = grid_for((size_t)m.rows * (m.cols / kMxBlock));
    if (dtype == WASTE_ACT_F32)
        dequantize_kernel<<<g, 256, 0, s>>>(m.codes, m.scales, m.rows, m.cols, static_cast<float *>(out), ld);
    else if (dtype == WASTE_ACT_BF16)
        dequantize_kernel<<<g, 256, 0, s>>>(m.codes, m.scales, m.rows, m.cols, static_cast<__nv_bfloat16 *>(out), ld);
    else
        dequantize_kernel<<<g, 256, 0, s>>>(m.codes, m.scales, m.rows, m.cols, static_cast<__half *>(out), ld);
    return cudaGetLastError();
}

} // namespace dense
} // namespace wm
