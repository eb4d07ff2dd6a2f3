// Internal declarations of the dense operators (waste_dense.h).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "waste_dense.h"

namespace wm {
namespace dense {

constexpr int kMxBlock = 32;     // values per scale
constexpr int kMxTileRows = 128; // rows of a scale tile
constexpr int kMxTileBytes = 512;

__host__ __device__ inline size_t mx_code_bytes(int rows, int cols) { return (size_t)rows * (cols / 2); }
__host__ __device__ inline size_t mx_scale_bytes(int rows, int cols) {
    return (size_t)((rows + kMxTileRows - 1) / kMxTileRows) * ((cols + 127) / 128) * kMxTileBytes;
}
// Byte of (row, block) in the scale tiles of a matrix with kb = ceil(cols / 128).
__host__ __device__ inline size_t mx_scale_at(int row, int block, int kb) {
    return ((size_t)(row >> 7) * kb + (block >> 2)) * kMxTileBytes + (row & 31) * 16 + ((row & 127) >> 5) * 4 +
           (block & 3);
}

inline size_t type_size(int dtype) { return dtype == WASTE_ACT_F32 ? 4 : 2; }

struct FfnFwd {
    int d, f, T, dtype, out_dtype, mode;
    const void *x, *wg, *wu, *wd;
    void *out, *g, *u; // g, u may be null
    void *a;           // workspace [T][f]
};
struct FfnBwd {
    int d, f, T, dtype, grad_dtype, accumulate;
    const void *dy, *x, *g, *u, *wg, *wu, *wd;
    void *dx, *dwg, *dwu, *dwd; // dx or the three dw may be null
    void *a, *dg, *du;          // workspace [T][f] each
};
struct Mx4Mat {
    const uint8_t *codes, *scales;
    int rows, cols;
};

cudaError_t launch_ffn_forward(const FfnFwd &P, cudaStream_t s);
cudaError_t launch_ffn_backward(const FfnBwd &P, cudaStream_t s);
cudaError_t launch_mx4_quantize(const void *x, int dtype, int rows, int cols, int64_t ld, uint8_t *codes,
                                uint8_t *scales, cudaStream_t s);
cudaError_t launch_mx4_dequantize(const Mx4Mat &m, void *out, int dtype, int64_t ld, cudaStream_t s);
cudaError_t launch_mx4_matmul(const Mx4Mat &a, const Mx4Mat &b, void *out, int out_dtype, int mode, cudaStream_t s);
// a = silu(x gate^T) * (x up^T), quantised into codes and scales ([x.rows][gate.rows]; the scale
// bytes of rows past the end are not written).
cudaError_t launch_mx4_gated(const Mx4Mat &x, const Mx4Mat &gate, const Mx4Mat &up, uint8_t *codes, uint8_t *scales,
                             cudaStream_t s);
// *out |= whether a device wait of these kernels gave up since the last call (cleared).
cudaError_t ffn_timeout(uint32_t *out);
cudaError_t mx4_timeout(uint32_t *out);

#ifdef __CUDACC__
// E2M1 value of a 4-bit code.
__device__ __forceinline__ float mx_value(uint32_t code) {
    const uint32_t n = code & 7u;
    // 0, 0.5 (the only subnormal), then (1 + m / 2) 2^(e - 1)
    const float v = n < 2 ? 0.5f * (float)n : __uint_as_float((((n >> 1) + 126u) << 23) | ((n & 1u) << 22));
    return code & 8u ? -v : v;
}
// The power of two of a scale byte (2^-127 is a subnormal of fp32); 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// Nearest E2M1 magnitude code of x >= 0 (ties to the even code, past 6 to 6): the number of
// borders passed, a border itself going up where the upper code is even.
__device__ __forceinline__ uint32_t mx_round(float x) {
    return (x > 0.25f) + (x >= 0.75f) + (x > 1.25f) + (x >= 1.75f) + (x > 2.5f) + (x >= 3.5f) + (x > 5.f);
}

// One block: its 32 codes (four words, lower columns in lower bits) and its scale byte.
__device__ __forceinline__ uint8_t mx_quantize(const float (&v)[kMxBlock], uint32_t (&w)[4]) {
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < kMxBlock; ++j) big = max(big, __float_as_uint(v[j]) & 0x7fffffffu); // order of magnitudes
    // exponent field of the largest magnitude = floor(log2) + 127 (0: zero or subnormal)
    const int field = (int)(big >> 23);
    const bool bad = field == 255;
    const int e = max(-127, field - 127 - 2);
    w[0] = w[1] = w[2] = w[3] = 0;
    if (!bad) {
#pragma unroll
        for (int j = 0; j < kMxBlock; ++j) {
            const uint32_t c = mx_round(ldexpf(fabsf(v[j]), -e)) | (__float_as_uint(v[j]) >> 31 << 3);
            w[j >> 3] |= c << (4 * (j & 7));
        }
    }
    return bad ? 255 : (uint8_t)(e + 127);
}
#endif

} // namespace dense
} // namespace wm
