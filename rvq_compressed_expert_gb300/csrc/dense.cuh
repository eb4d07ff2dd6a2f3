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
    float *sums;       // and skinny_bytes(T)
};
struct FfnBwd {
    int d, f, T, dtype, grad_dtype, accumulate;
    const void *dy, *x, *g, *u, *wg, *wu, *wd;
    void *dx, *dwg, *dwu, *dwd; // dx or the three dw may be null
    void *a, *dg, *du;          // workspace [T][f] each
    float *sums;                // and skinny_bytes(T)
};
struct Mx4Mat {
    const uint8_t *codes, *scales;
    int rows, cols;
};

// Calls of at most so many tokens take the kernels that read the weights straight into registers
// (dense_gemv.cu); their a is fp32 in the workspace.
constexpr int kGemvTokens = 1;
constexpr int kMxGemvTokens = 2;
// Calls of at most so many tokens keep what rounding a (dg, du) to 16 bits leaves too, and multiply
// both parts: with few tokens the error of a few large values is not averaged out, and the products
// are bound by the weights' way from memory or the gradients' to it.
constexpr int kSplitTokens = 32;
// Calls of at most so many tokens may take the kernel with the weights on the MMA's row side
// (dense_skinny.cuh; an estimate decides there), which splits k over at most so many CTAs; their partial
// sums stand in the workspace.
constexpr int kSkinnyTokens = 208, kSkinnyCtas = 160;
inline int pad_tokens(int T) { return (T + 15) / 16 * 16; }
// Bytes of partial sums for T tokens or fewer.
inline size_t skinny_bytes(int T) {
    const int few = T < kSplitTokens ? T : kSplitTokens, all = T < kSkinnyTokens ? T : kSkinnyTokens;
    const int n = 2 * pad_tokens(few) > pad_tokens(all) ? 2 * pad_tokens(few) : pad_tokens(all);
    return (size_t)kSkinnyCtas * n * 128 * 4;
}
// Shared memory in which those of 4-bit weights stage nt rows of n quantised values.
__host__ __device__ inline size_t mx_gemv_smem(int n, int nt) { return (size_t)nt * (n * 2 + (n / 32 + 15) / 16 * 16); }
constexpr size_t kMxGemvSmem = 48 << 10; // what a kernel may take without asking

cudaError_t launch_ffn_forward(const FfnFwd &P, cudaStream_t s);
cudaError_t launch_ffn_gemv(const FfnFwd &P, cudaStream_t s);
cudaError_t launch_mx4_ffn_gemv(const void *x, int x_dtype, int T, const Mx4Mat &gate, const Mx4Mat &up,
                                const Mx4Mat &down, float *a, void *out, int out_dtype, int mode, cudaStream_t s);
// out = x w^T of one or two rows x, and whether this is the quicker way.
bool mx4_gemv_wins(const Mx4Mat &x, const Mx4Mat &w);
cudaError_t launch_mx4_gemv(const Mx4Mat &x, const Mx4Mat &w, void *out, int out_dtype, int mode, cudaStream_t s);
cudaError_t launch_ffn_backward(const FfnBwd &P, cudaStream_t s);
cudaError_t launch_mx4_quantize(const void *x, int dtype, int rows, int cols, int64_t ld, uint8_t *codes,
                                uint8_t *scales, cudaStream_t s);
cudaError_t launch_mx4_dequantize(const Mx4Mat &m, void *out, int dtype, int64_t ld, cudaStream_t s);
// after_own: the kernel before this one in the stream is one of these operators' and does not write b.
cudaError_t launch_mx4_matmul(const Mx4Mat &a, const Mx4Mat &b, void *out, int out_dtype, int mode, bool after_own,
                              cudaStream_t s);
// a = silu(x gate^T) * (x up^T), quantised into codes and scales ([x.rows][gate.rows]; the scale
// bytes of rows past the end are not written).  Behind launch_mx4_quantize of x; next: the codes
// of the product behind it.
cudaError_t launch_mx4_gated(const Mx4Mat &x, const Mx4Mat &gate, const Mx4Mat &up, const Mx4Mat &next,
                             uint8_t *codes, uint8_t *scales, cudaStream_t s);
// One CTA that waits on a barrier of its own (see waste_dense_debug_wait).
cudaError_t launch_debug_wait(int polls, int arrive, cudaStream_t s);
// *out |= whether a device wait of these kernels gave up since the last call (cleared).
cudaError_t ffn_timeout(uint32_t *out);
cudaError_t mx4_timeout(uint32_t *out);

#ifdef __CUDACC__
// By the approximate exponential and quotient: relative errors of 2^-22 and of the argument's rounding,
// |g| 2^-23: far below what one rounding to 16 or 4 bits behind it leaves, and below the rounding of bf16's two
// parts; in fp32 (one token) and beside fp16's two parts (2^-22) it is the larger error of a.  Below 2^-126 (g < -87.3) the
// quotient is 0, by definition for divisors past 2^126, and so is what is multiplied with it.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// The power of two of a scale byte (2^-127 is a subnormal of fp32); 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// Exponent of a block whose largest magnitude has the fp32 bits `big`: its exponent field is
// floor(log2) + 127 (0 for zero and subnormals).  255 in the field: the block holds an infinity
// or a NaN.
__device__ __forceinline__ int mx_exponent(uint32_t big) { return max(-127, (int)(big >> 23) - 127 - 2); }
__device__ __forceinline__ bool mx_bad(uint32_t big) { return big >= 0x7f800000u; }
// 2^-e: a normal fp32 number for every block exponent (-127 .. 125), so the product with it is
// exact unless it underflows, far below half the smallest code.
__device__ __forceinline__ float mx_inverse(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }
// Eight E2M1 codes (v[0] in the lowest bits): nearest, ties to the even code, past 6 to 6.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}
// Eight codes as halves (exact).
__device__ __forceinline__ void mx_halves8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// The values of eight codes.
__device__ __forceinline__ void mx_values8(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    mx_halves8(w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
// One block held by one thread: its 32 codes and its scale byte.
__device__ __forceinline__ uint8_t mx_quantize(const float (&v)[kMxBlock], uint32_t (&w)[4]) {
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < kMxBlock; ++j) big = max(big, __float_as_uint(v[j]) & 0x7fffffffu);
    const bool bad = mx_bad(big);
    const int e = mx_exponent(big);
    const float inv = mx_inverse(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = v[8 * i + j] * inv;
        w[i] = bad ? 0 : mx_codes8(x);
    }
    return bad ? 255 : (uint8_t)(e + 127);
}
#endif

} // namespace dense
} // namespace wm
