// Microscaled 4-bit matrices: quantisation and its inverse.
//
// Both are one pass, bound by memory: a value is read once (2 or 4 bytes), its 4-bit code and its
// share of a scale byte (1/32) written, or the other way round.  A lane takes 8 consecutive
// values, so a warp's accesses are whole lines of one row (256 columns) and a block is four
// neighbouring lanes: its largest magnitude is two shuffles away, and the four scale bytes that
// stand together in a scale tile are gathered by two more into one word.  The roundings are the
// hardware's e2m1 conversions.  A warp keeps its 256 columns and walks down the rows, kRows of
// them in flight at once to cover the memory's latency.
#include "dense.cuh"
#include "dense_tc.cuh"

namespace wm {
namespace dense {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSegment = 256; // columns of a warp
constexpr int kRows = 4;      // rows of a warp in flight

// 8 consecutive values: one or two 16-byte pieces.
template <class T> struct Eight {
    uint4 q[sizeof(T) / 2];
};
template <class T> __device__ __forceinline__ Eight<T> load8(const T *p) {
    Eight<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}
template <class T> __device__ __forceinline__ void store8(T *p, const Eight<T> &v) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = v.q[i];
}
__device__ __forceinline__ void unpack8(const Eight<float> &a, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<const float *>(a.q)[i];
}
__device__ __forceinline__ void unpack8(const Eight<__nv_bfloat16> &a, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.q)[i]);
}
__device__ __forceinline__ void unpack8(const Eight<__half> &a, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __half2float(reinterpret_cast<const __half *>(a.q)[i]);
}
__device__ __forceinline__ void pack8(const float (&v)[8], Eight<float> &a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) reinterpret_cast<float *>(a.q)[i] = v[i];
}
__device__ __forceinline__ void pack8(const float (&v)[8], Eight<__nv_bfloat16> &a) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<__nv_bfloat162 *>(a.q)[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void pack8(const float (&v)[8], Eight<__half> &a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<__half2 *>(a.q)[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
}

// Where a warp works: its segment, its first row and the distance to its next.
struct Walk {
    int col, row, step;
};
__device__ __forceinline__ Walk walk(int cols) {
    const int nseg = (cols + kSegment - 1) / kSegment;
    const int w = blockIdx.x * kWarps + (threadIdx.x >> 5), all = gridDim.x * kWarps;
    Walk k;
    k.col = (w % nseg) * kSegment + (threadIdx.x & 31) * 8;
    k.row = w / nseg;
    k.step = all / nseg; // warps past the last whole round have nothing to do
    if (k.row >= k.step) k.row = 0x7fffffff;
    return k;
}

template <class T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T *__restrict__ x, int rows, int cols, int64_t ld,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const int lane = threadIdx.x & 31, kb = (cols + 127) / 128;
    const Walk K = walk(cols);
    const bool in = K.col < cols;
    tc::grid_wait();
    tc::grid_release();
    for (int64_t r0 = K.row; r0 < rows; r0 += (int64_t)kRows * K.step) {
        Eight<T> a[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (in && r < rows) a[i] = load8(x + r * ld + K.col);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (r >= rows) break;
            float v[8];
            uint32_t big = 0;
            if (in) {
                unpack8(a[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) big = max(big, __float_as_uint(v[j]) & 0x7fffffffu);
            }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const bool bad = mx_bad(big);
            const int e = mx_exponent(big);
            // blocks past the last column have scale 0
            uint32_t s = in ? (bad ? 255u : (uint32_t)(e + 127)) << (8 * ((lane >> 2) & 3)) : 0u;
            s |= __shfl_xor_sync(0xffffffffu, s, 4);
            s |= __shfl_xor_sync(0xffffffffu, s, 8);
            if ((lane & 15) == 0 && in)
                *reinterpret_cast<uint32_t *>(scales + mx_scale_at((int)r, K.col / kMxBlock, kb)) = s;
            if (in) {
                const float inv = mx_inverse(e);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= inv;
                *reinterpret_cast<uint32_t *>(codes + (size_t)r * (cols / 2) + K.col / 2) = bad ? 0 : mx_codes8(v);
            }
        }
    }
    // the scale words of the last tile's rows past the end
    const int pad = (128 - (rows & 127)) & 127;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)pad * kb; i += (int64_t)gridDim.x * kThreads)
        *reinterpret_cast<uint32_t *>(scales + mx_scale_at(rows + (int)(i / kb), (int)(i % kb) * 4, kb)) = 0;
}

template <class T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int rows, int cols,
                                                              T *__restrict__ out, int64_t ld) {
    const int kb = (cols + 127) / 128;
    const Walk K = walk(cols);
    tc::grid_wait();
    tc::grid_release();
    if (K.col >= cols) return;
    for (int64_t r0 = K.row; r0 < rows; r0 += (int64_t)kRows * K.step) {
        uint32_t w[kRows];
        uint8_t s[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (r < rows) {
                w[i] = __ldg(reinterpret_cast<const uint32_t *>(codes + (size_t)r * (cols / 2) + K.col / 2));
                s[i] = __ldg(scales + mx_scale_at((int)r, K.col / kMxBlock, kb));
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (r >= rows) break;
            float v[8];
            mx_values8(w[i], v);
            const float p = mx_scale(s[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= p;
            Eight<T> a;
            pack8(v, a);
            store8(out + r * ld + K.col, a);
        }
    }
}

// Warps for every (segment, kRows rows), at most four full rounds of the GPU's.
int grid_for(int rows, int cols) {
    const int64_t nseg = (cols + kSegment - 1) / kSegment;
    const int64_t need = nseg * (((int64_t)rows + kRows - 1) / kRows);
    const int64_t most = (int64_t)device_sm_count() * 32;
    int64_t g = (need + kWarps - 1) / kWarps;
    if (g > most) g = most;
    // at least one whole round over a row
    const int64_t least = (nseg + kWarps - 1) / kWarps;
    return (int)(g < least ? least : g);
}

// A launch that may begin while the kernel before it ends (the kernels wait for it themselves).
template <class... P, class... A> cudaError_t launch(void (*kernel)(P...), int grid, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <class T>
cudaError_t quantize(const void *x, int rows, int cols, int64_t ld, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    return launch(quantize_kernel<T>, grid_for(rows, cols), s, static_cast<const T *>(x), rows, cols, ld, codes, scales);
}
template <class T> cudaError_t dequantize(const Mx4Mat &m, void *out, int64_t ld, cudaStream_t s) {
    return launch(dequantize_kernel<T>, grid_for(m.rows, m.cols), s, m.codes, m.scales, m.rows, m.cols,
                  static_cast<T *>(out), ld);
}

} // namespace

cudaError_t launch_mx4_quantize(const void *x, int dtype, int rows, int cols, int64_t ld, uint8_t *codes,
                                uint8_t *scales, cudaStream_t s) {
    return dtype == WASTE_ACT_F32    ? quantize<float>(x, rows, cols, ld, codes, scales, s)
           : dtype == WASTE_ACT_BF16 ? quantize<__nv_bfloat16>(x, rows, cols, ld, codes, scales, s)
                                     : quantize<__half>(x, rows, cols, ld, codes, scales, s);
}

cudaError_t launch_mx4_dequantize(const Mx4Mat &m, void *out, int dtype, int64_t ld, cudaStream_t s) {
    return dtype == WASTE_ACT_F32    ? dequantize<float>(m, out, ld, s)
           : dtype == WASTE_ACT_BF16 ? dequantize<__nv_bfloat16>(m, out, ld, s)
                                     : dequantize<__half>(m, out, ld, s);
}

} // namespace dense
} // namespace wm
