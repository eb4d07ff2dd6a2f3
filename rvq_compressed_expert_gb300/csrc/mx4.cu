// Microscaled 4-bit matrices: quantisation and its inverse.
//
// Both are one pass, bound by memory once the instructions per value are few: a value is read once
// (2 or 4 bytes), its 4-bit code and its share of a scale byte (1/32) written, or the other way
// round.  A warp's accesses are whole lines of one row, and it walks down the rows, several of them
// in flight at once to cover the memory's latency.
//
// quantize: a lane takes 16 consecutive values, so a block is two neighbouring lanes, its largest
// magnitude one shuffle away, and the four scale bytes that stand together in a scale tile are
// gathered by two more into one word.  With 8 values a lane the work per block is spread over twice
// the lanes: 66.4 us against 46.6 us (6.4 TB/s) for 16383 x 7168 bf16.
// dequantize: a lane makes 16 bytes of output, so that every store instruction of a warp is
// contiguous: 48.8 us for the same matrix (6.1 TB/s), 59.4 us with 32 bytes a lane.
// The roundings are the hardware's e2m1 conversions.  Loads are ordinary ones, not read-only: the kernel before may
// still write what is read here when this one begins.
#include "dense.cuh"
#include "dense_tc.cuh"

namespace wm {
namespace dense {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 16; // values of a lane (quantize)
constexpr int kRows = 2; // rows of a warp in flight (quantize)

// A lane's values: 16-byte pieces.
template <class T> struct Held {
    static constexpr int kPieces = kPer * (int)sizeof(T) / 16;
    uint4 q[kPieces];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) q[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) reinterpret_cast<uint4 *>(p)[i] = q[i];
    }
    __device__ __forceinline__ uint32_t word(int i) const { return reinterpret_cast<const uint32_t *>(q)[i]; }
    __device__ __forceinline__ uint32_t &word(int i) { return reinterpret_cast<uint32_t *>(q)[i]; }
};

// The largest magnitude's fp32 bits (a NaN's stay a NaN's).
__device__ __forceinline__ uint32_t largest(const Held<float> &a) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) big = max(big, a.word(i) & 0x7fffffffu);
    return big;
}
// 16-bit types: two at a time, NaN kept.
template <class H2> __device__ __forceinline__ H2 largest2(const uint32_t *w) {
    H2 m;
    *reinterpret_cast<uint32_t *>(&m) = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < kPer / 2; ++i) {
        H2 v;
        *reinterpret_cast<uint32_t *>(&v) = w[i] & 0x7fff7fffu;
        m = __hmax2_nan(m, v);
    }
    return m;
}
__device__ __forceinline__ uint32_t largest(const Held<__nv_bfloat16> &a) {
    const __nv_bfloat162 m = largest2<__nv_bfloat162>(reinterpret_cast<const uint32_t *>(a.q));
    return __float_as_uint(__bfloat162float(__hmax_nan(m.x, m.y))) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t largest(const Held<__half> &a) {
    const __half2 m = largest2<__half2>(reinterpret_cast<const uint32_t *>(a.q));
    return __float_as_uint(__half2float(__hmax_nan(m.x, m.y))) & 0x7fffffffu;
}

// Values 8 j .. 8 j + 7.
__device__ __forceinline__ void unpack8(const Held<float> &a, int j, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a.word(8 * j + i));
}
__device__ __forceinline__ void unpack8(const Held<__nv_bfloat16> &a, int j, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a.word(4 * j + i) << 16);
        v[2 * i + 1] = __uint_as_float(a.word(4 * j + i) & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const Held<__half> &a, int j, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = a.word(4 * j + i);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
// A lane's output (dequantize): 16 bytes.
template <class T> struct Out {
    static constexpr int kPer = 8, kRows = 4;
    using Codes = uint32_t;
    static __device__ __forceinline__ uint32_t two(float a, float b, __nv_bfloat16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint32_t two(float a, float b, __half) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint4 make(Codes c, float p) {
        float v[8];
        mx_values8(c, v);
        return make_uint4(two(v[0] * p, v[1] * p, T()), two(v[2] * p, v[3] * p, T()), two(v[4] * p, v[5] * p, T()),
                          two(v[6] * p, v[7] * p, T()));
    }
};
template <> struct Out<float> {
    static constexpr int kPer = 4, kRows = 8;
    using Codes = uint16_t;
    static __device__ __forceinline__ uint4 make(Codes c, float p) {
        float v[8];
        mx_values8(c, v);
        return make_uint4(__float_as_uint(v[0] * p), __float_as_uint(v[1] * p), __float_as_uint(v[2] * p),
                          __float_as_uint(v[3] * p));
    }
};

// Where a warp works: its segment, its first row and the distance to its next.
struct Walk {
    int col, row, step;
};
template <int kLane> __device__ __forceinline__ Walk walk(int cols) {
    const int nseg = (cols + 32 * kLane - 1) / (32 * kLane);
    const int w = blockIdx.x * kWarps + (threadIdx.x >> 5), all = gridDim.x * kWarps;
    Walk k;
    k.col = ((w % nseg) * 32 + (threadIdx.x & 31)) * kLane;
    k.row = w / nseg;
    k.step = all / nseg; // warps past the last whole round have nothing to do
    if (k.row >= k.step) k.row = 0x7fffffff;
    return k;
}

template <class T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T *x, int rows, int cols, int64_t ld, uint8_t *codes,
                                                            uint8_t *scales) {
    const int lane = threadIdx.x & 31, kb = (cols + 127) / 128;
    const Walk K = walk<kPer>(cols);
    const bool in = K.col < cols;
    tc::grid_wait_release();
    for (int64_t r0 = K.row; r0 < rows; r0 += (int64_t)kRows * K.step) {
        Held<T> a[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (in && r < rows) a[i].load(x + r * ld + K.col);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (r >= rows) break;
            uint32_t big = in ? largest(a[i]) : 0;
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            const bool bad = mx_bad(big);
            const int e = mx_exponent(big);
            // blocks past the last column have scale 0
            uint32_t s = in ? (bad ? 255u : (uint32_t)(e + 127)) << (8 * ((lane >> 1) & 3)) : 0u;
            s |= __shfl_xor_sync(0xffffffffu, s, 2);
            s |= __shfl_xor_sync(0xffffffffu, s, 4);
            if ((lane & 7) == 0 && in)
                *reinterpret_cast<uint32_t *>(scales + mx_scale_at((int)r, K.col / kMxBlock, kb)) = s;
            if (in) {
                const float inv = mx_inverse(e);
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[8];
                    unpack8(a[i], j, v);
#pragma unroll
                    for (int l = 0; l < 8; ++l) v[l] *= inv;
                    w[j] = bad ? 0 : mx_codes8(v);
                }
                *reinterpret_cast<uint2 *>(codes + (size_t)r * (cols / 2) + K.col / 2) = make_uint2(w[0], w[1]);
            }
        }
    }
    // the scale words of the last tile's rows past the end
    const int pad = (128 - (rows & 127)) & 127;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < (int64_t)pad * kb; i += (int64_t)gridDim.x * kThreads)
        *reinterpret_cast<uint32_t *>(scales + mx_scale_at(rows + (int)(i / kb), (int)(i % kb) * 4, kb)) = 0;
}

template <class T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t *codes, const uint8_t *scales, int rows,
                                                              int cols, T *out, int64_t ld) {
    constexpr int kLane = Out<T>::kPer, kDeep = Out<T>::kRows;
    using Codes = typename Out<T>::Codes;
    const int kb = (cols + 127) / 128;
    const Walk K = walk<kLane>(cols);
    tc::grid_wait_release();
    if (K.col >= cols) return;
    for (int64_t r0 = K.row; r0 < rows; r0 += (int64_t)kDeep * K.step) {
        Codes w[kDeep];
        uint8_t s[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (r < rows) {
                w[i] = *reinterpret_cast<const Codes *>(codes + (size_t)r * (cols / 2) + K.col / 2);
                s[i] = scales[mx_scale_at((int)r, K.col / kMxBlock, kb)];
            }
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int64_t r = r0 + (int64_t)i * K.step;
            if (r >= rows) break;
            *reinterpret_cast<uint4 *>(out + r * ld + K.col) = Out<T>::make(w[i], mx_scale(s[i]));
        }
    }
}

// Warps for every piece of `lane` x 32 columns and `deep` rows, at most four full rounds of the
// GPU's; extra: words written besides, by all threads.
int grid_for(int rows, int cols, int lane, int deep, int64_t extra) {
    const int64_t nseg = (cols + 32 * lane - 1) / (32 * lane);
    const int64_t need = nseg * (((int64_t)rows + deep - 1) / deep);
    const int64_t most = (int64_t)device_sm_count() * 32;
    int64_t g = (need + kWarps - 1) / kWarps;
    if (g > most) g = most;
    // at least one whole round over a row, and some threads for the rest
    const int64_t least = (nseg + kWarps - 1) / kWarps;
    if (g < least) g = least;
    const int64_t rest = (extra + kThreads - 1) / kThreads;
    if (g < rest) g = rest < device_sm_count() ? rest : (g > device_sm_count() ? g : device_sm_count());
    return (int)g;
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
    const int64_t pad = (int64_t)((128 - (rows & 127)) & 127) * ((cols + 127) / 128);
    return launch(quantize_kernel<T>, grid_for(rows, cols, kPer, kRows, pad), s, static_cast<const T *>(x), rows, cols, ld, codes, scales);
}
template <class T> cudaError_t dequantize(const Mx4Mat &m, void *out, int64_t ld, cudaStream_t s) {
    return launch(dequantize_kernel<T>, grid_for(m.rows, m.cols, Out<T>::kPer, Out<T>::kRows, 0), s, m.codes, m.scales, m.rows, m.cols,
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
