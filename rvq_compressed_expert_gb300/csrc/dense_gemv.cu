// The gated feed-forward block for a few tokens (decode), and the 4-bit product of as many rows: the
// weights are read once, straight into registers, and that reading is all that takes time.
//
// Two launches.  gate_up: one column f of the block, its gate and up rows streamed (16 bytes a lane,
// several pieces in flight) against the tokens' x, added across the lanes, a = silu(g) u written
// in fp32.  down: a warp takes a few rows of Wd against a.  No shared memory
// ring, no tensor memory and no sums across CTAs: what bounds both is memory latency times
// bandwidth, so every SM holds as many loads in flight as its registers allow.  down does not
// depend on gate_up for its weights: it is launched while gate_up runs and asks for its first rows
// before it waits for a.  a never leaves fp32, so only the output is rounded.
//
// Against the tensor cores, d 7168, f 1536, weights from memory: one token of 16 bits 14.8 us here and
// 20.4 there (dense_skinny.cuh), two 25.7 here and 20.4 there; 4-bit weights, one token 9.8 us here
// and 17.0 there, two 15.6, three 20.6, four 22.8 (there 17.0 for all): the multiplications grow with the
// tokens.
#include "dense.cuh"
#include "dense_tc.cuh"

namespace wm {
namespace dense {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kDownRows = 2;

// Weights, streamed once: no place in L1, which keeps x (or a), and from L2 (relaxed at the GPU's scope), where what
// complete kernels wrote is: some are asked for before the kernel's own wait.  Nothing is read by read-only
// loads: these kernels begin while the one before them ends, which may write what they read.
__device__ __forceinline__ uint4 load_stream(const void *p) {
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_stream8(const uint8_t *p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void widen(uint32_t w, float &lo, float &hi, __nv_bfloat16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void widen(uint32_t w, float &lo, float &hi, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x;
    hi = f.y;
}
template <class T> __device__ __forceinline__ void widen8(const uint4 &q, float (&v)[8]) {
    widen(q.x, v[0], v[1], T());
    widen(q.y, v[2], v[3], T());
    widen(q.z, v[4], v[5], T());
    widen(q.w, v[6], v[7], T());
}
__device__ __forceinline__ float add_lanes(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

template <class T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }

template <class O> __device__ __forceinline__ void put(void *out, size_t at, float v, int add) {
    O &o = static_cast<O *>(out)[at];
    o = narrow<O>(add ? (float)o + v : v);
}
__device__ __forceinline__ void put_as(int dtype, void *out, size_t at, float v, int add) {
    if (dtype == WASTE_ACT_F32)
        put<float>(out, at, v, add);
    else if (dtype == WASTE_ACT_BF16)
        put<__nv_bfloat16>(out, at, v, add);
    else
        put<__half>(out, at, v, add);
}

// ---- 16-bit weights, one token ---------------------------------------------------------------

constexpr int kPieces = 4;    // pieces of 256 k of each row in flight in a warp (gate_up)
constexpr int kRowPieces = 6; // the same of each row in down

// A CTA takes one column, its Q warps share the k and meet in shared memory.  Q so that a warp's
// pieces are on the way at once (8 past k = 4096, else 4); small CTAs, so that the SMs stay full
// to the end.  Block of one token, d 7168, f 1536: a column a warp 19.2 us, two columns a CTA with 4
// warps and 7 pieces each 17.1, one column with 4 warps of 7 16.0, 8 warps of 4 15.3; d 2048, f 768:
// 8 warps 5.6, 4 warps 4.9.
template <class T, int Q>
__global__ void __launch_bounds__(Q * 32) gate_up_kernel(const T *x, const T *wg, const T *wu, float *a, T *g, T *u,
                                                         int d, int f) {
    __shared__ float2 sums[Q];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, col = blockIdx.x;
    tc::grid_wait_release();
    const int all = (d + 255) / 256, first = all * part / Q, last = all * (part + 1) / Q;
    float sg = 0.f, su = 0.f;
    const T *pg = wg + (size_t)col * d, *pu = wu + (size_t)col * d;
    for (int p0 = first; p0 < last; p0 += kPieces) {
        uint4 qg[kPieces], qu[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int k = (p0 + i) * 256 + lane * 8;
            const bool in = p0 + i < last && k < d;
            qg[i] = in ? load_stream(pg + k) : make_uint4(0, 0, 0, 0);
            qu[i] = in ? load_stream(pu + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int k = (p0 + i) * 256 + lane * 8;
            if (p0 + i >= last || k >= d) break;
            float vg[8], vu[8], vx[8];
            widen8<T>(qg[i], vg);
            widen8<T>(qu[i], vu);
            widen8<T>(*reinterpret_cast<const uint4 *>(x + k), vx);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sg = fmaf(vg[j], vx[j], sg);
                su = fmaf(vu[j], vx[j], su);
            }
        }
    }
    sg = add_lanes(sg);
    su = add_lanes(su);
    if (lane == 0) sums[part] = make_float2(sg, su);
    __syncthreads();
    if (threadIdx.x) return;
    float cg = 0.f, cu = 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        cg += sums[i].x;
        cu += sums[i].y;
    }
    a[col] = silu(cg) * cu;
    if (g) {
        g[col] = narrow<T>(cg);
        u[col] = narrow<T>(cu);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) down_kernel(const float *a, const T *wd, void *out, int out_dtype, int add,
                                                        int d, int f) {
    const int lane = threadIdx.x & 31, row = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kDownRows;
    float s[kDownRows] = {};
    uint4 q[kDownRows][kRowPieces];
    const auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kRowPieces; ++i)
#pragma unroll
            for (int r = 0; r < kDownRows; ++r) {
                const int k = k0 + 256 * i;
                q[r][i] = k < f && row + r < d ? load_stream(wd + (size_t)(row + r) * f + k) : make_uint4(0, 0, 0, 0);
            }
    };
    fetch(lane * 8); // the kernel before this one made a, not Wd
    tc::grid_wait_release();
    for (int k0 = lane * 8; k0 - lane * 8 < f;) {
#pragma unroll
        for (int i = 0; i < kRowPieces; ++i) {
            const int k = k0 + 256 * i;
            if (k >= f) break;
            const float4 *p = reinterpret_cast<const float4 *>(a + k);
            const float4 y = p[0], z = p[1];
            const float v[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
            for (int r = 0; r < kDownRows; ++r) {
                float w[8];
                widen8<T>(q[r][i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[r] = fmaf(w[j], v[j], s[r]);
            }
        }
        k0 += 256 * kRowPieces;
        if (k0 - lane * 8 < f) fetch(k0);
    }
#pragma unroll
    for (int r = 0; r < kDownRows; ++r) {
        const float y = add_lanes(s[r]);
        if (lane == r && row + r < d) put_as(out_dtype, out, row + r, y, add);
    }
}

template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <class T> cudaError_t forward(const FfnFwd &P, cudaStream_t s) {
    const bool far = P.d > 4096;
    const cudaError_t e =
        launch(far ? gate_up_kernel<T, 8> : gate_up_kernel<T, 4>, P.f, far ? 256 : 128, 0, s,
               static_cast<const T *>(P.x), static_cast<const T *>(P.wg), static_cast<const T *>(P.wu),
               static_cast<float *>(P.a), static_cast<T *>(P.g), static_cast<T *>(P.u), P.d, P.f);
    if (e != cudaSuccess) return e;
    constexpr int kPer = kWarps * kDownRows;
    return launch(down_kernel<T>, (P.d + kPer - 1) / kPer, kThreads, 0, s, static_cast<const float *>(P.a),
                  static_cast<const T *>(P.wd), P.out, P.out_dtype, P.mode, P.d, P.f);
}

// ---- microscaled 4-bit weights ---------------------------------------------------------------
// The same two launches.  x (then a) is quantised by every CTA for itself into shared memory --
// a few thousand values, less than one launch's latency -- as the halves its codes stand for and
// the blocks' exponents.  A lane takes whole blocks of 32: the products of two E2M1 values are
// multiples of 1/4 up to 36, so eight of them add up exactly in an fp16 lane; a block's sum is
// exact and meets its two powers of two in fp32.

constexpr int kMxDownRows = 4;
constexpr int kMxWarps = 8, kMxThreads = kMxWarps * 32;

// A staged row: 16-byte piece j of block b at (j * nb + b), then the scale bytes (mx_gemv_smem).

template <class T> __device__ __forceinline__ void block_of(const T *p, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32 * (int)sizeof(T) / 16; ++i) {
        const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
        if constexpr (sizeof(T) == 4) {
            v[4 * i] = __uint_as_float(q.x), v[4 * i + 1] = __uint_as_float(q.y);
            v[4 * i + 2] = __uint_as_float(q.z), v[4 * i + 3] = __uint_as_float(q.w);
        } else {
            widen(q.x, v[8 * i], v[8 * i + 1], T());
            widen(q.y, v[8 * i + 2], v[8 * i + 3], T());
            widen(q.z, v[8 * i + 4], v[8 * i + 5], T());
            widen(q.w, v[8 * i + 6], v[8 * i + 7], T());
        }
    }
}
template <class T> __device__ __forceinline__ void stage(const T *x, int T_, int n, uint8_t *smem) {
    const int nb = n / 32;
    for (int i = threadIdx.x; i < T_ * nb; i += kMxThreads) {
        const int t = i / nb, b = i - t * nb;
        uint8_t *base = smem + t * mx_gemv_smem(n, 1);
        float v[32];
        block_of(x + (size_t)t * n + b * 32, v);
        uint32_t w[4];
        base[n * 2 + b] = mx_quantize(v, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            mx_halves8(w[j], h);
            reinterpret_cast<uint4 *>(base)[j * nb + b] = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    __syncthreads();
}
// The same of rows that are 4-bit already.
__device__ __forceinline__ void stage_codes(const Mx4Mat &x, uint8_t *smem) {
    const int nb = x.cols / 32, kb = (x.cols + 127) / 128;
    for (int i = threadIdx.x; i < x.rows * nb; i += kMxThreads) {
        const int t = i / nb, b = i - t * nb;
        uint8_t *base = smem + t * mx_gemv_smem(x.cols, 1);
        const uint4 q = reinterpret_cast<const uint4 *>(x.codes + (size_t)t * (x.cols / 2))[b];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        base[x.cols * 2 + b] = x.scales[mx_scale_at(t, b, kb)];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            mx_halves8(w[j], h);
            reinterpret_cast<uint4 *>(base)[j * nb + b] = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    __syncthreads();
}
// Sum of the 32 products of a weight block and a staged block, exact.
__device__ __forceinline__ float dot32(const uint4 &codes, const uint8_t *base, int nb, int b) {
    float s = 0.f;
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        __half2 acc = __float2half2_rn(0.f);
#pragma unroll
        for (int j = 2 * p; j < 2 * p + 2; ++j) {
            uint32_t h[4];
            mx_halves8(w[j], h);
            const uint4 q = reinterpret_cast<const uint4 *>(base)[j * nb + b];
            const uint32_t y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc = __hfma2(*reinterpret_cast<const __half2 *>(&h[i]), *reinterpret_cast<const __half2 *>(&y[i]), acc);
        }
        const float2 f = __half22float2(acc);
        s += f.x + f.y;
    }
    return s;
}
// v 2^(a + b - 254) for two scale bytes, in two steps that stay in range; NaN for byte 255.
__device__ __forceinline__ float scaled(float v, uint32_t a, uint32_t b) {
    const int e = (int)(a + b) - 254, h = e >> 1;
    const float p = __uint_as_float((uint32_t)max(h + 127, 1) << 23);
    const float q = __uint_as_float((uint32_t)max(e - h + 127, 1) << 23);
    v = v * p * q;
    return a == 255u || b == 255u ? __uint_as_float(0x7fc00000u) : v;
}

template <class T, int NT>
__global__ void __launch_bounds__(kMxThreads) mx_gate_up_kernel(const T *x, Mx4Mat wg, Mx4Mat wu, float *a, int T_) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int U = 4;
    const int d = wg.cols, f = wg.rows, nb = d / 32, kb = (d + 127) / 128;
    const int lane = threadIdx.x & 31, col = blockIdx.x * kMxWarps + (threadIdx.x >> 5);
    tc::grid_wait_release();
    uint4 q[2][U];
    uint32_t sc[2][U];
    const auto fetch = [&](int b0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int b = b0 + 32 * i;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const Mx4Mat &W = m ? wu : wg;
                const bool in = b < nb && col < f;
                q[m][i] = in ? load_stream(W.codes + (size_t)col * (d / 2) + b * 16) : make_uint4(0, 0, 0, 0);
                sc[m][i] = in ? load_stream8(W.scales + mx_scale_at(col, b, kb)) : 0;
            }
        }
    };
    fetch(lane); // the first rows are on their way while x is quantised
    stage(x, T_, d, smem);
    if (col >= f) return;
    float sg[NT] = {}, su[NT] = {};
    for (int b0 = lane; b0 < nb;) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int b = b0 + 32 * i;
            if (b >= nb) break;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= T_) break;
                const uint8_t *base = smem + t * mx_gemv_smem(d, 1);
                const uint32_t sx = base[d * 2 + b];
                sg[t] += scaled(dot32(q[0][i], base, nb, b), sx, sc[0][i]);
                su[t] += scaled(dot32(q[1][i], base, nb, b), sx, sc[1][i]);
            }
        }
        b0 += 32 * U;
        if (b0 - lane < nb) fetch(b0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float cg = add_lanes(sg[t]), cu = add_lanes(su[t]);
        if (lane == t && t < T_) a[(size_t)t * f + col] = silu(cg) * cu;
    }
}

// out = x W^T for one or two rows x: fp32 (down: a, quantised here), or 4-bit already.  R rows of W a
// warp, U blocks of each on the way at once in a lane.
template <int NT, int R, int U, bool kQuantised>
__global__ void __launch_bounds__(kMxThreads) mx_rows_kernel(const float *a, Mx4Mat x, Mx4Mat w, void *out,
                                                             int out_dtype, int add, int T_) {
    static_assert(R * NT <= 32, "a lane for each sum");
    extern __shared__ __align__(16) uint8_t smem[];
    const int n = w.cols, rows = w.rows, nb = n / 32, kb = (n + 127) / 128;
    const int lane = threadIdx.x & 31, row = (blockIdx.x * kMxWarps + (threadIdx.x >> 5)) * R;
    uint4 q[R][U];
    uint32_t sc[R][U];
    const auto fetch = [&](int b0) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int b = b0 + 32 * i;
                const bool in = b < nb && row + r < rows;
                q[r][i] = in ? load_stream(w.codes + (size_t)(row + r) * (n / 2) + b * 16) : make_uint4(0, 0, 0, 0);
                sc[r][i] = in ? load_stream8(w.scales + mx_scale_at(row + r, b, kb)) : 0;
            }
    };
    if constexpr (!kQuantised) fetch(lane); // the kernel before this one made a, not W
    tc::grid_wait_release();
    if constexpr (kQuantised) {
        fetch(lane);
        stage_codes(x, smem);
    } else {
        stage(a, T_, n, smem);
    }
    float s[R][NT] = {};
    for (int b0 = lane; b0 < nb;) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int b = b0 + 32 * i;
            if (b >= nb) break;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= T_) break;
                const uint8_t *base = smem + t * mx_gemv_smem(n, 1);
                const uint32_t sx = base[n * 2 + b];
#pragma unroll
                for (int r = 0; r < R; ++r) s[r][t] += scaled(dot32(q[r][i], base, nb, b), sx, sc[r][i]);
            }
        }
        b0 += 32 * U;
        if (b0 - lane < nb) fetch(b0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float y = add_lanes(s[r][t]);
            if (lane == r * NT + t && t < T_ && row + r < rows)
                put_as(out_dtype, out, (size_t)t * rows + row + r, y, add);
        }
}

template <class T, int NT>
cudaError_t mx_forward(const T *x, int T_, const Mx4Mat &gate, const Mx4Mat &up, const Mx4Mat &down, float *a, void *out,
                       int out_dtype, int mode, cudaStream_t s) {
    cudaError_t e = launch(mx_gate_up_kernel<T, NT>, (gate.rows + kMxWarps - 1) / kMxWarps, kMxThreads, (int)mx_gemv_smem(gate.cols, T_), s,
                           x, gate, up, a, T_);
    if (e != cudaSuccess) return e;
    constexpr int kPer = kMxWarps * kMxDownRows;
    return launch(mx_rows_kernel<NT, kMxDownRows, 2, false>, (down.rows + kPer - 1) / kPer, kMxThreads,
                  (int)mx_gemv_smem(down.cols, T_), s, static_cast<const float *>(a), Mx4Mat{}, down, out, out_dtype, mode, T_);
}
template <class T>
cudaError_t mx_forward_any(const void *x, int T_, const Mx4Mat &gate, const Mx4Mat &up, const Mx4Mat &down, float *a,
                           void *out, int out_dtype, int mode, cudaStream_t s) {
    const T *p = static_cast<const T *>(x);
    return T_ == 1 ? mx_forward<T, 1>(p, T_, gate, up, down, a, out, out_dtype, mode, s)
                   : mx_forward<T, 2>(p, T_, gate, up, down, a, out, out_dtype, mode, s);
}

template <int NT, int R, int U>
cudaError_t mx_product(const Mx4Mat &x, const Mx4Mat &w, void *out, int out_dtype, int mode, cudaStream_t s) {
    constexpr int kPer = kMxWarps * R;
    return launch(mx_rows_kernel<NT, R, U, true>, (w.rows + kPer - 1) / kPer, kMxThreads, (int)mx_gemv_smem(w.cols, x.rows), s,
                  static_cast<const float *>(nullptr), x, w, out, out_dtype, mode, x.rows);
}
// Rows of W from which on four of them a warp still give every SM a CTA.
int many_rows() { return kMxWarps * kMxDownRows * device_sm_count(); }

} // namespace

// Products of one or two rows that the multiplications here do not hold up more than the tensor-core
// kernel's setup and exchange would.  Here and there, us (rows x columns x k): 1 x 1536 x 7168 3.7 and
// 7.2, 1 x 7168 x 1536 3.8 and 5.5, 1 x 7168 x 7168 9.7 and 11.4, 1 x 100000 x 2048 30.3 and 28.3; 2 x 1536 x
// 7168 5.2 and 7.2, 2 x 2048 x 2048 2.8 and 5.8, 2 x 7168 x 1536 6.1 and 5.6, 2 x 7168 x 7168 17.8 and 11.1.
bool mx4_gemv_wins(const Mx4Mat &x, const Mx4Mat &w) {
    if (x.rows > kMxGemvTokens || mx_gemv_smem(x.cols, x.rows) > kMxGemvSmem) return false;
    const int64_t values = (int64_t)w.rows * w.cols;
    return x.rows == 1 ? values <= 1 << 27 : values <= 1 << 24 && w.rows < many_rows();
}

cudaError_t launch_mx4_gemv(const Mx4Mat &x, const Mx4Mat &w, void *out, int out_dtype, int mode, cudaStream_t s) {
    return x.rows == 2                 ? mx_product<2, 1, 8>(x, w, out, out_dtype, mode, s)
           : w.rows >= many_rows() ? mx_product<1, kMxDownRows, 2>(x, w, out, out_dtype, mode, s)
                                       : mx_product<1, 1, 8>(x, w, out, out_dtype, mode, s);
}

cudaError_t launch_ffn_gemv(const FfnFwd &P, cudaStream_t s) {
    return P.dtype == WASTE_ACT_BF16 ? forward<__nv_bfloat16>(P, s) : forward<__half>(P, s);
}

cudaError_t launch_mx4_ffn_gemv(const void *x, int x_dtype, int T, const Mx4Mat &gate, const Mx4Mat &up,
                                const Mx4Mat &down, float *a, void *out, int out_dtype, int mode, cudaStream_t s) {
    return x_dtype == WASTE_ACT_F32    ? mx_forward_any<float>(x, T, gate, up, down, a, out, out_dtype, mode, s)
           : x_dtype == WASTE_ACT_BF16 ? mx_forward_any<__nv_bfloat16>(x, T, gate, up, down, a, out, out_dtype, mode, s)
                                       : mx_forward_any<__half>(x, T, gate, up, down, a, out, out_dtype, mode, s);
}

} // namespace dense
} // namespace wm
