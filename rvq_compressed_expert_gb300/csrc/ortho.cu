// Updates made orthogonal by Newton-Schulz products (waste_train.h).
//
// X holds 2^10 times its value in two fp16 parts, hi + lo; products take hi and sum in fp32.  The factor keeps what is
// small (A starts with entries of 1e-5 and less) above fp16's subnormals and what is large (62 at most, checked for the coefficients) in its range.
// With hi alone the error of one rounding stays in X: for a gradient of low rank it lies outside the rank's space, where
// every step makes it 3.4 times larger (4 % for rank 8, 15 % for rank 1).  B = b A + c A^2 keeps its diagonal apart
// in fp32: near the end it is the largest part of B, and its rounding would be the largest error (1.7e-3 with
// it in fp16, 0.9e-3 without, G Gaussian).  The diagonal multiplies hi while noise can still grow, so that
// B X stays in X's space, and hi + lo in the last step but one.  The last step takes hi alone: what its rounding leaves
// is not multiplied by a step any more.
//
// A step is three products: A = X X^T (its tiles on and below the diagonal, the long side in shares, partial sums added by
// gram_kernel, or a tile at once where shares would cost more than they save), B from A^2, and X from B X, whose epilogue reads and writes both parts of X.  Small matrices do all steps in
// one launch (the last step included, with both parts of X).  Measured: 1536 x 7168 bf16 382 to 391 us (floor 143 us of MMAs: 272 GFLOP; by launch, cold and one
// by one, a step: A 21 us, its sum 10, B 14, X 30 to 35; G's norm and start 23), four 7168 x 1536 fp32 added to bf16 weights
// 1.17 to 1.25 ms (floor 571: a step's A 62 us, its sum 14, B 27, X 102 to 130, whose floor is 70: its epilogue's 350 MB go past
// what L2 holds; A is 168 items on 76 pairs, three waves, for a floor of 36; norm and start 87), eight 128 x 256 33 us in one
// launch of 15 products.
#include <type_traits>

#include "tile_mma.cuh"

namespace wm {
namespace train {

namespace {

constexpr float kUp = 1024.f, kDown = 1.f / 1024.f;
constexpr int kFlat = 256; // threads of the kernels that are not products

template <class T, int V> struct alignas(V == 8 ? 16 : sizeof(T)) Piece {
    T v[V];
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A sum over the CTA, in thread 0; part: a float a warp.
__device__ __forceinline__ float block_sum(float v, float *part) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < (int)blockDim.x / 32; ++w) v += part[w];
    return v;
}

// Sum of squares of the values that each(f) hands to f (every thread its own, the same each time), in three ranges so
// that none leaves fp32: below 2^-45 times 2^80, past 2^45 times 2^-80, and the rest (NaN among it); in thread 0.  Where
// the CTA's largest magnitude is in the middle range one sum of all is enough: what underflows there is nothing
// beside it.
template <class F> __device__ __forceinline__ void squares_of(const F &each, float *part, float (&s)[3]) {
    float most = 0.f;
    s[0] = s[1] = s[2] = 0.f;
    each([&](float v) {
        most = fmaxf(most, fabsf(v));
        s[2] = fmaf(v, v, s[2]);
    });
    const bool far = __syncthreads_or(most > 0x1p45f), some = __syncthreads_or(most >= 0x1p-45f);
    if (far || !some) {
        s[2] = 0.f;
        each([&](float v) {
            const float m = fabsf(v), up = v * 0x1p80f, down = v * 0x1p-80f;
            if (m < 0x1p-45f)
                s[0] = fmaf(up, up, s[0]);
            else if (m > 0x1p45f)
                s[1] = fmaf(down, down, s[1]);
            else
                s[2] = fmaf(v, v, s[2]);
        });
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] = block_sum(s[k], part);
}

// Of each matrix (`size` values, in pieces of V): sums [count][kOrthoParts][3].
template <class T, int V>
__global__ void __launch_bounds__(kFlat) squares_kernel(const T *g, int64_t size, float *sums) {
    __shared__ float part[kFlat / 32];
    tc::grid_wait_release();
    const int64_t n = size / V, i0 = n * blockIdx.x / kOrthoParts, i1 = n * (blockIdx.x + 1) / kOrthoParts;
    const Piece<T, V> *p = reinterpret_cast<const Piece<T, V> *>(g + (size_t)blockIdx.y * size);
    float s[3];
    squares_of(
        [&](auto f) {
#pragma unroll 4
            for (int64_t i = i0 + threadIdx.x; i < i1; i += kFlat) {
                const Piece<T, V> q = p[i];
#pragma unroll
                for (int k = 0; k < V; ++k) f((float)q.v[k]);
            }
        },
        part, s);
    if (threadIdx.x < 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) sums[((size_t)blockIdx.y * kOrthoParts + blockIdx.x) * 3 + k] = s[k];
}

// What G is multiplied with: |G| = f 2^e, 1/2 <= f < 2, so by two exact powers of two, then by 2^10 / f.
struct Factor {
    float a, b, f;
    __device__ __forceinline__ float operator()(float v) const { return v * a * b * f; }
};
__device__ __forceinline__ float power(int e) { return __int_as_float((e + 127) << 23); } // -126 .. 127
// From the sum in the three ranges.
__device__ __forceinline__ Factor factor_of(float low, float high, float rest) {
    // |G|^2 = s 2^(2 shift)
    const int shift = high > 0.f ? 80 : rest > 0.f ? 0 : -80;
    const float s = high > 0.f ? high + rest * 0x1p-80f * 0x1p-80f : rest > 0.f ? rest + low * 0x1p-80f * 0x1p-80f : low;
    if (!isfinite(s + rest)) return Factor{1.f, 1.f, __int_as_float(0x7fc00000)};
    if (s == 0.f) return Factor{1.f, 1.f, 0.f};
    const float r = sqrtf(s); // 2^-75 .. 2^64: a normal number
    const int e = ((__float_as_int(r) >> 23) & 255) - 127;
    const int down = -e - shift, half = down / 2; // within -144 .. 155
    return Factor{power(half), power(down - half), kUp / (r * power(-e))};
}

// 2^10 G / |G| in two parts, V columns at a time.
template <class T, int V>
__global__ void __launch_bounds__(kFlat)
    start_kernel(const T *g, int rows, int cols, int ldx, const float *sums, __half *hi, __half *lo) {
    __shared__ Factor shared;
    __shared__ float part[kFlat / 32];
    tc::grid_wait_release();
    float all[3] = {0.f, 0.f, 0.f};
    sums += (size_t)blockIdx.y * kOrthoParts * 3;
#pragma unroll
    for (int i = threadIdx.x; i < kOrthoParts; i += kFlat)
#pragma unroll
        for (int k = 0; k < 3; ++k) all[k] += sums[3 * i + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) all[k] = block_sum(all[k], part);
    if (threadIdx.x == 0) shared = factor_of(all[0], all[1], all[2]);
    __syncthreads();
    const Factor f = shared;
    const uint32_t per = ldx / V;
    const int64_t n = (int64_t)rows * per;
    g += (size_t)blockIdx.y * rows * cols;
#pragma unroll 2
    for (int64_t i = (int64_t)blockIdx.x * kFlat + threadIdx.x; i < n; i += (int64_t)gridDim.x * kFlat) {
        const uint32_t r = n >> 32 ? (uint32_t)(i / per) : (uint32_t)i / per;
        const int c = (int)(i - (int64_t)r * per) * V;
        Piece<T, V> q = {};
        if (V > 1 || c < cols) q = *reinterpret_cast<const Piece<T, V> *>(g + (size_t)r * cols + c);
        Piece<__half, V> h, l;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float v = f((float)q.v[k]);
            h.v[k] = __float2half_rn(v);
            l.v[k] = __float2half_rn(v - __half2float(h.v[k]));
        }
        const size_t to = (size_t)blockIdx.y * n + i;
        reinterpret_cast<Piece<__half, V> *>(hi)[to] = h;
        reinterpret_cast<Piece<__half, V> *>(lo)[to] = l;
    }
}

// What the three products of a step have in common: `count` matrices of M x N results, tiles of 128 * cg x BN.
struct Stack {
    int BN, high, tm, tn, count, M, K;
    void set(int cg, int bn, int n, int m, int cols, int k) {
        BN = bn, high = kBM * cg, M = m, K = k, count = n;
        tm = (m + high - 1) / high;
        tn = (cols + bn - 1) / bn;
    }
    __device__ __forceinline__ int tiles() const { return count * tm * tn; }
    __device__ __forceinline__ Spot spot(int t) const {
        const int z = t / (tm * tn), r = t - z * tm * tn;
        // groups of rows of tiles, columns moving slowest inside a group
        const int group = 2048 / high, per = group * tn, g = r / per, top = g * group, gm = min(group, tm - top), i = r - g * per;
        Spot T;
        T.am = (top + i % gm) * high;
        T.bm = T.n = i / gm * BN;
        T.az = T.bz = z;
        T.ak = T.bk = 0;
        T.pieces = (K + 63) >> 6;
        T.left = 64;
        T.m = z * M + T.am;
        T.z = z;
        T.rows = M - T.am;
        return T;
    }
};
// 32 columns of rows of a matrix of M x ld halves
__device__ __forceinline__ void put_halves(Out32 &o, const Spot &T, const CUtensorMap *map, int M, int ld, int n, const float (&v)[32]) {
    put3_as(WASTE_ACT_F16, o, map, n, ld, o.m - T.z * M, T.z, v);
}
// Tile t of those on and below a diagonal, row by row.
__host__ __device__ __forceinline__ void triangle(int t, int &i, int &j) {
    i = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - i * (i + 1) / 2;
}
// Partial sums of A = X X^T (kMn: X^T X): [matrix][share of k][tile][side][side], fp32.
template <bool kMn> struct GramJob {
    static constexpr bool kAmn = kMn, kBmn = kMn, kMask = false, kReads = false, kTwoPieces = false, kRagged = false;
    CUtensorMap ta, tb, to;
    void *out;
    int side, tri, slices, count, pieces;
    __device__ void begin(uint8_t *) const {}
    __device__ __forceinline__ int tiles(const uint8_t *) const { return count * slices * tri; }
    __device__ __forceinline__ Spot spot(const uint8_t *, int t) const {
        const int s = t / tri, z = s / slices, share = s - z * slices;
        int i, j;
        triangle(t - s * tri, i, j);
        const int k0 = (int)((long long)pieces * share / slices), k1 = (int)((long long)pieces * (share + 1) / slices);
        Spot T;
        T.am = i * side;
        T.bm = j * side;
        T.az = T.bz = z;
        T.ak = T.bk = k0 * 64;
        T.pieces = k1 - k0;
        T.left = 64;
        T.m = t * side;
        T.n = 0;
        T.rows = side;
        return T;
    }
    using Held = Nothing;
    using In = Nothing;
    __device__ __forceinline__ void ahead(const Spot &, int, int, int) const {}
    __device__ __forceinline__ void fetch(const Out32 &, const Spot &, int, Held &) const {}
    __device__ __forceinline__ void turn(const Out32 &, uint4 *, const Held &, In &) const {}
    __device__ __forceinline__ void tile(Out32 &o, const Spot &, int n, const float (&v)[32], const In &) const {
        dense::put32_as(WASTE_ACT_F32, o, &to, out, side, n, side, true, false, v);
    }
};
// A = X X^T (kMn: X^T X) at once.
template <bool kMn> struct WholeGramJob {
    static constexpr bool kAmn = kMn, kBmn = kMn, kMask = false, kReads = false, kTwoPieces = true, kRagged = false;
    CUtensorMap ta, tb, to;
    Stack s;
    int ldm;
    __device__ void begin(uint8_t *) const {}
    __device__ __forceinline__ int tiles(const uint8_t *) const { return s.tiles(); }
    __device__ __forceinline__ Spot spot(const uint8_t *, int t) const { return s.spot(t); }
    using Held = Nothing;
    using In = Nothing;
    __device__ __forceinline__ void tile(Out32 &o, const Spot &T, int n, const float (&v)[32], const In &) const {
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = v[i] * kDown;
        put_halves(o, T, &to, s.M, ldm, n, x);
    }
};
// A from its partial sums, both halves: a CTA takes 64 x 64 values of a tile.
__global__ void __launch_bounds__(kFlat) gram_kernel(const float *parts, int side, int tri, int slices, int m, int ldm, __half *a) {
    __shared__ __half turn[64][66];
    tc::grid_wait_release();
    const int per = side / 64, z = blockIdx.y, tile = blockIdx.x / (per * per), sub = blockIdx.x % (per * per);
    int i, j;
    triangle(tile, i, j);
    const int r0 = i * side + sub / per * 64, c0 = j * side + sub % per * 64; // of the matrix
    if (r0 < c0 || r0 >= m || c0 >= m) return; // above the diagonal, or past the end
    const size_t step = (size_t)tri * side * side;
    const float *p = parts + ((size_t)z * slices * tri + tile) * side * side + (size_t)(sub / per * 64) * side + sub % per * 64;
    __half *to = a + (size_t)z * m * ldm;
    for (int e = threadIdx.x; e < 64 * 16; e += kFlat) {
        const int r = e / 16, c = e % 16 * 4;
        float4 v = {};
#pragma unroll 4
        for (int s = 0; s < slices; ++s) {
            const float4 q = *reinterpret_cast<const float4 *>(p + s * step + (size_t)r * side + c);
            v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
        }
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) turn[r][c + k] = __float2half_rn(x[k] * kDown);
    }
    __syncthreads();
    const bool cross = r0 == c0;
    for (int e = threadIdx.x; e < 64 * 32; e += kFlat) { // the block, and turned round
        const int r = e / 32, c = e % 32 * 2;
#pragma unroll
        for (int side2 = 0; side2 < 2; ++side2) {
            if (side2 && cross) break;
            const int row = (side2 ? c0 : r0) + r, col = (side2 ? r0 : c0) + c;
            if (row >= m || col >= ldm) continue;
            __half x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) x[k] = side2 || (cross && c + k > r) ? turn[c + k][r] : turn[r][c + k];
            *reinterpret_cast<__half2 *>(to + (size_t)row * ldm + col) = __halves2half2(x[0], x[1]);
        }
    }
}
// B = b A + c A^2, its diagonal apart
struct SquareJob {
    static constexpr bool kAmn = false, kBmn = false, kMask = false, kReads = true, kTwoPieces = false, kRagged = false;
    CUtensorMap ta, tb, to;
    Stack s;
    const void *a;
    float *diag;
    int ldm;
    float b, c;
    __device__ void begin(uint8_t *) const {}
    __device__ __forceinline__ int tiles(const uint8_t *) const { return s.tiles(); }
    __device__ __forceinline__ Spot spot(const uint8_t *, int t) const { return s.spot(t); }
    using Held = Block<2>;
    struct In {
        uint4 q[4];
    };
    __device__ __forceinline__ void ahead(const Spot &, int, int, int) const {}
    __device__ __forceinline__ void fetch(const Out32 &o, const Spot &, int n, Held &h) const { h.fetch(o, a, ldm, n, ldm); }
    __device__ __forceinline__ void turn(const Out32 &o, uint4 *t, const Held &h, In &in) const { h.turn(o, t, in.q); }
    __device__ __forceinline__ void tile(Out32 &o, const Spot &T, int n, const float (&v)[32], const In &in) const {
        float x[32];
        halves(in.q, false, x);
        const int row = o.m - T.az * s.M + o.lane; // of its matrix
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = fmaf(c, v[i] * kDown, b * x[i]);
            if (n + i == row) {
                if (o.lane < o.rows) diag[(size_t)T.az * ldm + row] = x[i] * kDown;
                x[i] = 0.f;
            }
        }
        put_halves(o, T, &to, s.M, ldm, n, x);
    }
};
// X <- a X + B X (kTall: a X + X B), the last one to the caller's memory
// kAdd: the last one added to what is there
template <bool kTall, bool kLast, bool kAdd> struct StepJob {
    static constexpr bool kAmn = false, kBmn = !kTall, kMask = false, kReads = true, kTwoPieces = false, kRagged = false;
    CUtensorMap ta, tb, thi, tlo;
    Stack s;
    const void *hi, *lo;
    const float *diag;
    int ldx, ldm;
    float a;
    int full;    // the diagonal multiplies both parts
    int keep_lo; // the next step takes both
    Out<kAdd> out; // of the last step
    float scale;
    __device__ void begin(uint8_t *) const {}
    __device__ __forceinline__ int tiles(const uint8_t *) const { return s.tiles(); }
    __device__ __forceinline__ Spot spot(const uint8_t *, int t) const { return s.spot(t); }
    __device__ __forceinline__ void ahead(const Spot &T, int r, int half, int BN) const {
        if (r >= T.rows) return;
        const int w = min(BN, ldx - T.n);
        if (w > 0 && !(kLast && half))
            ask_l2(static_cast<const __half *>(half ? lo : hi) + (size_t)(T.m + r) * ldx + T.n, w * 2);
        if constexpr (kAdd) out.ahead(T.m + r, T.n, half, BN);
    }
    struct Held {
        Block<2> hi, lo;
        std::conditional_t<kAdd, typename Out<kAdd>::Held, Nothing> base;
    };
    struct In {
        uint4 hi[4], lo[4];
        typename Out<kAdd>::In base;
    };
    __device__ __forceinline__ void fetch(const Out32 &o, const Spot &, int n, Held &h) const {
        h.hi.fetch(o, hi, ldx, n, ldx);
        if constexpr (!kLast) h.lo.fetch(o, lo, ldx, n, ldx);
        if constexpr (kAdd) out.fetch(o, n, h.base);
    }
    __device__ __forceinline__ void turn(const Out32 &o, uint4 *t, const Held &h, In &in) const {
        h.hi.turn(o, t, in.hi);
        if constexpr (!kLast) h.lo.turn(o, t, in.lo);
        if constexpr (kAdd) out.turn(o, t, h.base, in.base);
    }
    __device__ __forceinline__ void tile(Out32 &o, const Spot &T, int n, const float (&v)[32], const In &in) const {
        float x[32], l[32];
        halves(in.hi, false, x);
        if constexpr (!kLast) halves(in.lo, false, l);
        const float *d = diag + (size_t)T.az * ldm;
        float dr = 0.f;
        if (!kTall && o.lane < o.rows) dr = d[o.m - T.az * s.M + o.lane];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            float4 dc = {dr, dr, dr, dr};
            if (kTall) dc = n + j < ldm ? *reinterpret_cast<const float4 *>(d + n + j) : float4{};
            const float dd[4] = {dc.x, dc.y, dc.z, dc.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = j + k;
                const float w = kLast ? x[i] : x[i] + l[i];
                x[i] = fmaf(a, w, fmaf(dd[k], full ? w : x[i], v[i] * kDown));
            }
        }
        if constexpr (kLast) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= scale;
            out.put(o, T, n, x, in.base);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) l[i] = x[i] - __half2float(__float2half_rn(x[i]));
            put_halves(o, T, &thi, s.M, ldx, n, x);
            if (keep_lo) put_halves(o, T, &tlo, s.M, ldx, n, l);
        }
    }
};

// ---- small matrices: all steps in one launch, one CTA a matrix
//
// X (short side first, 128 rows) stays in shared memory: hi in the layout of an MMA operand with 128-byte swizzle, which
// serves A = X X^T with the long side as k and B X with the rows as k alike, lo in the same layout beside it.  A, and
// B in its place, have 32 KB more.  A step is three products of a few hundred nanoseconds, each followed by its epilogue
// and a barrier.
constexpr int kSmallRows = 128, kSmallCols = 320, kSmallThreads = 512;
constexpr int kSlab = 16384; // 128 rows x 64 columns

// Byte of row r, columns 8 i .. 8 i + 7 in slabs of 64 columns.
__device__ __forceinline__ uint32_t place(int r, int i) { return (i >> 3) * kSlab + r * 128 + (((i & 7) ^ (r & 7)) << 4); }
__device__ __forceinline__ uint4 pack_halves(const float (&v)[8]) { return dense::piece_of(v, __half()); }

template <class O> __device__ __forceinline__ void put_one(O *p, float v, int add) { *p = dense::round_to<O>(add ? (float)*p + v : v); }
__device__ __forceinline__ void put_value(void *p, int dtype, size_t i, float v, int add) {
    if (dtype == WASTE_ACT_F32)
        put_one(static_cast<float *>(p) + i, v, add);
    else if (dtype == WASTE_ACT_BF16)
        put_one(static_cast<__nv_bfloat16 *>(p) + i, v, add);
    else
        put_one(static_cast<__half *>(p) + i, v, add);
}

template <class T, bool kTall>
__global__ void __launch_bounds__(kSmallThreads)
    small_kernel(const T *g, int m, int n, int steps, float ca, float cb, float cc, void *out, int out_dtype, int add, float scale) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ float part[kSmallThreads / 32], diag[kSmallRows];
    __shared__ Factor shared;
    __shared__ __align__(8) uint64_t bar_word;
    __shared__ uint32_t tmem_slot;
    const int slabs = (n + 63) / 64, tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    uint8_t *hi = smem, *lo = smem + slabs * kSlab, *mat = lo + slabs * kSlab;
    const uint32_t hi_at = tc::smem_u32(hi), mat_at = tc::smem_u32(mat), bar = tc::smem_u32(&bar_word);
    if (tid == 0) {
        tc::mbar_init(bar, 1);
        tc::mbar_init_fence();
    }
    if (warp == 0) tc::tmem_alloc(tc::smem_u32(&tmem_slot), kTmemCols); // one CTA an SM: by its registers, too
    tc::grid_wait_release();

    // ---- G, by pieces of 8 of X's columns: thread t holds t, t + 512, .. in registers, all asked for at once
    g += (size_t)blockIdx.x * m * n;
    const int per = slabs * 8;
    constexpr int kMost = kSmallRows * kSmallCols / 8 / kSmallThreads;
    float x0[kMost][8];
    const auto row = [&](int i) { return kTall ? i % kSmallRows : i / per; }; // neighbours read neighbouring values
    const auto col = [&](int i) { return kTall ? i / kSmallRows : i % per; };
#pragma unroll
    for (int p = 0; p < kMost; ++p) {
        float(&v)[8] = x0[p];
        const int i = p * kSmallThreads + tid, r = row(i), c = col(i) * 8;
        const bool in = i < kSmallRows * per && r < m;
        if (!kTall && sizeof(T) == 2 && n % 8 == 0) {
            Piece<T, 8> q = {};
            if (in && c < n) q = *reinterpret_cast<const Piece<T, 8> *>(g + r * n + c);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = (float)q.v[k];
        } else if (!kTall && n % 4 == 0 && sizeof(T) == 4) {
            float4 q[2] = {};
            if (in && c < n) q[0] = *reinterpret_cast<const float4 *>(g + r * n + c);
            if (in && c + 4 < n) q[1] = *reinterpret_cast<const float4 *>(g + r * n + c + 4);
            v[0] = q[0].x, v[1] = q[0].y, v[2] = q[0].z, v[3] = q[0].w, v[4] = q[1].x, v[5] = q[1].y, v[6] = q[1].z, v[7] = q[1].w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = in && c + k < n ? (float)g[kTall ? (c + k) * m + r : r * n + c + k] : 0.f;
        }
    }
    float s[3];
    squares_of(
        [&](auto f) {
#pragma unroll
            for (int p = 0; p < kMost; ++p)
#pragma unroll
                for (int k = 0; k < 8; ++k) f(x0[p][k]);
        },
        part, s);
    if (tid == 0) shared = factor_of(s[0], s[1], s[2]);
    __syncthreads();
    const Factor f = shared;
#pragma unroll
    for (int p = 0; p < kMost; ++p) {
        const int i = p * kSmallThreads + tid;
        if (i >= kSmallRows * per) break;
        float(&v)[8] = x0[p], l[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = f(v[k]);
            l[k] = v[k] - __half2float(__float2half_rn(v[k]));
        }
        const uint32_t at = place(row(i), col(i));
        *reinterpret_cast<uint4 *>(hi + at) = pack_halves(v);
        *reinterpret_cast<uint4 *>(lo + at) = pack_halves(l);
    }

    // ---- steps
    const int q = warp & 3, r = 32 * q + lane, first = 32 * (warp >> 2), step = kSmallThreads / 4; // this thread's row and columns
    uint32_t phase = 0;
    bool ok = true;
    // one product: what the threads wrote is there for it, and its sums are there for them
    const auto product = [&](auto issue) {
        tc::fence_proxy_async();
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        if (warp == 0) {
            if (tc::elect_one()) {
                issue();
                tc::mma_commit(bar);
            }
            __syncwarp();
        }
        const bool mine = tc::mbar_wait(bar, phase);
        phase ^= 1;
        ok = !__syncthreads_or(!mine);
        tc::fence_after_sync();
    };
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0), wide = 128; // A's and B's sums in the first 128, X's behind them
    const uint64_t hi_desc = tc::desc_sw128(hi_at, kSlab), mat_desc = tc::desc_sw128(mat_at, kSlab);
    constexpr uint32_t square = tc::idesc_half(kSmallRows, kSmallRows, false, false, false);
    const auto sums = [&](uint32_t col, uint32_t (&v)[32]) {
        tc::tmem_ld32(tmem + col + ((uint32_t)(32 * q) << 16), v);
        tc::tmem_wait_ld(v);
    };
    for (int i = 0; i < steps && ok; ++i) {
        product([&] {
            for (int k = 0; k < 4 * slabs; ++k) {
                const uint64_t d = hi_desc + (uint64_t)((k / 4 * kSlab + k % 4 * 32) >> 4);
                tc::mma_f16(tmem, d, d, square, k > 0);
            }
        });
        if (!ok) break;
        for (int c = first; c < kSmallRows; c += step) {
            uint32_t v[32];
            sums(c, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(v[8 * j + k]) * kDown;
                *reinterpret_cast<uint4 *>(mat + place(r, c / 8 + j)) = pack_halves(x);
            }
        }
        product([&] {
            for (int k = 0; k < 8; ++k) {
                const uint64_t d = mat_desc + (uint64_t)((k / 4 * kSlab + k % 4 * 32) >> 4);
                tc::mma_f16(tmem, d, d, square, k > 0);
            }
        });
        if (!ok) break;
        for (int c = first; c < kSmallRows; c += step) {
            uint32_t v[32];
            sums(c, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 *at = reinterpret_cast<uint4 *>(mat + place(r, c / 8 + j));
                float x[8];
                dense::widen8(false, *at, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[k] = fmaf(cc, __uint_as_float(v[8 * j + k]) * kDown, cb * x[k]);
                    if (c + 8 * j + k == r) {
                        diag[r] = x[k] * kDown;
                        x[k] = 0.f;
                    }
                }
                *at = pack_halves(x);
            }
        }
        product([&] {
            for (int h = 0; h < slabs; h += 4) { // 256 columns at most in one MMA
                const int cols = 64 * (slabs - h < 4 ? slabs - h : 4);
                const uint32_t id = tc::idesc_half(kSmallRows, cols, false, false, true);
                for (int k = 0; k < 8; ++k)
                    tc::mma_f16(tmem + wide + 64 * h, mat_desc + (uint64_t)((k / 4 * kSlab + k % 4 * 32) >> 4),
                                hi_desc + (uint64_t)((h * kSlab + k * 2048) >> 4), id, k > 0);
            }
        });
        if (!ok) break;
        const bool last = i + 1 == steps, full = i + 2 >= steps;
        const float d = diag[r];
        for (int c = first; c < 64 * slabs; c += step) {
            uint32_t v[32];
            sums(wide + c, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = place(r, c / 8 + j);
                float x[8], l[8];
                dense::widen8(false, *reinterpret_cast<const uint4 *>(hi + at), x);
                dense::widen8(false, *reinterpret_cast<const uint4 *>(lo + at), l);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float w = x[k] + l[k];
                    x[k] = fmaf(ca, w, fmaf(d, full ? w : x[k], __uint_as_float(v[8 * j + k]) * kDown));
                }
                if (!last) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) l[k] = x[k] - __half2float(__float2half_rn(x[k]));
                    *reinterpret_cast<uint4 *>(hi + at) = pack_halves(x);
                    *reinterpret_cast<uint4 *>(lo + at) = pack_halves(l);
                    continue;
                }
                if (r >= m) continue;
                const int c0 = c + 8 * j;
                const size_t mat0 = (size_t)blockIdx.x * m * n;
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= scale;
                if (kTall) { // neighbouring lanes, neighbouring values
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (c0 + k < n) put_value(out, out_dtype, mat0 + (size_t)(c0 + k) * m + r, x[k], add);
                } else {
                    dense::put_as(out_dtype, out, mat0 + (size_t)r * n + c0, c0, n, n % 8 == 0, add, x);
                }
            }
        }
    }
    if (!ok && tid == 0) atomicOr(&dense::g_dense_timeout, 1u);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
}

template <class T, bool kTall> cudaError_t small(const Ortho &P, cudaStream_t s) {
    static SmemAttr attr;
    const auto kernel = small_kernel<T, kTall>;
    const int m = kTall ? P.cols : P.rows, n = kTall ? P.rows : P.cols;
    const int smem = (2 * ((n + 63) / 64) + 2) * kSlab + 1024;
    const cudaError_t e = ensure_smem(attr, reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_behind(kernel, dim3(P.count), dim3(kSmallThreads), smem, s, static_cast<const T *>(P.g), m, n, P.steps, P.a, P.b, P.c, P.out,
                         P.out_dtype, P.add, P.scale * kDown);
}

// Tiles of 128 * cg x BN for `count` results of M x N over `pieces` of k: the quickest by whole waves of tiles, each as
// long as its operands and what its epilogue reads (`extra` bytes a value) need into an SM (100 B/ns) or as its
// MMAs take.  An MN-major B comes in columns of 64.
struct Shape {
    int cg, BN;
};
Shape shape(int count, int M, int N, int pieces, bool b_mn, int extra, int sms) {
    Shape best{1, 64};
    double least = 1e30;
    for (int cg = 1; cg <= 2; ++cg)
        for (int BN = 64; BN <= 256; BN += 32) {
            if (cg == 2 && M <= kBM) continue;
            if (BN > 64 && BN - 32 >= N) break;
            const long long tiles = (long long)count * ((M + kBM * cg - 1) / (kBM * cg)) * ((N + BN - 1) / BN), slots = sms / cg;
            const double in = pieces * (kBM * kRowBytes + (double)dense::stage_b_bytes(BN, cg, b_mn)) + kBM * BN * extra;
            const double load = in / 100., mma = pieces * BN * 1.31, out = kBM * BN * 0.1; // the last tile's epilogue
            const double t = (double)((tiles + slots - 1) / slots) * (load > mma ? load : mma) + out;
            if (t < least) least = t, best = Shape{cg, BN};
        }
    return best;
}
template <class J> cudaError_t launch(int cg, int BN, const J &job, long long tiles, int sms, cudaStream_t s) {
    TileArgs T = {};
    T.BN = BN;
    return cg == 2 ? launch_tiles_as<2>(T, job, false, 0, tiles, sms, s) : launch_tiles_as<1>(T, job, false, 0, tiles, sms, s);
}

template <bool kTall, bool kAdd> cudaError_t steps(const Ortho &P, const OrthoParts &W, cudaStream_t s) {
    const int m = kTall ? P.cols : P.rows, n = kTall ? P.rows : P.cols, sms = device_sm_count();
    uint8_t *hi[2] = {P.ws + W.hi[0], P.ws + W.hi[1]}, *lo = P.ws + W.lo, *A = P.ws + W.a, *B = P.ws + W.b;
    float *diag = reinterpret_cast<float *>(P.ws + W.diag), *parts = reinterpret_cast<float *>(P.ws + W.gram);
    const size_t xs = (size_t)P.rows * W.ldx, ss = (size_t)m * W.ldm;
    const int pieces = (m + 63) / 64;
    const Shape qs = shape(P.count, m, m, pieces, false, 2, sms), xx = shape(P.count, P.rows, P.cols, pieces, !kTall, 4, sms);
    const int gcg = W.side == 256 ? 2 : 1, long_pieces = (n + 63) / 64;
    const bool whole = W.slices == 0;
    const Shape gs = whole ? shape(P.count, m, m, long_pieces, kTall, 0, sms) : Shape{gcg, W.side};
    cudaError_t e = cudaSuccess;
    const auto x_map = [&](CUtensorMap *t, int i, int box) {
        if (e == cudaSuccess) e = stack_map(t, hi[i], P.cols, P.rows, P.count, W.ldx, xs, box);
    };
    const auto s_map = [&](CUtensorMap *t, const void *p, int box) {
        if (e == cudaSuccess) e = stack_map(t, p, m, m, P.count, W.ldm, ss, box);
    };
    const auto o_map = [&](CUtensorMap *t, void *p, int rows, int ld) { // a stack of halves
        if (e == cudaSuccess) e = store_map3(t, p, WASTE_ACT_F16, P.count, rows, ld);
    };
    GramJob<kTall> G = {};
    SquareJob Q = {};
    StepJob<kTall, false, false> S = {};
    StepJob<kTall, true, kAdd> L = {};
    G.out = parts;
    G.side = W.side, G.tri = W.tri, G.slices = W.slices, G.count = P.count, G.pieces = (n + 63) / 64;
    const long long items = (long long)P.count * W.tri * W.slices;
    if (!whole) e = dense::store_map(&G.to, parts, 4, (int)(items * W.side), W.side);
    WholeGramJob<kTall> D = {};
    D.s.set(gs.cg, gs.BN, P.count, m, m, n);
    o_map(&D.to, A, m, W.ldm);
    D.ldm = W.ldm;
    Q.s.set(qs.cg, qs.BN, P.count, m, m, m);
    s_map(&Q.ta, A, kBM);
    s_map(&Q.tb, A, qs.BN / qs.cg);
    o_map(&Q.to, B, m, W.ldm);
    Q.a = A, Q.diag = diag, Q.ldm = W.ldm, Q.b = P.b, Q.c = P.c;
    S.s.set(xx.cg, xx.BN, P.count, P.rows, P.cols, m);
    s_map(kTall ? &S.tb : &S.ta, B, kTall ? xx.BN / xx.cg : kBM);
    o_map(&S.tlo, lo, P.rows, W.ldx);
    S.lo = lo, S.diag = diag, S.ldx = W.ldx, S.ldm = W.ldm, S.a = P.a;
    if (e == cudaSuccess) e = L.out.set(P.out, P.count, P.rows, P.cols, P.out_dtype);
    CUtensorMap ga[2], gb[2], sx[2], st[2];
    for (int i = 0; i < 2; ++i) {
        x_map(&ga[i], i, kTall ? 64 : kBM);
        x_map(&gb[i], i, kTall ? 64 : gs.BN / gs.cg);
        x_map(&sx[i], i, kTall ? kBM : 64);
        o_map(&st[i], hi[i], P.rows, W.ldx);
    }
    const int per = W.side / 64;
    for (int i = 0; i < P.steps && e == cudaSuccess; ++i) {
        const int from = i & 1;
        G.ta = D.ta = ga[from], G.tb = D.tb = gb[from];
        e = whole ? launch(gs.cg, gs.BN, D, (long long)P.count * D.s.tm * D.s.tn, sms, s) : launch(gcg, W.side, G, items, sms, s);
        if (e == cudaSuccess && !whole)
            e = launch_behind(gram_kernel, dim3(W.tri * per * per, P.count), dim3(kFlat), 0, s, parts, W.side, W.tri, W.slices, m, W.ldm,
                              reinterpret_cast<__half *>(A));
        if (e == cudaSuccess) e = launch(qs.cg, qs.BN, Q, (long long)P.count * Q.s.tm * Q.s.tn, sms, s);
        if (e != cudaSuccess) break;
        const long long tiles = (long long)P.count * S.s.tm * S.s.tn;
        (kTall ? S.ta : S.tb) = sx[from];
        S.hi = hi[from];
        S.full = i + 2 >= P.steps;
        if (i + 1 < P.steps) {
            S.thi = st[from ^ 1];
            S.keep_lo = i + 2 < P.steps;
            e = launch(xx.cg, xx.BN, S, tiles, sms, s);
        } else {
            L.ta = S.ta, L.tb = S.tb, L.s = S.s, L.hi = S.hi, L.lo = S.lo, L.diag = S.diag, L.ldx = S.ldx, L.ldm = S.ldm, L.a = S.a;
            L.full = S.full, L.scale = P.scale * kDown;
            e = launch(xx.cg, xx.BN, L, tiles, sms, s);
        }
    }
    return e;
}

template <class T, int V> cudaError_t start(const Ortho &P, const OrthoParts &W, cudaStream_t s) {
    float *sums = reinterpret_cast<float *>(P.ws + W.sums);
    const T *g = static_cast<const T *>(P.g);
    cudaError_t e = launch_behind(squares_kernel<T, V>, dim3(kOrthoParts, P.count), dim3(kFlat), 0, s, g, (int64_t)P.rows * P.cols, sums);
    if (e != cudaSuccess) return e;
    const int64_t blocks = ((int64_t)P.rows * (W.ldx / V) + 2 * kFlat - 1) / (2 * kFlat), most = 16 * device_sm_count();
    return launch_behind(start_kernel<T, V>, dim3((unsigned)(blocks < most ? blocks : most), P.count), dim3(kFlat), 0, s, g, P.rows, P.cols,
                         W.ldx, sums, reinterpret_cast<__half *>(P.ws + W.hi[0]), reinterpret_cast<__half *>(P.ws + W.lo));
}

} // namespace

cudaError_t launch_ortho(const Ortho &P, cudaStream_t s) {
    const OrthoParts W = ortho_parts(P.count, P.rows, P.cols);
    const bool tall = P.rows > P.cols;
    const int m = tall ? P.cols : P.rows, n = tall ? P.rows : P.cols;
    if (m <= kSmallRows && n <= kSmallCols) {
        const auto go = [&](auto t) {
            using T = decltype(t);
            return tall ? small<T, true>(P, s) : small<T, false>(P, s);
        };
        return P.g_dtype == WASTE_ACT_F32 ? go(float()) : P.g_dtype == WASTE_ACT_BF16 ? go(__nv_bfloat16()) : go(__half());
    }
    const auto go = [&](auto t) {
        using T = decltype(t);
        return P.cols % 8 ? start<T, 1>(P, W, s) : start<T, 8>(P, W, s);
    };
    const cudaError_t e = P.g_dtype == WASTE_ACT_F32 ? go(float()) : P.g_dtype == WASTE_ACT_BF16 ? go(__nv_bfloat16()) : go(__half());
    if (e != cudaSuccess) return e;
    if (P.add) return tall ? steps<true, true>(P, W, s) : steps<false, true>(P, W, s);
    return tall ? steps<true, false>(P, W, s) : steps<false, false>(P, W, s);
}
cudaError_t ortho_word(uint32_t **word) { return dense::timeout_word(word); }
cudaError_t ortho_timeout(uint32_t *out) { return dense::read_and_clear_timeout(out); }

} // namespace train
} // namespace wm
