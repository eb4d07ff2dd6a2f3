// Products grouped by expert (waste_train.h): y_r = x_r W_e^T, dx_r = dy_r W_e, dW_e = dy_e^T x_e over rows sorted
// by expert, as tiles of tile_mma.cuh.
//
// The offsets stay on the device: every CTA reads them, adds up the experts' tiles in shared memory, and finds each of
// its tiles by bisection.  A tile has rows of one expert alone: TMA loads start at any row, what the last tile of an
// expert loads of the next one's rows is never stored, and in dW, where rows are summed over, the rows
// behind the expert's last are cleared in shared memory.
#include <type_traits>

#include "tile_mma.cuh"

namespace wm {
namespace train {

cudaError_t stack_map(CUtensorMap *m, const void *p, int cols, int rows, int mats, size_t ld, size_t step, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)mats};
    const cuuint64_t strides[2] = {ld * 2, step * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    return dense::encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

namespace {

__device__ uint32_t g_bad_offsets;

// Offsets as the kernels use them: what does not ascend within 0 .. rows is replaced by the nearest that does.
struct Offsets {
    const int32_t *p;
    int E, rows;
    // Into first[0 .. E]; with tn > 0 also the tiles of all experts before each, of `high` rows and tn
    // columns of tiles, into before[0 .. E].
    __device__ void read(int *first, int *before, int high, int tn) const {
        for (int e = threadIdx.x; e <= E; e += kTileThreads) first[e] = p[e];
        __syncthreads();
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x, per = (E + 32) / 32, e0 = min(E + 1, lane * per), e1 = min(E + 1, e0 + per);
            int most = 0;
            bool bad = false;
            for (int e = e0; e < e1; ++e) {
                const int v = first[e];
                bad |= v < 0 || v > rows || (e > 0 && v < first[e - 1]);
                most = max(most, min(v, rows));
            }
            // the largest up to each lane's first
            int up = most;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up = max(up, v);
            }
            up = __shfl_up_sync(0xffffffffu, up, 1);
            if (lane == 0) up = 0;
            if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) atomicOr(&g_bad_offsets, 1u);
            int last = up;
            for (int e = e0; e < e1; ++e) first[e] = last = max(last, min(first[e], rows));
            __syncwarp();
            if (tn > 0) {
                int sum = 0;
                for (int e = e0; e < e1; ++e)
                    if (e > 0) sum += (first[e] - first[e - 1] + high - 1) / high * tn;
                int at = sum;
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, at, o);
                    if (lane >= o) at += v;
                }
                at -= sum;
                for (int e = e0; e < e1; ++e) {
                    if (e > 0) at += (first[e] - first[e - 1] + high - 1) / high * tn;
                    before[e] = at;
                }
            }
        }
        __syncthreads();
    }
};

// Results by row: y (W K-major) and dx (W MN-major).
template <int kCG, bool kWmn, bool kAdd> struct RowsJob {
    static constexpr bool kAmn = false, kBmn = kWmn, kMask = false, kReads = kAdd;
    CUtensorMap ta, tb;
    Out<kAdd> out;
    Offsets off;
    int BN, tn, pieces;
    static constexpr int kHigh = kBM * kCG;
    __device__ void begin(uint8_t *smem) const {
        int *first = reinterpret_cast<int *>(smem);
        off.read(first, first + off.E + 1, kHigh, tn);
    }
    __device__ __forceinline__ int tiles(const uint8_t *smem) const { return reinterpret_cast<const int *>(smem)[2 * off.E + 1]; }
    __device__ __forceinline__ Spot spot(const uint8_t *smem, int t) const {
        const int *first = reinterpret_cast<const int *>(smem), *before = first + off.E + 1;
        int e = 0; // the last with before[e] <= t
        for (int b = 1 << (31 - __clz(off.E)); b; b >>= 1)
            if (e + b <= off.E && before[e + b] <= t) e += b;
        const int r = t - before[e], r0 = first[e], n = first[e + 1] - r0, tm = (n + kHigh - 1) / kHigh;
        // groups of 16 row tiles (of 128), columns moving slowest inside a group
        constexpr int kGroup = 16 / kCG;
        const int per = kGroup * tn, g = r / per, top = g * kGroup, gm = min(kGroup, tm - top), i = r - g * per;
        const int mi = top + i % gm, ni = i / gm;
        Spot T;
        T.am = T.m = r0 + mi * kHigh;
        T.az = 0;
        T.bm = T.n = ni * BN;
        T.bz = e;
        T.ak = T.bk = 0;
        T.pieces = pieces;
        T.left = 64;
        T.rows = n - mi * kHigh;
        return T;
    }
    using Held = typename Out<kAdd>::Held;
    using In = typename Out<kAdd>::In;
    __device__ __forceinline__ void ahead(const Spot &T, int r, int half, int BN) const {
        if (r < T.rows) out.ahead(T.m + r, T.n, half, BN);
    }
    __device__ __forceinline__ void fetch(const Out32 &o, const Spot &, int n, Held &h) const { out.fetch(o, n, h); }
    __device__ __forceinline__ void turn(const Out32 &o, uint4 *t, const Held &h, In &in) const { out.turn(o, t, h, in); }
    __device__ __forceinline__ void tile(Out32 &o, const Spot &, int n, const float (&v)[32], const In &in) const {
        out.put(o, n, v, in);
    }
};

// dW: the rows are what is summed over.
template <int kCG, bool kAdd> struct WeightsJob {
    static constexpr int kHigh = kBM * kCG;
    static constexpr bool kAmn = true, kBmn = true, kMask = true, kReads = kAdd;
    CUtensorMap ta, tb;
    Out<kAdd> out;
    Offsets off;
    int BN, tm, tn, M;
    __device__ void begin(uint8_t *smem) const { off.read(reinterpret_cast<int *>(smem), nullptr, 0, 0); }
    __device__ __forceinline__ int tiles(const uint8_t *) const { return off.E * tm * tn; }
    __device__ __forceinline__ Spot spot(const uint8_t *smem, int t) const {
        const int *first = reinterpret_cast<const int *>(smem);
        const int e = t / (tm * tn), r = t - e * tm * tn, mi = r % tm, ni = r / tm;
        const int r0 = first[e], n = first[e + 1] - r0;
        Spot T;
        T.am = mi * kHigh;
        T.bm = T.n = ni * BN;
        T.az = T.bz = 0;
        T.ak = T.bk = r0;
        T.pieces = (n + 63) >> 6;
        T.left = n - ((T.pieces - 1) << 6);
        T.m = e * M + mi * kHigh;
        T.rows = M - mi * kHigh;
        return T;
    }
    using Held = typename Out<kAdd>::Held;
    using In = typename Out<kAdd>::In;
    __device__ __forceinline__ void ahead(const Spot &T, int r, int half, int BN) const {
        if (r < T.rows) out.ahead(T.m + r, T.n, half, BN);
    }
    __device__ __forceinline__ void fetch(const Out32 &o, const Spot &, int n, Held &h) const { out.fetch(o, n, h); }
    __device__ __forceinline__ void turn(const Out32 &o, uint4 *t, const Held &h, In &in) const { out.turn(o, t, h, in); }
    __device__ __forceinline__ void tile(Out32 &o, const Spot &T, int n, const float (&v)[32], const In &in) const {
        if (T.pieces || !kAdd) out.put(o, n, v, in);
    }
};

constexpr std::integral_constant<int, 1> kOne;
constexpr std::integral_constant<int, 2> kTwo;
constexpr std::true_type kYes;
constexpr std::false_type kNo;

// Whole widths of 32 columns, 256 at most.
int width(int n) { return n >= 256 ? 256 : n <= 64 ? 64 : (n + 31) / 32 * 32; }

// Pairs of CTAs, with tiles of 256 rows, from so many rows an expert on (their mean: the offsets are on the device).
bool pairs(const Group &G) { return G.rows / G.E >= 160; }

template <int kCG, bool kWmn, bool kAdd>
cudaError_t rows_product(const Group &G, const void *a, int K, const void *w, int N, void *out, int out_dtype, cudaStream_t s) {
    RowsJob<kCG, kWmn, kAdd> J = {};
    TileArgs P = {};
    P.BN = J.BN = width(N);
    J.off = {G.offsets, G.E, G.rows};
    J.tn = (N + J.BN - 1) / J.BN;
    J.pieces = (K + 63) / 64;
    cudaError_t e = stack_map(&J.ta, a, K, G.rows, 1, K, (size_t)K * G.rows, kBM);
    if (e == cudaSuccess) e = stack_map(&J.tb, w, G.k, G.n, G.E, G.k, (size_t)G.k * G.n, kWmn ? 64 : J.BN / kCG);
    if (e == cudaSuccess) e = J.out.set(out, G.rows, N, out_dtype);
    if (e != cudaSuccess) return e;
    const long long most = ((long long)G.rows / J.kHigh + (G.E < G.rows ? G.E : G.rows)) * J.tn;
    return launch_tiles_as<kCG>(P, J, G.dtype == WASTE_ACT_BF16, (size_t)(G.E + 1) * 8, most, device_sm_count(), s);
}

template <int kCG, bool kAdd>
cudaError_t weights_product(const Group &G, const void *dy, const void *x, void *dw, int grad_dtype, cudaStream_t s) {
    WeightsJob<kCG, kAdd> J = {};
    TileArgs P = {};
    P.BN = J.BN = width(G.k);
    J.off = {G.offsets, G.E, G.rows};
    J.M = G.n;
    J.tm = (G.n + J.kHigh - 1) / J.kHigh;
    J.tn = (G.k + J.BN - 1) / J.BN;
    cudaError_t e = stack_map(&J.ta, dy, G.n, G.rows, 1, G.n, (size_t)G.n * G.rows, 64);
    if (e == cudaSuccess) e = stack_map(&J.tb, x, G.k, G.rows, 1, G.k, (size_t)G.k * G.rows, 64);
    if (e == cudaSuccess) e = J.out.set(dw, G.E * G.n, G.k, grad_dtype);
    if (e != cudaSuccess) return e;
    return launch_tiles_as<kCG>(P, J, G.dtype == WASTE_ACT_BF16, (size_t)(G.E + 1) * 4, (long long)G.E * J.tm * J.tn,
                                device_sm_count(), s);
}

} // namespace

cudaError_t launch_group_forward(const Group &G, const void *x, const void *w, void *y, int out_dtype, int add, cudaStream_t s) {
    const auto go = [&](auto cg, auto adds) {
        return rows_product<decltype(cg)::value, false, decltype(adds)::value>(G, x, G.k, w, G.n, y, out_dtype, s);
    };
    return pairs(G) ? (add ? go(kTwo, kYes) : go(kTwo, kNo)) : add ? go(kOne, kYes) : go(kOne, kNo);
}
cudaError_t launch_group_dx(const Group &G, const void *dy, const void *w, void *dx, cudaStream_t s) {
    return pairs(G) ? rows_product<2, true, false>(G, dy, G.n, w, G.k, dx, G.dtype, s)
                    : rows_product<1, true, false>(G, dy, G.n, w, G.k, dx, G.dtype, s);
}
cudaError_t launch_group_dw(const Group &G, const void *dy, const void *x, void *dw, int grad_dtype, int add, cudaStream_t s) {
    const auto go = [&](auto cg, auto adds) {
        return weights_product<decltype(cg)::value, decltype(adds)::value>(G, dy, x, dw, grad_dtype, s);
    };
    return pairs(G) && G.n > kBM ? (add ? go(kTwo, kYes) : go(kTwo, kNo)) : add ? go(kOne, kYes) : go(kOne, kNo);
}

cudaError_t group_status(uint32_t *timeout, uint32_t *offsets) {
    cudaError_t e = dense::read_and_clear_timeout(timeout);
    uint32_t v = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_bad_offsets, sizeof v);
    const uint32_t zero = 0;
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_bad_offsets, &zero, sizeof zero);
    *offsets |= v;
    return e;
}

} // namespace train
} // namespace wm
