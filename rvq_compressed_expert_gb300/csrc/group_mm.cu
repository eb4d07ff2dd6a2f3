// Products grouped by expert (waste_train.h): y_r = x_r W_e^T, dx_r = dy_r W_e, dW_e = dy_e^T x_e over rows sorted
// by expert, as tiles of tile_mma.cuh.
//
// The offsets stay on the device: every CTA reads them, adds up the experts' tiles in shared memory, and finds each of
// its tiles by bisection.
//
// y and dx: the matrices are on the MMA's row side (128 rows, 256 for a pair of CTAs) and the expert's rows on its column
// side, whose width is a multiple of 16 (32), so that little is computed for rows that are not there: an expert's
// rows are cut into equal shares of at most 256, or 64 (rows_plan).  With the rows on the row side, in tiles of 256, a
// batch of uneven popularity (126 to 2048 rows an expert) wastes 20 %.  The sums are turned round in shared memory on
// their way out.
// Loads start at any row; what the last share of an expert loads of the next one's rows is never stored.
// dW: its rows are what is summed over; those behind the expert's last are cleared in shared memory.
//
// Measured (bf16, k 7168, n 1536; popularity falling as 1 / rank^1.1; floors at 6.75 TB/s and 1.90 PFLOP/s): 16 rows of 16
// experts 63 us (floor 52: W's 352 MB; 256 tiles of 96 x 16 on 152 SMs make two rounds, the second not full); 2048
// rows over 384 experts 975 us = 7.1 TB/s of W; 32768 rows over 64 experts, back through down, 478 us cold and 531 to 550 in long
// runs at 1.65 GHz (floor 379; cuBLAS takes 408 for one matrix of as many rows), their gradients 1130 to 1190 us (floor
// 758; dx 470, the rest dW).  dW is bound by its epilogue, not by memory or MMAs (8192 rows over 16 experts: DRAM 39 %,
// tensor pipe 56 %, 142 us; dx, the same operations, 77 % and 112): a tile's sums go out in boxes of 32 rows x 64 bytes, one
// behind another, 2.1 us for an SM's 128 x 256 values in bf16 however few rows they sum (64 matrices of 1536 x 7168 from 64,
// 128 and 256 rows each: 312, 302, 361 us), which MMAs hide only where sums are long (512 rows 527 us, MMAs 379; 1024 832
// and 758; 2048 1545 and 1516).  In fp32 3.5 us, added to bf16 3.7, added to fp32 7.8 (2.8 GB read and written: 5.9).
// Added y (mode 1) goes out lane by lane: 1536 to 7168, 32768 rows 1038 us against 463.
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

cudaError_t store_map3(CUtensorMap *m, void *p, int dtype, int mats, int rows, int cols) {
    const size_t size = dense::type_size(dtype);
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)mats};
    const cuuint64_t strides[2] = {cols * size, cols * size * rows};
    const cuuint32_t box[3] = {(cuuint32_t)(64 / size), 32, 1};
    return dense::encode_map(m, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, p, dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

namespace {

__device__ uint32_t g_bad_offsets;

// Offsets as the kernels use them: what does not ascend within 0 .. rows is replaced by the nearest that does.
struct Offsets {
    const int32_t *p;
    int E, rows, share; // share: rows of an expert in one tile, at most
    // Into first[0 .. E]; and the shares (of at most `share` rows) of all experts before each into before[0 .. E], if not null.
    __device__ void read(int *first, int *before) const {
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
            if (before) {
                int sum = 0;
                for (int e = e0; e < e1; ++e)
                    if (e > 0) sum += (first[e] - first[e - 1] + share - 1) / share;
                int at = sum;
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, at, o);
                    if (lane >= o) at += v;
                }
                at -= sum;
                for (int e = e0; e < e1; ++e) {
                    if (e > 0) at += (first[e] - first[e - 1] + share - 1) / share;
                    before[e] = at;
                }
            }
        }
        __syncthreads();
    }
};

// Results by row: y (W K-major) and dx (W MN-major).
template <int kCG, bool kWmn, bool kAdd> struct RowsJob {
    static constexpr bool kAmn = kWmn, kBmn = false, kMask = false, kReads = false, kTwoPieces = true, kRagged = true;
    static constexpr int kUnit = 16 * kCG, kTall = kBM * kCG;
    CUtensorMap ta, ta_low, tb, tb_low, to;
    Offsets off;
    int N, pieces;
    void *out;
    int dtype;
    // shared memory: first[E + 1], before[E + 1], height of a tile, tiles down
    __device__ void begin(uint8_t *smem) const {
        int *first = reinterpret_cast<int *>(smem), *before = first + off.E + 1;
        off.read(first, before);
        if (threadIdx.x == 0) {
            // few tiles: lower ones where they fill the GPU's rounds better (each costs what its rows of W and of x need);
            // 16 experts of 1536 rows on 152 SMs: 192 tiles of 128 make two rounds, 256 of 96 two shorter ones.
            // (Without x's rows in the cost, dx of 40 experts of 100 rows, 5120 to 1536, took 64: 196 us against 139.)
            int best = kTall;
            if (kCG == 1) {
                int least = 0x7fffffff;
                const int cols = max(16, (first[off.E] - first[0]) / max(1, before[off.E]));
                for (int h = kBM; h >= (kWmn ? 64 : 32); h -= kWmn ? 64 : 32) {
                    const long long tiles = (long long)before[off.E] * ((N + h - 1) / h);
                    if (tiles > 16 * (int)gridDim.x) break; // many rounds: as they are
                    const int t = (int)((tiles + gridDim.x - 1) / gridDim.x) * (h + cols);
                    if (t < least) least = t, best = h;
                }
            }
            before[off.E + 1] = best;
            before[off.E + 2] = (N + best - 1) / best;
        }
        __syncthreads();
    }
    __device__ __forceinline__ int tiles(const uint8_t *smem) const {
        const int *before = reinterpret_cast<const int *>(smem) + off.E + 1;
        return before[off.E] * before[off.E + 2];
    }
    __device__ __forceinline__ Spot spot(const uint8_t *smem, int t) const {
        const int *first = reinterpret_cast<const int *>(smem), *before = first + off.E + 1;
        const int high = before[off.E + 1], tm = before[off.E + 2], u = t / tm;
        int e = 0; // the last with before[e] <= u
        for (int b = 1 << (31 - __clz(off.E)); b; b >>= 1)
            if (e + b <= off.E && before[e + b] <= u) e += b;
        const int r = t - before[e] * tm, r0 = first[e], n = first[e + 1] - r0, shares = before[e + 1] - before[e];
        // groups of 8 shares, W's rows moving slowest inside a group: the tiles in flight share their operands in L2
        const int per = 8 * tm, g = r / per, top = g * 8, gm = min(8, shares - top), i = r - g * per;
        const int share = top + i % gm, mi = i / gm;
        const int each = ((n + shares - 1) / shares + kUnit - 1) / kUnit * kUnit, left = n - share * each;
        Spot T;
        T.am = T.m = mi * high;
        T.az = e;
        T.bm = T.n = r0 + share * each;
        T.bz = 0;
        T.ak = T.bk = 0;
        T.pieces = pieces;
        T.left = min(each, left); // rows that are there
        T.rows = min(high, N - mi * high);
        T.cols = min(each, (left + kUnit - 1) / kUnit * kUnit);
        T.high = high / kCG;
        return T;
    }
    using Held = Nothing;
    using In = Nothing;
    // 32 columns of y (lane = column, o.rows of them there) of 32 rows from n on
    __device__ __forceinline__ void tile(Out32 &o, const Spot &T, int n, const float (&v)[32], const In &) const {
        const int rows = T.n + T.left - n;
        if (rows <= 0) return;
        if (!kAdd && rows >= 32) {
            if (dtype == WASTE_ACT_F32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t *t = reinterpret_cast<uint32_t *>(o.next());
                    if (o.lane / 16 == h)
#pragma unroll
                        for (int i = 0; i < 32; ++i) t[dense::turned(i, o.lane % 16 / 4, 4) * 4 + o.lane % 4] = __float_as_uint(v[i]);
                    send(o, t, o.m + 16 * h, n, 16 * h < o.rows);
                }
            } else {
                uint16_t *t = reinterpret_cast<uint16_t *>(o.next());
                // two rows at a time: their values of a column, rounded together
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const uint32_t w = dtype == WASTE_ACT_BF16 ? dense::two(v[i], v[i + 1], __nv_bfloat16()) : dense::two(v[i], v[i + 1], __half());
                    t[dense::turned(i, o.lane / 8, 4) * 8 + o.lane % 8] = (uint16_t)w;
                    t[dense::turned(i + 1, o.lane / 8, 4) * 8 + o.lane % 8] = (uint16_t)(w >> 16);
                }
                send(o, t, o.m, n, true);
            }
            return;
        }
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint4 *t = o.next();
            float *f = reinterpret_cast<float *>(t);
            if (o.lane / 16 == h)
#pragma unroll
                for (int i = 0; i < 32; ++i) f[dense::turned(i, o.lane % 16 / 4, 4) * 4 + o.lane % 4] = v[i];
            __syncwarp();
            const size_t at = (size_t)n * N + o.m + 16 * h;
            const int cols = N - o.m - 16 * h;
            if (dtype == WASTE_ACT_F32)
                dense::drain(t, static_cast<float *>(out) + at, N, rows, cols, true, kAdd, o.lane);
            else if (dtype == WASTE_ACT_BF16)
                dense::drain(t, static_cast<__nv_bfloat16 *>(out) + at, N, rows, cols, true, kAdd, o.lane);
            else
                dense::drain(t, static_cast<__half *>(out) + at, N, rows, cols, true, kAdd, o.lane);
        }
    }
    __device__ __forceinline__ void send(Out32 &o, const void *t, int x, int y, bool any) const {
        tc::fence_proxy_async();
        __syncwarp();
        if (o.lane == 0 && any) tc::tma_store(&to, x, y, tc::smem_u32(t));
    }
};

// dW: the rows are what is summed over.
template <int kCG, bool kAdd> struct WeightsJob {
    static constexpr int kHigh = kBM * kCG;
    static constexpr bool kAmn = true, kBmn = true, kMask = true, kReads = kAdd, kTwoPieces = !kAdd, kRagged = false;
    CUtensorMap ta, tb;
    Out<kAdd> out;
    Offsets off;
    int BN, tm, tn, M;
    __device__ void begin(uint8_t *smem) const { off.read(reinterpret_cast<int *>(smem), nullptr); }
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
        T.z = e;
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
        if (T.pieces || !kAdd) out.put(o, T, n, v, in);
    }
};

constexpr std::integral_constant<int, 1> kOne;
constexpr std::integral_constant<int, 2> kTwo;
constexpr std::true_type kYes;
constexpr std::false_type kNo;

// Whole widths of 32 columns, 256 at most.
int width(int n) { return n >= 256 ? 256 : n <= 64 ? 64 : (n + 31) / 32 * 32; }

// Pairs of CTAs from so many rows an expert on (their mean: the offsets are on the device): they halve the bytes of W
// an SM takes in for its columns, which counts once W is not what memory is read for.
bool pairs(const Group &G) { return G.rows / G.E >= 160; }
// For dW, whose sums are over an expert's rows, from more on: short sums leave the two CTAs waiting for each other's
// epilogues (40 x 1536 x 5120: 256 rows 205 us in pairs, 159 apart; 400 rows 253 and 259; 64 experts of 512 rows 540 and 615).
bool weight_pairs(const Group &G) { return G.rows / G.E >= 384 && G.n > kBM; }

// Columns of dW's tiles: as many as there are, 256 at most, or 64 by single CTAs where those leave SMs without work, by what
// the rounds of tiles take into an SM for a piece of the rows (dx and dW of 684 rows of one expert, 1192 x 152: 21.7 us and
// 16.1; two of 2985 rows, 1592 x 136: 43.8 and 36.9).
struct WeightsPlan {
    int BN;
    bool pair;
};
WeightsPlan weights_plan(const Group &G) {
    const int sms = device_sm_count();
    const auto cost = [&](const WeightsPlan &P) {
        const int high = P.pair ? 2 * kBM : kBM, slots = P.pair ? sms / 2 : sms;
        const long long tiles = (long long)G.E * ((G.n + high - 1) / high) * ((G.k + P.BN - 1) / P.BN);
        return (tiles + slots - 1) / slots * (kBM + P.BN / (P.pair ? 2 : 1));
    };
    const WeightsPlan wide{width(G.k), weight_pairs(G)}, narrow{64, false};
    return 5 * cost(narrow) < 4 * cost(wide) ? narrow : wide;
}

// What the tiles of y or dx (N columns) take into an SM for a piece of k, by rounds of tiles, were the rows spread evenly:
// single CTAs take the best of the heights that begin() has.
long long rows_cost(const Group &G, int N, int share, bool pair, bool mn, int sms) {
    const long long experts = G.E < G.rows ? G.E : G.rows, n = (G.rows + experts - 1) / experts, cuts = (n + share - 1) / share;
    const long long unit = pair ? 32 : 16, cols = ((n + cuts - 1) / cuts + unit - 1) / unit * unit, shares = experts * cuts;
    const auto rounds = [&](int high, int slots) { return (shares * ((N + high - 1) / high) + slots - 1) / slots; };
    if (pair) return rounds(2 * kBM, sms / 2) * (kBM + cols / 2);
    long long best = rounds(kBM, sms) * (kBM + cols);
    for (int h = kBM; h > 0; h -= mn ? 64 : 32) {
        const long long c = rounds(h, sms) * (h + cols);
        if (c < best) best = c;
    }
    return best;
}

// Rows of an expert in one tile, and whether a pair of CTAs takes it.  64 where there are few, so that the stages, which
// have room for as many, hold more of W on its way (one token, 16 rows of 16 experts: 73 us with 256, 59 with 64); and where
// wide tiles leave SMs without work (229 rows of one expert, 1912 to 104: 17.8 us and 12.7; 4 x 1150 rows, 184 to 216: 9.5 and 8.0).
struct RowsPlan {
    int share;
    bool pair;
};
RowsPlan rows_plan(const Group &G, int N, bool mn) {
    const RowsPlan P{G.rows / G.E < 32 ? 64 : 256, pairs(G)};
    const int sms = device_sm_count();
    const bool narrow = P.share > 64 && 5 * rows_cost(G, N, 64, false, mn, sms) < 4 * rows_cost(G, N, P.share, P.pair, mn, sms);
    return narrow ? RowsPlan{64, false} : P;
}

template <int kCG, bool kWmn, bool kAdd>
cudaError_t rows_product(const Group &G, int share, const void *a, int K, const void *w, int N, void *out, int out_dtype, cudaStream_t s) {
    RowsJob<kCG, kWmn, kAdd> J = {};
    TileArgs P = {};
    P.BN = J.off.share = share;
    J.off.p = G.offsets, J.off.E = G.E, J.off.rows = G.rows;
    J.N = N;
    J.pieces = (K + 63) / 64;
    J.out = out;
    J.dtype = out_dtype;
    cudaError_t e = stack_map(&J.ta, w, G.k, G.n, G.E, G.k, (size_t)G.k * G.n, kWmn ? 64 : kBM);
    if (e == cudaSuccess) e = stack_map(&J.ta_low, w, G.k, G.n, G.E, G.k, (size_t)G.k * G.n, 32);
    if (e == cudaSuccess) e = stack_map(&J.tb, a, K, G.rows, 1, K, (size_t)K * G.rows, 64);
    if (e == cudaSuccess) e = stack_map(&J.tb_low, a, K, G.rows, 1, K, (size_t)K * G.rows, 16);
    if (e == cudaSuccess) e = dense::store_map(&J.to, out, (int)dense::type_size(out_dtype), G.rows, N);
    if (e != cudaSuccess) return e;
    const long long shares = (long long)G.rows / P.BN + (G.E < G.rows ? G.E : G.rows);
    const int low = kCG == 2 ? J.kTall : kWmn ? 64 : 32;
    return launch_tiles_as<kCG>(P, J, G.dtype == WASTE_ACT_BF16, (size_t)(G.E + 2) * 8, shares * ((N + low - 1) / low),
                                device_sm_count(), s);
}

template <int kCG, bool kAdd>
cudaError_t weights_product(const Group &G, int BN, const void *dy, const void *x, void *dw, int grad_dtype, cudaStream_t s) {
    WeightsJob<kCG, kAdd> J = {};
    TileArgs P = {};
    P.BN = J.BN = BN;
    J.off = {G.offsets, G.E, G.rows, 0};
    J.M = G.n;
    J.tm = (G.n + J.kHigh - 1) / J.kHigh;
    J.tn = (G.k + J.BN - 1) / J.BN;
    cudaError_t e = stack_map(&J.ta, dy, G.n, G.rows, 1, G.n, (size_t)G.n * G.rows, 64);
    if (e == cudaSuccess) e = stack_map(&J.tb, x, G.k, G.rows, 1, G.k, (size_t)G.k * G.rows, 64);
    if (e == cudaSuccess) e = J.out.set(dw, G.E, G.n, G.k, grad_dtype);
    if (e != cudaSuccess) return e;
    return launch_tiles_as<kCG>(P, J, G.dtype == WASTE_ACT_BF16, (size_t)(G.E + 1) * 4, (long long)G.E * J.tm * J.tn,
                                device_sm_count(), s);
}

} // namespace

cudaError_t launch_group_forward(const Group &G, const void *x, const void *w, void *y, int out_dtype, int add, cudaStream_t s) {
    const RowsPlan R = rows_plan(G, G.n, false);
    const auto go = [&](auto cg, auto adds) {
        return rows_product<decltype(cg)::value, false, decltype(adds)::value>(G, R.share, x, G.k, w, G.n, y, out_dtype, s);
    };
    return R.pair ? (add ? go(kTwo, kYes) : go(kTwo, kNo)) : add ? go(kOne, kYes) : go(kOne, kNo);
}
cudaError_t launch_group_dx(const Group &G, const void *dy, const void *w, void *dx, cudaStream_t s) {
    const RowsPlan R = rows_plan(G, G.k, true);
    return R.pair ? rows_product<2, true, false>(G, R.share, dy, G.n, w, G.k, dx, G.dtype, s)
                  : rows_product<1, true, false>(G, R.share, dy, G.n, w, G.k, dx, G.dtype, s);
}
cudaError_t launch_group_dw(const Group &G, const void *dy, const void *x, void *dw, int grad_dtype, int add, cudaStream_t s) {
    const WeightsPlan W = weights_plan(G);
    const auto go = [&](auto cg, auto adds) {
        return weights_product<decltype(cg)::value, decltype(adds)::value>(G, W.BN, dy, x, dw, grad_dtype, s);
    };
    return W.pair ? (add ? go(kTwo, kYes) : go(kTwo, kNo)) : add ? go(kOne, kYes) : go(kOne, kNo);
}

cudaError_t group_word(uint32_t **word) { return dense::timeout_word(word); }
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
