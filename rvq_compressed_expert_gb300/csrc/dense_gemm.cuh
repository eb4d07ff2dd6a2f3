// The tensor-core product of the dense operators: D[m][n] = sum_k A[m][k] B[n][k] in fp32, on
// tcgen05.mma, with an epilogue that takes the sums on their way out.
//
// A CTA makes 128 x BN tiles (BN <= 256), or two CTAs together 256 x BN ones (cg = 2: each loads 128
// rows of A and half of B, and the tensor cores of both read both halves, so a tile needs two
// thirds of the bytes at BN = 256).  One thread moves 128-byte-wide pieces of A and B (64
// 16-bit or 256 4-bit values of k) into a ring of shared-memory stages by TMA; one thread issues
// the MMAs on full stages into one of two TMEM accumulators; eight warps take the other one out
// through the epilogue meanwhile.  Rows, columns and k past the matrices' ends arrive as zeros
// (TMA's fill), so any size works; the epilogue leaves them out.
//
// Two launch shapes (plan(), below):
//   S = 1: a persistent grid, one CTA per SM, each (or each pair) taking every so-manieth tile.
//   S > 1: where there are few tiles, a cluster of S CTAs per tile, each with its share of k; the
//          partial sums meet through distributed shared memory, each CTA adding up its share of
//          the tile in rank order (the same bits every time) and running the epilogue on it.
//
// What bounds it: at 256 x 256 a stage brings 32 KB into an SM for 512 cycles of MMAs, and an SM takes
// in about 100 B/ns, so loads and MMAs are near balance, and long 16-bit products run at the power
// limit.  Measured, calls one behind another, range over GPUs: block of 4096 tokens (d 7168, f 1536, bf16, g and u
// kept) 168 to 175 us = 1.54 to 1.61 PFLOP/s, its gradients 347 to 358 us = 1.51 to 1.56 PFLOP/s (cuBLAS sustains
// 1.71 on a square product); 4-bit 4096 x 7168 x 7168 68 to 71 us = 5.9 to 6.2 PFLOP/s, tensor pipe 63 % active.
//
// Waits are bounded: one that gives up (a second or so; for a tile's product longer, by its k) latches
// g_dense_timeout, which waste_dense_status reports, and the CTA winds up.
#pragma once

#include "dense.cuh"
#include "dense_tc.cuh"

namespace wm {
namespace dense {

// kOne: up to three independent products of one k in one launch; kSum: the same, each the sum of two;
// kPair: two products with the same A in one tile (columns [0, BN/2) by b0, the rest by b1).
enum { kOne, kPair, kSum };
enum { kHalf, kMx4 };

constexpr int kBM = 128;
constexpr int kRowBytes = 128; // bytes of one row of a stage
constexpr int kMaxStages = 8;
constexpr int kMaxProb = 3;
constexpr uint32_t kSmemBudget = 227 * 1024;
constexpr uint32_t kPieceBytes = 2048; // an epilogue warp's 32 rows x 64 bytes on their way out
constexpr uint32_t kBarBytes = 256;
constexpr int kThreads = 352; // loader, issuer, allocator, eight epilogue warps
constexpr int kTmemCols = 512;

struct Prob {
    int M, N, tm, tn, begin; // sizes, tiles, first tile
};
struct GemmArgs {
    CUtensorMap ta[kMaxProb], tb[kMaxProb];   // kPair: tb[0], tb[1] are the two products'
    CUtensorMap ta2[kMaxProb], tb2[kMaxProb]; // kSum: where pieces of k past kb_seg come from
    CUtensorMap sa, sb[2]; // 4-bit operands: their scale tiles, [row tile * skb + tile of blocks]
    Prob prob[kMaxProb];
    int nprob, tiles;
    int BN, S, stages, nacc;
    int kb_seg; // k pieces of the first part of a sum
    int kb;     // k pieces in all (kSum: twice as many)
    int K, skb;
    uint32_t idesc, smem;
    // early_b: B does not come from the kernel before this one, so its first pieces are asked for
    // before waiting for that kernel
    int early_b;
    // bytes that the next kernel reads and L2 can hold, asked for behind the own loads (or 0)
    const uint8_t *ahead;
    size_t ahead_bytes;
};

// Bytes of a stage in one CTA: 128 rows of A, its rows of B, the scale tiles of both.
__host__ __device__ inline uint32_t stage_b_bytes(int BN, int cg, bool b_mn) {
    const int rows = BN / cg;
    return (uint32_t)(b_mn ? (rows + 63) / 64 * 64 : rows) * kRowBytes;
}
__host__ __device__ inline uint32_t stage_size(int BN, int cg, bool b_mn, bool mx4) {
    const uint32_t n = kBM * kRowBytes + stage_b_bytes(BN, cg, b_mn) + (mx4 ? 1024u * (1 + (BN + 127) / 128) : 0u);
    return (n + 1023) & ~1023u;
}

struct Tile {
    int p, m0, n0, rows; // n0: first column of b0 (kPair: of both)
};
template <int kForm, int kCG> __device__ __forceinline__ Tile tile_at(const GemmArgs &P, int t, int rank) {
    int p = 0;
    if (kForm != kPair)
        while (p + 1 < P.nprob && t >= P.prob[p + 1].begin) ++p;
    const Prob &Q = P.prob[p];
    t -= Q.begin;
    // groups of 16 row tiles, columns moving slowest inside a group: the tiles in flight share
    // their operands in L2
    constexpr int kGroup = 16 / kCG;
    const int per = kGroup * Q.tn, g = t / per, first = g * kGroup, gm = min(kGroup, Q.tm - first), r = t - g * per;
    Tile o;
    o.p = p;
    o.m0 = (first + r % gm) * kBM * kCG + (kCG == 2 ? rank * kBM : 0);
    o.n0 = (r / gm) * (kForm == kPair ? P.BN / 2 : P.BN);
    o.rows = min(kBM, Q.M - o.m0); // none (or fewer) in a pair's second CTA
    return o;
}

// A warp's common answer, which the compiler knows to be common.
__device__ __forceinline__ bool all(bool v) { return __all_sync(0xffffffffu, v); }

// A wait for a whole tile's product, by the clock: 1.1 s, and 2 us for each piece of k (one takes 0.2 to 0.4).  Polls do
// not tell the time: one returns when another wait of the CTA ends, so beside the loop over k 2^18 of them were over
// in 60 ms.
__device__ __forceinline__ bool wait_tile(uint32_t bar, uint32_t parity, int pieces) {
    constexpr int kPolls = 1024;
    if (tc::mbar_wait(bar, parity, kPolls)) return true;
    const uint64_t end = tc::clock_ns() + 1100000000ull + 2000ull * (uint32_t)pieces;
    do {
        if (tc::mbar_wait(bar, parity, kPolls)) return true;
    } while (tc::clock_ns() < end);
    return false;
}

// One word in each translation unit that has kernels; read_and_clear_timeout reads its own.
static __device__ uint32_t g_dense_timeout;

// Its address, for the test aids.
static inline cudaError_t timeout_word(uint32_t **word) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_dense_timeout);
}
static inline cudaError_t read_and_clear_timeout(uint32_t *out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_dense_timeout, sizeof v);
    const uint32_t zero = 0;
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_dense_timeout, &zero, sizeof zero);
    *out |= v;
    return e;
}

// One stage of 4-bit operands: its scale tiles to tensor memory (a pair: each CTA's A rows, and all
// of B's, in both), and its MMAs, two to a half.  The scales have columns of their own for each
// stage (the stage is full again only after the MMAs that read them are done).  left: k from here on.
template <int kCG, int kNrt>
__device__ __forceinline__ void issue_mx4(uint32_t d, uint64_t da, uint64_t db, uint32_t sf, uint64_t ds, uint32_t idesc,
                                          int left, uint32_t acc) {
    const uint32_t id1 = idesc | (2u << 4) | (2u << 29); // the upper byte pair of the scale words
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h && left <= 128) return;
        const uint32_t fa = sf + 4 * h, fb = sf + 8 + 4 * kNrt * h;
#pragma unroll
        for (int i = 0; i <= kNrt; ++i) {
            const uint32_t to = i ? fb + 4 * (i - 1) : fa;
            const uint64_t from = ds + (uint64_t)((1024 * i + 512 * h) >> 4);
            if (kCG == 2)
                tc::copy_scales_pair(to, from);
            else
                tc::copy_scales(to, from);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j && left <= 128 * h + 64) return;
            const uint64_t off = (uint64_t)(2 * (2 * h + j));
            if (kCG == 2)
                tc::mma_mx4_pair(d, da + off, db + off, j ? id1 : idesc, fa, fb, acc);
            else
                tc::mma_mx4(d, da + off, db + off, j ? id1 : idesc, fa, fb, acc);
            acc = 1;
        }
    }
}

// v += the W floats at shared address src of each CTA of the cluster, in rank order; the loads of
// up to eight ranks are in flight at once, 8 floats at a time.
template <int W> __device__ __forceinline__ void add_ranks(uint32_t src, int S, float (&v)[W]) {
#pragma unroll
    for (int j = 0; j < W; j += 8) {
        float4 x[8][2];
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s < S) {
                const uint32_t a = tc::map_rank(src + 4 * j, s);
                x[s][0] = tc::ld_cluster(a);
                x[s][1] = tc::ld_cluster(a + 16);
            }
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s < S) {
                v[j] += x[s][0].x, v[j + 1] += x[s][0].y, v[j + 2] += x[s][0].z, v[j + 3] += x[s][0].w;
                v[j + 4] += x[s][1].x, v[j + 5] += x[s][1].y, v[j + 6] += x[s][1].z, v[j + 7] += x[s][1].w;
            }
    }
}

// An epilogue warp's 32 rows: the first, how many of them there are, and shared memory for two pieces of
// them, taken in turn (a copy may still read the other).
struct Out32 {
    uint4 *turn;
    int m, rows, lane, flip;
    __device__ __forceinline__ uint4 *next() {
        if (lane == 0) {
            tc::close_stores();
            tc::stores_read<1>();
        }
        __syncwarp();
        flip ^= 1;
        return turn + flip * (kPieceBytes / 16);
    }
};

// W columns of a row (kPair: of both products) from tensor memory to registers; complete after
// taken().
template <int W, int kForm> struct Sums {
    alignas(16) uint32_t v[W];
    alignas(16) uint32_t w[kForm == kPair ? W : 1];
    __device__ __forceinline__ void take(uint32_t src, int cols) {
        if constexpr (W == 32) {
            tc::tmem_ld32(src, v);
            if constexpr (kForm == kPair) tc::tmem_ld32(src + cols, w);
        } else {
            tc::tmem_ld16n(src, v);
            if constexpr (kForm == kPair) tc::tmem_ld16n(src + cols, w);
        }
    }
    __device__ __forceinline__ void taken() {
        tc::tmem_wait_ld(v);
        if constexpr (kForm == kPair) tc::tmem_wait_ld(w);
    }
    // to the partial sums' row
    __device__ __forceinline__ void keep(float4 *part, int cols, int c) const {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            part[c / 4 + i] = *reinterpret_cast<const float4 *>(&v[4 * i]);
            if constexpr (kForm == kPair) part[(cols + c) / 4 + i] = *reinterpret_cast<const float4 *>(&w[4 * i]);
        }
    }
    // 32 rows (the warp's) from row m on, `rows` of them valid
    template <class Epi>
    __device__ __forceinline__ void give(const Epi &epi, const Tile &T, Out32 &o, int c) const {
        const auto &x = *reinterpret_cast<const float(*)[W]>(v);
        if constexpr (kForm == kPair)
            epi.template tile<W>(o, T.p, T.n0 + c, x, *reinterpret_cast<const float(*)[W]>(w));
        else
            epi.template tile<W>(o, T.p, T.n0 + c, x, x);
    }
};

template <int kCG, int kKind, int kForm, bool kAmn, bool kBmn, class Epi>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs P, const __grid_constant__ Epi epi) {
    extern __shared__ __align__(1024) uint8_t smem_raw[]; // stages, pieces on their way out, barriers
    const uint32_t smem0 = tc::smem_u32(smem_raw), base = smem0;
    const uint32_t bars_at = P.smem - kBarBytes;
    const uint32_t bars = smem0 + bars_at; // full[8], empty[8], accfull[2], accempty[2]
    const uint32_t bar_full = bars, bar_empty = bars + 64, bar_accf = bars + 128, bar_acce = bars + 144;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + bars_at + 160);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem_raw + bars_at + 164);
    const uint32_t drain = bars + 168;

    // one value a warp, and known to be: the loops' addresses stay in uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int BN = P.BN, S = kCG == 2 ? 1 : P.S;
    const uint32_t a_bytes = kBM * kRowBytes, b_bytes = stage_b_bytes(BN, kCG, kBmn);
    const uint32_t s_off = a_bytes + b_bytes, stage_bytes = stage_size(BN, kCG, kBmn, kKind == kMx4);
    const int nrt = (BN + 127) >> 7; // scale tiles of B
    const int rank = kCG == 2 ? (int)(blockIdx.x & 1) : S > 1 ? (int)(blockIdx.x % S) : 0; // in the cluster
    const bool leads = kCG == 1 || rank == 0; // issues the MMAs

    if (warp == 0 && P.early_b) tc::see_complete(); // while the others set up
    if (tid == 32) {
        for (int i = 0; i < P.stages; ++i) {
            tc::mbar_init(bar_full + 8 * i, 1);
            tc::mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar_accf + 8 * i, 1);
            tc::mbar_init(bar_acce + 8 * i, 8 * kCG);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::mbar_init_fence();
    }
    if (warp == 2) {
        if (kCG == 2)
            tc::tmem_alloc_pair(tc::smem_u32(tmem_slot), kTmemCols);
        else
            tc::tmem_alloc(tc::smem_u32(tmem_slot), kTmemCols);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (kCG == 2) tc::cluster_sync(); // the other CTA's barriers are up
    tc::fence_after_sync();
    constexpr uint32_t tmem = 0; // all columns are this CTA's, so they start at the first
    if (*tmem_slot != tmem && tid == 0) *abort_flag = 1;
    if (warp != 0) tc::grid_wait(); // warp 0's loader may have B's first pieces to ask for before

    const int kb0 = S > 1 ? (int)((long long)P.kb * rank / S) : 0;
    const int kb1 = S > 1 ? (int)((long long)P.kb * (rank + 1) / S) : P.kb;
    const int tile0 = S > 1 ? (int)blockIdx.x / S : (int)blockIdx.x / kCG;
    const int step = S > 1 ? P.tiles : (int)gridDim.x / kCG;
    const auto acc_at = [&](int buf) { return tmem + buf * (kKind == kMx4 ? BN : 256); };

    if (warp == 0) {
        // ---- loader (the warp walks the loop, an elected lane issues).  A pair's CTAs load their own
        // rows of A and their half of B; the bytes of both count on the first one's barrier, which
        // announces them.
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        const uint32_t full0 = kCG == 2 ? tc::map_rank(bar_full, 0) : bar_full;
        const auto load = [](uint32_t dst, const CUtensorMap *m, int x, int y, uint32_t bar) {
            if (kCG == 2)
                tc::tma_load_pair(dst, m, x, y, bar);
            else
                tc::tma_load(dst, m, x, y, bar);
        };
        const auto load_a = [&](const Tile &T, int kb, int st) {
            const uint32_t sa = base + st * stage_bytes, full = full0 + 8 * st;
            const bool second = kForm == kSum && kb >= P.kb_seg;
            const int k = second ? kb - P.kb_seg : kb;
            const CUtensorMap *ta = second ? &P.ta2[T.p] : &P.ta[T.p];
            const int kx = kKind == kMx4 ? k * kRowBytes : k * 64;
            if (kAmn) {
                for (int i = 0; i < kBM / 64; ++i) load(sa + i * 8192, ta, T.m0 + 64 * i, kx, full);
            } else {
                load(sa, ta, kx, T.m0, full);
            }
            if (kKind == kMx4) load(sa + s_off, &P.sa, 0, (T.m0 >> 7) * P.skb + 2 * k, full);
        };
        // also announces the bytes of the whole stage
        const auto load_b = [&](const Tile &T, int kb, int st) {
            const uint32_t sb = base + st * stage_bytes + a_bytes, full = full0 + 8 * st;
            const bool second = kForm == kSum && kb >= P.kb_seg;
            const int k = second ? kb - P.kb_seg : kb;
            const CUtensorMap *tb = second ? &P.tb2[T.p] : &P.tb[kForm == kPair ? (kCG == 2 ? rank : 0) : T.p];
            const int kx = kKind == kMx4 ? k * kRowBytes : k * 64;
            const int n0 = T.n0 + (kCG == 2 && kForm != kPair ? rank * (BN / 2) : 0);
            if (leads)
                tc::mbar_arrive_expect_tx(bar_full + 8 * st,
                                          kCG * (a_bytes + b_bytes + (kKind == kMx4 ? 1024u * (1 + nrt) : 0u)));
            if (kBmn) {
                for (uint32_t i = 0; i * 8192 < b_bytes; ++i) load(sb + i * 8192, tb, n0 + 64 * i, kx, full);
            } else {
                load(sb, tb, kx, n0, full);
                if (kForm == kPair && kCG == 1) load(sb + b_bytes / 2, &P.tb[1], kx, n0, full);
            }
            if (kKind == kMx4)
                for (int i = 0; i < nrt; ++i)
                    load(sb + b_bytes + 1024 * (1 + i), &P.sb[kForm == kPair ? i : 0], 0,
                         ((T.n0 >> 7) + (kForm == kPair ? 0 : i)) * P.skb + 2 * k, full);
        };
        int early = 0;
        if (P.early_b && tile0 < P.tiles) {
            early = min(P.stages, kb1 - kb0);
            const Tile T = tile_at<kForm, kCG>(P, tile0, rank);
            if (tc::elect_one())
                for (int i = 0; i < early; ++i) load_b(T, kb0 + i, i);
            __syncwarp();
        }
        tc::grid_wait_release();
        for (int t = tile0; t < P.tiles && ok; t += step) {
            const Tile T = tile_at<kForm, kCG>(P, t, rank);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (issued >= early) {
                    if (!all(tc::mbar_wait(bar_empty + 8 * st, ph ^ 1))) {
                        ok = false;
                        break;
                    }
                }
                if (tc::elect_one()) {
                    if (issued >= early) load_b(T, kb, st);
                    load_a(T, kb, st);
                }
                __syncwarp();
                ++issued;
                if (++st == P.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (P.ahead_bytes && lane == 0) {
            // this CTA's share, in pieces of 16 KiB
            const size_t n = (P.ahead_bytes + 16383) >> 14;
            for (size_t i = blockIdx.x; i < n; i += gridDim.x) {
                const size_t left = P.ahead_bytes - (i << 14);
                tc::prefetch_l2(P.ahead + (i << 14), left < 16384 ? (uint32_t)left : 16384u);
            }
        }
        if (!ok) {
            // copies in flight land before the CTA goes: the last rounds' full barriers
            if (lane == 0) *abort_flag = 1;
            const int n = min(issued, P.stages);
            for (int i = 0; i < n && leads; ++i) {
                const int j = issued - n + i;
                tc::mbar_wait(bar_full + 8 * (j % P.stages), (j / P.stages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leads) {
            // ---- MMA issuer.  The whole warp walks the loop and one elected lane issues, so that
            // addresses and descriptors stay in the warp's uniform registers, where the tensor
            // core takes them from: a loop inside "if (lane == 0)" moves each operand there anew.
            const auto commit = [](uint32_t bar) {
                if (kCG == 2)
                    tc::mma_commit_pair(bar);
                else
                    tc::mma_commit(bar);
            };
            int st = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true;
            const uint64_t scales0 = tc::desc_scales(base + s_off);
            const uint64_t desc0 = tc::desc_sw128(base, kKind == kHalf ? 8192 : 16);
            for (int t = tile0; t < P.tiles && ok; t += step, ++it) {
                const int buf = P.nacc == 2 ? it & 1 : 0;
                const uint32_t use = P.nacc == 2 ? it >> 1 : it;
                if (!all(tc::mbar_wait(bar_acce + 8 * buf, (use & 1) ^ 1))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t d = acc_at(buf);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!all(tc::mbar_wait(bar_full + 8 * st, ph))) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint64_t da = desc0 + (uint64_t)((st * stage_bytes) >> 4), db = da + (uint64_t)(a_bytes >> 4);
                    if (tc::elect_one()) {
                        if (kKind == kHalf) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint64_t dj = da + (uint64_t)(j * ((kAmn ? 2048 : 32) >> 4));
                                const uint64_t ej = db + (uint64_t)(j * ((kBmn ? 2048 : 32) >> 4));
                                const uint32_t acc = j > 0 || kb > kb0;
                                if (kCG == 2)
                                    tc::mma_f16_pair(d, dj, ej, P.idesc, acc);
                                else
                                    tc::mma_f16(d, dj, ej, P.idesc, acc);
                            }
                        } else {
                            const uint32_t sf = tmem + P.nacc * BN + st * (8 + 8 * nrt);
                            const uint64_t ds = scales0 + (uint64_t)((st * stage_bytes) >> 4);
                            const int left = P.K - kb * 256;
                            if (nrt == 2)
                                issue_mx4<kCG, 2>(d, da, db, sf, ds, P.idesc, left, kb > kb0);
                            else
                                issue_mx4<kCG, 1>(d, da, db, sf, ds, P.idesc, left, kb > kb0);
                        }
                        commit(bar_empty + 8 * st);
                        if (kb + 1 == kb1) commit(bar_accf + 8 * buf);
                    }
                    __syncwarp();
                    if (++st == P.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) {
                if (lane == 0) *abort_flag = 1;
                if (tc::elect_one()) commit(drain);
                tc::mbar_wait(drain, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 3) {
        // ---- epilogue: two warps for each quarter of the lanes (rows); they take its pieces of 32
        // columns in turn
        const int q = warp & 3, half = (warp - 3) >> 2, r = 32 * q + lane;
        const int cols = kForm == kPair ? BN / 2 : BN;
        // split k: this CTA's partial sums go to shared memory, rows padded by 16 bytes
        float4 *part = S > 1 ? reinterpret_cast<float4 *>(smem_raw) + r * (BN / 4 + 1) : nullptr;
        Out32 out{reinterpret_cast<uint4 *>(smem_raw + P.stages * stage_bytes) + (warp - 3) * (2 * kPieceBytes / 16), 0, 0,
                  lane, 0};
        int it = 0;
        for (int t = tile0; t < P.tiles; t += step, ++it) {
            const Tile T = tile_at<kForm, kCG>(P, t, rank);
            const int buf = P.nacc == 2 ? it & 1 : 0;
            const uint32_t use = P.nacc == 2 ? it >> 1 : it;
            if constexpr (Epi::kAhead)
                if (S == 1 && r < T.rows && half == 0) epi.ahead(T.m0 + r, T.n0, cols);
            bool ok = true;
            if (lane == 0) ok = wait_tile(bar_accf + 8 * buf, use & 1, kb1 - kb0);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                *abort_flag = 1;
                break;
            }
            tc::fence_after_sync();
            const uint32_t src = acc_at(buf) + ((uint32_t)(32 * q) << 16);
            const auto free_acc = [&] {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (leads)
                        tc::mbar_arrive(bar_acce + 8 * buf);
                    else
                        tc::mbar_arrive_cluster(tc::map_rank(bar_acce + 8 * buf, 0));
                }
            };
            const bool any = 32 * q < T.rows;
            out.m = T.m0 + 32 * q;
            out.rows = T.rows - 32 * q;
            if constexpr (kKind == kMx4) {
                // one accumulator (the other's place holds scales): all of it to registers first,
                // so that the next tile's MMAs wait for the reading alone
                constexpr int kHeld = kForm == kPair ? 2 : 4;
                Sums<32, kForm> x[kHeld];
                if (any) {
#pragma unroll
                    for (int i = 0; i < kHeld; ++i)
                        if (64 * i + 32 * half < cols) x[i].take(src + 64 * i + 32 * half, cols);
#pragma unroll
                    for (int i = 0; i < kHeld; ++i)
                        if (64 * i + 32 * half < cols) x[i].taken();
                }
                free_acc();
                const auto out_one = [&](const Sums<32, kForm> &s, int c) {
                    if (c >= cols) return;
                    if (!part)
                        s.give(epi, T, out, c);
                    else if (r < T.rows)
                        s.keep(part, cols, c);
                };
                if (any) { // written out: as a loop this is not unrolled, and x goes to local memory
                    out_one(x[0], 32 * half);
                    out_one(x[1], 64 + 32 * half);
                    if constexpr (kHeld == 4) {
                        out_one(x[2], 128 + 32 * half);
                        out_one(x[3], 192 + 32 * half);
                    }
                }
            } else {
                if (any) {
                    for (int c = 32 * half; c < cols; c += 64) {
                        if (c + 32 <= cols) {
                            Sums<32, kForm> x;
                            x.take(src + c, cols);
                            x.taken();
                            if (!part)
                                x.give(epi, T, out, c);
                            else if (r < T.rows)
                                x.keep(part, cols, c);
                        } else {
                            Sums<16, kForm> x;
                            x.take(src + c, cols);
                            x.taken();
                            if (!part)
                                x.give(epi, T, out, c);
                            else if (r < T.rows)
                                x.keep(part, cols, c);
                        }
                    }
                }
                free_acc();
            }
        }
        if (lane == 0) {
            tc::close_stores();
            tc::stores_done();
        }
        __syncwarp();
    }
    if (S > 1) {
        __syncthreads();
        tc::cluster_sync();
        const Tile T = tile_at<kForm, kCG>(P, tile0, rank);
        constexpr int W = Epi::kWidth, kLanes = Epi::kLanes;
        const int cols = kForm == kPair ? BN / 2 : BN, nc = cols / W, items = T.rows * nc / kLanes;
        // items of W columns for kLanes lanes each, a contiguous share for each CTA of the cluster
        const int i1 = (int)((long long)items * (rank + 1) / S) * kLanes;
        for (int i = (int)((long long)items * rank / S) * kLanes + tid; i < i1; i += kThreads) {
            const int rr = i / nc, c = (i - rr * nc) * W;
            float v[W], w[W];
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] = w[j] = 0.f;
            const uint32_t src = base + (uint32_t)(rr * (BN + 4) + c) * 4;
            add_ranks<W>(src, S, v);
            if (kForm == kPair) add_ranks<W>(src + 4 * cols, S, w);
            epi.template row<W>(T.p, T.m0 + rr, T.n0 + c, v, w);
        }
        tc::cluster_sync(); // no CTA leaves while another reads its sums
    }
    tc::fence_before_sync();
    __syncthreads();
    if (kCG == 2) tc::cluster_sync(); // nor while its memory takes part in the other's MMAs or barriers
    tc::fence_after_sync();
    if (tid == 0 && *abort_flag) atomicOr(&g_dense_timeout, 1u);
    if (warp == 2) {
        if (kCG == 2)
            tc::tmem_dealloc_pair(tmem, kTmemCols);
        else
            tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- tensor maps (host) --------------------------------------------------------------------

// A tiled tensor map of rank 2 or 3 (strides in bytes, of all dimensions but the first).
cudaError_t encode_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *p, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion l2);

// A tensor map over rows x row_bytes bytes (contiguous rows): boxes of box_rows rows x 128 bytes,
// 128-byte swizzle, zeros past the ends.  unit: bytes of one coordinate step (2 or 1).
cudaError_t make_map(CUtensorMap *m, const void *p, int unit, int rows, size_t row_bytes, int box_rows);

// A tensor map over scale tiles (512 bytes each): boxes of two tiles.
cudaError_t make_scale_map(CUtensorMap *m, const void *p, size_t tiles);

// A tensor map to store a matrix of rows x cols values of 2 or 4 bytes by (cols * bytes % 16 == 0): boxes
// of 32 rows x 64 bytes, 64-byte swizzle.
cudaError_t store_map(CUtensorMap *m, void *p, int bytes, int rows, int cols);

// ---- epilogues -----------------------------------------------------------------------------
// kTurns: tile() needs the shared memory of Out32, and maps() makes tensor maps of the outputs for it.
// ahead(m, n, cols) (kAhead): row m of a tile will be taken from column n on.  row<W>(p, m, n, c, c2): W consecutive sums of row m from column n of problem p (n a multiple
// of W; kLanes neighbouring lanes take neighbouring pieces at once); columns at or past N are left out.  tile<W>(o, p, n, c, c2): the same for the 32 rows of
// a warp, lane = row, all lanes together.

template <class O> __device__ __forceinline__ O round_to(float v);
template <> __device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half round_to<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float round_to<float>(float v) { return v; }

template <class O> struct Pack {
    uint4 q;
    __device__ float get(int i) const { return (float)reinterpret_cast<const O *>(&q)[i]; }
};

// A 16-byte piece of rounded values, two at a time where the type allows.
__device__ __forceinline__ uint4 piece_of(const float *v, float) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint32_t two(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t two(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <class O> __device__ __forceinline__ uint4 piece_of(const float *v, O t) {
    return make_uint4(two(v[0], v[1], t), two(v[2], v[3], t), two(v[4], v[5], t), two(v[6], v[7], t));
}

// W values to p[0..W) (columns n..): whole 16-byte pieces where the row allows, add: to what is there.
template <class O, int W>
__device__ __forceinline__ void put(O *p, int n, int N, bool vec, bool add, const float (&v)[W]) {
    constexpr int kPer = 16 / sizeof(O);
    static_assert(W % kPer == 0, "whole pieces");
#pragma unroll
    for (int i = 0; i < W; i += kPer) {
        if (vec && n + i + kPer <= N) {
            float w[kPer];
            Pack<O> o;
            if (add) o.q = *reinterpret_cast<const uint4 *>(p + i);
#pragma unroll
            for (int j = 0; j < kPer; ++j) w[j] = add ? o.get(j) + v[i + j] : v[i + j];
            *reinterpret_cast<uint4 *>(p + i) = piece_of(w, O());
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (n + i + j < N) p[i + j] = round_to<O>(add ? (float)p[i + j] + v[i + j] : v[i + j]);
        }
    }
}
template <int W>
__device__ __forceinline__ void put_as(int dtype, void *out, size_t at, int n, int N, bool vec, bool add,
                                       const float (&v)[W]) {
    if (dtype == WASTE_ACT_F32)
        put(static_cast<float *>(out) + at, n, N, vec, add, v);
    else if (dtype == WASTE_ACT_BF16)
        put(static_cast<__nv_bfloat16 *>(out) + at, n, N, vec, add, v);
    else
        put(static_cast<__half *>(out) + at, n, N, vec, add, v);
}
// What rounding v to the 16-bit type leaves, rounded to it (in fp16 below 2^-14, so for |v| < 2^-3, to
// multiples of 2^-24); nothing where it leaves the type's range.
template <int W>
__device__ __forceinline__ void put_rest(int dtype, void *out, size_t at, int n, int N, const float (&v)[W]) {
    float r[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float h = dtype == WASTE_ACT_BF16 ? (float)__float2bfloat16_rn(v[i]) : (float)__float2half_rn(v[i]);
        r[i] = isinf(h) ? 0.f : v[i] - h;
    }
    put_as(dtype, out, at, n, N, true, false, r);
}

// The same for the 32 rows of a warp, lane = row: the values cross through shared memory in pieces of 64
// bytes a row.  map: a tensor map over the matrix (store_map), whose copies take the rounded values
// from there and leave out what is past its ends; or null (rows without whole 16-byte pieces, sums added
// to what is there): the fp32 values go in, and drain() takes them out, consecutive lanes
// consecutive pieces of a row.  A lane storing its own row touches 32 rows with every instruction:
// 2048 x 7168 x 1536 in 4 bits to bf16 22.0 us that way, 18.8 with pieces stored by the lanes, 15.7 by copies.
__device__ __forceinline__ int turned(int row, int piece, int pieces) {
    // pieces is 2 or 4; permuted so that neither the writes (lane = row) nor the reads (lane = piece)
    // meet in a bank (the maps' 64-byte swizzle)
    return row * pieces + (piece ^ ((row * pieces >> 3) & (pieces - 1)));
}
// 16 columns of `rows` rows; out: their first value, cols: columns of the matrix from there on.
template <class O>
__device__ __forceinline__ void drain(const uint4 *turn, O *out, size_t ld, int rows, int cols, bool vec, bool add, int lane) {
    struct alignas(4 * sizeof(O)) Four {
        O v[4];
    };
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int at = 32 * i + lane, row = at / 4, piece = at % 4, c = 4 * piece;
        const uint4 q = turn[turned(row, piece, 4)];
        const float x[4] = {__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w)};
        O *p = out + (size_t)row * ld + c;
        if (row >= rows) continue;
        if (vec && c + 4 <= cols) {
            Four y;
            if (add) y = *reinterpret_cast<const Four *>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j) y.v[j] = round_to<O>(add ? (float)y.v[j] + x[j] : x[j]);
            *reinterpret_cast<Four *>(p) = y;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < cols) p[j] = round_to<O>(add ? (float)p[j] + x[j] : x[j]);
        }
    }
}
// 64 bytes of each row through a map
template <class O>
__device__ __forceinline__ void send(Out32 &o, const CUtensorMap *map, int n, int N, const float *v) {
    constexpr int kPer = 16 / (int)sizeof(O);
    uint4 *turn = o.next();
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[turned(o.lane, i, 4)] = piece_of(v + kPer * i, O());
    tc::fence_proxy_async();
    __syncwarp();
    if (o.lane == 0 && n < N) tc::tma_store(map, n, o.m, tc::smem_u32(turn));
}
template <int W>
__device__ __forceinline__ void put32_as(int dtype, Out32 &o, const CUtensorMap *map, void *out, size_t ld, int n, int N,
                                         bool vec, bool add, const float (&v)[W]) {
    if (W == 32 && map) {
        if (dtype == WASTE_ACT_BF16) {
            send<__nv_bfloat16>(o, map, n, N, v);
        } else if (dtype == WASTE_ACT_F16) {
            send<__half>(o, map, n, N, v);
        } else {
            send<float>(o, map, n, N, v);
            send<float>(o, map, n + 16, N, v + 16);
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < W; h += 16) {
        uint4 *turn = o.next();
#pragma unroll
        for (int i = 0; i < 4; ++i) turn[turned(o.lane, i, 4)] = piece_of(v + h + 4 * i, 0.f);
        __syncwarp();
        const size_t at = (size_t)o.m * ld + n + h;
        const int cols = N - n - h;
        if (dtype == WASTE_ACT_F32)
            drain(turn, static_cast<float *>(out) + at, ld, o.rows, cols, vec, add, o.lane);
        else if (dtype == WASTE_ACT_BF16)
            drain(turn, static_cast<__nv_bfloat16 *>(out) + at, ld, o.rows, cols, vec, add, o.lane);
        else
            drain(turn, static_cast<__half *>(out) + at, ld, o.rows, cols, vec, add, o.lane);
    }
}
// W columns of a 16-bit matrix for the 32 rows of a warp, lane = row (rows of N % 8 == 0 columns;
// zeros past the ends).
template <int W>
__device__ __forceinline__ void get32(Out32 &o, const void *src, size_t ld, int n, int N, uint4 (&q)[W / 8]) {
    constexpr int kPieces = W / 8;
    uint4 *turn = o.next();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int at = 32 * i + o.lane, row = at / kPieces, piece = at % kPieces, c = n + 8 * piece;
        const bool in = row < o.rows && c < N;
        const uint16_t *p = static_cast<const uint16_t *>(src) + (size_t)(o.m + row) * ld + c;
        turn[turned(row, piece, kPieces)] = in ? *reinterpret_cast<const uint4 *>(p) : uint4{};
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) q[i] = turn[turned(o.lane, i, kPieces)];
}

// 8 values of a 16-bit type
__device__ __forceinline__ void widen8(bool bf16, const uint4 &q, float (&v)[8]) {
    if (bf16) {
        const Pack<__nv_bfloat16> p{q};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p.get(i);
    } else {
        const Pack<__half> p{q};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p.get(i);
    }
}

struct Store {
    static constexpr int kWidth = 8, kLanes = 1;
    static constexpr bool kTurns = true;
    static constexpr bool kAhead = false;
    CUtensorMap map[kMaxProb];
    void *out[kMaxProb];
    int ld[kMaxProb];
    int dtype, add, vec;
    bool whole; // by the maps
    cudaError_t maps(const GemmArgs &G) {
        whole = vec && !add;
        cudaError_t e = cudaSuccess;
        for (int i = 0; whole && i < G.nprob && e == cudaSuccess; ++i)
            e = store_map(&map[i], out[i], (int)type_size(dtype), G.prob[i].M, ld[i]);
        return e;
    }
    // selected, not indexed: an index would put a copy of the whole in local memory, whose loads
    // miss the little L1 that the stages leave
    __device__ __forceinline__ void *to(int p) const { return p == 0 ? out[0] : p == 1 ? out[1] : out[2]; }
    __device__ __forceinline__ int row_of(int p) const { return p == 0 ? ld[0] : p == 1 ? ld[1] : ld[2]; }
    template <int W>
    __device__ __forceinline__ void row(int p, int m, int n, const float (&c)[W], const float (&)[W]) const {
        const int w = row_of(p);
        put_as(dtype, to(p), (size_t)m * w + n, n, w, vec, add, c);
    }
    template <int W>
    __device__ __forceinline__ void tile(Out32 &o, int p, int n, const float (&c)[W], const float (&)[W]) const {
        const int w = row_of(p);
        put32_as(dtype, o, whole ? &map[p] : nullptr, to(p), w, n, w, vec, add, c);
    }
};

// a = silu(g) u; g and u kept if asked for.  f % 8 == 0, so rows hold whole 16-byte pieces.
struct Gated {
    static constexpr int kWidth = 8, kLanes = 1;
    static constexpr bool kTurns = true;
    static constexpr bool kAhead = false;
    CUtensorMap map[3];
    void *a, *g, *u;
    int f, dtype;
    cudaError_t maps(const GemmArgs &G) {
        void *p[3] = {a, g, u};
        cudaError_t e = cudaSuccess;
        for (int i = 0; i < 3 && p[i] && e == cudaSuccess; ++i) e = store_map(&map[i], p[i], 2, G.prob[0].M, f);
        return e;
    }
    template <int W>
    __device__ __forceinline__ void row(int, int m, int n, const float (&cg)[W], const float (&cu)[W]) const {
        const size_t at = (size_t)m * f + n;
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = cg[i] * sigmoid(cg[i]) * cu[i];
        put_as(dtype, a, at, n, f, true, false, v);
        if (g) {
            put_as(dtype, g, at, n, f, true, false, cg);
            put_as(dtype, u, at, n, f, true, false, cu);
        }
    }
    template <int W>
    __device__ __forceinline__ void tile(Out32 &o, int, int n, const float (&cg)[W], const float (&cu)[W]) const {
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = cg[i] * sigmoid(cg[i]) * cu[i];
        put32_as(dtype, o, &map[0], a, f, n, f, true, false, v);
        if (g) {
            put32_as(dtype, o, &map[1], g, f, n, f, true, false, cg);
            put32_as(dtype, o, &map[2], u, f, n, f, true, false, cu);
        }
    }
};

// da -> a, dg, du from the kept g and u, which are asked of L2 while the tile's product runs.
struct GatedGrad {
    static constexpr int kWidth = 8, kLanes = 1;
    static constexpr bool kTurns = true;
    static constexpr bool kAhead = true;
    CUtensorMap map[3];
    const void *g, *u;
    void *a, *dg, *du;
    int f, dtype;
    cudaError_t maps(const GemmArgs &G) {
        void *p[3] = {a, dg, du};
        cudaError_t e = cudaSuccess;
        for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = store_map(&map[i], p[i], 2, G.prob[0].M, f);
        return e;
    }
    void *a_lo, *dg_lo, *du_lo; // what rounding them left, or null (row() alone)
    __device__ __forceinline__ void ahead(int m, int n, int cols) const {
        const char *pg = static_cast<const char *>(g) + ((size_t)m * f + n) * 2;
        const char *pu = static_cast<const char *>(u) + ((size_t)m * f + n) * 2;
        const int bytes = min(cols, f - n) * 2;
        for (int i = 0; i < bytes; i += 128) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(pg + i));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(pu + i));
        }
    }
    // one piece of 8 columns: a, dg and du
    __device__ __forceinline__ void grads(const uint4 &qg, const uint4 &qu, const float *da, float *x, float *y,
                                          float *z) const {
        float gv[8], uv[8];
        widen8(dtype == WASTE_ACT_BF16, qg, gv);
        widen8(dtype == WASTE_ACT_BF16, qu, uv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid(gv[j]), silu = gv[j] * s;
            x[j] = silu * uv[j];
            y[j] = da[j] * (uv[j] * (s * (1.f + gv[j] * (1.f - s)))); // no factor past the result's range
            z[j] = da[j] * silu;
        }
    }
    template <int W>
    __device__ __forceinline__ void row(int, int m, int n, const float (&da)[W], const float (&)[W]) const {
        static_assert(W == 8, "one piece");
        if (n >= f) return; // f % 8 == 0
        const size_t at = (size_t)m * f + n;
        float x[8], y[8], z[8];
        grads(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(g) + at),
              *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(u) + at), da, x, y, z);
        put_as(dtype, a, at, n, f, true, false, x);
        put_as(dtype, dg, at, n, f, true, false, y);
        put_as(dtype, du, at, n, f, true, false, z);
        if (a_lo) {
            put_rest(dtype, a_lo, at, n, f, x);
            put_rest(dtype, dg_lo, at, n, f, y);
            put_rest(dtype, du_lo, at, n, f, z);
        }
    }
    template <int W>
    __device__ __forceinline__ void tile(Out32 &o, int, int n, const float (&da)[W], const float (&)[W]) const {
        uint4 qg[W / 8], qu[W / 8];
        get32<W>(o, g, f, n, f, qg);
        get32<W>(o, u, f, n, f, qu);
        float x[W], y[W], z[W];
#pragma unroll
        for (int i = 0; i < W / 8; ++i) grads(qg[i], qu[i], da + 8 * i, x + 8 * i, y + 8 * i, z + 8 * i);
        put32_as(dtype, o, &map[0], a, f, n, f, true, false, x);
        put32_as(dtype, o, &map[1], dg, f, n, f, true, false, y);
        put32_as(dtype, o, &map[2], du, f, n, f, true, false, z);
    }
};

// ---- host side -----------------------------------------------------------------------------

// L2 holds this much of the next kernel's weights beside what is in flight.
constexpr size_t kAheadMost = 48u << 20;

// Launch shape from the sizes alone: tile width, CTAs per tile that split k, and CTAs (1 or 2)
// that make one tile together, for n products of sizes (M, N) and kb pieces of k.  pair: a tile
// holds BN / 2 columns of each of two products.
struct Plan {
    int BN, S, cg;
    double ns; // estimated
};
int clusters_at_once(int S); // clusters of S CTAs that run at once
Plan plan(const int *M, const int *N, int n, int kb, bool pair, bool mx4, int sms, bool heavy = false);

// Fills in the plan and the tiles.
inline void set_shape(GemmArgs &G, const Plan &L, const int *M, const int *N, int n, bool pair) {
    G.BN = L.BN;
    G.S = L.S;
    G.nprob = n;
    G.tiles = 0;
    const int h = kBM * L.cg, w = pair ? L.BN / 2 : L.BN;
    for (int i = 0; i < n; ++i) {
        G.prob[i] = Prob{M[i], N[i], (M[i] + h - 1) / h, (N[i] + w - 1) / w, G.tiles};
        G.tiles += G.prob[i].tm * G.prob[i].tn;
    }
}
// Rows of B's boxes (K-major).
inline int box_rows_b(const Plan &L, bool pair) { return pair || L.cg == 2 ? L.BN / 2 : L.BN; }

template <int kCG, int kKind, int kForm, bool kAmn, bool kBmn, class Epi>
cudaError_t launch_gemm_as(GemmArgs &G, Epi &epi, int sms, cudaStream_t s) {
    static SmemAttr attr;
    const auto kernel = gemm_kernel<kCG, kKind, kForm, kAmn, kBmn, Epi>;
    const uint32_t stage = stage_size(G.BN, kCG, kBmn, kKind == kMx4);
    const uint32_t turn = Epi::kTurns ? 8 * 2 * kPieceBytes : 0;
    G.stages = (int)((kSmemBudget - kBarBytes - turn) / stage);
    // 4-bit: a sixth stage makes it slower (the prompt of 2048 tokens 59.9 -> 61.3 us)
    const int most_stages = kKind == kMx4 && G.BN == 256 ? 5 : kMaxStages;
    if (G.stages > most_stages) G.stages = most_stages;
    G.nacc = 2;
    if (kKind == kMx4) { // the stages' scales take tensor memory too
        const int per = 8 + 8 * ((G.BN + 127) / 128);
        if (2 * G.BN + G.stages * per > kTmemCols) G.nacc = 1;
    }
    const uint32_t smem = G.smem = G.stages * stage + turn + kBarBytes;
    cudaError_t e = ensure_smem(attr, reinterpret_cast<const void *>(kernel), (int)smem);
    if constexpr (Epi::kTurns)
        if (e == cudaSuccess && G.S == 1) e = epi.maps(G);
    if (e != cudaSuccess) return e;
    // The launch may begin while the kernel before it in the stream ends (grid_wait holds back
    // everything that touches memory): its setup hides behind that kernel's tail.
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int most = sms / kCG, ctas = kCG == 2 ? 2 : G.S;
    cfg.gridDim = dim3(G.S > 1 ? G.tiles * G.S : (G.tiles < most ? G.tiles : most) * kCG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (ctas > 1) {
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = ctas;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, G, epi);
}
template <int kKind, int kForm, bool kAmn, bool kBmn, class Epi>
cudaError_t launch_gemm(GemmArgs &G, const Plan &L, Epi epi, int sms, cudaStream_t s) {
    return L.cg == 2 ? launch_gemm_as<2, kKind, kForm, kAmn, kBmn>(G, epi, sms, s)
                     : launch_gemm_as<1, kKind, kForm, kAmn, kBmn>(G, epi, sms, s);
}

} // namespace dense
} // namespace wm
