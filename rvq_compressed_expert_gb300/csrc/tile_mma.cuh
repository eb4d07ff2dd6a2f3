// The tensor-core product of the training operators: tiles of D = A B^T in fp32 on tcgen05.mma, where a job says
// which tiles there are, where a tile's operands lie and what becomes of its sums.  Built from dense_gemm.cuh's parts.
//
// A persistent grid, one CTA per SM: one warp moves 128-byte-wide pieces of A and B (64 16-bit values of k) into a
// ring of shared-memory stages by TMA, one issues the MMAs on full stages into one of two TMEM accumulators, eight
// take the other one out through the job's epilogue.  Operands are three-dimensional maps (matrix, row, column), so
// that a matrix of a stack ends where it ends; parts past its ends arrive as zeros.
//
// A job J (a kernel argument, with its tensor maps ta and tb) has
//   kAmn, kBmn   operands that lie with m (or n) contiguous (MN-major) rather than k
//   kReads       an epilogue that reads
//   kTwoPieces   an epilogue that reads nothing and has registers for two pieces of 32 columns at once
//   kRagged      tiles of their own heights and widths: A also comes in boxes of 32 rows (ta_low), B (K-major) in boxes
//                of 64 and 16 (tb, tb_low)
//   kMask        tiles whose k ends inside a piece that holds other values: those are cleared in shared memory
//   begin(smem)  by all threads, once what the kernel before wrote is visible; smem: P.job_bytes of its own
//   tiles(smem), spot(smem, t): how many, and which
//   ahead(spot, r, half, BN): row r of a later tile will be read besides: may be asked of L2 (two lanes a row)
//   fetch(out, spot, n, held), turn(out, shared, held, in), tile(out, spot, n, v, in): the sums v of 32 rows and 32 columns
//                from n on (lane = row, all lanes together), with what the epilogue reads besides: asked for ahead of
//                the sums (held), then brought to the lanes' rows (in)
// What bounds it: a pair's 256 x 256 tile brings 32 KB a piece of k into each SM for 512 cycles of MMAs, about what an SM
// takes in (100 B/ns), so an epilogue that reads costs nearly its share of bytes; long runs are at the power limit.
// Waits are bounded, as dense_gemm.cuh's.
#pragma once

#include "dense_gemm.cuh"
#include "train.cuh"

namespace wm {
namespace train {

using dense::all;
using dense::kBM;
using dense::kMaxStages;
using dense::kPieceBytes;
using dense::kRowBytes;
using dense::kSmemBudget;
using dense::kTmemCols;
using dense::Out32;
constexpr int kTileThreads = dense::kThreads;
constexpr uint32_t kTileBars = 320; // bytes of barriers

struct Spot {
    int am, az, bm, bz; // A's and B's first row (m, n) and matrix
    int ak, bk;         // their first k
    int pieces, left;   // pieces of k; how many k of the last one count (kMask)
    int m, n, rows;     // place in the result: first row (of all matrices'), first column, rows that are the tile's
    int z;              // matrix of the result
    // kRagged: columns of the tile (a multiple of 16 a CTA), and the rows of A that each CTA loads (of 32, MN-major 64)
    int cols = 0, high = 0;
};
struct TileArgs {
    int BN, stages;
    uint32_t idesc, smem, job_bytes;
};

// One box of one matrix of a stack; the second form from either CTA of a pair, its bytes counting on an mbarrier of
// either (a shared::cluster address).
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t mbar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
                 "[%2];" ::"r"(dst),
                 "l"(m), "r"(mbar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_load3_pair(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t mbar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(m), "r"(mbar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// 32 rows x 32 columns of a matrix of 2 or 4 byte values, on their way: consecutive lanes hold consecutive 16 bytes of a
// row (rows of whole 16-byte pieces; zeros past the ends), to be turned round in shared memory.
template <int kBytes> struct Block {
    static constexpr int kPieces = 2 * kBytes, kPer = 16 / kBytes;
    uint4 q[kPieces];
    __device__ __forceinline__ void fetch(const Out32 &o, const void *src, size_t ld, int n, int N) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int at = 32 * i + o.lane, row = at / kPieces, c = n + kPer * (at % kPieces);
            const uint8_t *p = static_cast<const uint8_t *>(src) + ((size_t)(o.m + row) * ld + c) * kBytes;
            q[i] = row < o.rows && c < N ? *reinterpret_cast<const uint4 *>(p) : uint4{};
        }
    }
    // this lane's row: its 16-byte pieces, in order.  t: the warp's own kPieceBytes (not those that copies leave from,
    // which would have to have left)
    __device__ __forceinline__ void turn(const Out32 &o, uint4 *t, uint4 (&out)[kPieces]) const {
#pragma unroll
        for (int h = 0; h < kPieces; h += 4) { // four pieces a row at a time
            __syncwarp();
            if constexpr (kPieces == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 32 * i + o.lane;
                    t[dense::turned(at / 4, at % 4, 4)] = q[i];
                }
            } else {
                // pieces h .. h + 3 of each row: of 8 lanes those 4 that hold them
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 32 * i + o.lane;
                    if (at % 8 / 4 == h / 4) t[dense::turned(at / 8, at % 4, 4)] = q[i];
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) out[h + i] = t[dense::turned(o.lane, i, 4)];
        }
    }
};
__device__ __forceinline__ void halves(const uint4 (&q)[4], bool bf16, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) dense::widen8(bf16, q[i], *reinterpret_cast<float(*)[8]>(&v[8 * i]));
}

// Ask L2 for `bytes` bytes from p on.
__device__ __forceinline__ void ask_l2(const void *p, int bytes) {
    for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p) + i));
}

struct Nothing {};

// The copy out for a stack of matrices, a box of 32 rows and 64 bytes ending where its matrix ends: a tile's last
// rows go the same way as all others (lane by lane they take longer than the rest of the tile: 63 matrices of 240 x 5376
// zeros 65 us, 256 rows 37).
__device__ __forceinline__ void tma_store3(const CUtensorMap *m, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m), "r"(src),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// A map for it: rows of cols values (whole 16-byte pieces).
cudaError_t store_map3(CUtensorMap *m, void *p, int dtype, int mats, int rows, int cols);
template <class O>
__device__ __forceinline__ void send3(Out32 &o, const CUtensorMap *map, int n, int N, int row, int z, const float *v) {
    constexpr int kPer = 16 / (int)sizeof(O);
    uint4 *turn = o.next();
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[dense::turned(o.lane, i, 4)] = dense::piece_of(v + kPer * i, O());
    tc::fence_proxy_async();
    __syncwarp();
    if (o.lane == 0 && n < N) tma_store3(map, n, row, z, tc::smem_u32(turn));
}
// 32 columns from n on of up to 32 rows from `row` on, lane = row.
__device__ __forceinline__ void put3_as(int dtype, Out32 &o, const CUtensorMap *map, int n, int N, int row, int z, const float (&v)[32]) {
    if (dtype == WASTE_ACT_BF16) {
        send3<__nv_bfloat16>(o, map, n, N, row, z, v);
    } else if (dtype == WASTE_ACT_F16) {
        send3<__half>(o, map, n, N, row, z, v);
    } else {
        send3<float>(o, map, n, N, row, z, v);
        send3<float>(o, map, n + 16, N, row, z, v + 16);
    }
}

// A result in memory: written, or (kAdd) added to what is there.
template <bool kAdd> struct Out {
    CUtensorMap map;
    void *p;
    int M, N, dtype, vec; // M x N: a matrix; vec: rows of whole 16-byte pieces, for copies and blocks
    cudaError_t set(void *out, int mats, int rows, int cols, int type) {
        p = out, M = rows, N = cols, dtype = type;
        vec = (size_t)cols * dense::type_size(type) % 16 == 0;
        return vec ? store_map3(&map, out, type, mats, rows, cols) : cudaSuccess;
    }
    // what is there, to be added to
    struct Held {
        Block<4> wide;
    };
    using In = std::conditional_t<kAdd, float[32], Nothing>;
    // half a row of BN columns from n on
    __device__ __forceinline__ void ahead(size_t m, int n, int half, int BN) const {
        const int size = dtype == WASTE_ACT_F32 ? 4 : 2, c = n + half * (BN / 2), cols = min(BN / 2, N - c);
        if (cols > 0) ask_l2(static_cast<const char *>(p) + (m * N + c) * size, cols * size);
    }
    __device__ __forceinline__ void fetch(const Out32 &o, int n, Held &h) const {
        if (!vec) return;
        if (dtype == WASTE_ACT_F32)
            h.wide.fetch(o, p, N, n, N);
        else
            reinterpret_cast<Block<2> &>(h.wide).fetch(o, p, N, n, N);
    }
    __device__ __forceinline__ void turn(const Out32 &o, uint4 *t, const Held &h, float (&base)[32]) const {
        if (!vec) return;
        if (dtype == WASTE_ACT_F32) {
            h.wide.turn(o, t, reinterpret_cast<uint4(&)[8]>(base));
        } else {
            uint4 q[4];
            reinterpret_cast<const Block<2> &>(h.wide).turn(o, t, q);
            halves(q, dtype == WASTE_ACT_BF16, base);
        }
    }
    __device__ __forceinline__ void put(Out32 &o, const Spot &T, int n, const float (&v)[32], const In &base) const {
        const int row = o.m - T.z * M; // of its matrix
        if (!vec) {
            dense::put32_as(dtype, o, nullptr, p, N, n, N, N % 4 == 0, kAdd, v);
        } else if constexpr (kAdd) {
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = base[i] + v[i];
            put3_as(dtype, o, &map, n, N, row, T.z, x);
        } else {
            put3_as(dtype, o, &map, n, N, row, T.z, v);
        }
    }
};

// Bytes of a stage in one CTA of cg.
inline uint32_t tile_stage(int BN, int cg, bool b_mn) { return dense::stage_size(BN, cg, b_mn, false); }

// tc::mbar_wait for an arrival from the pair's other CTA, which is to be seen to have written its shared memory.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
    for (int it = 0; it < tc::kWaitPolls; ++it) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (ok) return true;
        if (it > 64) __nanosleep(128);
    }
    return false;
}

// Zeros in rows first .. end - 1 of a stage's slabs (64 rows of 128 bytes each, a row one k), by one warp, seen by MMAs
// behind it: others' values, a NaN among them maybe, must not meet zeros of the other operand.
__device__ __forceinline__ void mask_rows(uint8_t *stage, int first, int end, int slabs, int lane) {
    const int n = (end - first) * 8;
    for (int i = lane; i < n * slabs; i += 32) {
        const int s = i / n, j = i - s * n;
        *reinterpret_cast<uint4 *>(stage + s * 8192 + first * 128 + j * 16) = uint4{};
    }
    tc::fence_proxy_async();
    __syncwarp();
}

// Shared memory of the eight epilogue warps: two pieces each on their way out, one on its way in.
template <class J> constexpr uint32_t kTurnBytes = 8 * (J::kReads ? 3 : 2) * kPieceBytes;

template <int kCG, class J>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(const __grid_constant__ TileArgs P, const __grid_constant__ J job) {
    extern __shared__ __align__(1024) uint8_t smem_raw[]; // stages, pieces on their way out, the job's, barriers
    const uint32_t base = tc::smem_u32(smem_raw);
    const uint32_t bars_at = P.smem - kTileBars;
    const uint32_t bars = base + bars_at;
    const uint32_t bar_full = bars, bar_empty = bars + 64, bar_accf = bars + 128, bar_acce = bars + 144;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + bars_at + 160);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem_raw + bars_at + 164);
    const uint32_t drain = bars + 168, bar_mask = bars + 176, bar_land = bars + 240;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int BN = P.BN;
    constexpr uint32_t a_bytes = kBM * kRowBytes;
    const uint32_t b_bytes = dense::stage_b_bytes(BN, kCG, J::kBmn);
    const uint32_t stage_bytes = dense::stage_size(BN, kCG, J::kBmn, false);
    const int rank = kCG == 2 ? (int)(blockIdx.x & 1) : 0;
    const bool leads = kCG == 1 || rank == 0;
    uint8_t *turns = smem_raw + P.stages * stage_bytes, *mine = turns + kTurnBytes<J>;

    if (tid == 32) {
        for (int i = 0; i < P.stages; ++i) {
            tc::mbar_init(bar_full + 8 * i, 1);
            tc::mbar_init(bar_empty + 8 * i, 1);
            tc::mbar_init(bar_mask + 8 * i, kCG); // one a stage: who clears may be further along than the issuer
            tc::mbar_init(bar_land + 8 * i, 1);
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
    tc::grid_wait_release();
    job.begin(mine);
    tc::fence_before_sync();
    __syncthreads();
    if (kCG == 2) tc::cluster_sync(); // the other CTA's barriers are up
    tc::fence_after_sync();
    constexpr uint32_t tmem = 0; // all columns are this CTA's, so they start at the first
    if (*tmem_slot != tmem && tid == 0) *abort_flag = 1;

    const int tiles = job.tiles(mine), tile0 = (int)blockIdx.x / kCG, step = (int)gridDim.x / kCG;

    if (warp == 0) {
        // ---- loader (the warp walks the loop, an elected lane issues)
        int st = 0, issued = 0;
        uint32_t ph = 0, land = 0, there = 0; // a bit a stage: uses of bar_land so far, whether the last load was one
        bool ok = true;
        const uint32_t full0 = kCG == 2 ? tc::map_rank(bar_full, 0) : bar_full;
        for (int t = tile0; t < tiles && ok; t += step) {
            const Spot T = job.spot(mine, t);
            const int am = T.am + rank * kBM, bm = T.bm + (kCG == 2 ? rank * ((J::kRagged ? T.cols : BN) / 2) : 0);
            for (int kb = 0; kb < T.pieces; ++kb) {
                if (!all(tc::mbar_wait(bar_empty + 8 * st, ph ^ 1))) {
                    ok = false;
                    break;
                }
                if (tc::elect_one()) {
                    const uint32_t sa = base + st * stage_bytes, sb = sa + a_bytes;
                    // a piece to be masked counts on a barrier of its own in each CTA, for the warp that clears
                    const bool own = J::kMask && kb + 1 == T.pieces && T.left < 64;
                    const uint32_t full = own ? bar_land + 8 * st : full0 + 8 * st;
                    const uint32_t bytes = J::kRagged ? (uint32_t)(T.high + T.cols / kCG) * kRowBytes : a_bytes + b_bytes;
                    if (own) {
                        tc::mbar_arrive_expect_tx(bar_land + 8 * st, bytes);
                        if (leads) tc::mbar_arrive(bar_full + 8 * st);
                    } else if (leads) {
                        tc::mbar_arrive_expect_tx(bar_full + 8 * st, kCG * bytes);
                    }
                    const auto load = [&](uint32_t dst, const CUtensorMap *m, int x, int y, int z) {
                        if (kCG == 2 && !(J::kMask && own))
                            tma_load3_pair(dst, m, x, y, z, full);
                        else
                            tma_load3(dst, m, x, y, z, full);
                    };
                    const int ka = T.ak + kb * 64, kk = T.bk + kb * 64;
                    if (J::kAmn) {
                        for (int i = 0; i < (J::kRagged ? T.high : kBM) / 64; ++i) load(sa + i * 8192, &job.ta, am + 64 * i, ka, T.az);
                    } else if (J::kRagged && T.high < kBM) {
                        if constexpr (J::kRagged)
                            for (int i = 0; i < T.high; i += 32) load(sa + i * kRowBytes, &job.ta_low, ka, am + i, T.az);
                    } else {
                        load(sa, &job.ta, ka, am, T.az);
                    }
                    if (J::kBmn) {
                        for (uint32_t i = 0; i * 8192 < b_bytes; ++i) load(sb + i * 8192, &job.tb, bm + 64 * i, kk, T.bz);
                    } else if constexpr (J::kRagged) {
                        const int n = T.cols / kCG;
                        int i = 0;
                        for (; i + 64 <= n; i += 64) load(sb + i * kRowBytes, &job.tb, kk, bm + i, T.bz);
                        for (; i < n; i += 16) load(sb + i * kRowBytes, &job.tb_low, kk, bm + i, T.bz);
                    } else {
                        load(sb, &job.tb, kk, bm, T.bz);
                    }
                }
                __syncwarp();
                if (J::kMask) {
                    const uint32_t own = kb + 1 == T.pieces && T.left < 64;
                    land ^= own << st;
                    there = (there & ~(1u << st)) | own << st;
                }
                ++issued;
                if (++st == P.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok) { // copies in flight land before the CTA goes
            if (lane == 0) *abort_flag = 1;
            const int n = min(issued, P.stages);
            for (int i = 0; i < n && leads; ++i) {
                const int j = issued - n + i;
                tc::mbar_wait(bar_full + 8 * (j % P.stages), (j / P.stages) & 1);
            }
            for (int i = 0; J::kMask && i < P.stages; ++i)
                if (there >> i & 1) tc::mbar_wait(bar_land + 8 * i, (land >> i & 1) ^ 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leads) {
            // ---- MMA issuer
            const auto commit = [](uint32_t bar) {
                if (kCG == 2)
                    tc::mma_commit_pair(bar);
                else
                    tc::mma_commit(bar);
            };
            int st = 0, it = 0;
            uint32_t ph = 0, masked = 0;
            bool ok = true;
            static_assert(!J::kMask || (J::kAmn && J::kBmn), "a row of a stage is one k");
            const uint64_t desc0 = tc::desc_sw128(base, 8192);
            for (int t = tile0; t < tiles && ok; t += step) {
                const Spot T = job.spot(mine, t);
                if (T.pieces == 0) continue;
                const int buf = it & 1, use = it >> 1;
                ++it;
                if (!all(tc::mbar_wait(bar_acce + 8 * buf, (use & 1) ^ 1))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t d = tmem + buf * 256;
                const uint32_t idesc = J::kRagged ? (P.idesc & ~(63u << 17)) | (uint32_t)(T.cols >> 3) << 17 : P.idesc;
                for (int kb = 0; kb < T.pieces; ++kb) {
                    if (!all(tc::mbar_wait(bar_full + 8 * st, ph))) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint64_t da = desc0 + (uint64_t)((st * stage_bytes) >> 4), db = da + (uint64_t)(a_bytes >> 4);
                    int steps = 4;
                    if (J::kMask && kb + 1 == T.pieces && T.left < 64) {
                        steps = (T.left + 15) >> 4;
                        // cleared, in both CTAs: these are a piece behind at most, the pieces before have come from both
                        if (!all(wait_cluster(bar_mask + 8 * st, masked >> st & 1))) {
                            ok = false;
                            break;
                        }
                        masked ^= 1u << st;
                        tc::fence_after_sync();
                    }
                    if (tc::elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (J::kMask && j >= steps) break;
                            const uint64_t dj = da + (uint64_t)(j * ((J::kAmn ? 2048 : 32) >> 4));
                            const uint64_t ej = db + (uint64_t)(j * ((J::kBmn ? 2048 : 32) >> 4));
                            if (kCG == 2)
                                tc::mma_f16_pair(d, dj, ej, idesc, j > 0 || kb > 0);
                            else
                                tc::mma_f16(d, dj, ej, idesc, j > 0 || kb > 0);
                        }
                        commit(bar_empty + 8 * st);
                        if (kb + 1 == T.pieces) commit(bar_accf + 8 * buf);
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
    } else if (warp == 2) {
        if (J::kMask) {
            // ---- clears what is not the tile's in this CTA's part of a stage as soon as it is there, often ahead of the MMAs
            // before it, and says so to the issuer
            int st = 0, pieces = 0; // since the last wait: it takes as long as all of them
            uint32_t used = 0;      // a bit a stage: the parity of the barrier that it lands on
            for (int t = tile0; t < tiles; t += step) {
                const Spot T = job.spot(mine, t);
                if (T.pieces == 0) continue;
                const int last = (st + T.pieces - 1) % P.stages;
                st = (st + T.pieces) % P.stages;
                pieces += T.pieces;
                if (T.left == 64) continue;
                if (!all(dense::wait_tile(bar_land + 8 * last, used >> last & 1, pieces))) {
                    if (lane == 0) *abort_flag = 1;
                    break;
                }
                pieces = 0;
                used ^= 1u << last;
                mask_rows(smem_raw + last * stage_bytes, T.left, (T.left + 15) & ~15, (int)((a_bytes + b_bytes) >> 13), lane);
                if (lane == 0) {
                    if (leads)
                        tc::mbar_arrive(bar_mask + 8 * last);
                    else
                        tc::mbar_arrive_cluster(tc::map_rank(bar_mask + 8 * last, 0));
                }
            }
        }
        __syncwarp();
    } else if (warp >= 3) {
        // ---- epilogue: two warps for each quarter of the lanes (rows); they take its pieces of 32 columns in turn
        const int q = warp & 3, half = (warp - 3) >> 2;
        Out32 out{reinterpret_cast<uint4 *>(turns) + (warp - 3) * (2 * kPieceBytes / 16), 0, 0, lane, 0};
        uint4 *turned = reinterpret_cast<uint4 *>(turns + 8 * 2 * kPieceBytes) + (warp - 3) * (kPieceBytes / 16);
        int it = 0;
        for (int t = tile0; t < tiles; t += step) {
            Spot T = job.spot(mine, t);
            T.m += rank * kBM;
            T.rows -= rank * kBM;
            const bool any = 32 * q < T.rows, empty = T.pieces == 0;
            out.m = T.m + 32 * q;
            out.rows = T.rows - 32 * q;
            const int buf = it & 1, use = it >> 1;
            if constexpr (J::kReads)
                if (t + step < tiles) job.ahead(job.spot(mine, t + step), 32 * q + rank * kBM + lane, half, BN);
            const uint32_t src = tmem + buf * 256 + ((uint32_t)(32 * q) << 16);
            const int width = J::kRagged ? T.cols : BN;
            const auto ready = [&] { // the tile's sums
                if (empty) return true;
                ++it;
                bool ok = true;
                if (lane == 0) ok = dense::wait_tile(bar_accf + 8 * buf, use & 1, T.pieces);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) *abort_flag = 1;
                tc::fence_after_sync();
                return ok;
            };
            const auto free_acc = [&] {
                if (empty) return;
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (leads)
                        tc::mbar_arrive(bar_acce + 8 * buf);
                    else
                        tc::mbar_arrive_cluster(tc::map_rank(bar_acce + 8 * buf, 0));
                }
            };
            if constexpr (J::kTwoPieces) {
                // nothing but the sums: two pieces to registers at once, so that the next tile's MMAs may follow while
                // the last two are on their way out
                if (!ready()) break;
                alignas(16) uint32_t v[32], w[32];
                const auto take = [&](int c) {
                    if (any && !empty) {
                        if (c < width) tc::tmem_ld32(src + c, v);
                        if (c + 64 < width) tc::tmem_ld32(src + c + 64, w);
                        if (c < width) tc::tmem_wait_ld(v);
                        if (c + 64 < width) tc::tmem_wait_ld(w);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = w[k] = 0;
                    }
                };
                const auto give = [&](int c) {
                    if (any && c < width) job.tile(out, T, T.n + c, reinterpret_cast<const float(&)[32]>(v), {});
                    if (any && c + 64 < width) job.tile(out, T, T.n + c + 64, reinterpret_cast<const float(&)[32]>(w), {});
                };
                take(32 * half);
                if (width <= 128) {
                    free_acc();
                    give(32 * half);
                } else {
                    give(32 * half);
                    take(128 + 32 * half);
                    free_acc();
                    give(128 + 32 * half);
                }
            } else {
                typename J::Held held;
                if (any) job.fetch(out, T, T.n + 32 * half, held);
                if (!ready()) break;
                for (int c = 32 * half; any && c < BN; c += 64) { // BN is a multiple of 32
                    alignas(16) uint32_t v[32];
                    if (empty) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0;
                    } else {
                        tc::tmem_ld32(src + c, v);
                        tc::tmem_wait_ld(v);
                    }
                    typename J::In in;
                    job.turn(out, turned, held, in);
                    if (c + 64 < BN) job.fetch(out, T, T.n + c + 64, held);
                    job.tile(out, T, T.n + c, reinterpret_cast<const float(&)[32]>(v), in);
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
    tc::fence_before_sync();
    __syncthreads();
    if (kCG == 2) tc::cluster_sync(); // no CTA leaves while its memory takes part in the other's MMAs or barriers
    tc::fence_after_sync();
    if (tid == 0 && *abort_flag) atomicOr(&dense::g_dense_timeout, 1u);
    if (warp == 2) {
        if (kCG == 2)
            tc::tmem_dealloc_pair(tmem, kTmemCols);
        else
            tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// A map over `mats` matrices of rows x cols 16-bit values, ld values from row to row and `step` from matrix to
// matrix: boxes of box_rows rows x 64 values of one of them, 128-byte swizzle, zeros past its ends.
cudaError_t stack_map(CUtensorMap *m, const void *p, int cols, int rows, int mats, size_t ld, size_t step, int box_rows);

// Fills in the rest of P (BN set) and launches: at most `tiles` tiles (an upper bound).
template <int kCG, class J>
cudaError_t launch_tiles_as(TileArgs &P, const J &job, bool bf16, size_t job_bytes, long long tiles, int sms, cudaStream_t s) {
    static SmemAttr attr;
    const auto kernel = tile_kernel<kCG, J>;
    const uint32_t stage = tile_stage(P.BN, kCG, J::kBmn), turn = kTurnBytes<J>;
    P.job_bytes = (uint32_t)round_up(job_bytes, 16);
    P.stages = (int)((kSmemBudget - kTileBars - turn - P.job_bytes) / stage);
    if (P.stages > kMaxStages) P.stages = kMaxStages;
    if (P.stages < 2) return cudaErrorInvalidValue;
    P.smem = P.stages * stage + turn + P.job_bytes + kTileBars;
    P.idesc = tc::idesc_half(kBM * kCG, P.BN, bf16, J::kAmn, J::kBmn);
    cudaError_t e = ensure_smem(attr, reinterpret_cast<const void *>(kernel), (int)P.smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kCG;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    const int most = sms / kCG;
    cfg.gridDim = dim3((tiles < most ? (int)tiles : most) * kCG);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = P.smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = kCG == 2 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P, job);
}

} // namespace train
} // namespace wm
