// The tensor-core product of the dense operators for few rows (a batch of decoding sequences, a
// short prompt): out[t][n] = sum_k x[t][k] W[n][k] with the weights' rows on the MMA's 128-row side
// and the tokens on its column side.
//
// With few tokens the product is bound by the weights' way from memory, and what one SM can take
// in is bound too (about 100 B/ns): in 128-row tiles of tokens (dense_gemm.cuh) most of a stage
// would be the tokens' rows, loaded again for every tile.  Here a stage is 128 rows of each weight
// matrix and only as many columns as there are tokens, so nearly all of it is weights that are read
// once.  Where there are fewer tiles than SMs a tile is split over k by a cluster (S CTAs, 1 where no more run at
// once or k is short), so that more of the SMs take part.
//
// The sums leave tensor memory transposed (a lane is a weight row) into rows per token, each CTA of a
// cluster adds up its share of them in rank order, and they go through the same epilogues as
// dense_gemm.cuh's.  They meet in L2, in a part of the workspace: an SM reads another's shared memory
// at about 13 B/ns, L2 at 100 (block of 131 tokens, d 7168, f 1536: 27.0 us and 24.8).  One tile per CTA.
//
// A token operand may come in two parts (lo: what rounding it to 16 bits left): their columns stand
// side by side in one MMA and are added with the ranks.  The weights are on the way before the
// kernel waits for the one before it, unless that one may have written them.
#pragma once

#include "dense_gemm.cuh"

namespace wm {
namespace dense {

struct SkinnyArgs {
    CUtensorMap ta[2]; // weights (kPair: both products'; else the two parts of a sum)
    CUtensorMap tb[2]; // tokens (the two parts of a sum)
    CUtensorMap tl[2]; // their low parts
    int T, N, npad, lo;       // tokens, columns of the result, tokens padded to 16, low part too
    int tiles, S, stages, cols;
    int kb, kb_seg;
    uint32_t idesc;
    int early_w;
    const uint8_t *ahead;
    size_t ahead_bytes;
    float *sums; // S > 1: [CTA][token][128], kSkinnyCtas of them at most
};

__host__ __device__ inline uint32_t skinny_stage(int nt) { return (uint32_t)(kBM + nt) * kRowBytes; }

// v += the W floats at p + s * step for each s < S, in that order; from L2 (another SM wrote them).
template <int W> __device__ __forceinline__ void add_parts(const float *p, size_t step, int S, float (&v)[W]) {
    static_assert(W == 8, "two pieces");
    float4 x[8][2];
#pragma unroll
    for (int s = 0; s < 8; ++s)
        if (s < S) {
            x[s][0] = __ldcg(reinterpret_cast<const float4 *>(p + s * step));
            x[s][1] = __ldcg(reinterpret_cast<const float4 *>(p + s * step) + 1);
        }
#pragma unroll
    for (int s = 0; s < 8; ++s)
        if (s < S) {
            v[0] += x[s][0].x, v[1] += x[s][0].y, v[2] += x[s][0].z, v[3] += x[s][0].w;
            v[4] += x[s][1].x, v[5] += x[s][1].y, v[6] += x[s][1].z, v[7] += x[s][1].w;
        }
}

template <int kForm, bool kAmn, class Epi>
__global__ void __launch_bounds__(kThreads, 1) skinny_kernel(const __grid_constant__ SkinnyArgs P,
                                                             const __grid_constant__ Epi epi) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kCols = kForm == kPair ? kBM / 2 : kBM; // columns of the result in a tile
    constexpr int kRow = kBM + 4;                         // floats of a token's row of sums
    const uint32_t smem0 = tc::smem_u32(smem_raw);
    const uint32_t base = (smem0 + kBarBytes + 1023) & ~1023u;
    const uint32_t bar_full = smem0, bar_empty = smem0 + 64, bar_acc = smem0 + 128, drain = smem0 + 136;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + 160);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem_raw + 164);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int S = P.S, nt = P.npad * (1 + P.lo);
    const uint32_t b_at = kBM * kRowBytes, stage_bytes = skinny_stage(nt);
    const int rank = S > 1 ? (int)(blockIdx.x % S) : 0, tile = (int)blockIdx.x / S;
    const int n0 = tile * kCols;
    const int kb0 = (int)((long long)P.kb * rank / S), kb1 = (int)((long long)P.kb * (rank + 1) / S);

    if (warp == 0 && P.early_w) tc::see_complete(); // while the others set up
    if (tid == 32) {
        for (int i = 0; i < P.stages; ++i) {
            tc::mbar_init(bar_full + 8 * i, 1);
            tc::mbar_init(bar_empty + 8 * i, 1);
        }
        tc::mbar_init(bar_acc, 1);
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::mbar_init_fence();
    }
    if (warp == 2) tc::tmem_alloc(tc::smem_u32(tmem_slot), P.cols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    if (warp != 0) tc::grid_wait();

    if (warp == 0) {
        // ---- loader
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        // also announces the bytes of the whole stage
        const auto load_w = [&](int kb, int st) {
            const uint32_t at = base + st * stage_bytes, full = bar_full + 8 * st;
            const bool second = kForm == kSum && kb >= P.kb_seg;
            const int kx = (second ? kb - P.kb_seg : kb) * 64;
            tc::mbar_arrive_expect_tx(full, stage_bytes);
            if (kForm == kPair) { // 64 rows of each
                tc::tma_load(at, &P.ta[0], kx, n0, full);
                tc::tma_load(at + b_at / 2, &P.ta[1], kx, n0, full);
            } else if (kAmn) {
                tc::tma_load(at, &P.ta[second ? 1 : 0], n0, kx, full);
                tc::tma_load(at + 8192, &P.ta[second ? 1 : 0], n0 + 64, kx, full);
            } else {
                tc::tma_load(at, &P.ta[second ? 1 : 0], kx, n0, full);
            }
        };
        const auto load_t = [&](int kb, int st) {
            const uint32_t at = base + st * stage_bytes + b_at, full = bar_full + 8 * st;
            const bool second = kForm == kSum && kb >= P.kb_seg;
            const int kx = (second ? kb - P.kb_seg : kb) * 64;
            tc::tma_load(at, &P.tb[second ? 1 : 0], kx, 0, full);
            if (P.lo) tc::tma_load(at + P.npad * kRowBytes, &P.tl[second ? 1 : 0], kx, 0, full);
        };
        const int early = P.early_w ? min(P.stages, kb1 - kb0) : 0;
        if (tc::elect_one())
            for (int i = 0; i < early; ++i) load_w(kb0 + i, i);
        __syncwarp();
        tc::grid_wait_release();
        for (int kb = kb0; kb < kb1; ++kb) {
            if (issued >= early && !all(tc::mbar_wait(bar_empty + 8 * st, ph ^ 1))) {
                ok = false;
                break;
            }
            if (tc::elect_one()) {
                if (issued >= early) load_w(kb, st);
                load_t(kb, st);
            }
            __syncwarp();
            ++issued;
            if (++st == P.stages) {
                st = 0;
                ph ^= 1;
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
        if (!ok) { // copies in flight land before the CTA goes
            if (lane == 0) *abort_flag = 1;
            const int n = min(max(issued, early), P.stages);
            for (int i = 0; i < n; ++i) {
                const int j = max(issued, early) - n + i;
                tc::mbar_wait(bar_full + 8 * (j % P.stages), (j / P.stages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        const uint64_t desc0 = tc::desc_sw128(base, 8192);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!all(tc::mbar_wait(bar_full + 8 * st, ph))) {
                ok = false;
                break;
            }
            tc::fence_after_sync();
            const uint64_t da = desc0 + (uint64_t)((st * stage_bytes) >> 4), db = da + (uint64_t)(b_at >> 4);
            if (tc::elect_one()) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc::mma_f16(tmem, da + (uint64_t)(j * ((kAmn ? 2048 : 32) >> 4)), db + (uint64_t)(2 * j), P.idesc,
                                j > 0 || kb > kb0);
                tc::mma_commit(bar_empty + 8 * st);
                if (kb + 1 == kb1) tc::mma_commit(bar_acc);
            }
            __syncwarp();
            if (++st == P.stages) {
                st = 0;
                ph ^= 1;
            }
        }
        if (!ok) {
            if (lane == 0) *abort_flag = 1;
            if (tc::elect_one()) tc::mma_commit(drain);
            tc::mbar_wait(drain, 0);
        }
        __syncwarp();
    } else if (warp >= 3) {
        // ---- sums to shared memory, a row of 128 per token (padded by 16 bytes); two warps for
        // each quarter of the lanes, 16 tokens at a time in turn
        const int q = warp & 3, half = (warp - 3) >> 2;
        bool ok = true;
        if (lane == 0) ok = wait_tile(bar_acc, 0, kb1 - kb0);
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
            *abort_flag = 1;
        } else {
            tc::fence_after_sync();
            const uint32_t src = tmem + ((uint32_t)(32 * q) << 16);
            float *part = reinterpret_cast<float *>(smem_raw + (base - smem0)) + 32 * q + lane;
            float *out = P.sums + (size_t)blockIdx.x * nt * kBM + 32 * q + lane;
            for (int c = 16 * half; c < nt; c += 32) {
                uint32_t v[16];
                tc::tmem_ld16n(src + c, v);
                tc::tmem_wait_ld(v);
                if (S == 1) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c + j) * kRow] = __uint_as_float(v[j]);
                } else {
                    const int left = P.T - (c < P.npad ? c : c - P.npad); // tokens from here on
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < left) __stcg(out + (size_t)(c + j) * kBM, __uint_as_float(v[j]));
                }
            }
            tc::fence_before_sync();
        }
    }
    __syncthreads();
    if (S > 1) tc::cluster_sync();
    {
        constexpr int W = Epi::kWidth, kPerRow = kCols / W;
        const int items = P.T * kPerRow;
        const int i1 = (int)((long long)items * (rank + 1) / S);
        for (int i = (int)((long long)items * rank / S) + tid; i < i1; i += kThreads) {
            const int t = i / kPerRow, c = (i % kPerRow) * W;
            if (n0 + c >= P.N) continue;
            float v[W], w[W];
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] = w[j] = 0.f;
            const int row = S > 1 ? kBM : kRow;
            const float *src = S > 1 ? P.sums + (size_t)tile * S * nt * kBM : reinterpret_cast<float *>(smem_raw + (base - smem0));
            src += (size_t)t * row + c;
            const auto add = [&](const float *p, float(&x)[W]) {
                if (S > 1) {
                    add_parts<W>(p, (size_t)nt * kBM, S, x);
                } else {
#pragma unroll
                    for (int j = 0; j < W; ++j) x[j] += p[j];
                }
            };
            add(src, v);
            if (kForm == kPair) add(src + kCols, w);
            if (kForm != kPair && P.lo) {
                add(src + P.npad * row, w);
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] += w[j];
            }
            epi.template row<W>(0, t, n0 + c, v, w);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (tid == 0 && *abort_flag) atomicOr(&g_dense_timeout, 1u);
    if (warp == 2) tc::tmem_dealloc(tmem, P.cols);
}

// How many CTAs split a tile's k -- as many as shorten it and still run at once -- and the estimated
// time in ns, on the scale of plan().  The sums' exchange grows with the tokens.
struct SkinnyPlan {
    int S;
    double ns;
};
inline SkinnyPlan skinny_plan(int T, int N, int kb, bool pair, int nt, int sms) {
    const int cols = pair ? kBM / 2 : kBM, tiles = (N + cols - 1) / cols;
    SkinnyPlan best{1, 1e30};
    for (int S = 1; S <= 8 && S <= kb; ++S) {
        if (S > 1 && (tiles > clusters_at_once(S) || tiles * S > kSkinnyCtas)) continue;
        const int waves = S > 1 ? 1 : (tiles + sms - 1) / sms;
        const double t = 3000.0 + (double)waves * ((kb + S - 1) / S) * skinny_stage(nt) / 100.0 +
                         (S > 1 ? 500.0 + T * (kBM * 4 / 40.0) : 0.0);
        if (t < best.ns) best = SkinnyPlan{S, t};
    }
    return best;
}
// Whether a product of T tokens takes this kernel rather than 128-row tiles of tokens.  Measured here and
// there, forward, bf16, weights from memory, both products, us: d 7168, f 1536, 3 tokens 20.6 and 27.5, 64
// 22.7 and 25.2, 131 24.8 and 29.7, 192 26.4 and 29.5, 256 30.1 and 30.1; d 4096, f 1024, 64 13.7 and 16.4,
// 131 16.4 and 19.5, 192 18.1 and 19.3, 256 20.7 and 19.8; d 2048, f 768, 131 12.4 and 13.3, 256 14.4 and
// 13.1.  The two estimates' difference is not trusted for the fewest.
static_assert(kSplitTokens <= 48, "a in two parts is read by this kernel alone");
inline bool skinny_wins(int T, int N, int kb, bool pair, int sms) {
    if (T > kSkinnyTokens) return false;
    return T <= 48 || skinny_plan(T, N, kb, pair, pad_tokens(T), sms).ns < plan(&T, &N, 1, kb, pair, false, sms).ns;
}

// G: maps, T, N, lo, kb, kb_seg, early_w set; the rest is filled in here.
template <int kForm, bool kAmn, class Epi>
cudaError_t launch_skinny(SkinnyArgs &G, bool bf16, const Epi &epi, int sms, cudaStream_t s) {
    static SmemAttr attr;
    const auto kernel = skinny_kernel<kForm, kAmn, Epi>;
    constexpr int kCols = kForm == kPair ? kBM / 2 : kBM;
    const int nt = G.npad * (1 + G.lo);
    const uint32_t stage = skinny_stage(nt);
    G.tiles = (G.N + kCols - 1) / kCols;
    G.S = skinny_plan(G.T, G.N, G.kb, kForm == kPair, nt, sms).S;
    G.idesc = tc::idesc_half(kBM, nt, bf16, kAmn, false);
    // what one CTA will use, at least the room of its sums if they stay there
    const uint32_t most = (kSmemBudget - kBarBytes - 1024) / stage, need = (uint32_t)(G.kb + G.S - 1) / G.S;
    const uint32_t sums = (uint32_t)nt * (kBM + 4) * 4;
    G.stages = (int)(need < most ? need : most);
    if (G.stages > kMaxStages) G.stages = kMaxStages;
    if (G.stages < 1) return cudaErrorInvalidValue;
    uint32_t ring = G.stages * stage;
    if (G.S == 1 && ring < sums) ring = sums;
    G.cols = 32;
    while (G.cols < nt) G.cols *= 2;
    const uint32_t smem = kBarBytes + 1024 + ring;
    if (G.cols > kTmemCols || smem > kSmemBudget) return cudaErrorInvalidValue;
    cudaError_t e = ensure_smem(attr, reinterpret_cast<const void *>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = G.S;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(G.tiles * G.S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = G.S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, G, epi);
}

} // namespace dense
} // namespace wm
