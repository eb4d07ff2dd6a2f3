// The gated feed-forward block on 16-bit weights, forward and backward, as tensor-core products
// (dense_gemm.cuh).
//
// forward   1. (x Wg^T, x Wu^T) in one launch, both products of a tile side by side, a = silu(g) u
//              (and g, u if kept) in the epilogue;  2. y = a Wd^T.
// backward  1. da = dy Wd, a / dg / du in the epilogue from the kept g and u;
//           2. dx = dg Wg + du Wu, one sum over both products;
//           3. dWg = dg^T x, dWu = du^T x, dWd = dy^T a, three products of T terms in one launch.  It waits
//              for 2 as well, though it needs 1 alone: what a launch of the call made is read behind a wait of
//              the reader's own (running beside 2 on the strength of 2's wait: 19.1 us instead of 19.8 for
//              333 tokens, d 1032, f 264, 48.2 instead of 49.0 for one token, d 7168, f 1536).
// Where a product runs over a matrix's rows (Wd, Wg, Wu in 1 and 2, everything in 3) the tiles go
// to the tensor core MN-major, as they lie in memory: nothing is transposed.
#include "dense_skinny.cuh"

namespace wm {
namespace dense {

namespace {

int pieces(int k) { return (k + 63) / 64; }

cudaError_t half_map(CUtensorMap *m, const void *p, int rows, int cols, int box_rows) {
    return make_map(m, p, 2, rows, (size_t)cols * 2, box_rows);
}

// a in two 16-bit parts: its rounding and what that left, one above the other.
struct GatedSplit {
    static constexpr int kWidth = 8;
    void *hi, *lo, *g, *u;
    int f, dtype;
    template <int W>
    __device__ __forceinline__ void row(int, int m, int n, const float (&cg)[W], const float (&cu)[W]) const {
        const size_t at = (size_t)m * f + n;
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = cg[i] * sigmoid(cg[i]) * cu[i];
        put_as(dtype, hi, at, n, f, true, false, v);
        if (lo) put_rest(dtype, lo, at, n, f, v);
        if (g) {
            put_as(dtype, g, at, n, f, true, false, cg);
            put_as(dtype, u, at, n, f, true, false, cu);
        }
    }
};

SkinnyArgs skinny(int T, int N, int K, float *sums) {
    SkinnyArgs G = {};
    G.T = T;
    G.N = N;
    G.npad = pad_tokens(T);
    G.kb = G.kb_seg = pieces(K);
    G.sums = sums;
    return G;
}

} // namespace

cudaError_t launch_ffn_forward(const FfnFwd &P, cudaStream_t s) {
    if (P.T <= kGemvTokens) return launch_ffn_gemv(P, s);
    const int sms = device_sm_count();
    const bool bf16 = P.dtype == WASTE_ACT_BF16, split = P.T <= kSplitTokens;
    void *lo = split ? static_cast<uint16_t *>(P.a) + (size_t)P.T * P.f : nullptr;
    cudaError_t e;
    // few tiles: bound by the weights' way from memory, which the next kernel's can follow at once
    // while this one adds up and ends
    const size_t wd = (size_t)P.d * P.f * 2, ahead = wd <= kAheadMost ? wd : 0;
    if (skinny_wins(P.T, P.f, pieces(P.d), true, sms)) {
        SkinnyArgs G = skinny(P.T, P.f, P.d, P.sums);
        if ((e = half_map(&G.ta[0], P.wg, P.f, P.d, kBM / 2)) != cudaSuccess) return e;
        if ((e = half_map(&G.ta[1], P.wu, P.f, P.d, kBM / 2)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[0], P.x, P.T, P.d, G.npad)) != cudaSuccess) return e;
        G.ahead = static_cast<const uint8_t *>(P.wd);
        G.ahead_bytes = ahead;
        e = launch_skinny<kPair, false>(G, bf16, GatedSplit{P.a, lo, P.g, P.u, P.f, P.dtype}, sms, s);
    } else {
        GemmArgs G = {};
        G.K = P.d;
        G.kb = G.kb_seg = pieces(P.d);
        const Plan L = plan(&P.T, &P.f, 1, G.kb, true, false, sms);
        set_shape(G, L, &P.T, &P.f, 1, true);
        G.idesc = tc::idesc_half(kBM * L.cg, G.BN, bf16, false, false);
        if ((e = half_map(&G.ta[0], P.x, P.T, P.d, kBM)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[0], P.wg, P.f, P.d, box_rows_b(L, true))) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[1], P.wu, P.f, P.d, box_rows_b(L, true))) != cudaSuccess) return e;
        if (G.S > 1) {
            G.ahead = static_cast<const uint8_t *>(P.wd);
            G.ahead_bytes = ahead;
        }
        e = launch_gemm<kHalf, kPair, false, false>(G, L, Gated{{}, P.a, P.g, P.u, P.f, P.dtype}, sms, s);
    }
    if (e != cudaSuccess) return e;
    Store st = {};
    st.out[0] = P.out;
    st.ld[0] = P.d;
    st.dtype = P.out_dtype;
    st.add = P.mode;
    st.vec = 1; // d % 8 == 0
    if (skinny_wins(P.T, P.d, pieces(P.f), false, sms)) {
        SkinnyArgs G = skinny(P.T, P.d, P.f, P.sums);
        G.early_w = 1;
        G.lo = split;
        if ((e = half_map(&G.ta[0], P.wd, P.d, P.f, kBM)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[0], P.a, P.T, P.f, G.npad)) != cudaSuccess) return e;
        if (split && (e = half_map(&G.tl[0], lo, P.T, P.f, G.npad)) != cudaSuccess) return e;
        return launch_skinny<kOne, false>(G, bf16, st, sms, s);
    }
    GemmArgs G = {};
    G.K = P.f;
    G.kb = G.kb_seg = pieces(P.f);
    const Plan L = plan(&P.T, &P.d, 1, G.kb, false, false, sms);
    set_shape(G, L, &P.T, &P.d, 1, false);
    G.idesc = tc::idesc_half(kBM * L.cg, G.BN, bf16, false, false);
    if ((e = half_map(&G.ta[0], P.a, P.T, P.f, kBM)) != cudaSuccess) return e;
    if ((e = half_map(&G.tb[0], P.wd, P.d, P.f, box_rows_b(L, false))) != cudaSuccess) return e;
    G.early_b = 1;
    return launch_gemm<kHalf, kOne, false, false>(G, L, st, sms, s);
}

cudaError_t launch_ffn_backward(const FfnBwd &P, cudaStream_t s) {
    const int sms = device_sm_count();
    const bool bf16 = P.dtype == WASTE_ACT_BF16;
    // few tokens: a, dg and du in two parts
    const bool split = P.T <= kSplitTokens;
    const auto rest = [&](void *p) { return split ? static_cast<uint16_t *>(p) + (size_t)P.T * P.f : nullptr; };
    void *a_lo = rest(P.a), *dg_lo = rest(P.dg), *du_lo = rest(P.du);
    const GatedGrad grad{{}, P.g, P.u, P.a, P.dg, P.du, P.f, P.dtype, a_lo, dg_lo, du_lo};
    cudaError_t e;
    if (skinny_wins(P.T, P.f, pieces(P.d), false, sms)) {
        SkinnyArgs G = skinny(P.T, P.f, P.d, P.sums);
        if ((e = half_map(&G.ta[0], P.wd, P.d, P.f, 64)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[0], P.dy, P.T, P.d, G.npad)) != cudaSuccess) return e;
        e = launch_skinny<kOne, true>(G, bf16, grad, sms, s);
        if (e != cudaSuccess) return e;
    } else {
        GemmArgs G = {};
        G.K = P.d;
        G.kb = G.kb_seg = pieces(P.d);
        const Plan L = plan(&P.T, &P.f, 1, G.kb, false, false, sms, true);
        set_shape(G, L, &P.T, &P.f, 1, false);
        G.idesc = tc::idesc_half(kBM * L.cg, G.BN, bf16, false, true);
        if ((e = half_map(&G.ta[0], P.dy, P.T, P.d, kBM)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[0], P.wd, P.d, P.f, 64)) != cudaSuccess) return e;
        e = launch_gemm<kHalf, kOne, false, true>(G, L, grad, sms, s);
        if (e != cudaSuccess) return e;
    }
    if (P.dx && skinny_wins(P.T, P.d, 2 * pieces(P.f), false, sms)) {
        SkinnyArgs G = skinny(P.T, P.d, P.f, P.sums);
        G.kb = 2 * G.kb_seg;
        G.early_w = 1;
        G.lo = split;
        const void *w[2] = {P.wg, P.wu}, *t[2] = {P.dg, P.du}, *l[2] = {dg_lo, du_lo};
        for (int i = 0; i < 2; ++i) {
            if (split && (e = half_map(&G.tl[i], l[i], P.T, P.f, G.npad)) != cudaSuccess) return e;
            if ((e = half_map(&G.ta[i], w[i], P.f, P.d, 64)) != cudaSuccess) return e;
            if ((e = half_map(&G.tb[i], t[i], P.T, P.f, G.npad)) != cudaSuccess) return e;
        }
        Store st = {};
        st.out[0] = P.dx;
        st.ld[0] = P.d;
        st.dtype = P.dtype;
        st.vec = 1;
        e = launch_skinny<kSum, true>(G, bf16, st, sms, s);
        if (e != cudaSuccess) return e;
    } else if (P.dx) {
        GemmArgs G = {};
        G.K = P.f;
        G.kb_seg = pieces(P.f);
        G.kb = 2 * G.kb_seg;
        const Plan L = plan(&P.T, &P.d, 1, G.kb, false, false, sms);
        set_shape(G, L, &P.T, &P.d, 1, false);
        G.idesc = tc::idesc_half(kBM * L.cg, G.BN, bf16, false, true);
        if ((e = half_map(&G.ta[0], P.dg, P.T, P.f, kBM)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[0], P.wg, P.f, P.d, 64)) != cudaSuccess) return e;
        if ((e = half_map(&G.ta2[0], P.du, P.T, P.f, kBM)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb2[0], P.wu, P.f, P.d, 64)) != cudaSuccess) return e;
        G.early_b = 1;
        Store st = {};
        st.out[0] = P.dx;
        st.ld[0] = P.d;
        st.dtype = P.dtype;
        st.vec = 1;
        e = launch_gemm<kHalf, kSum, false, true>(G, L, st, sms, s);
        if (e != cudaSuccess) return e;
    }
    if (!P.dwg) return cudaSuccess;
    const int M[3] = {P.f, P.f, P.d}, N[3] = {P.d, P.d, P.f};
    GemmArgs G = {};
    G.K = P.T;
    G.kb_seg = pieces(P.T);
    G.kb = split ? 2 * G.kb_seg : G.kb_seg; // the low parts' products behind the others'
    const Plan L = plan(M, N, 3, G.kb, false, false, sms);
    set_shape(G, L, M, N, 3, false);
    G.idesc = tc::idesc_half(kBM * L.cg, G.BN, bf16, true, true);
    const void *a[3] = {P.dg, P.du, P.dy}, *b[3] = {P.x, P.x, P.a};
    const void *a2[3] = {dg_lo, du_lo, P.dy}, *b2[3] = {P.x, P.x, a_lo};
    void *out[3] = {P.dwg, P.dwu, P.dwd};
    Store st = {};
    for (int i = 0; i < 3; ++i) {
        if ((e = half_map(&G.ta[i], a[i], P.T, M[i], 64)) != cudaSuccess) return e;
        if ((e = half_map(&G.tb[i], b[i], P.T, N[i], 64)) != cudaSuccess) return e;
        if (split && (e = half_map(&G.ta2[i], a2[i], P.T, M[i], 64)) != cudaSuccess) return e;
        if (split && (e = half_map(&G.tb2[i], b2[i], P.T, N[i], 64)) != cudaSuccess) return e;
        st.out[i] = out[i];
        st.ld[i] = N[i];
    }
    st.dtype = P.grad_dtype;
    st.add = P.accumulate;
    st.vec = 1;
    return split ? launch_gemm<kHalf, kSum, true, true>(G, L, st, sms, s)
                 : launch_gemm<kHalf, kOne, true, true>(G, L, st, sms, s);
}

namespace {
__global__ void __launch_bounds__(32) debug_wait_kernel(int polls, int arrive) {
    __shared__ __align__(8) uint64_t bar;
    const uint32_t at = tc::smem_u32(&bar);
    if (threadIdx.x == 0) {
        tc::mbar_init(at, 1);
        tc::mbar_init_fence();
        if (arrive) tc::mbar_arrive(at);
    }
    __syncwarp();
    if (!all(tc::mbar_wait(at, 0, polls)) && threadIdx.x == 0) atomicOr(&g_dense_timeout, 1u);
}
} // namespace
cudaError_t launch_debug_wait(int polls, int arrive, cudaStream_t s) {
    debug_wait_kernel<<<1, 32, 0, s>>>(polls, arrive);
    return cudaGetLastError();
}

cudaError_t ffn_timeout(uint32_t *out) { return read_and_clear_timeout(out); }

} // namespace dense
} // namespace wm
