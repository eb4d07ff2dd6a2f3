// Products of microscaled 4-bit matrices on the block-scaled tensor core (dense_gemm.cuh): codes
// and scales go to it as they lie in memory.
#include "dense_gemm.cuh"

namespace wm {
namespace dense {

namespace {

// a = silu(g) u, quantised block by block (32 columns of a row) on its way out: a thread's block of a
// tile, or four lanes' of a row of split sums (a few rows: the loads of 32 columns of every part one after
// another took longest; block of 3 tokens, d 7168, f 1536, 20.7 us by one lane, 16.8 by four).
// The scale bytes between the last block and the next multiple of four are zeroed: the product
// that reads them multiplies them with zero codes.
struct GatedMx4 {
    static constexpr int kWidth = 8, kLanes = 4;
    static constexpr bool kTurns = false, kAhead = false;
    uint8_t *codes, *scales;
    int f, kb;
    __device__ __forceinline__ void scale(int m, int n, uint8_t s) const {
        uint8_t *sp = scales + mx_scale_at(m, n / kMxBlock, kb);
        *sp = s;
        if (n + kMxBlock == f)
            for (int b = n / kMxBlock + 1, j = 1; b & 3; ++b, ++j) sp[j] = 0;
    }
    template <int W>
    __device__ __forceinline__ void row(int, int m, int n, const float (&g)[W], const float (&u)[W]) const {
        static_assert(W == 8, "a quarter of a block");
        if (n >= f) return; // f % 32 == 0: all four lanes or none
        float v[W];
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            v[i] = g[i] * sigmoid(g[i]) * u[i];
            big = max(big, __float_as_uint(v[i]) & 0x7fffffffu);
        }
        const uint32_t four = 0xfu << (threadIdx.x & 28);
        big = max(big, __shfl_xor_sync(four, big, 1));
        big = max(big, __shfl_xor_sync(four, big, 2));
        const bool bad = mx_bad(big);
        const int e = mx_exponent(big);
        const float inv = mx_inverse(e);
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] *= inv;
        *reinterpret_cast<uint32_t *>(codes + (size_t)m * (f / 2) + n / 2) = bad ? 0 : mx_codes8(v);
        if (n % kMxBlock == 0) scale(m, n, bad ? 255 : (uint8_t)(e + 127));
    }
    template <int W>
    __device__ __forceinline__ void tile(const Out32 &o, int, int n, const float (&g)[W], const float (&u)[W]) const {
        static_assert(W == kMxBlock, "one block a row");
        if (o.lane >= o.rows || n >= f) return;
        const int m = o.m + o.lane;
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = g[i] * sigmoid(g[i]) * u[i];
        uint32_t w[4];
        scale(m, n, mx_quantize(v, w));
        *reinterpret_cast<uint4 *>(codes + (size_t)m * (f / 2) + n / 2) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Maps of an operand's codes and scales.
cudaError_t maps(CUtensorMap *codes, CUtensorMap *scales, const Mx4Mat &x, int box_rows) {
    const cudaError_t e = make_map(codes, x.codes, 1, x.rows, (size_t)x.cols / 2, box_rows);
    if (e != cudaSuccess) return e;
    return make_scale_map(scales, x.scales, mx_scale_bytes(x.rows, x.cols) / kMxTileBytes);
}

// Everything but B's maps.
cudaError_t common(GemmArgs &G, Plan &L, const Mx4Mat &a, const Mx4Mat &b, bool pair, int sms) {
    G.K = a.cols;
    G.kb = G.kb_seg = (a.cols + 255) / 256;
    G.skb = (a.cols + 127) / 128;
    L = plan(&a.rows, &b.rows, 1, G.kb, pair, true, sms);
    set_shape(G, L, &a.rows, &b.rows, 1, pair);
    G.idesc = tc::idesc_mx4(kBM * L.cg, G.BN, 0);
    return maps(&G.ta[0], &G.sa, a, kBM);
}

} // namespace

cudaError_t launch_mx4_matmul(const Mx4Mat &a, const Mx4Mat &b, void *out, int out_dtype, int mode, bool after_own,
                              cudaStream_t s) {
    if (mx4_gemv_wins(a, b)) return launch_mx4_gemv(a, b, out, out_dtype, mode, s);
    const int sms = device_sm_count();
    GemmArgs G = {};
    Plan L;
    cudaError_t e = common(G, L, a, b, false, sms);
    if (e == cudaSuccess) e = maps(&G.tb[0], &G.sb[0], b, box_rows_b(L, false));
    if (e != cudaSuccess) return e;
    G.early_b = after_own;
    Store st = {};
    st.out[0] = out;
    st.ld[0] = b.rows;
    st.dtype = out_dtype;
    st.add = mode;
    st.vec = (size_t)b.rows * type_size(out_dtype) % 16 == 0;
    return launch_gemm<kMx4, kOne, false, false>(G, L, st, sms, s);
}

cudaError_t launch_mx4_gated(const Mx4Mat &x, const Mx4Mat &gate, const Mx4Mat &up, const Mx4Mat &next,
                             uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int sms = device_sm_count();
    GemmArgs G = {};
    Plan L;
    cudaError_t e = common(G, L, x, gate, true, sms);
    if (e == cudaSuccess) e = maps(&G.tb[0], &G.sb[0], gate, box_rows_b(L, true));
    if (e == cudaSuccess) e = maps(&G.tb[1], &G.sb[1], up, box_rows_b(L, true));
    if (e != cudaSuccess) return e;
    G.early_b = 1;
    const size_t bytes = mx_code_bytes(next.rows, next.cols);
    if (G.S > 1 && bytes <= kAheadMost) {
        G.ahead = next.codes;
        G.ahead_bytes = bytes;
    }
    const int f = gate.rows;
    return launch_gemm<kMx4, kPair, false, false>(G, L, GatedMx4{codes, scales, f, (f + 127) / 128}, sms, s);
}

cudaError_t mx4_timeout(uint32_t *out) { return read_and_clear_timeout(out); }

} // namespace dense
} // namespace wm
