// Products of microscaled 4-bit matrices on the block-scaled tensor core (dense_gemm.cuh): codes
// and scales go to it as they lie in memory.
#include "dense_gemm.cuh"

namespace wm {
namespace dense {

namespace {

// a = silu(g) u, quantised block by block (32 columns of a row, one thread's) on its way out.
// The scale bytes between the last block and the next multiple of four are zeroed: the product
// that reads them multiplies them with zero codes.
struct GatedMx4 {
    static constexpr int kWidth = 32;
    uint8_t *codes, *scales;
    int f, kb;
    template <int W>
    __device__ __forceinline__ void row(int, int m, int n, const float (&g)[W], const float (&u)[W]) const {
        static_assert(W == kMxBlock, "one block a row");
        if (n >= f) return;
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = g[i] * sigmoid(g[i]) * u[i];
        uint32_t w[4];
        uint8_t *sp = scales + mx_scale_at(m, n / kMxBlock, kb);
        *sp = mx_quantize(v, w);
        *reinterpret_cast<uint4 *>(codes + (size_t)m * (f / 2) + n / 2) = make_uint4(w[0], w[1], w[2], w[3]);
        if (n + W == f)
            for (int b = n / kMxBlock + 1, j = 1; b & 3; ++b, ++j) sp[j] = 0;
    }
};

cudaError_t mx_map(CUtensorMap *m, const Mx4Mat &x, int box_rows) {
    return make_map(m, x.codes, 1, x.rows, (size_t)x.cols / 2, box_rows);
}

GemmArgs common(const Mx4Mat &a, const Mx4Mat &b, bool pair, int sms) {
    GemmArgs G = {};
    G.K = a.cols;
    G.kb = G.kb_seg = (a.cols + 255) / 256;
    const Plan L = plan(&a.rows, &b.rows, 1, G.kb, pair, true, sms);
    G.BN = L.BN;
    G.S = L.S;
    G.nacc = G.BN <= 128 ? 2 : 1; // the scales of the stages take tensor memory too
    set_problems(G, &a.rows, &b.rows, 1, pair);
    G.idesc = tc::idesc_mx4(kBM, G.BN, 0);
    G.sa = a.scales;
    G.sb[0] = b.scales;
    G.skb = (a.cols + 127) / 128;
    G.nbt = (b.rows + kMxTileRows - 1) / kMxTileRows;
    return G;
}

} // namespace

cudaError_t launch_mx4_matmul(const Mx4Mat &a, const Mx4Mat &b, void *out, int out_dtype, int mode, bool after_own,
                              cudaStream_t s) {
    const int sms = device_sm_count();
    GemmArgs G = common(a, b, false, sms);
    G.early_b = after_own;
    cudaError_t e = mx_map(&G.ta[0], a, kBM);
    if (e == cudaSuccess) e = mx_map(&G.tb[0], b, G.BN);
    if (e != cudaSuccess) return e;
    Store st = {};
    st.out[0] = out;
    st.ld[0] = b.rows;
    st.dtype = out_dtype;
    st.add = mode;
    st.vec = (size_t)b.rows * type_size(out_dtype) % 16 == 0;
    return launch_gemm<kMx4, kOne, false, false>(G, st, sms, s);
}

cudaError_t launch_mx4_gated(const Mx4Mat &x, const Mx4Mat &gate, const Mx4Mat &up, const Mx4Mat &next,
                             uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int sms = device_sm_count();
    GemmArgs G = common(x, gate, true, sms);
    G.sb[1] = up.scales;
    G.early_b = 1;
    const size_t bytes = mx_code_bytes(next.rows, next.cols);
    if (G.S > 1 && bytes <= kAheadMost) {
        G.ahead = next.codes;
        G.ahead_bytes = bytes;
    }
    cudaError_t e = mx_map(&G.ta[0], x, kBM);
    if (e == cudaSuccess) e = mx_map(&G.tb[0], gate, G.BN / 2);
    if (e == cudaSuccess) e = mx_map(&G.tb[1], up, G.BN / 2);
    if (e != cudaSuccess) return e;
    const int f = gate.rows;
    return launch_gemm<kMx4, kPair, false, false>(G, GatedMx4{codes, scales, f, (f + 127) / 128}, sms, s);
}

cudaError_t mx4_timeout(uint32_t *out) { return read_and_clear_timeout(out); }

} // namespace dense
} // namespace wm
