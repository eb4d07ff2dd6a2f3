// Host side of the dense operators' products: tensor maps, launch shapes, the timeout word.
#include <algorithm>

#include "dense_gemm.cuh"

namespace wm {
namespace dense {

namespace {
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}
} // namespace

cudaError_t make_map(CUtensorMap *m, const void *p, int unit, int rows, size_t row_bytes, int box_rows) {
    const EncodeFn fn = encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {row_bytes / unit, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / unit), (cuuint32_t)box_rows};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r = fn(m, unit == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                          const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_scale_map(CUtensorMap *m, const void *p, size_t tiles) {
    const EncodeFn fn = encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {kMxTileBytes / 4, (cuuint64_t)tiles};
    const cuuint64_t strides[1] = {kMxTileBytes};
    const cuuint32_t box[2] = {kMxTileBytes / 4, 2};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(p), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The estimate: pieces of k one after another, each as long as its MMAs or as its bytes need into
// one SM (about 100 B/ns), whole waves of tiles; splitting k costs the exchange of the sums.
Plan plan(const int *M, const int *N, int n, int kb, bool pair, bool mx4, int sms) {
    Plan best{256, 1, 1};
    double best_t = 1e30;
    int rows = 0;
    for (int i = 0; i < n; ++i) rows = std::max(rows, std::min(M[i], kBM));
    const auto consider = [&](int BN, int cg, int S) {
        const int w = pair ? BN / 2 : BN, h = kBM * cg;
        long long tiles = 0;
        for (int i = 0; i < n; ++i) tiles += (long long)((M[i] + h - 1) / h) * ((N[i] + w - 1) / w);
        const double mma = mx4 ? BN * 0.75 : BN * 1.08, feed = (rows + BN / cg) * 128.0 / 100.0;
        const double piece = std::max(mma, feed);
        const double out = 500.0 + rows * BN * 0.05; // the last tile's way out; the others' is hidden
        const double waves = (double)((tiles * S * cg + sms - 1) / sms);
        const double t = S == 1 ? waves * kb * piece + out
                                : waves * (((kb + S - 1) / S) * piece + out + 1500.0 + rows * BN * 0.02);
        if (t < best_t * 0.98) {
            best_t = t;
            best = Plan{BN, S, cg};
        }
    };
    // 4-bit: whole scale tiles (128 rows) of each product; 16-bit: any multiple of 32
    for (int BN = 256; BN >= (mx4 && pair ? 256 : 128); BN -= mx4 ? 128 : 32)
        if (rows == kBM) consider(BN, 2, 1);
    for (int BN = 256; BN >= (mx4 && pair ? 256 : 128); BN -= 128)
        for (int S = 1; S <= 8 && S <= kb; ++S) consider(BN, 1, S);
    return best;
}

} // namespace dense
} // namespace wm
