// Host side of the dense operators' products: tensor maps, launch shapes, the timeout word.
#include <algorithm>
#include <atomic>

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

// In a host thread that has not used CUDA yet no context is current, and the driver
// refuses (the runtime would make the device's own current by itself): it is made current, once a thread.
cudaError_t encode_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *p, const cuuint64_t *dims,
                       const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion l2) {
    const EncodeFn fn = encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t one[3] = {1, 1, 1};
    const auto call = [&] {
        return fn(m, type, rank, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, l2,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaSetDevice(dev);
        if (e != cudaSuccess) return e;
        r = call();
    }
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {
// A two-dimensional map.
cudaError_t encode(CUtensorMap *m, CUtensorMapDataType type, const void *p, const cuuint64_t (&dims)[2], cuuint64_t stride,
                   const cuuint32_t (&box)[2], CUtensorMapSwizzle swizzle, CUtensorMapL2promotion l2) {
    return encode_map(m, type, 2, p, dims, &stride, box, swizzle, l2);
}
} // namespace

cudaError_t make_map(CUtensorMap *m, const void *p, int unit, int rows, size_t row_bytes, int box_rows) {
    return encode(m, unit == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, p,
                  {row_bytes / unit, (cuuint64_t)rows}, row_bytes, {(cuuint32_t)(kRowBytes / unit), (cuuint32_t)box_rows},
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

cudaError_t store_map(CUtensorMap *m, void *p, int bytes, int rows, int cols) {
    return encode(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32, p,
                  {(cuuint64_t)cols, (cuuint64_t)rows}, (cuuint64_t)cols * bytes, {(cuuint32_t)(64 / bytes), 32},
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

cudaError_t make_scale_map(CUtensorMap *m, const void *p, size_t tiles) {
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, p, {kMxTileBytes / 4, (cuuint64_t)tiles}, kMxTileBytes,
                  {kMxTileBytes / 4, 2}, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

namespace {
// Takes as much of an SM as the products' CTAs do, to ask how many clusters of them fit.
__global__ void __launch_bounds__(kThreads, 1) cluster_probe_kernel() {}
} // namespace

// Clusters of S CTAs (2..8) that run at once on the current device: SMs come in groups that a
// cluster does not cross, so fewer than SMs / S (on one GB300: 76, 46, 36, 28, 23, 15, 15).  0: none.
int clusters_at_once(int S) {
    static std::atomic<int> cache[kMaxDevices][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int n = cache[dev][S].load(std::memory_order_relaxed);
    if (n == 0) {
        static SmemAttr attr;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = S;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(S);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBudget;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (ensure_smem(attr, reinterpret_cast<const void *>(cluster_probe_kernel), kSmemBudget) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, cluster_probe_kernel, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return 0;
        }
        cache[dev][S].store(n, std::memory_order_relaxed);
    }
    return n;
}

// The estimate, in ns: whole waves of tiles, each as long as its bytes need into one SM (its MMAs
// are shorter, or as long, and the way out of all but the last is behind the next one's loads); what a pair
// costs more than a CTA alone, and with 4-bit operands, whose scales both CTAs copy, much more; for
// split k the exchange of the sums, and only one wave (a second one waits for whole clusters to end:
// twice the time).  Its constants are fitted to 1,365 measured launches (16 to 3000 rows, 256 to 7168
// columns and k, both kinds, every shape below): over these it picks a launch 0.7 % slower than the best
// one, in the geometric mean (with the same for 4 bits 1.6 %: 509 x 7168 x 1536 in pairs 8.1 us, without 7.0).
// heavy: an epilogue that reads and writes several matrices (the gradients': for 333 tokens, d 1032, f
// 264 four CTAs a tile make the backward 22.7 -> 19.2 us).
Plan plan(const int *M, const int *N, int n, int kb, bool pair, bool mx4, int sms, bool heavy) {
    Plan best{256, 1, 1, 1e30};
    int rows = 0;
    for (int i = 0; i < n; ++i) rows = std::max(rows, std::min(M[i], kBM));
    const auto consider = [&](int BN, int cg, int S) {
        const int w = pair ? BN / 2 : BN, h = kBM * cg;
        long long tiles = 0;
        for (int i = 0; i < n; ++i) tiles += (long long)((M[i] + h - 1) / h) * ((N[i] + w - 1) / w);
        const int slots = S > 1 ? clusters_at_once(S) : sms / cg;
        if (slots < 1) return;
        const long long waves = (tiles + slots - 1) / slots;
        if (S > 1 && waves > 1) return;
        const double piece = (kBM + BN / cg) * kRowBytes / 80.0;
        double t = (cg == 1 ? 0.0 : mx4 ? 4000.0 : 1570.0) + (double)waves * ((kb + S - 1) / S) * piece;
        if (S > 1) t += 3400.0 + rows * BN * 0.43;
        if (heavy) t += rows * BN * 0.6 / S; // split k splits the way out too
        if (t < best.ns) best = Plan{BN, S, cg, t};
    };
    // 4-bit: whole scale tiles (128 rows) of each product; 16-bit: any multiple of 32
    const int least = mx4 ? (pair ? 256 : 128) : 64;
    for (int BN = 256; BN >= least; BN -= mx4 ? 128 : 32)
        if (rows == kBM) consider(BN, 2, 1);
    for (int BN = 256; BN >= least; BN /= 2)
        for (int S = 1; S <= 8 && S <= kb; ++S) consider(BN, 1, S);
    return best;
}

} // namespace dense
} // namespace wm
