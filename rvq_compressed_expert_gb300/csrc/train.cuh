// Internal declarations of the training operators (waste_train.h).
#pragma once

#include "dense.cuh"
#include "dense_tc.cuh"
#include "waste_train.h"

namespace wm {
namespace train {

// Rows of memory, ld elements apart.
struct Rows {
    void *p;
    int64_t ld;
};
struct NormFwd {
    int d, T, x_dtype, y_dtype, w_dtype;
    float eps;
    const void *w, *b; // or null
    Rows x, y;
    float *mean, *rstd; // or null
};
struct NormBwd {
    int d, T, x_dtype, y_dtype, w_dtype, grad_dtype, accumulate;
    const void *w; // or null
    Rows x, dy, dx; // dx.p may be null
    const float *mean, *rstd;
    void *dw, *db; // or null
    float *parts;  // workspace: [norm_parts][2][d]
};
// Partial sums of dw and db: so many rows of them at most.
constexpr int kNormParts = 304;
inline size_t norm_bytes(int d, int T) { return round_up((size_t)(T < kNormParts ? T : kNormParts) * 2 * d * 4, 256); }

struct Group {
    int E, k, n, dtype, rows;
    const int32_t *offsets;
};
// y = x W^T by expert, dx = dy W, dW = dy^T x.
cudaError_t launch_group_forward(const Group &G, const void *x, const void *w, void *y, int out_dtype, int add, cudaStream_t s);
cudaError_t launch_group_dx(const Group &G, const void *dy, const void *w, void *dx, cudaStream_t s);
cudaError_t launch_group_dw(const Group &G, const void *dy, const void *x, void *dw, int grad_dtype, int add, cudaStream_t s);
// *timeout |= whether a wait gave up, *offsets |= whether offsets were out of order, since the last call (cleared).
cudaError_t group_status(uint32_t *timeout, uint32_t *offsets);

// Newton-Schulz: the matrices of a call and its workspace.
struct Ortho {
    int count, rows, cols, steps;
    float a, b, c;
    const void *g;
    int g_dtype;
    void *out;
    int out_dtype, add;
    float scale;
    uint8_t *ws;
};
// What stands in the workspace, from its start: X in two halves (the first of them twice, taken in turn), A and
// b A + c A^2 without its diagonal, that diagonal, partial sums of squares, and A's partial sums.
constexpr int kOrthoParts = 512; // of a matrix
struct OrthoParts {
    size_t hi[2], lo, a, b, diag, sums, gram, total;
    int ldx, ldm;
    int side, tri, slices; // of A: tiles of side x side, those on and below its diagonal, in so many shares of k
};
// A is made in tiles of 256 x 256 by pairs of CTAs (of 128 x 128 by one where it is no larger).  Either those on and below its
// diagonal, the long side split into shares: as many as shorten the waves of tiles (a piece of k takes about 370 ns, 410 in those) by
// more than their fp32 partial sums, written and read again, cost; these are added up by a launch of their own, about 6
// us.  Or, where that costs more than it saves (0 shares), all of its tiles at once.  The workspace has to have one
// size everywhere, so this counts with the SMs of the one device the library is for.
inline int gram_slices(int count, int across, int pieces, int side) {
    const int slots = side == 256 ? 76 : 152;
    const long long tiles = (long long)count * across * (across + 1) / 2, all = (long long)count * across * across;
    int best = 0;
    double least = (double)((all + slots - 1) / slots) * pieces * 410.;
    for (int s = 1; s <= 16 && s <= pieces; ++s) {
        const double waves = (double)((tiles * s + slots - 1) / slots);
        const double t = waves * ((pieces + s - 1) / s) * 370. + (double)(tiles * s) * side * side * 8. / 5000. + 6000.;
        if (t < least) least = t, best = s;
    }
    return best;
}
inline OrthoParts ortho_parts(int count, int rows, int cols) {
    const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    OrthoParts p;
    p.side = m > 128 ? 256 : 128;
    const int across = (m + p.side - 1) / p.side;
    p.tri = across * (across + 1) / 2;
    p.slices = gram_slices(count, across, (n + 63) / 64, p.side);
    p.ldx = (cols + 7) / 8 * 8;
    p.ldm = (m + 7) / 8 * 8;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t o = at;
        at += round_up(bytes, 256);
        return o;
    };
    const size_t x = (size_t)count * rows * p.ldx * 2, s = (size_t)count * m * p.ldm * 2;
    p.hi[0] = take(x), p.hi[1] = take(x), p.lo = take(x);
    p.a = take(s), p.b = take(s);
    p.diag = take((size_t)count * p.ldm * 4);
    p.sums = take((size_t)count * kOrthoParts * 3 * 4);
    p.gram = take((size_t)count * p.tri * p.slices * p.side * p.side * 4);
    p.total = at;
    return p;
}
cudaError_t launch_ortho(const Ortho &P, cudaStream_t s);
cudaError_t ortho_timeout(uint32_t *out);

cudaError_t launch_norm_forward(const NormFwd &P, cudaStream_t s);
cudaError_t launch_norm_backward(const NormBwd &P, cudaStream_t s);
cudaError_t norm_timeout(uint32_t *out);

// Where each unit's kernels say that a wait gave up; and a CTA that lets one do so, by the unit's own wait (the norm's:
// wait_row, three of them and settle), for waste_train_debug_wait.
cudaError_t norm_word(uint32_t **word);
cudaError_t group_word(uint32_t **word);
cudaError_t ortho_word(uint32_t **word);
cudaError_t launch_debug_wait(uint32_t *word, bool rows, int polls, int arrive, cudaStream_t s);

#ifdef __CUDACC__
// The norm's wait for a row: one that gives up (1.1 s at most) says so in *word, and then none of the CTA's is waited for
// any more.
__device__ __forceinline__ void wait_row(uint32_t bar, uint32_t parity, volatile uint32_t *gave_up, uint32_t *word,
                                         int polls = tc::kWaitPolls) {
    if (*gave_up) return;
    if (!tc::mbar_wait(bar, parity, polls)) {
        *gave_up = 1;
        atomicOr(word, 1u);
    }
}
// Behind a wait that gave up: time for copies on their way to land before the CTA goes.
__device__ __forceinline__ void settle(volatile uint32_t *gave_up) {
    if (*gave_up)
        for (int i = 0; i < 64; ++i) __nanosleep(1 << 14);
}
#endif

// A launch that may begin while the kernel before it in the stream ends; the kernel waits for that one itself
// (tc::grid_wait_release) before it touches memory.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

} // namespace train
} // namespace wm
