// Host side of waste_dense.h: argument checks, workspace layout and the launches of each call.
#include "checks.cuh"
#include "tc_dev.cuh"
#include "train.cuh"

using namespace wm;
using namespace wm::dense;

namespace {

int check_ffn(const waste_ffn_config *c, int32_t T) {
    if (!c) return fail(WASTE_EINVAL, "config is NULL");
    if (c->abi_version != WASTE_MOE_ABI_VERSION)
        return fail(WASTE_EINVAL, "abi_version %u, library speaks %u", c->abi_version, WASTE_MOE_ABI_VERSION);
    if (c->d <= 0 || c->d % 8) return fail(WASTE_EINVAL, "d = %d must be a positive multiple of 8", c->d);
    if (c->f <= 0 || c->f % 8) return fail(WASTE_EINVAL, "f = %d must be a positive multiple of 8", c->f);
    if (!half_type(c->dtype)) return fail(WASTE_EINVAL, "dtype = %d: bf16 or fp16", c->dtype);
    if (c->d > kMostRows || c->f > kMostRows) return fail(WASTE_EINVAL, "d = %d, f = %d: at most 2^30", c->d, c->f);
    if (T < 0 || T > kMostRows) return fail(WASTE_EINVAL, "T = %d outside [0, 2^30]", T);
    return WASTE_OK;
}

// One [T][f] buffer of the workspace; a forward call of few tokens keeps 32 bits of each value in
// it, so the size for T tokens also covers every smaller call.
static_assert(kGemvTokens <= kSplitTokens, "32 bits of a");
size_t ffn_part(const waste_ffn_config *c, int32_t T) {
    const size_t few = T < kSplitTokens ? T : kSplitTokens, half = (size_t)T * c->f * 2, full = few * c->f * 4;
    return round_up(half > full ? half : full, 256);
}

// And for a call of few tokens its partial sums (a forward of kGemvTokens has none).
size_t ffn_bytes(const waste_ffn_config *c, int32_t T, bool backward) {
    const int parts = backward ? 3 : 1, few = T < kSkinnyTokens ? T : kSkinnyTokens;
    const size_t all = parts * ffn_part(c, T);
    if (few <= (backward ? 0 : kGemvTokens)) return all;
    const size_t with_sums = parts * ffn_part(c, few) + skinny_bytes(few);
    return all > with_sums ? all : with_sums;
}

int check_mx4_shape(int32_t rows, int32_t cols) {
    if (rows < 0 || rows > kMostRows) return fail(WASTE_EINVAL, "rows = %d outside [0, 2^30]", rows);
    if (cols <= 0 || cols % kMxBlock || cols > kMostRows)
        return fail(WASTE_EINVAL, "cols = %d must be a positive multiple of 32, at most 2^30", cols);
    return WASTE_OK;
}

int check_mx4_x(const void *x, int dtype, int cols, int64_t ld, const char *name) {
    if (!any_type(dtype)) return fail(WASTE_EINVAL, "dtype = %d: fp32, bf16 or fp16", dtype);
    if (ld < cols || ld * (int64_t)type_size(dtype) % 16)
        return fail(WASTE_EINVAL, "row stride %lld: at least cols = %d and a multiple of 16 bytes", (long long)ld, cols);
    const void *p[] = {x};
    const char *n[] = {name};
    return check_ptrs(p, n, 1);
}

int check_mx4_ffn(const waste_mx4_ffn_config *c, int32_t T) {
    if (!c) return fail(WASTE_EINVAL, "config is NULL");
    if (c->abi_version != WASTE_MOE_ABI_VERSION)
        return fail(WASTE_EINVAL, "abi_version %u, library speaks %u", c->abi_version, WASTE_MOE_ABI_VERSION);
    if (c->d <= 0 || c->d % kMxBlock) return fail(WASTE_EINVAL, "d = %d must be a positive multiple of 32", c->d);
    if (c->f <= 0 || c->f % kMxBlock) return fail(WASTE_EINVAL, "f = %d must be a positive multiple of 32", c->f);
    if (c->d > kMostRows || c->f > kMostRows) return fail(WASTE_EINVAL, "d = %d, f = %d: at most 2^30", c->d, c->f);
    if (T < 0 || T > kMostRows) return fail(WASTE_EINVAL, "T = %d outside [0, 2^30]", T);
    return WASTE_OK;
}

struct Mx4FfnParts {
    size_t xc, xs, ac, as, af, total;
};
Mx4FfnParts mx4_ffn_parts(const waste_mx4_ffn_config *c, int32_t T) {
    Mx4FfnParts p;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += round_up(bytes, 256);
        return o;
    };
    p.xc = take(mx_code_bytes(T, c->d));
    p.xs = take(mx_scale_bytes(T, c->d));
    p.ac = take(mx_code_bytes(T, c->f));
    p.as = take(mx_scale_bytes(T, c->f));
    // calls of few tokens keep a in fp32 instead
    p.af = take((size_t)(T < kMxGemvTokens ? T : kMxGemvTokens) * c->f * 4);
    p.total = at;
    return p;
}

} // namespace

extern "C" {

int waste_dense_status(void) {
    uint32_t timeout = 0, offsets = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = ffn_timeout(&timeout);
    if (e == cudaSuccess) e = mx4_timeout(&timeout);
    if (e == cudaSuccess) e = train::group_status(&timeout, &offsets);
    if (e == cudaSuccess) e = train::ortho_timeout(&timeout);
    if (e == cudaSuccess) e = train::norm_timeout(&timeout);
    if (e != cudaSuccess) return done(e, "reading the status");
    if (timeout) return fail(WASTE_ETIMEOUT, "a device wait of a dense operator gave up");
    if (offsets) return fail(WASTE_EINVAL, "offsets of a product grouped by expert fall or leave the rows");
    return ok();
}

int waste_dense_debug_wait(int32_t polls, int32_t arrive, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    if (polls < 0 || polls > tc::kWaitPolls) return fail(WASTE_EINVAL, "polls = %d outside [0, 2^18]", polls);
    if (arrive != 0 && arrive != 1) return fail(WASTE_EINVAL, "arrive = %d", arrive);
    return done(launch_debug_wait(polls ? polls : tc::kWaitPolls, arrive, reinterpret_cast<cudaStream_t>(stream)), "wait kernel");
}

int waste_ffn_workspace(const waste_ffn_config *cfg, int32_t T, int32_t backward, size_t *bytes) {
    const int rc = check_ffn(cfg, T);
    if (rc) return rc;
    if (!bytes) return fail(WASTE_EINVAL, "bytes is NULL");
    *bytes = ffn_bytes(cfg, T, backward);
    return ok();
}

int waste_ffn_forward(const waste_ffn_config *cfg, const void *d_x, int32_t T, const void *d_w_gate,
                      const void *d_w_up, const void *d_w_down, void *d_out, int32_t out_dtype, int32_t mode,
                      void *d_g, void *d_u, void *d_workspace, size_t workspace_bytes, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_ffn(cfg, T);
    if (rc) return rc;
    if (out_dtype != cfg->dtype && out_dtype != WASTE_ACT_F32)
        return fail(WASTE_EINVAL, "out_dtype = %d: the config's dtype or fp32", out_dtype);
    if (mode != 0 && mode != 1) return fail(WASTE_EINVAL, "mode = %d", mode);
    if (!d_g != !d_u) return fail(WASTE_EINVAL, "g and u: both or neither");
    if (T == 0) return ok();
    const void *p[] = {d_x, d_w_gate, d_w_up, d_w_down, d_out, d_g, d_u};
    const char *n[] = {"x", "w_gate", "w_up", "w_down", "out", "g", "u"};
    rc = check_ptrs(p, n, d_g ? 7 : 5);
    const size_t need = ffn_bytes(cfg, T, false), w = (size_t)cfg->d * cfg->f * 2, tf = (size_t)T * cfg->f * 2;
    if (!rc) rc = check_workspace(d_workspace, workspace_bytes, need);
    if (rc) return rc;
    // x is read by the first launch alone, out written by the last: the two may overlap
    const Span x{d_x, (size_t)T * cfg->d * 2, "x"}, out{d_out, (size_t)T * cfg->d * type_size(out_dtype), "out"};
    const Span ws{d_workspace, need, "workspace"}, g{d_g, tf, "g"}, u{d_u, tf, "u"};
    const Span wg{d_w_gate, w, "w_gate"}, wu{d_w_up, w, "w_up"}, wd{d_w_down, w, "w_down"};
    const Span kept[] = {ws, g, u, out, x, wg, wu, wd}, last[] = {out, wg, wu, wd};
    if ((rc = check_apart(kept, 3, 8)) || (rc = check_apart(last, 1, 4))) return rc;
    FfnFwd P{cfg->d, cfg->f, T, cfg->dtype, out_dtype, mode, d_x, d_w_gate, d_w_up, d_w_down, d_out, d_g, d_u,
             d_workspace, reinterpret_cast<float *>(static_cast<char *>(d_workspace) + ffn_part(cfg, T))};
    return done(launch_ffn_forward(P, reinterpret_cast<cudaStream_t>(stream)), "gated feed-forward");
}

int waste_ffn_backward(const waste_ffn_config *cfg, const void *d_dy, int32_t T, const void *d_x, const void *d_g,
                       const void *d_u, const void *d_w_gate, const void *d_w_up, const void *d_w_down, void *d_dx,
                       void *d_dw_gate, void *d_dw_up, void *d_dw_down, int32_t grad_dtype, int32_t accumulate,
                       void *d_workspace, size_t workspace_bytes, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_ffn(cfg, T);
    if (rc) return rc;
    if (grad_dtype != cfg->dtype && grad_dtype != WASTE_ACT_F32)
        return fail(WASTE_EINVAL, "grad_dtype = %d: the config's dtype or fp32", grad_dtype);
    if (accumulate != 0 && accumulate != 1) return fail(WASTE_EINVAL, "accumulate = %d", accumulate);
    const bool dw = d_dw_gate != nullptr;
    if ((d_dw_up != nullptr) != dw || (d_dw_down != nullptr) != dw)
        return fail(WASTE_EINVAL, "dw_gate, dw_up and dw_down: all or none");
    if (!d_dx && !dw) return ok();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dw) {
        const void *p[] = {d_dw_gate, d_dw_up, d_dw_down};
        const char *n[] = {"dw_gate", "dw_up", "dw_down"};
        if ((rc = check_ptrs(p, n, 3))) return rc;
    }
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        const size_t bytes = (size_t)cfg->d * cfg->f * type_size(grad_dtype);
        if (dw && !accumulate) {
            void *w[] = {d_dw_gate, d_dw_up, d_dw_down};
            for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = cudaMemsetAsync(w[i], 0, bytes, s);
        }
        return done(e, "clearing the gradients");
    }
    const void *p[] = {d_dy, d_x, d_g, d_u, d_w_gate, d_w_up, d_w_down, d_dx};
    const char *n[] = {"dy", "x", "g", "u", "w_gate", "w_up", "w_down", "dx"};
    rc = check_ptrs(p, n, d_dx ? 8 : 7);
    const size_t part = ffn_part(cfg, T), need = ffn_bytes(cfg, T, true), wn = (size_t)cfg->d * cfg->f;
    if (!rc) rc = check_workspace(d_workspace, workspace_bytes, need);
    if (rc) return rc;
    const size_t td = (size_t)T * cfg->d * 2, tf = (size_t)T * cfg->f * 2, gn = wn * type_size(grad_dtype);
    const Span spans[] = {{d_workspace, need, "workspace"}, {d_dx, td, "dx"}, {d_dw_gate, gn, "dw_gate"},
                          {d_dw_up, gn, "dw_up"}, {d_dw_down, gn, "dw_down"}, {d_dy, td, "dy"}, {d_x, td, "x"},
                          {d_g, tf, "g"}, {d_u, tf, "u"}, {d_w_gate, wn * 2, "w_gate"}, {d_w_up, wn * 2, "w_up"},
                          {d_w_down, wn * 2, "w_down"}};
    if ((rc = check_apart(spans, 5, 12))) return rc;
    char *w = static_cast<char *>(d_workspace);
    FfnBwd P{cfg->d, cfg->f,  T,      cfg->dtype, grad_dtype, accumulate, d_dy, d_x,      d_g,         d_u, d_w_gate,
             d_w_up, d_w_down, d_dx, d_dw_gate,  d_dw_up,    d_dw_down,  w,    w + part, w + 2 * part,
             reinterpret_cast<float *>(w + 3 * part)};
    return done(launch_ffn_backward(P, s), "gated feed-forward gradients");
}

int waste_mx4_layout(int32_t rows, int32_t cols, size_t *code_bytes, size_t *scale_bytes) {
    const int rc = check_mx4_shape(rows, cols);
    if (rc) return rc;
    if (code_bytes) *code_bytes = mx_code_bytes(rows, cols);
    if (scale_bytes) *scale_bytes = mx_scale_bytes(rows, cols);
    return ok();
}

int waste_mx4_quantize(const void *d_x, int32_t dtype, int32_t rows, int32_t cols, int64_t ld, uint8_t *d_codes,
                       uint8_t *d_scales, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_mx4_shape(rows, cols);
    if (rc || rows == 0) return rc ? rc : ok();
    rc = check_mx4_x(d_x, dtype, cols, ld, "x");
    const void *p[] = {d_codes, d_scales};
    const char *n[] = {"codes", "scales"};
    if (!rc) rc = check_ptrs(p, n, 2);
    if (rc) return rc;
    const size_t size = type_size(dtype);
    const Span spans[] = {{d_codes, mx_code_bytes(rows, cols), "codes"}, {d_scales, mx_scale_bytes(rows, cols), "scales"},
                          {d_x, cols * size, "x", (size_t)rows, ld * size}};
    if ((rc = check_apart(spans, 2, 3))) return rc;
    return done(launch_mx4_quantize(d_x, dtype, rows, cols, ld, d_codes, d_scales,
                                    reinterpret_cast<cudaStream_t>(stream)),
                "4-bit quantisation");
}

int waste_mx4_dequantize(const uint8_t *d_codes, const uint8_t *d_scales, int32_t rows, int32_t cols, void *d_out,
                         int32_t dtype, int64_t ld, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_mx4_shape(rows, cols);
    if (rc || rows == 0) return rc ? rc : ok();
    rc = check_mx4_x(d_out, dtype, cols, ld, "out");
    const void *p[] = {d_codes, d_scales};
    const char *n[] = {"codes", "scales"};
    if (!rc) rc = check_ptrs(p, n, 2);
    if (rc) return rc;
    const size_t size = type_size(dtype);
    const Span out{d_out, cols * size, "out", (size_t)rows, ld * size};
    if (meet({d_codes, mx_code_bytes(rows, cols), "codes"}, out)) return fail(WASTE_EINVAL, "out overlaps codes");
    if (meet({d_scales, mx_scale_bytes(rows, cols), "scales"}, out)) return fail(WASTE_EINVAL, "out overlaps scales");
    return done(launch_mx4_dequantize(Mx4Mat{d_codes, d_scales, rows, cols}, d_out, dtype, ld,
                                      reinterpret_cast<cudaStream_t>(stream)),
                "4-bit dequantisation");
}

int waste_mx4_matmul(int32_t M, int32_t N, int32_t K, const uint8_t *d_a_codes, const uint8_t *d_a_scales,
                     const uint8_t *d_b_codes, const uint8_t *d_b_scales, void *d_out, int32_t out_dtype,
                     int32_t mode, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_mx4_shape(M, K);
    if (rc) return rc;
    if (N < 1 || N > kMostRows) return fail(WASTE_EINVAL, "N = %d outside [1, 2^30]", N);
    if (!any_type(out_dtype)) return fail(WASTE_EINVAL, "out_dtype = %d: fp32, bf16 or fp16", out_dtype);
    if (mode != 0 && mode != 1) return fail(WASTE_EINVAL, "mode = %d", mode);
    if (M == 0) return ok();
    const void *p[] = {d_a_codes, d_a_scales, d_b_codes, d_b_scales, d_out};
    const char *n[] = {"a_codes", "a_scales", "b_codes", "b_scales", "out"};
    rc = check_ptrs(p, n, 5);
    if (rc) return rc;
    const Span spans[] = {{d_out, (size_t)M * N * type_size(out_dtype), "out"},
                          {d_a_codes, mx_code_bytes(M, K), "a_codes"},
                          {d_a_scales, mx_scale_bytes(M, K), "a_scales"},
                          {d_b_codes, mx_code_bytes(N, K), "b_codes"},
                          {d_b_scales, mx_scale_bytes(N, K), "b_scales"}};
    if ((rc = check_apart(spans, 1, 5))) return rc;
    return done(launch_mx4_matmul(Mx4Mat{d_a_codes, d_a_scales, M, K}, Mx4Mat{d_b_codes, d_b_scales, N, K}, d_out,
                                  out_dtype, mode, false, reinterpret_cast<cudaStream_t>(stream)),
                "4-bit product");
}

int waste_mx4_ffn_workspace(const waste_mx4_ffn_config *cfg, int32_t T, size_t *bytes) {
    const int rc = check_mx4_ffn(cfg, T);
    if (rc) return rc;
    if (!bytes) return fail(WASTE_EINVAL, "bytes is NULL");
    *bytes = mx4_ffn_parts(cfg, T).total;
    return ok();
}

int waste_mx4_ffn_forward(const waste_mx4_ffn_config *cfg, const void *d_x, int32_t x_dtype, int32_t T, void *d_out,
                          int32_t out_dtype, int32_t mode, void *d_workspace, size_t workspace_bytes,
                          waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_mx4_ffn(cfg, T);
    if (rc) return rc;
    if (!any_type(x_dtype) || !any_type(out_dtype))
        return fail(WASTE_EINVAL, "x_dtype = %d, out_dtype = %d: fp32, bf16 or fp16", x_dtype, out_dtype);
    if (mode != 0 && mode != 1) return fail(WASTE_EINVAL, "mode = %d", mode);
    if (T == 0) return ok();
    const void *p[] = {d_x,
                       cfg->d_gate_codes,
                       cfg->d_gate_scales,
                       cfg->d_up_codes,
                       cfg->d_up_scales,
                       cfg->d_down_codes,
                       cfg->d_down_scales,
                       d_out};
    const char *n[] = {"x", "gate_codes", "gate_scales", "up_codes", "up_scales", "down_codes", "down_scales", "out"};
    rc = check_ptrs(p, n, 8);
    const Mx4FfnParts W = mx4_ffn_parts(cfg, T);
    if (!rc) rc = check_workspace(d_workspace, workspace_bytes, W.total);
    if (rc) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(d_workspace);
    const int d = cfg->d, f = cfg->f;
    // x is read by the first launch alone, out written by the last: the two may overlap
    const size_t wide = mx_code_bytes(f, d), tall = mx_code_bytes(d, f), ws = mx_scale_bytes(f, d), ds = mx_scale_bytes(d, f);
    const Span spans[] = {{d_workspace, W.total, "workspace"},
                          {d_out, (size_t)T * d * type_size(out_dtype), "out"},
                          {cfg->d_gate_codes, wide, "gate_codes"},
                          {cfg->d_gate_scales, ws, "gate_scales"},
                          {cfg->d_up_codes, wide, "up_codes"},
                          {cfg->d_up_scales, ws, "up_scales"},
                          {cfg->d_down_codes, tall, "down_codes"},
                          {cfg->d_down_scales, ds, "down_scales"}};
    if ((rc = check_apart(spans, 2, 8))) return rc;
    if (meet(spans[0], {d_x, (size_t)T * d * type_size(x_dtype), "x"})) return fail(WASTE_EINVAL, "workspace overlaps x");
    const Mx4Mat gate{cfg->d_gate_codes, cfg->d_gate_scales, f, d}, up{cfg->d_up_codes, cfg->d_up_scales, f, d},
        down{cfg->d_down_codes, cfg->d_down_scales, d, f};
    if (T <= kMxGemvTokens && mx_gemv_smem(d, T) <= kMxGemvSmem && mx_gemv_smem(f, T) <= kMxGemvSmem)
        return done(launch_mx4_ffn_gemv(d_x, x_dtype, T, gate, up, down, reinterpret_cast<float *>(w + W.af), d_out,
                                        out_dtype, mode, s),
                    "4-bit gated feed-forward");
    cudaError_t e = launch_mx4_quantize(d_x, x_dtype, T, d, d, w + W.xc, w + W.xs, s);
    if (e == cudaSuccess)
        e = launch_mx4_gated(Mx4Mat{w + W.xc, w + W.xs, T, d}, gate, up, down, w + W.ac, w + W.as, s);
    if (e == cudaSuccess)
        e = launch_mx4_matmul(Mx4Mat{w + W.ac, w + W.as, T, f}, down, d_out, out_dtype, mode, true, s);
    return done(e, "4-bit gated feed-forward");
}

} // extern "C"
