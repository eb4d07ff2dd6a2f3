// Host side of waste_train.h: argument checks, workspace layout and the launches of each call.
#include <cmath>

#include "checks.cuh"
#include "train.cuh"

using namespace wm;
using namespace wm::dense;
using namespace wm::train;

namespace {

int check_abi(uint32_t v) {
    if (v != WASTE_MOE_ABI_VERSION) return fail(WASTE_EINVAL, "abi_version %u, library speaks %u", v, WASTE_MOE_ABI_VERSION);
    return WASTE_OK;
}
int check_flag(int32_t v, const char *name) { return v == 0 || v == 1 ? WASTE_OK : fail(WASTE_EINVAL, "%s = %d", name, v); }

// ---- layer norm
int check_norm(const waste_norm_config *c, int32_t T) {
    if (!c) return fail(WASTE_EINVAL, "config is NULL");
    if (int rc = check_abi(c->abi_version)) return rc;
    if (c->d < 1 || c->d > kMostRows) return fail(WASTE_EINVAL, "d = %d outside [1, 2^30]", c->d);
    if (!any_type(c->x_dtype) || !any_type(c->y_dtype) || !any_type(c->w_dtype))
        return fail(WASTE_EINVAL, "x_dtype = %d, y_dtype = %d, w_dtype = %d: fp32, bf16 or fp16", c->x_dtype, c->y_dtype, c->w_dtype);
    if (!(c->eps >= 0.f) || std::isinf(c->eps)) return fail(WASTE_EINVAL, "eps = %g must be finite and not negative", (double)c->eps);
    if (T < 0 || T > kMostRows) return fail(WASTE_EINVAL, "T = %d outside [0, 2^30]", T);
    return WASTE_OK;
}
int check_at(const void *p, int dtype, const char *name) {
    if (!p) return fail(WASTE_EINVAL, "%s is NULL", name);
    if (!aligned(p, type_size(dtype))) return fail(WASTE_EINVAL, "%s must be aligned to its type", name);
    return WASTE_OK;
}
int check_rows(const void *p, int dtype, int64_t ld, int32_t d, const char *name) {
    if (int rc = check_at(p, dtype, name)) return rc;
    if (ld < d || ld > ((int64_t)1 << 40)) return fail(WASTE_EINVAL, "row stride of %s %lld: d = %d to 2^40", name, (long long)ld, d);
    return WASTE_OK;
}
Span rows_span(const void *p, int dtype, int64_t ld, int32_t d, int32_t T, const char *name) {
    const size_t size = type_size(dtype);
    return T < 2 ? Span{p, d * size, name} : Span{p, d * size, name, (size_t)T, ld * size};
}
// Whether two spans of rows share a byte.  Rows of one stride may lie between each other's; of unlike strides they
// are taken to meet where their ranges do.
bool rows_meet(const Span &a, const Span &b) {
    if (a.rows == 1) return meet(a, b);
    if (b.rows == 1) return meet(b, a);
    if (!a.p || !b.p) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uintptr_t a1 = a0 + (a.rows - 1) * a.pitch + a.row_bytes, b1 = b0 + (b.rows - 1) * b.pitch + b.row_bytes;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.pitch != b.pitch) return true;
    // b's rows begin `off` behind a's, modulo the pitch
    const size_t off = b0 >= a0 ? (b0 - a0) % a.pitch : (a.pitch - (a0 - b0) % a.pitch) % a.pitch;
    return off < a.row_bytes || off + b.row_bytes > a.pitch;
}
int check_norm_apart(const Span *s, int n, int all) {
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < all; ++j)
            if (s[i].p && s[j].p && rows_meet(s[i], s[j])) return fail(WASTE_EINVAL, "%s overlaps %s", s[i].name, s[j].name);
    return WASTE_OK;
}

// ---- products grouped by expert
int check_group(const waste_group_config *c, int32_t rows, const int32_t *offsets) {
    if (!c) return fail(WASTE_EINVAL, "config is NULL");
    if (int rc = check_abi(c->abi_version)) return rc;
    if (c->n_experts < 1 || c->n_experts > kMaxExperts)
        return fail(WASTE_EINVAL, "n_experts = %d outside [1, %d]", c->n_experts, kMaxExperts);
    if (c->k <= 0 || c->k % 8 || c->n <= 0 || c->n % 8)
        return fail(WASTE_EINVAL, "k = %d and n = %d must be positive multiples of 8", c->k, c->n);
    if ((int64_t)c->k * c->n_experts > kMostRows || (int64_t)c->n * c->n_experts > kMostRows)
        return fail(WASTE_EINVAL, "E = %d, k = %d, n = %d: E k and E n at most 2^30", c->n_experts, c->k, c->n);
    if (!half_type(c->dtype)) return fail(WASTE_EINVAL, "dtype = %d: bf16 or fp16", c->dtype);
    if (rows < 0 || rows > kMostRows) return fail(WASTE_EINVAL, "rows = %d outside [0, 2^30]", rows);
    if (!offsets || !aligned(offsets, 4)) return fail(WASTE_EINVAL, "offsets are NULL or not 4-byte aligned");
    return WASTE_OK;
}

// ---- orthogonalised updates
// The largest |p(s)| for s in [0, most], p(s) = a s + b s^3 + c s^5: at the end or where p' is zero.
double largest(const waste_ortho_config *c, double most) {
    const auto p = [&](double s) { return std::fabs(s * (c->a + s * s * (c->b + s * s * c->c))); };
    double top = p(most);
    const double qa = 5. * c->c, qb = 3. * c->b, qc = c->a, disc = qb * qb - 4. * qa * qc;
    double roots[2] = {-1., -1.}; // of qa t^2 + qb t + qc in t = s^2
    if (qa == 0.) {
        if (qb != 0.) roots[0] = -qc / qb;
    } else if (disc >= 0.) {
        roots[0] = (-qb + std::sqrt(disc)) / (2. * qa);
        roots[1] = (-qb - std::sqrt(disc)) / (2. * qa);
    }
    for (double t : roots)
        if (t > 0. && t < most * most) top = std::fmax(top, p(std::sqrt(t)));
    return top;
}
int check_ortho(const waste_ortho_config *c) {
    if (!c) return fail(WASTE_EINVAL, "config is NULL");
    if (int rc = check_abi(c->abi_version)) return rc;
    if (c->count < 0 || c->count > 65535) return fail(WASTE_EINVAL, "count = %d outside [0, 65535]", c->count);
    if (c->rows < 1 || c->cols < 1 || c->rows > kMostRows || c->cols > kMostRows)
        return fail(WASTE_EINVAL, "rows = %d, cols = %d outside [1, 2^30]", c->rows, c->cols);
    const int m = c->rows < c->cols ? c->rows : c->cols;
    if (m > 1 << 15) return fail(WASTE_EINVAL, "rows = %d, cols = %d: the shorter side at most 2^15", c->rows, c->cols);
    if ((int64_t)c->count * c->rows > kMostRows) return fail(WASTE_EINVAL, "count = %d, rows = %d: %d rows at most", c->count, c->rows, kMostRows);
    if (c->steps < 1 || c->steps > 32) return fail(WASTE_EINVAL, "steps = %d outside [1, 32]", c->steps);
    if (!std::isfinite(c->a) || !std::isfinite(c->b) || !std::isfinite(c->c))
        return fail(WASTE_EINVAL, "coefficients %g, %g, %g", (double)c->a, (double)c->b, (double)c->c);
    // singular values s <= most: A's are s^2, B's b s^2 + c s^4, and their entries no larger; 2^10 times them are fp16
    constexpr double kRange = 62.;
    double most = 1.;
    for (int i = 0; i < c->steps; ++i) {
        const auto q = [&](double t) { return std::fabs(t * (c->b + t * c->c)); };
        const double top = most * most, bend = c->c != 0.f ? -c->b / (2. * c->c) : 0.;
        double b = q(top);
        if (bend > 0. && bend < top) b = std::fmax(b, q(bend));
        if (!(top <= kRange) || !(b <= kRange)) // NaN too
            return fail(WASTE_EINVAL, "coefficients %g, %g, %g leave the range of step %d", (double)c->a, (double)c->b, (double)c->c, i + 1);
        most = std::fmax(1., largest(c, most)); // 1: singular values that stay where they are
    }
    if (!(most <= kRange))
        return fail(WASTE_EINVAL, "coefficients %g, %g, %g leave the range of the last step", (double)c->a, (double)c->b, (double)c->c);
    return WASTE_OK;
}

} // namespace

extern "C" {

int waste_norm_forward(const waste_norm_config *cfg, const void *d_x, int64_t ld_x, int32_t T, const void *d_w,
                       const void *d_b, void *d_y, int64_t ld_y, float *d_mean, float *d_rstd, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_norm(cfg, T);
    if (rc) return rc;
    if (!d_mean != !d_rstd) return fail(WASTE_EINVAL, "mean and rstd: both or neither");
    if (T == 0) return ok();
    const int d = cfg->d;
    if ((rc = check_rows(d_x, cfg->x_dtype, ld_x, d, "x")) || (rc = check_rows(d_y, cfg->y_dtype, ld_y, d, "y"))) return rc;
    if (d_w && (rc = check_at(d_w, cfg->w_dtype, "w"))) return rc;
    if (d_b && (rc = check_at(d_b, cfg->w_dtype, "b"))) return rc;
    if (d_mean && ((rc = check_at(d_mean, 0, "mean")) || (rc = check_at(d_rstd, 0, "rstd")))) return rc;
    const size_t wn = d * type_size(cfg->w_dtype);
    const bool in_place = d_y == d_x && cfg->y_dtype == cfg->x_dtype && (T < 2 || ld_y == ld_x);
    const Span spans[] = {rows_span(d_y, cfg->y_dtype, ld_y, d, T, "y"), {d_mean, (size_t)T * 4, "mean"},
                          {d_rstd, (size_t)T * 4, "rstd"}, {d_w, wn, "w"}, {d_b, wn, "b"},
                          in_place ? Span{nullptr, 0, "x"} : rows_span(d_x, cfg->x_dtype, ld_x, d, T, "x")};
    if ((rc = check_norm_apart(spans, 3, 6))) return rc;
    const NormFwd P{d, T, cfg->x_dtype, cfg->y_dtype, cfg->w_dtype, cfg->eps, d_w, d_b, {const_cast<void *>(d_x), ld_x},
                    {d_y, ld_y}, d_mean, d_rstd};
    return done(launch_norm_forward(P, reinterpret_cast<cudaStream_t>(stream)), "layer norm");
}

int waste_norm_workspace(const waste_norm_config *cfg, int32_t T, size_t *bytes) {
    const int rc = check_norm(cfg, T);
    if (rc) return rc;
    if (!bytes) return fail(WASTE_EINVAL, "bytes is NULL");
    *bytes = norm_bytes(cfg->d, T);
    return ok();
}

int waste_norm_backward(const waste_norm_config *cfg, const void *d_dy, int64_t ld_dy, const void *d_x, int64_t ld_x,
                        int32_t T, const float *d_mean, const float *d_rstd, const void *d_w, void *d_dx, int64_t ld_dx,
                        void *d_dw, void *d_db, int32_t grad_dtype, int32_t accumulate, void *d_workspace,
                        size_t workspace_bytes, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_norm(cfg, T);
    if (rc) return rc;
    const int d = cfg->d;
    if (grad_dtype != cfg->w_dtype && grad_dtype != WASTE_ACT_F32)
        return fail(WASTE_EINVAL, "grad_dtype = %d: the config's w_dtype or fp32", grad_dtype);
    if ((rc = check_flag(accumulate, "accumulate"))) return rc;
    if (!d_dx && !d_dw && !d_db) return ok();
    if (d_dw && (rc = check_at(d_dw, grad_dtype, "dw"))) return rc;
    if (d_db && (rc = check_at(d_db, grad_dtype, "db"))) return rc;
    const size_t gn = d * type_size(grad_dtype);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        if (d_dw && !accumulate) e = cudaMemsetAsync(d_dw, 0, gn, s);
        if (d_db && !accumulate && e == cudaSuccess) e = cudaMemsetAsync(d_db, 0, gn, s);
        return done(e, "clearing the gradients");
    }
    if ((rc = check_rows(d_x, cfg->x_dtype, ld_x, d, "x")) || (rc = check_rows(d_dy, cfg->y_dtype, ld_dy, d, "dy"))) return rc;
    if (d_dx && (rc = check_rows(d_dx, cfg->x_dtype, ld_dx, d, "dx"))) return rc;
    if ((rc = check_at(d_mean, 0, "mean")) || (rc = check_at(d_rstd, 0, "rstd"))) return rc;
    if (d_w && (rc = check_at(d_w, cfg->w_dtype, "w"))) return rc;
    const size_t need = d_dw || d_db ? norm_bytes(d, T) : 0;
    if ((rc = check_workspace(d_workspace, workspace_bytes, need))) return rc;
    const bool in_place = d_dx && d_dx == d_dy && cfg->y_dtype == cfg->x_dtype && (T < 2 || ld_dy == ld_dx);
    const Span spans[] = {d_dx ? rows_span(d_dx, cfg->x_dtype, ld_dx, d, T, "dx") : Span{nullptr, 0, "dx"},
                          {d_dw, gn, "dw"}, {d_db, gn, "db"}, {need ? d_workspace : nullptr, need, "workspace"},
                          rows_span(d_x, cfg->x_dtype, ld_x, d, T, "x"), {d_mean, (size_t)T * 4, "mean"},
                          {d_rstd, (size_t)T * 4, "rstd"}, {d_w, d * type_size(cfg->w_dtype), "w"},
                          rows_span(d_dy, cfg->y_dtype, ld_dy, d, T, "dy")};
    if ((rc = check_norm_apart(spans, 4, 8))) return rc;
    for (int i = in_place ? 1 : 0; i < 4; ++i)
        if (spans[i].p && rows_meet(spans[i], spans[8])) return fail(WASTE_EINVAL, "%s overlaps dy", spans[i].name);
    const NormBwd P{d, T, cfg->x_dtype, cfg->y_dtype, cfg->w_dtype, grad_dtype, accumulate, d_w, {const_cast<void *>(d_x), ld_x},
                    {const_cast<void *>(d_dy), ld_dy}, {d_dx, ld_dx}, d_mean, d_rstd, d_dw, d_db, static_cast<float *>(d_workspace)};
    return done(launch_norm_backward(P, s), "layer norm gradients");
}

int waste_group_forward(const waste_group_config *cfg, const void *d_x, int32_t rows, const int32_t *d_offsets,
                        const void *d_w, void *d_out, int32_t out_dtype, int32_t mode, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_group(cfg, rows, d_offsets);
    if (rc) return rc;
    if (out_dtype != cfg->dtype && out_dtype != WASTE_ACT_F32)
        return fail(WASTE_EINVAL, "out_dtype = %d: the config's dtype or fp32", out_dtype);
    if ((rc = check_flag(mode, "mode"))) return rc;
    if (rows == 0) return ok();
    const void *p[] = {d_x, d_w, d_out};
    const char *n[] = {"x", "w", "out"};
    if ((rc = check_ptrs(p, n, 3))) return rc;
    const int E = cfg->n_experts;
    const Span spans[] = {{d_out, (size_t)rows * cfg->n * type_size(out_dtype), "out"}, {d_x, (size_t)rows * cfg->k * 2, "x"},
                          {d_w, (size_t)E * cfg->n * cfg->k * 2, "w"}, {d_offsets, (size_t)(E + 1) * 4, "offsets"}};
    if ((rc = check_apart(spans, 1, 4))) return rc;
    return done(launch_group_forward({E, cfg->k, cfg->n, cfg->dtype, rows, d_offsets}, d_x, d_w, d_out, out_dtype, mode,
                                     reinterpret_cast<cudaStream_t>(stream)),
                "product grouped by expert");
}

int waste_group_backward(const waste_group_config *cfg, const void *d_dy, const void *d_x, int32_t rows,
                         const int32_t *d_offsets, const void *d_w, void *d_dx, void *d_dw, int32_t grad_dtype,
                         int32_t accumulate, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_group(cfg, rows, d_offsets);
    if (rc) return rc;
    if (grad_dtype != cfg->dtype && grad_dtype != WASTE_ACT_F32)
        return fail(WASTE_EINVAL, "grad_dtype = %d: the config's dtype or fp32", grad_dtype);
    if ((rc = check_flag(accumulate, "accumulate"))) return rc;
    const void *p[] = {d_dy, d_dx, d_w, d_dw, d_x};
    const char *n[] = {"dy", "dx", "w", "dw", "x"};
    const int E = cfg->n_experts;
    const size_t wn = (size_t)E * cfg->n * cfg->k;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (d_dw && (rc = check_ptrs(p + 3, n + 3, rows ? 2 : 1))) return rc;
    if (rows == 0) {
        const bool clear = d_dw && !accumulate;
        return done(clear ? cudaMemsetAsync(d_dw, 0, wn * type_size(grad_dtype), s) : cudaSuccess, "clearing the gradients");
    }
    if (!d_dx && !d_dw) return ok();
    if ((rc = check_ptrs(p, n, d_dx ? 3 : 1))) return rc;
    const Span spans[] = {{d_dx, (size_t)rows * cfg->k * 2, "dx"}, {d_dw, wn * type_size(grad_dtype), "dw"},
                          {d_dy, (size_t)rows * cfg->n * 2, "dy"}, {d_x, (size_t)rows * cfg->k * 2, "x"},
                          {d_w, wn * 2, "w"}, {d_offsets, (size_t)(E + 1) * 4, "offsets"}};
    if ((rc = check_apart(spans, 2, 6))) return rc;
    const Group G{E, cfg->k, cfg->n, cfg->dtype, rows, d_offsets};
    cudaError_t e = d_dx ? launch_group_dx(G, d_dy, d_w, d_dx, s) : cudaSuccess;
    if (e == cudaSuccess && d_dw) e = launch_group_dw(G, d_dy, d_x, d_dw, grad_dtype, accumulate, s);
    return done(e, "gradients grouped by expert");
}

int waste_ortho_workspace(const waste_ortho_config *cfg, size_t *bytes) {
    const int rc = check_ortho(cfg);
    if (rc) return rc;
    if (!bytes) return fail(WASTE_EINVAL, "bytes is NULL");
    *bytes = ortho_parts(cfg->count, cfg->rows, cfg->cols).total;
    return ok();
}

int waste_ortho_update(const waste_ortho_config *cfg, const void *d_g, int32_t g_dtype, void *d_out, int32_t out_dtype,
                       float scale, int32_t mode, void *d_workspace, size_t workspace_bytes, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    int rc = check_ortho(cfg);
    if (rc) return rc;
    if (!any_type(g_dtype)) return fail(WASTE_EINVAL, "g_dtype = %d: fp32, bf16 or fp16", g_dtype);
    if ((rc = check_flag(mode, "mode"))) return rc;
    if (mode ? !any_type(out_dtype) : out_dtype != WASTE_ACT_BF16)
        return fail(WASTE_EINVAL, "out_dtype = %d: bf16, or any type with mode 1", out_dtype);
    if (!std::isfinite(scale)) return fail(WASTE_EINVAL, "scale = %g", (double)scale);
    if (cfg->count == 0) return ok();
    const void *p[] = {d_g, d_out};
    const char *n[] = {"g", "out"};
    if ((rc = check_ptrs(p, n, 2))) return rc;
    const size_t need = ortho_parts(cfg->count, cfg->rows, cfg->cols).total, size = (size_t)cfg->count * cfg->rows * cfg->cols;
    if ((rc = check_workspace(d_workspace, workspace_bytes, need))) return rc;
    const Span spans[] = {{d_out, size * type_size(out_dtype), "out"}, {d_workspace, need, "workspace"},
                          {d_g, size * type_size(g_dtype), "g"}};
    if ((rc = check_apart(spans, 2, 3))) return rc;
    const Ortho P{cfg->count, cfg->rows, cfg->cols, cfg->steps, cfg->a, cfg->b, cfg->c, d_g, g_dtype, d_out, out_dtype, mode, scale,
                  static_cast<uint8_t *>(d_workspace)};
    return done(launch_ortho(P, reinterpret_cast<cudaStream_t>(stream)), "orthogonalised update");
}

int waste_train_debug_wait(int32_t unit, int32_t polls, int32_t arrive, waste_stream_t stream) {
    const NvtxRange nvtx_range(__func__);
    if (unit < 0 || unit > 2) return fail(WASTE_EINVAL, "unit = %d outside [0, 2]", unit);
    if (polls < 0 || polls > tc::kWaitPolls) return fail(WASTE_EINVAL, "polls = %d outside [0, 2^18]", polls);
    if (int rc = check_flag(arrive, "arrive")) return rc;
    uint32_t *word = nullptr;
    cudaError_t e = unit == 0 ? norm_word(&word) : unit == 1 ? group_word(&word) : ortho_word(&word);
    if (e == cudaSuccess)
        e = train::launch_debug_wait(word, unit == 0, polls ? polls : tc::kWaitPolls, arrive, reinterpret_cast<cudaStream_t>(stream));
    return done(e, "wait kernel");
}

} // extern "C"
