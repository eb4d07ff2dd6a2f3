/*
 * waste_train.h -- C ABI of the operators that train the layer around the routed RVQ experts of
 * waste_moe.h on NVIDIA GB300 (sm_103a), before its matrices are encoded: the layer norm in front of router
 * and experts with its gradients, products grouped by expert with theirs, and updates made orthogonal by
 * Newton-Schulz products.
 *
 * Conventions: those of waste_dense.h (device pointers of the current device; calls enqueue on a stream,
 * allocate nothing and may be captured; arguments are checked on the host before anything is launched; what a
 * call writes overlaps nothing else of it unless the call says so; a workspace holds nothing between calls
 * and serves one call at a time; the same inputs give the same bits; sizes up to 2^30).  dtype arguments are
 * WASTE_ACT_F32, WASTE_ACT_BF16 and WASTE_ACT_F16.  waste_dense_status reports these operators' device waits too.
 */
#ifndef WASTE_TRAIN_H
#define WASTE_TRAIN_H

#include "waste_dense.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Test aid, as waste_dense_debug_wait: the wait is latched as one of the layer norm's (unit 0), of the products grouped by
 * expert (1) or of the orthogonalised updates (2). */
int waste_train_debug_wait(int32_t unit, int32_t polls, int32_t arrive, waste_stream_t stream);

/* ---- layer norm -------------------------------------------------------------------------
 * Over each row of d >= 1 values: mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
 *   y = (x - mu) r w + b
 * and, with xh = (x - mu) r and g = dy w,
 *   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum over rows of dy xh,  db = sum over rows of dy.
 * Statistics and sums are fp32; y, dx, dw and db are rounded once.  So a row's sum and its sum of squares about the
 * mean have to lie in fp32's range: where the squares leave it (distances of 1.8e19 / sqrt(d) and more) r is 0 and y is b.
 * Rows are contiguous, ld elements apart (ld >= d), pointers aligned to their type: 16-byte aligned rows of d % 8 == 0
 * values take the quick way. */
typedef struct {
    uint32_t abi_version; /* must equal WASTE_MOE_ABI_VERSION */
    int32_t d;
    int32_t x_dtype; /* of x and dx */
    int32_t y_dtype; /* of y and dy */
    int32_t w_dtype; /* of w and b */
    float eps;       /* finite, >= 0 */
} waste_norm_config;

/* y [T][d].  d_w or d_b NULL: ones, zeros.  d_mean, d_rstd [T] fp32: receive mu and r for the gradients, or
 * both NULL.  y may be x itself (same address, type and ld); rows of unlike strides may not lie in one range.
 * T >= 0; T == 0 does nothing.  A row with an infinity or a NaN becomes NaN, other rows are not touched by it. */
int waste_norm_forward(const waste_norm_config *cfg, const void *d_x, int64_t ld_x, int32_t T, const void *d_w,
                       const void *d_b, void *d_y, int64_t ld_y, float *d_mean, float *d_rstd, waste_stream_t stream);

/* Bytes of workspace of a backward call of T tokens that asks for dw or db (no less for fewer tokens).  Host
 * arithmetic only; it does not pass 2432 d bytes (and a rounding up to 256), whatever T is. */
int waste_norm_workspace(const waste_norm_config *cfg, int32_t T, size_t *bytes);

/* Gradients for dy [T][d] of a forward call with this x that kept mean and rstd.  d_w NULL: ones.
 *   d_dx  [T][d] or NULL: not computed; may be dy itself (same address, type and ld)
 *   d_dw, d_db  [d] of grad_dtype (fp32 or w_dtype), or NULL: not computed
 *   accumulate 0: dw and db are written; 1: added to what is there (one rounding)
 * T == 0: dw and db become zero with accumulate 0.  No workspace is needed where dw and db are NULL. */
int waste_norm_backward(const waste_norm_config *cfg, const void *d_dy, int64_t ld_dy, const void *d_x, int64_t ld_x,
                        int32_t T, const float *d_mean, const float *d_rstd, const void *d_w, void *d_dx, int64_t ld_dx,
                        void *d_dw, void *d_db, int32_t grad_dtype, int32_t accumulate, void *d_workspace,
                        size_t workspace_bytes, waste_stream_t stream);

/* ---- products grouped by expert ------------------------------------------------------------
 * W [E][n][k]; the rows of x [rows][k] are sorted by expert: expert e has rows offsets[e] .. offsets[e + 1] - 1.
 *   y_r = x_r W_e^T,   dx_r = dy_r W_e,   dW_e = sum over e's rows of dy_r^T x_r
 * offsets [E + 1] int32 stand on the device and are not read by the host: they do not fall and lie in
 * 0 .. rows.  Where they do not, nothing outside the buffers is touched, outputs are undefined and
 * waste_dense_status reports WASTE_EINVAL.  Rows before offsets[0] and from offsets[E] on belong to no
 * expert: y and dx there are left as they were.  k and n positive multiples of 8, 1 <= E <= 4096,
 * rows, E n and E k at most 2^30; x, W, y, dy, dx of dtype (bf16 or fp16), sums in fp32. */
typedef struct {
    uint32_t abi_version; /* must equal WASTE_MOE_ABI_VERSION */
    int32_t n_experts;    /* E */
    int32_t k;            /* columns of x */
    int32_t n;            /* columns of y */
    int32_t dtype;        /* WASTE_ACT_BF16 or WASTE_ACT_F16 */
} waste_group_config;

/* y [rows][n] of out_dtype (cfg->dtype or WASTE_ACT_F32); mode 0: out = y, mode 1: out += y (one rounding). */
int waste_group_forward(const waste_group_config *cfg, const void *d_x, int32_t rows, const int32_t *d_offsets,
                        const void *d_w, void *d_out, int32_t out_dtype, int32_t mode, waste_stream_t stream);

/* Gradients for dy [rows][n].
 *   d_dx  [rows][k] of cfg->dtype, or NULL: not computed (then d_w may be NULL)
 *   d_dw  [E][n][k] of grad_dtype (cfg->dtype or WASTE_ACT_F32), or NULL: not computed (then d_x may be NULL)
 *   accumulate 0: dW is written (zeros for an expert without rows); 1: added to what is there (one rounding) */
int waste_group_backward(const waste_group_config *cfg, const void *d_dy, const void *d_x, int32_t rows,
                         const int32_t *d_offsets, const void *d_w, void *d_dx, void *d_dw, int32_t grad_dtype,
                         int32_t accumulate, waste_stream_t stream);

/* ---- orthogonalised updates (Newton-Schulz) ------------------------------------------------
 * For each of `count` matrices G [rows][cols], with the short side first (transposed where rows > cols):
 *   X = G / |G|_F;  `steps` times  X <- a X + (b A + c A^2) X,  A = X X^T
 * which moves every singular value of G towards 1 and keeps its singular vectors.  A zero matrix gives
 * zeros; one with an infinity or a NaN gives NaN throughout, the others are not touched by it.
 * Products take fp16 operands scaled by 2^10 and sum in fp32; X is held in two fp16 parts (22 bits) and the
 * diagonal of b A + c A^2 in fp32.  Five steps of 3.4445, -4.7750, 2.0315 are off the exact result by 1e-3 of its norm
 * or so, below bf16's rounding of it, for full and for low rank; eight by 2e-3, and what converges by less.  A step
 * multiplies by a what rounding leaves outside the space of a G of low rank, in any arithmetic: with a^steps past
 * 1e5 (ten steps of 3.4445; fp32 products are no better) the result for such a G is not near the exact one. */
typedef struct {
    uint32_t abi_version; /* must equal WASTE_MOE_ABI_VERSION */
    int32_t count;        /* matrices, >= 0 */
    int32_t rows, cols;   /* >= 1; the shorter of them at most 2^15 */
    int32_t steps;        /* 1 .. 32 */
    /* checked: for singular values s from [0, 1] on, s^2 and |b s^2 + c s^4| stay within 62 over the steps (fp16's
     * range, scaled): 3.4445, -4.7750, 2.0315 and what converges do */
    float a, b, c;
} waste_ortho_config;

int waste_ortho_workspace(const waste_ortho_config *cfg, size_t *bytes);

/* out [count][rows][cols] of out_dtype from d_g of g_dtype:
 *   mode 0: out = scale X (out_dtype WASTE_ACT_BF16);
 *   mode 1: out += scale X (any type, one rounding: a weight and its update).  fp32 weights too receive X as it is held:
 *           off by 1e-3 of the update's norm or so, not by fp32's rounding
 * out may not be G. */
int waste_ortho_update(const waste_ortho_config *cfg, const void *d_g, int32_t g_dtype, void *d_out, int32_t out_dtype,
                       float scale, int32_t mode, void *d_workspace, size_t workspace_bytes, waste_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* WASTE_TRAIN_H */
