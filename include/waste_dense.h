/*
 * waste_dense.h -- C ABI of the dense operators that stand beside the routed RVQ experts of
 * waste_moe.h on NVIDIA GB300 (sm_103a): the gated feed-forward block of a dense (always-on)
 * expert with its gradients, and microscaled 4-bit matrices (MXFP4) with their product.
 *
 * The block is the same one the routed experts compute from their codes (waste_moe_forward):
 *   g = x Wg^T,  u = x Wu^T            [T][f]
 *   a = silu(g) * u,  silu(z) = z / (1 + exp(-z))
 *   y = a Wd^T                         [T][d]
 * with Wg, Wu [f][d] and Wd [d][f] row-major, and its gradients
 *   da = dy Wd,  du = da silu(g),  dg = da u s (1 + g (1 - s)),  s = 1 / (1 + exp(-g))
 *   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T a.
 *
 * Conventions (those of waste_moe.h): d_* are device pointers of the current device, owned by
 * the caller; calls that take a stream enqueue on it and return, allocate nothing and may be
 * captured into a CUDA graph; arguments are checked on the host before anything is launched;
 * the return value is WASTE_OK or a negative waste_status whose message is
 * waste_moe_last_error().  Matrices are row-major without padding unless a row stride is an
 * argument, and no size is past 2^30.  Pointers are 16-byte aligned, workspaces 256-byte aligned.
 * A workspace holds nothing between calls; two calls that may run at the same time (two streams, two
 * captured graphs), or are made at the same time by two host threads, need one each.  What a call
 * writes (its workspace too) overlaps nothing else of the call, unless the call says so: WASTE_EINVAL
 * where it does.  The same inputs give the same bits: no sum depends on the order in which blocks run.
 */
#ifndef WASTE_DENSE_H
#define WASTE_DENSE_H

#include "waste_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { WASTE_ACT_F16 = 2 }; /* beside WASTE_ACT_F32 and WASTE_ACT_BF16 */

/* Synchronises the device; WASTE_ETIMEOUT if a bounded device wait of one of these operators
 * gave up on the current device since the last call of this (outputs since then are not to be
 * used, and the context is to be treated as unusable, as after waste_moe_stats), else WASTE_OK. */
int waste_dense_status(void);

/* Test aid for that report: one CTA on `stream` waits, by the operators' own wait, on a barrier that
 * nobody else arrives at, and latches the timeout if the wait gives up.  polls: 1 .. 2^18 polls of up to 4 us
 * before it does, or 0: the operators' limit (2^18: 1.1 s).  arrive 1: the wait is over when it begins, and
 * nothing is latched.  The context stays usable; the library never calls it. */
int waste_dense_debug_wait(int32_t polls, int32_t arrive, waste_stream_t stream);

/* ---- gated feed-forward block ---------------------------------------------------------
 * d % 8 == 0, f % 8 == 0, both positive; dtype WASTE_ACT_BF16 or WASTE_ACT_F16: the type of x,
 * the weights, g, u, dy and dx.  Sums are held in fp32; a, dg and du are rounded once to dtype
 * on their way into the next product.  Calls of at most 32 tokens keep what that rounding leaves as
 * well, rounded to dtype too: a value v is then off by at most 2^-16 |v| in bf16, and in fp16, whose
 * rests become subnormal for |v| < 2^-3, by the larger of 2^-22 |v| and 2^-25; an infinite x, weight or dy
 * may then give NaN where one product would give an infinity.  (A forward of one token keeps a in fp32.) */
typedef struct {
    uint32_t abi_version; /* must equal WASTE_MOE_ABI_VERSION */
    int32_t d;            /* hidden size */
    int32_t f;            /* width of the block */
    int32_t dtype;        /* WASTE_ACT_BF16 or WASTE_ACT_F16 */
} waste_ffn_config;

/* Bytes of workspace that a forward (backward = 0) or backward (1) call of T tokens needs.
 * Host arithmetic only. */
int waste_ffn_workspace(const waste_ffn_config *cfg, int32_t T, int32_t backward, size_t *bytes);

/* y into d_out [T][d] of type out_dtype (cfg->dtype or WASTE_ACT_F32).
 *   mode 0: out = y;  mode 1: out += y (the sum is rounded once to out_dtype)
 *   d_g, d_u  [T][f] of cfg->dtype: receive g and u for waste_ffn_backward, or both NULL
 * d_out may overlap d_x (x is read before anything is written there).
 * T >= 0; T == 0 does nothing. */
int waste_ffn_forward(const waste_ffn_config *cfg, const void *d_x, int32_t T, const void *d_w_gate,
                      const void *d_w_up, const void *d_w_down, void *d_out, int32_t out_dtype, int32_t mode,
                      void *d_g, void *d_u, void *d_workspace, size_t workspace_bytes, waste_stream_t stream);

/* Gradients of a forward call with the same x and weights that kept g and u.
 *   d_dx [T][d] of cfg->dtype, or NULL: not computed
 *   d_dw_gate, d_dw_up [f][d], d_dw_down [d][f] of type grad_dtype (cfg->dtype or
 *   WASTE_ACT_F32), or all three NULL: not computed
 *   accumulate 0: the weights' gradients are written; 1: added to what is there (one rounding
 *   to grad_dtype).  dx is always written.
 * T == 0: dx is untouched; with accumulate 0 the weights' gradients become zero. */
int waste_ffn_backward(const waste_ffn_config *cfg, const void *d_dy, int32_t T, const void *d_x, const void *d_g,
                       const void *d_u, const void *d_w_gate, const void *d_w_up, const void *d_w_down, void *d_dx,
                       void *d_dw_gate, void *d_dw_up, void *d_dw_down, int32_t grad_dtype, int32_t accumulate,
                       void *d_workspace, size_t workspace_bytes, waste_stream_t stream);

/* ---- microscaled 4-bit matrices (MXFP4) -------------------------------------------------
 * The OCP Microscaling format with E2M1 elements: blocks of 32 consecutive columns of a row
 * share a power of two.  rows >= 0, cols positive with cols % 32 == 0.
 *   codes  [rows][cols / 2] bytes: two E2M1 codes a byte, the even column in the low half;
 *          code = sign << 3 | n, n = 0..7 for 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   scales E8M0 bytes s (the power of two is 2^(s - 127); 255 = NaN: every value of the block
 *          is NaN) in tiles of 128 rows x 4 blocks, the order in which the tensor core takes
 *          them: with kb = ceil(cols / 128), the byte of row r and block k is at
 *          ((r / 128) * kb + k / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + k % 4.
 *          The bytes of rows and blocks past the end are zero (waste_mx4_quantize writes them);
 *          other values there may turn results of the last blocks into NaN. */
int waste_mx4_layout(int32_t rows, int32_t cols, size_t *code_bytes, size_t *scale_bytes);

/* Quantise d_x [rows][cols] (dtype WASTE_ACT_F32, _BF16 or _F16; consecutive rows ld >= cols
 * elements apart, ld a multiple of 16 bytes): per block with largest magnitude m the exponent
 * is e = max(-127, floor(log2 m) - 2) (m = 0: -127), codes are v 2^-e rounded to the nearest
 * E2M1 value, ties to the even code, magnitudes past 6 to 6; the sign of a zero is kept.  A
 * block that holds an infinity or a NaN gets scale 255 and codes 0. */
int waste_mx4_quantize(const void *d_x, int32_t dtype, int32_t rows, int32_t cols, int64_t ld, uint8_t *d_codes,
                       uint8_t *d_scales, waste_stream_t stream);

/* The values that codes and scales stand for, rounded to dtype, rows ld elements apart (what
 * lies between the rows is left as it was). */
int waste_mx4_dequantize(const uint8_t *d_codes, const uint8_t *d_scales, int32_t rows, int32_t cols, void *d_out,
                         int32_t dtype, int64_t ld, waste_stream_t stream);

/* C = A B^T of MXFP4 matrices A [M][K] and B [N][K], summed in fp32, into d_out [M][N] of type
 * out_dtype (WASTE_ACT_F32, _BF16 or _F16); mode 0: out = C, mode 1: out += C (one rounding).
 * M >= 0, N >= 1; M == 0 does nothing.  A and B may be the same matrix. */
int waste_mx4_matmul(int32_t M, int32_t N, int32_t K, const uint8_t *d_a_codes, const uint8_t *d_a_scales,
                     const uint8_t *d_b_codes, const uint8_t *d_b_scales, void *d_out, int32_t out_dtype,
                     int32_t mode, waste_stream_t stream);

/* The gated feed-forward block with MXFP4 weights: x is quantised as by waste_mx4_quantize, g
 * and u are fp32 sums, a = silu(g) * u in fp32 is quantised by the same rules, y = a Wd^T.
 * d % 32 == 0, f % 32 == 0; x [T][d] of type x_dtype (WASTE_ACT_F32, _BF16 or _F16); out [T][d]
 * and mode as in waste_mx4_matmul; d_out may overlap d_x. */
typedef struct {
    uint32_t abi_version; /* must equal WASTE_MOE_ABI_VERSION */
    int32_t d;
    int32_t f;
    const uint8_t *d_gate_codes, *d_gate_scales; /* Wg [f][d] */
    const uint8_t *d_up_codes, *d_up_scales;     /* Wu [f][d] */
    const uint8_t *d_down_codes, *d_down_scales; /* Wd [d][f] */
} waste_mx4_ffn_config;

int waste_mx4_ffn_workspace(const waste_mx4_ffn_config *cfg, int32_t T, size_t *bytes);
int waste_mx4_ffn_forward(const waste_mx4_ffn_config *cfg, const void *d_x, int32_t x_dtype, int32_t T, void *d_out,
                          int32_t out_dtype, int32_t mode, void *d_workspace, size_t workspace_bytes,
                          waste_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* WASTE_DENSE_H */
