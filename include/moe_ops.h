/*
 * moe_ops.h -- C ABI of the operators around the single-GPU MoE layer of
 * moe.h: the RMS norm in front of it (with the residual's addition and an
 * 8-bit output), expert blocks in MXFP8, and the backward passes of the norm,
 * of the grouped SwiGLU experts and of the combine.
 *
 * The conventions of moe.h hold: caller-owned 16-byte aligned device buffers,
 * contiguous row-major matrices, no allocation, no copy to the host and no
 * synchronisation (every call may be captured in a HIP graph), arguments
 * checked on the host before anything is enqueued, the same status codes, and
 * bitwise repeatable results (no atomics).  All pointers belong to the device
 * that is current at the call, and `stream` to that device.  A workspace
 * holds nothing between calls: it need not be initialised, calls that share
 * one must be ordered, and one sized for max_rows (or T) rows serves every
 * call with fewer.  Outputs must not overlap inputs or one another
 * except where a call says so.  Rows past the last expert's row are not
 * touched in any output.
 *
 * Types: MOE_F32 and MOE_BF16 rows; sums, statistics and gradients of
 * parameters that are sums over rows accumulate in float32 or more (of MXFP8
 * products see below), and every output is rounded once, to nearest even
 * (bfloat16 and 8-bit results below 2^-126 after the step of a float32 there,
 * 2^-149).  A non-finite input makes the outputs that depend on it non-finite
 * or undefined, and no others.
 *
 * MXFP8 is the OCP microscaling format that gfx950's matrix instructions read
 * directly: e4m3 elements (torch.float8_e4m3fn), and for every 32 consecutive
 * elements of a row one scale byte b that stands for 2^(b - 127) (E8M0).  A
 * row of K elements (a multiple of 32) has MOE_MX_PITCH(K) scale bytes: the
 * K / 32 scales, then zeros up to a multiple of 4.  The scale the library
 * writes is the smallest 2^e, e >= -127, with max|v| / 2^e <= 448, so no
 * element saturates.
 */
#ifndef MOE_OPS_MI355X_H
#define MOE_OPS_MI355X_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scale bytes of an MXFP8 row of K elements. */
#define MOE_MX_PITCH(K) (((K) + 127) / 128 * 4)
/* Added to dt = MOE_BF16: the gate and up projections that a training block
 * saves take 16 bits each, not a float32. */
#define MOE_GU_16 0x100

/*
 * moe_rmsnorm -- the norm between the residual stream and the layer.
 *
 *   s[t]    = x[t] + residual[t], added in float32 and rounded to dt (the new
 *             residual stream); s = x when residual == NULL
 *   rstd[t] = 1 / sqrt(mean_h(s[t][h]^2) + eps)
 *   y[t][h] = s[t][h] * rstd[t] * weight[h]
 *
 *   x, residual, sum, y: [T][H] dtype dt; weight[H] dtype dt; rstd[T] float32.
 *   y8[T][H] and y8_scale[T][MOE_MX_PITCH(H)]: MXFP8 of y before y's own
 *   rounding (for moe_grouped_ffn_mxfp8; the router takes y).  sum, y, y8 with
 *   y8_scale, and rstd may each be NULL, but not all of them.  sum and y may be
 *   x or residual themselves (and not each other).  eps >= 0 and finite; with
 *   eps = 0 a row of zeros has no norm and gives NaN.  H a multiple of 32, at
 *   most 16384, and T * min(64 * ceil(H / 512), 1024) below 2^32, the threads of
 *   a launch with a block per row (more rows: MOE_ERR_UNSUPPORTED).
 */
int moe_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int T, int H,
                int dt, void* sum, void* y, void* y8, uint8_t* y8_scale, float* rstd, void* stream);

/*
 * moe_rmsnorm_backward -- gradients of moe_rmsnorm.
 *   With xh = s * rstd and g = dy * weight:
 *   dx[t]      = rstd * (g - xh * mean_h(g * xh)) + dsum[t]
 *   dweight[h] = sum_t dy[t][h] * xh[t][h]                     (float32)
 *
 *   s: the summed rows the norm was taken of (sum, or x without a residual);
 *   rstd as moe_rmsnorm wrote it.  dsum (may be NULL): the gradient arriving at
 *   `sum` from its other uses.  dx is the gradient of x and of residual alike;
 *   it may be dy, s or dsum itself.  dy, dsum, s, dx: [T][H] dtype dt.  xh, g and
 *   their products are float32, and must not leave its range.
 *   T = 0 writes dweight = 0.  ws: moe_rmsnorm_backward_workspace_size bytes.
 */
size_t moe_rmsnorm_backward_workspace_size(int T, int H, int dt);
int moe_rmsnorm_backward(const void* dy, const void* dsum, const void* s, const void* weight,
                         const float* rstd, int T, int H, int dt, void* dx, float* dweight,
                         void* ws, size_t ws_bytes, void* stream);

/*
 * moe_combine_backward -- gradients of moe_combine.
 *   For every (t, j) with row = dst_row[t][j] >= 0:
 *     dy_perm[row] = topk_w[t][j] * dy[t]                      (dtype y_perm_dt)
 *     dtopk_w[t][j] = sum_h dy[t][h] * y_perm[row][h]          (float32)
 *   and dtopk_w[t][j] = 0 where dst_row[t][j] < 0.  The gradient of y_shared
 *   is dy itself.  dst_row names rows of y_perm and dy_perm (what it
 *   holds is not checked), every row at most once, as moe_permute writes it;
 *   rows it does not name keep what dy_perm held (so in a padded layout,
 *   whose blank rows moe_grouped_ffn_backward reads as well, clear dy_perm
 *   first).  dy_perm may be y_perm itself, where no row of it is blank.
 *   Limits of moe_combine, and H and T as for moe_rmsnorm.
 */
int moe_combine_backward(const void* dy, int dt, const void* y_perm, int y_perm_dt,
                         const int32_t* dst_row, const float* topk_w, int T, int k, int H,
                         void* dy_perm, float* dtopk_w, void* stream);

/*
 * moe_grouped_ffn_train / moe_grouped_ffn_backward -- moe_grouped_ffn with
 * what its backward pass needs, and that pass.
 *   For expert i and every row r in [offsets[i], offsets[i+1]), with
 *   a = x_perm[r], or x[src_token[r]] when x_perm == NULL:
 *     forward   g = W_gate a, u = W_up a, h = SiLU(g) * u, y_perm[r] = W2 h,
 *               gu[r] = [g | u]  ([max_rows][2*I_loc])
 *     backward  dh = W2^T dy_perm[r]
 *               dg = dh * u * SiLU'(g), du = dh * SiLU(g),
 *               SiLU'(g) = s (1 + g (1 - s)), s = 1 / (1 + exp(-g))
 *               dx_perm[r] = W_gate^T dg + W_up^T du
 *               dw13[i] = sum_r [dg | du] a^T,  dw2[i] = sum_r dy_perm[r] h^T
 *   gu is float32 and holds g and u unrounded; or, with dt = MOE_BF16 |
 *   MOE_GU_16 in both calls, it has 16 bits per value and half the memory (the
 *   Python binding goes by gu's type: a bfloat16 tensor is taken as such
 *   storage).  What the 16-bit form holds is for these two calls alone, and no
 *   bfloat16 numbers: four consecutive columns, from a multiple of 4 on, share
 *   an exponent, and each value is off by at most 2^-11 of itself plus 2^-17 of
 *   the largest of its four.  A value that is not finite makes the other three
 *   undefined.
 *   The backward pass reads g and u from gu and forms h anew.  h, dg and du are
 *   rounded to dt before the products that read them, as h is in the forward
 *   pass, so a gradient passes one such rounding between its two products, as
 *   the output does (bfloat16, against float64, in 2-norm: y_perm and the
 *   gradients 2.35e-3 with a float32 gu, the gradients 2.37e-3 with 16 bits).
 *
 *   dy_perm, dx_perm, y_perm: [max_rows][H]; dw13, dw2: shapes of w13, w2; all
 *   dtype dt.  dx_perm may be NULL, and dw13 and dw2 together may be NULL (not
 *   all three).  An expert without rows gets zero gradients; max_rows = 0
 *   writes them for every expert.  The gradient of token t's row in the
 *   gathered form is the sum of its copies' dx_perm rows: moe_combine with
 *   weights 1.  Shape limits of moe_grouped_ffn; H and I_loc at most
 *   65536, H * I_loc and max_rows at most 2^30 (in bfloat16 H * I_loc below
 *   2^30), and shapes that a launch of fewer than 2^32 threads does not cover
 *   are MOE_ERR_UNSUPPORTED: in float32 from 1.7e10 elements of dx_perm, dw13
 *   and dw2 together, in bfloat16 from 2^28 rows or 2.7e11 elements.
 *   An expert whose offsets leave [0, max_rows] or decrease is treated as one
 *   without rows; the others' ranges must not overlap.  With src_token, every source must be a row of x; a source of
 *   -1 reads row 0.  For the padded layout of moe_permute_capacity pass its
 *   x_perm to both, and rows of zeros in dy_perm for its blank rows: they then
 *   add nothing to any gradient.
 */
size_t moe_grouped_ffn_train_workspace_size(int max_rows, int E_loc, int H, int I_loc, int dt);
int moe_grouped_ffn_train(const void* x_perm, const void* x, const int32_t* src_token,
                          const int32_t* offsets, int E_loc, int max_rows, int H, int I_loc,
                          const void* w13, const void* w2, int dt, void* gu, void* y_perm,
                          void* ws, size_t ws_bytes, void* stream);
size_t moe_grouped_ffn_backward_workspace_size(int max_rows, int E_loc, int H, int I_loc, int dt);
int moe_grouped_ffn_backward(const void* dy_perm, const void* x_perm, const void* x,
                             const int32_t* src_token, const int32_t* offsets, int E_loc,
                             int max_rows, int H, int I_loc, const void* w13, const void* w2,
                             int dt, const void* gu, void* dx_perm, void* dw13, void* dw2,
                             void* ws, size_t ws_bytes, void* stream);

/*
 * moe_grouped_ffn_mxfp8 -- moe_grouped_ffn on MXFP8 rows and weights.
 *   g, u, y are products of the values the elements and scales stand for; h =
 *   SiLU(g) * u is brought to MXFP8 (blocks of 32 along I_loc) between the two
 *   products.  The 8-bit matrix instructions add blocks of 64 or 128 products
 *   with about 16 significant bits, and the blocks in float32, so an h next to
 *   an e4m3 border (one in some 2000) may round to its other neighbour: 2.0e-3
 *   from the formula in 2-norm where exact sums leave 1.7e-3.  With few rows g
 *   and u are summed in float32 throughout, so a row's last bits may differ with
 *   the batch that it is in.
 *
 *   x8[*][H] with x_scale[*][MOE_MX_PITCH(H)], rows gathered by src_token, or
 *   row r itself when src_token == NULL;
 *   w13[E_loc][2*I_loc][H] with w13_scale[E_loc][2*I_loc][MOE_MX_PITCH(H)];
 *   w2[E_loc][H][I_loc] with w2_scale[E_loc][H][MOE_MX_PITCH(I_loc)];
 *   y_perm[max_rows][H] of dtype y_dt.  Elements must be finite, scale bytes
 *   below 255 and the values they stand for below 2^127; those below 2^-126 may
 *   count as zero.  Limits (H * I_loc at
 *   most 2^30), offsets and sources as for moe_grouped_ffn_train (a source of -1 gives a meaningless row, which
 *   moe_combine does not read).
 */
size_t moe_grouped_ffn_mxfp8_workspace_size(int max_rows, int E_loc, int H, int I_loc);
int moe_grouped_ffn_mxfp8(const void* x8, const uint8_t* x_scale, const int32_t* src_token,
                          const int32_t* offsets, int E_loc, int max_rows, int H, int I_loc,
                          const void* w13, const uint8_t* w13_scale, const void* w2,
                          const uint8_t* w2_scale, void* y_perm, int y_dt, void* ws,
                          size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_OPS_MI355X_H */
