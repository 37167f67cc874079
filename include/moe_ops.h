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
 * holds nothing between calls: it need not be initialised, and calls that
 * share one must be ordered.  Outputs must not overlap inputs or one another
 * except where a call says so.  Rows past the last expert's row are not
 * touched in any output.
 *
 * Types: MOE_F32 and MOE_BF16 rows; sums, statistics and gradients of
 * parameters that are sums over rows accumulate in float32, and every output
 * is rounded once, to nearest even.  A non-finite input makes the outputs that
 * depend on it non-finite or undefined, and no others.
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
 *   y8_scale, and rstd may each be NULL, but not all of them.  sum may be x or
 *   residual itself.  eps >= 0 and finite.  H a multiple of 32, at most 16384.
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
 *   it may be dy, s or dsum itself.  dy, dsum, s, dx: [T][H] dtype dt.
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
 *   is dy itself.  dst_row names every row at most once, as moe_permute writes
 *   it; rows it does not name keep what dy_perm held.  dy_perm may be y_perm
 *   itself.  Limits of moe_combine, and H at most 16384.
 */
int moe_combine_backward(const void* dy, int dt, const void* y_perm, int y_perm_dt,
                         const int32_t* dst_row, const float* topk_w, int T, int k, int H,
                         void* dy_perm, float* dtopk_w, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_OPS_MI355X_H */
