// C ABI entry points of the operators around the layer: argument checks,
// workspace layout and kernel sequencing.  Declarations and the full contract
// are in include/moe_ops.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <climits>
#include <cmath>

#include "moe_ops.h"
#include "moe_host.h"
#include "moe_kernels.h"
#include "moe_ops_kernels.h"

using namespace moe;

namespace {

template <typename... P>
bool any_misaligned(const P*... p) {
  return !(... && aligned16(p));   // a null pointer counts as aligned
}

int check_row_width(int H) {
  const int st = check_hidden(H);
  if (st) return st;
  return H > OPS_MAX_H ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
// A block per row: a launch holds fewer than 2^32 threads.
bool rows_fit(int T, int H) { return (long long)T * row_threads(H) < (1ll << 32); }

// Shapes of an expert block beside the layer's own.
int check_block(int max_rows, int E_loc, int H, int I_loc) {
  if (E_loc < 1 || max_rows < 0 || I_loc <= 0) return MOE_ERR_INVALID_ARG;
  const int st = check_hidden(H);
  if (st) return st;
  if (I_loc % 32 || E_loc > 1024 || H > OPS_MAX_DIM || I_loc > OPS_MAX_DIM ||
      (long long)H * I_loc > OPS_MAX_HI || max_rows > OPS_MAX_ROWS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
// The rows' type of a training block's dt, which may say that gu has 16 bits per value.
int rows_dt(int dt) { return dt == (MOE_BF16 | MOE_GU_16) ? MOE_BF16 : dt; }
int check_train(int max_rows, int E_loc, int H, int I_loc, int dt) {
  if (!valid_dt(dt)) return MOE_ERR_INVALID_ARG;
  const int st = check_block(max_rows, E_loc, H, I_loc);
  if (st) return st;
  // an expert's W13 within the 2^32 - 1 bytes that a buffer descriptor can span
  if (dt == MOE_BF16 && (long long)H * I_loc >= OPS_MAX_HI) return MOE_ERR_UNSUPPORTED;
  return train_fits(max_rows, E_loc, H, I_loc, dt) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
int check_mx(int max_rows, int E_loc, int H, int I_loc) {
  const int st = check_block(max_rows, E_loc, H, I_loc);
  if (st) return st;
  return mx_fits(max_rows, E_loc, H, I_loc) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int moe_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int T, int H,
                int dt, void* sum, void* y, void* y8, uint8_t* y8_scale, float* rstd,
                void* stream) {
  if (!valid_dt(dt) || T < 0 || !(eps >= 0.f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
  const int st = check_row_width(H);
  if (st) return st;
  if (!rows_fit(T, H)) return MOE_ERR_UNSUPPORTED;
  if (!y8 != !y8_scale) return MOE_ERR_INVALID_ARG;
  if (!sum && !y && !y8 && !rstd) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(x, residual, weight, sum, y, y8, y8_scale, rstd)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !weight) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_rmsnorm(x, residual, weight, eps, T, H, dt, sum, y, y8, y8_scale, rstd,
                                   static_cast<hipStream_t>(stream)));
}

size_t moe_rmsnorm_backward_workspace_size(int T, int H, int dt) {
  if (T < 0 || !valid_dt(dt) || check_row_width(H) != MOE_OK) return 0;
  return align_up((size_t)(T > 0 ? rmsnorm_bwd_blocks(T) : 1) * H * 4);
}

int moe_rmsnorm_backward(const void* dy, const void* dsum, const void* s, const void* weight,
                         const float* rstd, int T, int H, int dt, void* dx, float* dweight,
                         void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dt(dt) || T < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_row_width(H);
  if (st) return st;
  if (!dweight || (T > 0 && (!dy || !s || !weight || !rstd || !dx))) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(dy, dsum, s, weight, rstd, dx, dweight, ws)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ws || ws_bytes < moe_rmsnorm_backward_workspace_size(T, H, dt)))
    return MOE_ERR_WORKSPACE;
  return hip_status(launch_rmsnorm_bwd(dy, dsum, s, weight, rstd, T, H, dt, dx, dweight,
                                       static_cast<float*>(ws), static_cast<hipStream_t>(stream)));
}

int moe_combine_backward(const void* dy, int dt, const void* y_perm, int y_perm_dt,
                         const int32_t* dst_row, const float* topk_w, int T, int k, int H,
                         void* dy_perm, float* dtopk_w, void* stream) {
  if (!valid_dt(dt) || !valid_dt(y_perm_dt) || T < 0 || k < 1) return MOE_ERR_INVALID_ARG;
  const int st = check_row_width(H);
  if (st) return st;
  if (k > KMAX || !fits_int(T, k) || !rows_fit(T, H)) return MOE_ERR_UNSUPPORTED;
  if (any_misaligned(dy, y_perm, dst_row, topk_w, dy_perm, dtopk_w)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!dy || !y_perm || !dst_row || !topk_w || !dy_perm || !dtopk_w) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_combine_bwd(dy, dt, y_perm, y_perm_dt, dst_row, topk_w, T, k, H,
                                       dy_perm, dtopk_w, static_cast<hipStream_t>(stream)));
}

size_t moe_grouped_ffn_train_workspace_size(int max_rows, int E_loc, int H, int I_loc, int dt) {
  dt = rows_dt(dt);
  if (check_train(max_rows, E_loc, H, I_loc, dt) != MOE_OK) return 0;
  return align_up((size_t)(max_rows > 0 ? max_rows : 1) * I_loc * elt_bytes(dt));
}

int moe_grouped_ffn_train(const void* x_perm, const void* x, const int32_t* src_token,
                          const int32_t* offsets, int E_loc, int max_rows, int H, int I_loc,
                          const void* w13, const void* w2, int dt, void* gu, void* y_perm,
                          void* ws, size_t ws_bytes, void* stream) {
  const bool gu16 = dt != rows_dt(dt);
  dt = rows_dt(dt);
  const int st = check_train(max_rows, E_loc, H, I_loc, dt);
  if (st) return st;
  if (any_misaligned(x_perm, x, src_token, offsets, w13, w2, gu, y_perm, ws))
    return MOE_ERR_INVALID_ARG;
  if (max_rows == 0) return MOE_OK;
  if (!offsets || !w13 || !w2 || !gu || !y_perm || (!x_perm && (!x || !src_token)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_grouped_ffn_train_workspace_size(max_rows, E_loc, H, I_loc, dt))
    return MOE_ERR_WORKSPACE;
  const TrainFfn f{x_perm ? x_perm : x, x_perm ? nullptr : src_token, offsets, E_loc, max_rows, H,
                   I_loc, dt, w13, w2, gu, gu16, ws};
  return hip_status(launch_train_forward(f, y_perm, static_cast<hipStream_t>(stream)));
}

size_t moe_grouped_ffn_backward_workspace_size(int max_rows, int E_loc, int H, int I_loc, int dt) {
  dt = rows_dt(dt);
  if (check_train(max_rows, E_loc, H, I_loc, dt) != MOE_OK) return 0;
  const size_t eb = elt_bytes(dt), rows = max_rows > 0 ? max_rows : 1;
  return align_up(rows * I_loc * eb) + align_up(rows * I_loc * eb * 2) + align_up(rows * H * eb);
}

int moe_grouped_ffn_backward(const void* dy_perm, const void* x_perm, const void* x,
                             const int32_t* src_token, const int32_t* offsets, int E_loc,
                             int max_rows, int H, int I_loc, const void* w13, const void* w2,
                             int dt, const void* gu, void* dx_perm, void* dw13, void* dw2,
                             void* ws, size_t ws_bytes, void* stream) {
  const bool gu16 = dt != rows_dt(dt);
  dt = rows_dt(dt);
  const int st = check_train(max_rows, E_loc, H, I_loc, dt);
  if (st) return st;
  if (!dw13 != !dw2 || (!dx_perm && !dw2)) return MOE_ERR_INVALID_ARG;
  if (any_misaligned(dy_perm, x_perm, x, src_token, offsets, w13, w2, gu, dx_perm, dw13, dw2, ws))
    return MOE_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (max_rows == 0) {
    if (!dw2) return MOE_OK;
    const size_t bytes = (size_t)E_loc * H * I_loc * elt_bytes(dt);
    MOE_TRY(launch_zero(dw2, bytes, s));
    return hip_status(launch_zero(dw13, 2 * bytes, s));
  }
  // (x is read by dw13 only)
  if (!dy_perm || !offsets || !w13 || !w2 || !gu || (dw2 && !x_perm && (!x || !src_token)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_grouped_ffn_backward_workspace_size(max_rows, E_loc, H, I_loc, dt))
    return MOE_ERR_WORKSPACE;
  Carver c(ws);
  void* h = c.take<char>((size_t)max_rows * I_loc * elt_bytes(dt));
  void* dgu = c.take<char>((size_t)max_rows * I_loc * elt_bytes(dt) * 2);
  void* xp = c.take<char>((size_t)max_rows * H * elt_bytes(dt));
  const TrainFfn f{x_perm ? x_perm : x, x_perm ? nullptr : src_token, offsets, E_loc, max_rows, H,
                   I_loc, dt, w13, w2, const_cast<void*>(gu), gu16, h};
  return hip_status(launch_train_backward(f, dy_perm, dgu, xp, dx_perm, dw13, dw2, s));
}

size_t moe_grouped_ffn_mxfp8_workspace_size(int max_rows, int E_loc, int H, int I_loc) {
  if (check_mx(max_rows, E_loc, H, I_loc) != MOE_OK) return 0;
  const size_t rows = max_rows > 0 ? max_rows : 1;
  // h in MXFP8, or in float32 where few rows take that form: the larger of the
  // two for any count up to max_rows, so that a program's largest batch sizes
  // the workspace for all
  const size_t f = rows < mx_float_rows(I_loc) ? rows : mx_float_rows(I_loc);
  const size_t h8 = align_up(rows * I_loc) + align_up(rows * MOE_MX_PITCH(I_loc));
  const size_t hf = align_up(f * I_loc * 4);
  return h8 > hf ? h8 : hf;
}

int moe_grouped_ffn_mxfp8(const void* x8, const uint8_t* x_scale, const int32_t* src_token,
                          const int32_t* offsets, int E_loc, int max_rows, int H, int I_loc,
                          const void* w13, const uint8_t* w13_scale, const void* w2,
                          const uint8_t* w2_scale, void* y_perm, int y_dt, void* ws,
                          size_t ws_bytes, void* stream) {
  if (!valid_dt(y_dt)) return MOE_ERR_INVALID_ARG;
  const int st = check_mx(max_rows, E_loc, H, I_loc);
  if (st) return st;
  if (any_misaligned(x8, x_scale, src_token, offsets, w13, w13_scale, w2, w2_scale, y_perm, ws))
    return MOE_ERR_INVALID_ARG;
  if (max_rows == 0) return MOE_OK;
  if (!x8 || !x_scale || !offsets || !w13 || !w13_scale || !w2 || !w2_scale || !y_perm)
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_grouped_ffn_mxfp8_workspace_size(max_rows, E_loc, H, I_loc))
    return MOE_ERR_WORKSPACE;
  Carver c(ws);
  uint8_t* h8 = c.take<uint8_t>((size_t)max_rows * I_loc);   // (float32 h leaves hs unused)
  uint8_t* hs = c.take<uint8_t>((size_t)max_rows * MOE_MX_PITCH(I_loc));
  const MxFfn f{static_cast<const uint8_t*>(x8), x_scale, src_token, offsets, E_loc, max_rows, H,
                I_loc, static_cast<const uint8_t*>(w13), w13_scale,
                static_cast<const uint8_t*>(w2), w2_scale, h8, hs, y_perm, y_dt};
  return hip_status(launch_mx_ffn(f, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
