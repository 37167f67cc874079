// Host-side launchers of the operators around the layer (internal to the
// library; the entry points are in ops_abi.hip, their contract in
// include/moe_ops.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int OPS_MAX_H = 16384;   // row elements the one-block-per-row kernels hold

// Zero `bytes` (a multiple of 16) by a kernel, which a graph replays safely.
hipError_t launch_zero(void* p, size_t bytes, hipStream_t st);

// norm.hip; H a multiple of 32, at most OPS_MAX_H
hipError_t launch_rmsnorm(const void* x, const void* residual, const void* w, float eps, int T,
                          int H, int dt, void* sum, void* y, void* y8, void* y8_scale, float* rstd,
                          hipStream_t st);
int rmsnorm_bwd_blocks(int T);     // rows of `part`
hipError_t launch_rmsnorm_bwd(const void* dy, const void* dsum, const void* s, const void* w,
                              const float* rstd, int T, int H, int dt, void* dx, float* dw,
                              float* part, hipStream_t st);
hipError_t launch_combine_bwd(const void* dy, int dt, const void* y_perm, int y_perm_dt,
                              const int32_t* dst_row, const float* w, int T, int k, int H,
                              void* dy_perm, float* dw, hipStream_t st);

}  // namespace moe
