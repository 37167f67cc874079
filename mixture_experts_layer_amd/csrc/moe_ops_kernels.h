// Host-side launchers of the operators around the layer (internal to the
// library; the entry points are in ops_abi.hip, their contract in
// include/moe_ops.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace moe {

constexpr int OPS_MAX_H = 16384;   // row elements the one-block-per-row kernels hold

// Zero `bytes` (a multiple of 16) by a kernel, which a graph replays safely.
hipError_t launch_zero(void* p, size_t bytes, hipStream_t st);

// norm.hip; H a multiple of 32, at most OPS_MAX_H
int row_threads(int H);            // threads of the block that takes a row
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

// ffn_train.hip: the grouped SwiGLU experts in training.  H, I multiples of 32.
struct TrainFfn {
  const void* x;            // token rows, gathered by src_token, or permuted rows
  const int32_t* src_token; // or null
  const int32_t* offsets;   // [E + 1]
  int E, max_rows, H, I, dt;
  const void* w13;
  const void* w2;
  void* gu;                 // [max_rows][2 I]: written by the forward pass, read by the backward
  bool gu16;                // its form: 16 bits per value (bfloat16 rows only), else float32
  void* h;                  // [max_rows][I], workspace
};
constexpr int OPS_MAX_DIM = 65536;               // H and I of the expert blocks
constexpr long long OPS_MAX_HI = 1ll << 30;      // H * I: 32-bit offsets inside an expert
constexpr int OPS_MAX_ROWS = 1 << 30;            // rows of the expert blocks
// whether every launch of a shape holds fewer than 2^32 threads
bool train_fits(int max_rows, int E, int H, int I, int dt);
bool mx_fits(int max_rows, int E, int H, int I);
hipError_t launch_train_forward(const TrainFfn& f, void* y, hipStream_t st);
// dgu: [max_rows][2 I], workspace; x_perm: [max_rows][H], workspace of the
// gathered form; dx, or dw13 with dw2, may be null
hipError_t launch_train_backward(const TrainFfn& f, const void* dy, void* dgu, void* x_perm,
                                 void* dx, void* dw13, void* dw2, hipStream_t st);

// ffn_mxfp8.hip: the grouped SwiGLU experts on MXFP8 rows and weights.
struct MxFfn {
  const uint8_t* x8;        // rows of H, gathered by src_token (or null: permuted)
  const uint8_t* x_scale;
  const int32_t* src_token;
  const int32_t* offsets;   // [E + 1]
  int E, max_rows, H, I;
  const uint8_t* w13;
  const uint8_t* w13_scale;
  const uint8_t* w2;
  const uint8_t* w2_scale;
  uint8_t* h8;              // workspace: h [max_rows][I] in e4m3 and its scales,
                            // or in float32 (mx_float_rows at most)
  uint8_t* h_scale;
  void* y;
  int y_dt;
};
size_t mx_float_rows(int I);        // most rows whose h is kept in float32
hipError_t launch_mx_ffn(const MxFfn& f, hipStream_t st);

}  // namespace moe
