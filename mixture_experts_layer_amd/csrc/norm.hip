// RMS norm in front of the MoE layer, with the residual's addition and an
// MXFP8 output, and its backward pass, gfx950.
//
//   s = x + residual (rounded to the row type: the residual stream),
//   rstd = 1 / sqrt(mean(s^2) + eps),   y = s * rstd * w.
//
// Both directions are memory-bound.  A block of up to 1024 threads holds one
// row in registers, 8 consecutive elements (16 bytes of bfloat16) per thread
// and step, so every input is read once and the row never goes back to memory
// between its statistics and its outputs.  Measured on MI355X (a large copy:
// 5.09 TB/s): 8192 x 4096 bfloat16 with a residual to sum, y and MXFP8 52 to 55
// us, 5.5 TB/s; backward of 8191 x 7168 with dsum 96 us, 4.9 TB/s; one row of 4096
// 2.8 us, a launch and one chain of loads.
#include "moe_ops_device.h"
#include "moe_ops_kernels.h"

namespace moe {

struct NormArgs {
  const void* x;
  const void* residual;   // or null
  const void* w;
  void* sum;              // or null
  void* y;                // or null
  uint8_t* y8;            // or null
  uint8_t* y8_scale;
  float* rstd;            // or null
  float eps;
  int H, n_chunk, pitch;
};

// The statistic and the products are taken in float64: the memory's time hides
// them, neither a row's squares nor s * w, whose product with rstd may be an
// ordinary number again, leave the range, and an element next to a rounding
// border falls on the side that the formula says, whatever the order of the sum.
//
// On the way to 8 bits and to bfloat16 a value passes float32 rounded to odd
// (a last bit of 1 stands for "and a little more"), so that it is rounded once:
// through the nearest float32 some 5 to 15 of 33 million elements landed on a
// border and went to its wrong side.
//
// The four threads of a quad hold one MXFP8 block (4 x 8 elements): its
// largest magnitude is two lane exchanges away.  No __restrict__: sum and y
// may be x or residual themselves (a thread reads its elements of a row
// before any thread of the block writes).
__device__ __forceinline__ float to_odd_f32(double v) {
  uint2 u = __builtin_bit_cast(uint2, v);
  u.x = (u.x & 0x1fffffffu ? u.x | 0x20000000u : u.x) & 0xe0000000u;
  return (float)__builtin_bit_cast(double, u);
}

template <bool BF16, int NV>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormArgs a) {
  __shared__ double red[16];
  const size_t t = blockIdx.x, rb = row_bytes(BF16, a.H);
  const char* xr = static_cast<const char*>(a.x) + t * rb;
  const char* rr = static_cast<const char*>(a.residual) + t * rb;
  Chunk<BF16> v[NV], r[NV], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < a.n_chunk) {
      v[i].load(xr, c);
      if (a.residual) r[i].load(rr, c);
      w[i].load(a.w, c);
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < a.n_chunk) {
      float f[8];
      if (a.residual) {
        float q[8];
        v[i].get(f);
        r[i].get(q);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += q[e];
        v[i].set(f);      // the stream's own rounding; the norm is of what is stored
      }
      v[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fma((double)f[e], (double)f[e], ss);
    }
  }
  const double rstd = 1.0 / sqrt(block_sum(ss, red) / a.H + (double)a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[t] = (float)rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < a.n_chunk) {
      if (a.sum) v[i].store(static_cast<char*>(a.sum) + t * rb, c);
      float f[8], q[8], y[8];
      v[i].get(f);
      w[i].get(q);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double p = (double)f[e] * (double)q[e] * rstd;   // (the first product is exact)
        f[e] = to_odd_f32(p);
        y[e] = BF16 ? f[e] : (float)p;
      }
      if (a.y) {
        Chunk<BF16> o;
        o.set(y);
        o.store(static_cast<char*>(a.y) + t * rb, c);
      }
      if (a.y8) {     // (n_chunk is a multiple of 4: whole quads come here)
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
        const uint32_t b = mx_scale_byte(quad_max(m));
        const float k = mx_inv_scale(b);
        const uint2 o = make_uint2(mx_pack4(f[0] * k, f[1] * k, f[2] * k, f[3] * k),
                                   mx_pack4(f[4] * k, f[5] * k, f[6] * k, f[7] * k));
        *reinterpret_cast<uint2*>(a.y8 + t * a.H + 8 * c) = o;
        if ((c & 3) == 0) a.y8_scale[t * a.pitch + (c >> 2)] = (uint8_t)b;
      }
    }
  }
  // the scale row's last bytes, where H is no multiple of 128
  if (a.y8 && (int)threadIdx.x < a.pitch - a.H / 32)
    a.y8_scale[t * a.pitch + a.H / 32 + threadIdx.x] = 0;
}

// ---------------------------------------------------------------------------
// Backward.  With xh = s * rstd and g = dy * w:
//   dx = rstd * (g - xh * mean(g * xh)) + dsum,   dw = sum_t dy * xh.
// A block takes every gridDim-th row and keeps its columns' dw sums in
// registers; the blocks' sums go to the workspace and a second launch (3 us
// for 77 rows, 5 us for 512 blocks of 7168) adds them in block order, so dw does
// not depend on timing.
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  const void* dy;
  const void* dsum;       // or null
  const void* s;
  const void* w;
  const float* rstd;
  void* dx;
  float* part;            // [gridDim.x][H]
  int T, H, n_chunk;
};

template <bool BF16, int NV>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[2][16];
  const size_t rb = row_bytes(BF16, a.H);
  Chunk<BF16> w[NV];
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < a.n_chunk) w[i].load(a.w, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  }
  Chunk<BF16> dy[NV], s[NV], ds[NV];
  float rs = 0.f;
  auto fetch = [&](unsigned t) {
    rs = a.rstd[t];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < a.n_chunk) {
        dy[i].load(static_cast<const char*>(a.dy) + t * rb, c);
        s[i].load(static_cast<const char*>(a.s) + t * rb, c);
        if (a.dsum) ds[i].load(static_cast<const char*>(a.dsum) + t * rb, c);
      }
    }
  };
  const unsigned T = a.T;      // (unsigned: the step past the last row may leave int)
  unsigned t = blockIdx.x;
  int turn = 0;
  if (t < T) fetch(t);
  for (; t < T; t += gridDim.x, turn ^= 1) {
    const float rstd = rs;
    float xh[NV][8], g[NV][8], dot = 0.f;
    Chunk<BF16> dsum[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      dsum[i] = ds[i];
      if (c < a.n_chunk) {
        float d[8], q[8];
        dy[i].get(d);
        s[i].get(xh[i]);
        w[i].get(q);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[i][e] *= rstd;
          g[i][e] = d[e] * q[e];
          acc[i][e] = fmaf(d[e], xh[i][e], acc[i][e]);
          dot = fmaf(g[i][e], xh[i][e], dot);
        }
      }
    }
    // the next row's loads fly during this row's reduction and stores
    if (t + gridDim.x < T) fetch(t + gridDim.x);
    const float m = block_sum(dot, red[turn]) / (float)a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < a.n_chunk) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd * (g[i][e] - xh[i][e] * m);
        if (a.dsum) {
          float q[8];
          dsum[i].get(q);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += q[e];
        }
        Chunk<BF16> out;
        out.set(o);
        out.store(static_cast<char*>(a.dx) + t * rb, c);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < a.n_chunk) {
      float4* p = reinterpret_cast<float4*>(a.part + (size_t)blockIdx.x * a.H) + 2 * c;
      p[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      p[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// dw[c] = sum over n rows of part[.][c]: 32 columns per block, 32 threads per
// column over the rows, then their sums in order.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* part, int n, int H,
                                                          float* out) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;     // H is a multiple of 32
  float v = 0.f;
#pragma unroll 8
  for (int i = r; i < n; i += 32) v += part[(size_t)i * H + col];
  s[r][c] = v;
  __syncthreads();
  if (r == 0) {
    for (int i = 1; i < 32; ++i) v += s[i][c];
    out[col] = v;
  }
}

// ---------------------------------------------------------------------------
// Backward of the combine, y[t] = sum_j w[t][j] * y_perm[dst_row[t][j]]:
//   dy_perm[dst_row[t][j]] = w[t][j] * dy[t],   dw[t][j] = <dy[t], y_perm[row]>.
// Rows belong to one (token, slot) each, so a block per token writes its own
// rows and no two blocks meet.  dy[t] stays in registers over the slots.
// Memory-bound: T = 8192, k = 8, H = 4096 in bfloat16 takes 228 us, 5.0 TB/s.  With
// fewer tokens than CUs each busy CU moves all slots of its token, and the others
// nothing: T = 33, k = 8, H = 7168 7 us, 0.24 MB per block.
// ---------------------------------------------------------------------------
struct CombineBwdArgs {
  const void* dy;
  const void* y_perm;
  const int32_t* dst_row;
  const float* w;
  void* dy_perm;
  float* dw;
  int k, H, n_chunk;
};

constexpr int CB_SLOTS = 8;    // slots whose rows are in flight together

template <bool DY_BF16, bool Y_BF16, int NV>
__global__ __launch_bounds__(1024) void combine_bwd_kernel(CombineBwdArgs a) {
  __shared__ float red[16][CB_SLOTS];
  const size_t t = blockIdx.x;
  const size_t rb = row_bytes(Y_BF16, a.H);
  float d[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) d[i][e] = 0.f;
    if (c < a.n_chunk) {
      Chunk<DY_BF16> v;
      v.load(static_cast<const char*>(a.dy) + t * row_bytes(DY_BF16, a.H), c);
      v.get(d[i]);
    }
  }
  for (int j0 = 0; j0 < a.k; j0 += CB_SLOTS) {
    int row[CB_SLOTS];
    float dot[CB_SLOTS];
#pragma unroll
    for (int u = 0; u < CB_SLOTS; ++u) {
      row[u] = j0 + u < a.k ? a.dst_row[t * a.k + j0 + u] : -1;
      dot[u] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= a.n_chunk) continue;
      Chunk<Y_BF16> y[CB_SLOTS];
#pragma unroll
      for (int u = 0; u < CB_SLOTS; ++u)
        if (row[u] >= 0) y[u].load(static_cast<const char*>(a.y_perm) + row[u] * rb, c);
#pragma unroll
      for (int u = 0; u < CB_SLOTS; ++u) {
        if (row[u] < 0) continue;
        const float wj = a.w[t * a.k + j0 + u];
        float f[8];
        y[u].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot[u] = fmaf(d[i][e], f[e], dot[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = wj * d[i][e];
        y[u].set(f);
        y[u].store(static_cast<char*>(a.dy_perm) + row[u] * rb, c);
      }
    }
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
    for (int u = 0; u < CB_SLOTS; ++u) {
      const float v = wave_sum_f(dot[u]);
      if (lane == 0) red[wid][u] = v;
    }
    lds_barrier();
    if (threadIdx.x < CB_SLOTS && j0 + (int)threadIdx.x < a.k) {
      float v = 0.f;
      for (int w = 0; w < (int)(blockDim.x >> 6); ++w) v += red[w][threadIdx.x];
      a.dw[t * a.k + j0 + threadIdx.x] = v;    // 0 for a slot without a row
    }
    lds_barrier();
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
__global__ void fill_zero16_kernel(uint4* p, size_t n) {
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n;
       i += (size_t)gridDim.x * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

hipError_t launch_zero(void* p, size_t bytes, hipStream_t st) {
  const size_t n = bytes / 16;
  if (n == 0) return hipSuccess;
  const size_t blocks = (n + 255) / 256;
  fill_zero16_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, st>>>(
      static_cast<uint4*>(p), n);
  return hipGetLastError();
}

// Threads per row and 8-element chunks per thread: one chunk per thread up to
// 8192 elements, two beyond (the block limit of 1024 threads).
int row_threads(int H) {
  const int n = H / 8;
  return n >= 1024 ? 1024 : (n + 63) / 64 * 64;
}

template <bool BF16>
static hipError_t norm_launch(const NormArgs& a, int T, hipStream_t st) {
  const int nt = row_threads(a.H);
  if (a.n_chunk <= nt) rmsnorm_kernel<BF16, 1><<<T, nt, 0, st>>>(a);
  else rmsnorm_kernel<BF16, 2><<<T, nt, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm(const void* x, const void* residual, const void* w, float eps, int T,
                          int H, int dt, void* sum, void* y, void* y8, void* y8_scale, float* rstd,
                          hipStream_t st) {
  if (T <= 0) return hipSuccess;
  if (H / 8 > 2048) return hipErrorInvalidValue;
  const NormArgs a{x, residual, w, sum, y, static_cast<uint8_t*>(y8),
                   static_cast<uint8_t*>(y8_scale), rstd, eps, H, H / 8, (H + 127) / 128 * 4};
  return dt == 1 ? norm_launch<true>(a, T, st) : norm_launch<false>(a, T, st);
}

// Blocks of the backward pass: two per CU, each with at least a row.
int rmsnorm_bwd_blocks(int T) { return T < 512 ? T : 512; }

template <bool BF16>
static hipError_t norm_bwd_launch(const NormBwdArgs& a, int blocks, hipStream_t st) {
  const int nt = row_threads(a.H);
  if (a.n_chunk <= nt) rmsnorm_bwd_kernel<BF16, 1><<<blocks, nt, 0, st>>>(a);
  else rmsnorm_bwd_kernel<BF16, 2><<<blocks, nt, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const void* dy, const void* dsum, const void* s, const void* w,
                              const float* rstd, int T, int H, int dt, void* dx, float* dw,
                              float* part, hipStream_t st) {
  if (T <= 0) return launch_zero(dw, (size_t)H * 4, st);
  if (H / 8 > 2048) return hipErrorInvalidValue;
  const NormBwdArgs a{dy, dsum, s, w, rstd, dx, part, T, H, H / 8};
  const int blocks = rmsnorm_bwd_blocks(T);
  hipError_t err = dt == 1 ? norm_bwd_launch<true>(a, blocks, st)
                           : norm_bwd_launch<false>(a, blocks, st);
  if (err != hipSuccess) return err;
  column_sum_kernel<<<H / 32, 1024, 0, st>>>(part, blocks, H, dw);
  return hipGetLastError();
}

template <bool DY, bool Y>
static hipError_t combine_bwd_launch(const CombineBwdArgs& a, int T, hipStream_t st) {
  const int nt = row_threads(a.H);
  if (a.n_chunk <= nt) combine_bwd_kernel<DY, Y, 1><<<T, nt, 0, st>>>(a);
  else combine_bwd_kernel<DY, Y, 2><<<T, nt, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* dy, int dt, const void* y_perm, int y_perm_dt,
                              const int32_t* dst_row, const float* w, int T, int k, int H,
                              void* dy_perm, float* dw, hipStream_t st) {
  if (T <= 0) return hipSuccess;
  if (H / 8 > 2048) return hipErrorInvalidValue;
  const CombineBwdArgs a{dy, y_perm, dst_row, w, dy_perm, dw, k, H, H / 8};
  if (dt == 1)
    return y_perm_dt == 1 ? combine_bwd_launch<true, true>(a, T, st)
                          : combine_bwd_launch<true, false>(a, T, st);
  return y_perm_dt == 1 ? combine_bwd_launch<false, true>(a, T, st)
                        : combine_bwd_launch<false, false>(a, T, st);
}

}  // namespace moe
