// Grouped SwiGLU experts on MXFP8 rows and weights, gfx950.
//
//   h = MXFP8(SiLU(W_gate a) * (W_up a)),   y = W2 h
//
// Both products run on v_mfma_scale_f32_*_f8f6f4, which multiplies e4m3
// elements and applies one E8M0 scale per 32 of them on either side, so the
// scales cost no vector instructions: a lane's operand register brings the
// scale byte of its row's 32-element block.  The instruction sums a block of
// 64 or 128 products with about 16 significant bits (measured: 1.5e-5 of the
// result on blocks of normal data, against 2^-4 of an element's own
// rounding) and accumulates blocks in float32.
//
// In 32x32x64, lane l holds row l % 32 and, in its two 16-byte halves, the
// elements 16 (l / 32) + [0, 16) of block 0 and of block 1; the scale of
// block b is taken from the lanes with l / 32 == b.  In 16x16x128, lane l
// holds row l % 16, elements 16 (l / 16) and 64 + 16 (l / 16) on, and block b's
// scale is taken from the lanes with l / 16 == b.
//
// Few rows per expert: the weights are the traffic, and the direct kernel
// streams them from memory into the operands.  Many rows: the tiled kernel,
// operands staged through LDS.
#include <algorithm>
#include <type_traits>

#include "moe_kernels.h"
#include "moe_ops_device.h"
#include "moe_ops_kernels.h"

namespace moe {

typedef int i32x4_v __attribute__((ext_vector_type(4)));
typedef int i32x8_v __attribute__((ext_vector_type(8)));

struct MxArgs {
  const uint8_t* A;           // rows [*][K]
  const uint8_t* As;          // their scales [*][pitch]
  const int32_t* src_token;   // or null: row r reads A row r
  const int32_t* offsets;
  int E, max_rows;
  const uint8_t* B;           // weights [E][b_rows][K]
  const uint8_t* Bs;          // their scales [E][b_rows][pitch]
  int K, N, b_rows;           // N: output columns (SWIGLU: I, up rows at N + n)
  int pitch, out_pitch;       // scale bytes per row of K and of N elements
  void* Y;                    // [rows][N]: SWIGLU: e4m3, else bfloat16 or float32
  uint8_t* Ys;                // SWIGLU: [rows][out_pitch]
};

// Scale bytes of the blocks past the end read as 2^0 (they multiply zeros;
// whatever a caller left there must not turn them into NaN).  blocks: 32-element
// blocks that the dword's four bytes may still cover.
__device__ __forceinline__ int mx_valid_scales(int s, int blocks) {
  const uint32_t keep = blocks >= 4 ? 0xffffffffu : (1u << (8 * blocks)) - 1u;
  return (int)(((uint32_t)s & keep) | (0x7f7f7f7fu & ~keep));
}

// ---------------------------------------------------------------------------
// Tiled kernel: TM rows x TN weight rows per block, contraction in chunks of
// 128 bytes, STAGES buffers.  An LDS row holds 8 chunks of 16 bytes, chunk c of
// row r at c ^ (r / 2 % 8); behind the rows of a stage lie their scale dwords
// (the four blocks of the chunk).  SWIGLU: TN / 2 gate rows, then the matching
// up rows, as in the bfloat16 kernels.
// ---------------------------------------------------------------------------
template <int TM_, int TN_, int STAGES_, int WM_, int WN_>
struct MxCfg {
  static constexpr int TM = TM_, TN = TN_, STAGES = STAGES_, WM = WM_, WN = WN_, TK = 128;
  static constexpr int NW = WM * WN, NTHR = NW * 64;
  static constexpr int WTM = TM / WM, WTN = TN / WN, MFM = WTM / 32, MFN = WTN / 32;
  static constexpr int ABYTES = TM * TK, BBYTES = TN * TK;
  static constexpr int SCALES = (TM + TN) * 4;
  static constexpr int SBYTES = ABYTES + BBYTES + SCALES;
  static constexpr int ALOADS = ABYTES / 1024 / NW, BLOADS = BBYTES / 1024 / NW;
  static constexpr int SLOADS = (TM + TN) / 64;       // scale loads per stage, in all
  static constexpr int PITCH = TN * 2 + 16;           // staged output row
  static constexpr int LDS = STAGES * SBYTES > TM * PITCH ? STAGES * SBYTES : TM * PITCH;
  static_assert(NW == 8 && ALOADS * 8192 == ABYTES && BLOADS * 8192 == BBYTES, "load split");
  static_assert(SLOADS <= NW && TM % 64 == 0 && TN % 64 == 0, "one scale load per wave");
  static_assert(LDS <= 160 * 1024 && SBYTES % 256 == 0, "LDS per block");
};

__device__ __forceinline__ int mx_swz(int r) { return (r >> 1) & 7; }

template <class C, bool SWIGLU, bool OUT_BF16, bool GATHER>
__global__ __launch_bounds__(C::NTHR, 1) void mx_tile_kernel(MxArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int COLS = SWIGLU ? C::TN / 2 : C::TN;
  const int NT = (a.N + COLS - 1) / COLS;
  TileScan scan;
  scan.init(a.offsets, a.E, C::TM, a.max_rows);
  int b = blockIdx.x;
  const int n_active = scan.total * NT, per = n_active >> 3;
  if (b >= n_active) return;
  if (b < per * 8) b = (b & 7) * per + (b >> 3);       // contiguous numbers share an XCD's L2
  const RowTile t = scan.find(a.offsets, a.E, C::TM, a.max_rows, b / NT);
  const int te = (t.end - t.off + C::TM - 1) / C::TM, li = b - t.first * NT;
  const int n_t = li / te;
  const int r0 = t.off + (li - n_t * te) * C::TM, r1 = min(r0 + C::TM, t.end);
  const int n0 = n_t * COLS;
  const uint8_t* Be = a.B + (size_t)t.e * a.b_rows * a.K;
  const uint8_t* Bse = a.Bs + (size_t)t.e * a.b_rows * a.pitch;

  auto b_row = [&](int rt) {      // weight row of tile row rt; past the end, the last one
    if (SWIGLU) return rt < COLS ? min(n0 + rt, a.N - 1) : a.N + min(n0 + rt - COLS, a.N - 1);
    return min(n0 + rt, a.N - 1);
  };
  const int kchunk = (lane & 7) ^ mx_swz(wid * 8 + (lane >> 3));    // the same for every load
  const uint8_t* ap[GATHER ? C::ALOADS : 1];
  uint32_t ao[C::ALOADS], bo[C::BLOADS];
#pragma unroll
  for (int j = 0; j < C::ALOADS; ++j) {
    const int row = min(r0 + (wid + 8 * j) * 8 + (lane >> 3), r1 - 1);
    ao[j] = (uint32_t)(row - r0) * a.K + kchunk * 16;
    if constexpr (GATHER) ap[j] = a.A + (size_t)max(a.src_token[row], 0) * a.K + kchunk * 16;
  }
#pragma unroll
  for (int j = 0; j < C::BLOADS; ++j)
    bo[j] = (uint32_t)b_row((wid + 8 * j) * 8 + (lane >> 3)) * (uint32_t)a.K + kchunk * 16;
  const uint8_t* abase = a.A + (size_t)r0 * a.K;
  // scales: wave w loads those of tile rows [64 w, 64 w + 64) of A then B
  const uint8_t* sp = nullptr;
  if (wid < C::SLOADS) {
    const int rt = wid * 64 + lane;
    if (wid < C::TM / 64) {
      const int row = min(r0 + rt, r1 - 1);
      sp = a.As + (size_t)(GATHER ? max(a.src_token[row], 0) : row) * a.pitch;
    } else {
      sp = Bse + (size_t)b_row(rt - C::TM) * a.pitch;
    }
  }

  const int nk = (a.K + C::TK - 1) / C::TK;
  auto issue = [&](int ks, int buf) {
    unsigned char* sa = smem + buf * C::SBYTES + wid * 1024;
    unsigned char* sb = sa + C::ABYTES;
    // 16-byte chunks past the contraction's end re-read the first
    const uint32_t back = ks * C::TK + kchunk * 16 >= a.K ? kchunk * 16 : 0;
#pragma unroll
    for (int j = 0; j < C::ALOADS; ++j) {
      if constexpr (GATHER)
        __builtin_amdgcn_global_load_lds((gbl_void_t*)(ap[j] + ks * C::TK - back),
                                         (lds_void_t*)(sa + 8192 * j), 16, 0, 0);
      else
        buffer_load_lds16(abase, 0xffffffffu, sa + 8192 * j, ao[j] - back, ks * C::TK);
    }
#pragma unroll
    for (int j = 0; j < C::BLOADS; ++j)
      buffer_load_lds16(Be, 0xffffffffu, sb + 8192 * j, bo[j] - back, ks * C::TK);
    if (wid < C::SLOADS)
      __builtin_amdgcn_global_load_lds(
          (gbl_void_t*)(sp + ks * 4),
          (lds_void_t*)(smem + buf * C::SBYTES + C::ABYTES + C::BBYTES + wid * 256), 4, 0, 0);
  };
  auto zero_tail = [&](unsigned char* sa, int left) {
    for (int i = threadIdx.x; i < (C::TM + C::TN) * 8; i += C::NTHR)
      if (((i & 7) ^ mx_swz(i >> 3)) * 16 >= left)
        reinterpret_cast<uint4*>(sa)[i] = make_uint4(0, 0, 0, 0);
    lds_barrier();
  };

  const int wm = wid / C::WN, wn = wid % C::WN;
  const int lrow = lane & 31, khalf = lane >> 5;
  int nbase[C::MFN];
#pragma unroll
  for (int ni = 0; ni < C::MFN; ++ni) {
    if (SWIGLU) {
      constexpr int HALF = C::MFN / 2;
      nbase[ni] = (ni < HALF ? 0 : COLS) + wn * (C::WTN / 2) + (ni % HALF) * 32;
    } else {
      nbase[ni] = wn * C::WTN + ni * 32;
    }
  }
  // rows of a wave's subtiles start at multiples of 32, so one swizzle does
  const int swz = mx_swz(lrow);
  auto frag = [&](const unsigned char* base, int row0, int step) {
    const unsigned char* p = base + (row0 + lrow) * C::TK;
    const i32x4_v lo = *reinterpret_cast<const i32x4_v*>(p + (((step * 4 + khalf) ^ swz) * 16));
    const i32x4_v hi = *reinterpret_cast<const i32x4_v*>(p + (((step * 4 + 2 + khalf) ^ swz) * 16));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x16_t acc[C::MFM][C::MFN];
#pragma unroll
  for (int i = 0; i < C::MFM; ++i)
#pragma unroll
    for (int j = 0; j < C::MFN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

#pragma unroll
  for (int s0 = 0; s0 < C::STAGES - 1; ++s0)
    if (s0 < nk) issue(s0, s0);
  constexpr int NL = C::ALOADS + C::BLOADS;    // at least so many per stage and wave
  for (int ks = 0; ks < nk; ++ks) {
    if (C::STAGES > 2 && ks + 1 < nk) wait_stage_barrier<(C::STAGES - 2) * NL>();
    else wait_stage_barrier<0>();
    if (ks + C::STAGES - 1 < nk) issue(ks + C::STAGES - 1, (ks + C::STAGES - 1) % C::STAGES);
    unsigned char* sa = smem + (ks % C::STAGES) * C::SBYTES;
    const unsigned char* sb = sa + C::ABYTES;
    const int* sc = reinterpret_cast<const int*>(sb + C::BBYTES);
    const int left = a.K - ks * C::TK;
    if (left < C::TK) zero_tail(sa, left);
    // this lane's blocks: byte 0 of the shifted dword in step 0, byte 2 in step 1
    int as[C::MFM], bs[C::MFN];
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi)
      as[mi] = (int)((uint32_t)mx_valid_scales(sc[wm * C::WTM + mi * 32 + lrow], left >> 5) >>
                     (8 * khalf));
#pragma unroll
    for (int ni = 0; ni < C::MFN; ++ni)
      bs[ni] = (int)((uint32_t)mx_valid_scales(sc[C::TM + nbase[ni] + lrow], left >> 5) >>
                     (8 * khalf));
    auto step = [&](auto step_c) {
      constexpr int S = decltype(step_c)::value;
      i32x8_v af[C::MFM], bf[C::MFN];
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni) bf[ni] = frag(sb, nbase[ni], S);
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi) af[mi] = frag(sa, wm * C::WTM + mi * 32, S);
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
        for (int ni = 0; ni < C::MFN; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              bf[ni], af[mi], acc[mi][ni], 0, 0, 2 * S, bs[ni], 2 * S, as[mi]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
  }

  // ---- epilogue; acc[mi][ni][4 q + r]: row mi * 32 + lrow, column nbase + 8 q + 4 khalf + r
  const int nrows = r1 - r0;
  lds_barrier();
  if constexpr (SWIGLU) {
    // h: a lane and the one 32 away hold a row's 32 columns of a subtile,
    // which are one MXFP8 block.  Staged as [row][COLS] bytes, the scale bytes
    // of the row's blocks behind them.
    constexpr int HALF = C::MFN / 2, HP = COLS + 16;
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi) {
      unsigned char* so = smem + (wm * C::WTM + mi * 32 + lrow) * HP;
#pragma unroll
      for (int ni = 0; ni < HALF; ++ni) {
        float h[16], m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          h[i] = silu_fast(acc[mi][ni][i]) * acc[mi][ni + HALF][i];
          m = fmaxf(m, fabsf(h[i]));
        }
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m),
                                                        false, false);
        const uint32_t sb8 = mx_scale_byte(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
        const float k = mx_inv_scale(sb8);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint32_t*>(so + nbase[ni] + 8 * q + 4 * khalf) =
              mx_pack4(h[4 * q] * k, h[4 * q + 1] * k, h[4 * q + 2] * k, h[4 * q + 3] * k);
        if (khalf == 0)
          so[COLS + (nbase[ni] >> 5)] = n0 + nbase[ni] < a.N ? (unsigned char)sb8 : 0;
      }
    }
    lds_barrier();
    uint8_t* Y = static_cast<uint8_t*>(a.Y);
    constexpr int CPR = COLS / 16;
    for (int c = threadIdx.x; c < C::TM * CPR; c += C::NTHR) {
      const int r = c / CPR, cc = c - r * CPR;
      if (r < nrows && n0 + cc * 16 < a.N)
        *reinterpret_cast<uint4*>(Y + (size_t)(r0 + r) * a.N + n0 + cc * 16) =
            *reinterpret_cast<const uint4*>(smem + r * HP + cc * 16);
    }
    for (int r = threadIdx.x; r < nrows; r += C::NTHR)
      *reinterpret_cast<uint32_t*>(a.Ys + (size_t)(r0 + r) * a.out_pitch + (n0 >> 5)) =
          *reinterpret_cast<const uint32_t*>(smem + r * HP + COLS);
    static_assert(!SWIGLU || COLS == 128, "a tile's scales are one dword");
  } else if constexpr (OUT_BF16) {
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2*>(smem + (wm * C::WTM + mi * 32 + lrow) * C::PITCH +
                                    (nbase[ni] + 8 * q + 4 * khalf) * 2) =
              make_uint2(cvt_bf16x2(acc[mi][ni][4 * q], acc[mi][ni][4 * q + 1]),
                         cvt_bf16x2(acc[mi][ni][4 * q + 2], acc[mi][ni][4 * q + 3]));
    lds_barrier();
    bf16_t* Y = static_cast<bf16_t*>(a.Y);
    constexpr int CPR = COLS / 8;
    for (int c = threadIdx.x; c < C::TM * CPR; c += C::NTHR) {
      const int r = c / CPR, cc = c - r * CPR;
      if (r < nrows && n0 + cc * 8 < a.N)
        st_nt16(Y + (size_t)(r0 + r) * a.N + n0 + cc * 8,
                *reinterpret_cast<const uint4*>(smem + r * C::PITCH + cc * 16));
    }
  } else {
    float* Y = static_cast<float*>(a.Y);
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi) {
      const int r = wm * C::WTM + mi * 32 + lrow;
      if (r >= nrows) continue;
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni) {
        if (n0 + nbase[ni] >= a.N) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(Y + (size_t)(r0 + r) * a.N + n0 + nbase[ni] + 8 * q +
                                     4 * khalf) =
              make_float4(acc[mi][ni][4 * q], acc[mi][ni][4 * q + 1], acc[mi][ni][4 * q + 2],
                          acc[mi][ni][4 * q + 3]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Direct kernel: 16 rows of one expert against weights streamed from memory
// into the operands of v_mfma_scale_f32_16x16x128 (weights first, so
// accumulator lane l holds columns 4 (l / 16) + i of row l % 16).  A block's
// waves are CW groups of KW: each group takes its own output columns (SWIGLU:
// 32 of h, two gate and two up tiles; else one tile of 16), and its waves
// split the contraction and meet in LDS, in wave order.
// ---------------------------------------------------------------------------
constexpr int MXD_U = 2;     // contraction steps of 128 whose loads are in flight together

__device__ __forceinline__ i32x4_v ld_nt16(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const i32x4_v*>(p));
}

template <bool SWIGLU, bool OUT_BF16, int CW, int KW>
__global__ __launch_bounds__(CW * KW * 64) void mx_direct_kernel(MxArgs a) {
  constexpr int NT = SWIGLU ? 4 : 1, COLS = SWIGLU ? 32 : 16, NTHR = CW * KW * 64;
  constexpr int RED = NT * 4 * 65;              // floats of one wave's partial sums
  __shared__ float red[CW * KW * RED];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wid / KW, kw = wid % KW;
  const int n_cb = (a.N + CW * COLS - 1) / (CW * COLS);
  TileScan scan;
  scan.init(a.offsets, a.E, 16, a.max_rows);
  const int tile = blockIdx.x / n_cb;
  if (tile >= scan.total) return;
  const RowTile t = scan.find(a.offsets, a.E, 16, a.max_rows, tile);
  const int r0 = t.off + (tile - t.first) * 16, r1 = min(r0 + 16, t.end);
  const int nb = (blockIdx.x - tile * n_cb) * CW * COLS;     // the block's first column
  const int n0 = nb + cw * COLS;
  const int lr = lane & 15, lg = lane >> 4;
  const int row = min(r0 + lr, r1 - 1);
  const size_t src = a.src_token ? max(a.src_token[row], 0) : row;
  const uint8_t* xa = a.A + src * a.K;
  const uint8_t* xs = a.As + src * a.pitch;
  const uint8_t* wp[NT];
  const uint8_t* ws[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    // (a group past the last column re-reads row 0: N is a multiple of 32)
    const int n = (n0 < a.N ? n0 : 0) + (SWIGLU ? (i & 1) * 16 + (i >> 1) * a.N : 0) + lr;
    const size_t w = (size_t)t.e * a.b_rows + n;
    wp[i] = a.B + w * a.K;
    ws[i] = a.Bs + w * a.pitch;
  }
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int steps = (a.K + 127) / 128;
  const int s0 = steps * kw / KW, s1 = steps * (kw + 1) / KW;
  for (int s = s0; s < s1; s += MXD_U) {
    i32x4_v w[MXD_U][NT][2], x[MXD_U][2];
    int wsc[MXD_U][NT], xsc[MXD_U];
#pragma unroll
    for (int u = 0; u < MXD_U; ++u) {
      // (a step past this wave's share re-reads its last and is not multiplied;
      // 16 bytes past the contraction's end re-read the row's first)
      const int st = min(s + u, s1 - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = st * 128 + h * 64 + lg * 16, ko = k < a.K ? k : 0;
#pragma unroll
        for (int i = 0; i < NT; ++i) w[u][i][h] = ld_nt16(wp[i] + ko);
        x[u][h] = *reinterpret_cast<const i32x4_v*>(xa + ko);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) wsc[u][i] = *reinterpret_cast<const int*>(ws[i] + st * 4);
      xsc[u] = *reinterpret_cast<const int*>(xs + st * 4);
    }
#pragma unroll
    for (int u = 0; u < MXD_U; ++u) {
      if (s + u >= s1) break;
      const int left = a.K - (s + u) * 128;
      if (left < 128) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h * 64 + lg * 16 >= left) {
            x[u][h] = i32x4_v{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NT; ++i) w[u][i][h] = i32x4_v{0, 0, 0, 0};
          }
        }
      }
      const i32x8_v xf = __builtin_shufflevector(x[u][0], x[u][1], 0, 1, 2, 3, 4, 5, 6, 7);
      const int xsv = (int)((uint32_t)mx_valid_scales(xsc[u], left >> 5) >> (8 * lg));
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const i32x8_v wf = __builtin_shufflevector(w[u][i][0], w[u][i][1], 0, 1, 2, 3, 4, 5, 6, 7);
        const int wsv = (int)((uint32_t)mx_valid_scales(wsc[u][i], left >> 5) >> (8 * lg));
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc[i], 0, 0, 0, wsv, 0,
                                                                  xsv);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[wid * RED + (i * 4 + q) * 65 + lane] = acc[i][q];
  __syncthreads();
  // outputs of the block: 16 rows x CW * COLS columns, columns fastest
  constexpr int BC = CW * COLS;
  for (int o = threadIdx.x; o < 16 * BC; o += NTHR) {
    const int m = o / BC, c = o - m * BC, g = c / COLS, n = c - g * COLS;
    const int at = (n & 3) * 65 + m + 16 * ((n & 15) >> 2) + (SWIGLU ? (n >> 4) * 4 * 65 : 0);
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const float* p = red + (g * KW + k) * RED + at;
      v += p[0];
      if (SWIGLU) u += p[SWIGLU ? 8 * 65 : 0];
    }
    const bool live = r0 + m < r1 && nb + c < a.N;
    if constexpr (SWIGLU) {
      // 32 consecutive lanes hold a row's block (16 * BC and NTHR are
      // multiples of 64, so whole waves take part)
      const float h = silu_fast(v) * u;
      float mx = fabsf(h);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
      const uint32_t b8 = mx_scale_byte(mx);
      const float hk = h * mx_inv_scale(b8);
      if (live) {
        static_cast<uint8_t*>(a.Y)[(size_t)(r0 + m) * a.N + nb + c] =
            (uint8_t)(mx_pack4(hk, hk, hk, hk) & 0xff);
        if ((c & 31) == 0) a.Ys[(size_t)(r0 + m) * a.out_pitch + ((nb + c) >> 5)] = (uint8_t)b8;
      }
    } else if (live) {
      const size_t yi = (size_t)(r0 + m) * a.N + nb + c;
      if (OUT_BF16) static_cast<bf16_t*>(a.Y)[yi] = (bf16_t)(cvt_bf16x2(v, v) & 0xffff);
      else static_cast<float*>(a.Y)[yi] = v;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using MxBig = MxCfg<256, 256, 2, 2, 4>;
using MxMed = MxCfg<128, 256, 3, 2, 4>;

static long long mx_row_tiles(int max_rows, int E, int BM) {
  const long long bound = ((long long)max_rows + (long long)E * (BM - 1)) / BM;
  return bound < max_rows ? bound : max_rows;
}

template <class C, bool SWIGLU, bool OUT_BF16, bool GATHER>
static hipError_t launch_mx_tile_t(const MxArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> lds_set{0};
  hipError_t err = ensure_lds_limit(
      reinterpret_cast<const void*>(&mx_tile_kernel<C, SWIGLU, OUT_BF16, GATHER>), C::LDS, lds_set);
  if (err != hipSuccess) return err;
  constexpr int cols = SWIGLU ? C::TN / 2 : C::TN;
  const long long grid = mx_row_tiles(a.max_rows, a.E, C::TM) * ((a.N + cols - 1) / cols);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  mx_tile_kernel<C, SWIGLU, OUT_BF16, GATHER><<<(unsigned)grid, C::NTHR, C::LDS, st>>>(a);
  return hipGetLastError();
}

template <bool SWIGLU, bool OUT_BF16, int CW, int KW>
static hipError_t launch_mx_direct_t(const MxArgs& a, hipStream_t st) {
  constexpr int cols = CW * (SWIGLU ? 32 : 16);
  const long long grid = mx_row_tiles(a.max_rows, a.E, 16) * ((a.N + cols - 1) / cols);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  mx_direct_kernel<SWIGLU, OUT_BF16, CW, KW><<<(unsigned)grid, CW * KW * 64, 0, st>>>(a);
  return hipGetLastError();
}

enum MxPath { MX_DIRECT, MX_MED, MX_BIG };
static MxPath mx_path(int max_rows, int E) {
  const int mean = (max_rows + E - 1) / E;
  return mean <= 8 ? MX_DIRECT : mean < 384 ? MX_MED : MX_BIG;
}

template <bool SWIGLU, bool OUT_BF16>
static hipError_t launch_mx(const MxArgs& a, MxPath path, hipStream_t st) {
  if (path == MX_DIRECT) {
    if constexpr (SWIGLU) return launch_mx_direct_t<true, true, 1, 8>(a, st);
    else return launch_mx_direct_t<false, OUT_BF16, 4, 2>(a, st);
  }
  if constexpr (SWIGLU) {
    if (a.src_token)
      return path == MX_BIG ? launch_mx_tile_t<MxBig, true, true, true>(a, st)
                            : launch_mx_tile_t<MxMed, true, true, true>(a, st);
  }
  return path == MX_BIG ? launch_mx_tile_t<MxBig, SWIGLU, OUT_BF16, false>(a, st)
                        : launch_mx_tile_t<MxMed, SWIGLU, OUT_BF16, false>(a, st);
}

hipError_t launch_mx_ffn(const MxFfn& f, hipStream_t st) {
  const MxPath path = mx_path(f.max_rows, f.E);
  const int pH = (f.H + 127) / 128 * 4, pI = (f.I + 127) / 128 * 4;
  const MxArgs up{f.x8, f.x_scale, f.src_token, f.offsets, f.E, f.max_rows, f.w13, f.w13_scale,
                  f.H, f.I, 2 * f.I, pH, pI, f.h8, f.h_scale};
  hipError_t err = launch_mx<true, true>(up, path, st);
  if (err != hipSuccess) return err;
  const MxArgs down{f.h8, f.h_scale, nullptr, f.offsets, f.E, f.max_rows, f.w2, f.w2_scale,
                    f.I, f.H, f.H, pI, 0, f.y, nullptr};
  return f.y_dt == 1 ? launch_mx<false, true>(down, path, st)
                     : launch_mx<false, false>(down, path, st);
}

}  // namespace moe
