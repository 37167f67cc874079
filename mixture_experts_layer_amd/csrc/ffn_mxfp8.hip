// Grouped SwiGLU experts on MXFP8 rows and weights, gfx950.
//
//   h = MXFP8(SiLU(W_gate a) * (W_up a)),   y = W2 h
//
// The products run on v_mfma_scale_f32_*_f8f6f4 (the gate/up product of few
// rows on bfloat16, below), which multiplies e4m3 elements and applies one E8M0
// scale per 32 of them on either side, so the scales cost no vector
// instructions: a lane's operand register brings the scale byte of its row's
// 32-element block.  The instruction sums a block of 64 or 128 products with
// about 16 significant bits (measured: 2e-5 of the result on blocks of normal
// data, against 2^-4 of an element's own rounding) and accumulates blocks in
// float32.
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
//
// Measured on MI355X, Qwen3 shape (128 experts, H 4096, I 1536): T = 64 462 us,
// 5.3 TB/s of weights (a large copy: 5.1); T = 8192 gate/up 1.10 ms and down 0.61,
// 1.4-1.5 PFLOP/s.  There neither memory (2.6 TB/s) nor the matrix cores (busy
// 0.36-0.39) are full: 256-row tiles have one block per CU and two stages, so
// every chunk of 128 waits for the last of its own loads.
// One token of an eighth of it (I 192): 11 us in two launches, latency.
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

// One output tile: rows [r0, r1) of expert e, columns from n0 on.
template <class C, bool SWIGLU, bool OUT_BF16, bool GATHER>
__device__ __forceinline__ void mx_tile(const MxArgs& a, unsigned char* smem, int e, int r0, int r1,
                                        int n0) {
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int COLS = SWIGLU ? C::TN / 2 : C::TN;
  const uint8_t* Be = a.B + (size_t)e * a.b_rows * a.K;
  const uint8_t* Bse = a.Bs + (size_t)e * a.b_rows * a.pitch;

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
      // (64 rows per load; counted waits, beyond two stages, need them all)
      if (C::STAGES == 2 && j > 0 && 64 * j >= r1 - r0) break;
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
  // LIVE: the wave's 32-row subtiles that hold rows
  auto contract = [&](auto live_c) {
    constexpr int LIVE = decltype(live_c)::value;
    for (int ks = 0; ks < nk; ++ks) {
      if (C::STAGES > 2 && ks + 1 < nk) wait_stage_barrier<(C::STAGES - 2) * NL>();
      else wait_stage_barrier<0>();
      if (ks + C::STAGES - 1 < nk) issue(ks + C::STAGES - 1, (ks + C::STAGES - 1) % C::STAGES);
      unsigned char* sa = smem + (ks % C::STAGES) * C::SBYTES;
      const unsigned char* sb = sa + C::ABYTES;
      const int* sc = reinterpret_cast<const int*>(sb + C::BBYTES);
      const int left = a.K - ks * C::TK;
      if (left < C::TK) zero_tail(sa, left);
      if constexpr (LIVE > 0) {
        int as[C::MFM], bs[C::MFN];
        // this lane's blocks: byte 0 of the shifted dword in step 0, byte 2 in step 1
#pragma unroll
        for (int mi = 0; mi < LIVE; ++mi)
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
          for (int mi = 0; mi < LIVE; ++mi) af[mi] = frag(sa, wm * C::WTM + mi * 32, S);
#pragma unroll
          for (int mi = 0; mi < LIVE; ++mi)
#pragma unroll
            for (int ni = 0; ni < C::MFN; ++ni)
              acc[mi][ni] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  bf[ni], af[mi], acc[mi][ni], 0, 0, 2 * S, bs[ni], 2 * S, as[mi]);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
      }
    }
  };
  // (a wave without rows only loads; each case is a loop of its own)
  const int live = r1 - r0 - wm * C::WTM;
  constexpr int HALF_M = (C::MFM + 1) / 2;
  if (live > 32 * HALF_M) contract(std::integral_constant<int, C::MFM>{});
  else if (live > 32) contract(std::integral_constant<int, HALF_M>{});
  else if (live > 0) contract(std::integral_constant<int, 1>{});
  else contract(std::integral_constant<int, 0>{});

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

// Row tiles as in the bfloat16 training products: 256 rows while an expert has
// them, a last tile of at most 128 or 64 rows in a shape with a third stage, and
// those behind the expert's other tiles.
using MxT256 = MxCfg<256, 256, 2, 2, 4>;
using MxT128 = MxCfg<128, 256, 3, 2, 4>;
using MxT64 = MxCfg<64, 256, 3, 2, 4>;
constexpr int MX_TM = MxT256::TM, MX_TN = MxT256::TN;
constexpr int MX_LDS = std::max({MxT256::LDS, MxT128::LDS, MxT64::LDS});

template <bool SWIGLU, bool OUT_BF16, bool GATHER>
__global__ __launch_bounds__(512, 2) void mx_tile_kernel(MxArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  constexpr int COLS = SWIGLU ? MX_TN / 2 : MX_TN;
  const int NT = (a.N + COLS - 1) / COLS;
  RowBlock t;
  if (!row_block<MX_TM>(a.offsets, a.E, a.max_rows, NT, blockIdx.x, t)) return;
  const int r0 = t.r0, r1 = t.r1, n0 = t.n * COLS;
  if (r1 - r0 > 128) mx_tile<MxT256, SWIGLU, OUT_BF16, GATHER>(a, smem, t.e, r0, r1, n0);
  else if (r1 - r0 > 64) mx_tile<MxT128, SWIGLU, OUT_BF16, GATHER>(a, smem, t.e, r0, r1, n0);
  else mx_tile<MxT64, SWIGLU, OUT_BF16, GATHER>(a, smem, t.e, r0, r1, n0);
}

// ---------------------------------------------------------------------------
// Direct kernel: 16 rows of one expert against weights streamed from memory
// into the operands of v_mfma_scale_f32_16x16x128, or, in MX_UP, widened to
// bfloat16 and into those of v_mfma_f32_16x16x32_bf16 (weights first, so
// accumulator lane l holds columns 4 (l / 16) + i of row l % 16).  A block's 8
// waves are CW groups of KW = 8 / CW: each group takes its own output columns,
// and its waves split the contraction and meet in LDS, in wave order.  A wave
// keeps two batches of U = 2 steps of 128 in flight, one being multiplied.
//   MX_UP      8 columns of h per group: 8 gate and the matching 8 up rows
//              share an operand.  Blocks of 32 or more columns store h as
//              MXFP8; narrower ones, which do not hold whole blocks of 32,
//              store it in float32;
//   MX_DOWN    16 columns of y per group, from MXFP8 h;
//   MX_DOWN32  the same from float32 h, which the block brings to MXFP8 in LDS
//              first (the same bits).
// ---------------------------------------------------------------------------
// The 8-bit matrix instructions add their products to about 16 bits (2e-5 of a
// sum measured, whichever form).  That is far below y's own rounding, but moves
// an h that lies next to an e4m3 border over it, an eighth of its value: about one
// h in 2000.  In a batch of thousands that is noise (2.0e-3 from the formula,
// 1.7e-3 with exact sums); in a small one a single h shows.  So the gate/up
// product of few rows, which waits for memory anyway, runs on bfloat16 values
// (exact: 4 significant bits, the block's power of two folded in) whose sums are
// good to 1e-7.
enum MxMode { MX_UP, MX_DOWN, MX_DOWN32 };

// 8 e4m3 elements times the power of two of scale byte `b`, as bfloat16
__device__ __forceinline__ bf16x8_t mx_widen(uint32_t lo, uint32_t hi, uint32_t b) {
  const float s = __uint_as_float(b << 23);      // (only the exponent is read)
  const bf16x2_v p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
  const bf16x2_v p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
  const bf16x2_v p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
  const bf16x2_v p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
  const uint4 v = make_uint4(__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                             __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3));
  return __builtin_bit_cast(bf16x8_t, v);
}

__device__ __forceinline__ i32x4_v ld_nt16(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const i32x4_v*>(p));
}

constexpr int MXD_MAX_LDS_K = 2048;    // contraction of MX_DOWN32: h rows in LDS

template <int MODE, bool OUT_BF16, int CW>
__global__ __launch_bounds__(512, 4) void mx_direct_kernel(MxArgs a) {
  constexpr int COLS = MODE == MX_UP ? 8 : 16, U = 2, KW = 8 / CW, RED = 4 * 65;
  constexpr bool QUANT = MODE == MX_UP && CW * COLS >= 32;
  extern __shared__ __attribute__((aligned(16))) unsigned char hbuf[];   // MX_DOWN32
  __shared__ float red[8 * RED];
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
  // the row's source is loaded here and turned into addresses only once the
  // first weights are on their way
  int src = a.src_token ? a.src_token[row] : row;
  const uint8_t* xa = a.A;
  const uint8_t* xs = a.As;
  // (a group past the last column re-reads column 0; N is a multiple of 32)
  const int nc = n0 < a.N ? n0 : 0;
  const size_t wrow = (size_t)t.e * a.b_rows +
                      (MODE == MX_UP ? nc + (lr & 7) + (lr >> 3) * a.N : nc + lr);
  const uint8_t* wp = a.B + wrow * a.K;
  const uint8_t* ws = a.Bs + wrow * a.pitch;

  const int steps = (a.K + 127) / 128;
  const int s0 = steps * kw / KW, s1 = steps * (kw + 1) / KW;
  const int hp = steps * 128 + 16, hsp = steps * 4;       // MX_DOWN32: LDS rows of h, of scales
  unsigned char* hscale = hbuf + 16 * hp;
  // A batch's rows ride with its weights: loads return in order, so rows asked
  // for after the next batch's weights would wait for those.
  struct Batch {
    i32x4_v w[U][2], x[U][2];
    int wsc[U], xsc[U];
  };
  // (a step past this wave's share re-reads its last and is not multiplied;
  // 16 bytes past the contraction's end re-read the row's first)
  auto load_w = [&](Batch& b, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = min(s + u, max(s1, 1) - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = st * 128 + h * 64 + lg * 16;
        b.w[u][h] = ld_nt16(wp + (k < a.K ? k : 0));
      }
      b.wsc[u] = *reinterpret_cast<const int*>(ws + st * 4);
    }
  };
  auto load_x = [&](Batch& b, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = min(s + u, max(s1, 1) - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = st * 128 + h * 64 + lg * 16;
        if constexpr (MODE == MX_DOWN32)
          b.x[u][h] = *reinterpret_cast<const i32x4_v*>(hbuf + lr * hp + k);
        else
          b.x[u][h] = *reinterpret_cast<const i32x4_v*>(xa + (k < a.K ? k : 0));
      }
      b.xsc[u] = *reinterpret_cast<const int*>(
          MODE == MX_DOWN32 ? hscale + lr * hsp + st * 4 : xs + st * 4);
    }
  };
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](Batch& b, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
      const int left = a.K - (s + u) * 128;
      if (left < 128) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h * 64 + lg * 16 >= left) b.x[u][h] = b.w[u][h] = i32x4_v{0, 0, 0, 0};
      }
      const uint32_t xs4 = mx_valid_scales(b.xsc[u], left >> 5);
      const uint32_t ws4 = mx_valid_scales(b.wsc[u], left >> 5);
      if constexpr (MODE == MX_UP) {
        // (16 bytes at 64 h + 16 lg: block 2 h + lg / 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int sh = 16 * h + 8 * (lg >> 1);
          const uint32_t xb = (xs4 >> sh) & 0xff, wb = (ws4 >> sh) & 0xff;
          const i32x4_v x = b.x[u][h], w = b.w[u][h];
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_widen(w[0], w[1], wb),
                                                        mx_widen(x[0], x[1], xb), acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_widen(w[2], w[3], wb),
                                                        mx_widen(x[2], x[3], xb), acc, 0, 0, 0);
        }
        continue;
      }
      const i32x8_v xf = __builtin_shufflevector(b.x[u][0], b.x[u][1], 0, 1, 2, 3, 4, 5, 6, 7);
      const i32x8_v wf = __builtin_shufflevector(b.w[u][0], b.w[u][1], 0, 1, 2, 3, 4, 5, 6, 7);
      const int xsv = (int)(xs4 >> (8 * lg));
      const int wsv = (int)(ws4 >> (8 * lg));
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc, 0, 0, 0, wsv, 0, xsv);
    }
  };
  Batch b0, b1;
  load_w(b0, s0);
  if constexpr (MODE == MX_DOWN32) {
    // the rows' h to MXFP8: 8 elements per thread, four threads to a block of
    // 32; rows past the tile and steps past the contraction are zeros
    const int n8 = steps * 16;
    for (int i = threadIdx.x; i < 16 * n8; i += 512) {
      const int m = i / n8, c = i - m * n8;
      float f[8];
      if (r0 + m < r1 && c * 8 < a.K) {
        Chunk<false> v;
        v.load(a.A + (size_t)(r0 + m) * a.K * 4, c);
        v.get(f);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
      }
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
      const uint32_t b8 = mx_scale_byte(quad_max(mx));
      const float k = mx_inv_scale(b8);
      *reinterpret_cast<uint2*>(hbuf + m * hp + c * 8) =
          make_uint2(mx_pack4(f[0] * k, f[1] * k, f[2] * k, f[3] * k),
                     mx_pack4(f[4] * k, f[5] * k, f[6] * k, f[7] * k));
      if ((c & 3) == 0) hscale[m * hsp + (c >> 2)] = (unsigned char)b8;
    }
    __syncthreads();
  } else {
    asm volatile("" : "+v"(src)::"memory");      // the wait for the source lands here
    xa = a.A + (size_t)max(src, 0) * a.K;
    xs = a.As + (size_t)max(src, 0) * a.pitch;
  }
  load_x(b0, s0);
  for (int s = s0; s < s1; s += 2 * U) {
    if (s + U < s1) {
      load_w(b1, s + U);
      load_x(b1, s + U);
    }
    multiply(b0, s);
    if (s + U >= s1) break;
    if (s + 2 * U < s1) {
      load_w(b0, s + 2 * U);
      load_x(b0, s + 2 * U);
    }
    multiply(b1, s + U);
  }

#pragma unroll
  for (int q = 0; q < 4; ++q) red[wid * RED + q * 65 + lane] = acc[q];
  __syncthreads();
  // outputs of the block: 16 rows x CW * COLS columns, columns fastest
  constexpr int BC = CW * COLS;
  for (int o = threadIdx.x; o < 16 * BC; o += 512) {
    const int m = o / BC, c = o - m * BC, g = c / COLS, n = c - g * COLS;
    const int at = (n & 3) * 65 + m + 16 * (n >> 2);
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const float* p = red + (g * KW + k) * RED + at;
      v += p[0];
      if (MODE == MX_UP) u += p[MODE == MX_UP ? 32 : 0];   // the up sums lie 32 lanes on
    }
    const bool live = r0 + m < r1 && nb + c < a.N;
    const size_t yi = (size_t)(r0 + m) * a.N + nb + c;
    if constexpr (QUANT) {
      // 32 consecutive lanes hold a row's block (BC is a multiple of 32, and
      // whole waves take part)
      const float h = silu_fast(v) * u;
      float mx = fabsf(h);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
      const uint32_t b8 = mx_scale_byte(mx);
      const float hk = h * mx_inv_scale(b8);
      if (live) {
        static_cast<uint8_t*>(a.Y)[yi] = (uint8_t)(mx_pack4(hk, hk, hk, hk) & 0xff);
        if ((c & 31) == 0) a.Ys[(size_t)(r0 + m) * a.out_pitch + ((nb + c) >> 5)] = (uint8_t)b8;
      }
    } else if (live) {
      if constexpr (MODE == MX_UP) static_cast<float*>(a.Y)[yi] = silu_fast(v) * u;
      else if (OUT_BF16) static_cast<bf16_t*>(a.Y)[yi] = (bf16_t)(cvt_bf16x2(v, v) & 0xffff);
      else static_cast<float*>(a.Y)[yi] = v;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static long long mx_row_tiles(int max_rows, int E, int BM) {
  const long long bound = ((long long)max_rows + (long long)E * (BM - 1)) / BM;
  return bound < max_rows ? bound : max_rows;
}

// (the direct kernel takes few rows, so fewer and smaller blocks)
bool mx_fits(int max_rows, int E, int H, int I) {
  const long long cols = std::max((I + MX_TN / 2 - 1) / (MX_TN / 2), (H + MX_TN - 1) / MX_TN);
  return mx_row_tiles(max_rows, E, MX_TM) * cols * 512 < (1ll << 32);
}

template <bool SWIGLU, bool OUT_BF16, bool GATHER>
static hipError_t launch_mx_tile_t(const MxArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> lds_set{0};
  hipError_t err = ensure_lds_limit(
      reinterpret_cast<const void*>(&mx_tile_kernel<SWIGLU, OUT_BF16, GATHER>), MX_LDS, lds_set);
  if (err != hipSuccess) return err;
  constexpr int cols = SWIGLU ? MX_TN / 2 : MX_TN;
  const long long grid = mx_row_tiles(a.max_rows, a.E, MX_TM) * ((a.N + cols - 1) / cols);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  mx_tile_kernel<SWIGLU, OUT_BF16, GATHER><<<(unsigned)grid, 512, MX_LDS, st>>>(a);
  return hipGetLastError();
}

template <int MODE, bool OUT_BF16, int CW>
static hipError_t launch_mx_direct_t(const MxArgs& a, hipStream_t st) {
  constexpr int cols = CW * (MODE == MX_UP ? 8 : 16);
  const long long grid = mx_row_tiles(a.max_rows, a.E, 16) * ((a.N + cols - 1) / cols);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  int lds = 0;
  if (MODE == MX_DOWN32) {
    const int steps = (a.K + 127) / 128;
    lds = 16 * (steps * 128 + 16) + 16 * steps * 4;
  }
  mx_direct_kernel<MODE, OUT_BF16, CW><<<(unsigned)grid, 512, lds, st>>>(a);
  return hipGetLastError();
}
// Which kernel takes each product.  Measured on MI355X, replayed from a graph
// (us; up kernel / down kernel; d<n>: direct with n column groups per block; the
// direct gate/up products on bfloat16 take 1-3% more of the whole):
//   I/P = 192, 8 experts x 1 row:     d1/d8 11.4  d2/d8 13.7  d4/d8 20.1  tiles 40.2
//     49 experts:                     d1/d8 42.4  d2/d8 44.8  tiles 59.2
//     87 experts:                     d1/d8 69.9  tiles/d8 64.4  tiles 74.8
//   I = 1536, 8 experts:              d2/d8 44.9  d1/d8 45.9  tiles 51.3
//     15 experts:                     d2/d8 73.8  tiles 67.2
//   I = 2048, H = 7168, 8 experts:    d4/tiles 88.7  d2/d8 98.4  tiles 110
//     13 experts:                     d2/d8 155   tiles 138
//   I = 14336, 2 experts:             tiles/d2 74.3  tiles/d8 147  d4/d8 173  tiles 207
//     8 experts, 4 rows each:         tiles/d2 345   tiles 367
//   many rows per expert (direct / tiles; outputs as row tiles of 16 x I / 8):
//     248:  936 rows, 4 experts, I 32, H 2976     18.3 / 52.4
//     256:  1024 rows, 1 expert, I 32, H 768      9.8 / 23.0
//     1260: 330 rows, 1 expert, I 480, H 192      17.3 / 23.1
//     1728: 1024 rows, 8 experts, I 192, H 4096   64.2 / 64.5
//     2568: 1710 rows, 1 expert, I 192, H 128     25.4 / 17.8
//     5280: 7016 rows, 4 experts, I 96, H 1312    92.7 / 33.7
// The tiled kernel streams faster (5.1 against 4.1 TB/s) but needs a block of
// 1 MB of weights per CU; a contraction of one or two steps gains nothing from
// its pipeline; and the direct kernel's 16-row tiles read the weights again
// for every 16 rows.
constexpr int MX_MIN_BLOCKS = 160;    // gate/up tiles below which the direct kernel streams faster
struct MxPlan {
  bool up_direct, down_direct;
  int cw_up, cw_down;     // direct kernels: column groups per block
  bool h_float;           // h in float32 between the products
};
static MxPlan mx_plan(int max_rows, int E, int H, int I) {
  MxPlan p{};
  const int mean = max_rows / E + (max_rows % E != 0);
  // experts with rows, were every row's expert drawn alike, and their row tiles
  const double touched = E * (1.0 - __builtin_pow(1.0 - 1.0 / E, (double)max_rows));
  const double tiles = std::max(touched, max_rows / 128.0);
  // few rows per expert, or so few outputs of the gate/up product that 8-column
  // blocks of 16 rows do not fill the CUs
  const bool few = mean <= 64 || (max_rows / 16 + touched) * (I / 8) <= 1536;
  p.up_direct = few && tiles * ((I + 127) / 128) < MX_MIN_BLOCKS;
  p.down_direct = few && (I <= 256 || tiles * ((H + 255) / 256) < 256);
  const int steps = (I + 127) / 128;
  p.cw_down = steps <= 16 ? 8 : steps <= 48 ? 4 : 2;
  p.cw_up = 4;
  if (p.up_direct && p.down_direct && I <= MXD_MAX_LDS_K)
    p.cw_up = touched * (I / 8) < 1024 ? 1 : 2;
  p.h_float = p.up_direct && p.cw_up < 4;
  return p;
}

template <bool OUT_BF16>
static hipError_t launch_mx_down(const MxArgs& a, const MxPlan& p, hipStream_t st) {
  if (!p.down_direct) return launch_mx_tile_t<false, OUT_BF16, false>(a, st);
  if (p.h_float) return launch_mx_direct_t<MX_DOWN32, OUT_BF16, 8>(a, st);   // I is short there
  return p.cw_down == 8   ? launch_mx_direct_t<MX_DOWN, OUT_BF16, 8>(a, st)
         : p.cw_down == 4 ? launch_mx_direct_t<MX_DOWN, OUT_BF16, 4>(a, st)
                          : launch_mx_direct_t<MX_DOWN, OUT_BF16, 2>(a, st);
}

// h is float32 only under a direct up kernel, so with fewer than
// MX_MIN_BLOCKS / ceil(I / 128) row tiles, which max_rows / 128 never exceeds.
size_t mx_float_rows(int I) { return (size_t)128 * MX_MIN_BLOCKS / ((I + 127) / 128); }

hipError_t launch_mx_ffn(const MxFfn& f, hipStream_t st) {
  const MxPlan p = mx_plan(f.max_rows, f.E, f.H, f.I);
  const int pH = (f.H + 127) / 128 * 4, pI = (f.I + 127) / 128 * 4;
  const MxArgs up{f.x8, f.x_scale, f.src_token, f.offsets, f.E, f.max_rows, f.w13, f.w13_scale,
                  f.H, f.I, 2 * f.I, pH, pI, f.h8, f.h_scale};
  const hipError_t err = !p.up_direct  ? f.src_token ? launch_mx_tile_t<true, true, true>(up, st)
                                                     : launch_mx_tile_t<true, true, false>(up, st)
                         : p.cw_up == 1 ? launch_mx_direct_t<MX_UP, true, 1>(up, st)
                         : p.cw_up == 2 ? launch_mx_direct_t<MX_UP, true, 2>(up, st)
                                        : launch_mx_direct_t<MX_UP, true, 4>(up, st);
  if (err != hipSuccess) return err;
  const MxArgs down{f.h8, f.h_scale, nullptr, f.offsets, f.E, f.max_rows, f.w2, f.w2_scale,
                    f.I, f.H, f.H, pI, 0, f.y, nullptr};
  return f.y_dt == 1 ? launch_mx_down<true>(down, p, st) : launch_mx_down<false>(down, p, st);
}

}  // namespace moe
