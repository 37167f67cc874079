// The grouped SwiGLU experts in training, gfx950: the forward pass that keeps
// the gate and up projections, and the backward pass.
//
// Six matrix products over the same ragged rows (R rows of expert e, a the
// gathered token rows):
//
//   gate/up   [g u] = a W13^T           rows x (2I), over H      + SwiGLU
//   down      y = h W2^T                rows x H,    over I
//   dh        dh = dy W2                rows x I,    over H      + its backward
//   dx        dx = [dg du] W13          rows x H,    over 2I
//   dW2       dW2 = dy^T h              H x I,       over rows
//   dW13      dW13 = [dg du]^T a        2I x H,      over rows
//
// One kernel computes them all: a tile of TM x TN outputs per block, operands
// staged through LDS in chunks of TK = 64 along the contraction, products by
// v_mfma_f32_32x32x16_bf16.  What differs is how an operand lies in memory:
//
//   contraction contiguous (KC): LDS holds [row][64], a fragment is one 16-byte
//     LDS read of a row's 8 consecutive elements;
//   contraction across rows (MC): LDS holds [k][columns] as in memory, and
//     ds_read_b64_tr_b16 transposes on the way to the registers -- each
//     16-lane group reads 4 k-rows of 16 columns and lane i receives column
//     i's 4 values -- so no transposed copy of a weight, a gradient or an
//     activation is ever written.
//
// Both reach LDS by 16-byte direct loads (1 KB per wave instruction).
//
// Measured on MI355X.  Mixtral shape, 8 experts, T = 4096 (R = 8192 rows), gu of 16
// bits: gate/up 1.98 ms, down 0.95, dh 1.14, dx 1.83, both weight gradients 3.07:
// 0.84 to 1.05 PFLOP/s, matrix cores busy 0.49-0.55 at 1.84-1.91 GHz (dh 0.43: its
// epilogue moves 1.2 GB; with a float32 gu 1.6 GB, dh 1.21 ms and gate/up 2.00).
// Qwen3 shape, 128 experts, 32 rows each: bound by the weights and their
// gradients, 14.5 GB in 2.63 ms.
#include <algorithm>
#include <type_traits>

#include "moe_kernels.h"
#include "moe_ops_device.h"
#include "moe_ops_kernels.h"

namespace moe {

typedef _Float16 f16x2_v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_v __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8_t tr_join(u32x2_v lo, u32x2_v hi) {
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3));
}

__device__ __forceinline__ uint32_t lds_addr(const unsigned char* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) unsigned char*)p;
}

enum Epilogue { EPI_STORE, EPI_SWIGLU, EPI_DSWIGLU };

struct GemmArgs {
  const bf16_t* A;            // rows of the outputs' rows (or, in a weight gradient, columns)
  const bf16_t* B;
  long long lda, ldb;         // elements between memory rows
  long long b_stride;         // elements between experts' B (weights)
  const int32_t* src_token;   // GATHER: row r of A is row src_token[r]
  const int32_t* offsets;
  int E, max_rows;
  int M, N, K;                // rows of a weight gradient; output columns; contraction (weights)
  int up_off;                 // EPI_SWIGLU: up rows of B; EPI_DSWIGLU: up columns of gu
  bf16_t* out;                // outputs; EPI_DSWIGLU: [dg du]
  long long ldo;
  long long out_stride;       // elements between experts' outputs (weight gradients)
  bf16_t* out2;               // EPI_SWIGLU, EPI_DSWIGLU: h [rows][N]
  void* gu;                   // [rows][2 N] of EPI_SWIGLU (written) and EPI_DSWIGLU (read)
  bool gu16;                  // its form: 16 bits per value, else float32
};

// Tile shape: TM x TN outputs, STAGES buffers of 64 along the contraction,
// WM x WN waves of (TM / WM) x (TN / WN) outputs each.
template <int TM_, int TN_, int TK_, int STAGES_, int WM_, int WN_>
struct GemmCfg {
  static constexpr int TM = TM_, TN = TN_, TK = TK_, STAGES = STAGES_, WM = WM_, WN = WN_;
  static constexpr int NW = WM * WN, NTHR = NW * 64;
  static constexpr int WTM = TM / WM, WTN = TN / WN, MFM = WTM / 32, MFN = WTN / 32;
  static constexpr int ABYTES = TM * TK * 2, BBYTES = TN * TK * 2, SBYTES = ABYTES + BBYTES;
  static constexpr int ALOADS = ABYTES / 1024 / NW, BLOADS = BBYTES / 1024 / NW;
  static constexpr int PITCH = TN * 2 + 16;       // staged output row
  static constexpr int LDS = STAGES * SBYTES > TM * PITCH ? STAGES * SBYTES : TM * PITCH;
  static_assert(ALOADS * NW * 1024 == ABYTES && BLOADS * NW * 1024 == BBYTES, "load split");
  static_assert(WTM % 32 == 0 && WTN % 64 == 0, "wave tile");
  static_assert(LDS <= 160 * 1024, "LDS per block");
};

// KC tile [row][TK]: 16-byte chunks, chunk c of row r at c ^ (r / 2 % 8) for 8
// chunks per row, c ^ (r / 4 % 4) for 4: the 16 lanes that read one chunk of 16
// rows then cover the banks once.
template <int TK>
__device__ __forceinline__ int kc_swz(int r) {
  return TK == 64 ? (r >> 1) & 7 : (r >> 2) & 3;
}
// MC tile [k][TN or TM columns]: 64-byte segments, segment s of row k at
// s ^ (k % 4): the four k-rows of 64 bytes that half a wave reads lie in
// different quarters of the banks.
__device__ __forceinline__ int mc_chunk(int k, int chunk) { return chunk ^ ((k & 3) << 2); }

// Transposing LDS reads of N fragments (32 columns x 16 k-rows each, ROW bytes
// per k-row) at LDS addresses at[] + OFF.  One asm block that ends with the
// wait for what it reads: the compiler's own bookkeeping makes the builtin
// form wait for every LDS-direct load in flight, which emptied the load
// pipeline at each chunk (the products by W2 and W13 ran 20% below the
// transpose-free ones).  The other wave of the SIMD multiplies meanwhile.
template <int OFF, int ROW>
__device__ __forceinline__ void tr_read(const uint32_t (&at)[2], bf16x8_t (&f)[2]) {
  u32x2_v a0, a1, b0, b1;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
      "ds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
      "ds_read_b64_tr_b16 %2, %5 offset:%6\n\t"
      "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(a0), "=&v"(a1), "=&v"(b0), "=&v"(b1)
      : "v"(at[0]), "v"(at[1]), "n"(OFF), "n"(OFF + 4 * ROW)
      : "memory");
  f[0] = tr_join(a0, a1);
  f[1] = tr_join(b0, b1);
}
template <int OFF, int ROW>
__device__ __forceinline__ void tr_read(const uint32_t (&at)[4], bf16x8_t (&f)[4]) {
  u32x2_v a0, a1, b0, b1, c0, c1, d0, d1;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
      "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
      "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
      "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
      "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
      "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(a0), "=&v"(a1), "=&v"(b0), "=&v"(b1), "=&v"(c0), "=&v"(c1), "=&v"(d0), "=&v"(d1)
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF), "n"(OFF + 4 * ROW)
      : "memory");
  f[0] = tr_join(a0, a1);
  f[1] = tr_join(b0, b1);
  f[2] = tr_join(c0, c1);
  f[3] = tr_join(d0, d1);
}

// Four consecutive elements, aligned to them.
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}

// The 16-bit form of gu: four consecutive values, scaled by a power of two so
// that the largest lies in [2^-8, 2^-7), as IEEE halves, whose two upper
// exponent bits are then zero; in their place stand the 8 bits of the largest
// value's float32 exponent, two in each half.  In bfloat16, in the same memory,
// a value would keep 8 significant bits, here 11 (gradients 3.5e-3 from float64
// there, 2.4e-3 here), and the range is float32's all the same.  A
// value that is not finite takes the group's largest code and exponent 255,
// which reads as infinite.
__device__ __forceinline__ uint2 gu_pack4(float a, float b, float c, float d) {
  const uint32_t top = max(max(__float_as_uint(a) & 0x7f800000u, __float_as_uint(b) & 0x7f800000u),
                           max(__float_as_uint(c) & 0x7f800000u, __float_as_uint(d) & 0x7f800000u));
  const int e = (int)(top >> 23);
  constexpr float MOST = 0x1.ffcp-8f;      // the largest half below 2^-7
  auto half = [&](float v) { return fminf(fmaxf(ldexpf(v, 119 - e), -MOST), MOST); };
  const uint32_t lo =
      __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_v){half(a), half(b)}, f16x2_v));
  const uint32_t hi =
      __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_v){half(c), half(d)}, f16x2_v));
  return make_uint2(lo | (e & 3) << 13 | (e >> 2 & 3) << 29, hi | (e >> 4 & 3) << 13 | (e >> 6) << 29);
}
// (a row of the 16-bit form)
__device__ __forceinline__ void load4(const bf16_t* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const int e = (int)((v.x >> 13 & 3) | (v.x >> 27 & 12) | (v.y >> 9 & 48) | (v.y >> 23 & 192));
  const f32x2_v lo = __builtin_convertvector(__builtin_bit_cast(f16x2_v, v.x & 0x9fff9fffu), f32x2_v);
  const f32x2_v hi = __builtin_convertvector(__builtin_bit_cast(f16x2_v, v.y & 0x9fff9fffu), f32x2_v);
  f[0] = ldexpf(lo[0], e - 119); f[1] = ldexpf(lo[1], e - 119);
  f[2] = ldexpf(hi[0], e - 119); f[3] = ldexpf(hi[1], e - 119);
}

// One output tile: rows [r0, r1) (of expert e; in a weight gradient, rows of the
// parameter), columns from n0 on, a contraction of K (from memory row krow0 on).
template <class C, bool WGRAD, bool BKC, int EPI, bool GATHER>
__device__ __forceinline__ void gemm_tile(const GemmArgs& a, unsigned char* smem, int e, int r0,
                                          int r1, int n0, int K, int krow0) {
  constexpr bool AKC = !WGRAD;
  static_assert(!WGRAD || (!BKC && EPI == EPI_STORE && !GATHER), "weight gradients");
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int COLS = EPI == EPI_SWIGLU ? C::TN / 2 : C::TN;
  const bf16_t* Be = WGRAD ? a.B : a.B + (size_t)e * a.b_stride;

  // ---- lanes' sources.  Rows and columns past the end read the last one (or
  // the first column): their products are not stored.
  // KC: one load covers KRPI rows; the chunk this lane loads of its row is the
  // same for every load (rows step by NW * KRPI, a multiple of 16)
  constexpr int KCPR = C::TK / 8, KRPI = 64 / KCPR;
  static_assert(C::NW == 8, "chunk of a lane");
  const int kchunk = (lane % KCPR) ^ kc_swz<C::TK>(wid * KRPI + lane / KCPR);
  const unsigned char* abase;
  const unsigned char* bbase;
  uint32_t ao[C::ALOADS], bo[C::BLOADS];
  const unsigned char* ap[AKC && GATHER ? C::ALOADS : 1];
  if constexpr (AKC) {
    abase = reinterpret_cast<const unsigned char*>(a.A + (size_t)r0 * a.lda);
#pragma unroll
    for (int j = 0; j < C::ALOADS; ++j) {
      const int rt = (wid + C::NW * j) * KRPI + lane / KCPR;
      const int row = min(r0 + rt, r1 - 1);
      ao[j] = (uint32_t)((size_t)(row - r0) * a.lda * 2 + kchunk * 16);
      if constexpr (GATHER)
        ap[j] = reinterpret_cast<const unsigned char*>(a.A + (size_t)max(a.src_token[row], 0) * a.lda) +
                kchunk * 16;
    }
  } else {
    constexpr int CPR = C::TM / 8, RPI = 64 / CPR;
    abase = reinterpret_cast<const unsigned char*>(a.A + (size_t)krow0 * a.lda);
#pragma unroll
    for (int j = 0; j < C::ALOADS; ++j) {
      const int k = (wid + C::NW * j) * RPI + lane / CPR;
      const int col = r0 + mc_chunk(k, lane % CPR) * 8;
      ao[j] = (uint32_t)((size_t)k * a.lda * 2 + (col < a.M ? col : 0) * 2);
    }
  }
  constexpr int BCPR = C::TN / 8, BRPI = 64 / BCPR;
  if constexpr (BKC) {
    bbase = reinterpret_cast<const unsigned char*>(Be);
#pragma unroll
    for (int j = 0; j < C::BLOADS; ++j) {
      const int rt = (wid + C::NW * j) * KRPI + lane / KCPR;
      int row;
      if (EPI == EPI_SWIGLU)
        row = rt < COLS ? min(n0 + rt, a.N - 1) : a.up_off + min(n0 + rt - COLS, a.N - 1);
      else
        row = min(n0 + rt, a.N - 1);
      bo[j] = (uint32_t)((size_t)row * a.ldb * 2 + kchunk * 16);
    }
  } else {
    bbase = reinterpret_cast<const unsigned char*>(WGRAD ? Be + (size_t)krow0 * a.ldb : Be);
#pragma unroll
    for (int j = 0; j < C::BLOADS; ++j) {
      const int k = (wid + C::NW * j) * BRPI + lane / BCPR;
      const int col = n0 + mc_chunk(k, lane % BCPR) * 8;
      bo[j] = (uint32_t)((size_t)k * a.ldb * 2 + (col < a.N ? col : 0) * 2);
    }
  }

  const int nk = (K + C::TK - 1) / C::TK;
  // `part`: the last chunk holds fewer than TK; what lies past the end re-reads
  // valid rows or columns (and is zeroed in LDS before the products)
  auto issue_as = [&](int ks, int buf, auto part_c, bool do_a, bool do_b) {
    constexpr bool PART = decltype(part_c)::value;
    unsigned char* sa = smem + buf * C::SBYTES + wid * 1024;
    unsigned char* sb = sa + C::ABYTES;
    const int left = K - ks * C::TK;
    const uint32_t kback = PART && kchunk * 8 >= left ? kchunk * 16 : 0;   // KC: to chunk 0
    auto mc_back = [&](int k, long long ld) {                              // MC: to the last row
      return PART && k >= left ? (uint32_t)((k - left + 1) * ld * 2) : 0u;
    };
    if (do_a) {
      if constexpr (AKC) {
#pragma unroll
        for (int j = 0; j < C::ALOADS; ++j) {
          // (counted waits, beyond two stages, need them all)
          if (C::STAGES == 2 && j > 0 && C::NW * KRPI * j >= r1 - r0) break;
          if constexpr (GATHER)
            __builtin_amdgcn_global_load_lds((gbl_void_t*)(ap[j] + (size_t)ks * (C::TK * 2) - kback),
                                             (lds_void_t*)(sa + C::NW * j * 1024), 16, 0, 0);
          else
            buffer_load_lds16(abase, 0xffffffffu, sa + C::NW * j * 1024, ao[j] - kback,
                              (uint32_t)ks * (C::TK * 2));
        }
      } else {
        constexpr int CPR = C::TM / 8, RPI = 64 / CPR;
        const unsigned char* base = abase + (size_t)ks * C::TK * a.lda * 2;
#pragma unroll
        for (int j = 0; j < C::ALOADS; ++j)
          buffer_load_lds16(base, 0xffffffffu, sa + C::NW * j * 1024,
                            ao[j] - mc_back((wid + C::NW * j) * RPI + lane / CPR, a.lda), 0);
      }
    }
    if (!do_b) return;
    if constexpr (BKC) {
#pragma unroll
      for (int j = 0; j < C::BLOADS; ++j)
        buffer_load_lds16(bbase, 0xffffffffu, sb + C::NW * j * 1024, bo[j] - kback,
                          (uint32_t)ks * (C::TK * 2));
    } else {
      const unsigned char* base = bbase + (size_t)ks * C::TK * a.ldb * 2;
#pragma unroll
      for (int j = 0; j < C::BLOADS; ++j)
        buffer_load_lds16(base, 0xffffffffu, sb + C::NW * j * 1024,
                          bo[j] - mc_back((wid + C::NW * j) * BRPI + lane / BCPR, a.ldb), 0);
    }
  };
  auto issue = [&](int ks, int buf, bool do_a = true, bool do_b = true) {
    if (K - ks * C::TK >= C::TK) issue_as(ks, buf, std::false_type{}, do_a, do_b);
    else issue_as(ks, buf, std::true_type{}, do_a, do_b);
  };
  // zero what the last chunk holds past its `left` rows or columns
  auto zero_tail = [&](unsigned char* sa, unsigned char* sb, int left) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    auto kc = [&](unsigned char* p, int rows) {
      for (int i = threadIdx.x; i < rows * KCPR; i += C::NTHR)
        if (((i % KCPR) ^ kc_swz<C::TK>(i / KCPR)) * 8 >= left) reinterpret_cast<uint4*>(p)[i] = z;
    };
    auto mc = [&](unsigned char* p, int cols) {
      for (int i = left * (cols / 8) + threadIdx.x; i < C::TK * (cols / 8); i += C::NTHR)
        reinterpret_cast<uint4*>(p)[i] = z;
    };
    if constexpr (AKC) kc(sa, C::TM); else mc(sa, C::TM);
    if constexpr (BKC) kc(sb, C::TN); else mc(sb, C::TN);
    lds_barrier();
  };

  // ---- fragments
  const int wm = wid / C::WN, wn = wid % C::WN;
  const int lrow = lane & 31, khalf = lane >> 5;
  const int trk = 8 * khalf + ((lane & 15) >> 2);                        // MC: this lane's k-row,
  const int trc = ((lane >> 4) & 1) * 32 + (lane & 3) * 8;               // byte inside a segment
  int nbase[C::MFN];
#pragma unroll
  for (int ni = 0; ni < C::MFN; ++ni) {
    if (EPI == EPI_SWIGLU) {
      constexpr int HALF = C::MFN / 2;
      nbase[ni] = (ni < HALF ? 0 : COLS) + wn * (C::WTN / 2) + (ni % HALF) * 32;
    } else {
      nbase[ni] = wn * C::WTN + ni * 32;
    }
  }
  int aoff[C::MFM], asw[C::MFM], boff[C::MFN], bsw[C::MFN];
#pragma unroll
  for (int mi = 0; mi < C::MFM; ++mi) {
    const int r = wm * C::WTM + mi * 32;
    asw[mi] = kc_swz<C::TK>(r + lrow);
    aoff[mi] = AKC ? (r + lrow) * (C::TK * 2)
                   : trk * (C::TM * 2) + (((r >> 5) ^ (trk & 3)) << 6) + trc;
  }
#pragma unroll
  for (int ni = 0; ni < C::MFN; ++ni) {
    const int r = nbase[ni];
    bsw[ni] = kc_swz<C::TK>(r + lrow);
    boff[ni] = BKC ? (r + lrow) * (C::TK * 2)
                   : trk * (C::TN * 2) + (((r >> 5) ^ (trk & 3)) << 6) + trc;
  }
  // fragments of step KK (16 along the contraction); KC by ordinary LDS reads,
  // which the compiler schedules, MC by tr_read
  auto load_a = [&](const unsigned char* sa, auto kk_c, bf16x8_t (&af)[C::MFM], auto live_c) {
    constexpr int KK = decltype(kk_c)::value;
    if constexpr (AKC) {
#pragma unroll
      for (int mi = 0; mi < decltype(live_c)::value; ++mi)
        af[mi] = *reinterpret_cast<const bf16x8_t*>(sa + aoff[mi] +
                                                    (((KK * 2 + khalf) ^ asw[mi]) * 16));
    } else {
      uint32_t at[C::MFM];
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi) at[mi] = lds_addr(sa) + aoff[mi];
      tr_read<KK * 16 * C::TM * 2, C::TM * 2>(at, af);
    }
  };
  auto load_b = [&](const unsigned char* sb, auto kk_c, bf16x8_t (&bf)[C::MFN]) {
    constexpr int KK = decltype(kk_c)::value;
    if constexpr (BKC) {
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni)
        bf[ni] = *reinterpret_cast<const bf16x8_t*>(sb + boff[ni] +
                                                    (((KK * 2 + khalf) ^ bsw[ni]) * 16));
    } else {
      uint32_t at[C::MFN];
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni) at[ni] = lds_addr(sb) + boff[ni];
      tr_read<KK * 16 * C::TN * 2, C::TN * 2>(at, bf);
    }
  };

  f32x16_t acc[C::MFM][C::MFN];
#pragma unroll
  for (int i = 0; i < C::MFM; ++i)
#pragma unroll
    for (int j = 0; j < C::MFN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // LIVE: the wave's 32-row subtiles that hold rows
  auto multiply = [&](const unsigned char* sa, const unsigned char* sb, auto live_c, auto&& first,
                      auto&& second) {
    constexpr int STEPS = C::TK / 16, LIVE = decltype(live_c)::value;
    if constexpr (LIVE > 0) {
      bf16x8_t af[2][C::MFM], bf[2][C::MFN];
      auto load = [&](auto kk_c) {
        constexpr int KK = decltype(kk_c)::value;
        load_a(sa, kk_c, af[KK & 1], live_c);
        load_b(sb, kk_c, bf[KK & 1]);
      };
      auto step = [&](auto kk_c) {
        constexpr int KK = decltype(kk_c)::value, CUR = KK & 1;
        // KC only: the next step's LDS reads go out ahead of this step's
        // products; transposed reads wait where they stand
        constexpr bool AHEAD = AKC && BKC;
        if constexpr (!AHEAD) load(kk_c);
        else if constexpr (KK == 0) load(kk_c);
        if constexpr (AHEAD && KK + 1 < STEPS) load(std::integral_constant<int, KK + 1>{});
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (KK == 0) first();
        if constexpr (KK == 1) second();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int mi = 0; mi < LIVE; ++mi)
#pragma unroll
          for (int ni = 0; ni < C::MFN; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[CUR][ni], af[CUR][mi],
                                                                  acc[mi][ni], 0, 0, 0);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      if constexpr (STEPS > 2) {
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
      }
    }
  };

  constexpr int NL = C::ALOADS + C::BLOADS;
  if (nk > 0) {
#pragma unroll
    for (int s0 = 0; s0 < C::STAGES - 1; ++s0)
      if (s0 < nk) issue(s0, s0);
  }
  auto contract = [&](auto live_c) {
    for (int ks = 0; ks < nk; ++ks) {
      // chunk ks has landed once at most the younger chunks' loads are
      // outstanding; past the barrier that holds for every wave, and nobody
      // still reads the buffer refilled below
      static_assert(C::STAGES <= 4, "counted waits");
      const int younger = min(nk - 1 - ks, C::STAGES - 2);
      if (younger == 2) wait_stage_barrier<(C::STAGES > 3 ? 2 : 0) * NL>();
      else if (younger == 1) wait_stage_barrier<(C::STAGES > 2 ? 1 : 0) * NL>();
      else wait_stage_barrier<0>();
      const bool more = ks + C::STAGES - 1 < nk;
      const int next = ks + C::STAGES - 1, nbuf = next % C::STAGES;
      // The chunk's loads go out before its products; where B is transposed on
      // the way, A's behind the first step's LDS reads and B's behind its
      // products (dx 1.69 -> 1.55 ms; the other products ran 0-5% slower so).
      constexpr bool SPREAD = !WGRAD && !BKC && decltype(live_c)::value > 0;
      if (!SPREAD && more) issue(next, nbuf);
      unsigned char* sa = smem + (ks % C::STAGES) * C::SBYTES;
      unsigned char* sb = sa + C::ABYTES;
      const int left = K - ks * C::TK;
      if (left < C::TK) zero_tail(sa, sb, left);     // (K is a multiple of 8 where KC)
      multiply(
          sa, sb, live_c, [&] { if (SPREAD && more) issue(next, nbuf, true, false); },
          [&] { if (SPREAD && more) issue(next, nbuf, false, true); });
    }
  };
  // An expert's last tile may hold few rows: a wave without rows only loads,
  // and one with at most half its subtiles skips the products of the others.
  // (Each case is a loop of its own, chosen once per wave.)
  const int live = r1 - r0 - wm * C::WTM;      // rows of this wave's part
  constexpr int HALF_M = (C::MFM + 1) / 2;
  if (WGRAD || live > 32 * HALF_M) contract(std::integral_constant<int, C::MFM>{});
  else if (live > 32) contract(std::integral_constant<int, HALF_M>{});
  else if (live > 0) contract(std::integral_constant<int, 1>{});
  else contract(std::integral_constant<int, 0>{});

  // ---- epilogue: output tiles leave through LDS, whole lines at a time.
  // acc[mi][ni][4 q + r] is row m0 + lrow, column nbase + 8 q + 4 khalf + r.
  const int nrows = r1 - r0;
  bf16_t* out = WGRAD ? a.out + (size_t)e * a.out_stride : a.out;
  auto put = [&](int mi, int col, uint32_t lo, uint32_t hi) {
    *reinterpret_cast<uint2*>(smem + (wm * C::WTM + mi * 32 + lrow) * C::PITCH + col * 2) =
        make_uint2(lo, hi);
  };
  // the staged tile, COLS columns of T, to y's columns from n0 on
  auto store = [&](auto* y, long long ld) {
    constexpr int EPC = 16 / sizeof(*y), CPR = COLS / EPC;    // 16-byte chunks per row
    for (int c = threadIdx.x; c < C::TM * CPR; c += C::NTHR) {
      const int r = c / CPR, cc = c - r * CPR;
      if (r < nrows && n0 + cc * EPC < a.N)
        st_nt16(y + (size_t)(r0 + r) * ld + n0 + cc * EPC,
                *reinterpret_cast<const uint4*>(smem + r * C::PITCH + cc * 16));
    }
  };
  lds_barrier();      // every wave is done reading the stage buffers
  if constexpr (EPI == EPI_STORE) {
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          put(mi, nbase[ni] + 8 * q + 4 * khalf,
              cvt_bf16x2(acc[mi][ni][4 * q], acc[mi][ni][4 * q + 1]),
              cvt_bf16x2(acc[mi][ni][4 * q + 2], acc[mi][ni][4 * q + 3]));
    lds_barrier();
    store(out, a.ldo);
  }
  if constexpr (EPI == EPI_SWIGLU) {
    // g, u (TN / 2 columns of float32 fill a staged row of TN bfloat16; of 16
    // bits both fit side by side), then h
    constexpr int HALF = C::MFN / 2;
    if (a.gu16) {
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
        for (int ni = 0; ni < C::MFN; ++ni)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& v = acc[mi][ni];
            const uint2 p = gu_pack4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            put(mi, nbase[ni] + 8 * q + 4 * khalf, p.x, p.y);
          }
      lds_barrier();
      constexpr int CPR = COLS / 8;
      for (int c = threadIdx.x; c < C::TM * 2 * CPR; c += C::NTHR) {
        const int r = c / (2 * CPR), cc = c - r * (2 * CPR), half = cc / CPR;
        const int col = n0 + (cc - half * CPR) * 8;
        if (r < nrows && col < a.N)
          st_nt16(static_cast<bf16_t*>(a.gu) + (size_t)(r0 + r) * (2 * (size_t)a.N) +
                      half * a.up_off + col,
                  *reinterpret_cast<const uint4*>(smem + r * C::PITCH + cc * 16));
      }
      lds_barrier();
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
          for (int ni = 0; ni < HALF; ++ni)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16_t& v = acc[mi][ni + half * HALF];
              *reinterpret_cast<float4*>(smem + (wm * C::WTM + mi * 32 + lrow) * C::PITCH +
                                         (nbase[ni] + 8 * q + 4 * khalf) * 4) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
        lds_barrier();
        store(static_cast<float*>(a.gu) + half * a.up_off, 2LL * a.N);
        lds_barrier();
      }
    }
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
      for (int ni = 0; ni < HALF; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float h[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            h[r] = silu_fast(acc[mi][ni][4 * q + r]) * acc[mi][ni + HALF][4 * q + r];
          put(mi, nbase[ni] + 8 * q + 4 * khalf, cvt_bf16x2(h[0], h[1]), cvt_bf16x2(h[2], h[3]));
        }
    lds_barrier();
    store(a.out2, a.N);
  }
  if constexpr (EPI == EPI_DSWIGLU) {
    // dg, du and h of each element from dh (the accumulator, never rounded)
    // and the saved g and u, 32 rows of every wave at a time: the three
    // results of those rows fill LDS side by side and leave together (h after
    // the others where LDS holds two)
    constexpr int RB = C::WM * 32, REGION = RB * C::PITCH;
    constexpr bool THREE = 3 * REGION <= C::LDS;
    static_assert(2 * REGION <= C::LDS, "staged rows");
    auto rows = [&](const auto* gu) {
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi) {
        const int row = min(r0 + wm * C::WTM + mi * 32 + lrow, r1 - 1);
        const auto* gr = gu + (size_t)row * (2 * (size_t)a.N);
        unsigned char* so = smem + (wm * 32 + lrow) * C::PITCH;
        uint2 hp[C::MFN][4];
#pragma unroll
        for (int ni = 0; ni < C::MFN; ++ni) {
          const int col = n0 + nbase[ni] < a.N ? n0 + nbase[ni] : 0;   // whole 32s in or out
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = col + 8 * q + 4 * khalf;
            float g[4], u[4], dg[4], du[4], h[4];
            load4(gr + c, g);
            load4(gr + a.N + c, u);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float dh = acc[mi][ni][4 * q + r];
              const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g[r])), sg = g[r] * s;
              h[r] = sg * u[r];
              dg[r] = dh * u[r] * (s + sg * (1.0f - s));
              du[r] = dh * sg;
            }
            uint2* p = reinterpret_cast<uint2*>(so + (nbase[ni] + 8 * q + 4 * khalf) * 2);
            p[0] = make_uint2(cvt_bf16x2(dg[0], dg[1]), cvt_bf16x2(dg[2], dg[3]));
            p[REGION / 8] = make_uint2(cvt_bf16x2(du[0], du[1]), cvt_bf16x2(du[2], du[3]));
            hp[ni][q] = make_uint2(cvt_bf16x2(h[0], h[1]), cvt_bf16x2(h[2], h[3]));
            if (THREE) p[2 * REGION / 8] = hp[ni][q];
          }
        }
        auto leave = [&](bf16_t* y, long long ld, int region) {
          constexpr int CPR = C::TN / 8;
          for (int c = threadIdx.x; c < RB * CPR; c += C::NTHR) {
            const int r = c / CPR, cc = c - r * CPR, col = n0 + cc * 8;
            const int rt = (r >> 5) * C::WTM + mi * 32 + (r & 31);     // row of the tile
            if (rt < nrows && col < a.N)
              st_nt16(y + (size_t)(r0 + rt) * ld + col,
                      *reinterpret_cast<const uint4*>(smem + region + r * C::PITCH + cc * 16));
          }
        };
        lds_barrier();
        leave(out, a.ldo, 0);
        leave(out + a.up_off, a.ldo, REGION);
        if constexpr (!THREE) {
          lds_barrier();
#pragma unroll
          for (int ni = 0; ni < C::MFN; ++ni)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint2*>(so + (nbase[ni] + 8 * q + 4 * khalf) * 2) = hp[ni][q];
          lds_barrier();
        }
        leave(a.out2, a.N, THREE ? 2 * REGION : 0);
        lds_barrier();
      }
    };
    if (a.gu16) rows(static_cast<const bf16_t*>(a.gu));
    else rows(static_cast<const float*>(a.gu));
  }
}

// Row tiles of an expert: 256 rows while it has them; the last tile, if it
// holds at most 128 or 64, in a shape of its own whose shorter stages leave LDS
// for three and four of them.  (Few rows leave nothing to hide a load's
// latency behind but other loads: with two stages a last tile of 6 rows took as
// long as a full one.)  At least 64 rows' worth of weights per block either way.
using GemmT256 = GemmCfg<256, 256, 64, 2, 2, 4>;
using GemmT128 = GemmCfg<128, 256, 64, 3, 2, 4>;
using GemmT64 = GemmCfg<64, 256, 64, 4, 2, 4>;
constexpr int GEMM_TM = GemmT256::TM, GEMM_TN = GemmT256::TN;
constexpr int GEMM_LDS = std::max({GemmT256::LDS, GemmT128::LDS, GemmT64::LDS});

template <bool BKC, int EPI, bool GATHER>
__global__ __launch_bounds__(512, 2) void train_rows_kernel(GemmArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  constexpr int COLS = EPI == EPI_SWIGLU ? GEMM_TN / 2 : GEMM_TN;
  const int NT = (a.N + COLS - 1) / COLS;
  RowBlock t;
  if (!row_block<GEMM_TM>(a.offsets, a.E, a.max_rows, NT, blockIdx.x, t)) return;
  const int r0 = t.r0, r1 = t.r1, n0 = t.n * COLS;
  if (r1 - r0 > 128)
    gemm_tile<GemmT256, false, BKC, EPI, GATHER>(a, smem, t.e, r0, r1, n0, a.K, 0);
  else if (r1 - r0 > 64)
    gemm_tile<GemmT128, false, BKC, EPI, GATHER>(a, smem, t.e, r0, r1, n0, a.K, 0);
  else
    gemm_tile<GemmT64, false, BKC, EPI, GATHER>(a, smem, t.e, r0, r1, n0, a.K, 0);
}

// Weight gradients: contractions as long as an expert has rows, often a few
// hundred, so a block's start and its output are a good part of its time:
// chunks of 32 rows and 128 x 256 outputs leave room for two blocks per CU, one
// computing while the other stores (Mixtral shape, 1024 rows per expert: dW2
// 1.04 -> 0.95 ms; 32 rows per expert: 0.43 -> 0.30 ms, 5.3 TB/s of stores).
using GemmW = GemmCfg<128, 256, 32, 2, 2, 4>;

// One launch for both parameters: blocks [0, grid0) take a0, the rest a1.
__global__ __launch_bounds__(512, 4) void train_wgrad_kernel(GemmArgs a0, GemmArgs a1, int grid0) {
  const bool second = (int)blockIdx.x >= grid0;
  const GemmArgs a = second ? a1 : a0;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  constexpr int GROUP = 8;      // column tiles side by side
  const int NT = (a.N + GemmW::TN - 1) / GemmW::TN, MT = (a.M + GemmW::TM - 1) / GemmW::TM;
  const int n_active = a.E * MT * NT, per = n_active >> 3;
  int b = second ? (int)blockIdx.x - grid0 : (int)blockIdx.x;
  if (b < per * 8) b = (b & 7) * per + (b >> 3);
  const int e = b / (MT * NT), li = b - e * MT * NT;
  const int g = li / (MT * GROUP), rem = li - g * MT * GROUP, Gc = min(GROUP, NT - g * GROUP);
  const int m_t = rem / Gc, n0 = (g * GROUP + (rem - m_t * Gc)) * GemmW::TN;
  const int r0 = m_t * GemmW::TM, r1 = min(r0 + GemmW::TM, a.M);
  const int o = a.offsets[e], K = expert_tiles(o, a.offsets[e + 1], 1, a.max_rows);
  gemm_tile<GemmW, true, false, EPI_STORE, false>(a, smem, e, r0, r1, n0, K, K ? o : 0);
}

// ---------------------------------------------------------------------------
// a_perm[r] = x[src_token[r]] for the rows of valid experts: dW13 reads its rows
// in order (with the gather inside the product's loads it ran 15-20% slower at
// 512-1024 rows per expert, more than the copy costs).  A wave per row.
// ---------------------------------------------------------------------------
constexpr int GR_ROWS = 16;      // rows per block of 4 waves

__global__ __launch_bounds__(256) void train_gather_kernel(const uint4* x, const int32_t* src_token,
                                                           const int32_t* offsets, int E,
                                                           int max_rows, int vecs, uint4* out) {
  const int lane = threadIdx.x & 63;
  const int row0 = blockIdx.x * GR_ROWS + (threadIdx.x >> 6) * (GR_ROWS / 4);
  bool mine[GR_ROWS / 4] = {};
  for (int e = lane; e < E; e += 64) {
    const int o = offsets[e], end = offsets[e + 1];
    if (expert_tiles(o, end, 1, max_rows) == 0) continue;
#pragma unroll
    for (int i = 0; i < GR_ROWS / 4; ++i) mine[i] |= row0 + i >= o && row0 + i < end;
  }
#pragma unroll
  for (int i = 0; i < GR_ROWS / 4; ++i) {
    if (__ballot(mine[i]) == 0) continue;
    const size_t row = row0 + i;
    const uint4* s = x + (size_t)max(src_token[row], 0) * vecs;
    for (int c = lane; c < vecs; c += 64) out[row * vecs + c] = s[c];
  }
}

// ---------------------------------------------------------------------------
// float32: the same products by v_mfma_f32_16x16x4_f32 straight from memory.
// The float32 layer is small (the toy layer has 16 rows per expert), so a
// block takes 32 x 32 outputs and its 4 waves split the contraction in
// interleaved chunks of 16, each with the next chunk's loads in flight; they
// meet in LDS in wave order.  (WAVES: a wave takes 32 x 32 outputs of a weight
// gradient alone, where a few rows per expert leave nothing to split.)  A lane's
// four elements of a chunk feed four products: element i of lane l stands for
// k = 4 (l / 16) + i in both operands.  The toy layer's step takes 34 us, four
// dependent launches bound by each wave's chain of loads, 4 to 16 chunks long (dx
// contracts over 2 I: 15 us; 64 x 64 tiles of plain multiply-adds: 343 us the
// step); three to six chunks in flight took 36 to 45.  Larger layers reach a
// quarter of the float32 product rate (8 experts of 128 rows, H 1024, I 512: 252
// us, 38 TFLOP/s): a 32 x 32 tile loads an operand byte for every 8 operations.
// ---------------------------------------------------------------------------
struct F32GemmArgs {
  const float* A;
  const float* B;
  long long lda, ldb, b_stride;
  const int32_t* src_token;
  const int32_t* offsets;
  int E, max_rows, M, N, K, up_off;
  float* out;
  long long ldo, out_stride;
  float* out2;
  const float* gu;
};

constexpr int F32_T = 32;

constexpr int f32_lds(int EPI) { return 4 * F32_T * ((EPI == EPI_SWIGLU ? 4 : 2) * 16 + 4); }

template <bool WGRAD, bool BKC, int EPI, bool WAVES>
__device__ __forceinline__ void f32_tile(const F32GemmArgs& a, int block, float* lds) {
  constexpr int T = F32_T, NB = EPI == EPI_SWIGLU ? 4 : 2;    // 16-column operands (gate, then up)
  constexpr int PITCH = NB * 16 + 4;
  auto red = reinterpret_cast<float(*)[T][PITCH]>(lds);
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int NT = a.N / T, tile = WAVES ? block * 4 + wid : block, n0 = (tile % NT) * T;
  int e, r0, r1, K, krow0 = 0;
  if constexpr (WGRAD) {
    const int MT = a.M / T, li = tile / NT;
    e = li / MT;
    if (e >= a.E) return;
    r0 = (li - e * MT) * T;
    r1 = r0 + T;
    const int o = a.offsets[e];
    K = expert_tiles(o, a.offsets[e + 1], 1, a.max_rows);
    krow0 = K ? o : 0;
  } else {
    TileScan scan;
    scan.init(a.offsets, a.E, T, a.max_rows);
    const int m_t = tile / NT;
    if (m_t >= scan.total) return;
    const RowTile t = scan.find(a.offsets, a.E, T, a.max_rows, m_t);
    e = t.e;
    r0 = t.off + (m_t - t.first) * T;
    r1 = min(r0 + T, t.end);
    K = a.K;
  }
  const int lr = lane & 15, lg = lane >> 4;
  // (a weight gradient's gathered B starts at row 0: its rows are looked up)
  const float* B = !WGRAD            ? a.B + (size_t)e * a.b_stride
                   : a.src_token ? a.B
                                 : a.B + (size_t)krow0 * a.ldb;
  const float* ap[2];
  const float* bp[NB];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (WGRAD) {
      ap[i] = a.A + (size_t)krow0 * a.lda + r0 + 16 * i + lr;
    } else {
      const int row = min(r0 + 16 * i + lr, r1 - 1);
      ap[i] = a.A + (size_t)(a.src_token ? max(a.src_token[row], 0) : row) * a.lda;
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int n = n0 + (i & 1) * 16 + lr + (i >> 1) * a.up_off;
    bp[i] = BKC ? B + (size_t)n * a.ldb : B + n;
  }
  // elements k + [0, 4) of a row, or of a column (zeros past the end: only a
  // weight gradient's contraction ends inside a chunk)
  auto along = [&](const float* p, int k) {
    const float4 v = *reinterpret_cast<const float4*>(p + k);
    return f32x4_t{v.x, v.y, v.z, v.w};
  };
  auto across = [&](const float* p, long long ld, int k, const int32_t* src) {
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0.f;
      if (!WGRAD || k + i < K)
        v[i] = p[(size_t)(src ? max(src[krow0 + k + i], 0) : k + i) * ld];
    }
    return v;
  };
  struct Chunk16 {
    f32x4_t a[2], b[NB];
  };
  auto load = [&](Chunk16& c, int s) {
    const int k = s * 16 + 4 * lg;
#pragma unroll
    for (int i = 0; i < 2; ++i) c.a[i] = WGRAD ? across(ap[i], a.lda, k, nullptr) : along(ap[i], k);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      c.b[i] = BKC ? along(bp[i], k) : across(bp[i], a.ldb, k, WGRAD ? a.src_token : nullptr);
  };
  f32x4_t acc[2][NB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Chunk16& c) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(c.b[j][q], c.a[i][q], acc[i][j], 0, 0, 0);
  };
  const int steps = (K + 15) / 16;
  constexpr int ds = WAVES ? 1 : 4;
  Chunk16 c0, c1;
  int s = WAVES ? 0 : wid;
  if (s < steps) load(c0, s);
  for (; s < steps; s += 2 * ds) {
    if (s + ds < steps) load(c1, s + ds);
    multiply(c0);
    if (s + ds >= steps) break;
    if (s + 2 * ds < steps) load(c0, s + 2 * ds);
    multiply(c1);
  }
  float* out = WGRAD ? a.out + (size_t)e * a.out_stride : a.out;
  // lane l holds columns 4 (l / 16) + [0, 4) of row l % 16 of every operand pair
  if constexpr (WAVES) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        *reinterpret_cast<float4*>(out + (size_t)(r0 + 16 * i + lr) * a.ldo + n0 + 16 * j +
                                   4 * lg) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<float4*>(&red[wid][16 * i + lr][16 * j + 4 * lg]) =
          make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
  __syncthreads();
  for (int o = threadIdx.x; o < T * T; o += 256) {
    const int m = o / T, n = o % T, row = r0 + m, col = n0 + n;
    if (row >= r1) continue;
    float v = 0.f, w = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v += red[k][m][n];
      if (EPI == EPI_SWIGLU) w += red[k][m][EPI == EPI_SWIGLU ? 32 + n : n];
    }
    float* p = out + (size_t)row * a.ldo + col;
    if constexpr (EPI == EPI_STORE) {
      *p = v;
    } else if constexpr (EPI == EPI_SWIGLU) {
      p[0] = v;
      p[a.up_off] = w;
      a.out2[(size_t)row * a.N + col] = silu(v) * w;
    } else {
      const float* gr = a.gu + (size_t)row * (2 * (size_t)a.N) + col;
      const float g = gr[0], u = gr[a.N], sig = 1.0f / (1.0f + expf(-g)), sg = g * sig;
      p[0] = v * u * (sig + sg * (1.0f - sig));
      p[a.up_off] = v * sg;
      a.out2[(size_t)row * a.N + col] = sg * u;
    }
  }
}

template <bool BKC, int EPI>
__global__ __launch_bounds__(256) void train_f32_kernel(F32GemmArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[f32_lds(EPI)];
  f32_tile<false, BKC, EPI, false>(a, blockIdx.x, lds);
}
// dx, dW13 and dW2, which need dh's results but not one another's, in one
// launch: blocks from 0, from b13 and from b2 on.
template <bool WAVES>
__global__ __launch_bounds__(256) void train_f32_grads_kernel(F32GemmArgs ax, F32GemmArgs a13,
                                                              F32GemmArgs a2, int b13, int b2) {
  __shared__ __attribute__((aligned(16))) float lds[f32_lds(EPI_STORE)];
  const int b = blockIdx.x;
  if (b < b13) f32_tile<false, false, EPI_STORE, false>(ax, b, lds);
  else if (b < b2) f32_tile<true, false, EPI_STORE, WAVES>(a13, b - b13, lds);
  else f32_tile<true, false, EPI_STORE, WAVES>(a2, b - b2, lds);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static long long row_tiles(int max_rows, int E, int BM) {
  const long long bound = ((long long)max_rows + (long long)E * (BM - 1)) / BM;
  return bound < max_rows ? bound : max_rows;
}
static long long cdivl(long long a, long long b) { return (a + b - 1) / b; }

// (N, M and a weight's contraction are multiples of 32)
static long long f32_row_blocks(const F32GemmArgs& a) {
  return row_tiles(a.max_rows, a.E, F32_T) * (a.N / F32_T);
}
static long long f32_wgrad_blocks(const F32GemmArgs& a, bool waves) {
  const long long tiles = (long long)a.E * (a.M / F32_T) * (a.N / F32_T);
  return waves ? cdivl(tiles, 4) : tiles;
}

template <bool BKC, int EPI, bool GATHER>
static hipError_t launch_rows(const GemmArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> lds_set{0};
  hipError_t err = ensure_lds_limit(
      reinterpret_cast<const void*>(&train_rows_kernel<BKC, EPI, GATHER>), GEMM_LDS, lds_set);
  if (err != hipSuccess) return err;
  const long long nt = cdivl(a.N, EPI == EPI_SWIGLU ? GEMM_TN / 2 : GEMM_TN);
  const long long grid = row_tiles(a.max_rows, a.E, GEMM_TM) * nt;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  train_rows_kernel<BKC, EPI, GATHER><<<(unsigned)grid, 512, GEMM_LDS, st>>>(a);
  return hipGetLastError();
}

bool train_fits(int max_rows, int E, int H, int I, int dt) {
  long long threads;
  if (dt == 0) {
    const long long rows = row_tiles(max_rows, E, F32_T), h = H / F32_T, i = I / F32_T;
    threads = 256 * std::max(rows * i, rows * h + 3 * E * h * i);
  } else {
    const long long rows = row_tiles(max_rows, E, GEMM_TM), cols = GEMM_TN;
    const long long row_blocks = rows * std::max(cdivl(I, cols / 2), cdivl(H, cols));
    const long long grad_blocks = E * (cdivl(2 * I, GemmW::TM) * cdivl(H, GemmW::TN) +
                                       cdivl(H, GemmW::TM) * cdivl(I, GemmW::TN));
    threads = std::max(512 * std::max(row_blocks, grad_blocks), cdivl(max_rows, GR_ROWS) * 256);
  }
  return threads < (1ll << 32);
}

static long long wgrad_blocks(const GemmArgs& a) {
  return a.E * cdivl(a.M, GemmW::TM) * cdivl(a.N, GemmW::TN);
}
static hipError_t launch_wgrad(const GemmArgs& a, const GemmArgs& b, hipStream_t st) {
  static std::atomic<uint64_t> lds_set{0};
  hipError_t err = ensure_lds_limit(reinterpret_cast<const void*>(&train_wgrad_kernel), GemmW::LDS,
                                    lds_set);
  if (err != hipSuccess) return err;
  const long long grid0 = wgrad_blocks(a), grid = grid0 + wgrad_blocks(b);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  train_wgrad_kernel<<<(unsigned)grid, 512, GemmW::LDS, st>>>(a, b, (int)grid0);
  return hipGetLastError();
}

template <bool BKC, int EPI>
static hipError_t launch_f32(const F32GemmArgs& a, hipStream_t st) {
  const long long grid = f32_row_blocks(a);
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  train_f32_kernel<BKC, EPI><<<(unsigned)grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

// One product's operands: rows of A against an expert's B (a weight gradient:
// b_stride 0, M and N its rows and columns).
struct Product {
  const void* A;
  long long lda;
  const void* B;
  long long ldb, b_stride;
  const int32_t* src;
  int M, N, K, up_off;
  void* out;
  long long ldo, out_stride;
  void* out2;
};
static GemmArgs bf16_args(const TrainFfn& f, const Product& p) {
  return GemmArgs{(const bf16_t*)p.A, (const bf16_t*)p.B, p.lda, p.ldb, p.b_stride, p.src,
                  f.offsets, f.E, f.max_rows, p.M, p.N, p.K, p.up_off, (bf16_t*)p.out, p.ldo,
                  p.out_stride, (bf16_t*)p.out2, f.gu, f.gu16};
}
static F32GemmArgs f32_args(const TrainFfn& f, const Product& p) {
  return F32GemmArgs{(const float*)p.A, (const float*)p.B, p.lda, p.ldb, p.b_stride, p.src,
                     f.offsets, f.E, f.max_rows, p.M, p.N, p.K, p.up_off, (float*)p.out, p.ldo,
                     p.out_stride, (float*)p.out2,
                     static_cast<const float*>(f.gu)};
}
template <bool BKC, int EPI>
static hipError_t rows_product(const TrainFfn& f, const Product& p, hipStream_t st) {
  if (f.dt == 0) return launch_f32<BKC, EPI>(f32_args(f, p), st);
  if constexpr (EPI == EPI_SWIGLU)
    if (p.src) return launch_rows<BKC, EPI, true>(bf16_args(f, p), st);
  return launch_rows<BKC, EPI, false>(bf16_args(f, p), st);
}

hipError_t launch_train_forward(const TrainFfn& f, void* y, hipStream_t st) {
  const long long H = f.H, I = f.I;
  const Product up{f.x, H, f.w13, H, 2 * I * H, f.src_token, 0, f.I, f.H, f.I, f.gu, 2 * I, 0, f.h};
  const hipError_t err = rows_product<true, EPI_SWIGLU>(f, up, st);
  if (err != hipSuccess) return err;
  const Product down{f.h, I, f.w2, I, H * I, nullptr, 0, f.H, f.I, 0, y, H, 0, nullptr};
  return rows_product<true, EPI_STORE>(f, down, st);
}

hipError_t launch_train_backward(const TrainFfn& f, const void* dy, void* dgu, void* x_perm,
                                 void* dx, void* dw13, void* dw2, hipStream_t st) {
  const long long H = f.H, I = f.I;
  const Product pdh{dy, H, f.w2, I, H * I, nullptr, 0, f.I, f.H, f.I, dgu, 2 * I, 0, f.h};
  const Product pdx{dgu, 2 * I, f.w13, H, 2 * I * H, nullptr, 0, f.H, 2 * f.I, 0, dx, H, 0, nullptr};
  Product p13{dgu, 2 * I, f.x, H, 0, f.src_token, 2 * f.I, f.H, 0, 0, dw13, H, 2 * I * H, nullptr};
  const Product p2{dy, H, f.h, I, 0, nullptr, f.H, f.I, 0, 0, dw2, I, H * I, nullptr};
  hipError_t err = rows_product<false, EPI_DSWIGLU>(f, pdh, st);
  if (err != hipSuccess) return err;
  if (f.dt == 0) {
    // the rest in one launch
    // Few rows per expert: a wave per tile of a weight gradient (4 and 64 rows
    // for each of 64 experts, H 1024, I 512, the step: 582 -> 355 and 890 -> 790
    // us).  Many rows or few tiles: four waves split the rows (8 experts of 1024
    // rows 412 -> 392 us; one of 1024, H = I = 64, 110 -> 42).
    const bool waves = f.max_rows <= 64ll * f.E;
    const F32GemmArgs ax = f32_args(f, pdx), a13 = f32_args(f, p13), a2 = f32_args(f, p2);
    const long long gx = dx ? f32_row_blocks(ax) : 0, g13 = dw13 ? f32_wgrad_blocks(a13, waves) : 0;
    const long long grid = gx + g13 + (dw2 ? f32_wgrad_blocks(a2, waves) : 0);
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    (waves ? train_f32_grads_kernel<true> : train_f32_grads_kernel<false>)<<<
        (unsigned)grid, 256, 0, st>>>(ax, a13, a2, (int)gx, (int)(gx + g13));
    return hipGetLastError();
  }
  if (dx && (err = rows_product<false, EPI_STORE>(f, pdx, st)) != hipSuccess) return err;
  if (!dw2) return hipSuccess;
  if (f.src_token) {
    train_gather_kernel<<<(unsigned)cdivl(f.max_rows, GR_ROWS), 256, 0, st>>>(
        static_cast<const uint4*>(f.x), f.src_token, f.offsets, f.E, f.max_rows, f.H / 8,
        static_cast<uint4*>(x_perm));
    if ((err = hipGetLastError()) != hipSuccess) return err;
    p13.B = x_perm;
    p13.src = nullptr;
  }
  return launch_wgrad(bf16_args(f, p13), bf16_args(f, p2), st);
}

}  // namespace moe
