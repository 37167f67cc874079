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
#include <algorithm>
#include <type_traits>

#include "moe_kernels.h"
#include "moe_ops_device.h"
#include "moe_ops_kernels.h"

namespace moe {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef const __attribute__((address_space(4))) int32_t* const_i32_t;

enum Epilogue { EPI_STORE, EPI_SWIGLU, EPI_DSWIGLU };

struct GemmArgs {
  const bf16_t* A;            // rows of the outputs' rows (or, in a weight gradient, columns)
  const bf16_t* B;
  long long lda, ldb;         // elements between memory rows
  long long b_stride;         // elements between experts' B (weights)
  const int32_t* src_token;   // gathered operand: A by rows, or B in a weight gradient
  const int32_t* offsets;
  int E, max_rows;
  int M, N, K;                // rows of a weight gradient; output columns; contraction (weights)
  int up_off;                 // EPI_SWIGLU: up rows of B; EPI_DSWIGLU: up columns of gu
  bf16_t* out;                // outputs; EPI_DSWIGLU: [dg du]
  long long ldo;
  long long out_stride;       // elements between experts' outputs (weight gradients)
  bf16_t* out2;               // EPI_SWIGLU, EPI_DSWIGLU: h [rows][N]
  float* gu;                  // [rows][2 N] of EPI_SWIGLU (written) and EPI_DSWIGLU (read)
  int group;                  // column tiles that run side by side
};

// Tile shape: TM x TN outputs, STAGES buffers of 64 along the contraction,
// WM x WN waves of (TM / WM) x (TN / WN) outputs each.
template <int TM_, int TN_, int STAGES_, int WM_, int WN_, int MINB_>
struct GemmCfg {
  static constexpr int TM = TM_, TN = TN_, STAGES = STAGES_, WM = WM_, WN = WN_, MINB = MINB_;
  static constexpr int TK = 64;
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

// KC tile [row][64]: 8 chunks of 16 bytes per row, chunk c of row r at
// c ^ (r / 2 % 8): the 16 lanes that read one chunk of 16 rows then cover the
// banks once.
__device__ __forceinline__ int kc_swz(int r) { return (r >> 1) & 7; }
// MC tile [k][TN or TM columns]: 64-byte segments, segment s of row k at
// s ^ (k % 4): the four k-rows of 64 bytes that half a wave reads lie in
// different quarters of the banks.
__device__ __forceinline__ int mc_chunk(int k, int chunk) { return chunk ^ ((k & 3) << 2); }

template <class C, bool WGRAD, bool BKC, int EPI, bool GATHER>
__global__ __launch_bounds__(C::NTHR, C::MINB) void train_gemm_kernel(GemmArgs a) {
  constexpr bool AKC = !WGRAD;
  static_assert(!WGRAD || (!BKC && EPI == EPI_STORE), "weight gradients contract over rows");
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int COLS = EPI == EPI_SWIGLU ? C::TN / 2 : C::TN;
  const int NT = (a.N + COLS - 1) / COLS;

  // ---- the block's expert, row range [r0, r1), column n0, contraction K
  int b = blockIdx.x, e, r0, r1, n_t, K, krow0 = 0;
  if constexpr (WGRAD) {
    const int MT = (a.M + C::TM - 1) / C::TM, n_active = a.E * MT * NT, per = n_active >> 3;
    if (b < per * 8) b = (b & 7) * per + (b >> 3);      // contiguous numbers share an XCD's L2
    e = b / (MT * NT);
    const int li = b - e * MT * NT;
    const int g = li / (MT * a.group), rem = li - g * MT * a.group;
    const int Gc = min(a.group, NT - g * a.group);
    const int m_t = rem / Gc;
    n_t = g * a.group + (rem - m_t * Gc);
    r0 = m_t * C::TM;
    r1 = min(r0 + C::TM, a.M);
    const int o = a.offsets[e], end = a.offsets[e + 1];
    K = expert_tiles(o, end, 1, a.max_rows);
    krow0 = K ? o : 0;
  } else {
    TileScan scan;
    scan.init(a.offsets, a.E, C::TM, a.max_rows);
    const int n_active = scan.total * NT, per = n_active >> 3;
    if (b >= n_active) return;
    if (b < per * 8) b = (b & 7) * per + (b >> 3);
    const RowTile t = scan.find(a.offsets, a.E, C::TM, a.max_rows, b / NT);
    e = t.e;
    const int te = (t.end - t.off + C::TM - 1) / C::TM, li = b - t.first * NT;
    const int g = li / (te * a.group), rem = li - g * te * a.group;
    const int Gc = min(a.group, NT - g * a.group);
    const int m_t = rem / Gc;
    n_t = g * a.group + (rem - m_t * Gc);
    r0 = t.off + m_t * C::TM;
    r1 = min(r0 + C::TM, t.end);
    K = a.K;
  }
  const int n0 = n_t * COLS;
  const bf16_t* Be = WGRAD ? a.B : a.B + (size_t)e * a.b_stride;

  // ---- lanes' sources.  Rows and columns past the end read the last one (or
  // the first column): their products are not stored.
  // KC: the chunk this lane loads of its row, the same for every load
  // (rows step by 64); row wid * 8 + lane / 8 of the first
  static_assert(C::NW == 8, "chunk of a lane");
  const int kchunk = (lane & 7) ^ kc_swz(wid * 8 + (lane >> 3));
  const unsigned char* abase;
  const unsigned char* bbase;
  uint32_t ao[C::ALOADS], bo[C::BLOADS];
  const unsigned char* ap[AKC && GATHER ? C::ALOADS : 1];
  if constexpr (AKC) {
    abase = reinterpret_cast<const unsigned char*>(a.A + (size_t)r0 * a.lda);
#pragma unroll
    for (int j = 0; j < C::ALOADS; ++j) {
      const int rt = (wid + C::NW * j) * 8 + (lane >> 3);
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
      const int rt = (wid + C::NW * j) * 8 + (lane >> 3);
      int row;
      if (EPI == EPI_SWIGLU)
        row = rt < COLS ? min(n0 + rt, a.N - 1) : a.up_off + min(n0 + rt - COLS, a.N - 1);
      else
        row = min(n0 + rt, a.N - 1);
      bo[j] = (uint32_t)((size_t)row * a.ldb * 2 + kchunk * 16);
    }
  } else {
    bbase = reinterpret_cast<const unsigned char*>(WGRAD ? Be + (GATHER ? 0 : (size_t)krow0 * a.ldb)
                                                         : Be);
#pragma unroll
    for (int j = 0; j < C::BLOADS; ++j) {
      const int k = (wid + C::NW * j) * BRPI + lane / BCPR;
      const int col = n0 + mc_chunk(k, lane % BCPR) * 8;
      bo[j] = (uint32_t)((GATHER ? 0 : (size_t)k * a.ldb * 2) + (col < a.N ? col : 0) * 2);
    }
  }

  const int nk = (K + C::TK - 1) / C::TK;
  // gathered rows of a weight gradient: the sources of the next chunk's rows,
  // uniform in the wave (scalar loads), one chunk ahead of their use
  int tok[WGRAD && GATHER ? C::BLOADS : 1][BRPI];
  auto load_tok = [&](int ks) {
    if constexpr (WGRAD && GATHER) {
      const_i32_t st = (const_i32_t)(uintptr_t)(a.src_token + krow0);
#pragma unroll
      for (int j = 0; j < C::BLOADS; ++j)
#pragma unroll
        for (int p = 0; p < BRPI; ++p)
          tok[j][p] = st[min(ks * C::TK + (wid + C::NW * j) * BRPI + p, K - 1)];
    }
  };
  // `part`: the last chunk holds fewer than TK; what lies past the end re-reads
  // valid rows or columns (and is zeroed in LDS before the products)
  auto issue_as = [&](int ks, int buf, auto part_c) {
    constexpr bool PART = decltype(part_c)::value;
    unsigned char* sa = smem + buf * C::SBYTES + wid * 1024;
    unsigned char* sb = sa + C::ABYTES;
    const int left = K - ks * C::TK;
    const uint32_t kback = PART && kchunk * 8 >= left ? kchunk * 16 : 0;   // KC: to chunk 0
    auto mc_back = [&](int k, long long ld) {                              // MC: to the last row
      return PART && k >= left ? (uint32_t)((k - left + 1) * ld * 2) : 0u;
    };
    if constexpr (AKC) {
#pragma unroll
      for (int j = 0; j < C::ALOADS; ++j) {
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
    if constexpr (BKC) {
#pragma unroll
      for (int j = 0; j < C::BLOADS; ++j)
        buffer_load_lds16(bbase, 0xffffffffu, sb + C::NW * j * 1024, bo[j] - kback,
                          (uint32_t)ks * (C::TK * 2));
    } else if constexpr (WGRAD && GATHER) {
#pragma unroll
      for (int j = 0; j < C::BLOADS; ++j) {
        int t = tok[j][0];
#pragma unroll
        for (int p = 1; p < BRPI; ++p) t = lane / BCPR == p ? tok[j][p] : t;
        __builtin_amdgcn_global_load_lds(
            (gbl_void_t*)(bbase + (size_t)max(t, 0) * a.ldb * 2 + bo[j]),
            (lds_void_t*)(sb + C::NW * j * 1024), 16, 0, 0);
      }
      load_tok(ks + 1);
    } else {
      const unsigned char* base = bbase + (size_t)ks * C::TK * a.ldb * 2;
#pragma unroll
      for (int j = 0; j < C::BLOADS; ++j)
        buffer_load_lds16(base, 0xffffffffu, sb + C::NW * j * 1024,
                          bo[j] - mc_back((wid + C::NW * j) * BRPI + lane / BCPR, a.ldb), 0);
    }
  };
  auto issue = [&](int ks, int buf) {
    if (K - ks * C::TK >= C::TK) issue_as(ks, buf, std::false_type{});
    else issue_as(ks, buf, std::true_type{});
  };
  // zero what the last chunk holds past its `left` rows or columns
  auto zero_tail = [&](unsigned char* sa, unsigned char* sb, int left) {
    const uint4 z = make_uint4(0, 0, 0, 0);
    auto kc = [&](unsigned char* p, int rows) {
      for (int i = threadIdx.x; i < rows * 8; i += C::NTHR)
        if (((i & 7) ^ kc_swz(i >> 3)) * 8 >= left) reinterpret_cast<uint4*>(p)[i] = z;
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
    asw[mi] = kc_swz(r + lrow);
    aoff[mi] = AKC ? (r + lrow) * 128
                   : trk * (C::TM * 2) + (((r >> 5) ^ (trk & 3)) << 6) + trc;
  }
#pragma unroll
  for (int ni = 0; ni < C::MFN; ++ni) {
    const int r = nbase[ni];
    bsw[ni] = kc_swz(r + lrow);
    boff[ni] = BKC ? (r + lrow) * 128
                   : trk * (C::TN * 2) + (((r >> 5) ^ (trk & 3)) << 6) + trc;
  }
  auto tr_frag = [&](const unsigned char* p, int row_bytes) {
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * row_bytes));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto load_frags = [&](const unsigned char* sa, const unsigned char* sb, int kk, bf16x8_t* af,
                        bf16x8_t* bf) {
    const int c = kk * 2 + khalf;
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi) {
      if constexpr (AKC)
        af[mi] = *reinterpret_cast<const bf16x8_t*>(sa + aoff[mi] + ((c ^ asw[mi]) * 16));
      else
        af[mi] = tr_frag(sa + aoff[mi] + kk * 16 * (C::TM * 2), C::TM * 2);
    }
#pragma unroll
    for (int ni = 0; ni < C::MFN; ++ni) {
      if constexpr (BKC)
        bf[ni] = *reinterpret_cast<const bf16x8_t*>(sb + boff[ni] + ((c ^ bsw[ni]) * 16));
      else
        bf[ni] = tr_frag(sb + boff[ni] + kk * 16 * (C::TN * 2), C::TN * 2);
    }
  };

  f32x16_t acc[C::MFM][C::MFN];
#pragma unroll
  for (int i = 0; i < C::MFM; ++i)
#pragma unroll
    for (int j = 0; j < C::MFN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  auto multiply = [&](const unsigned char* sa, const unsigned char* sb) {
    constexpr int STEPS = C::TK / 16;
    bf16x8_t af[2][C::MFM], bf[2][C::MFN];
    load_frags(sa, sb, 0, af[0], bf[0]);
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk) {
      const int cur = kk & 1;
      if (kk + 1 < STEPS) load_frags(sa, sb, kk + 1, af[cur ^ 1], bf[cur ^ 1]);
      __builtin_amdgcn_sched_barrier(0);   // the next step's LDS reads stay ahead
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
        for (int ni = 0; ni < C::MFN; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[cur][ni], af[cur][mi],
                                                                acc[mi][ni], 0, 0, 0);
    }
  };

  constexpr int NL = C::ALOADS + C::BLOADS;
  if (nk > 0) {
    load_tok(0);
#pragma unroll
    for (int s0 = 0; s0 < C::STAGES - 1; ++s0)
      if (s0 < nk) issue(s0, s0);
  }
  for (int ks = 0; ks < nk; ++ks) {
    // chunk ks has landed once at most the younger chunks' loads are
    // outstanding; past the barrier that holds for every wave, and nobody
    // still reads the buffer refilled below
    if (C::STAGES > 2 && ks + 1 < nk) wait_stage_barrier<(C::STAGES - 2) * NL>();
    else wait_stage_barrier<0>();
    if (ks + C::STAGES - 1 < nk) issue(ks + C::STAGES - 1, (ks + C::STAGES - 1) % C::STAGES);
    unsigned char* sa = smem + (ks % C::STAGES) * C::SBYTES;
    unsigned char* sb = sa + C::ABYTES;
    const int left = K - ks * C::TK;
    if (left < C::TK) zero_tail(sa, sb, left);     // (K is a multiple of 8 where KC)
    multiply(sa, sb);
  }

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
    // g, u (TN / 2 columns of float32 fill a staged row of TN bfloat16), then h
    constexpr int HALF = C::MFN / 2;
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
      store(a.gu + half * a.up_off, 2LL * a.N);
      lds_barrier();
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
    // and the saved g and u; dg and du share the accumulator's register
    uint32_t hp[C::MFM][C::MFN][8];
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi) {
      const int row = min(r0 + wm * C::WTM + mi * 32 + lrow, r1 - 1);
      const float* gr = a.gu + (size_t)row * (2 * (size_t)a.N);
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni) {
        const int col = n0 + nbase[ni] < a.N ? n0 + nbase[ni] : 0;   // whole 32s in or out
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = col + 8 * q + 4 * khalf;
          const float4 g4 = *reinterpret_cast<const float4*>(gr + c);
          const float4 u4 = *reinterpret_cast<const float4*>(gr + a.N + c);
          const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
          float h[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float dh = acc[mi][ni][4 * q + r];
            const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g[r]));
            const float sg = g[r] * s;
            h[r] = sg * u[r];
            const uint32_t p = cvt_bf16x2(dh * u[r] * (s + sg * (1.0f - s)), dh * sg);
            acc[mi][ni][4 * q + r] = __uint_as_float(p);
          }
          hp[mi][ni][2 * q] = cvt_bf16x2(h[0], h[1]);
          hp[mi][ni][2 * q + 1] = cvt_bf16x2(h[2], h[3]);
        }
        // g and u of one subtile at a time: all of them at once would spill
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    auto pass = [&](int which) {
#pragma unroll
      for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
        for (int ni = 0; ni < C::MFN; ++ni)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t p[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) p[r] = __float_as_uint(acc[mi][ni][4 * q + r]);
            const uint32_t sel = which ? 0x07060302u : 0x05040100u;   // high halves, or low
            put(mi, nbase[ni] + 8 * q + 4 * khalf, __builtin_amdgcn_perm(p[1], p[0], sel),
                __builtin_amdgcn_perm(p[3], p[2], sel));
          }
    };
    pass(0);
    lds_barrier();
    store(out, a.ldo);
    lds_barrier();
    pass(1);
    lds_barrier();
    store(out + a.up_off, a.ldo);
    lds_barrier();
#pragma unroll
    for (int mi = 0; mi < C::MFM; ++mi)
#pragma unroll
      for (int ni = 0; ni < C::MFN; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          put(mi, nbase[ni] + 8 * q + 4 * khalf, hp[mi][ni][2 * q], hp[mi][ni][2 * q + 1]);
    lds_barrier();
    store(a.out2, a.N);
  }
}

// ---------------------------------------------------------------------------
// float32: the same products on 64 x 64 tiles by plain multiply-adds (the
// float32 layer is small).
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

template <bool WGRAD, bool BKC, int EPI>
__global__ __launch_bounds__(256) void train_f32_kernel(F32GemmArgs a) {
  constexpr int T = 64, TK = 16;
  __shared__ float sa[TK][T + 1], sb[TK][T + 1], su[EPI == EPI_SWIGLU ? TK : 1][T + 1];
  const int tid = threadIdx.x;
  const int NT = (a.N + T - 1) / T;
  int e, r0, r1, K, krow0 = 0;
  const int n0 = (blockIdx.x % NT) * T;
  if constexpr (WGRAD) {
    const int MT = (a.M + T - 1) / T, li = blockIdx.x / NT;
    e = li / MT;
    r0 = (li - e * MT) * T;
    r1 = min(r0 + T, a.M);
    const int o = a.offsets[e], end = a.offsets[e + 1];
    K = expert_tiles(o, end, 1, a.max_rows);
    krow0 = K ? o : 0;
  } else {
    TileScan scan;
    scan.init(a.offsets, a.E, T, a.max_rows);
    const int tile = blockIdx.x / NT;
    if (tile >= scan.total) return;
    const RowTile t = scan.find(a.offsets, a.E, T, a.max_rows, tile);
    e = t.e;
    r0 = t.off + (tile - t.first) * T;
    r1 = min(r0 + T, t.end);
    K = a.K;
  }
  const float* B = WGRAD ? a.B : a.B + (size_t)e * a.b_stride;
  float acc[4][4] = {}, acu[4][4] = {};
  const int tm = tid >> 4, tn = tid & 15;       // rows tm + 16 i, columns tn + 16 j
  for (int k0 = 0; k0 < K; k0 += TK) {
    for (int i = tid; i < TK * T; i += 256) {
      // consecutive threads along the operand's contiguous direction
      const int ak = WGRAD ? i / T : i % TK, am = WGRAD ? i % T : i / TK;
      const int bk = BKC ? i % TK : i / T, bn = BKC ? i / TK : i % T;
      float va = 0.f, vb = 0.f, vu = 0.f;
      if (k0 + ak < K && r0 + am < r1) {
        if constexpr (WGRAD) {
          va = a.A[(size_t)(krow0 + k0 + ak) * a.lda + r0 + am];
        } else {
          const int row = a.src_token ? max(a.src_token[r0 + am], 0) : r0 + am;
          va = a.A[(size_t)row * a.lda + k0 + ak];
        }
      }
      if (k0 + bk < K && n0 + bn < a.N) {
        if constexpr (BKC) {
          vb = B[(size_t)(n0 + bn) * a.ldb + k0 + bk];
          if (EPI == EPI_SWIGLU) vu = B[(size_t)(a.up_off + n0 + bn) * a.ldb + k0 + bk];
        } else if constexpr (WGRAD) {
          const int kr = krow0 + k0 + bk, row = a.src_token ? max(a.src_token[kr], 0) : kr;
          vb = B[(size_t)row * a.ldb + n0 + bn];
        } else {
          vb = B[(size_t)(k0 + bk) * a.ldb + n0 + bn];
        }
      }
      sa[ak][am] = va;
      sb[bk][bn] = vb;
      if (EPI == EPI_SWIGLU) su[EPI == EPI_SWIGLU ? bk : 0][bn] = vu;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(sa[k][tm + 16 * i], sb[k][tn + 16 * j], acc[i][j]);
          if (EPI == EPI_SWIGLU)
            acu[i][j] = fmaf(sa[k][tm + 16 * i], su[EPI == EPI_SWIGLU ? k : 0][tn + 16 * j],
                             acu[i][j]);
        }
    __syncthreads();
  }
  float* out = WGRAD ? a.out + (size_t)e * a.out_stride : a.out;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = r0 + tm + 16 * i, col = n0 + tn + 16 * j;
      if (row >= r1 || col >= a.N) continue;
      float* o = out + (size_t)row * a.ldo + col;
      if constexpr (EPI == EPI_STORE) {
        *o = acc[i][j];
      } else if constexpr (EPI == EPI_SWIGLU) {
        o[0] = acc[i][j];
        o[a.up_off] = acu[i][j];
        a.out2[(size_t)row * a.N + col] = silu(acc[i][j]) * acu[i][j];
      } else {
        const float* gr = a.gu + (size_t)row * (2 * (size_t)a.N) + col;
        const float g = gr[0], u = gr[a.N], s = 1.0f / (1.0f + expf(-g)), sg = g * s;
        o[0] = acc[i][j] * u * (s + sg * (1.0f - s));
        o[a.up_off] = acc[i][j] * sg;
        a.out2[(size_t)row * a.N + col] = sg * u;
      }
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using GemmBig = GemmCfg<256, 256, 2, 2, 4, 1>;
using GemmMed = GemmCfg<128, 256, 3, 2, 4, 1>;

static long long row_tiles(int max_rows, int E, int BM) {
  const long long bound = ((long long)max_rows + (long long)E * (BM - 1)) / BM;
  return bound < max_rows ? bound : max_rows;
}
static long long cdivl(long long a, long long b) { return (a + b - 1) / b; }

template <class C, bool WGRAD, bool BKC, int EPI, bool GATHER>
static hipError_t launch_gemm_t(const GemmArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> lds_set{0};
  hipError_t err = ensure_lds_limit(
      reinterpret_cast<const void*>(&train_gemm_kernel<C, WGRAD, BKC, EPI, GATHER>), C::LDS, lds_set);
  if (err != hipSuccess) return err;
  constexpr int cols = EPI == EPI_SWIGLU ? C::TN / 2 : C::TN;
  const long long nt = cdivl(a.N, cols);
  const long long grid = (WGRAD ? a.E * cdivl(a.M, C::TM) : row_tiles(a.max_rows, a.E, C::TM)) * nt;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  train_gemm_kernel<C, WGRAD, BKC, EPI, GATHER><<<(unsigned)grid, C::NTHR, C::LDS, st>>>(a);
  return hipGetLastError();
}

template <bool WGRAD, bool BKC, int EPI>
static hipError_t launch_gemm(const GemmArgs& a, hipStream_t st) {
  const int mean = (int)cdivl(a.max_rows, a.E);
  const bool big = WGRAD ? true : mean >= 384;
  if constexpr (EPI == EPI_SWIGLU || WGRAD) {
    if (a.src_token)
      return big ? launch_gemm_t<GemmBig, WGRAD, BKC, EPI, true>(a, st)
                 : launch_gemm_t<GemmMed, WGRAD, BKC, EPI, true>(a, st);
  }
  return big ? launch_gemm_t<GemmBig, WGRAD, BKC, EPI, false>(a, st)
             : launch_gemm_t<GemmMed, WGRAD, BKC, EPI, false>(a, st);
}

template <bool WGRAD, bool BKC, int EPI>
static hipError_t launch_f32(const F32GemmArgs& a, hipStream_t st) {
  const long long nt = cdivl(a.N, 64);
  const long long grid = (WGRAD ? a.E * cdivl(a.M, 64) : row_tiles(a.max_rows, a.E, 64)) * nt;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  train_f32_kernel<WGRAD, BKC, EPI><<<(unsigned)grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

// One product in either type.
template <bool WGRAD, bool BKC, int EPI>
static hipError_t product(const TrainFfn& f, const void* A, long long lda, const void* B,
                          long long ldb, long long b_stride, bool gather, int M, int N, int K,
                          int up_off, void* out, long long ldo, long long out_stride, void* out2,
                          hipStream_t st) {
  const int32_t* src = gather ? f.src_token : nullptr;
  if (f.dt == 0) {
    const F32GemmArgs a{(const float*)A, (const float*)B, lda, ldb, b_stride, src, f.offsets, f.E,
                        f.max_rows, M, N, K, up_off, (float*)out, ldo, out_stride, (float*)out2,
                        f.gu};
    return launch_f32<WGRAD, BKC, EPI>(a, st);
  }
  const GemmArgs a{(const bf16_t*)A, (const bf16_t*)B, lda, ldb, b_stride, src, f.offsets, f.E,
                   f.max_rows, M, N, K, up_off, (bf16_t*)out, ldo, out_stride, (bf16_t*)out2,
                   f.gu, WGRAD ? 4 : 1};
  return launch_gemm<WGRAD, BKC, EPI>(a, st);
}

hipError_t launch_train_forward(const TrainFfn& f, void* y, hipStream_t st) {
  const long long H = f.H, I = f.I;
  hipError_t err = product<false, true, EPI_SWIGLU>(f, f.x, H, f.w13, H, 2 * I * H, true, 0, f.I,
                                                    f.H, f.I, f.dt == 0 ? f.gu : nullptr, 2 * I, 0,
                                                    f.h, st);
  if (err != hipSuccess) return err;
  return product<false, true, EPI_STORE>(f, f.h, I, f.w2, I, H * I, false, 0, f.H, f.I, 0, y, H, 0,
                                         nullptr, st);
}

hipError_t launch_train_backward(const TrainFfn& f, const void* dy, void* dgu, void* dx, void* dw13,
                                 void* dw2, hipStream_t st) {
  const long long H = f.H, I = f.I;
  hipError_t err = product<false, false, EPI_DSWIGLU>(f, dy, H, f.w2, I, H * I, false, 0, f.I, f.H,
                                                      f.I, dgu, 2 * I, 0, f.h, st);
  if (err != hipSuccess) return err;
  if (dx) {
    err = product<false, false, EPI_STORE>(f, dgu, 2 * I, f.w13, H, 2 * I * H, false, 0, f.H,
                                           2 * f.I, 0, dx, H, 0, nullptr, st);
    if (err != hipSuccess) return err;
  }
  if (!dw2) return hipSuccess;
  err = product<true, false, EPI_STORE>(f, dy, H, f.h, I, 0, false, f.H, f.I, 0, 0, dw2, I, H * I,
                                        nullptr, st);
  if (err != hipSuccess) return err;
  return product<true, false, EPI_STORE>(f, dgu, 2 * I, f.x, H, 0, true, 2 * f.I, f.H, 0, 0, dw13, H,
                                         2 * I * H, nullptr, st);
}

}  // namespace moe
