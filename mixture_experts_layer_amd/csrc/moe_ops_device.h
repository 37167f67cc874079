// Device helpers of the operators around the layer (norm, MXFP8 experts,
// backward passes): rows in 8-element chunks, bfloat16 rounding by the
// hardware conversion, MXFP8 blocks, and the lookup of an expert's row tile.
#pragma once
#include "moe_device.h"

namespace moe {

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));
typedef float f32x2_v __attribute__((ext_vector_type(2)));

// Two floats to packed bfloat16, to nearest even; NaN stays NaN (one
// v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_v){lo, hi}, bf16x2_v));
}

// 16 bytes, not to be read again by this launch
__device__ __forceinline__ void st_nt16(void* p, const uint4& v) {
  typedef unsigned int v4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store((v4){v.x, v.y, v.z, v.w}, reinterpret_cast<v4*>(p));
}

// 8 consecutive elements of a bfloat16 or float32 row.
template <bool BF16>
struct Chunk {
  uint4 raw[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* row, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(row) + (BF16 ? c : 2 * c);
    raw[0] = p[0];
    if (!BF16) raw[BF16 ? 0 : 1] = p[1];
  }
  __device__ __forceinline__ void get(float* f) const {
    if (BF16) {
      unpack_bf16x8(raw[0], f);
    } else {
      const uint4 a = raw[0], b = raw[BF16 ? 0 : 1];
      f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
      f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
      f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    if (BF16) {
      raw[0] = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                          cvt_bf16x2(f[6], f[7]));
    } else {
      raw[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
      raw[BF16 ? 0 : 1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                     __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
  }
  __device__ __forceinline__ void store(void* row, int c) const {
    uint4* p = reinterpret_cast<uint4*>(row) + (BF16 ? c : 2 * c);
    p[0] = raw[0];
    if (!BF16) p[1] = raw[BF16 ? 0 : 1];
  }
};

__device__ __forceinline__ size_t row_bytes(bool bf16, int H) { return (size_t)H * (bf16 ? 2 : 4); }

// Sum over the 64 lanes of a wave in float64, the same bits in every lane: the
// lane exchanges of wave_sum_f on both halves of the value.
__device__ __forceinline__ double wave_sum_d(double v) {
  auto dpp = [](double x, auto ctrl) {
    const uint2 u = __builtin_bit_cast(uint2, x);
    const uint2 r = make_uint2(
        __builtin_amdgcn_update_dpp(0, (int)u.x, decltype(ctrl)::value, 0xF, 0xF, false),
        __builtin_amdgcn_update_dpp(0, (int)u.y, decltype(ctrl)::value, 0xF, 0xF, false));
    return __builtin_bit_cast(double, r);
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  v += dpp(v, std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
  v += dpp(v, std::integral_constant<int, 0x141>{});   // row_half_mirror
  v += dpp(v, std::integral_constant<int, 0x140>{});   // row_mirror
  uint2 u = __builtin_bit_cast(uint2, v);
  auto lo = __builtin_amdgcn_permlane16_swap(u.x, u.x, false, false);
  auto hi = __builtin_amdgcn_permlane16_swap(u.y, u.y, false, false);
  v = __builtin_bit_cast(double, make_uint2(lo[0], hi[0])) +
      __builtin_bit_cast(double, make_uint2(lo[1], hi[1]));
  u = __builtin_bit_cast(uint2, v);
  lo = __builtin_amdgcn_permlane32_swap(u.x, u.x, false, false);
  hi = __builtin_amdgcn_permlane32_swap(u.y, u.y, false, false);
  return __builtin_bit_cast(double, make_uint2(lo[0], hi[0])) +
         __builtin_bit_cast(double, make_uint2(lo[1], hi[1]));
}

// Sum over a block of whole waves, the same bits in every thread: each wave's
// sum, then the waves' sums in wave order.  `red`: one float per wave, not
// read or written by anyone between two calls' barriers (callers alternate).
__device__ __forceinline__ float wave_sum(float v) { return wave_sum_f(v); }
__device__ __forceinline__ double wave_sum(double v) { return wave_sum_d(v); }
template <typename F>
__device__ __forceinline__ F block_sum(F v, F* red) {
  v = wave_sum(v);
  const int nw = blockDim.x >> 6;
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  lds_barrier();
  F s = red[0];
  for (int w = 1; w < nw; ++w) s += red[w];
  return s;
}

// Largest of the four lanes of a quad (lanes 4q .. 4q + 3), in every lane.
__device__ __forceinline__ float quad_max(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                         0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF,
                                         0xF, false));
  };
  v = fmaxf(v, dpp(v, std::integral_constant<int, 0xB1>{}));   // quad_perm [1,0,3,2]
  return fmaxf(v, dpp(v, std::integral_constant<int, 0x4E>{}));   // quad_perm [2,3,0,1]
}

// ---------------------------------------------------------------------------
// MXFP8 (OCP microscaling): 32 elements share the scale 2^(byte - 127); an
// element is e4m3 (largest finite 448 = 1.75 * 2^8).  The byte is the least
// one for which no element of the block exceeds 448 after scaling: with
// max|v| = 1.m * 2^(E - 127) that is E - 8, one more if 1.m > 1.75, and at
// least 0.  (The format's own suggestion, floor(log2 max|v|) - 8, saturates
// every block whose largest element lies above 1.75 * 2^n; the larger scale
// costs such a block one bit at the small end instead.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7fffffffu;
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(b, 0);
}
// 2^(127 - byte), the factor an element is multiplied by (byte <= 248)
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// four scaled values to e4m3, to nearest even
__device__ __forceinline__ uint32_t mx_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// ---------------------------------------------------------------------------
// Row tiles of the experts, looked up by each wave in the offsets themselves
// (no map to build in a launch of its own): expert e has ceil(count / BM)
// tiles, numbered expert after expert.  An expert whose range is not within
// [0, max_rows], or runs backwards, has none.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int expert_tiles(int o, int end, int BM, int max_rows) {
  return o >= 0 && o < end && end <= max_rows ? (end - o + BM - 1) / BM : 0;
}

struct RowTile {
  int e, off, end;   // expert and its row range
  int first;         // number of its first tile
};

// TALL: tiles of more than BM / 2 rows; SHORT: an expert's last tile of fewer.
enum RowTiles { ALL_TILES, TALL_TILES, SHORT_TILES };
template <RowTiles KIND>
__device__ __forceinline__ int row_tiles_of(int o, int end, int BM, int max_rows) {
  const int n = expert_tiles(o, end, BM, max_rows);
  if (KIND == ALL_TILES || n == 0) return n;
  const int has_short = end - o - (n - 1) * BM <= BM / 2;
  return KIND == SHORT_TILES ? has_short : n - has_short;
}

template <RowTiles KIND>
struct TileScanOf {
  int per, incl, n;  // experts per lane, tiles up to and of this lane's experts
  int total;

  // every lane of a wave takes part; E <= 1024
  __device__ __forceinline__ void init(const int32_t* offsets, int E, int BM, int max_rows) {
    const int lane = threadIdx.x & 63;
    per = (E + 63) >> 6;
    n = 0;
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e < E) n += row_tiles_of<KIND>(offsets[e], offsets[e + 1], BM, max_rows);
    }
    incl = wave_inclusive_scan(n);
    total = __builtin_amdgcn_readlane(incl, 63);
  }
  // the expert of tile `tile` < total (the same in every lane)
  __device__ __forceinline__ RowTile find(const int32_t* offsets, int E, int BM, int max_rows,
                                          int tile) const {
    const int lane = threadIdx.x & 63;
    const int L = __builtin_ctzll(__ballot(incl > tile));
    RowTile r{0, 0, 0, 0};
    if (lane == L) {
      int base = incl - n;
      for (int j = 0; j < per; ++j) {
        const int e = lane * per + j;
        if (e >= E) break;
        const int o = offsets[e], end = offsets[e + 1];
        const int nt = row_tiles_of<KIND>(o, end, BM, max_rows);
        if (tile < base + nt) {
          r = RowTile{e, o, end, base};
          break;
        }
        base += nt;
      }
    }
    return RowTile{__builtin_amdgcn_readlane(r.e, L), __builtin_amdgcn_readlane(r.off, L),
                   __builtin_amdgcn_readlane(r.end, L), __builtin_amdgcn_readlane(r.first, L)};
  }
};
using TileScan = TileScanOf<ALL_TILES>;

// Which tile block `li` of an expert's ceil(rows / TM) x NT tiles computes.  Row
// tiles of more than TM / 2 rows first, the short last one behind them: a CU left
// with a short tile at the end waits less.  Within the first, the 32 blocks of an
// XCD take all row tiles of a column while they are few, else 4 columns side by
// side (one column of 32 row tiles ran 10-25% slower).
struct TileOrder {
  int m, n;
};
__device__ __forceinline__ TileOrder tile_order(int rows, int TM, int NT, int li) {
  const int te = (rows + TM - 1) / TM, last = rows - (te - 1) * TM;
  const int tall = last > TM / 2 ? te : te - 1;
  if (li >= tall * NT) return TileOrder{te - 1, li - tall * NT};
  const int group = tall > 8 ? 4 : 1;
  const int g = li / (tall * group), rem = li - g * tall * group, Gc = min(group, NT - g * group);
  const int m = rem / Gc;
  return TileOrder{m, g * group + (rem - m * Gc)};
}

// The rows and the column tile of block `b` of a kernel of TM-row tiles, one
// block per CU, and NT column tiles; false if there are no more blocks.  Blocks of
// contiguous numbers share an XCD's L2.  While the tall tiles make few rounds of
// the 256 CUs, every one of them comes before any short one: mixed in, 16 short
// tiles made a third, nearly empty round of tall ones (Mixtral shape, 7 experts
// of 1024 rows and one of 1025: 9.49 -> 8.64 ms a training step; 988 to 1070 rows
// each: 9.49 -> 8.80; MXFP8 1.68 -> 1.58 and 1.74 -> 1.66 ms).  Otherwise a short
// tile follows its expert's tall ones, whose weights it then finds in the caches
// (Qwen3 shape, MXFP8: 512 rows per expert, 16 rounds, 1551 us against 1569 with
// the short tiles last; 270 rows, 8 rounds, 0.7 short tiles for every tall one,
// 1027 against 1167).
constexpr int TALL_ROUNDS = 8;
struct RowBlock {
  int e, r0, r1, n;
};
__device__ __forceinline__ int xcd_order(int b, int n) {
  const int per = n >> 3;
  return b < per * 8 ? (b & 7) * per + (b >> 3) : b;
}
template <int TM>
__device__ __forceinline__ bool row_block(const int32_t* offsets, int E, int max_rows, int NT,
                                          int b, RowBlock& out) {
  TileScanOf<TALL_TILES> tall;
  tall.init(offsets, E, TM, max_rows);
  TileScanOf<SHORT_TILES> rest;
  rest.init(offsets, E, TM, max_rows);
  const int n_tall = tall.total * NT, n_all = n_tall + rest.total * NT;
  if (b >= n_all) return false;
  RowTile t;
  TileOrder o;
  if (n_tall > TALL_ROUNDS * 256 || rest.total * 3LL > tall.total) {
    TileScan all;
    all.per = tall.per;
    all.incl = tall.incl + rest.incl;
    all.n = tall.n + rest.n;
    b = xcd_order(b, n_all);
    t = all.find(offsets, E, TM, max_rows, b / NT);
    o = tile_order(t.end - t.off, TM, NT, b - t.first * NT);
  } else if (b < n_tall) {
    b = xcd_order(b, n_tall);
    t = tall.find(offsets, E, TM, max_rows, b / NT);
    o = tile_order(t.end - t.off, TM, NT, b - t.first * NT);
  } else {
    b = xcd_order(b - n_tall, n_all - n_tall);
    t = rest.find(offsets, E, TM, max_rows, b / NT);
    o = TileOrder{(t.end - t.off - 1) / TM, b - t.first * NT};
  }
  out.e = t.e;
  out.r0 = t.off + o.m * TM;
  out.r1 = min(out.r0 + TM, t.end);
  out.n = o.n;
  return true;
}

}  // namespace moe
