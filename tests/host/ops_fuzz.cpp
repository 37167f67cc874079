// Host-side argument fuzzing of include/moe_ops.h, built with sanitizers on
// the host pass (no GPU needed).  Every call here is a pure host query or
// carries an argument that the host checks reject, so nothing is ever
// enqueued.  Shapes are judged by the header's words, written apart from the
// library's checks, in 128-bit integers.  Exit status 0 and a final "ok" line
// mean every check held and the sanitizers found nothing.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "moe_ops.h"

namespace {

typedef __int128 wide;

uint64_t g_state = 0x2545f4914f6cdd1dull;
uint32_t next_u32() {            // xorshift64*
  g_state ^= g_state >> 12;
  g_state ^= g_state << 25;
  g_state ^= g_state >> 27;
  return (uint32_t)((g_state * 0x2545f4914f6cdd1dull) >> 32);
}
template <int N>
int pick(const int (&v)[N]) { return v[next_u32() % N]; }
int log_int(int bits) {          // 1 .. 2^bits, spread over the logarithm
  const double e = next_u32() / 4294967296.0 * bits;
  return (int)std::exp2(e);
}

int g_fail = 0;
#define CHECK(cond, ...)                                  \
  do {                                                    \
    if (!(cond)) {                                        \
      std::fprintf(stderr, "check failed: %s: ", #cond);  \
      std::fprintf(stderr, __VA_ARGS__);                  \
      std::fprintf(stderr, "\n");                         \
      if (++g_fail > 20) std::exit(1);                    \
    }                                                     \
  } while (0)

alignas(16) unsigned char g_buf[64];     // a stand-in: only its address is read
void* const P = g_buf;
void* const MIS = g_buf + 4;
uint8_t* const P8 = g_buf;
float* const PF = reinterpret_cast<float*>(g_buf);
int32_t* const PI = reinterpret_cast<int32_t*>(g_buf);

const int kRows[] = {INT_MIN, -1, 0, 1, 2, 15, 16, 63, 64, 65, 255, 256, 257, 8192, 65536, (1 << 22) - 1,
                     1 << 22, (1 << 26) - 1, 1 << 26, (1 << 28) - 16, 1 << 28, 1 << 29, 1 << 30, (1 << 30) + 1,
                     INT_MAX};
const int kWidth[] = {INT_MIN, -32, 0, 1, 31, 32, 48, 64, 96, 512, 544, 4096, 8192, 14336, 16384, 16416, 32768, 65504,
                      65536, 65568, INT_MAX - 31, INT_MAX};
const int kExperts[] = {INT_MIN, -1, 0, 1, 2, 8, 60, 128, 1000, 1024, 1025, INT_MAX};
const int kDt[] = {INT_MIN, -1, 0, 1, 2, MOE_GU_16, MOE_BF16 | MOE_GU_16, 2 | MOE_GU_16, INT_MAX};

wide cdiv(wide a, wide b) { return (a + b - 1) / b; }

bool row_ok(int H) { return H > 0 && H % 32 == 0 && H <= 16384; }
bool rows_ok(int T, int H) {
  const wide t = 64 * cdiv(H, 512);
  return T >= 0 && row_ok(H) && (wide)T * (t < 1024 ? t : 1024) < ((wide)1 << 32);
}
bool block_ok(int rows, int E, int H, int I) {
  return rows >= 0 && rows <= (1 << 30) && E >= 1 && E <= 1024 && H > 0 && H % 32 == 0 && H <= 65536 && I > 0 &&
         I % 32 == 0 && I <= 65536 && (wide)H * I <= ((wide)1 << 30);
}
bool train_dt(int dt) { return dt == 0 || dt == 1 || dt == (MOE_BF16 | MOE_GU_16); }

}  // namespace

int main(int argc, char** argv) {
  const int iters = argc > 1 ? std::atoi(argv[1]) : 20000;
  long long accepted = 0;
  for (int it = 0; it < iters; ++it) {
    const bool edge = it & 1;
    const int T = edge ? pick(kRows) : log_int(30);
    const int H = edge ? pick(kWidth) : 32 * log_int(11), I = edge ? pick(kWidth) : 32 * log_int(11);
    const int E = edge ? pick(kExperts) : log_int(10), dt = edge ? pick(kDt) : (int)(next_u32() & 1);
    const int k = edge ? (int)(next_u32() % 40) - 3 : 1 + (int)(next_u32() % 32);
    const bool mis = next_u32() & 1;

    // ---- norm: each call without an input, misaligned, or of a refused shape
    const bool t01 = dt == 0 || dt == 1;
    {
      const int st = moe_rmsnorm(T > 0 && !mis ? nullptr : P, nullptr, P, mis ? -1.f : 1e-6f, T, H, dt, P, nullptr,
                                 nullptr, nullptr, nullptr, nullptr);
      const bool shape = t01 && rows_ok(T, H);
      CHECK(st != MOE_OK || (T == 0 && !mis && shape), "norm T %d H %d dt %d", T, H, dt);
      if (t01 && T >= 0 && row_ok(H) && !mis && T > 0)
        CHECK(st == (rows_ok(T, H) ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED), "norm T %d H %d: %d", T, H, st);
    }
    {
      const size_t n = moe_rmsnorm_backward_workspace_size(T, H, dt);
      CHECK((n > 0) == (T >= 0 && t01 && row_ok(H)), "norm backward size T %d H %d", T, H);
      if (n > 0) {
        ++accepted;
        CHECK(n >= (size_t)H * 4 && n <= (size_t)512 * H * 4, "norm backward size %zu", n);
        if (T < INT_MAX) CHECK(n <= moe_rmsnorm_backward_workspace_size(T + 1, H, dt), "monotone");
        if (T > 0)
          CHECK(moe_rmsnorm_backward(P, P, P, P, PF, T, H, dt, P, PF, P, n - 1, nullptr) == MOE_ERR_WORKSPACE,
                "norm backward short workspace");
      }
      CHECK(moe_rmsnorm_backward(P, P, P, P, PF, T, H, dt, P, nullptr, P, n, nullptr) != MOE_OK,
            "norm backward without dweight");
      CHECK(moe_rmsnorm_backward(P, P, mis ? MIS : P, P, PF, T, H, dt, mis ? P : MIS, PF, P, n, nullptr) != MOE_OK,
            "norm backward misaligned");
    }
    {
      const int st = moe_combine_backward(P, dt, P, next_u32() & 1, PI, PF, T, k, H, mis ? MIS : P, mis ? PF : nullptr,
                                          nullptr);
      CHECK(st != MOE_OK || (T == 0 && !mis), "combine backward T %d k %d H %d", T, k, H);
      if (t01 && T > 0 && k >= 1 && row_ok(H)) {
        const bool fits = k <= 32 && (wide)T * k <= INT_MAX && rows_ok(T, H);
        CHECK(st == (fits ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED), "combine T %d k %d H %d: %d", T, k, H, st);
      }
    }

    // ---- expert blocks: a size of 0 goes with a rejected call, another with a
    // call that a workspace one byte short stops
    const bool blk = block_ok(T, E, H, I);
    const int rows = T;
    {
      const int rdt = dt & ~MOE_GU_16;
      const size_t f = moe_grouped_ffn_train_workspace_size(rows, E, H, I, dt);
      const size_t b = moe_grouped_ffn_backward_workspace_size(rows, E, H, I, dt);
      CHECK((f > 0) == (b > 0), "train sizes of rows %d E %d H %d I %d dt %d", rows, E, H, I, dt);
      if (f > 0) {
        ++accepted;
        const wide n = rows > 0 ? rows : 1, eb = rdt == 0 ? 4 : 2;
        CHECK(blk && train_dt(dt), "train accepted rows %d E %d H %d I %d dt %d", rows, E, H, I, dt);
        CHECK(rdt == 0 || (wide)4 * H * I <= 0xffffffffll, "W13 of %d x %d", H, I);
        CHECK((wide)f >= n * I * eb && (wide)f < n * I * eb + 256, "train size %zu", f);
        CHECK((wide)b >= n * eb * (3 * (wide)I + H) && (wide)b < n * eb * (3 * (wide)I + H) + 768, "size %zu", b);
        if (rows > 0) {
          CHECK(f >= moe_grouped_ffn_train_workspace_size(rows - 1, E, H, I, dt), "monotone");
          CHECK(b >= moe_grouped_ffn_backward_workspace_size(rows - 1, E, H, I, dt), "monotone");
          CHECK(moe_grouped_ffn_train(nullptr, P, PI, PI, E, rows, H, I, P, P, dt, P, P, P, f - 1, nullptr) ==
                    MOE_ERR_WORKSPACE, "train short workspace");
          CHECK(moe_grouped_ffn_backward(P, nullptr, P, PI, PI, E, rows, H, I, P, P, dt, P, P, P, P, P, b - 1,
                                         nullptr) == MOE_ERR_WORKSPACE, "backward short workspace");
        }
      } else if (rows > 0) {
        const int want = !blk || !train_dt(dt) ? 0 : MOE_ERR_UNSUPPORTED;
        const int s1 = moe_grouped_ffn_train(P, P, PI, PI, E, rows, H, I, P, P, dt, P, P, P, SIZE_MAX, nullptr);
        const int s2 = moe_grouped_ffn_backward(P, P, P, PI, PI, E, rows, H, I, P, P, dt, P, P, P, P, P, SIZE_MAX,
                                                nullptr);
        CHECK(s1 == s2 && s1 != MOE_OK && (!want || s1 == want), "rejected train rows %d E %d: %d %d", rows, E, s1, s2);
      }
      CHECK(moe_grouped_ffn_backward(P, P, P, PI, PI, E, rows, H, I, P, P, dt, P, P, nullptr, P, P, SIZE_MAX,
                                     nullptr) != MOE_OK, "dw2 without dw13");
      CHECK(moe_grouped_ffn_train(P, nullptr, nullptr, PI, E, rows, H, I, MIS, P, dt, P, P, P, SIZE_MAX, nullptr) !=
                MOE_OK, "train misaligned");
    }
    {
      const size_t n = moe_grouped_ffn_mxfp8_workspace_size(rows, E, H, I);
      const int y_dt = (int)(next_u32() & 1);
      if (n > 0) {
        ++accepted;
        CHECK(blk, "mxfp8 accepted rows %d E %d H %d I %d", rows, E, H, I);
        CHECK((wide)n >= (wide)(rows > 0 ? rows : 1) * (I + (wide)MOE_MX_PITCH(I)), "mxfp8 size %zu", n);
        if (rows > 0) {
          CHECK(n >= moe_grouped_ffn_mxfp8_workspace_size(rows - 1, E, H, I), "monotone");
          CHECK(moe_grouped_ffn_mxfp8(P, P8, PI, PI, E, rows, H, I, P, P8, P, P8, P, y_dt, P, n - 1, nullptr) ==
                    MOE_ERR_WORKSPACE, "mxfp8 short workspace");
        }
      } else if (rows > 0) {
        CHECK(moe_grouped_ffn_mxfp8(P, P8, PI, PI, E, rows, H, I, P, P8, P, P8, P, y_dt, P, SIZE_MAX, nullptr) != MOE_OK,
              "rejected mxfp8 rows %d E %d H %d I %d", rows, E, H, I);
      }
      CHECK(moe_grouped_ffn_mxfp8(P, P8, nullptr, PI, E, rows, H, I, P, P8, P, mis ? P8 + 1 : P8, P, mis ? y_dt : 7, P,
                                  SIZE_MAX, nullptr) != MOE_OK, "mxfp8 misaligned or of no type");
    }
  }
  if (g_fail) return 1;
  std::printf("ok %d cases, %lld with an accepted shape\n", iters, accepted);
  return 0;
}
