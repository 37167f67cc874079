// Host helpers shared by the C ABI's entry points: argument checks, workspace
// carving and status conversion.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <climits>

#include "moe.h"

namespace moe {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int elt_bytes(int dt) { return dt == MOE_F32 ? 4 : 2; }
inline bool valid_dt(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline int cdiv(int a, int b) { return a / b + (a % b != 0); }   // a >= 0, b > 0, no overflow

// Bump allocator over the caller's workspace (or a size count when base == 0).
struct Carver {
  char* base;
  size_t used = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(size_t bytes) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += align_up(bytes);
    return p;
  }
};

// Token-pair and logit counts are int on the device: T * E (logits; k <= E,
// so this bounds the T * k pairs as well) must fit an int.
inline bool fits_int(long long a, long long b) { return a * b <= INT_MAX; }

inline int check_hidden(int H) {
  if (H <= 0) return MOE_ERR_INVALID_ARG;
  if (H % 32) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

#define MOE_TRY(expr)                      \
  do {                                     \
    hipError_t _e = (expr);                \
    if (_e != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
