// Host-side status helpers shared by the C ABI sources: the thread's error message, the argument
// checks and the translation of HIP errors.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/ft_moe.h"

namespace ftk {

// the text of ft_moe_last_error() on this host thread
inline thread_local char g_err[512] = {0};

inline int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

inline int ok() {
  g_err[0] = 0;
  return FT_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(FT_E_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define REQUIRE(cond, code, ...) \
  do {                           \
    if (!(cond)) return fail(code, __VA_ARGS__); \
  } while (0)

#define CHECK_PTR(p, name) \
  do {                                                               \
    if ((p) == nullptr) return fail(FT_E_INVAL, "%s is null", name); \
    if (!aligned16(p)) return fail(FT_E_INVAL, "%s is not 16-byte aligned", name); \
  } while (0)

// The n of FT_N_SLOTS(n) in a call's flags; 0: not given.
constexpr int kSlotFlags = 0x7fffff00;
inline int flag_slots(int flags) { return (flags & kSlotFlags) >> 8; }

inline int check_tek(int T, int E, int k) {
  REQUIRE(T >= 0, FT_E_INVAL, "T must be >= 0 (got %d)", T);
  REQUIRE(E >= 1 && E <= 1024, FT_E_INVAL, "E must be in [1, 1024] (got %d)", E);
  REQUIRE(k >= 1 && k <= E && k <= 32, FT_E_INVAL, "k must be in [1, min(E, 32)] (got k=%d, E=%d)", k, E);
  REQUIRE((long long)T * k <= (1LL << 30), FT_E_INVAL, "T*k too large (%lld)", (long long)T * k);
  return FT_OK;
}

}  // namespace ftk
