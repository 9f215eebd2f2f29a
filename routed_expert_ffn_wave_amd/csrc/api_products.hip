// C ABI of the bf16 products, SwiGLU rows and low-rank adapters (declared in include/ft_moe_products.h): host-side
// validation and kernel launches on the caller's stream.  Nothing here allocates, synchronises or throws across the ABI.
#include <hip/hip_runtime.h>

#include "../../include/ft_moe_products.h"
#include "ft_api.h"
#include "ft_products.h"

namespace {

using namespace ftk;

constexpr int kMaxCols = 1 << 20;

int check_groups(int rows, const char* rows_name, int E, int N, int K, int flags, int known) {
  REQUIRE((flags & ~known) == 0, FT_E_INVAL, "unknown flags 0x%x", flags & ~known);
  REQUIRE(E >= 1 && E <= 1024, FT_E_INVAL, "E must be in [1, 1024] (got %d)", E);
  REQUIRE(rows >= 0 && rows <= (1 << 30), FT_E_INVAL, "%s must be in [0, 2^30] (got %d)", rows_name, rows);
  REQUIRE(N > 0 && N % 8 == 0 && N <= kMaxCols, FT_E_INVAL, "N must be a positive multiple of 8, at most 2^20 (got %d)", N);
  REQUIRE(K > 0 && K % 8 == 0 && K <= kMaxCols, FT_E_INVAL, "K must be a positive multiple of 8, at most 2^20 (got %d)", K);
  return FT_OK;
}

int check_slots(int n_slots, const int32_t* slot_of, const char* name, int E) {
  REQUIRE(n_slots >= 1, FT_E_INVAL, "n_slots must be >= 1 (got %d)", n_slots);
  REQUIRE(slot_of || E <= n_slots, FT_E_INVAL, "%s is needed for E = %d and %d slots", name, E, n_slots);
  if (slot_of) CHECK_PTR(slot_of, name);
  return FT_OK;
}

int run_grouped(int kind, const char* what, const char* in_name, const char* out_name, const uint16_t* in, int P, const uint16_t* w,
                int n_slots, int N, int K, const int32_t* offsets, const int32_t* slot_of, int E, void* out, int flags,
                hipStream_t stream) {
  int rc = check_groups(P, "P", E, N, K, flags, FT_OUT_BF16);
  if (rc) return rc;
  REQUIRE(n_slots >= 1, FT_E_INVAL, "n_slots must be >= 1 (got %d)", n_slots);
  if (P == 0) return ok();
  if ((rc = check_slots(n_slots, slot_of, "slot_of_expert", E))) return rc;
  CHECK_PTR(in, in_name);
  CHECK_PTR(w, "w");
  CHECK_PTR(offsets, "offsets");
  CHECK_PTR(out, out_name);
  const GroupedArgs a{{offsets, slot_of, E, P, (uint32_t)n_slots}, in, w, N, K, out, (flags & FT_OUT_BF16) != 0};
  const hipError_t e = launch_grouped(kind, a, stream);
  REQUIRE(e != hipErrorNotSupported, FT_E_UNSUPPORTED, "product too large (%d rows, N=%d, K=%d, E=%d)", P, N, K, E);
  return hip_status(e, what);
}

int check_swiglu(int rows, int I) {
  REQUIRE(rows >= 0, FT_E_INVAL, "rows must be >= 0 (got %d)", rows);
  REQUIRE(I > 0 && I % 8 == 0 && I <= kMaxCols, FT_E_INVAL, "I must be a positive multiple of 8, at most 2^20 (got %d)", I);
  // a thread 8 values; a launch counts its threads, whole blocks of them, in 32 bits
  REQUIRE(((long long)rows * (I / 8) + 255) / 256 * 256 < (1LL << 32), FT_E_UNSUPPORTED, "rows too large (%d rows of %d values)", rows, I);
  return FT_OK;
}

size_t lora_ws(int T, int E, int r, int N, int K) { return (size_t)lora_splits(T, E, r, N, K) * T * r * sizeof(float); }

}  // namespace

extern "C" {

size_t ft_moe_grouped_matmul_wgrad_workspace(int N, int K, int E) {
  return N <= 0 || N > kMaxCols || K <= 0 || K > kMaxCols || E < 1 || E > 1024 ? 0 : wgrad_workspace(N, K, E);
}

int ft_moe_grouped_matmul(const uint16_t* a, int P, const uint16_t* w, int n_slots, int N, int K, const int32_t* offsets,
                          const int32_t* slot_of_expert, int E, void* out, int flags, hipStream_t stream) {
  try {
    return run_grouped(0, "ft_moe_grouped_matmul launch", "a", "out", a, P, w, n_slots, N, K, offsets, slot_of_expert, E, out, flags,
                       stream);
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_grouped_matmul: unexpected exception");
  }
}

int ft_moe_grouped_matmul_grad(const uint16_t* dout, int P, const uint16_t* w, int n_slots, int N, int K,
                               const int32_t* offsets, const int32_t* slot_of_expert, int E, void* da, int flags,
                               hipStream_t stream) {
  try {
    return run_grouped(1, "ft_moe_grouped_matmul_grad launch", "dout", "da", dout, P, w, n_slots, N, K, offsets, slot_of_expert, E, da,
                       flags, stream);
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_grouped_matmul_grad: unexpected exception");
  }
}

int ft_moe_grouped_matmul_wgrad(const uint16_t* dout, const uint16_t* a, int P, int N, int K, const int32_t* offsets,
                                const int32_t* slot_of_expert, int E, void* dw, void* ws, size_t ws_bytes, int flags,
                                hipStream_t stream) {
  try {
    int rc = check_groups(P, "P", E, N, K, flags, FT_OUT_BF16 | FT_ADD_TO_OUT | kSlotFlags);
    if (rc) return rc;
    const bool bf16 = (flags & FT_OUT_BF16) != 0, add = (flags & FT_ADD_TO_OUT) != 0;
    REQUIRE(!(bf16 && add), FT_E_INVAL, "FT_ADD_TO_OUT needs an fp32 dw");
    const int n = flag_slots(flags);
    REQUIRE(slot_of_expert || n == 0, FT_E_INVAL, "FT_N_SLOTS without slot_of_expert");
    if (P == 0 && add) return ok();
    if (P > 0) {
      CHECK_PTR(dout, "dout");
      CHECK_PTR(a, "a");
    }
    CHECK_PTR(offsets, "offsets");
    if (slot_of_expert) CHECK_PTR(slot_of_expert, "slot_of_expert");
    CHECK_PTR(dw, "dw");
    const size_t need = wgrad_workspace(N, K, E);
    if (need) CHECK_PTR(ws, "ws");
    REQUIRE(ws_bytes >= need, FT_E_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
    const WgradArgs args{{offsets, slot_of_expert, E, P, n ? (uint32_t)n : 0x80000000u}, dout, a, N, K, dw, bf16, add, ws};
    const hipError_t e = launch_wgrad(args, stream);
    REQUIRE(e != hipErrorNotSupported, FT_E_UNSUPPORTED, "gradient too large (N=%d, K=%d, E=%d)", N, K, E);
    return hip_status(e, "ft_moe_grouped_matmul_wgrad launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_grouped_matmul_wgrad: unexpected exception");
  }
}

int ft_moe_swiglu(const uint16_t* gu, int rows, int I, uint16_t* h, hipStream_t stream) {
  try {
    const int rc = check_swiglu(rows, I);
    if (rc) return rc;
    if (rows == 0) return ok();
    CHECK_PTR(gu, "gu");
    CHECK_PTR(h, "h");
    return hip_status(launch_swiglu(gu, nullptr, rows, I, h, stream), "ft_moe_swiglu launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_swiglu: unexpected exception");
  }
}

int ft_moe_swiglu_grad(const uint16_t* gu, const uint16_t* dh, int rows, int I, uint16_t* dgu, hipStream_t stream) {
  try {
    const int rc = check_swiglu(rows, I);
    if (rc) return rc;
    if (rows == 0) return ok();
    CHECK_PTR(gu, "gu");
    CHECK_PTR(dh, "dh");
    CHECK_PTR(dgu, "dgu");
    return hip_status(launch_swiglu(gu, dh, rows, I, dgu, stream), "ft_moe_swiglu_grad launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_swiglu_grad: unexpected exception");
  }
}

size_t ft_moe_lora_workspace(int T, int E, int r, int N, int K) {
  if (T <= 0 || T >= (1 << 24) || E < 1 || E > 1024 || r <= 0 || r > 256 || N <= 0 || N > kMaxCols || K <= 0 || K > kMaxCols) return 0;
  return lora_ws(T, E, r, N, K);
}

int ft_moe_lora(const void* base, const uint16_t* x, int T, const uint16_t* a, const uint16_t* b, const float* scale,
                int n_slots, int r, int N, int K, const int32_t* offsets, const int32_t* gather,
                const int32_t* slot_of_adapter, int E, void* out, void* ws, size_t ws_bytes, int flags, hipStream_t stream) {
  try {
    int rc = check_groups(T, "T", E, N, K, flags, FT_OUT_BF16);
    if (rc) return rc;
    REQUIRE(r > 0 && r % 8 == 0 && r <= 256, FT_E_INVAL, "r must be a positive multiple of 8, at most 256 (got %d)", r);
    REQUIRE(n_slots >= 1, FT_E_INVAL, "n_slots must be >= 1 (got %d)", n_slots);
    // items in an int whatever the table holds (from 0 over E + 1 offsets to T, one that does not ascend can give all rows to every
    // second of E + 2 groups): at most 16 rows by 256 columns each, or 64 hidden rows by 64 of at most 256 columns in up to 16 shares of K
    REQUIRE(T < (1 << 24) && (T / 16 + 8LL) * ((E + 3) / 2) * ((N + 255) / 256 > 16 ? (N + 255) / 256 : 16) < (1LL << 31) - (1 << 16),
            FT_E_UNSUPPORTED, "T too large (%d rows, N=%d, E=%d)", T, N, E);
    if (T == 0) return ok();
    if ((rc = check_slots(n_slots, slot_of_adapter, "slot_of_adapter", E))) return rc;
    CHECK_PTR(base, "base");
    CHECK_PTR(x, "x");
    CHECK_PTR(a, "a");
    CHECK_PTR(b, "b");
    if (scale) CHECK_PTR(scale, "scale");
    CHECK_PTR(offsets, "offsets");
    CHECK_PTR(gather, "gather");
    CHECK_PTR(out, "out");
    const size_t need = lora_ws(T, E, r, N, K);
    if (need) CHECK_PTR(ws, "ws");
    REQUIRE(ws_bytes >= need, FT_E_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
    const LoraArgs args{{offsets, slot_of_adapter, E, T, (uint32_t)n_slots}, gather, x, a, b, scale, base, out, r, N, K,
                        (flags & FT_OUT_BF16) != 0, (float*)ws};
    return hip_status(launch_lora(args, stream), "ft_moe_lora launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_lora: unexpected exception");
  }
}

}  // extern "C"
