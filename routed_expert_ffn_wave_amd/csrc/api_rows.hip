// C ABI of the row calls (declared in include/ft_moe_rows.h): host-side validation and kernel launches
// on the caller's stream.  Nothing here allocates, synchronises or throws across the ABI.
#include <hip/hip_runtime.h>

#include "../../include/ft_moe_rows.h"
#include "ft_api.h"
#include "ft_rows.h"

namespace {

using namespace ftk;

int check_flags(int flags, int known) {
  REQUIRE((flags & ~known) == 0, FT_E_INVAL, "unknown flags 0x%x", flags & ~known);
  return FT_OK;
}

// 8-bit rows of K values and the work of quantising `rows` of them
int check_rows_fp8(int rows, int K, const char* rows_name, const char* K_name) {
  REQUIRE(rows >= 0, FT_E_INVAL, "%s must be >= 0 (got %d)", rows_name, rows);
  REQUIRE(K > 0 && K % 16 == 0 && K <= (1 << 20), FT_E_INVAL, "%s must be a positive multiple of 16, at most 2^20 (got %d)",
          K_name, K);
  REQUIRE(launch_fits((long long)rows * fp8_scale_cols(K), kRowsScales, kRowsThreads), FT_E_UNSUPPORTED,
          "%s too large (%d rows of %d values)", rows_name, rows, K);
  return FT_OK;
}

int check_pairs(int T, int E, int k, int d, int multiple) {
  int rc = check_tek(T, E, k);
  if (rc) return rc;
  REQUIRE(d > 0 && d % multiple == 0 && d <= (1 << 20), FT_E_INVAL,
          "d must be a positive multiple of %d, at most 2^20 (got %d)", multiple, d);
  // 1024 values: 4 KiB in fp32
  REQUIRE(launch_fits((long long)T * ((d + 1023) / 1024), kDispatchWaves, kDispatchThreads), FT_E_UNSUPPORTED,
          "T too large (%d tokens of %d values)", T, d);
  return FT_OK;
}

#define CHECK_TAB()                                        \
  do {                                                     \
    CHECK_PTR(ids, "ids");                                 \
    CHECK_PTR(inv, "inv");                                 \
    if (slot_of_expert) CHECK_PTR(slot_of_expert, "slot_of_expert"); \
    REQUIRE(slot_of_expert || flag_slots(flags) == 0, FT_E_INVAL, "FT_N_SLOTS without slot_of_expert"); \
  } while (0)

PairTab pair_tab(const int32_t* ids, const int32_t* inv, const int32_t* slot_of, int T, int E, int k, int flags) {
  const int n = flag_slots(flags);
  return PairTab{ids, inv, slot_of, E, k, T * k, n ? (uint32_t)n : 0x80000000u};
}

int check_matmul(int rows, const char* rows_name, int N, int K, int E, int flags) {
  int rc = check_flags(flags, FT_OUT_BF16);
  if (rc) return rc;
  REQUIRE(rows >= 0 && rows <= (1 << 30), FT_E_INVAL, "%s must be in [0, 2^30] (got %d)", rows_name, rows);
  REQUIRE(N > 0 && N <= (1 << 24), FT_E_INVAL, "N must be in [1, 2^24] (got %d)", N);
  REQUIRE(K > 0 && K % 16 == 0 && K <= (1 << 20), FT_E_INVAL, "K must be a positive multiple of 16, at most 2^20 (got %d)", K);
  REQUIRE(((long long)rows / 16 + 1 + E) * ((N + 15) / 16) < (1LL << 31), FT_E_UNSUPPORTED,
          "product too large (%d rows, N=%d)", rows, N);
  return FT_OK;
}

int run_matmul(const Fp8MatmulArgs& m, const char* what, hipStream_t stream) {
  const hipError_t e = launch_fp8_matmul(m, stream);
  REQUIRE(e != hipErrorNotSupported, FT_E_UNSUPPORTED, "product too large (%d rows, N=%d, E=%d)", m.M, m.N, m.E);
  return hip_status(e, what);
}

}  // namespace

extern "C" {

int ft_moe_fp8_scale_cols(int K) { return K > 0 ? (int)((K + 511LL) / 512 * 4) : 0; }

int ft_moe_quant_fp8(const void* x, int rows, int K, uint8_t* codes, float* scales, int flags, hipStream_t stream) {
  try {
    int rc = check_rows_fp8(rows, K, "rows", "K");
    if (rc) return rc;
    if ((rc = check_flags(flags, FT_ROWS_F32))) return rc;
    if (rows == 0) return ok();
    CHECK_PTR(x, "x");
    CHECK_PTR(codes, "codes");
    CHECK_PTR(scales, "scales");
    return hip_status(launch_rows_fp8(flags & FT_ROWS_F32 ? ROWS_F32 : ROWS_BF16, x, rows, K, codes, scales, nullptr, stream),
                      "ft_moe_quant_fp8 launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_quant_fp8: unexpected exception");
  }
}

int ft_moe_swiglu_fp8(const uint16_t* gu, int rows, int I, uint8_t* codes, float* scales, hipStream_t stream) {
  try {
    int rc = check_rows_fp8(rows, I, "rows", "I");
    if (rc) return rc;
    if (rows == 0) return ok();
    CHECK_PTR(gu, "gu");
    CHECK_PTR(codes, "codes");
    CHECK_PTR(scales, "scales");
    return hip_status(launch_rows_fp8(ROWS_SWIGLU, gu, rows, I, codes, scales, nullptr, stream), "ft_moe_swiglu_fp8 launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_swiglu_fp8: unexpected exception");
  }
}

int ft_moe_dispatch(const void* x, const int32_t* ids, const int32_t* inv, const int32_t* slot_of_expert, int T, int E,
                    int k, int d, void* x_sorted, int flags, hipStream_t stream) {
  try {
    int rc = check_pairs(T, E, k, d, 8);
    if (rc) return rc;
    if ((rc = check_flags(flags, FT_ROWS_F32 | kSlotFlags))) return rc;
    if (T == 0) return ok();
    CHECK_PTR(x, "x");
    CHECK_TAB();
    CHECK_PTR(x_sorted, "x_sorted");
    const PairTab tab = pair_tab(ids, inv, slot_of_expert, T, E, k, flags);
    return hip_status(launch_dispatch(x, tab, T, d, x_sorted, (flags & FT_ROWS_F32) != 0, stream), "ft_moe_dispatch launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_dispatch: unexpected exception");
  }
}

int ft_moe_dispatch_fp8(const void* x, const int32_t* ids, const int32_t* inv, const int32_t* slot_of_expert, int T,
                        int E, int k, int d, uint8_t* codes, float* scales, int flags, hipStream_t stream) {
  try {
    int rc = check_pairs(T, E, k, d, 16);
    if (rc) return rc;
    if ((rc = check_rows_fp8(T, d, "T", "d"))) return rc;
    if ((rc = check_flags(flags, FT_ROWS_F32 | kSlotFlags))) return rc;
    if (T == 0) return ok();
    CHECK_PTR(x, "x");
    CHECK_TAB();
    CHECK_PTR(codes, "codes");
    CHECK_PTR(scales, "scales");
    const PairTab tab = pair_tab(ids, inv, slot_of_expert, T, E, k, flags);
    return hip_status(launch_rows_fp8(flags & FT_ROWS_F32 ? ROWS_F32 : ROWS_BF16, x, T, d, codes, scales, &tab, stream),
                      "ft_moe_dispatch_fp8 launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_dispatch_fp8: unexpected exception");
  }
}

int ft_moe_dispatch_grad(const void* dx_sorted, const int32_t* ids, const int32_t* inv, const int32_t* slot_of_expert,
                         int T, int E, int k, int d, void* dx, int flags, hipStream_t stream) {
  try {
    int rc = check_pairs(T, E, k, d, 8);
    if (rc) return rc;
    if ((rc = check_flags(flags, FT_ROWS_F32 | kSlotFlags))) return rc;
    if (T == 0) return ok();
    CHECK_PTR(dx_sorted, "dx_sorted");
    CHECK_TAB();
    CHECK_PTR(dx, "dx");
    const PairTab tab = pair_tab(ids, inv, slot_of_expert, T, E, k, flags);
    return hip_status(launch_dispatch_grad(dx_sorted, tab, T, d, dx, (flags & FT_ROWS_F32) != 0, stream),
                      "ft_moe_dispatch_grad launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_dispatch_grad: unexpected exception");
  }
}

int ft_moe_combine_grad(const void* dout, const uint16_t* y_sorted, const int32_t* ids, const float* w,
                        const int32_t* inv, const int32_t* slot_of_expert, int T, int E, int k, int d,
                        uint16_t* dy_sorted, float* dw, float* dlogits, int flags, hipStream_t stream) {
  try {
    int rc = check_pairs(T, E, k, d, 8);
    if (rc) return rc;
    if ((rc = check_flags(flags, FT_OUT_BF16 | kSlotFlags))) return rc;
    REQUIRE(T < (1 << 24), FT_E_UNSUPPORTED, "T too large (%d tokens, a block of 256 threads each)", T);
    if (T == 0) return ok();
    CHECK_PTR(dout, "dout");
    CHECK_PTR(y_sorted, "y_sorted");
    CHECK_PTR(w, "w");
    CHECK_TAB();
    CHECK_PTR(dy_sorted, "dy_sorted");
    CHECK_PTR(dw, "dw");
    if (dlogits) CHECK_PTR(dlogits, "dlogits");
    const PairTab tab = pair_tab(ids, inv, slot_of_expert, T, E, k, flags);
    return hip_status(launch_combine_grad(dout, y_sorted, w, tab, T, d, dy_sorted, dw, dlogits, (flags & FT_OUT_BF16) != 0,
                                          stream),
                      "ft_moe_combine_grad launch");
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_combine_grad: unexpected exception");
  }
}

int ft_moe_fp8_matmul(const uint8_t* a, const float* a_scales, int M, const uint8_t* w, const float* w_scales, int N,
                      int K, void* out, int flags, hipStream_t stream) {
  try {
    int rc = check_matmul(M, "M", N, K, 0, flags);
    if (rc) return rc;
    if (M == 0) return ok();
    CHECK_PTR(a, "a");
    CHECK_PTR(a_scales, "a_scales");
    CHECK_PTR(w, "w");
    CHECK_PTR(w_scales, "w_scales");
    CHECK_PTR(out, "out");
    Fp8MatmulArgs m{a, a_scales, w, w_scales, M, N, K, fp8_scale_cols(K), 1, nullptr, nullptr, 0, out,
                    (flags & FT_OUT_BF16) != 0};
    return run_matmul(m, "ft_moe_fp8_matmul launch", stream);
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_fp8_matmul: unexpected exception");
  }
}

int ft_moe_fp8_grouped_matmul(const uint8_t* a, const float* a_scales, int P, const uint8_t* w, const float* w_scales,
                              int n_slots, int N, int K, const int32_t* offsets, const int32_t* slot_of_expert, int E,
                              void* out, int flags, hipStream_t stream) {
  try {
    REQUIRE(E >= 1 && E <= 1024, FT_E_INVAL, "E must be in [1, 1024] (got %d)", E);
    REQUIRE(n_slots >= 1, FT_E_INVAL, "n_slots must be >= 1 (got %d)", n_slots);
    int rc = check_matmul(P, "P", N, K, E, flags);
    if (rc) return rc;
    if (P == 0) return ok();
    CHECK_PTR(a, "a");
    CHECK_PTR(a_scales, "a_scales");
    CHECK_PTR(w, "w");
    CHECK_PTR(w_scales, "w_scales");
    CHECK_PTR(offsets, "offsets");
    CHECK_PTR(slot_of_expert, "slot_of_expert");
    CHECK_PTR(out, "out");
    Fp8MatmulArgs m{a, a_scales, w, w_scales, P, N, K, fp8_scale_cols(K), n_slots, offsets, slot_of_expert, E, out,
                    (flags & FT_OUT_BF16) != 0};
    return run_matmul(m, "ft_moe_fp8_grouped_matmul launch", stream);
  } catch (...) {
    return fail(FT_E_INTERNAL, "ft_moe_fp8_grouped_matmul: unexpected exception");
  }
}

}  // extern "C"
