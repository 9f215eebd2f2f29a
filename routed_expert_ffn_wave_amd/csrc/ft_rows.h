// Launch interface of the row kernels (8-bit rows and products, dispatch, gradients).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ftk {

// Which pairs have a row, and where (the pair tables of ft_moe_route / ft_moe_permute).
struct PairTab {
  const int32_t* ids;      // [T][k]
  const int32_t* inv;      // [T][k]
  const int32_t* slot_of;  // [E], or null: every expert counts
  int E, k, TK;            // TK = T * k
  uint32_t slots;          // entries of slot_of outside [0, slots) name no matrix
  // row of flat pair f, or -1 when it has none; nothing is read out of bounds for any table contents
  __device__ __forceinline__ int row(int f) const {
    const int e = ids[f];
    if ((unsigned)e >= (unsigned)E) return -1;
    if (slot_of && (uint32_t)slot_of[e] >= slots) return -1;
    const int r = inv[f];
    return (unsigned)r < (unsigned)TK ? r : -1;
  }
};

inline __host__ __device__ int fp8_scale_cols(int K) { return (K + 511) / 512 * 4; }

// Whether `items` fit a launch of blocks of `threads` threads with `per` items each: a launch counts its threads, whole
// blocks of them, in 32 bits.
inline bool launch_fits(long long items, int per, int threads) {
  return (items + per - 1) / per * threads < (1LL << 32);
}

constexpr int kRowsThreads = 256, kRowsScales = 32;      // a block of the 8-bit rows: 8 lanes a scale
constexpr int kDispatchThreads = 256, kDispatchWaves = 4;  // a block of the dispatch: a wave moves 4 KiB of a token's row

enum { ROWS_BF16 = 0, ROWS_F32 = 1, ROWS_SWIGLU = 2 };
// 8-bit rows of `rows` rows of K values; tab: null, or the pairs whose rows get them
hipError_t launch_rows_fp8(int kind, const void* x, int rows, int K, uint8_t* codes, float* scales, const PairTab* tab,
                           hipStream_t s);
hipError_t launch_dispatch(const void* x, const PairTab& tab, int T, int d, void* x_sorted, bool f32, hipStream_t s);
hipError_t launch_dispatch_grad(const void* dxs, const PairTab& tab, int T, int d, void* dx, bool f32, hipStream_t s);
hipError_t launch_combine_grad(const void* dout, const uint16_t* y, const float* w, const PairTab& tab, int T, int d,
                               uint16_t* dy, float* dw, float* dlogits, bool dout_bf16, hipStream_t s);

// Product of 8-bit rows with block-scaled weights; E == 0: one matrix for all rows.
struct Fp8MatmulArgs {
  const uint8_t* a;    // [M][K]
  const float* sa;     // [M][S]
  const uint8_t* w;    // [n_slots][N][K]
  const float* sw;     // [n_slots][ceil(N/128)][ceil(K/128)]
  int M, N, K, S, n_slots;
  const int32_t* offsets;  // [E+1]
  const int32_t* slot_of;  // [E]
  int E;
  void* out;
  bool out_bf16;
};
hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t s);

}  // namespace ftk
