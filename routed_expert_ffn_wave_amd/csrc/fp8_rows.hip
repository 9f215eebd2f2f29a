// Rows to 8-bit rows: e4m3 codes with one fp32 scale per 128 values (the activation side of the FP8
// block linear of the FreeToken walk-through "深入FreeToken架构…全链路剖析", section 六), as they lie, in
// expert order, or of SiLU(g) * u.
//
// Per block of 128: top = max(|x|, 2^-100), code = nearest e4m3 of 448 x / top, scale = top / 448.
// Eight lanes hold a block, 16 values each: two 16-byte loads (bf16), one 16-byte store of codes, the
// maximum over three lane exchanges.  The quotient is formed without a division per value: with
// top = m 2^e, y = x * (448 / 2^e) is exact for bf16 x (8 + 3 significant bits), q0 = y * rcp(m), and one
// residual step q = q0 + (y - q0 m) * rcp(m).  For bf16 x a quotient is either a rounding border of
// e4m3 or at least 2^-13 away from one (numerator 11 bits, denominator 8, border 5), and a border is hit
// exactly by the residual step, so the codes are the exact ones.  (For fp32 x, y is rounded too: quotients are off by
// up to 3 roundings, and a code may be the other neighbour of a border that close.)
//
// In expert order a token's row is quantised once and its codes are stored at each of its k rows:
// x is read once instead of k times.
//
// Bound by HBM; a few rows by the launch.  Eight lanes a block keep every access at 16 bytes a lane (32 read as bf16)
// and the codes of a block on one 128-byte line, and a wave holds 8 blocks, so a single row of 7168 already takes 7
// waves.  Measured: SwiGLU of 43541 rows, I = 2048, 449 MB in 80 us (5.6 TB/s; a 4 GiB copy reaches 4.9); 4096
// rows of 2048 to 8 rows each, 86 MB in 15 us (5.8 TB/s); 16 rows of 7168 in 2.4 us.
#include "ft_device.h"
#include "ft_rows.h"

namespace ftk {
namespace {

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// maximum over the 8 lanes of a block (lane exchanges inside a row of 16 lanes)
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // mirror inside 8 lanes
  return v;
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  // 1 / (1 + 2^(-g log2 e)): exp2 overflows to infinity for very negative g and the product is -0
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
  return g * s * u;
}

template <int KIND>
__device__ __forceinline__ void load16(const void* x, size_t row, int K, int col, float (&v)[16]) {
  if constexpr (KIND == ROWS_F32) {
    const f32x4* p = (const f32x4*)((const float*)x + row * K + col);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 w = p[q];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = w[i];
    }
  } else {
    const u32x4* p = (const u32x4*)((const uint16_t*)x + row * (size_t)(KIND == ROWS_SWIGLU ? 2 * K : K) + col);
    const u32x4 w[2] = {p[0], p[1]};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_bits_to_f32(w[i / 4][i % 4] & 0xffffu);
      v[2 * i + 1] = __uint_as_float(w[i / 4][i % 4] & 0xffff0000u);
    }
    if constexpr (KIND == ROWS_SWIGLU) {
      const u32x4* pu = (const u32x4*)((const uint16_t*)x + row * (size_t)(2 * K) + K + col);
      const u32x4 u[2] = {pu[0], pu[1]};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[2 * i] = silu_mul(v[2 * i], bf16_bits_to_f32(u[i / 4][i % 4] & 0xffffu));
        v[2 * i + 1] = silu_mul(v[2 * i + 1], __uint_as_float(u[i / 4][i % 4] & 0xffff0000u));
      }
    }
  }
}

template <int KIND, bool SORT>
__global__ __launch_bounds__(256) void rows_fp8_kernel(const void* __restrict__ x, uint32_t nunits, int K, int S,
                                                       uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                       PairTab tab) {
  const int lane = threadIdx.x & 63, l8 = lane & 7;
  const uint32_t u = blockIdx.x * 32u + (threadIdx.x >> 3);
  if (u >= nunits) return;  // whole groups of 8 lanes
  const uint32_t row = u / (uint32_t)S, b = u - row * (uint32_t)S;
  const int col = (int)b * 128 + l8 * 16;
  const bool has = col < K;  // K % 16 == 0: a lane's 16 values are all inside or all outside
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (has) load16<KIND>(x, row, K, col, v);
  uint32_t m = 0;  // magnitudes compare as integers; NaN and infinity above every finite value
#pragma unroll
  for (int i = 0; i < 16; ++i) m = umax(m, __float_as_uint(v[i]) & 0x7fffffffu);
  const uint32_t top = umax(max8(m), 0x0d800000u);  // 2^-100
  const float mant = __uint_as_float((top & 0x007fffffu) | 0x3f800000u);
  const float c = __uint_as_float(((262u - (top >> 23)) << 23) | 0x00600000u);  // 448 / 2^e
  const float inv = __builtin_amdgcn_rcpf(mant);
  const bool finite = top < 0x7f800000u;
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = v[4 * i + j] * c;
      const float q0 = y * inv;
      q[j] = fmaf(fmaf(-q0, mant, y), inv, q0);
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    o[i] = finite ? (uint32_t)w : 0x7f7f7f7fu;
  }
  const float t = __uint_as_float(top), s0 = t * (1.0f / 448.0f);
  float scale = fmaf(fmaf(-s0, 448.0f, t), 1.0f / 448.0f, s0);  // t / 448, correctly rounded
  if (!finite) scale = __uint_as_float(0x7fc00000u);
  if ((int)b * 128 >= K) scale = 0.0f;
  if constexpr (SORT) {
    for (int j0 = 0; j0 < tab.k; j0 += 8) {
      const int mine = j0 + l8 < tab.k ? tab.row((int)row * tab.k + j0 + l8) : -1;
      const int n = min(8, tab.k - j0);
      for (int j = 0; j < n; ++j) {
        const int r = __shfl(mine, (lane & ~7) + j, 64);
        if (r < 0) continue;
        if (has) *(u32x4*)(codes + (size_t)r * K + col) = o;
        if (l8 == 0) scales[(size_t)r * S + b] = scale;
      }
    }
  } else {
    if (has) *(u32x4*)(codes + (size_t)row * K + col) = o;
    if (l8 == 0) scales[(size_t)row * S + b] = scale;
  }
}

}  // namespace

hipError_t launch_rows_fp8(int kind, const void* x, int rows, int K, uint8_t* codes, float* scales, const PairTab* tab,
                           hipStream_t s) {
  const int S = fp8_scale_cols(K);
  const uint32_t n = (uint32_t)rows * (uint32_t)S;  // the caller checked that it fits
  const dim3 grid((n + kRowsScales - 1) / kRowsScales), block(kRowsThreads);
  const PairTab t = tab ? *tab : PairTab{};
#define LAUNCH(KIND, SORT) \
  hipLaunchKernelGGL((rows_fp8_kernel<KIND, SORT>), grid, block, 0, s, x, n, K, S, codes, scales, t)
  if (kind == ROWS_SWIGLU)
    LAUNCH(ROWS_SWIGLU, false);
  else if (kind == ROWS_F32 && tab)
    LAUNCH(ROWS_F32, true);
  else if (kind == ROWS_F32)
    LAUNCH(ROWS_F32, false);
  else if (tab)
    LAUNCH(ROWS_BF16, true);
  else
    LAUNCH(ROWS_BF16, false);
#undef LAUNCH
  return hipGetLastError();
}

}  // namespace ftk
