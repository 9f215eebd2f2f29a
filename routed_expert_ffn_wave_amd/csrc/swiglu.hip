// SwiGLU of bf16 rows and its gradient: h = SiLU(g) u with SiLU(g) = g s, s = 1 / (1 + e^-g);
//   dg = dh u s (1 + g (1 - s)),  du = dh g s.
// fp32 in between, one rounding at the end.
// A thread has 8 columns of a row: 16-byte loads and stores, no LDS, all of the GPU's waves in flight.  Bound by memory: 32768 rows of 768
// columns 24.0 us forward (151 MB, 6.3 TB/s), 43.4 us back (252 MB, 5.8 TB/s) with other calls' rows in between; 21.7 and 36.2 on the same
// rows again, part of which the last-level cache still has.  Non-temporal stores as in store_rows (27.5 / 26.0, back 46.5 / 43.8).
#include "ft_device.h"
#include "ft_products.h"

namespace ftk {
namespace {

constexpr int ST = 256;

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  return (uint32_t)f32_to_bf16_bits(a) | ((uint32_t)f32_to_bf16_bits(b) << 16);
}
// e^-g past fp32's range gives s = 0 (g < -88.7), and -0 or 0 times a finite u
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

template <bool GRAD>
__global__ __launch_bounds__(ST) void swiglu_kernel(const uint16_t* gu, const uint16_t* dh, uint32_t chunks, uint32_t per_row, uint16_t* out) {
  const uint32_t i = blockIdx.x * ST + threadIdx.x;  // chunk of 8 columns
  if (i >= chunks) return;
  const uint32_t row = i / per_row, c = i - row * per_row;
  const size_t at = ((size_t)row * 2 * per_row + c) * 8, up = at + (size_t)per_row * 8;
  const u32x4 g = *(const u32x4*)(gu + at), u = *(const u32x4*)(gu + up);
  if constexpr (!GRAD) {
    u32x4 h;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float g0 = lo(g[q]), g1 = hi(g[q]);
      h[q] = pack(g0 * sigmoid(g0) * lo(u[q]), g1 * sigmoid(g1) * hi(u[q]));
    }
    __builtin_nontemporal_store(h, (u32x4*)(out + (size_t)i * 8));
  } else {
    const u32x4 d = *(const u32x4*)(dh + (size_t)i * 8);
    u32x4 dg, du;
    auto one = [](float g, float u, float d, float& dg, float& du) {
      const float s = sigmoid(g), gs = g * s;
      du = d * gs;
      dg = d * u * (s + gs * (1.0f - s));
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float a0, b0, a1, b1;
      one(lo(g[q]), lo(u[q]), lo(d[q]), a0, b0);
      one(hi(g[q]), hi(u[q]), hi(d[q]), a1, b1);
      dg[q] = pack(a0, a1);
      du[q] = pack(b0, b1);
    }
    __builtin_nontemporal_store(dg, (u32x4*)(out + at));
    __builtin_nontemporal_store(du, (u32x4*)(out + up));
  }
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* gu, const uint16_t* dh, long long rows, int I, uint16_t* out, hipStream_t s) {
  const long long chunks = rows * (I / 8);
  const dim3 grid((uint32_t)((chunks + ST - 1) / ST));
  if (dh)
    hipLaunchKernelGGL(swiglu_kernel<true>, grid, dim3(ST), 0, s, gu, dh, (uint32_t)chunks, (uint32_t)(I / 8), out);
  else
    hipLaunchKernelGGL(swiglu_kernel<false>, grid, dim3(ST), 0, s, gu, dh, (uint32_t)chunks, (uint32_t)(I / 8), out);
  return hipGetLastError();
}

}  // namespace ftk
