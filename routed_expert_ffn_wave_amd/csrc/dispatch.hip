// Token rows in expert order, their gradient, and the gradient of the weighted combine (the expert
// dispatch of the FreeToken walk-through "深入FreeToken架构…全链路剖析", section 一, for a training step).
//
// All three move rows and are bound by HBM.  They work per token, not per sorted row: a token's row is
// read once for its k copies (forward) and its k rows are summed in registers (gradient), so no atomics are
// needed and every sum has a fixed order.  Rows are taken in pieces of 16 bytes a lane.  A wave moves 4 KiB: with 4 loads
// in flight a lane, and with a block or more per compute unit from about 500 rows of 2048 on.  Measured:
//   dispatch, 4096 rows of 7168 to 8 rows each: 529 MB in 106 us (5.0 TB/s; a 4 GiB copy reaches 4.9)
//   its gradient, 1023 x 8 rows of 2048 in fp32: 75 MB in 12 us (6.1 TB/s)
//   combine's gradient, 4096 tokens x 8 rows of 2048: 288 MB in 48 - 60 us; 8 tokens: 6.5 us
#include "ft_device.h"
#include "ft_rows.h"

namespace ftk {
namespace {

constexpr int SEG_U = 4;  // 16-byte pieces per lane: a wave moves 4 KiB of one row

__device__ __forceinline__ void unpack8(const u32x4& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_bf16_bits(v[2 * i]) | ((uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16);
  return o;
}

// Lane j: the row of pair f0 + j, -1 without one (also from k on): one chain of loads for all k pairs.
__device__ __forceinline__ int rows_of(const PairTab& tab, int f0) {
  const int lane = threadIdx.x & 63;
  return lane < tab.k ? tab.row(f0 + lane) : -1;
}

// One wave per (token, 4 KiB of its row).  pieces: 16-byte pieces per row.
__global__ __launch_bounds__(256) void dispatch_kernel(const u32x4* __restrict__ x, PairTab tab, uint32_t nwork,
                                                       uint32_t nseg, int pieces, u32x4* __restrict__ xs) {
  const uint32_t wk = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (wk >= nwork) return;
  const uint32_t t = wk / nseg;
  const int p0 = (int)(wk - t * nseg) * (64 * SEG_U) + (threadIdx.x & 63);
  u32x4 v[SEG_U];
#pragma unroll
  for (int q = 0; q < SEG_U; ++q)
    if (p0 + 64 * q < pieces) v[q] = x[(size_t)t * pieces + p0 + 64 * q];
  const int rows = rows_of(tab, (int)t * tab.k);
  for (int j = 0; j < tab.k; ++j) {
    const int r = __builtin_amdgcn_readlane(rows, j);
    if (r < 0) continue;
#pragma unroll
    for (int q = 0; q < SEG_U; ++q)
      if (p0 + 64 * q < pieces) xs[(size_t)r * pieces + p0 + 64 * q] = v[q];
  }
}

// The same partition: dx[t] = sum_j dxs[row(t, j)], in fp32, j ascending.  JB rows are loaded before the
// first is added.
template <bool F32>
__global__ __launch_bounds__(256) void dispatch_grad_kernel(const u32x4* __restrict__ dxs, PairTab tab, uint32_t nwork,
                                                            uint32_t nseg, int pieces, u32x4* __restrict__ dx) {
  constexpr int JB = 4, NV = F32 ? 4 : 8;
  const uint32_t wk = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (wk >= nwork) return;
  const uint32_t t = wk / nseg;
  const int p0 = (int)(wk - t * nseg) * (64 * SEG_U) + (threadIdx.x & 63);
  const int rows = rows_of(tab, (int)t * tab.k);
  float acc[SEG_U][NV];
#pragma unroll
  for (int q = 0; q < SEG_U; ++q)
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[q][i] = 0.0f;
  for (int j0 = 0; j0 < tab.k; j0 += JB) {
    u32x4 v[JB][SEG_U];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int r = __builtin_amdgcn_readlane(rows, j0 + j);  // -1 from k on (k <= 32)
#pragma unroll
      for (int q = 0; q < SEG_U; ++q) {
        v[j][q] = u32x4{0, 0, 0, 0};
        if (r >= 0 && p0 + 64 * q < pieces) v[j][q] = dxs[(size_t)r * pieces + p0 + 64 * q];
      }
    }
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int q = 0; q < SEG_U; ++q) {
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[q][i] += __uint_as_float(v[j][q][i]);
        } else {
          float f[8];
          unpack8(v[j][q], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[q][i] += f[i];
        }
      }
  }
#pragma unroll
  for (int q = 0; q < SEG_U; ++q)
    if (p0 + 64 * q < pieces) {
      u32x4 o;
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(acc[q][i]);
      } else {
        o = pack8(acc[q]);
      }
      dx[(size_t)t * pieces + p0 + 64 * q] = o;
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sums of 8 values over the wave: lane l gets the sum of value l % 8.  Three exchanges halve the values a lane holds,
// three more add the 8 partial sums of a value: 10 exchanges instead of 48.
__device__ __forceinline__ float wave_sums8(const float (&v)[8]) {
  const int lane = threadIdx.x & 63;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // keep the values whose bit 0 is the lane's
    const float keep = lane & 1 ? v[2 * i + 1] : v[2 * i], give = lane & 1 ? v[2 * i] : v[2 * i + 1];
    a[i] = keep + __shfl_xor(give, 1, 64);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 2 ? a[2 * i + 1] : a[2 * i], give = lane & 2 ? a[2 * i] : a[2 * i + 1];
    b[i] = keep + __shfl_xor(give, 2, 64);
  }
  const float keep = lane & 4 ? b[1] : b[0], give = lane & 4 ? b[0] : b[1];
  float s = keep + __shfl_xor(give, 4, 64);
#pragma unroll
  for (int o = 8; o <= 32; o <<= 1) s += __shfl_xor(s, o, 64);
  return s;
}

// One block per token: dy rows, the k dot products dout . y, and the row of dlogits.  Eight pairs are taken together,
// so dout is read once for k <= 8, and eight rows of y are in flight.  The pair tables are read once, a lane per pair,
// beside the first piece of dout.  (With the tables read pair by pair, three dependent loads each, and every dot
// product reduced alone, the kernel took 51 us instead of 48 for 4096 tokens and 8.6 instead of 6.5 for 8.)
template <bool BF16>
__global__ __launch_bounds__(256) void combine_grad_kernel(const void* __restrict__ dout,
                                                           const uint16_t* __restrict__ y,
                                                           const float* __restrict__ w, PairTab tab, int d,
                                                           uint16_t* __restrict__ dy, float* __restrict__ dw,
                                                           float* __restrict__ dlogits) {
  constexpr int JB = 8;
  __shared__ float s_part[4][32];
  __shared__ float s_dl[32];
  __shared__ int s_id[32];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int f0 = t * tab.k;
  const bool on = lane < tab.k;
  const int rows = rows_of(tab, f0), id = on ? tab.ids[f0 + lane] : -1;
  const float wl = on ? w[f0 + lane] : 0.0f;
  for (int j0 = 0; j0 < tab.k; j0 += JB) {
    int r[JB];
    float wj[JB], acc[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      r[j] = __builtin_amdgcn_readlane(rows, j0 + j);
      wj[j] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j0 + j));
      acc[j] = 0.0f;
    }
    for (int c = tid * 8; c < d; c += 256 * 8) {
      float g[8];
      if constexpr (BF16) {
        unpack8(*(const u32x4*)((const uint16_t*)dout + (size_t)t * d + c), g);
      } else {
        const f32x4* p = (const f32x4*)((const float*)dout + (size_t)t * d + c);
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = a[i], g[4 + i] = b[i];
      }
      u32x4 yv[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j)
        if (r[j] >= 0) yv[j] = *(const u32x4*)(y + (size_t)r[j] * d + c);
#pragma unroll
      for (int j = 0; j < JB; ++j)
        if (r[j] >= 0) {
          float f[8], o[8];
          unpack8(yv[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[j] = fmaf(g[i], f[i], acc[j]);
            o[i] = wj[j] * g[i];
          }
          *(u32x4*)(dy + (size_t)r[j] * d + c) = pack8(o);
        }
    }
    const float s = wave_sums8(acc);
    if (lane < JB) s_part[wv][j0 + lane] = s;  // k <= 32: j0 + 7 < 32
  }
  __syncthreads();
  if (tid < 64) {
    const float a = on ? (s_part[0][lane] + s_part[1][lane]) + (s_part[2][lane] + s_part[3][lane]) : 0.0f;
    if (on) dw[f0 + lane] = a;
    if (dlogits) {
      const float mean = wave_sum(on ? wl * a : 0.0f);
      if (on) {
        s_dl[lane] = wl * (a - mean);
        s_id[lane] = id;
      }
    }
  }
  if (!dlogits) return;
  __syncthreads();
  for (int e = tid; e < tab.E; e += 256) {
    float v = 0.0f;
    for (int j = 0; j < tab.k; ++j)
      if (s_id[j] == e) v += s_dl[j];
    dlogits[(size_t)t * tab.E + e] = v;
  }
}

}  // namespace

hipError_t launch_dispatch(const void* x, const PairTab& tab, int T, int d, void* xs, bool f32, hipStream_t s) {
  const int pieces = d / 8 * (f32 ? 2 : 1);
  const uint32_t nseg = (uint32_t)(pieces + 64 * SEG_U - 1) / (64 * SEG_U), nwork = (uint32_t)T * nseg;
  hipLaunchKernelGGL(dispatch_kernel, dim3((nwork + kDispatchWaves - 1) / kDispatchWaves), dim3(kDispatchThreads), 0, s, (const u32x4*)x, tab, nwork, nseg, pieces,
                     (u32x4*)xs);
  return hipGetLastError();
}

hipError_t launch_dispatch_grad(const void* dxs, const PairTab& tab, int T, int d, void* dx, bool f32, hipStream_t s) {
  const int pieces = d / 8 * (f32 ? 2 : 1);
  const uint32_t nseg = (uint32_t)(pieces + 64 * SEG_U - 1) / (64 * SEG_U), nwork = (uint32_t)T * nseg;
  const dim3 grid((nwork + kDispatchWaves - 1) / kDispatchWaves), block(kDispatchThreads);
  if (f32)
    hipLaunchKernelGGL(dispatch_grad_kernel<true>, grid, block, 0, s, (const u32x4*)dxs, tab, nwork, nseg, pieces,
                       (u32x4*)dx);
  else
    hipLaunchKernelGGL(dispatch_grad_kernel<false>, grid, block, 0, s, (const u32x4*)dxs, tab, nwork, nseg, pieces,
                       (u32x4*)dx);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const void* dout, const uint16_t* y, const float* w, const PairTab& tab, int T, int d,
                               uint16_t* dy, float* dw, float* dlogits, bool dout_bf16, hipStream_t s) {
  if (dout_bf16)
    hipLaunchKernelGGL(combine_grad_kernel<true>, dim3(T), dim3(256), 0, s, dout, y, w, tab, d, dy, dw, dlogits);
  else
    hipLaunchKernelGGL(combine_grad_kernel<false>, dim3(T), dim3(256), 0, s, dout, y, w, tab, d, dy, dw, dlogits);
  return hipGetLastError();
}

}  // namespace ftk
