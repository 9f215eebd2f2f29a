// Products of 8-bit rows with block-scaled 8-bit weights, dense and grouped by expert (the FP8 block
// linear of the FreeToken walk-through "深入FreeToken架构…全链路剖析", section 六, over the expert groups of
// section 五):  out[m][n] = sum_b sa[m][b] sw[n/128][b] sum_{k in b} a[m][k] w[n][k],  b = blocks of 128.
//
// fp8_rows_kernel: few rows.  A block takes 16 NF weight rows and up to 16 MT activation rows over the whole of
// K; its 8 waves take the 128-blocks in turn and their sums meet in LDS in a fixed order, so a single row
// already keeps 8 waves a block busy with weight loads.  Codes are widened to bf16 (exact) and
// multiplied on v_mfma_f32_16x16x32_bf16: products exact, fp32 sums.  Bound by the weights' bytes.
#include "ft_device.h"
#include "ft_groups.h"
#include "ft_kernels.h"
#include "ft_rows.h"

namespace ftk {
namespace {

constexpr int RW = 8;  // waves per block

// 16 e4m3 codes as two operands of 8 bf16 values
__device__ __forceinline__ void widen(const u32x4& c, bf16x8 (&o)[2]) {
  uint32_t p[8];
  Chunk<FMT_FP8_B128>::decode(c, p);
  o[0] = __builtin_bit_cast(bf16x8, u32x4{p[0], p[1], p[2], p[3]});
  o[1] = __builtin_bit_cast(bf16x8, u32x4{p[4], p[5], p[6], p[7]});
}

struct Tile {
  int slot, row0, rows, n0;
};

template <int MT, int NF, bool BF16>
__device__ __forceinline__ void rows_tile(const Fp8MatmulArgs& a, const Tile& tl, float* s_part) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nb = (a.K + 127) / 128, nblk_n = (a.N + 127) / 128;
  // lane (r, g) holds row r and the 16-byte chunks g and g + 4 of a 128-block: any order of k that both
  // operands share is the same sum.  Rows past the end repeat the last one; their results are not stored.
  const uint8_t* wp[NF];
  const uint8_t* ap[MT];
  const float* sp[MT];
#pragma unroll
  for (int f = 0; f < NF; ++f) wp[f] = a.w + ((size_t)tl.slot * a.N + min(tl.n0 + 16 * f + r, a.N - 1)) * a.K;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const size_t row = (size_t)tl.row0 + min(16 * m + r, tl.rows - 1);
    ap[m] = a.a + row * a.K;
    sp[m] = a.sa + row * a.S;
  }
  const float* swp = a.sw + ((size_t)tl.slot * nblk_n + tl.n0 / 128) * nb;  // 16 NF rows lie in one 128-block
  f32x4 acc[MT][NF];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  for (int b = wv; b < nb; b += RW) {
    const float sw = swp[b];
    u32x4 wc[NF][2], ac[MT][2];
    float sa[MT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = b * 128 + (g + 4 * h) * 16;
      const bool in = c < a.K;  // chunks past K count as zero codes
#pragma unroll
      for (int f = 0; f < NF; ++f) wc[f][h] = in ? *(const u32x4*)(wp[f] + c) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int m = 0; m < MT; ++m) ac[m][h] = in ? *(const u32x4*)(ap[m] + c) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] = sp[m][b];
    f32x4 part[MT][NF];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) part[m][f] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 wb[NF][2], ab[2];
#pragma unroll
      for (int f = 0; f < NF; ++f) widen(wc[f][h], wb[f]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        widen(ac[m][h], ab);
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            part[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[f][q], ab[q], part[m][f], 0, 0, 0);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][f][i] = fmaf(part[m][f][i], sa[m] * sw, acc[m][f][i]);
  }
  // lane (r, g) of a fragment holds row (activation) r and columns 4 g .. 4 g + 3 of the 16 weight rows
  constexpr int NV = MT * NF * 256;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) *(f32x4*)(s_part + wv * NV + ((m * NF + f) * 16 + r) * 16 + 4 * g) = acc[m][f];
  __syncthreads();
  for (int i = threadIdx.x; i < NV; i += 64 * RW) {
    float v = s_part[i];
#pragma unroll
    for (int q = 1; q < RW; ++q) v += s_part[q * NV + i];
    const int fr = i >> 8, rr = (i >> 4) & 15, cc = i & 15;
    const int m = 16 * (fr / NF) + rr, n = tl.n0 + 16 * (fr % NF) + cc;
    if (m < tl.rows && n < a.N) {
      const size_t at = (size_t)(tl.row0 + m) * a.N + n;
      if (BF16)
        ((uint16_t*)a.out)[at] = f32_to_bf16_bits(v);
      else
        ((float*)a.out)[at] = v;
    }
  }
  __syncthreads();
}

template <int MT, int NF, bool BF16, bool GROUPED>
__global__ __launch_bounds__(64 * RW) void fp8_rows_kernel(Fp8MatmulArgs a) {
  __shared__ __attribute__((aligned(16))) float s_part[RW * MT * NF * 256];
  const int ntn = (a.N + 16 * NF - 1) / (16 * NF);
  if constexpr (!GROUPED) {
    const int mt = blockIdx.x / ntn, nt = blockIdx.x % ntn;
    rows_tile<MT, NF, BF16>(a, Tile{0, mt * 16 * MT, min(16 * MT, a.M - mt * 16 * MT), nt * 16 * NF}, s_part);
  } else {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int E2 = a.E + 2;
    GroupList gl{(int*)lds, (int*)lds + E2, (int*)lds + 2 * E2, (int*)lds + 3 * E2, 0};
    build_clipped_groups(a.slot_of, a.offsets, a.E, a.M, a.n_slots, gl, (int*)lds + 4 * E2,
                         [&](int cnt) { return (cnt + 16 * MT - 1) / (16 * MT) * ntn; });
    const int nitems = gl.item0[gl.n];
    for (int it = blockIdx.x; it < nitems; it += gridDim.x) {
      const int gi = find_group(gl.item0, gl.n, it);
      const int local = it - gl.item0[gi], mt = local / ntn, nt = local % ntn;
      const int m0 = mt * 16 * MT;
      rows_tile<MT, NF, BF16>(a, Tile{gl.slot[gi], gl.row0[gi] + m0, min(16 * MT, gl.cnt[gi] - m0), nt * 16 * NF},
                              s_part);
    }
  }
}

template <int MT, int NF, bool BF16>
hipError_t launch_rows(const Fp8MatmulArgs& a, hipStream_t s) {
  const long long ntn = (a.N + 16 * NF - 1) / (16 * NF), ntm = (a.M + 16 * MT - 1) / (16 * MT);
  if (a.E == 0) {
    hipLaunchKernelGGL((fp8_rows_kernel<MT, NF, BF16, false>), dim3((uint32_t)(ntn * ntm)), dim3(64 * RW), 0, s, a);
    return hipGetLastError();
  }
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = group_lds_bytes(a.E);
  hipError_t e = cache.get((const void*)fp8_rows_kernel<MT, NF, BF16, true>, 64 * RW, lds, &f);
  if (e != hipSuccess) return e;
  const long long upper = (ntm + (a.E < a.M ? a.E : a.M)) * ntn, most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL((fp8_rows_kernel<MT, NF, BF16, true>), dim3((uint32_t)(upper < most ? upper : most)), dim3(64 * RW),
                     lds, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t s) {
  if (a.out_bf16) return launch_rows<4, 1, true>(a, s);
  return launch_rows<4, 1, false>(a, s);
}

}  // namespace ftk
