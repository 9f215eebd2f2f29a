// Products of 8-bit rows with block-scaled 8-bit weights, dense and grouped by expert (the FP8 block
// linear of the FreeToken walk-through "深入FreeToken架构…全链路剖析", section 六, over the expert groups of
// section 五):  out[m][n] = sum_b sa[m][b] sw[n/128][b] sum_{k in b} a[m][k] w[n][k],  b = blocks of 128.
//
// fp8_rows_kernel: few rows.  A block takes 16 NF weight rows and up to 16 activation rows over the whole of
// K; its 8 waves take the 128-blocks in turn and their sums meet in LDS in a fixed order, so a single row
// already keeps 8 waves a block busy with weight loads.  Codes are widened to bf16 (exact) and
// multiplied on v_mfma_f32_16x16x32_bf16: products exact, fp32 sums.  Bound by the weights' bytes: 37 experts
// of 4096 x 7168 with one to three rows each, 1087 MB, in 183 us, 5.9 TB/s.  (More rows a block do not pay: a lane's
// 16-byte chunks of 16 different rows cost the address unit 64 cycles a load, where 8 lanes a row cost 16;
// 64 x 32 blocks of 128 rows took 28 us against 18 for the 64 x 64 tiles loaded through LDS.)
#include "fp8_choice.h"
#include "fp8_tile.h"
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

template <int NF, bool BF16>
__device__ __forceinline__ void rows_tile(const Fp8MatmulArgs& a, const Tile& tl, float* s_part) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nb = (a.K + 127) / 128, nblk_n = (a.N + 127) / 128;
  // lane (r, g) holds row r and the 16-byte chunks g and g + 4 of a 128-block: any order of k that both
  // operands share is the same sum.  Rows past the end repeat the last one; their results are not stored.
  const uint8_t* wb = a.w + ((size_t)tl.slot * a.N + tl.n0) * a.K;
  const uint8_t* ab = a.a + (size_t)tl.row0 * a.K;
  uint32_t wo[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) wo[f] = (uint32_t)min(16 * f + r, a.N - 1 - tl.n0) * (uint32_t)a.K + g * 16;
  const uint32_t row = (uint32_t)min(r, tl.rows - 1), ao = row * (uint32_t)a.K + g * 16;
  const float* sap = a.sa + (size_t)tl.row0 * a.S + row * (uint32_t)a.S;
  // 16 NF rows lie in one 128-block.  (lane >> 6 is 0, but by lane: vector loads, which complete in order, where a scalar
  // load is waited for together with every LDS operation.)
  const float* swp = a.sw + ((size_t)tl.slot * nblk_n + tl.n0 / 128) * nb + (lane >> 6);
  f32x4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4{0, 0, 0, 0};
  // A block's operands in registers: the next block is in flight while one is multiplied.
  struct Regs {
    u32x4 w[NF][2], a[2];
    float sa, sw;
  };
  auto load = [&](Regs& x, int b) {
    if (b * 128 + 128 <= a.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int f = 0; f < NF; ++f) x.w[f][h] = *(const u32x4*)(wb + (size_t)b * 128 + 64 * h + wo[f]);
        x.a[h] = *(const u32x4*)(ab + (size_t)b * 128 + 64 * h + ao);
      }
    } else {  // the short block, or none: chunks past K count as zero codes
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = b * 128 + (g + 4 * h) * 16 < a.K;
        const size_t at = in ? (size_t)b * 128 + 64 * h : 0;
        const u32x4 none = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < NF; ++f) x.w[f][h] = in ? *(const u32x4*)(wb + at + wo[f]) : none;
        x.a[h] = in ? *(const u32x4*)(ab + at + ao) : none;
      }
    }
    x.sa = sap[min(b, nb - 1)];
    x.sw = swp[min(b, nb - 1)];
  };
  auto multiply = [&](const Regs& x) {
    f32x4 part[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) part[f] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 wf[2], af[2];
      widen(x.a[h], af);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        widen(x.w[f][h], wf);
#pragma unroll
        for (int q = 0; q < 2; ++q) part[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[q], af[q], part[f], 0, 0, 0);
      }
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(part[f][i], x.sa * x.sw, acc[f][i]);
  };
  Regs even, odd;
  load(even, wv);
  for (int b = wv; b < nb; b += 2 * RW) {
    load(odd, b + RW);
    multiply(even);
    if (b + RW >= nb) break;
    load(even, b + 2 * RW);
    multiply(odd);
  }
  // lane (r, g) of a fragment holds activation row r and columns 4 g .. 4 g + 3 of the 16 weight rows
  constexpr int NV = NF * 256;
#pragma unroll
  for (int f = 0; f < NF; ++f) *(f32x4*)(s_part + wv * NV + (f * 16 + r) * 16 + 4 * g) = acc[f];
  __syncthreads();
  for (int i = threadIdx.x; i < NV; i += 64 * RW) {
    float v = s_part[i];
#pragma unroll
    for (int q = 1; q < RW; ++q) v += s_part[q * NV + i];
    const int m = (i >> 4) & 15, n = tl.n0 + 16 * (i >> 8) + (i & 15);
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

template <int NF, bool BF16, bool GROUPED>
__global__ __launch_bounds__(64 * RW) void fp8_rows_kernel(Fp8MatmulArgs a) {
  __shared__ __attribute__((aligned(16))) float s_part[RW * NF * 256];
  const int ntn = (a.N + 16 * NF - 1) / (16 * NF);
  if constexpr (!GROUPED) {
    const int mt = blockIdx.x / ntn, nt = blockIdx.x % ntn;
    rows_tile<NF, BF16>(a, Tile{0, mt * 16, min(16, a.M - mt * 16), nt * 16 * NF}, s_part);
  } else {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int E2 = a.E + 2;
    GroupList gl{(int*)lds, (int*)lds + E2, (int*)lds + 2 * E2, (int*)lds + 3 * E2, 0};
    build_clipped_groups(a.slot_of, a.offsets, a.E, a.M, a.n_slots, gl, (int*)lds + 4 * E2,
                         [&](int cnt) { return (cnt + 15) / 16 * ntn; });
    const int nitems = gl.item0[gl.n];
    for (int it = blockIdx.x; it < nitems; it += gridDim.x) {
      const int gi = find_group(gl.item0, gl.n, it);
      const int local = it - gl.item0[gi], m0 = local / ntn * 16, nt = local % ntn;
      rows_tile<NF, BF16>(a, Tile{gl.slot[gi], gl.row0[gi] + m0, min(16, gl.cnt[gi] - m0), nt * 16 * NF}, s_part);
    }
  }
}

template <int NF, bool BF16>
hipError_t launch_rows(const Fp8MatmulArgs& a, hipStream_t s) {
  const long long ntn = (a.N + 16 * NF - 1) / (16 * NF), ntm = (a.M + 15) / 16;
  if (a.E == 0) {
    hipLaunchKernelGGL((fp8_rows_kernel<NF, BF16, false>), dim3((uint32_t)(ntn * ntm)), dim3(64 * RW), 0, s, a);
    return hipGetLastError();
  }
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = group_lds_bytes(a.E);
  hipError_t e = cache.get((const void*)fp8_rows_kernel<NF, BF16, true>, 64 * RW, lds, &f);
  if (e != hipSuccess) return e;
  const long long upper = (ntm + (a.E < a.M ? a.E : a.M)) * ntn, most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL((fp8_rows_kernel<NF, BF16, true>), dim3((uint32_t)(upper < most ? upper : most)), dim3(64 * RW), lds, s, a);
  return hipGetLastError();
}

// Many rows: tiles of fp8_tile.h.  Blocks are placed on the 8 XCDs round-robin; each XCD gets a contiguous run
// of the tile list, so that tiles that run together share rows and weights through its L2.
template <class C, bool BF16, bool GROUPED>
__global__ __launch_bounds__(C::NT, 2) void fp8_tile_kernel(Fp8MatmulArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int ntn = (a.N + C::BN - 1) / C::BN;
  const int per = gridDim.x / 8, lb = (blockIdx.x % 8) * per + blockIdx.x / 8;  // gridDim.x % 8 == 0
  if constexpr (!GROUPED) {
    const int ntm = (a.M + C::BM - 1) / C::BM;
    if (lb >= ntm * ntn) return;
    // bands of 4 row tiles, weight tiles within a band in turn
    constexpr int BAND = 4;
    const int band = lb / (BAND * ntn), h = min(BAND, ntm - band * BAND), in = lb - band * BAND * ntn;
    const int mt = band * BAND + in % h, nt = in / h;
    fp8_tile<C, BF16>(a, TileJob{0, mt * C::BM, min(C::BM, a.M - mt * C::BM), nt * C::BN}, lds);
  } else {
    const int E2 = a.E + 2;
    int* li = (int*)(lds + C::LDS);
    GroupList gl{li, li + E2, li + 2 * E2, li + 3 * E2, 0};
    build_clipped_groups(a.slot_of, a.offsets, a.E, a.M, a.n_slots, gl, li + 4 * E2,
                         [&](int cnt) { return (cnt + C::BM - 1) / C::BM * ntn; });
    const int nitems = gl.item0[gl.n];
    for (int it = lb; it < nitems; it += gridDim.x) {
      const int gi = find_group(gl.item0, gl.n, it);
      const int local = __builtin_amdgcn_readfirstlane(it - gl.item0[gi]);
      const int slot = __builtin_amdgcn_readfirstlane(gl.slot[gi]);
      const int row0 = __builtin_amdgcn_readfirstlane(gl.row0[gi]), cnt = __builtin_amdgcn_readfirstlane(gl.cnt[gi]);
      const int m0 = local / ntn * C::BM, nt = local % ntn;
      fp8_tile<C, BF16>(a, TileJob{slot, row0 + m0, min(C::BM, cnt - m0), nt * C::BN}, lds);
    }
  }
}

template <class C, bool BF16>
hipError_t launch_dense_tiles(const Fp8MatmulArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const long long ntn = (a.N + C::BN - 1) / C::BN, ntm = (a.M + C::BM - 1) / C::BM;
  hipError_t e = cache.get((const void*)fp8_tile_kernel<C, BF16, false>, C::NT, C::LDS, &f);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((fp8_tile_kernel<C, BF16, false>), dim3((uint32_t)((ntn * ntm + 7) / 8 * 8)), dim3(C::NT), C::LDS, s, a);
  return hipGetLastError();
}

template <class C, bool BF16>
hipError_t launch_grouped_tiles(const Fp8MatmulArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const long long ntn = (a.N + C::BN - 1) / C::BN, ntm = (a.M + C::BM - 1) / C::BM;
  const size_t lds = C::LDS + group_lds_bytes(a.E);
  hipError_t e = cache.get((const void*)fp8_tile_kernel<C, BF16, true>, C::NT, lds, &f);
  if (e != hipSuccess) return e;
  const long long upper = ((ntm + (a.E < a.M ? a.E : a.M)) * ntn + 7) / 8 * 8, most = (long long)f.per_cu * f.cus / 8 * 8;
  hipLaunchKernelGGL((fp8_tile_kernel<C, BF16, true>), dim3((uint32_t)(upper < most ? upper : most)), dim3(C::NT), lds, s, a);
  return hipGetLastError();
}

template <class C, bool BF16>
hipError_t launch_tiles(const Fp8MatmulArgs& a, hipStream_t s) {
  return a.E == 0 ? launch_dense_tiles<C, BF16>(a, s) : launch_grouped_tiles<C, BF16>(a, s);
}

}  // namespace

hipError_t launch_fp8_matmul(const Fp8MatmulArgs& a, hipStream_t s) {
  if (!a.out_bf16) {
    switch (choose<false>(a)) {
      case -1: return hipErrorNotSupported;
      case 0: return launch_rows<1, false>(a, s);
      case 1: return launch_rows<2, false>(a, s);
      case 2: return launch_tiles<SoloWide, false>(a, s);
      case 3: return launch_dense_tiles<PairWide, false>(a, s);
      case 4: return launch_tiles<TWide, false>(a, s);
      default: return launch_grouped_tiles<TWide256, false>(a, s);
    }
  }
  switch (choose<true>(a)) {
    case -1: return hipErrorNotSupported;
    case 0: return launch_rows<1, true>(a, s);
    case 1: return launch_rows<2, true>(a, s);
    case 2: return launch_tiles<Solo, true>(a, s);
    case 3: return launch_dense_tiles<Pair64, true>(a, s);
    case 4: return launch_dense_tiles<Pair128, true>(a, s);
    case 5: return launch_grouped_tiles<T64, true>(a, s);
    case 6: return launch_grouped_tiles<T128, true>(a, s);
    case 7: return launch_tiles<T128x256, true>(a, s);
    default: return launch_tiles<T256, true>(a, s);
  }
}

}  // namespace ftk
