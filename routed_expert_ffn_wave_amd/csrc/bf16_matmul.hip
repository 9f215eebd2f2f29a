// Products of bf16 rows with one matrix per expert, the gradient of the rows and the gradient of the matrices: what the
// expert FFN of a training step is made of (the expert groups of the FreeToken walk-through
// "深入FreeToken架构…全链路剖析", section 五).
//   forward        out[p][n]   = sum_k a[p][k] w[e][n][k]
//   rows           da[p][k]    = sum_n dout[p][n] w[e][n][k]
//   matrices       dw[e][n][k] = sum_{p of e} dout[p][n] a[p][k]
// bf16 products are exact in fp32 and added there by the matrix instructions; results are rounded once.
#include "bf16_tile.h"
#include "ft_groups.h"
#include "ft_kernels.h"
#include "ft_products.h"

namespace ftk {
namespace {

__device__ __forceinline__ bool group_of(const RowGroups& s, int e, int& slot, int& row0, int& cnt) {
  slot = s.slot_of ? s.slot_of[e] : e;
  row0 = min(max(s.offsets[e], 0), s.P);
  cnt = max(min(max(s.offsets[e + 1], 0), s.P) - row0, 0);
  return (uint32_t)slot < s.n_slots;
}

template <class ItemsOf>
__device__ __forceinline__ void list_groups(const RowGroups& s, GroupList& g, int* tmp, ItemsOf items_of) {
  build_group_list(
      s.E, g, tmp, [&](int e, int& slot, int& row0, int& cnt) { return e < s.E && group_of(s, e, slot, row0, cnt) && cnt > 0; }, items_of);
}

// A tile of up to BM rows takes the least of these heights that holds its rows.
template <int BM, bool GRAD, bool BF16>
__device__ __forceinline__ void grouped_tile(const GroupedArgs& a, int slot, int row0, int rows, int n0, uint8_t* lds) {
  using C = Bf16Cfg<BM, 256, 2, 4, BM == 64 ? 3 : 2>;
  const int cols = GRAD ? a.K : a.N, red = GRAD ? a.N : a.K;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint16_t* w = a.w + (size_t)slot * a.N * a.K;
  f32x4 acc[C::MF][C::NF];
  const Operand ro{a.a + (size_t)row0 * red, red, rows, nullptr, 0};
  const Operand co{GRAD ? w + n0 : w + (size_t)n0 * a.K, a.K, min(C::BN, cols - n0), nullptr, 0};
  bf16_tile<C, DIRECT, GRAD ? ACROSS : DIRECT>(ro, co, red, lds, acc);
  uint8_t* out = (uint8_t*)a.out + (size_t)row0 * cols * (BF16 ? 2 : 4);
  store_rows<C::MF, C::NF, BF16, false>(acc, out, cols, wv / C::WN * 16 * C::MF, rows, n0 + wv % C::WN * 16 * C::NF, cols, lane);
}

constexpr int kTileLds = 2 * (256 + 256) * 128;

// Blocks are placed on the 8 XCDs round-robin; each XCD gets a contiguous run of the tile list, so that tiles that run
// together share rows and matrices through its L2: bands of 4 row tiles, column tiles within a band in turn.
template <bool GRAD, bool BF16>
__global__ __launch_bounds__(512, 2) void grouped_tile_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int cols = GRAD ? a.K : a.N;
  const int ntn = (cols + 255) / 256;
  const int E2 = a.g.E + 2;
  int* li = (int*)(lds + kTileLds);
  GroupList gl{li, li + E2, li + 2 * E2, li + 3 * E2, 0};
  list_groups(a.g, gl, li + 4 * E2, [&](int cnt) { return (cnt + 255) / 256 * ntn; });
  const int nitems = gl.item0[gl.n];
  const int per = gridDim.x / 8, lb = (blockIdx.x % 8) * per + blockIdx.x / 8;  // gridDim.x % 8 == 0
  for (int it = lb; it < nitems; it += gridDim.x) {
    const int gi = find_group(gl.item0, gl.n, it);
    const int local = __builtin_amdgcn_readfirstlane(it - gl.item0[gi]);
    const int slot = __builtin_amdgcn_readfirstlane(gl.slot[gi]);
    const int row0 = __builtin_amdgcn_readfirstlane(gl.row0[gi]), cnt = __builtin_amdgcn_readfirstlane(gl.cnt[gi]);
    constexpr int BAND = 4;
    const int band = local / (BAND * ntn), h = min(BAND, (cnt + 255) / 256 - band * BAND), in = local - band * BAND * ntn;
    const int m0 = (band * BAND + in % h) * 256, n0 = in / h * 256, rows = min(256, cnt - m0);
    if (rows > 192)
      grouped_tile<256, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
    else if (rows > 128)
      grouped_tile<192, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
    else if (rows > 64)
      grouped_tile<128, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
    else
      grouped_tile<64, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
  }
}

template <class C, bool BF16, bool ADD>
__global__ __launch_bounds__(C::NT, 2) void wgrad_tile_kernel(WgradArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int ntm = (a.N + C::BM - 1) / C::BM, ntn = (a.K + C::BN - 1) / C::BN, tiles = ntm * ntn;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.x / tiles, t = blockIdx.x % tiles;
  int slot, row0, cnt;
  if (!group_of(a.g, e, slot, row0, cnt)) return;
  row0 = __builtin_amdgcn_readfirstlane(row0), cnt = __builtin_amdgcn_readfirstlane(cnt);
  if (ADD && cnt == 0) return;
  const int m0 = t / ntn * C::BM, n0 = t % ntn * C::BN;
  f32x4 acc[C::MF][C::NF];
  const Operand ro{a.dout + (size_t)row0 * a.N + m0, a.N, min(C::BM, a.N - m0), nullptr, 0};
  const Operand co{a.a + (size_t)row0 * a.K + n0, a.K, min(C::BN, a.K - n0), nullptr, 0};
  bf16_tile<C, ACROSS, ACROSS>(ro, co, cnt, lds, acc);
  uint8_t* out = (uint8_t*)a.dw + ((size_t)e * a.N + m0) * a.K * (BF16 ? 2 : 4);
  store_rows<C::MF, C::NF, BF16, ADD>(acc, out, a.K, wv / C::WN * 16 * C::MF, ro.rows, n0 + wv % C::WN * 16 * C::NF, a.K, lane);
}

template <bool GRAD, bool BF16>
hipError_t launch_tiles(const GroupedArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const int cols = GRAD ? a.K : a.N, E = a.g.E, P = a.g.P;
  const long long ntn = (cols + 255) / 256, ntm = (P + 255) / 256;
  if ((P / 256 + 2LL) * (E / 2 + 1) * ntn >= 1LL << 31) return hipErrorNotSupported;
  const size_t lds = kTileLds + group_lds_bytes(E);
  hipError_t e = cache.get((const void*)grouped_tile_kernel<GRAD, BF16>, 512, lds, &f);
  if (e != hipSuccess) return e;
  const long long upper = ((ntm + (E < P ? E : P)) * ntn + 7) / 8 * 8, most = (long long)f.per_cu * f.cus / 8 * 8;
  hipLaunchKernelGGL((grouped_tile_kernel<GRAD, BF16>), dim3((uint32_t)(upper < most ? upper : most)), dim3(512), lds, s, a);
  return hipGetLastError();
}

template <class C, bool BF16, bool ADD>
hipError_t launch_wgrad_tiles(const WgradArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const long long blocks = (long long)((a.N + C::BM - 1) / C::BM) * ((a.K + C::BN - 1) / C::BN) * a.g.E;
  if (blocks * C::NT >= 1LL << 32) return hipErrorNotSupported;
  hipError_t e = cache.get((const void*)wgrad_tile_kernel<C, BF16, ADD>, C::NT, C::LDS, &f);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((wgrad_tile_kernel<C, BF16, ADD>), dim3((uint32_t)blocks), dim3(C::NT), C::LDS, s, a);
  return hipGetLastError();
}

using T256 = Bf16Cfg<256, 256, 2, 4, 2>;

}  // namespace

hipError_t launch_grouped(int kind, const GroupedArgs& a, hipStream_t s) {
  if (kind == 0) return a.out_bf16 ? launch_tiles<false, true>(a, s) : launch_tiles<false, false>(a, s);
  return a.out_bf16 ? launch_tiles<true, true>(a, s) : launch_tiles<true, false>(a, s);
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  if (a.out_bf16) return launch_wgrad_tiles<T256, true, false>(a, s);
  return a.add ? launch_wgrad_tiles<T256, false, true>(a, s) : launch_wgrad_tiles<T256, false, false>(a, s);
}

}  // namespace ftk
