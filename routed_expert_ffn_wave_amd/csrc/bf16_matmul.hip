// Products of bf16 rows with one matrix per expert, the gradient of the rows and the gradient of the matrices: what the
// expert FFN of a training step is made of (the expert groups of the FreeToken walk-through
// "深入FreeToken架构…全链路剖析", section 五).
//   forward        out[p][n]   = sum_k a[p][k] w[e][n][k]
//   rows           da[p][k]    = sum_n dout[p][n] w[e][n][k]
//   matrices       dw[e][n][k] = sum_{p of e} dout[p][n] a[p][k]
// bf16 products are exact in fp32 and added there by the matrix instructions; results are rounded once.
//
// What bounds them.  Compute: 16384 rows of one 4096 x 7168 matrix take 680 - 710 us forward (1.36 - 1.41 PFLOP/s; the library 615) and
// 690 - 710 back (the library 700), 8 experts with 2048 rows each 780 us for the matrices (1.23 PFLOP/s; the library's dense
// product of that layout 1.0 - 1.2): without the loads 583 of 740 us, without the matrix instructions 623, so neither alone; the clock
// falls to 1.4 - 1.7 GHz under them.  Memory: 128 experts of 1536 x 2048 with 64 rows each 150 us (5.5 TB/s), 16 tokens 97 us (5.2); with
// 256 rows each 210 us, what L2 reads from beyond it at 5 TB/s.  4096 tokens, Zipf, 274 us: both in turn (1.24 GB and 206 GFLOP, 36 % of
// the matrix cores' cycles).
#include <algorithm>
#include <cmath>

#include "bf16_plan.h"
#include "bf16_tile.h"
#include "ft_groups.h"
#include "ft_kernels.h"
#include "ft_products.h"

namespace ftk {
namespace {

template <class ItemsOf>
__device__ __forceinline__ void list_groups(const RowGroups& s, GroupList& g, int* tmp, ItemsOf items_of) {
  build_group_list(
      s.E, g, tmp, [&](int e, int& slot, int& row0, int& cnt) { return e < s.E && group_of(s, e, slot, row0, cnt) && cnt > 0; }, items_of);
}

constexpr int kTileLds = 160 * 1024;  // all of a compute unit's
static_assert(group_lds_bytes(1024) <= kTileLds, "LDS");

// Tiles of W columns: 256 by up to 256 rows, or 128 by up to 128 rows where there are few tiles.
template <int W>
constexpr int kTallest = W;

template <int BM, int W, bool GRAD, bool BF16>
__device__ __forceinline__ void grouped_tile(const GroupedArgs& a, int slot, int row0, int rows, int n0, uint8_t* lds) {
  constexpr int NS = W == 128 ? (BM <= 64 ? 6 : 5) : BM <= 64 && !GRAD ? 4 : BM <= 128 ? 3 : 2;
  using C = Bf16Cfg<BM, W, W == 128 ? 4 : 2, W == 128 ? 2 : 4, NS, 1, 64, NS == 2 ? 3 : NS>;
  static_assert(C::LDS <= kTileLds, "LDS");
  const int cols = GRAD ? a.K : a.N, red = GRAD ? a.N : a.K;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint16_t* w = a.w + (size_t)slot * a.N * a.K;
  f32x4 acc[C::MF][C::NF];
  const Operand ro{a.a + (size_t)row0 * red, red, rows, nullptr, 0};
  const Operand co{GRAD ? w + n0 : w + (size_t)n0 * a.K, a.K, min(C::BN, cols - n0), nullptr, 0};
  // Experts begin at different stages of a forward product: rows of K values (4 KiB for K = 2048) that all begin at once meet in the
  // same memory channels (128 experts of 1536 x 2048 with 64 rows each: 200 -> 161 us; the rows' gradient reads whole memory rows).
  bf16_tile<C, DIRECT, GRAD ? ACROSS : DIRECT>(ro, co, red, lds, acc, GRAD ? 0 : (slot & 0xffff) * 7);
  uint8_t* out = (uint8_t*)a.out + (size_t)row0 * cols * (BF16 ? 2 : 4);
  store_rows<C::MF, C::NF, BF16, false>(acc, out, cols, wv / C::WN * 16 * C::MF, rows, n0 + wv % C::WN * 16 * C::NF, cols, this_lane());
}

// The height of the tiles of a group of cnt rows.
template <int W>
__device__ __forceinline__ int tile_rows(int cnt) {
  constexpr int STEP = W == 128 ? 64 : 32;
  const int ntm = (cnt + kTallest<W> - 1) / kTallest<W>;
  return ((cnt + ntm - 1) / ntm + STEP - 1) / STEP * STEP;
}

// Tile `local` of a group of cnt rows, cut into tiles of the same height: bands of 4 row tiles, column tiles within a band in turn.  A tile
// takes the least of the heights that holds its rows.
template <int W, bool GRAD, bool BF16>
__device__ __forceinline__ void grouped_item(const GroupedArgs& a, int slot, int row0, int cnt, int local, uint8_t* lds) {
  constexpr int BAND = 4;
  const int ntn = ((GRAD ? a.K : a.N) + W - 1) / W;
  const int ntm = (cnt + kTallest<W> - 1) / kTallest<W>, each = tile_rows<W>(cnt);
  const int band = local / (BAND * ntn), h = min(BAND, ntm - band * BAND), in = local - band * BAND * ntn;
  const int m0 = (band * BAND + in % h) * each, n0 = in / h * W, rows = min(each, cnt - m0);
  auto tile = [&](auto height) { grouped_tile<decltype(height)::value, W, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds); };
  if constexpr (W == 128) {
    if (rows > 64)
      tile(std::integral_constant<int, 128>{});
    else
      tile(std::integral_constant<int, 64>{});
  } else if (rows > 224)
    tile(std::integral_constant<int, 256>{});
  else if (rows > 192)
    tile(std::integral_constant<int, 224>{});
  else if (rows > 160)
    tile(std::integral_constant<int, 192>{});
  else if (rows > 128)
    tile(std::integral_constant<int, 160>{});
  else if (rows > 96)
    tile(std::integral_constant<int, 128>{});
  else if (rows > 64)
    tile(std::integral_constant<int, 96>{});
  else if (rows > 32)
    tile(std::integral_constant<int, 64>{});
  else
    tile(std::integral_constant<int, 32>{});
}

// Blocks are placed on the 8 XCDs round-robin; each XCD gets a contiguous run of the tile list, so that tiles that run
// together share rows and matrices through its L2, which holds little more than the stages that they have under way: they share
// only what they read in step.  So groups are cut into even tiles and long lists go by falling heights, and an XCD's tiles take equally long;
// XCDs begin at different rounds, or all would be bound by the matrix cores first and by memory later.  us, without order / with it:
// 4096 tokens, Zipf, top 8 of 128 experts of 1536 x 2048 297 / 279 (read by L2 1.39 -> 1.14 GB, 0.92 needed), 1024 tokens 158 / 145.
// (Each block a run of tiles of even cost: 343; queues with the tallest tiles first, as the matrix gradient has them, 5 % more than no order.)
template <int W, bool ORDERED, bool GRAD, bool BF16>
__global__ __launch_bounds__(512, 2) void grouped_tile_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int ntn = ((GRAD ? a.K : a.N) + W - 1) / W;
  const int per = gridDim.x / 8, x = blockIdx.x % 8, j = blockIdx.x / 8, lane = threadIdx.x & 63;  // gridDim.x % 8 == 0
  // The list lies where the stages will: every wave keeps what it says of this block's next 16 tiles, lanes 4 i .. 4 i + 3 tile i.
  for (int first = 0;; first += 16) {
    const int E = a.g.E, E2 = E + 2;
    int* li = (int*)lds;
    GroupList gl{li, li + E2, li + 2 * E2, li + 3 * E2, 0};
    auto tiles_of = [&](int cnt) { return (cnt + kTallest<W> - 1) / kTallest<W> * ntn; };
    int classes = 0;
    if constexpr (!ORDERED) {
      list_groups(a.g, gl, li + 4 * E2, tiles_of);
    } else {
      // The groups by falling class of their tiles' heights, classes that there are in turn.
      int* rows_of = li + 5 * E2;  // [E]: slot, first row, rows (0: none)
      int* present = rows_of + 3 * E;
      if (threadIdx.x == 0) *present = 0;
      __syncthreads();
      auto class_of = [](int cnt) { return 4 - (tile_rows<W>(cnt) + 63) / 64; };
      for (int e = threadIdx.x; e < E; e += 512) {
        int slot, row0, cnt;
        if (!group_of(a.g, e, slot, row0, cnt)) cnt = 0;
        rows_of[e] = slot, rows_of[E + e] = row0, rows_of[2 * E + e] = cnt;
        if (cnt > 0) atomicOr(present, 1 << class_of(cnt));
      }
      __syncthreads();
      classes = __builtin_amdgcn_readfirstlane(*present);
      const int E64 = (E + 63) / 64 * 64;
      build_group_list(
          __popc(classes) * E64, gl, li + 4 * E2,
          [&](int i, int& slot, int& row0, int& cnt) {
            const int pass = i / E64, e = i - pass * E64;
            if (e >= E) return false;
            int left = classes;
            for (int k = 0; k < pass; ++k) left &= left - 1;
            slot = rows_of[e], row0 = rows_of[E + e], cnt = rows_of[2 * E + e];
            return cnt > 0 && (left & -left) == 1 << class_of(cnt);
          },
          tiles_of);
    }
    const int nitems = gl.item0[gl.n], rounds = (nitems + (int)gridDim.x - 1) / (int)gridDim.x;
    // Each XCD begins at another round, and rounds are turned against each other: a block must not meet the same height always.
    const int mine = first + lane / 4, turned = classes & (classes - 1) ? (mine + x * rounds / 8) % max(rounds, 1) : mine;
    const int it = turned * (int)gridDim.x + x * per + (j + 7 * mine) % per;
    int word = mine < rounds ? 0 : -1;  // its slot, first row, rows (0: no tile in this round, -1: nor later), and number in the group
    if (mine < rounds && it < nitems) {
      const int gi = find_group(gl.item0, gl.n, it);
      word = lane % 4 == 3 ? it - gl.item0[gi] : (lane % 4 == 0 ? gl.slot : lane % 4 == 1 ? gl.row0 : gl.cnt)[gi];
    }
    __syncthreads();
    for (int r = 0; r < 16; ++r) {
      const int rows = __builtin_amdgcn_readlane(word, 4 * r + 2);
      if (rows < 0) return;
      if (rows > 0)
        grouped_item<W, GRAD, BF16>(a, __builtin_amdgcn_readlane(word, 4 * r), __builtin_amdgcn_readlane(word, 4 * r + 1), rows,
                                    __builtin_amdgcn_readlane(word, 4 * r + 3), lds);
    }
  }
}

// The sums of a block's four waves, each over a share of the reduction, added in their order and stored: rows < `rows` and
// columns n0 .. n0 + 63 < cols of out with ld values a row.
template <class C, bool BF16, bool ADD>
__device__ __forceinline__ void join_waves(const f32x4 (&acc)[C::MF][C::NF], void* out, size_t ld, int rows, int n0, int cols, uint8_t* lds) {
  constexpr int PITCH = 68;  // floats of a row of results in LDS, over the stages
  static_assert(C::KG == 4 && C::GW == 1 && C::NF == 4 && C::BM * PITCH * 4 <= C::RING, "a wave's results lie over its stages");
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
  float* mine = (float*)(lds + wv * C::RING);
#pragma unroll
  for (int m = 0; m < C::MF; ++m)
#pragma unroll
    for (int f = 0; f < 4; ++f) *(f32x4*)(mine + (16 * m + r) * PITCH + 16 * f + 4 * g) = acc[m][f];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * 16; i += 256) {
    const int row = i / 16, c = i % 16 * 4;
    const float* p = (const float*)lds + row * PITCH + c;
    f32x4 v = *(const f32x4*)p;
#pragma unroll
    for (int q = 1; q < 4; ++q) v += *(const f32x4*)(p + q * (C::RING / 4));
    if (n0 + c >= cols) continue;
    const size_t at = (size_t)row * ld + n0 + c;
    if constexpr (BF16) {
      *(u32x2*)((uint16_t*)out + at) = u32x2{(uint32_t)f32_to_bf16_bits(v[0]) | ((uint32_t)f32_to_bf16_bits(v[1]) << 16),
                                             (uint32_t)f32_to_bf16_bits(v[2]) | ((uint32_t)f32_to_bf16_bits(v[3]) << 16)};
    } else {
      if (ADD) v += *(const f32x4*)((const float*)out + at);
      *(f32x4*)((float*)out + at) = v;
    }
  }
  __syncthreads();  // the stages are free for the next tile
}

// Few rows an expert: BM rows by 64 columns a block, whose four waves have a share of the reduction each, with stages of
// their own and no barriers; their sums meet in LDS in a fixed order.
template <int BM, bool GRAD, bool BF16>
__device__ __forceinline__ void few_tile(const GroupedArgs& a, int slot, int row0, int rows, int n0, uint8_t* lds) {
  using C = Bf16Cfg<BM, 64, 1, 1, 2, 4>;
  const int cols = GRAD ? a.K : a.N, red = GRAD ? a.N : a.K, stages = (red + 63) / 64;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = stages * wv / 4 * 64, k1 = min(stages * (wv + 1) / 4 * 64, red);
  const uint16_t* w = a.w + (size_t)slot * a.N * a.K;
  f32x4 acc[C::MF][C::NF];
  const Operand ro{a.a + (size_t)row0 * red + k0, red, rows, nullptr, 0};
  const Operand co{GRAD ? w + (size_t)k0 * a.K + n0 : w + (size_t)n0 * a.K + k0, a.K, min(64, cols - n0), nullptr, 0};
  bf16_tile<C, DIRECT, GRAD ? ACROSS : DIRECT>(ro, co, k1 - k0, lds + wv * C::RING, acc);
  join_waves<C, BF16, false>(acc, (uint8_t*)a.out + (size_t)row0 * cols * (BF16 ? 2 : 4), cols, rows, n0, cols, lds);
}

// ROWS 16: 16 rows a tile, two blocks a compute unit; 64: the least of 16, 32 and 64 that holds a tile's rows.
template <int ROWS>
constexpr int kFewLds = ROWS == 16 ? 4 * 2 * (16 + 64) * 128 : 4 * 2 * (64 + 64) * 128;

template <int ROWS, bool GRAD, bool BF16>
__global__ __launch_bounds__(256) void grouped_few_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int cols = GRAD ? a.K : a.N;
  const int ntn = (cols + 63) / 64;
  const int E2 = a.g.E + 2;
  int* li = (int*)(lds + kFewLds<ROWS>);
  GroupList gl{li, li + E2, li + 2 * E2, li + 3 * E2, 0};
  list_groups(a.g, gl, li + 4 * E2, [&](int cnt) { return (cnt + ROWS - 1) / ROWS * ntn; });
  const int nitems = gl.item0[gl.n];
  for (int it = blockIdx.x; it < nitems; it += gridDim.x) {
    const int gi = find_group(gl.item0, gl.n, it);
    const int local = __builtin_amdgcn_readfirstlane(it - gl.item0[gi]);
    const int slot = __builtin_amdgcn_readfirstlane(gl.slot[gi]);
    const int row0 = __builtin_amdgcn_readfirstlane(gl.row0[gi]), cnt = __builtin_amdgcn_readfirstlane(gl.cnt[gi]);
    const int m0 = local / ntn * ROWS, n0 = local % ntn * 64, rows = min(ROWS, cnt - m0);
    if (ROWS > 16 && rows > 32)
      few_tile<64, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
    else if (ROWS > 16 && rows > 16)
      few_tile<32, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
    else
      few_tile<16, GRAD, BF16>(a, slot, row0 + m0, rows, n0, lds);
  }
}

template <class C, bool BF16, bool ADD, class Next>
__device__ __forceinline__ void wgrad_item(const WgradArgs& a, int e, int row0, int cnt, int t, uint8_t* lds, Next next) {
  const int ntn = (a.K + C::BN - 1) / C::BN, lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (ADD && cnt == 0) return next();
  // bands of 4 tiles along N, in turn along K: 32 that run together read 4 + 8 tiles' operands and not 1 + 28
  // (8 experts of 4096 x 7168 with 2048 rows each: 3.6 -> 1.5 GB read by L2, 849 -> 822 us)
  const int ntm = (a.N + C::BM - 1) / C::BM, band = t / (4 * ntn), h = min(4, ntm - band * 4), in = t - band * 4 * ntn;
  const int m0 = (band * 4 + in % h) * C::BM, n0 = in / h * C::BN;
  f32x4 acc[C::MF][C::NF];
  const Operand ro{a.dout + (size_t)row0 * a.N + m0, a.N, min(C::BM, a.N - m0), nullptr, 0};
  const Operand co{a.a + (size_t)row0 * a.K + n0, a.K, min(C::BN, a.K - n0), nullptr, 0};
  bf16_tile<C, ACROSS, ACROSS>(ro, co, cnt, lds, acc);
  next();
  uint8_t* out = (uint8_t*)a.dw + ((size_t)e * a.N + m0) * a.K * (BF16 ? 2 : 4);
  store_rows<C::MF, C::NF, BF16, ADD>(acc, out, a.K, wv / C::WN * 16 * C::MF, ro.rows, n0 + wv % C::WN * 16 * C::NF, a.K, lane);
}

template <class C, bool BF16, bool ADD>
__global__ __launch_bounds__(C::NT, 2) void wgrad_tile_kernel(WgradArgs a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int tiles = (a.N + C::BM - 1) / C::BM * ((a.K + C::BN - 1) / C::BN);
  const int e = blockIdx.x / tiles;
  int slot, row0, cnt;
  if (!group_of(a.g, e, slot, row0, cnt)) return;
  wgrad_item<C, BF16, ADD>(a, e, __builtin_amdgcn_readfirstlane(row0), __builtin_amdgcn_readfirstlane(cnt), blockIdx.x % tiles, lds, [] {});
}

template <class C, bool BF16, bool ADD>
__global__ __launch_bounds__(C::NT, 2) void wgrad_planned_kernel(WgradArgs a, int tiles, Plan* plan) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  run_plan(plan, tiles, [&](const PlanPart& part, int t, auto next) {
    wgrad_item<C, BF16, ADD>(a, part.expert, part.row0, part.rows, t, lds, next);
  });
}

// Few tiles: 64 x 64 a block, whose four waves have a share of the expert's rows each.
using WgradFew = Bf16Cfg<64, 64, 1, 1, 2, 4>;

template <bool BF16, bool ADD>
__global__ __launch_bounds__(256) void wgrad_few_kernel(WgradArgs a) {
  using C = WgradFew;
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int ntn = (a.K + 63) / 64, tiles = (a.N + 63) / 64 * ntn, e = blockIdx.x / tiles, t = blockIdx.x % tiles;
  int slot, row0, cnt;
  if (!group_of(a.g, e, slot, row0, cnt)) return;
  row0 = __builtin_amdgcn_readfirstlane(row0), cnt = __builtin_amdgcn_readfirstlane(cnt);
  if (ADD && cnt == 0) return;
  const int m0 = t / ntn * 64, n0 = t % ntn * 64, stages = (cnt + 63) / 64;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = stages * wv / 4 * 64, k1 = min(stages * (wv + 1) / 4 * 64, cnt);
  f32x4 acc[C::MF][C::NF];
  const Operand ro{a.dout + (size_t)(row0 + k0) * a.N + m0, a.N, min(64, a.N - m0), nullptr, 0};
  const Operand co{a.a + (size_t)(row0 + k0) * a.K + n0, a.K, min(64, a.K - n0), nullptr, 0};
  bf16_tile<C, ACROSS, ACROSS>(ro, co, k1 - k0, lds + wv * C::RING, acc);
  join_waves<C, BF16, ADD>(acc, (uint8_t*)a.dw + ((size_t)e * a.N + m0) * a.K * (BF16 ? 2 : 4), a.K, ro.rows, n0, a.K, lds);
}

constexpr long long kMostItems = (1LL << 31) - (1 << 16);  // counted in an int, with a launch's blocks added

template <int ROWS, bool GRAD, bool BF16>
hipError_t launch_few(const GroupedArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const int cols = GRAD ? a.K : a.N, E = a.g.E, P = a.g.P;
  const long long ntn = (cols + 63) / 64, ntm = (P + ROWS - 1) / ROWS;
  const size_t lds = kFewLds<ROWS> + group_lds_bytes(E);
  hipError_t e = cache.get((const void*)grouped_few_kernel<ROWS, GRAD, BF16>, 256, lds, &f);
  if (e != hipSuccess) return e;
  const long long upper = std::min<long long>(P, ntm + E) * ntn, most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL((grouped_few_kernel<ROWS, GRAD, BF16>), dim3((uint32_t)(upper < most ? upper : most)), dim3(256), lds, s, a);
  return hipGetLastError();
}

template <int W, bool ORDERED, bool GRAD, bool BF16>
hipError_t launch_tiles(const GroupedArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const int cols = GRAD ? a.K : a.N, E = a.g.E, P = a.g.P;
  const long long ntn = (cols + W - 1) / W, tiles = std::min<long long>(P, (P + kTallest<W> - 1) / kTallest<W> + E) * ntn;
  if ((P / kTallest<W> + 2LL) * (E / 2 + 1) * ntn >= kMostItems) return hipErrorNotSupported;
  hipError_t e = cache.get((const void*)grouped_tile_kernel<W, ORDERED, GRAD, BF16>, 512, kTileLds, &f);
  if (e != hipSuccess) return e;
  const long long upper = (tiles + 7) / 8 * 8, most = (long long)f.per_cu * f.cus / 8 * 8;
  hipLaunchKernelGGL((grouped_tile_kernel<W, ORDERED, GRAD, BF16>), dim3((uint32_t)(upper < most ? upper : most)), dim3(512), kTileLds, s, a);
  return hipGetLastError();
}

// Matrix gradients of more tiles than two a compute unit are planned.
long long wgrad_tiles(int N, int K, int E) { return (long long)((N + 255) / 256) * ((K + 255) / 256) * E; }
constexpr int kPlanFrom = 512;

template <class C, bool BF16, bool ADD>
hipError_t launch_wgrad_tiles(const WgradArgs& a, hipStream_t s) {
  static LaunchCache cache, planned;
  LaunchFacts f;
  const long long blocks = wgrad_tiles(a.N, a.K, a.g.E);
  if (blocks > kPlanFrom) {
    const int tiles = (int)(blocks / a.g.E);
    hipError_t e = planned.get((const void*)wgrad_planned_kernel<C, BF16, ADD>, C::NT, C::LDS, &f);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a.g, tiles, (Plan*)a.ws);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((wgrad_planned_kernel<C, BF16, ADD>), dim3(f.per_cu * f.cus), dim3(C::NT), C::LDS, s, a, tiles, (Plan*)a.ws);
    return hipGetLastError();
  }
  hipError_t e = cache.get((const void*)wgrad_tile_kernel<C, BF16, ADD>, C::NT, C::LDS, &f);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((wgrad_tile_kernel<C, BF16, ADD>), dim3((uint32_t)blocks), dim3(C::NT), C::LDS, s, a);
  return hipGetLastError();
}

template <bool BF16, bool ADD>
hipError_t launch_wgrad_few(const WgradArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const long long blocks = (long long)((a.N + 63) / 64) * ((a.K + 63) / 64) * a.g.E;
  hipError_t e = cache.get((const void*)wgrad_few_kernel<BF16, ADD>, 256, WgradFew::LDS, &f);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((wgrad_few_kernel<BF16, ADD>), dim3((uint32_t)blocks), dim3(256), WgradFew::LDS, s, a);
  return hipGetLastError();
}

// Four stages of 32 steps: 3 % less time than two of 64 (8 experts of 4096 x 7168 with 2048 rows each: 820 -> 808 us).  Where rows are
// DIRECT their pieces would be 64 bytes: 8 % more (16384 rows, 7168 -> 4096: 707 -> 764 us).
using T256 = Bf16Cfg<256, 256, 2, 4, 4, 1, 32>;

// Which kernel: 256-column tiles, or blocks of 64 columns whose waves share the reduction.  How the rows lie is known on the device
// only: as if experts were drawn evenly.  Two rules.  By times modelled for the rounds that the 256 compute units take, in us (a
// tile's start and end, and its stages of 64): what bounds products of many rows or few tiles.  The bytes are not in that model, and
// with few rows an expert they are the time: there it takes tiles for faster than they are.  So forward products of up to 16 rows an
// expert take the blocks whatever it says, by the times below.  Measured, us, 256-column tiles / 64-column blocks, bf16 results:
//   forward, 128 experts of 1536 x 2048, top 8 of   1 token  18.9 / 11.8    4  34.4 / 29.9    8  70.7 / 60.6    64  143.6 / 137.7
//                                                  256  148.8 / 147.3    512  154.1 / 160.8    4096 (Zipf)  274 / 533
//   rows' gradient, the same                         1  17.3 / 11.9    4  32.5 / 33.2    16  99.3 / 110.5    256  147.4 / 178.8
//   one matrix of 4096 x 4096, rows                 64  31.2 / 16.0    300  73.8 / 29.8
// With few rows the forward product is bound by the matrices' bytes, which the smaller blocks read at 5.7 - 6.1 TB/s, the larger
// ones at 5.3 - 5.6; in the rows' gradient, whose 64 columns are 128 bytes of a memory row, it is the other way round.
// Forward with up to 16 rows an expert elsewhere, 256-column tiles / 64-column blocks (/ 128-column tiles):
//   64 experts of 2048 x 1024, top 4 of   1 token  11.7 / 6.8    8  24.9 / 26.5    32  46.7 / 47.9    128  50.8 / 56.2
//   8 of 4096 x 8192, top 2               1        56.4 / 24.6   4  94.8 / 93.3 / 81.2    16  104.0 / 123.3 / 101.8
//   16 of 2048 x 2048, top 4              1        23.6 / 10.5   4  28.3 / 23.8    16  30.4 / 28.0
//   256 of 4096 x 7168, top 8             1        98.2 / 80.8  16  1002 / 975    128  2379 / 2375
// so that from some 4 rows an expert on the tiles win by up to a fifth where rows are long or experts few.
// Tiles of 128 columns where 256 leave units without one, or a round nearly empty (a tile's time as a share of a
// 256-column one's, 0.58 forward and 0.68 back, is fitted to these times, not derived).  us, 256 (or 64) / 128: 256 tokens, top 2 of 8 experts of
// 4096 x 4096 73 / 50, back 86 / 53; 300, top 4 of 16 of 2048 x 2048 32 / 25, back 33 / 27; 333, top 8 of 64, 40 here, of 2048 x 1032 56 / 49; but 128 experts
// with 128 rows each 161 / 168, 512 tokens, top 2 of 8, 81 / 89; back 77 tokens, top 4 of 32 of 2048 x 768 19.8 / 21.0, 64, top 2 of 8, 54.6 / 51.1.
// The list is put in order of heights where there are more than two rounds and heights to differ: it takes 1 - 2 us.
// 16 rows a block, two blocks a unit, where 64 would leave most units without one (64 rows, 4096 x 4096: 16.0 -> 12.2).
constexpr int kOrdered = 257;  // 256, the list in order
template <bool GRAD>
int choose(const GroupedArgs& a) {
  const int cols = GRAD ? a.K : a.N, red = GRAD ? a.N : a.K;
  const double held = a.g.slot_of ? std::min(1.0, (double)a.g.n_slots / a.g.E) : 1.0;
  const double rows = std::max(1.0, held * a.g.P), groups = std::max(1.0, held * a.g.E * (1.0 - std::exp(-(double)a.g.P / a.g.E)));
  const double each = rows / groups, stages = (red + 63) / 64;
  auto blocks = [&](int h, int w) { return std::max(groups, rows / h + (each > h ? 0.5 : 0.0) * groups) * ((cols + w - 1) / w); };
  auto rounds = [&](int h, int w) { return std::ceil(blocks(h, w) / 256); };
  const double tile = 3.5 + stages * (0.3 + 0.8 * std::min(each, 256.0) / 256);
  const double few = rounds(64, 64) * (3.5 + stages / 4 * 0.8), wide = rounds(256, 256) * tile;
  // (Groups of about 128 rows: many in two tiles.  A rows' gradient of few rows wants whole memory rows.)
  const double narrow = each <= 100 && !(GRAD && each < 12) ? rounds(128, 128) * (GRAD ? 0.68 : 0.58) * tile : wide;
  if (few < std::min(wide, narrow) || (!GRAD && each <= 16)) return blocks(64, 64) < 100 ? 16 : 64;
  if (narrow < wide) return 128;
  return each >= 48 && blocks(256, 256) > 512 ? kOrdered : 256;
}

template <bool GRAD, bool BF16>
hipError_t launch_grouped_as(const GroupedArgs& a, hipStream_t s) {
  // tiles of all groups in an int whatever the table holds: one that does not ascend can give all rows to every second expert
  if ((a.g.P / 16 + 2LL) * (a.g.E / 2 + 1) * (((GRAD ? a.K : a.N) + 63) / 64) >= kMostItems) return launch_tiles<256, true, GRAD, BF16>(a, s);
  switch (choose<GRAD>(a)) {
    case 16: return launch_few<16, GRAD, BF16>(a, s);
    case 64: return launch_few<64, GRAD, BF16>(a, s);
    case 128: return launch_tiles<128, false, GRAD, BF16>(a, s);
    case kOrdered: return launch_tiles<256, true, GRAD, BF16>(a, s);
    default: return launch_tiles<256, false, GRAD, BF16>(a, s);
  }
}

// Matrix gradients: 256 x 256 tiles, or 64 x 64 blocks whose waves share the rows, by times modelled for rounds of the 256
// compute units (rows as if drawn evenly).  Measured, us, tiles / blocks, fp32 results: 8 experts of 512 x 512 with 1024 rows 28.3 /
// 20.5, with 128 rows 12.0 / 9.7; 4 experts of 256 x 256 with 4096 rows 77 / 17; 8 experts of 1024 x 1024 with 1024 rows 32.8 / 54.2;
// 16 experts of 1024 x 512 with 512 rows 21.9 / 43.6.
// A tile reduces all rows of its expert, so that few tiles take as long as the popular expert's: 32768 rows of 16 experts of 512 x 512 45 us
// with even experts, 212 where one has 12000; of 64 of 512 x 1024 63 and 101 (one 4000); 8192 rows of 8 of 1536 x 2048 65 and 70.
// Adding to fp32 gradients (ADD) waits for the old values of a piece before the next piece's are asked for: 4096 tokens, Zipf, 128 experts of
// 1536 x 2048 820 us where writing takes 399, 8 experts of 4096 x 7168 with 2048 rows each 1051 and 828.
bool wgrad_few(const WgradArgs& a) {
  const double stages = std::ceil((double)a.g.P / a.g.E / 64), blocks = (double)((a.N + 63) / 64) * ((a.K + 63) / 64) * a.g.E;
  return blocks < 1 << 24 && std::ceil(blocks / 256) * (5 + stages / 4 * 1.1) < std::ceil(wgrad_tiles(a.N, a.K, a.g.E) / 256.0) * (4 + stages * 1.4);
}

template <bool BF16, bool ADD>
hipError_t launch_wgrad_as(const WgradArgs& a, hipStream_t s) {
  return wgrad_few(a) ? launch_wgrad_few<BF16, ADD>(a, s) : launch_wgrad_tiles<T256, BF16, ADD>(a, s);
}

}  // namespace

size_t wgrad_workspace(int N, int K, int E) { return wgrad_tiles(N, K, E) > kPlanFrom ? plan_bytes(E) : 0; }

hipError_t launch_grouped(int kind, const GroupedArgs& a, hipStream_t s) {
  if (kind == 0) return a.out_bf16 ? launch_grouped_as<false, true>(a, s) : launch_grouped_as<false, false>(a, s);
  return a.out_bf16 ? launch_grouped_as<true, true>(a, s) : launch_grouped_as<true, false>(a, s);
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  if (wgrad_tiles(a.N, a.K, a.g.E) >= kMostItems) return hipErrorNotSupported;
  if (a.out_bf16) return launch_wgrad_as<true, false>(a, s);
  return a.add ? launch_wgrad_as<false, true>(a, s) : launch_wgrad_as<false, false>(a, s);
}

}  // namespace ftk
