// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale_s (x[t] A_s^T) B_s^T,  s the slot of row t's adapter; rows without one: out[t] = base[t].
// The hidden rows h = x A^T (r values each) are held in fp32; the second product takes them as bf16 terms (the value cut to 8 bits, what that
// left, and for fp32 results what that one's left), which carry 16 bits of it, or all 24, and not 8.
//
// lora_small_kernel: few rows.  A block has 16 rows of one adapter and 256 columns and forms their hidden rows by itself, its
// waves sharing K; one launch, no workspace.  Bound by its chain of dependent loads (16 rows of 16 adapters 5.6 us in a graph, of which 3.6 are the
// launch) and, with more blocks, by the reads of x and A that the blocks of an adapter repeat from L2.
// lora_shrink_kernel, lora_expand_kernel: many rows.  The first forms hidden rows in tiles of 64 rows by splits of K, so that
// every compute unit has loads in flight; the second adds the splits up in their order and multiplies with B.  4096 rows of 5
// adapters, r = 64, 7168 -> 4096: 17.0 + 27.4 us, 16.9 + 49.7 in fp32.  The first streams x at 3.4 TB/s: latency, one or two blocks a unit (other splits, 128
// rows a block, another place in K to begin with: within 3 %); the second at 2.5 TB/s: its blocks' loads, sums and stores in turn.
#include <algorithm>

#include "bf16_tile.h"
#include "ft_groups.h"
#include "ft_kernels.h"
#include "ft_products.h"

namespace ftk {
namespace {

// Chunks of up to ROWS rows of one adapter; with `copy` also those of rows without one (slot -1): positions of adapters without a slot, from
// offsets[E] on (entry E) and before offsets[0] (entry E + 1).
template <int ROWS>
__device__ __forceinline__ int list_chunks(const RowGroups& s, bool copy, GroupList& g, int* lds) {
  const int E2 = s.E + 4;
  g = GroupList{lds, lds + E2, lds + 2 * E2, lds + 3 * E2, 0};
  build_group_list(
      s.E + 2, g, lds + 4 * E2,
      [&](int e, int& slot, int& row0, int& cnt) {
        const int first = s.offsets[min(e, s.E)], next = s.offsets[e < s.E ? e + 1 : 0];  // loads that wait for no branch
        slot = s.slot_of ? s.slot_of[min(e, s.E - 1)] : e;
        if (e >= s.E || (uint32_t)slot >= s.n_slots) slot = -1;
        row0 = e <= s.E ? min(max(first, 0), s.P) : 0;
        cnt = (e == s.E ? s.P : min(max(next, 0), s.P)) - row0;
        return e <= s.E + 1 && cnt > 0 && (copy || slot >= 0);
      },
      [](int cnt) { return (cnt + ROWS - 1) / ROWS; });
  return g.item0[g.n];
}
constexpr size_t list_lds(int E) { return group_lds_bytes(E + 2); }

// An item's rows: positions p0 .. p0 + rows - 1 of gather.
struct Chunk {
  int slot, p0, rows;
};
template <int ROWS>
__device__ __forceinline__ Chunk chunk_of(const GroupList& gl, int ch) {
  const int gi = find_group(gl.item0, gl.n, ch), first = (ch - gl.item0[gi]) * ROWS;
  return Chunk{__builtin_amdgcn_readfirstlane(gl.slot[gi]), __builtin_amdgcn_readfirstlane(gl.row0[gi] + first),
                 __builtin_amdgcn_readfirstlane(min(ROWS, gl.cnt[gi] - first))};
}

__device__ __forceinline__ bf16x8 load8(const uint16_t* p, bool in) {
  return in ? *(const bf16x8*)p : __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
}
// Bf16 terms that a hidden value is passed on as: with a bf16 result two hold more than it does, with an fp32 one three hold all of it.
constexpr int terms(bool bf16) { return bf16 ? 2 : 3; }
// The next term of v, of which v is left for the ones after: cut from v short of its end, so that every term has v's sign and none is 0
// beside a value that is not: an infinite value of b then gives infinities of one sign, not the NaN of a term of the other or of a 0.  The last one
// is rounded.  What is left of a cut is under 2^-7 of v and has 16 bits at most: two terms hold v within 2^-16, three all of it.  0, an
// infinity and a NaN are every term.
template <bool LAST>
__device__ __forceinline__ uint32_t next_term(float& v) {
  if constexpr (LAST) return f32_to_bf16_bits(v);
  const uint32_t bits = __float_as_uint(v);
  const bool some = (bits & 0x7fffffffu) - 1 < 0x7f7fffffu;  // finite and not 0
  const uint32_t cut = (bits - some) & 0xffff0000u;          // (a NaN that a sum gave keeps its upper bits)
  v = some ? v - __uint_as_float(cut) : v;
  return cut >> 16;
}
// four bf16 values plus four fp32, rounded
__device__ __forceinline__ u32x2 pack_sum(u32x2 base, f32x4 v) {
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    o[h] = (uint32_t)f32_to_bf16_bits(__uint_as_float(base[h] << 16) + v[2 * h]) |
           ((uint32_t)f32_to_bf16_bits(__uint_as_float(base[h] & 0xffff0000u) + v[2 * h + 1]) << 16);
  return o;
}

// ---- few rows

// 16 rows by 256 columns a block: its SW waves form the hidden rows from a share of K each, then 256 / SW columns.
template <int RF>
struct SmallCfg {
  static constexpr int SW = RF == 4 ? 4 : 8, NF = 16 / SW;
  using Tile = Bf16Cfg<16, 16 * RF, 1, 1, RF == 4 ? 3 : 2, SW>;  // RF 1: two blocks a compute unit
  static constexpr int KS = (RF + 1) / 2, PITCH = KS * 32 + 8;  // the second product's steps of 32
};

template <int RF, bool BF16>
__global__ __launch_bounds__(64 * SmallCfg<RF>::SW) void lora_small_kernel(LoraArgs a, bool copy) {
  using C = SmallCfg<RF>;
  using T = typename C::Tile;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  constexpr int TERMS = terms(BF16);
  __shared__ __attribute__((aligned(16))) uint16_t s_hidden[TERMS][16 * C::PITCH];
  GroupList gl;
  const int chunks = list_chunks<16>(a.g, copy, gl, (int*)(smem + T::LDS));
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (a.N + 255) / 256, stages = (a.K + 63) / 64;
  // Blocks are placed on the 8 XCDs round-robin; each XCD gets a contiguous run of the items, whose columns share x and A.
  const int xcd = blockIdx.x % 8, end = (int)((long long)chunks * ntn * (xcd + 1) / 8);  // gridDim.x % 8 == 0
  for (int it = (int)((long long)chunks * ntn * xcd / 8) + blockIdx.x / 8; it < end; it += gridDim.x / 8) {
    const Chunk c = chunk_of<16>(gl, it / ntn);
    const int n0 = it % ntn * 256 + wv * 16 * C::NF;
    const int t = r < c.rows ? a.gather[c.p0 + r] : -1;
    const bool real = (uint32_t)t < (uint32_t)a.g.P;
    // what does not depend on the hidden rows is loaded first
    const size_t at = (size_t)(real ? t : 0) * a.N + n0 + 4 * g;
    u32x4 base[C::NF];
#pragma unroll
    for (int f = 0; f < C::NF; ++f) {
      base[f] = u32x4{0, 0, 0, 0};
      if (real && n0 + 16 * f + 4 * g < a.N) {
        if constexpr (BF16) {
          const u32x2 b = *(const u32x2*)((const uint16_t*)a.base + at + 16 * f);
          base[f][0] = b[0], base[f][1] = b[1];
        } else {
          base[f] = *(const u32x4*)((const float*)a.base + at + 16 * f);
        }
      }
    }
    f32x4 acc[C::NF];
#pragma unroll
    for (int f = 0; f < C::NF; ++f) acc[f] = f32x4{0, 0, 0, 0};
    if (c.slot >= 0) {
      const float scale = a.scale ? a.scale[c.slot] : 1.0f;
      bf16x8 bf[C::KS][C::NF];
#pragma unroll
      for (int q = 0; q < C::KS; ++q)
#pragma unroll
        for (int f = 0; f < C::NF; ++f)
          bf[q][f] = load8(a.b + ((size_t)c.slot * a.N + min(n0 + 16 * f + r, a.N - 1)) * a.r + 32 * q + 8 * g, 32 * q + 8 * g < a.r);
      const int k0 = stages * wv / C::SW * 64, k1 = min(stages * (wv + 1) / C::SW * 64, a.K);
      const Operand ro{a.x + k0, a.K, c.rows, a.gather + c.p0, a.g.P};
      const Operand co{a.a + (size_t)c.slot * a.r * a.K + k0, a.K, a.r, nullptr, 0};
      f32x4 hid[1][RF];
      bf16_tile<T, GATHERED, DIRECT>(ro, co, k1 - k0, smem + wv * T::RING, hid);
      // lane (r, g) holds row r, columns 16 f + 4 g .. + 3; every wave's sums over its own stages
      float* mine = (float*)(smem + wv * T::RING);
#pragma unroll
      for (int f = 0; f < RF; ++f) *(f32x4*)(mine + (r * RF + f) * 16 + 4 * g) = hid[0][f];
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * C::KS * 32; i += 64 * C::SW) {
        const int row = i / (C::KS * 32), j = i % (C::KS * 32);
        float v = 0.0f;
        if (row < c.rows && j < a.r) {
#pragma unroll
          for (int q = 0; q < C::SW; ++q) v += ((const float*)(smem + q * T::RING))[row * RF * 16 + j];
        }
        unrolled<0, TERMS>([&](auto q) { s_hidden[decltype(q)::value][row * C::PITCH + j] = (uint16_t)next_term<decltype(q)::value == TERMS - 1>(v); });
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < C::KS; ++q) {
        bf16x8 hf[TERMS];
#pragma unroll
        for (int k = 0; k < TERMS; ++k) hf[k] = *(const bf16x8*)(s_hidden[k] + r * C::PITCH + 32 * q + 8 * g);
#pragma unroll
        for (int f = 0; f < C::NF; ++f)
#pragma unroll
          for (int k = 0; k < TERMS; ++k) acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[q][f], hf[k], acc[f], 0, 0, 0);
      }
#pragma unroll
      for (int f = 0; f < C::NF; ++f) acc[f] *= scale;
    }
#pragma unroll
    for (int f = 0; f < C::NF; ++f)
      if (real && n0 + 16 * f + 4 * g < a.N) {
        if constexpr (BF16) {
          u32x2 o{base[f][0], base[f][1]};
          if (c.slot >= 0) o = pack_sum(o, acc[f]);
          *(u32x2*)((uint16_t*)a.out + at + 16 * f) = o;
        } else {
          f32x4 o = __builtin_bit_cast(f32x4, base[f]);
          if (c.slot >= 0) o += acc[f];
          *(f32x4*)((float*)a.out + at + 16 * f) = o;
        }
      }
  }
}

// ---- many rows

// h[split][p][j] = sum over the split's k of x[gather[p]][k] A[j][k] for 64 positions p and BN columns j
template <int BN>
using ShrinkCfg = Bf16Cfg<64, BN, 2, 1, 4>;

template <int BN>
__global__ __launch_bounds__(128) void lora_shrink_kernel(LoraArgs a, int splits) {
  using C = ShrinkCfg<BN>;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  GroupList gl;
  const int chunks = list_chunks<64>(a.g, false, gl, (int*)(smem + C::LDS));
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ntj = (a.r + BN - 1) / BN, stages = (a.K + 63) / 64;
  for (int it = blockIdx.x; it < chunks * splits * ntj; it += gridDim.x) {
    const int split = it % splits, j0 = it / splits % ntj * BN;
    const Chunk c = chunk_of<64>(gl, it / splits / ntj);
    const int k0 = (int)((long long)stages * split / splits) * 64, k1 = min((int)((long long)stages * (split + 1) / splits) * 64, a.K);
    f32x4 acc[C::MF][C::NF];
    const Operand ro{a.x + k0, a.K, c.rows, a.gather + c.p0, a.g.P};
    const Operand co{a.a + ((size_t)c.slot * a.r + j0) * a.K + k0, a.K, min(BN, a.r - j0), nullptr, 0};
    bf16_tile<C, GATHERED, DIRECT>(ro, co, k1 - k0, smem, acc);
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < C::MF; ++m)
#pragma unroll
      for (int f = 0; f < C::NF; ++f) {
        const int row = (wv * C::MF + m) * 16 + r, j = j0 + 16 * f + 4 * g;
        if (row < c.rows && j < a.r) *(f32x4*)(a.ws + ((size_t)split * a.g.P + c.p0 + row) * a.r + j) = acc[m][f];
      }
  }
}

// 32 rows by 256 columns of out, 64 of the r columns at a time: B goes to LDS directly, the hidden rows are added up on
// the way there.
using ExpandB = Loader<DIRECT, 256, 4>;
constexpr int ER = 32, kHidden = ER * 128;  // bytes of a term of 64 columns
template <bool BF16>
constexpr int kExpandLds = terms(BF16) * kHidden + 256 * 128;  // the terms, B

template <bool BF16>
__global__ __launch_bounds__(256, 3) void lora_expand_kernel(LoraArgs a, int splits, bool copy) {
  constexpr int TERMS = terms(BF16), AT_B = TERMS * kHidden;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  GroupList gl;
  const int chunks = list_chunks<ER>(a.g, copy, gl, (int*)(smem + kExpandLds<BF16>));
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), ntn = (a.N + 255) / 256;
  for (int it = blockIdx.x; it < chunks * ntn; it += gridDim.x) {
    const Chunk c = chunk_of<ER>(gl, it / ntn);
    const int n0 = it % ntn * 256;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // laundered: addresses are formed here, not kept through the loop
    const int lane = tid & 63;
    Reader<DIRECT, ER, ER / 16> rr;
    Reader<DIRECT, 256, 4> rb;
    rr.open(0, lane);
    rb.open(wv * 64, lane);
    const float scale = a.scale && c.slot >= 0 ? a.scale[c.slot] : 1.0f;
    f32x4 acc[ER / 16][4];
#pragma unroll
    for (int m = 0; m < ER / 16; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
    // this lane's pieces of 4 columns of out (each_piece): rows 16 m + 4 mid + j; base is on its way while the sums are formed
    const int col = n0 + wv * 64 + 16 * (lane >> 4) + 4 * (lane & 3);
    using Piece = std::conditional_t<BF16, u32x2, f32x4>;
    int t[ER / 4];
    Piece base[ER / 4];
#pragma unroll
    for (int i = 0; i < ER / 4; ++i) {
      const int row = 16 * (i / 4) + 4 * ((lane >> 2) & 3) + i % 4;
      t[i] = row < c.rows && col < a.N ? a.gather[c.p0 + row] : -1;
    }
    auto load_base = [&] {
#pragma unroll
      for (int i = 0; i < ER / 4; ++i) {
        base[i] = Piece{};
        if ((uint32_t)t[i] < (uint32_t)a.g.P) base[i] = *(const Piece*)((const uint8_t*)a.base + ((size_t)t[i] * a.N + col) * (BF16 ? 2 : 4));
      }
    };
    if (c.slot < 0) {
      load_base();
    } else {
      for (int j0 = 0; j0 < a.r; j0 += 64) {
        const int red = min(64, a.r - j0);
        const Operand bo{a.b + ((size_t)c.slot * a.N + n0) * a.r + j0, a.r, min(256, a.N - n0), nullptr, 0};
        ExpandB lb;
        lb.open(bo, tid, red);
        unrolled<0, ExpandB::Q>([&](auto q) { lb.template issue<decltype(q)::value, AT_B>(lds_addr(smem) + wv * 1024); });
        if (j0 == 0) load_base();
        // pieces of 4 hidden values, ER / 16 a thread, splits four at a time so that their loads are under way together
        f32x4 v[ER / 16];
#pragma unroll
        for (int i = 0; i < ER / 16; ++i) v[i] = f32x4{0, 0, 0, 0};
        const int j = j0 + tid % 16 * 4;
        for (int q0 = 0; q0 < splits; q0 += 4) {
          f32x4 part[4][ER / 16];
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < ER / 16; ++i) {
              const int row = 16 * i + tid / 16;
              part[q][i] = f32x4{0, 0, 0, 0};
              if (q0 + q < splits && row < c.rows && j < a.r) part[q][i] = *(const f32x4*)(a.ws + ((size_t)(q0 + q) * a.g.P + c.p0 + row) * a.r + j);
            }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < ER / 16; ++i) v[i] += part[q][i];
        }
#pragma unroll
        for (int i = 0; i < ER / 16; ++i) {
          const int row = 16 * i + tid / 16;
          f32x4 h = v[i];
          uint8_t* to = smem + row * 128 + ((tid % 16 / 2 ^ Loader<DIRECT, ER, 4>::key(row)) << 4) + (tid & 1) * 8;
          unrolled<0, TERMS>([&](auto k) {
            constexpr bool LAST = decltype(k)::value == TERMS - 1;
            u32x2 pair;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float lo = h[2 * q], hi = h[2 * q + 1];
              pair[q] = next_term<LAST>(lo);
              pair[q] |= next_term<LAST>(hi) << 16;
              h[2 * q] = lo, h[2 * q + 1] = hi;
            }
            *(u32x2*)(to + decltype(k)::value * kHidden) = pair;
          });
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (red < 64) {
          ExpandB::clear(smem + AT_B, tid, red);
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        unrolled<0, 2>([&](auto half) {
          constexpr int H = decltype(half)::value;
          bf16x8 bf[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) bf[f] = rb.template read<H>(smem + AT_B, f);
#pragma unroll
          for (int m = 0; m < ER / 16; ++m) {
            bf16x8 hf[TERMS];
#pragma unroll
            for (int k = 0; k < TERMS; ++k) hf[k] = rr.template read<H>(smem + k * kHidden, m);
#pragma unroll
            for (int f = 0; f < 4; ++f)
#pragma unroll
              for (int k = 0; k < TERMS; ++k) acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[f], hf[k], acc[m][f], 0, 0, 0);
          }
        });
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // LDS is free for what comes next
      }
    }
    each_piece<ER / 16, false>(acc, lane, [&](int i, int, int, f32x4 v) {
      Piece o = base[i];
      if (c.slot >= 0) {
        v *= scale;
        if constexpr (BF16)
          o = pack_sum(o, v);
        else
          o += v;
      }
      if ((uint32_t)t[i] < (uint32_t)a.g.P) *(Piece*)((uint8_t*)a.out + ((size_t)t[i] * a.N + col) * (BF16 ? 2 : 4)) = o;
    });
  }
}

// Chunks of up to `rows` of T rows in E groups, at most.
long long chunks(int T, int E, int rows) { return std::min<long long>(T, (T + rows - 1LL) / rows + E); }

template <int RF, bool BF16>
hipError_t launch_small(const LoraArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = SmallCfg<RF>::Tile::LDS + list_lds(a.g.E);
  hipError_t e = cache.get((const void*)lora_small_kernel<RF, BF16>, SmallCfg<RF>::Tile::NT, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = (chunks(a.g.P, a.g.E + 2, 16) * ((a.N + 255) / 256) + 7) / 8 * 8, most = (long long)f.per_cu * f.cus / 8 * 8;
  hipLaunchKernelGGL((lora_small_kernel<RF, BF16>), dim3((uint32_t)(items < most ? items : most)), dim3(SmallCfg<RF>::Tile::NT), lds, s, a, a.base != a.out);
  return hipGetLastError();
}

template <int BN>
hipError_t launch_shrink(const LoraArgs& a, int splits, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = ShrinkCfg<BN>::LDS + list_lds(a.g.E);
  hipError_t e = cache.get((const void*)lora_shrink_kernel<BN>, 128, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = chunks(a.g.P, a.g.E, 64) * splits * ((a.r + BN - 1) / BN), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL(lora_shrink_kernel<BN>, dim3((uint32_t)(items < most ? items : most)), dim3(128), lds, s, a, splits);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_expand(const LoraArgs& a, int splits, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = kExpandLds<BF16> + list_lds(a.g.E);
  hipError_t e = cache.get((const void*)lora_expand_kernel<BF16>, 256, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = chunks(a.g.P, a.g.E + 2, ER) * ((a.N + 255) / 256), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL(lora_expand_kernel<BF16>, dim3((uint32_t)(items < most ? items : most)), dim3(256), lds, s, a, splits, a.base != a.out);
  return hipGetLastError();
}

// One kernel or two, by times modelled in us.  In the one every 256 columns' block reads its rows of x and A itself, which is what it
// takes past 4.5 us: blocks of an adapter run on one XCD, and share the 256 compute units' loads where there are more blocks than
// units, and in turn where one unit holds no more (two, with r > 16 one).  Measured, us in a graph with other calls' inputs in between,
// one kernel / two: 16 rows of 16 adapters, r = 16, 2048 -> 4096: 5.6 / 10.7; 32 rows of 32: 7.7 / 12.0; 256 rows of 16: 8.9 / 12.3; 512 rows: 12.3 / 13.6;
// 1024 rows: 17.6 / 15.7; 131 rows of 40, r = 8, 7168 -> 2048, fp32: 12.3 / 15.9; 64 rows of 64, r = 16, 4096 -> 4096: 14.1 / 15.3; 512 rows of 16: 15.9 / 14.3;
// 3000 rows of 7, 776 -> 520, r = 16: 9.6 / 14.2, r = 64: 20.7 / 16.7; 16 rows of 16, r = 64, 2048 -> 4096: 10.0 / 12.9, 7168 -> 4096: 17.0 / 14.5.
bool lora_small(int T, int E, int r, int N, int K) {
  const double ntn = (N + 255) / 256, blocks = chunks(T, E + 1, 16) * ntn, rows = std::min(16.0, std::max(1.0, (double)T / E));
  const double one = 4.5 + std::max(0.6, blocks / 256) * 38e-6 * (std::max(16, r) + rows) * K + std::max(0.0, r <= 16 ? blocks / 512 - 1 : 5 * (blocks / 256 - 1)) * 0.8;
  const double two = 9 + 0.4e-3 * K + 0.5e-3 * T + 0.0055 * chunks(T, E + 1, 32) * ntn;
  return r <= 64 && one < two;
}

}  // namespace

// Shares of K: 1.5 blocks a compute unit, at least 512 values each (both kernels, us, 2 / 4 / 6 / 8 shares: 4096 rows of 5 adapters,
// 7168 -> 4096, r = 64: 51.0 / 54.5 / 51.1 / 54.4; 1024 rows of 16, 4096 -> 4096, r = 16: 19.6 / 17.3 / 17.1 / 17.0; 131 rows of 40,
// 7168 -> 2048, r = 8: 20.5 / 16.3 / 15.4 / 14.6).  0: no hidden rows in memory.
int lora_splits(int T, int E, int r, int N, int K) {
  if (lora_small(T, E, r, N, K)) return 0;
  const long long c = chunks(T, E, 64), s = std::min<long long>({(384 + c / 2) / c, K / 512, 16});
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int T = a.g.P, splits = lora_splits(T, a.g.E, a.r, a.N, a.K);
  if (splits == 0) {
    if (a.bf16) return a.r <= 16 ? launch_small<1, true>(a, s) : a.r <= 32 ? launch_small<2, true>(a, s) : launch_small<4, true>(a, s);
    return a.r <= 16 ? launch_small<1, false>(a, s) : a.r <= 32 ? launch_small<2, false>(a, s) : launch_small<4, false>(a, s);
  }
  hipError_t e = a.r <= 16 ? launch_shrink<16>(a, splits, s)
               : a.r <= 32 ? launch_shrink<32>(a, splits, s) : launch_shrink<64>(a, splits, s);
  if (e != hipSuccess) return e;
  return a.bf16 ? launch_expand<true>(a, splits, s) : launch_expand<false>(a, splits, s);
}

}  // namespace ftk
