// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale_s (x[t] A_s^T) B_s^T,  s the slot of row t's adapter; rows without one: out[t] = base[t].
// The hidden rows h = x A^T (r values each) are held in fp32; the second product takes them as two bf16 terms (the value
// and what its rounding left), so that they carry 16 bits or more of it and not 8.
//
// lora_small_kernel: few rows.  A block has 16 rows of one adapter and 256 columns and forms their hidden rows by itself, its
// waves sharing K; one launch, no workspace.  Bound by its chain of dependent loads.
// lora_shrink_kernel, lora_expand_kernel: many rows.  The first forms hidden rows in tiles of 64 rows by splits of K, so that
// every compute unit has loads in flight; the second adds the splits up in their order and multiplies with B.
#include "bf16_tile.h"
#include "ft_groups.h"
#include "ft_kernels.h"
#include "ft_products.h"

namespace ftk {
namespace {

// Chunks of up to ROWS rows of one adapter; with `copy` also those of rows without one (slot -1).
template <int ROWS>
__device__ __forceinline__ int list_chunks(const RowGroups& s, bool copy, GroupList& g, int* lds) {
  const int E2 = s.E + 3;
  g = GroupList{lds, lds + E2, lds + 2 * E2, lds + 3 * E2, 0};
  build_group_list(
      s.E + 1, g, lds + 4 * E2,
      [&](int e, int& slot, int& row0, int& cnt) {
        if (e <= s.E) {
          row0 = min(max(s.offsets[e], 0), s.P);
          cnt = (e < s.E ? min(max(s.offsets[e + 1], 0), s.P) : s.P) - row0;
          slot = e == s.E ? -1 : s.slot_of ? s.slot_of[e] : e;
          if ((uint32_t)slot >= s.n_slots) slot = -1;
        }
        return cnt > 0 && (copy || slot >= 0);
      },
      [](int cnt) { return (cnt + ROWS - 1) / ROWS; });
  return g.item0[g.n];
}
constexpr size_t list_lds(int E) { return group_lds_bytes(E + 1); }

// An item's rows: positions p0 .. p0 + rows - 1 of gather.
struct Chunk16 {
  int slot, p0, rows;
};
template <int ROWS>
__device__ __forceinline__ Chunk16 chunk_of(const GroupList& gl, int ch) {
  const int gi = find_group(gl.item0, gl.n, ch), first = (ch - gl.item0[gi]) * ROWS;
  return Chunk16{__builtin_amdgcn_readfirstlane(gl.slot[gi]), __builtin_amdgcn_readfirstlane(gl.row0[gi] + first),
                 __builtin_amdgcn_readfirstlane(min(ROWS, gl.cnt[gi] - first))};
}

__device__ __forceinline__ bf16x8 load8(const uint16_t* p, bool in) {
  return in ? *(const bf16x8*)p : __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
}
__device__ __forceinline__ uint32_t pack_sum(uint32_t base, float a, float b) {
  return (uint32_t)f32_to_bf16_bits(__uint_as_float(base << 16) + a) |
         ((uint32_t)f32_to_bf16_bits(__uint_as_float(base & 0xffff0000u) + b) << 16);
}

// ---- few rows

constexpr int SW = 8;  // waves per block

template <int RF, bool BF16>
__global__ __launch_bounds__(64 * SW) void lora_small_kernel(LoraArgs a, bool copy) {
  constexpr int KS = (RF + 1) / 2, PITCH = KS * 32 + 8;  // the second product's steps of 32
  extern __shared__ __attribute__((aligned(16))) int lds[];
  __shared__ __attribute__((aligned(16))) float s_part[SW][RF * 256];
  __shared__ __attribute__((aligned(16))) uint16_t s_hi[16 * PITCH], s_lo[16 * PITCH];
  GroupList gl;
  const int chunks = list_chunks<16>(a.g, copy, gl, lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (a.N + 255) / 256;
  for (int it = blockIdx.x; it < chunks * ntn; it += gridDim.x) {
    const Chunk16 c = chunk_of<16>(gl, it / ntn);
    const int n0 = it % ntn * 256 + wv * 32;
    const int t = r < c.rows ? a.gather[c.p0 + r] : -1;
    const bool real = (uint32_t)t < (uint32_t)a.g.P;
    // what does not depend on the hidden rows is loaded first
    const size_t at = (size_t)(real ? t : 0) * a.N + n0 + 4 * g;
    u32x4 base[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
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
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    if (c.slot >= 0) {
      const float scale = a.scale ? a.scale[c.slot] : 1.0f;
      bf16x8 bf[KS][2];
#pragma unroll
      for (int q = 0; q < KS; ++q)
#pragma unroll
        for (int f = 0; f < 2; ++f)
          bf[q][f] = load8(a.b + ((size_t)c.slot * a.N + min(n0 + 16 * f + r, a.N - 1)) * a.r + 32 * q + 8 * g, 32 * q + 8 * g < a.r);
      f32x4 hid[RF];
#pragma unroll
      for (int f = 0; f < RF; ++f) hid[f] = f32x4{0, 0, 0, 0};
      const uint16_t* xp = a.x + (size_t)(real ? t : 0) * a.K;
      const uint16_t* ap = a.a + (size_t)c.slot * a.r * a.K;
      // U steps of 64 a turn and wave
      constexpr int U = RF <= 2 ? 4 : 2;
      for (int k0 = wv * 64 * U; k0 < a.K; k0 += 64 * U * SW) {
        bf16x8 xf[2 * U], af[RF][2 * U];
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
          const int k = k0 + 32 * u + 8 * g;
          xf[u] = load8(xp + k, k < a.K);
#pragma unroll
          for (int f = 0; f < RF; ++f) af[f][u] = load8(ap + (size_t)min(16 * f + r, a.r - 1) * a.K + k, k < a.K);
        }
#pragma unroll
        for (int u = 0; u < 2 * U; ++u)
#pragma unroll
          for (int f = 0; f < RF; ++f) hid[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[f][u], xf[u], hid[f], 0, 0, 0);
      }
      // lane (r, g) holds row r, columns 16 f + 4 g .. + 3
#pragma unroll
      for (int f = 0; f < RF; ++f) *(f32x4*)(&s_part[wv][(r * RF + f) * 16 + 4 * g]) = hid[f];
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * KS * 32; i += 64 * SW) {
        const int row = i / (KS * 32), j = i % (KS * 32);
        float v = 0.0f;
        if (row < c.rows && j < a.r) {
#pragma unroll
          for (int q = 0; q < SW; ++q) v += s_part[q][row * RF * 16 + j];
          v *= scale;
        }
        const uint16_t h = f32_to_bf16_bits(v);
        s_hi[row * PITCH + j] = h;
        s_lo[row * PITCH + j] = f32_to_bf16_bits(v - bf16_bits_to_f32(h));
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        const bf16x8 hf = *(const bf16x8*)(s_hi + r * PITCH + 32 * q + 8 * g), lf = *(const bf16x8*)(s_lo + r * PITCH + 32 * q + 8 * g);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[q][f], hf, acc[f], 0, 0, 0);
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[q][f], lf, acc[f], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
      if (real && n0 + 16 * f + 4 * g < a.N) {
        if constexpr (BF16) {
          u32x2 o{base[f][0], base[f][1]};
          if (c.slot >= 0) o = u32x2{pack_sum(o[0], acc[f][0], acc[f][1]), pack_sum(o[1], acc[f][2], acc[f][3])};
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
using ShrinkCfg = Bf16Cfg<64, BN, 2, 1, 3>;

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
    const Chunk16 c = chunk_of<64>(gl, it / splits / ntj);
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

// 64 rows by 256 columns of out
constexpr int EW = 4;  // waves per block
__host__ __device__ inline int hidden_pitch(int r) { return (r + 31) / 32 * 32 + 8; }

template <bool BF16>
__global__ __launch_bounds__(64 * EW) void lora_expand_kernel(LoraArgs a, int splits, bool copy) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  GroupList gl;
  const int chunks = list_chunks<64>(a.g, copy, gl, (int*)smem);
  const int RP = (a.r + 31) / 32 * 32, pitch = hidden_pitch(a.r);
  uint16_t* s_hi = (uint16_t*)(smem + list_lds(a.g.E));
  uint16_t* s_lo = s_hi + 64 * pitch;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (a.N + 255) / 256;
  for (int it = blockIdx.x; it < chunks * ntn; it += gridDim.x) {
    const Chunk16 c = chunk_of<64>(gl, it / ntn);
    const int n0 = it % ntn * 256 + wv * 64;
    int t[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) t[m] = 16 * m + r < c.rows ? a.gather[c.p0 + 16 * m + r] : -1;
    f32x4 acc[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
    if (c.slot >= 0) {
      const float scale = a.scale ? a.scale[c.slot] : 1.0f;
      for (int i = threadIdx.x; i < 64 * RP / 4; i += 64 * EW) {
        const int row = i / (RP / 4), j = i % (RP / 4) * 4;
        f32x4 v = f32x4{0, 0, 0, 0};
        if (row < c.rows && j < a.r) {
          const float* h = a.ws + (size_t)(c.p0 + row) * a.r + j;
          for (int q = 0; q < splits; ++q) v += *(const f32x4*)(h + (size_t)q * a.g.P * a.r);
          v *= scale;
        }
        u32x2 hi, lo;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint16_t h0 = f32_to_bf16_bits(v[2 * q]), h1 = f32_to_bf16_bits(v[2 * q + 1]);
          hi[q] = (uint32_t)h0 | ((uint32_t)h1 << 16);
          lo[q] = (uint32_t)f32_to_bf16_bits(v[2 * q] - bf16_bits_to_f32(h0)) | ((uint32_t)f32_to_bf16_bits(v[2 * q + 1] - bf16_bits_to_f32(h1)) << 16);
        }
        *(u32x2*)(s_hi + row * pitch + j) = hi;
        *(u32x2*)(s_lo + row * pitch + j) = lo;
      }
      __syncthreads();
      const uint16_t* bp = a.b + (size_t)c.slot * a.N * a.r;
      for (int j = 8 * g; j < RP; j += 32) {
        bf16x8 bf[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) bf[f] = load8(bp + (size_t)min(n0 + 16 * f + r, a.N - 1) * a.r + j, j < a.r);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const bf16x8 hf = *(const bf16x8*)(s_hi + (16 * m + r) * pitch + j), lf = *(const bf16x8*)(s_lo + (16 * m + r) * pitch + j);
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[f], hf, acc[m][f], 0, 0, 0);
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[f], lf, acc[m][f], 0, 0, 0);
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const bool real = (uint32_t)t[m] < (uint32_t)a.g.P;
      const size_t row = (size_t)(real ? t[m] : 0) * a.N;
      if constexpr (BF16) {
        swap_fours(acc[m]);  // 16 columns of a row in one lane
        const int n = n0 + 16 * g;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (real && n + 8 * h < a.N) {
            u32x4 o = *(const u32x4*)((const uint16_t*)a.base + row + n + 8 * h);
            if (c.slot >= 0) {
              const f32x4 x = acc[m][2 * h], y = acc[m][2 * h + 1];
              o = u32x4{pack_sum(o[0], x[0], x[1]), pack_sum(o[1], x[2], x[3]), pack_sum(o[2], y[0], y[1]), pack_sum(o[3], y[2], y[3])};
            }
            *(u32x4*)((uint16_t*)a.out + row + n + 8 * h) = o;
          }
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int n = n0 + 16 * f + 4 * g;
          if (real && n < a.N) {
            f32x4 o = *(const f32x4*)((const float*)a.base + row + n);
            if (c.slot >= 0) o += acc[m][f];
            *(f32x4*)((float*)a.out + row + n) = o;
          }
        }
      }
    }
  }
}

template <int RF, bool BF16>
hipError_t launch_small(const LoraArgs& a, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = list_lds(a.g.E);
  hipError_t e = cache.get((const void*)lora_small_kernel<RF, BF16>, 64 * SW, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = ((a.g.P + 15LL) / 16 + (a.g.E + 1 < a.g.P ? a.g.E + 1 : a.g.P)) * ((a.N + 255) / 256), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL((lora_small_kernel<RF, BF16>), dim3((uint32_t)(items < most ? items : most)), dim3(64 * SW), lds, s, a, a.base != a.out);
  return hipGetLastError();
}

template <int BN>
hipError_t launch_shrink(const LoraArgs& a, int splits, long long chunks, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = ShrinkCfg<BN>::LDS + list_lds(a.g.E);
  hipError_t e = cache.get((const void*)lora_shrink_kernel<BN>, 128, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = chunks * splits * ((a.r + BN - 1) / BN), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL(lora_shrink_kernel<BN>, dim3((uint32_t)(items < most ? items : most)), dim3(128), lds, s, a, splits);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_expand(const LoraArgs& a, int splits, long long chunks, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = list_lds(a.g.E) + (size_t)2 * 64 * hidden_pitch(a.r) * 2;
  hipError_t e = cache.get((const void*)lora_expand_kernel<BF16>, 64 * EW, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = chunks * ((a.N + 255) / 256), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL(lora_expand_kernel<BF16>, dim3((uint32_t)(items < most ? items : most)), dim3(64 * EW), lds, s, a, splits, a.base != a.out);
  return hipGetLastError();
}

// Few rows: a block reads its 16 rows' x and A itself, as often as there are 256 columns.
bool lora_small(int T, int E, int r, int K) { return r <= 64 && (long long)(r + 16) * K <= 1 << 18 && (T + 15) / 16 + (E < T ? E : T) <= 256; }

long long chunks64(int T, int E) { return (T + 63) / 64 + (E < T ? E : T); }

}  // namespace

// Shares of K: enough for three blocks a compute unit, at least 256 values each.  0: no hidden rows in memory.
int lora_splits(int T, int E, int r, int K) {
  if (lora_small(T, E, r, K)) return 0;
  long long s = 768 / chunks64(T, E);
  if (s > K / 256) s = K / 256;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int T = a.g.P, splits = lora_splits(T, a.g.E, a.r, a.K);
  if (splits == 0) {
    if (a.bf16) return a.r <= 16 ? launch_small<1, true>(a, s) : a.r <= 32 ? launch_small<2, true>(a, s) : launch_small<4, true>(a, s);
    return a.r <= 16 ? launch_small<1, false>(a, s) : a.r <= 32 ? launch_small<2, false>(a, s) : launch_small<4, false>(a, s);
  }
  hipError_t e = a.r <= 16 ? launch_shrink<16>(a, splits, chunks64(T, a.g.E), s)
               : a.r <= 32 ? launch_shrink<32>(a, splits, chunks64(T, a.g.E), s) : launch_shrink<64>(a, splits, chunks64(T, a.g.E), s);
  if (e != hipSuccess) return e;
  return a.bf16 ? launch_expand<true>(a, splits, chunks64(T, a.g.E + 1), s) : launch_expand<false>(a, splits, chunks64(T, a.g.E + 1), s);
}

}  // namespace ftk
