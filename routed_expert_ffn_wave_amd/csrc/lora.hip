// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale_s (x[t] A_s^T) B_s^T,  s the slot of row t's adapter; rows without one: out[t] = base[t].
// Two kernels.  The first forms the hidden rows h = x A^T (r values each) by splits of K, so that few rows keep many
// compute units busy; the second adds the splits up in a fixed order and multiplies with B.  Hidden values are held in
// fp32; the second product takes them as two bf16 terms (the value and what its rounding left), so that they carry 16 bits or
// more of it and not 8.
#include "ft_device.h"
#include "ft_groups.h"
#include "ft_kernels.h"
#include "ft_products.h"

namespace ftk {
namespace {

constexpr int LW = 4;  // waves per block

// Chunks of up to ROWS rows of one adapter; with COPY also those of rows without one (slot -1).
template <int ROWS, bool COPY>
__device__ __forceinline__ int list_chunks(const RowGroups& s, GroupList& g, int* lds) {
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
        return cnt > 0 && (COPY || slot >= 0);
      },
      [](int cnt) { return (cnt + ROWS - 1) / ROWS; });
  return g.item0[g.n];
}
size_t chunks_lds(int E) { return group_lds_bytes(E + 1); }

// h[split][p][j] = sum over the split's k of x[gather[p]][k] A[j][k] for 16 positions p, 16 RF columns j; the block's
// waves share the split in turns of 32 values.
template <int RF>
__global__ __launch_bounds__(64 * LW) void lora_shrink_kernel(LoraArgs a, int splits) {
  extern __shared__ __attribute__((aligned(16))) int lds[];
  __shared__ __attribute__((aligned(16))) float s_part[LW][RF * 256];
  GroupList gl;
  const int chunks = list_chunks<16, false>(a.g, gl, lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntj = (a.r + 16 * RF - 1) / (16 * RF), steps = (a.K + 31) / 32;
  for (int it = blockIdx.x; it < chunks * splits * ntj; it += gridDim.x) {
    const int split = it % splits, jt = it / splits % ntj, ch = it / splits / ntj;
    const int gi = find_group(gl.item0, gl.n, ch);
    const int p0 = gl.row0[gi] + (ch - gl.item0[gi]) * 16, rows = min(16, gl.row0[gi] + gl.cnt[gi] - p0), j0 = jt * 16 * RF;
    const int s0 = (int)((long long)steps * split / splits), s1 = (int)((long long)steps * (split + 1) / splits);
    const int t = a.gather[p0 + min(r, rows - 1)];
    const bool real = (uint32_t)t < (uint32_t)a.g.P;
    const uint16_t* xp = a.x + (size_t)(real ? t : 0) * a.K;
    const uint16_t* ap = a.a + ((size_t)gl.slot[gi] * a.r) * a.K;
    f32x4 acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[f] = f32x4{0, 0, 0, 0};
    const bf16x8 none = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
    for (int s = s0 + wv; s < s1; s += LW) {
      const int k = s * 32 + 8 * g;
      const bool in = k < a.K;
      const bf16x8 xf = in ? *(const bf16x8*)(xp + k) : none;
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const int j = min(j0 + 16 * f + r, a.r - 1);
        const bf16x8 af = in ? *(const bf16x8*)(ap + (size_t)j * a.K + k) : none;
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, xf, acc[f], 0, 0, 0);
      }
    }
    // lane (r, g) holds row r, columns 16 f + 4 g .. + 3
#pragma unroll
    for (int f = 0; f < RF; ++f) *(f32x4*)(&s_part[wv][(r * RF + f) * 16 + 4 * g]) = acc[f];
    __syncthreads();
    for (int i = threadIdx.x; i < RF * 256; i += 64 * LW) {
      float v = s_part[0][i];
#pragma unroll
      for (int q = 1; q < LW; ++q) v += s_part[q][i];
      const int row = i / (16 * RF), j = j0 + i % (16 * RF);
      if (row < rows && j < a.r) a.ws[((size_t)split * a.g.P + p0 + row) * a.r + j] = v;
    }
    __syncthreads();
  }
}

// 16 rows by 256 columns of out; RP: r rounded up to a multiple of 32
template <bool BF16>
__global__ __launch_bounds__(64 * LW) void lora_expand_kernel(LoraArgs a, int splits, bool copy) {
  extern __shared__ __attribute__((aligned(16))) int lds[];
  GroupList gl;
  const int chunks = copy ? list_chunks<16, true>(a.g, gl, lds) : list_chunks<16, false>(a.g, gl, lds);
  const int RP = (a.r + 31) / 32 * 32, pitch = RP + 8;
  uint16_t* s_hi = (uint16_t*)((uint8_t*)lds + ((size_t)(4 * (a.g.E + 3) + 4) * 4 + 15 & ~(size_t)15));
  uint16_t* s_lo = s_hi + 16 * pitch;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int ntn = (a.N + 255) / 256;
  for (int it = blockIdx.x; it < chunks * ntn; it += gridDim.x) {
    const int ch = it / ntn, n0 = it % ntn * 256 + wv * 64;
    const int gi = find_group(gl.item0, gl.n, ch);
    const int slot = gl.slot[gi], p0 = gl.row0[gi] + (ch - gl.item0[gi]) * 16, rows = min(16, gl.row0[gi] + gl.cnt[gi] - p0);
    const int t = r < rows ? a.gather[p0 + r] : -1;
    const bool real = (uint32_t)t < (uint32_t)a.g.P;
    f32x4 acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = f32x4{0, 0, 0, 0};
    if (slot >= 0) {
      const float scale = a.scale ? a.scale[slot] : 1.0f;
      for (int i = threadIdx.x; i < 16 * RP; i += 64 * LW) {
        const int row = i / RP, j = i % RP;
        float v = 0.0f;
        if (row < rows && j < a.r) {
          for (int q = 0; q < splits; ++q) v += a.ws[((size_t)q * a.g.P + p0 + row) * a.r + j];
          v *= scale;
        }
        const uint16_t h = f32_to_bf16_bits(v);
        s_hi[row * pitch + j] = h;
        s_lo[row * pitch + j] = f32_to_bf16_bits(v - bf16_bits_to_f32(h));
      }
      __syncthreads();
      const uint16_t* bp = a.b + (size_t)slot * a.N * a.r;
      const bf16x8 none = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
      for (int j = 8 * g; j < RP; j += 32) {
        const bf16x8 hf = *(const bf16x8*)(s_hi + r * pitch + j), lf = *(const bf16x8*)(s_lo + r * pitch + j);
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int n = min(n0 + 16 * f + r, a.N - 1);
          const bf16x8 bf = j < a.r ? *(const bf16x8*)(bp + (size_t)n * a.r + j) : none;
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf, hf, acc[f], 0, 0, 0);
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf, lf, acc[f], 0, 0, 0);
        }
      }
      __syncthreads();
    }
    if (real)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int n = n0 + 16 * f + 4 * g;
        if (n >= a.N) continue;
        const size_t at = (size_t)t * a.N + n;
        if (BF16) {
          const u32x2 b = *(const u32x2*)((const uint16_t*)a.base + at);
          u32x2 o = b;
          if (slot >= 0)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            o[h] = (uint32_t)f32_to_bf16_bits(__uint_as_float(b[h] << 16) + acc[f][2 * h]) |
                   ((uint32_t)f32_to_bf16_bits(__uint_as_float(b[h] & 0xffff0000u) + acc[f][2 * h + 1]) << 16);
          *(u32x2*)((uint16_t*)a.out + at) = o;
        } else {
          f32x4 o = *(const f32x4*)((const float*)a.base + at);
          if (slot >= 0) o += acc[f];
          *(f32x4*)((float*)a.out + at) = o;
        }
      }
  }
}

template <int RF>
hipError_t launch_shrink(const LoraArgs& a, int splits, long long chunks, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = chunks_lds(a.g.E);
  hipError_t e = cache.get((const void*)lora_shrink_kernel<RF>, 64 * LW, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = chunks * splits * ((a.r + 16 * RF - 1) / (16 * RF)), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL(lora_shrink_kernel<RF>, dim3((uint32_t)(items < most ? items : most)), dim3(64 * LW), lds, s, a, splits);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_expand(const LoraArgs& a, int splits, bool copy, long long chunks, hipStream_t s) {
  static LaunchCache cache;
  LaunchFacts f;
  const size_t lds = ((size_t)(4 * (a.g.E + 3) + 4) * 4 + 15 & ~(size_t)15) + 2 * 16 * ((a.r + 31) / 32 * 32 + 8) * 2;
  hipError_t e = cache.get((const void*)lora_expand_kernel<BF16>, 64 * LW, lds, &f);
  if (e != hipSuccess) return e;
  const long long items = chunks * ((a.N + 255) / 256), most = (long long)f.per_cu * f.cus;
  hipLaunchKernelGGL(lora_expand_kernel<BF16>, dim3((uint32_t)(items < most ? items : most)), dim3(64 * LW), lds, s, a, splits, copy);
  return hipGetLastError();
}

}  // namespace

// Shares of K: enough for two blocks a compute unit, at least 256 values each.
int lora_splits(int T, int E, int r, int K) {
  const long long chunks = (T + 15) / 16 + (E < T ? E : T);
  long long s = 512 / (chunks > 0 ? chunks : 1);
  if (s > K / 256) s = K / 256;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int T = a.g.P, splits = lora_splits(T, a.g.E, a.r, a.K);
  const bool copy = a.base != a.out;
  const long long chunks = (T + 15) / 16 + (a.g.E + 1 < T ? a.g.E + 1 : T);
  hipError_t e = a.r <= 16 ? launch_shrink<1>(a, splits, chunks, s)
               : a.r <= 32 ? launch_shrink<2>(a, splits, chunks, s) : launch_shrink<4>(a, splits, chunks, s);
  if (e != hipSuccess) return e;
  return a.bf16 ? launch_expand<true>(a, splits, copy, chunks, s) : launch_expand<false>(a, splits, copy, chunks, s);
}

}  // namespace ftk
