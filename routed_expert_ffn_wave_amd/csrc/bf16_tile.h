// Tiles of the bf16 products by expert: BM x BN results of out[i][j] = sum over the reduction of R[i][.] C[j][.], in
// stages of 64 steps.  An operand is DIRECT when its reduction is contiguous in memory (activation rows; the matrix of a
// forward product) and ACROSS when the reduction runs over its memory rows (the matrix of a rows' gradient, both operands of a
// matrix gradient).
//
// Both go through LDS, loaded there directly, 16 bytes a lane.  A DIRECT stage is rows of 128 bytes; an ACROSS stage is 64
// memory rows of the tile's columns, read back with the transposing LDS read (four rows by 16 columns per 16 lanes), so that
// either way a lane gets eight consecutive reduction steps of one row or column.  Chunks are permuted by a key of the row,
// applied to the global addresses, so that the lanes of a read touch all banks.
#pragma once
#include "fp8_tile.h"  // dma16, lds_addr, unrolled
#include "ft_device.h"

namespace ftk {

template <int BM_, int BN_, int WM_, int WN_, int NS_, int PER_>
struct Bf16Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;  // NS: stages in LDS
  static constexpr int PER = PER_;                                        // blocks per compute unit that the registers allow
  static constexpr int GW = WM * WN, NT = 64 * GW;
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;              // fragments of a wave
  static constexpr int QM = BM / (8 * GW), QN = BN / (8 * GW);            // loads of 16 bytes a lane and stage
  static constexpr int STAGE = (BM + BN) * 128, LDS = NS * STAGE;
  static_assert(BM % (8 * GW) == 0 && BN % (8 * GW) == 0, "load passes");
  static_assert(NF % 4 == 0, "groups of 64 columns meet in the epilogue");
  static_assert((NS - 1) * (QM + QN) <= 63, "what the load counter holds");
};

// One operand of a tile: `rows` rows (DIRECT) or columns (ACROSS) from `base` on, of a matrix with `ld` values a memory row.
struct Operand {
  const uint16_t* base;
  int ld, rows;
};

// An operand's loads into its part of a stage, B rows or columns wide, by GW waves.
template <bool ACROSS, int B, int GW>
struct Loader {
  static constexpr int Q = B / (8 * GW);
  static constexpr int CH = ACROSS ? B / 8 : 8;  // chunks of a row in LDS
  static constexpr int RP = 64 * GW / CH;        // rows of a load pass
  uint32_t off[Q];
  const uint8_t* p;
  size_t step;  // bytes from a stage to the next

  // Rows 0 - 3 and 8 - 11 of an ACROSS stage are read together (32 bytes each), as are 16 rows of a DIRECT one (16 bytes).
  static __device__ __forceinline__ int key(int row) {
    if (!ACROSS) return (row >> 1) & 7;
    return B == 64 ? (row & 2) | ((row >> 1) & 4) : 2 * ((row & 3) | ((row >> 1) & 4));
  }
  static __device__ __forceinline__ int row_of(int q, int tid) { return q * RP + tid / CH; }
  static __device__ __forceinline__ int chunk_of(int q, int tid) { return (tid % CH) ^ key(row_of(q, tid)); }

  // red: length of the reduction.  What lies past it, or past `rows`, repeats something inside.
  __device__ __forceinline__ void open(const Operand& o, int tid, int red) {
    p = (const uint8_t*)o.base;
    step = ACROSS ? (size_t)o.ld * 128 : 128;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = row_of(q, tid), c = chunk_of(q, tid);
      off[q] = ACROSS ? (uint32_t)min(r, red - 1) * (uint32_t)(o.ld * 2) + (uint32_t)min(c, (o.rows - 1) / 8) * 16
                      : (uint32_t)min(r, o.rows - 1) * (uint32_t)(o.ld * 2) + (uint32_t)(c * 8 < red ? c : 0) * 16;
    }
  }
  // The last stage is a short one of `left` < 64 steps.
  __device__ __forceinline__ void shorten(const Operand& o, int tid, int left) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = row_of(q, tid), c = chunk_of(q, tid);
      if (ACROSS)
        off[q] -= (uint32_t)(r - min(r, left - 1)) * (uint32_t)(o.ld * 2);
      else
        off[q] -= (uint32_t)(c * 8 < left ? 0 : c) * 16;
    }
  }
  // What a short stage holds past its end becomes 0.
  static __device__ __forceinline__ void clear(uint8_t* part, int tid, int left) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if ((ACROSS ? row_of(q, tid) : chunk_of(q, tid) * 8) >= left) *(u32x4*)(part + (q * 64 * GW + tid) * 16) = u32x4{0, 0, 0, 0};
  }
};

// Reads of an operand's fragments, 16 rows or columns by 32 steps, from its part of a stage.
template <bool ACROSS, int B, int F>
struct Reader {
  uint32_t off[ACROSS ? F : 1];
  __device__ __forceinline__ void open(int first, int lane) {  // first: the wave's first row or column
    const int r = lane & 15, g = lane >> 4;
    if constexpr (ACROSS) {
      const int row = 8 * g + (r >> 2), key = Loader<true, B, 1>::key(row);
#pragma unroll
      for (int f = 0; f < F; ++f) off[f] = row * B * 2 + (((first / 8 + 2 * f) ^ key) << 4) + (r & 3) * 8;
    } else {
      off[0] = (first + r) * 128 + ((g ^ Loader<false, B, 1>::key(r)) << 4);
    }
  }
  // half 0, 1: steps 0 - 31 and 32 - 63
  template <int half>
  __device__ __forceinline__ bf16x8 read(const uint8_t* part, int f) const {
    if constexpr (ACROSS) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* Lds;
      const uint8_t* at = part + off[f] + half * 32 * B * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(at + 4 * B * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *(const bf16x8*)(part + (off[0] ^ (half * 64)) + f * 2048);
    }
  }
};

// acc = the tile of R and C over `red` steps (0: zeros).  A wave's lane (r, g) gets row 16 m + r and columns
// 16 f + 4 g .. + 3 of its part.
//
// One pipeline over all stages, in halves of 32 steps: while the matrix instructions of a half run from registers, the next
// half's fragments are read from LDS into other registers.  The turn to the next stage comes before the second half, whose
// fragments have been read by then: from there on the buffer of this stage takes the loads of the stage NS ahead.
template <class C, bool RACROSS, bool CACROSS>
__device__ __forceinline__ void bf16_tile(const Operand& ro, const Operand& co, int red, uint8_t* lds, f32x4 (&acc)[C::MF][C::NF]) {
  constexpr int MF = C::MF, NF = C::NF, NS = C::NS, U = C::QM + C::QN;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv / C::WN, wn = wv % C::WN;
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  if (red <= 0) return;
  const int nb = (red + 63) / 64, left = red & 63;  // stages; the last has `left` steps if that is not 0
  Loader<RACROSS, C::BM, C::GW> lr;
  Loader<CACROSS, C::BN, C::GW> lc;
  lr.open(ro, tid, red);
  lc.open(co, tid, red);
  Reader<RACROSS, C::BM, MF> rr;
  Reader<CACROSS, C::BN, NF> rc;
  rr.open(wm * 16 * MF, lane);
  rc.open(wn * 16 * NF, lane);
  const uint32_t lds0 = lds_addr(lds) + wv * 1024;
  int fill = 0;
  uint32_t fill_lds = lds0;
  auto open = [&] {
    if (fill == nb - 1 && left && fill > 0) {
      lr.shorten(ro, tid, left);
      lc.shorten(co, tid, left);
    }
  };
  auto issue_unit = [&](auto u_) {
    constexpr int u = decltype(u_)::value;
    if constexpr (u < C::QM)
      dma16<u * C::GW * 1024>(lr.p, lr.off[u], fill_lds);
    else
      dma16<C::BM * 128 + (u - C::QM) * C::GW * 1024>(lc.p, lc.off[u - C::QM], fill_lds);
  };
  auto advance = [&] {
    ++fill;
    lr.p += lr.step;
    lc.p += lc.step;
    fill_lds = fill_lds + C::STAGE >= lds0 + C::LDS ? lds0 : fill_lds + C::STAGE;
  };
  auto clear = [&](uint8_t* st) {
    Loader<RACROSS, C::BM, C::GW>::clear(st, tid, left);
    Loader<CACROSS, C::BN, C::GW>::clear(st + C::BM * 128, tid, left);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  bf16x8 f0[NF + MF], f1[NF + MF];  // the fragments of a half: columns, then rows
  uint8_t* st = lds;
  auto frag = [&](const uint8_t* from, auto half, int n) {
    constexpr int H = decltype(half)::value;
    return n < NF ? rc.template read<H>(from + C::BM * 128, n) : rr.template read<H>(from, n - NF);
  };
  using Half0 = std::integral_constant<int, 0>;
  using Half1 = std::integral_constant<int, 1>;
  // Slots between a half's MM matrix instructions: fragment reads in the first three quarters, loads from the start on.
  constexpr int MM = MF * NF, RS = (MM - MM / 4) / (NF + MF), DS = MM / 2 / U > 0 ? MM / 2 / U : 1;
  static_assert(RS >= 1 && U * DS <= MM, "a half's reads and a stage's loads fit its matrix instructions");
  auto half = [&](bf16x8(&now)[NF + MF], bf16x8(&next)[NF + MF], const uint8_t* from, auto h, auto loads) {
#pragma unroll
    for (int i = 0; i < MM; ++i) {
      const int m = i / NF, f = i % NF;
      acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now[f], now[NF + m], acc[m][f], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (i % RS == 0 && i / RS < NF + MF) next[i / RS] = frag(from, h, i / RS);
      if constexpr (decltype(loads)::value)
        unrolled<0, U>([&](auto u) {
          if (decltype(u)::value * DS == i) issue_unit(u);
        });
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto after = [&](uint8_t* s) { return s + C::STAGE >= lds + C::LDS ? lds : s + C::STAGE; };

  while (fill < min(NS, nb)) {
    open();
    unrolled<0, U>(issue_unit);
    advance();
  }
  if (nb >= NS)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 1) * U) : "memory");
  else
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (nb == 1 && left) clear(st);
#pragma unroll
  for (int n = 0; n < NF + MF; ++n) f0[n] = frag(st, Half0{}, n);
  int b = 0;
  for (; b < nb - NS; ++b) {
    half(f0, f1, st, Half1{}, std::false_type{});
    // the next stage has landed for every wave, and every wave has read this one
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * U) : "memory");
    open();
    st = after(st);
    half(f1, f0, st, Half0{}, std::true_type{});
    advance();
  }
  for (; b < nb; ++b) {  // nothing left to load
    half(f0, f1, st, Half1{}, std::false_type{});
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    st = after(st);
    if (b == nb - 2 && left) clear(st);
    half(f1, f0, st, Half0{}, std::false_type{});  // past the last stage: read but unused
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the stages are free for the next tile
}

// Store a wave's results: rows m0 + 16 m + r < rows, columns from n0 on below cols (a multiple of 8) of out with ld
// values a row.
template <int MF, int NF, bool BF16, bool ADD>
__device__ __forceinline__ void store_rows(const f32x4 (&acc)[MF][NF], void* out, size_t ld, int m0, int rows, int n0, int cols, int lane) {
  // laundered, so that the addresses are formed here and not kept in registers through the pipeline
  asm volatile("" : "+v"(lane));
  const int r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int q = 0; q < MF * NF / 4; ++q) {
    const int m = q / (NF / 4), f0 = q % (NF / 4) * 4, row = m0 + 16 * m + r, n = n0 + 16 * f0;
    if constexpr (BF16) {
      // four lanes hold a row's 16 columns of every fragment in fours: swapped so that each holds 16 of one fragment
      uint32_t w[4][2];
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[f][h] = (uint32_t)f32_to_bf16_bits(acc[m][f0 + f][2 * h]) | ((uint32_t)f32_to_bf16_bits(acc[m][f0 + f][2 * h + 1]) << 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const auto x = __builtin_amdgcn_permlane32_swap(w[f][h], w[f + 2][h], false, false);
          w[f][h] = x[0], w[f + 2][h] = x[1];
        }
#pragma unroll
        for (int f = 0; f < 4; f += 2) {
          const auto x = __builtin_amdgcn_permlane16_swap(w[f][h], w[f + 1][h], false, false);
          w[f][h] = x[0], w[f + 1][h] = x[1];
        }
      }
      uint16_t* o = (uint16_t*)out + (size_t)row * ld + n + 16 * g;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (row < rows && n + 16 * g + 8 * h < cols) *(u32x4*)(o + 8 * h) = u32x4{w[2 * h][0], w[2 * h][1], w[2 * h + 1][0], w[2 * h + 1][1]};
    } else {
      float* o = (float*)out + (size_t)row * ld + n + 4 * g;
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (row < rows && n + 16 * f + 4 * g < cols) {
          f32x4 v = acc[m][f0 + f];
          if (ADD) v += *(const f32x4*)(o + 16 * f);
          *(f32x4*)(o + 16 * f) = v;
        }
    }
  }
}

}  // namespace ftk
