// Tiles of the bf16 products by expert: BM x BN results of out[i][j] = sum over the reduction of R[i][.] C[j][.], in
// stages of BK (64 or 32) steps.  An operand is DIRECT when its reduction is contiguous in memory (activation rows; the matrix of a
// forward product) and ACROSS when the reduction runs over its memory rows (the matrix of a rows' gradient, both operands of a
// matrix gradient).
//
// Both go through LDS, loaded there directly, 16 bytes a lane.  A DIRECT stage is rows of 2 BK bytes; an ACROSS stage is BK
// memory rows of the tile's columns, read back with the transposing LDS read (four rows by 16 columns per 16 lanes), so that
// either way a lane gets eight consecutive reduction steps of one row or column.  Chunks are permuted by a key of the row,
// applied to the global addresses, so that the lanes of a read touch all banks.
#pragma once
#include "fp8_tile.h"  // dma16, lds_addr, unrolled
#include "ft_device.h"

namespace ftk {

// One wave: lane l's 16 bytes at its address to LDS bytes lds + AT + 16 l.
template <int AT>
__device__ __forceinline__ void dma16_at(const uint8_t* from, uint32_t lds) {
  asm volatile("s_add_u32 m0, %1, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(lds), "i"(AT) : "memory", "scc");
}

// The lane, laundered: addresses are formed from it where they are used, not kept in registers from one tile of a block to the next.
__device__ __forceinline__ int this_lane() {
  int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
  asm volatile("" : "+v"(lane));
  return lane;
}

template <int BM_, int BN_, int WM_, int WN_, int NS_, int KG_ = 1, int BK_ = 64, int NSC_ = NS_>
struct Bf16Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_;
  static constexpr int NS = NS_, NSC = NSC_;  // stages of BK steps in LDS, of the rows and of the columns
  // KG > 1: a block is KG groups of waves, each with the whole tile, a share of the reduction and stages of its own.
  static constexpr int KG = KG_, GW = WM * WN, NT = 64 * GW * KG;
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;  // fragments of a wave
  // Loads of 16 bytes a lane and stage, whole passes of all lanes: rows past BM are loaded but not read.
  static constexpr int QM = (BM * BK + 512 * GW - 1) / (512 * GW), QN = BN * BK / (512 * GW), LM = QM * 512 * GW / BK;
  static constexpr int PM = LM * BK * 2, PN = BN * BK * 2, RING = NS * PM + NSC * PN, LDS = KG * RING;  // RING: a group's stages
  static_assert(BM % (16 * WM) == 0 && BN * BK % (512 * GW) == 0 && (BK == 64 || BK == 32), "fragments, load passes");
  static_assert(NSC == NS || (NSC == NS + 1 && BK == 64), "what the waits count");
  static_assert((NS - 1) * QM + (NSC - 1) * QN <= 63, "what the load counter holds");
};

enum { DIRECT = 0, ACROSS = 1, GATHERED = 2 };  // GATHERED: DIRECT rows named by a table

// One operand of a tile: `rows` rows (DIRECT) or columns (ACROSS) from `base` on, of a matrix with `ld` values a memory row.
// GATHERED: rows gather[0 ..] of the `total` rows at base; entries outside them count as row 0.
struct Operand {
  const uint16_t* base;
  int ld, rows;
  const int32_t* gather;
  int total;
};

// An operand's loads into its part of a stage, B rows or columns wide, by GW waves.
template <int MODE, int B, int GW, int BK = 64>
struct Loader {
  static constexpr int Q = B * BK / (512 * GW);
  static constexpr int CH = MODE == ACROSS ? B / 8 : BK / 8;  // chunks of a row in LDS
  static constexpr int RP = 64 * GW / CH;                     // rows of a load pass
  uint32_t off[Q];
  const uint8_t* at[MODE == GATHERED ? Q : 1];
  const uint8_t* p;
  size_t step;  // bytes from a stage to the next

  // Rows 0 - 3 and 8 - 11 of an ACROSS stage are read together (32 bytes each), as are 16 rows of a DIRECT one (16 bytes).
  static __device__ __forceinline__ int key(int row) {
    if (MODE != ACROSS) return BK == 64 ? (row >> 1) & 7 : ((row >> 1) ^ (row >> 2)) & 3;
    return B == 64 ? (row & 2) | ((row >> 1) & 4) : 2 * ((row & 3) | ((row >> 1) & 4));
  }
  static __device__ __forceinline__ int row_of(int q, int tid) { return q * RP + tid / CH; }
  static __device__ __forceinline__ int chunk_of(int q, int tid) { return (tid % CH) ^ key(row_of(q, tid)); }

  // red: length of the reduction.  What lies past it, or past `rows`, repeats something inside.
  __device__ __forceinline__ void open(const Operand& o, int tid, int red) {
    p = (const uint8_t*)o.base;
    step = MODE == ACROSS ? (size_t)o.ld * BK * 2 : BK * 2;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = row_of(q, tid), c = chunk_of(q, tid);
      if constexpr (MODE == GATHERED) {
        const int t = o.gather[min(r, o.rows - 1)];
        at[q] = p + (size_t)((uint32_t)t < (uint32_t)o.total ? t : 0) * o.ld * 2 + (c * 8 < red ? c : 0) * 16;
        continue;
      }
      off[q] = MODE == ACROSS ? (uint32_t)min(r, red - 1) * (uint32_t)(o.ld * 2) + (uint32_t)min(c, (o.rows - 1) / 8) * 16
                      : (uint32_t)min(r, o.rows - 1) * (uint32_t)(o.ld * 2) + (uint32_t)(c * 8 < red ? c : 0) * 16;
    }
  }
  // The last stage is a short one of `left` < BK steps.
  __device__ __forceinline__ void shorten(const Operand& o, int tid, int left) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = row_of(q, tid), c = chunk_of(q, tid);
      if (MODE == GATHERED)
        at[q] -= (c * 8 < left ? 0 : c) * 16;
      else if (MODE == ACROSS)
        off[q] -= (uint32_t)(r - min(r, left - 1)) * (uint32_t)(o.ld * 2);
      else
        off[q] -= (uint32_t)(c * 8 < left ? 0 : c) * 16;
    }
  }
  template <int q, int AT>
  __device__ __forceinline__ void issue(uint32_t lds) const {
    if constexpr (MODE == GATHERED)
      dma16_at<AT + q * GW * 1024>(at[q], lds);
    else
      dma16<AT + q * GW * 1024>(p, off[q], lds);
  }
  __device__ __forceinline__ void advance() {
    if constexpr (MODE == GATHERED)
#pragma unroll
      for (int q = 0; q < Q; ++q) at[q] += BK * 2;
    else
      p += step;
  }
  __device__ __forceinline__ void skip(int stages) {
    if constexpr (MODE == GATHERED)
#pragma unroll
      for (int q = 0; q < Q; ++q) at[q] += stages * BK * 2;
    else
      p += (long long)stages * (long long)step;
  }
  // What a short stage holds past its end becomes 0.
  static __device__ __forceinline__ void clear(uint8_t* part, int tid, int left) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if ((MODE == ACROSS ? row_of(q, tid) : chunk_of(q, tid) * 8) >= left) *(u32x4*)(part + (q * 64 * GW + tid) * 16) = u32x4{0, 0, 0, 0};
  }
};

// Reads of an operand's fragments, 16 rows or columns by 32 steps, from its part of a stage.
template <int MODE, int B, int F, int BK = 64>
struct Reader {
  uint32_t off[MODE == ACROSS ? F : 1];
  __device__ __forceinline__ void open(int first, int lane) {  // first: the wave's first row or column
    const int r = lane & 15, g = lane >> 4;
    if constexpr (MODE == ACROSS) {
      const int row = 8 * g + (r >> 2), key = Loader<ACROSS, B, 1>::key(row);
#pragma unroll
      for (int f = 0; f < F; ++f) off[f] = row * B * 2 + (((first / 8 + 2 * f) ^ key) << 4) + (r & 3) * 8;
    } else {
      off[0] = (first + r) * BK * 2 + ((g ^ Loader<DIRECT, B, 1, BK>::key(r)) << 4);
    }
  }
  // half 0, 1: steps 0 - 31 and 32 - 63 of the stage
  template <int half>
  __device__ __forceinline__ bf16x8 read(const uint8_t* part, int f) const {
    if constexpr (MODE == ACROSS) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* Lds;
      const uint8_t* at = part + off[f] + half * 32 * B * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(at + 4 * B * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *(const bf16x8*)(part + (off[0] ^ (half * 64)) + f * 32 * BK);
    }
  }
};

// acc = the tile of R and C over `red` steps (0: zeros).  A wave's lane (r, g) gets row 16 m + r and columns
// 16 f + 4 g .. + 3 of its part.  Groups of waves pass their own operands, `red` and part of `lds`; those of one wave run
// without barriers, and groups of several have to have the same number of stages.
//
// One pipeline over all stages, in halves of 32 steps: while the matrix instructions of a half run from registers, the next
// half's fragments are read from LDS into other registers.  The turn to the next stage comes before the half (a stage's second, with
// BK = 64) whose fragments have been read by then: from there on the buffers of this stage take the rows of the stage NS ahead and
// the columns of the one NSC ahead.  rotate: the stage to begin with, where all are whole ones (modulo their number).
//
// Columns are an expert's matrix, most of which comes from far memory, rows are shared by the tiles beside this one: with 256 rows
// all of the LDS holds two stages of rows and three of columns.  (Three of columns against two: 128 experts of 1536 x 2112 with 256
// rows each 231 -> 210 us, 16384 rows, 7168 -> 4096, 698 -> 687 us.  A touch of the lines of later stages instead, to have them in L2 in
// time, took 15 - 30 % longer: L2 holds little more than the stages that its 32 compute units have under way.)
//
// A wave's 128 x 64 results read 24 KB of LDS per 64 steps for 64 matrix instructions of 16 cycles; eight waves of a 256 x 256 tile
// and its loads need 2048 cycles of LDS at 128 bytes a cycle, and its matrix instructions 2048.  Four waves of 128 x 128 read a
// third less, but took 40 % longer (1026 against 714 us for 16384 rows, 7168 -> 4096: one wave a SIMD waits for every read and
// barrier, and 512 registers did not hold it).
template <class C, int RMODE, int CMODE>
__device__ __forceinline__ void bf16_tile(const Operand& ro, const Operand& co, int red, uint8_t* lds, f32x4 (&acc)[C::MF][C::NF],
                                          int rotate = 0) {
  constexpr int MF = C::MF, NF = C::NF, NS = C::NS, NSC = C::NSC, U = C::QM + C::QN;
  const int lane = this_lane(), wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % C::GW, tid = wv * 64 + lane;
  const int wm = wv / C::WN, wn = wv % C::WN;
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0, 0, 0, 0};
  if (red <= 0) return;
  const int nb = (red + C::BK - 1) / C::BK, left = red % C::BK;  // stages; the last has `left` steps if that is not 0
  Loader<RMODE, C::LM, C::GW, C::BK> lr;
  Loader<CMODE, C::BN, C::GW, C::BK> lc;
  lr.open(ro, tid, red);
  lc.open(co, tid, red);
  Reader<RMODE, C::LM, MF, C::BK> rr;
  Reader<CMODE, C::BN, NF, C::BK> rc;
  rr.open(wm * 16 * MF, lane);
  rc.open(wn * 16 * NF, lane);
  const uint32_t lds0 = lds_addr(lds) + wv * 1024;
  int wrap = 0;  // the number of stages after which the first follows (0: none)
  if (rotate > 0 && left == 0) {
    const int first = rotate % nb;
    wrap = first ? nb - first : 0;
    lr.skip(first);
    lc.skip(first);
  }
  int fill_r = 0, fill_c = 0;  // stages loaded
  // As many stages of both: rows and columns side by side, one pointer; otherwise all rows, then all columns.
  constexpr bool SAME = NSC == NS;
  constexpr int SR = SAME ? C::PM + C::PN : C::PM;
  uint32_t to_r = lds0, to_c = lds0 + NS * C::PM;
  // Before the loads of a stage, once each: the last may be a short one.
  auto open_r = [&] {
    if (fill_r == nb - 1 && left && fill_r > 0) {
      lr.shorten(ro, tid, left);
      if (SAME) lc.shorten(co, tid, left);
    }
  };
  auto open_c = [&] {
    if (!SAME && fill_c == nb - 1 && left && fill_c > 0) lc.shorten(co, tid, left);
  };
  auto issue_unit = [&](auto u_) {
    constexpr int u = decltype(u_)::value;
    if constexpr (u < C::QM)
      lr.template issue<u, 0>(to_r);
    else
      lc.template issue<u - C::QM, SAME ? C::PM : 0>(SAME ? to_r : to_c);
  };
  auto advance_r = [&] {
    lr.advance();
    if (++fill_r == wrap) lr.skip(-nb);
    to_r = to_r + SR >= lds0 + NS * SR ? lds0 : to_r + SR;
  };
  auto advance_c = [&] {
    lc.advance();
    if (++fill_c == wrap) lc.skip(-nb);
    to_c = to_c + C::PN >= lds0 + C::RING ? lds0 + NS * C::PM : to_c + C::PN;
  };
  auto advance = [&] {
    if constexpr (SAME) {
      ++fill_r;
      lr.advance();
      lc.advance();
      if (fill_r == wrap) lr.skip(-nb), lc.skip(-nb);
      to_r = to_r + SR >= lds0 + NS * SR ? lds0 : to_r + SR;
    } else {
      advance_r(), advance_c();
    }
  };
  auto meet = [] {
    if constexpr (C::GW > 1) asm volatile("s_barrier" ::: "memory");
  };
  uint8_t *sr = lds, *sc = lds + NS * C::PM;  // this stage
  auto cols = [&] { return SAME ? sr + C::PM : sc; };
  auto next_stage = [&] {
    sr = sr + SR >= lds + NS * SR ? lds : sr + SR;
    if (!SAME) sc = sc + C::PN >= lds + C::RING ? lds + NS * C::PM : sc + C::PN;
  };
  auto clear = [&] {
    Loader<RMODE, C::LM, C::GW, C::BK>::clear(sr, tid, left);
    Loader<CMODE, C::BN, C::GW, C::BK>::clear(cols(), tid, left);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    meet();
  };
  bf16x8 f0[NF + MF], f1[NF + MF];  // the fragments of a half: columns, then rows
  auto frag = [&](auto half, int n) {
    constexpr int H = decltype(half)::value;
    return n < NF ? rc.template read<H>(cols(), n) : rr.template read<H>(sr, n - NF);
  };
  using Half0 = std::integral_constant<int, 0>;
  using Half1 = std::integral_constant<int, 1>;
  // Slots between a half's MM matrix instructions: fragment reads in the first three quarters, loads in the first half.
  constexpr int MM = MF * NF, RD = MF + NF, RS = MM - MM / 4, US = MM / 2 > 0 ? MM / 2 : 1;
  auto half = [&](bf16x8(&now)[NF + MF], bf16x8(&next)[NF + MF], auto h, auto loads) {
    unrolled<0, MM>([&](auto slot) {
      constexpr int i = decltype(slot)::value, m = i / NF, f = i % NF;
      acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now[f], now[NF + m], acc[m][f], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // reads n with n RS / RD == i, loads u with u US / L == i
      unrolled<(i * RD + RS - 1) / RS, (i + 1) * RD <= RS * RD ? ((i + 1) * RD + RS - 1) / RS : (i * RD + RS - 1) / RS>([&](auto n) {
        if constexpr (decltype(n)::value < RD) next[decltype(n)::value] = frag(h, decltype(n)::value);
      });
      constexpr int L = decltype(loads)::value;
      if constexpr (L > 0 && i < US) unrolled<(i * L + US - 1) / US, ((i + 1) * L + US - 1) / US>(issue_unit);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using None = std::integral_constant<int, 0>;
  using Rows = std::integral_constant<int, C::QM>;
  using Both = std::integral_constant<int, U>;

  if constexpr (SAME) {
    while (fill_r < min(NS, nb)) {
      open_r();
      unrolled<0, U>(issue_unit);
      advance();
    }
  } else {
    while (fill_c < min(NSC, nb)) {
      const bool rows = fill_c < NS;
      if (rows) {
        open_r();
        unrolled<0, C::QM>(issue_unit);
      }
      open_c();
      unrolled<C::QM, U>(issue_unit);
      advance_c();
      if (rows) advance_r();
    }
  }
  if (nb >= NSC)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NS - 1) * C::QM + (NSC - 1) * C::QN) : "memory");
  else
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  meet();
  if (nb == 1 && left) clear();
#pragma unroll
  for (int n = 0; n < NF + MF; ++n) f0[n] = frag(Half0{}, n);
  int b = 0;
  // The next stage has landed for every wave, and every wave has read this one, whose buffers may be loaded again.
  auto turn = [&] {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NS - 2) * C::QM + (NSC - 2) * C::QN) : "memory");
    meet();
    open_r(), open_c();  // (a stage's loads follow at once; the columns have none left where only rows do)
    next_stage();
  };
  auto last_turn = [&] {  // nothing is left to load
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    meet();
    next_stage();
    if (b == nb - 2 && left) clear();
  };
  // (Past the last stage fragments are read but unused.)
  if constexpr (C::BK == 64) {
    for (; b < nb - NSC; ++b) {
      half(f0, f1, Half1{}, None{});
      turn();
      half(f1, f0, Half0{}, Both{});
      advance();
    }
    if (!SAME && b < nb - NS) {
      half(f0, f1, Half1{}, None{});
      turn();
      half(f1, f0, Half0{}, Rows{});
      advance_r();
      ++b;
    }
    for (; b < nb; ++b) {
      half(f0, f1, Half1{}, None{});
      last_turn();
      half(f1, f0, Half0{}, None{});
    }
  } else {
    for (; b < nb - NS - 1; b += 2) {
      turn();
      half(f0, f1, Half0{}, Both{});
      advance();
      turn();
      half(f1, f0, Half0{}, Both{});
      advance();
    }
    if (b < nb - NS) {  // an odd one: its successor is in f1
      turn();
      half(f0, f1, Half0{}, Both{});
      advance();
      ++b;
      last_turn();
      half(f1, f0, Half0{}, None{});
      ++b;
    }
    for (; b < nb; ++b) {
      last_turn();
      half(f0, f1, Half0{}, None{});
      if (++b >= nb) break;
      last_turn();
      half(f1, f0, Half0{}, None{});
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  meet();  // the stages are free for the next tile
}

// Four lanes (g = 0 .. 3) that hold 4 g .. 4 g + 3 of four fragments' 16 columns each, swapped so that lane g holds all of
// fragment g: v[j] columns 4 j .. 4 j + 3 of it.  V: 32-bit words a lane has of a fragment.
template <class V>
__device__ __forceinline__ void swap_fours(V (&v)[4]) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i) {
    uint32_t w[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const auto word = v[f][i];  // a value: the cast of a vector's element in place reads element 0
      w[f] = __builtin_bit_cast(uint32_t, word);
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const auto x = __builtin_amdgcn_permlane32_swap(w[f], w[f + 2], false, false);
      w[f] = x[0], w[f + 2] = x[1];
    }
#pragma unroll
    for (int f = 0; f < 4; f += 2) {
      const auto x = __builtin_amdgcn_permlane16_swap(w[f], w[f + 1], false, false);
      w[f] = x[0], w[f + 1] = x[1];
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) v[f][i] = __builtin_bit_cast(std::decay_t<decltype(v[0][0])>, w[f]);
  }
}

// The same four registers, now with the pieces of a row in neighbouring lanes: after swap_fours, registers and the low two
// lane bits change places.  (A memory instruction whose neighbouring lanes lie in different rows takes four times as
// long to send off: 64 cycles for 16 bytes a lane.)
template <class V>
__device__ __forceinline__ void swap_quads(V (&v)[4], int lane) {
  const bool odd = lane & 1, upper = lane & 2;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i) {
    int w[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const auto word = v[f][i];
      w[f] = __builtin_bit_cast(int, word);
    }
#pragma unroll
    for (int f = 0; f < 4; f += 2) {
      const int a = w[f], b = w[f + 1];
      const int na = __builtin_amdgcn_update_dpp(0, a, 0xB1, 0xf, 0xf, true), nb = __builtin_amdgcn_update_dpp(0, b, 0xB1, 0xf, 0xf, true);
      w[f] = odd ? nb : a;
      w[f + 1] = odd ? b : na;
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int a = w[f], b = w[f + 2];
      const int na = __builtin_amdgcn_update_dpp(0, a, 0x4E, 0xf, 0xf, true), nb = __builtin_amdgcn_update_dpp(0, b, 0x4E, 0xf, 0xf, true);
      w[f] = upper ? nb : a;
      w[f + 2] = upper ? b : na;
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) v[f][i] = __builtin_bit_cast(std::decay_t<decltype(v[0][0])>, w[f]);
  }
}

// A wave's results of 64 columns in whole pieces of rows.  put(i, row, column, piece): the i-th piece, row of the wave's part,
// column of the 64; a piece is 4 values in fp32, or 8 in bf16 (two fragment rows at a time; MF odd: one, in halves of 4).
template <int MF, bool BF16, class Put>
__device__ __forceinline__ void each_piece(const f32x4 (&acc)[MF][4], int lane, Put put) {
  const int up = lane >> 4, mid = (lane >> 2) & 3, low = lane & 3;
  if constexpr (!BF16) {
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      f32x4 v[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) v[f] = acc[m][f];
      swap_fours(v);
      swap_quads(v, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) put(4 * m + j, 16 * m + 4 * mid + j, 16 * up + 4 * low, v[j]);
    }
  } else {
#pragma unroll
    for (int m = 0; m < MF; m += 2) {
      // v[2 (f / 2) + m % 2]: the lane's columns of fragments f, f + 1, which lanes g, g + 1 swap to 8 in a row
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int mm = m + (k & 1) < MF ? m + (k & 1) : m;
        uint32_t w[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f32x4& p = acc[mm][(k & 2) + q];
            w[q][h] = (uint32_t)f32_to_bf16_bits(p[2 * h]) | ((uint32_t)f32_to_bf16_bits(p[2 * h + 1]) << 16);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto x = __builtin_amdgcn_permlane16_swap(w[0][h], w[1][h], false, false);
          v[k][h] = x[0], v[k][2 + h] = x[1];
        }
      }
      // lane bits 5, 4: g / 2 and f % 2; after the swap f / 2 and m % 2, the registers' g / 2 and f % 2
      swap_fours(v);
      const u32x4 t = v[1];
      v[1] = v[2], v[2] = t;
      swap_quads(v, lane);  // lane bits 1, 0: f % 2 and g / 2; the registers' are the row's
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m + (up & 1) < MF) put(2 * m + j, 16 * (m + (up & 1)) + 4 * mid + j, 32 * (up >> 1) + 8 * low, v[j]);
    }
  }
}

// Store a wave's results: rows m0 + 16 m + r < rows, columns from n0 on below cols (a multiple of 8) of out with ld
// values a row.  Stores are non-temporal: results that stay in L2 push out what other tiles read again, and the kernel that reads
// them next pays nothing for it, also where they are small.  us, plain / non-temporal: 4096 tokens, Zipf, 128 experts of 1536 x 2048 matrix
// gradient 417 / 395, rows' gradient 278 / 274; 333 tokens, 64 experts of 2048 x 1032, fp32, 55.3 / 51.8; SwiGLU of 32768 rows of 768 27.5 / 26.0;
// forward of a layer of 128 such experts, top 8, of 1 token 44.0 / 44.3, 256 265 / 262, 1024 318 / 304; with its way back 495 / 478, 977 / 928, 1139 / 1052.
template <int MF, int NF, bool BF16, bool ADD>
__device__ __forceinline__ void store_rows(const f32x4 (&acc)[MF][NF], void* out, size_t ld, int m0, int rows, int n0, int cols, int lane) {
  static_assert(NF == 4, "64 columns");
  // laundered, so that the addresses are formed here and not kept in registers through the pipeline
  asm volatile("" : "+v"(lane));
  each_piece<MF, BF16>(acc, lane, [&](int, int row, int col, auto piece) {
    row += m0, col += n0;
    if (row >= rows || col >= cols) return;
    if constexpr (BF16) {
      __builtin_nontemporal_store(piece, (u32x4*)((uint16_t*)out + (size_t)row * ld + col));
    } else {
      float* o = (float*)out + (size_t)row * ld + col;
      if (ADD) piece += *(const f32x4*)o;
      __builtin_nontemporal_store(piece, (f32x4*)o);
    }
  });
}

}  // namespace ftk
