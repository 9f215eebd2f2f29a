// Tiles of the 8-bit product for many rows: BM activation rows x BN weight rows per block, K steps of one
// 128-block, so that a step's partial products are scaled with one fp32 factor per activation row.
//
// A block's waves form a WM x WN grid; a wave holds (BM / WM) x (BN / WN) results as 16 x 16 fragments whose
// rows are weight rows and whose columns are activation rows: a lane's values of a fragment belong to one
// activation row, so one factor scales all four of them, and the four fragments of a wave take the weight
// rows in an order that leaves 16 consecutive columns of out in one lane.
//
// Both operands go through LDS, loaded there directly (16 bytes a lane) one to three steps ahead into the
// other stages.  Rows are 128 bytes in LDS; their eight 16-byte chunks are permuted by a key of the row so that
// the 16 lanes that read one chunk of 16 rows touch all banks.  The permutation is applied to the global
// addresses, which stay inside the same 128 bytes.
//
// What bounds it: 8192 x 4096 x 7168 with 256 x 256 tiles takes 205 - 255 us (1.9 - 2.35 PFLOP/s; the clock falls to
// about 1.5 GHz under it, and the time follows the clock the card gives).  Matrix instructions fill 58 - 65 % of
// the cycles.  Of 244 us, leaving out the loads gave 202, the LDS reads 223, the fp32 multiply-adds 222: no single one
// bounds it.  Registers only, the loop's matrix instructions with their multiply-adds run at 3.7 PFLOP/s.
// A wave's 128 x 64 results (256 x 256 tiles) read 24 KB of LDS per 32 matrix instructions, 64 x 64 read 16 KB per 16:
// larger tiles a wave need more than the 256 registers that two waves a SIMD have.
//
// Exact products (WIDE) convert codes to bf16 and take twice the matrix cycles: 8192 x 4096 x 7168 in 434 - 505 us.
// In its loop the conversions and multiply-adds do not run beside the matrix instructions (459 k cycles of matrix
// instructions and 395 k of others add up in 946 k), though the 8-bit loop's multiply-adds do; every wave converts operands that
// up to four waves share.  A loop ordered by hand like the 8-bit one took the same time; why is not known.
#pragma once
#include <type_traits>

#include "fp8_tile_cfg.h"
#include "ft_device.h"
#include "ft_rows.h"

namespace ftk {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// One wave: lane l's 16 (4) bytes at base + voff to LDS bytes lds + AT + 16 l (4 l).  M0 carries the LDS address (one
// wait state after writing it); nothing else in these kernels reads M0 (it serves indexed registers, interpolation
// and messages), so it is not put back.
template <int AT>
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds), "i"(AT)
               : "memory", "scc");
}
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(lds)
               : "memory");
}
// f(integral_constant<int, I>) for I = B .. E - 1
template <int B, int E, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    unrolled<B + 1, E>(f);
  }
}

// Position of 16-byte chunk c of a row in LDS.  A rows are read 16 in a row; the fragments of a wave's
// weight rows take rows 16 (r / 4) + 4 f + r % 4.
__device__ __forceinline__ int key_a(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int key_b(int row) { return ((row >> 1) & 1) | ((row >> 3) & 6); }

struct TileJob {
  int slot, row0, rows, n0;  // rows: activation rows of this tile, 1 .. BM
};

template <class C, bool BF16>
__device__ __forceinline__ void fp8_tile(const Fp8MatmulArgs& a, const TileJob& job, uint8_t* lds) {
  constexpr int MF = C::MF, NF = C::NF;
  const int lane = threadIdx.x & 63, gwv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = gwv / C::GW, wv = gwv % C::GW, tid = wv * 64 + lane;  // in the group
  const int r = lane & 15, g = lane >> 4;
  const int wm = wv / C::WN, wn = wv % C::WN;
  const int K = a.K, nb = (K + 127) / 128, nblk_n = (a.N + 127) / 128;
  const int b0 = nb * kg / C::KG, b1 = nb * (kg + 1) / C::KG;  // this group's blocks
  uint8_t* const block_lds = lds;
  lds += kg * C::GROUP;
  const uint32_t lds0 = lds_addr(lds);

  // ---- loads: rows past the end repeat the last one (their results are not stored)
  const int lrow = tid >> 3;
  auto ca = [&](int q) { return (tid & 7) ^ key_a(q * C::RQ + lrow); };
  auto cb = [&](int q) { return (tid & 7) ^ key_b(q * C::RQ + lrow); };
  const int wrows = min(C::BN, a.N - job.n0);
  uint32_t va[C::QA], vb[C::QB];
#pragma unroll
  for (int q = 0; q < C::QA; ++q) va[q] = (uint32_t)min(q * C::RQ + lrow, job.rows - 1) * (uint32_t)K + ca(q) * 16;
#pragma unroll
  for (int q = 0; q < C::QB; ++q) vb[q] = (uint32_t)min(q * C::RQ + lrow, wrows - 1) * (uint32_t)K + cb(q) * 16;
  const uint32_t vs = (uint32_t)min(tid, job.rows - 1) * (uint32_t)a.S * 4;
  const uint8_t* pa = a.a + (size_t)job.row0 * K + (size_t)b0 * 128;
  const uint8_t* pb = a.w + ((size_t)job.slot * a.N + job.n0) * K + (size_t)b0 * 128;
  const uint8_t* ps = (const uint8_t*)(a.sa + (size_t)job.row0 * a.S);
  const uint8_t* pw = (const uint8_t*)(a.sw + ((size_t)job.slot * nblk_n + job.n0 / 128) * nb);
  const int wblk = min((lane >> 2) & (C::BN > 128 ? C::BN / 128 - 1 : 0), nblk_n - 1 - job.n0 / 128);  // lane / 4's block of 128 weight rows
  const int nfull = K >> 7;  // whole blocks; a shorter one may follow
  // The loads of a stage, one at a time, in stage order: U units of 16 bytes a lane, and every fourth stage a load
  // of the next 4 steps' scales (the last wave's are the weights').  fill: the stage being loaded and its buffer.
  constexpr int U = C::QA + C::QB, NS = C::NS;
  int fill = b0;
  uint32_t fill_lds = lds0 + wv * 1024;
  auto issue_unit = [&](auto u_) {
    constexpr int u = decltype(u_)::value;
    if constexpr (u < C::QA)
      dma16<u * C::RQ * 128>(pa, va[u], fill_lds);
    else
      dma16<(C::BM + (u - C::QA) * C::RQ) * 128>(pb, vb[u - C::QA], fill_lds);
  };
  // Before a stage's units: its scales, and chunks of a short block past K load the block's first chunk (turn()
  // clears them).
  auto open = [&] {
    if ((fill & 3) == 0 || fill == b0) {
      const uint32_t half = (fill >> 2) & 1, first = fill & ~3;
      if (wv < C::BM / 64) dma16<C::SBUF>(ps + (size_t)first * 4, vs, lds0 + half * C::BM * 16 + wv * 1024);
      if (wv == C::GW - 1)
        dma4(pw, (uint32_t)(wblk * nb + min((int)first + (lane & 3), nb - 1)) * 4, lds0 + C::SW + half * 256);
    }
    if (fill == nfull) {
#pragma unroll
      for (int q = 0; q < C::QA; ++q) va[q] -= fill * 128 + ca(q) * 16 < K ? 0 : ca(q) * 16;
#pragma unroll
      for (int q = 0; q < C::QB; ++q) vb[q] -= fill * 128 + cb(q) * 16 < K ? 0 : cb(q) * 16;
    }
  };
  // After them: the next stage.
  auto advance = [&] {
    ++fill;
    pa += 128;
    pb += 128;
    fill_lds += C::STAGE;
    if (fill_lds >= lds0 + NS * C::STAGE) fill_lds -= NS * C::STAGE;
  };
  auto issue = [&] {
    open();
    unrolled<0, U>(issue_unit);
    advance();
  };

  // ---- fragment reads: byte offsets of this lane's chunks g and g + 4 inside a stage
  const int arow = wm * 16 * MF + r, brow = wn * 16 * NF + 16 * (r >> 2) + (r & 3);
  const uint32_t ra = arow * 128 + ((g ^ key_a(r)) << 4);
  // fragment f reads rows brow + 4 f: the key's bits 1, 4 and 5 of the row do not change with f
  const uint32_t rb = C::BM * 128 + brow * 128 + ((g ^ key_b(brow)) << 4);
  const uint32_t rs = C::SBUF + arow * 16, rw = C::SW + wn * 16 * NF / 128 * 16;

  f32x4 acc[MF][NF];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[m][f] = f32x4{0, 0, 0, 0};

  // this lane's two chunks of a fragment in the stage at `st`
  auto frag = [&](const uint8_t* st, uint32_t off) {
    const u32x4 lo = *(const u32x4*)(st + off), hi = *(const u32x4*)(st + (off ^ 64));
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  auto after = [&](const uint8_t* st) { return st + C::STAGE < lds + NS * C::STAGE ? st + C::STAGE : (const uint8_t*)lds; };
  auto sa_of = [&](int b, int m) {
    return *(const float*)(lds + rs + ((b >> 2) & 1) * C::BM * 16 + (b & 3) * 4 + m * 256);
  };
  auto sw_of = [&](int b) { return *(const float*)(lds + rw + ((b >> 2) & 1) * 256 + (b & 3) * 4); };
  // Before stage b is read: its loads have landed for every wave, and every wave is done with the stage before it,
  // whose buffer can be loaded again.  The chunks of a short block that lie past K become zero codes.
  // (The stages after it that are in flight, U loads or one more each, may stay so.)
  auto turn = [&](int b, const uint8_t* stage) {
    const int newer = min(NS - 2, b1 - 1 - b);
    if (NS == 4 && newer == 2)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * U) : "memory");
    else if (NS > 2 && newer == 1)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(U) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if constexpr (C::GW > 1) asm volatile("s_barrier" ::: "memory");
    if (b == nfull) {
      uint8_t* st = const_cast<uint8_t*>(stage) + tid * 16;
#pragma unroll
      for (int q = 0; q < C::QA; ++q)
        if (b * 128 + ca(q) * 16 >= K) *(u32x4*)(st + q * C::RQ * 128) = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < C::QB; ++q)
        if (b * 128 + cb(q) * 16 >= K) *(u32x4*)(st + C::BM * 128 + q * C::RQ * 128) = u32x4{0, 0, 0, 0};
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if constexpr (C::GW > 1) asm volatile("s_barrier" ::: "memory");
    }
  };

  // Groups of several waves share the block's barrier: each passes it as often as the one with most to do.
  auto even_out = [&] {
    if constexpr (C::KG > 1 && C::GW > 1)
      for (int i = b1 - b0 + (b0 <= nfull && nfull < b1); i < (nb + C::KG - 1) / C::KG + (nfull < nb); ++i) asm volatile("s_barrier" ::: "memory");
  };

  if (C::KG > 1 && b0 == b1) {
    // fewer blocks than groups
  } else if (C::GW > 1 && wm * 16 * MF >= job.rows) {
    // a wave without rows: its share of the loads and the turns
    while (fill < min(b0 + NS - 1, b1)) issue();
    const uint8_t* st = lds;
    for (int b = b0; b < b1; ++b, st = after(st)) {
      turn(b, st);
      if (fill < b1) issue();
    }
  } else if constexpr (!C::WIDE) {
    // The instruction stream is one pipeline over all steps, in groups of two fragment rows by four fragments:
    // each matrix instruction is followed by the multiply-adds of the fragment two instructions back and by
    // LDS reads of what comes a group later.  The turn from stage b to b + 1 comes before the last group of
    // step b, whose operands are in registers by then, and a weight fragment is read again, from
    // stage b + 1, right after its last use: every LDS read has 7 to 8 matrix instructions to land.
    constexpr int G = MF / 2;
    constexpr int SPREAD = 4 * U <= 8 * G * 2 ? 4 : 2;  // twice the matrix instructions per load
    static_assert(U * SPREAD / 2 > 8 && U * SPREAD / 2 <= 8 * G, "a stage's loads end before the next turn, in the next step");
    static_assert(G % 2 == 0, "the operand buffers alternate by group");
    i32x8 wf[NF], af[2][2];
    f32x4 part[4];
    float sa[2], sc[2] = {0.0f, 0.0f}, sw;
    part[2] = part[3] = f32x4{0, 0, 0, 0};
    auto fold = [&](f32x4& c, const f32x4& q, float s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = fmaf(q[i], s, c[i]);
      asm volatile("" : "+v"(c));  // here, not sunk to where it is next read
    };
    while (fill < min(b0 + NS - 1, b1)) issue();
    turn(b0, lds);
    if (fill < b1) issue();
#pragma unroll
    for (int f = 0; f < NF; ++f) wf[f] = frag(lds, rb + f * 512);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      af[0][i] = frag(lds, ra + i * 2048);
      sa[i] = sa_of(b0, i);
    }
    sw = sw_of(b0);
    const uint8_t* st = lds;
    for (int b = b0; b < b1; ++b) {
      const uint8_t* nx = after(st);  // past the last step: read but unused
      // the stage that takes the buffer freed by the last turn is loaded after it: first units in the last group of
      // a step, the others in the next step's
      bool filling = b > b0 && fill < b1;
#pragma unroll
      for (int p = 0; p < G; ++p) {
        if (p == G - 1) {
          if (filling) advance();
          filling = false;
          if (b + 1 < b1) {
            turn(b + 1, nx);
            filling = fill < b1;
            if (filling) open();
          }
        }
        const float before[2] = {sc[0], sc[1]};
        sc[0] = sa[0] * sw;
        sc[1] = sa[1] * sw;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          part[s & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[s >> 1], af[p & 1][s & 1], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          if (s < 2)
            fold(acc[(2 * p + MF - 2 + s) % MF][3], part[s + 2], before[s]);
          else
            fold(acc[2 * p + (s & 1)][(s - 2) >> 1], part[(s - 2) & 3], sc[s & 1]);
          const bool turned = p == G - 1;
          if (s == 0 || s == 2) af[(p + 1) & 1][s >> 1] = frag(turned ? nx : st, ra + (turned ? 0 : 2 * p + 2) * 2048 + (s >> 1) * 2048);
          if (s == 4) {
            sa[0] = sa_of(turned ? b + 1 : b, turned ? 0 : 2 * p + 2);
            sa[1] = sa_of(turned ? b + 1 : b, turned ? 1 : 2 * p + 3);
            if (turned) sw = sw_of(b + 1);
          }
          if (turned && (s & 1)) wf[s >> 1] = frag(nx, rb + (s >> 1) * 512);
          const int k = ((p + 1) % G) * 8 + s;
          unrolled<0, U>([&](auto u) {
            if (decltype(u)::value * SPREAD / 2 == k && filling) issue_unit(u);
          });
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      st = nx;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) fold(acc[MF - 2 + i][3], part[i + 2], sc[i]);
  } else {
    auto step = [&](int b, const uint8_t* st) {
      const float sw = sw_of(b);
      bf16x8 wf[NF][4];
      auto wide = [&](uint32_t off, bf16x8(&o)[4]) {
        const i32x8 c = frag(st, off);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          u32x4 p;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            p[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[2 * h + i], 1.0f, false));
            p[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)c[2 * h + i], 1.0f, true));
          }
          o[h] = __builtin_bit_cast(bf16x8, p);
        }
      };
#pragma unroll
      for (int f = 0; f < NF; ++f) wide(rb + f * 512, wf[f]);
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        bf16x8 af[4];
        wide(ra + m * 2048, af);
        const float sc = sa_of(b, m) * sw;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          f32x4 part = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int h = 0; h < 4; ++h) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[f][h], af[h], part, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][f][i] = fmaf(part[i], sc, acc[m][f][i]);
        }
      }
    };
    while (fill < min(b0 + NS - 1, b1)) issue();
    const uint8_t* st = lds;
    for (int b = b0; b < b1; ++b, st = after(st)) {
      turn(b, st);
      if (fill < b1) issue();
      step(b, st);
    }
  }
  // 16 consecutive results of a row
  auto store = [&](int row, int n, const f32x4 (&v)[4]) {
    if (row >= job.rows || n >= a.N) return;
    const size_t at = (size_t)(job.row0 + row) * a.N + n;
    const bool whole = n + 16 <= a.N && (a.N & (BF16 ? 7 : 3)) == 0;
    if constexpr (BF16) {
      uint16_t* o = (uint16_t*)a.out + at;
      if (whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4& p = v[2 * h + i / 2];
            w[i] = (uint32_t)f32_to_bf16_bits(p[2 * (i & 1)]) | ((uint32_t)f32_to_bf16_bits(p[2 * (i & 1) + 1]) << 16);
          }
          *(u32x4*)(o + 8 * h) = w;
        }
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + 4 * f + i < a.N) o[4 * f + i] = f32_to_bf16_bits(v[f][i]);
      }
    } else {
      float* o = (float*)a.out + at;
      if (whole) {
#pragma unroll
        for (int f = 0; f < 4; ++f) *(f32x4*)(o + 4 * f) = v[f];
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + 4 * f + i < a.N) o[4 * f + i] = v[f][i];
      }
    }
  };

  if constexpr (C::KG == 1) {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the stages are free for the next tile
    // lane (r, g), fragment row m: row wm 16 MF + 16 m + r, columns wn 64 + 16 g .. + 15
#pragma unroll
    for (int m = 0; m < MF; ++m) store(arow + 16 * m, job.n0 + wn * 16 * NF + 16 * g, acc[m]);
  } else {
    // every wave's results over its own stages, then the sums in the order of K
    float* mine = (float*)lds;
    even_out();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if constexpr (C::GW > 1) asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int f = 0; f < NF; ++f) *(f32x4*)(mine + (arow + 16 * m) * C::PITCH + wn * 16 * NF + 16 * g + 4 * f) = acc[m][f];
    __syncthreads();
    for (int i = threadIdx.x; i < C::BM * C::BN / 16; i += C::NT) {
      const int row = i / (C::BN / 16), n = i % (C::BN / 16) * 16;
      f32x4 v[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) v[f] = *(const f32x4*)((const float*)block_lds + row * C::PITCH + n + 4 * f);
#pragma unroll
      for (int q = 1; q < C::KG; ++q)
#pragma unroll
        for (int f = 0; f < 4; ++f) v[f] += *(const f32x4*)((const float*)(block_lds + q * C::GROUP) + row * C::PITCH + n + 4 * f);
      store(row, job.n0 + n, v);
    }
    __syncthreads();  // the stages are free for the next tile
  }
}

}  // namespace ftk
