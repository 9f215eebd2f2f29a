// Shape of a tile of the 8-bit product, and what it takes of a compute unit's LDS.
#pragma once

namespace ftk {

template <int BM_, int BN_, int WM_, int WN_, int NS_, bool WIDE_, int KG_ = 1>
struct TileCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;  // NS: stages in LDS
  static constexpr bool WIDE = WIDE_;  // codes widened to bf16 (exact products), else 8-bit matrix instructions
  // KG > 1: the block is KG groups of waves, each with the whole tile, a share of K and stages of its own; their
  // results are added at the end, in the order of K.  Groups of one wave run without barriers.
  static constexpr int KG = KG_, GW = WM * WN;  // waves of a group
  static constexpr int NT = 64 * GW * KG;
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;  // fragments of a wave
  static constexpr int RQ = 8 * GW;                           // rows of one load pass (8 lanes a row)
  static constexpr int QA = BM / RQ, QB = BN / RQ;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int SBUF = NS * STAGE;         // scales of 4 steps, twice: activations [BM][4] fp32,
  static constexpr int SW = SBUF + 2 * BM * 16;  // weights [BN / 128][4] in 256 bytes
  static constexpr int GROUP = SW + 2 * 256, LDS = KG * GROUP;
  static constexpr int PITCH = BN + 4;           // floats of a row of results in LDS (KG > 1), over the stages
  static_assert(BM % RQ == 0 && BN % RQ == 0 && BM % 64 == 0 && (BM / 64 < GW || (BM == 64 && GW == 1)), "load passes");
  static_assert(KG == 1 || BM * PITCH * 4 <= GROUP, "a group's results lie over its stages");
  static_assert(NS >= 2 && NS <= 4, "the scales of 4 steps are held twice");
  static_assert(NF == 4 && 128 % (BN / WN) == 0, "a wave's 64 weight rows share one scale");
};

}  // namespace ftk
