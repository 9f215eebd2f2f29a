// Which kernel takes a product of 8-bit rows: a model of host code alone, from sizes.
#pragma once
#include <algorithm>
#include <cmath>

#include "fp8_tile_cfg.h"
#include "ft_group_lds.h"
#include "ft_rows.h"

namespace ftk {

// Which kernel: the one whose blocks, taken in rounds of the 256 compute units (or as many times that as fit),
// are through first.  `step` stands for the time of one 128-block of K in a round, in us on an MI355X; `full`
// where rounds follow each other.  The constants are fitted to the times below, so that the fastest kernel there has the least
// cost: only their order within a list counts (the 16x32 kernel has 0.26 beside the bf16 kernels by expert and 0.19 beside the
// fp32 ones, and takes the same time).  By expert, over 800 measured sizes (4 to 256 experts, N of 256 to 4096, K of 256
// to 7168, 1 to 4096 tokens) the kernel chosen takes 7 % more time than the fastest on average, and over 15 % more at every
// sixth size.  M rows x 4096 columns, K = 7168, us a call (bf16 results; / 2, / 4: that many shares of K):
//   M             16     32     64     128    256    512    1024   2048   4096   8192
//   16x16         10.2   18.3   34     65     -      -      -      -      -      -
//   16x32         14.0   13.4   24     46     88     -      -      -      -      -
//   64x64 / 4     15.3   15.1   16.1   18.5   19.3   34.8   67     131    261    533
//   64x128 / 2    -      -      25     25     26     27     50     98     194    -
//   128x128 / 2   -      -      -      36     36     36     38     75     147    -
//   128x256       -      47     48     49     49     50     50     60     117    263 - 311
//   256x256       -      -      -      71     74     75     75     79     99     206 - 249
// and fp32 results:
//   16x32         -      -      -      -      88     -      -      -      -      -
//   64x64 / 4     -      -      20     21     23     44     81     153    -      -
//   128x128 / 2   -      -      53     55     56     58     62     121    -      -
//   128x128       -      -      64     65     67     71     72     117    -      434 - 505
// A block alone on its compute unit waits for its loads: two shares of K, each with stages and waves of its own, keep twice as many in
// flight (64x128 and 128x128 without: 41 and 45 at 256 rows).  By expert, where tiles follow each other, the unshared
// ones serve better (64 tokens below: 74 us for 64x128 against 83 with shares).
//
// By expert, `group` where rounds follow each other, `light` where a group fills half a tile or less (waves
// without rows wait only; bound by the weights' bytes).  us for T tokens, top 8:
//   128 experts of 1536 x 2048, T =  4      16     64     256    1024     256 experts, 96 held, of 4096 x 7168, T =  64     256    1024   8192
//   16x32                            21.4   50.7   83     125    362                                                 427    549    1430   -
//   64x64 / 4                        25     63     102    105    149                                                 504    552    588    -
//   64x128                           20.9   43.6   74     77     104                                                 433    471    509    1747
//   128x128                          28.8   54.2   85     87     98                                                  437    484    497    1331
//   128x256                          18.9   42.7   75     78     90                                                  428    464    482    1066
//   256x256                          23.3   52.7   89     90     101                                                 530    558    578    1062
// and fp32 results:
//   16x32                            21.5   49.8   82     122    362                                                 427    552    1433   -
//   64x64 / 4                        29.5   70.3   108    110    160                                                 512    574    620    -
//   128x128                          32.9   60.3   92     94     109                                                 573    590    607    1880
//   128x256                          24.4   46.5   80     85     112                                                 466    493    515    1765
struct Choice {
  int rows, cols, per;
  float step, full, group, light;
  int lds;  // of the tiles kernels, 0 for the others
  float many;  // > 0: a round of one block a unit from kManyExperts on
};
using Solo = TileCfg<64, 64, 1, 1, 2, false, 4>;
using SoloWide = TileCfg<64, 64, 1, 1, 2, true, 4>;
using Pair64 = TileCfg<64, 128, 1, 2, 3, false, 2>;    // dense only, as kNever says
using Pair128 = TileCfg<128, 128, 2, 2, 2, false, 2>;  // dense only
using PairWide = TileCfg<128, 128, 2, 2, 2, true, 2>;  // dense only
using T64 = TileCfg<64, 128, 1, 2, 3, false>;          // by expert only
using T128 = TileCfg<128, 128, 2, 2, 4, false>;        // by expert only
using T128x256 = TileCfg<128, 256, 2, 4, 3, false>;
using T256 = TileCfg<256, 256, 2, 4, 2, false>;
using TWide = TileCfg<128, 128, 2, 2, 2, true>;
using TWide256 = TileCfg<128, 256, 2, 4, 3, true>;  // by expert only
constexpr int kLds = 160 * 1024;  // of a compute unit
// From 350 experts on their table leaves room for one 64x128 block where two fit beside fewer.  256 blocks alone took 0.92 - 1.0 us
// a step, half of 512 two by two 0.66 - 0.77, 256 64x64 blocks of as many experts 0.54 - 0.6: `many`, to the scale of the
// constants they stand beside.  512 tokens, top 8 of 384 experts of 520 x 1040: 55 us with 128x256, chosen so, against 75 for
// 64x128; 4096 tokens 94 with 128x128 against 144; over 280 sizes of 384 to 1024 experts 2 % less time, none slower.  (fp32 128x128
// fits once from 735 experts on; counting that chose slower kernels for 768 and 1024 experts, 2 % more time over 130 sizes.)
constexpr int many_experts() {
  int E = 1;
  while (2 * (T64::LDS + group_lds_bytes(E)) <= kLds) ++E;
  return E;
}
constexpr int kManyExperts = many_experts();
constexpr float kNever = 1e30f;
constexpr Choice kBf16[] = {{16, 16, 1, 0.18f, 0.18f, 0.18f, 0.18f, 0},
                            {16, 32, 1, 0.26f, 0.26f, 0.26f, 0.26f, 0},
                            {64, 64, 1, 0.33f, 0.31f, 0.32f, 0.32f, Solo::LDS, 0.4f},
                            {64, 128, 1, 0.48f, 0.44f, kNever, kNever, Pair64::LDS},
                            {128, 128, 1, 0.66f, 0.66f, kNever, kNever, Pair128::LDS},
                            {64, 128, 2, 0.71f, kNever, 0.95f, 0.95f, T64::LDS, 0.57f},
                            {128, 128, 1, 0.78f, kNever, 0.82f, 0.82f, T128::LDS},
                            {128, 256, 1, 0.93f, 1.15f, 1.25f, 0.85f, T128x256::LDS},
                            {256, 256, 1, 1.4f, 2.0f, 2.2f, 2.2f, T256::LDS}};
constexpr Choice kF32[] = {{16, 16, 1, 0.18f, 0.18f, 0.18f, 0.18f, 0},
                           {16, 32, 1, 0.26f, 0.26f, 0.19f, 0.19f, 0},
                           {64, 64, 1, 0.37f, 0.36f, 0.5f, 0.46f, SoloWide::LDS},
                           {128, 128, 1, 1.05f, 1.08f, kNever, kNever, PairWide::LDS},
                           {128, 128, 2, 1.2f, 2.0f, 2.15f, 1.7f, TWide::LDS},
                           {128, 256, 1, 1.5f, kNever, 1.95f, 1.45f, TWide256::LDS}};

// Rows with a slot and groups that have any, where only the device knows: as if experts were drawn evenly.
struct Spread {
  double rows, groups;
};
inline Spread spread(const Fp8MatmulArgs& a) {
  const double held = std::min(1.0, (double)a.n_slots / a.E);
  return {std::max(1.0, held * a.M), std::max(1.0, held * a.E * (1.0 - std::exp(-(double)a.M / a.E)))};
}

inline double cost(const Choice& c, const Fp8MatmulArgs& a) {
  if (c.lds + (a.E > 0 ? group_lds_bytes(a.E) : 0) > kLds) return kNever;
  // Counts that have to fit: the threads of a dense launch (at most 512 a block, blocks in multiples of 8) in 32 bits, the
  // tiles of all groups in an int whatever the table holds (one that does not ascend can give all rows to every second
  // expert).
  const double ntn = (a.N + c.cols - 1) / c.cols;
  if (a.E == 0 ? ((a.M + c.rows - 1) / c.rows) * ntn > (1 << 23) - 8
               : (a.M / c.rows + 2.0) * (a.E / 2 + 1) * ntn >= 2147483648.0)
    return kNever;
  double chunks = (a.M + c.rows - 1) / c.rows, round = c.full;
  int per = c.per;
  if (a.E > 0) {  // each group has half a chunk to spare
    const Spread p = spread(a);
    chunks = std::max(p.groups, p.rows / c.rows + 0.5 * p.groups);
    round = 2 * p.rows <= c.rows * p.groups ? c.light : c.group;
    if (a.E >= kManyExperts && c.many > 0) round = c.many, per = 1;
  }
  const double blocks = chunks * ntn;
  return blocks <= 256 && round < kNever ? c.step : std::ceil(blocks / (256.0 * per)) * round;
}

// -1: none fits
template <bool BF16>
int choose(const Fp8MatmulArgs& a) {
  const Choice* c = BF16 ? kBf16 : kF32;
  // A few rows a group: bound by the weights' bytes, and with long rows 16 x 32 blocks stream them fastest (top 8 of
  // 256 experts, 96 resident, K = 7168, 16 / 32 tokens: 176 - 198 / 281 us, 5.9 TB/s; 64 x 128 tiles 207 / 293,
  // 64 x 64 210; with K = 2048 and 4 / 16 tokens 21 / 52 us against 20 / 44 for 64 x 128; where between the two lengths
  // the border lies was not measured)
  if (a.E > 0 && a.K >= 4096) {
    const Spread p = spread(a);
    if (p.rows <= 3 * p.groups && cost(c[1], a) < kNever) return 1;
  }
  const int n = BF16 ? sizeof(kBf16) / sizeof(Choice) : sizeof(kF32) / sizeof(Choice);
  int best = 0;
  for (int i = 1; i < n; ++i)
    if (cost(c[i], a) < cost(c[best], a)) best = i;
  return cost(c[best], a) < kNever ? best : -1;
}

}  // namespace ftk
