// The choice among the kernels of the 8-bit product.
#include <cstdio>

#include "../../routed_expert_ffn_wave_amd/csrc/fp8_choice.h"

using namespace ftk;

static int g_bad = 0;
#define EXPECT(cond, ...) ((cond) ? (void)0 : (void)(g_bad = 1, std::printf(__VA_ARGS__), std::printf("\n")))

static Fp8MatmulArgs by_expert(int P, int N, int K, int n_slots, int E) {
  Fp8MatmulArgs a{};
  a.M = P, a.N = N, a.K = K, a.n_slots = n_slots, a.E = E;
  return a;
}

// Two blocks of 64x128 share a compute unit only where its LDS holds both beside the table of experts.
static void blocks_that_fit() {
  const Choice& c = kBf16[5];
  EXPECT(c.rows == 64 && c.cols == 128 && c.per == 2, "entry 5 is not 64x128");
  for (int E = 1; E <= 1024; ++E) {
    const int fit = (int)(160 * 1024 / (c.lds + group_lds_bytes(E)));
    const double blocks = E * 32.0;  // one chunk of rows for each expert
    if (blocks <= 256) continue;
    const double rounds = cost(c, by_expert(64 * E, 4096, 2048, E, E)) / c.group;
    // one block a unit takes more than half of the time of two
    EXPECT(fit > 1 || rounds > 0.55 * blocks / 256, "%d experts: %g rounds, %d blocks a unit", E, rounds, fit);
  }
  const struct {
    int T, N, K, E, best[3];
  } measured[] = {{512, 520, 1040, 384, {7, 7, 7}}, {4096, 520, 1040, 384, {7, 8, 6}}, {4096, 520, 2048, 384, {7, 8, 6}},
                  {512, 520, 1040, 512, {7, 7, 7}}, {512, 520, 2048, 512, {7, 7, 7}}, {512, 1536, 2048, 256, {7, 7, 7}}};
  for (const auto& m : measured) {
    const int got = choose<true>(by_expert(8 * m.T, m.N, m.K, m.E, m.E));
    EXPECT(got == m.best[0] || got == m.best[1] || got == m.best[2], "%d tokens, %d experts of %d x %d: kernel %d", m.T, m.E, m.N, m.K,
           got);
  }
}

// A dense launch's threads, blocks in multiples of 8, stay under 2^32.
static void dense_launches() {
  Fp8MatmulArgs a{};
  a.K = 16, a.n_slots = 1;
  for (int tiles = (1 << 23) - 18; tiles <= (1 << 23); tiles += 2) {
    a.N = 512, a.M = (tiles / 2 - 1) * 256 + 1;  // so many tiles of the largest kernel, more of every other one
    for (int bf16 = 0; bf16 < 2; ++bf16) {
      const int got = bf16 ? choose<true>(a) : choose<false>(a);
      const bool fits = bf16 && (tiles + 7) / 8 * 8LL * T256::NT < 1LL << 32;
      EXPECT((got >= 0) == fits, "%d tiles, bf16 %d: kernel %d", tiles, bf16, got);
    }
  }
  EXPECT(launch_fits((1LL << 29) - 32, 32, 256) && !launch_fits((1LL << 29) - 31, 32, 256), "launch_fits");
}

int main() {
  blocks_that_fit();
  dense_launches();
  return g_bad;
}
