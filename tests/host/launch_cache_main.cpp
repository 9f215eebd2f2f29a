// LaunchCache against stand-ins for the runtime's calls: the blocks of a call follow its own dynamic LDS, whatever
// sizes came before it, and the kernel's limit only grows.
#include <cstdio>
#include <initializer_list>

#include "../../routed_expert_ffn_wave_amd/csrc/ft_kernels.h"

static int g_dev = 0, g_queries = 0;
static size_t g_limit[4] = {};

extern "C" {
hipError_t hipGetDevice(int* d) { return *d = g_dev, hipSuccess; }
hipError_t hipGetLastError() { return hipErrorInvalidValue; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { return *v = 256, hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int lds) {
  if ((size_t)lds < g_limit[g_dev]) std::printf("limit lowered to %d\n", lds);
  return g_limit[g_dev] = lds, hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t lds) {
  ++g_queries;
  if (lds > g_limit[g_dev]) return hipErrorInvalidValue;
  return *n = (int)(160 * 1024 / (lds + 1)), hipSuccess;
}
}

int main() {
  static ftk::LaunchCache cache;
  int bad = 0;
  auto expect = [&](size_t lds, int per_cu) {
    ftk::LaunchFacts f{};
    const hipError_t e = cache.get((const void*)&g_dev, 256, lds, &f);
    if (e != hipSuccess || f.per_cu != per_cu || f.cus != 256) {
      std::printf("device %d, %zu bytes: status %d, %d blocks, expected %d\n", g_dev, lds, (int)e, f.per_cu, per_cu);
      bad = 1;
    }
  };
  for (int dev : {0, 1, 0}) {
    g_dev = dev;
    for (size_t lds : {70000, 90000, 70000, 0, 160000, 70000, 30000, 90000})
      expect(lds, lds == 0 ? 163840 : (int)(163840 / (lds + 1)));
  }
  const int known = g_queries;
  expect(70000, 2);
  if (g_queries != known) bad = 1, std::printf("asked again for a known size\n");
  for (int pass = 0; pass < 2; ++pass) {  // a size for each of 16 batches in turn, two shapes
    const int before = g_queries;
    for (int q = 1; q <= 16; ++q) expect(1000 * q, 163840 / (1000 * q + 1)), expect(1000 * q + 500, 163840 / (1000 * q + 501));
    if (pass && g_queries != before) bad = 1, std::printf("asked again for 32 sizes\n");
  }
  for (size_t lds = 1000; lds < 60000; lds += 1000) expect(lds, (int)(163840 / (lds + 1)));  // more sizes than are kept
  expect(70000, 2);
  expect(163839, 1);
  expect(400000, 1);  // the caller's launch fails, not the count
  return bad;
}
