// Launch interface of the bf16 products by expert, SwiGLU rows and low-rank adapters.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ftk {

// Rows of expert e: offsets[e] .. offsets[e+1] - 1, clipped to [0, P); its matrix: slot_of[e], or e where slot_of is null.
struct RowGroups {
  const int32_t* offsets;  // [E+1]
  const int32_t* slot_of;  // [E] or null
  int E, P;
  uint32_t n_slots;  // slots outside [0, n_slots) name no matrix
};

// kind 0: out[P][N] = a[P][K] w^T; 1: out[P][K] = a[P][N] w (the rows' gradient); w [n_slots][N][K]
struct GroupedArgs {
  RowGroups g;
  const uint16_t *a, *w;
  int N, K;
  void* out;
  bool out_bf16;
};
hipError_t launch_grouped(int kind, const GroupedArgs& a, hipStream_t s);

// dw[E][N][K] = dout[P][N]^T a[P][K] by expert, or += with add (fp32)
struct WgradArgs {
  RowGroups g;
  const uint16_t *dout, *a;
  int N, K;
  void* dw;
  bool out_bf16, add;
  void* ws;
};
size_t wgrad_workspace(int N, int K, int E);  // bytes of ws (0: none is needed)
hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s);

// h[rows][I] = SiLU(g) u of gu[rows][2 I]; with dh: out[rows][2 I] = its gradient
hipError_t launch_swiglu(const uint16_t* gu, const uint16_t* dh, long long rows, int I, uint16_t* out, hipStream_t s);

// out[t] = base[t] + scale (x[t] a^T) b^T by adapter
struct LoraArgs {
  RowGroups g;            // groups of positions of `gather`, P = T
  const int32_t* gather;  // [T]
  const uint16_t *x, *a, *b;
  const float* scale;  // [n_slots] or null
  const void* base;
  void* out;
  int r, N, K;
  bool bf16;  // base and out
  float* ws;  // [splits][T][r]
};
int lora_splits(int T, int E, int r, int N, int K);  // 0: the call needs no ws
hipError_t launch_lora(const LoraArgs& a, hipStream_t s);

}  // namespace ftk
