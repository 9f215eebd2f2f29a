// Order of the tiles of a large matrix gradient: long ones first, from queues.
//
// A tile takes as many stages as its expert has rows, so that a fixed share of the list leaves most of the GPU waiting for
// the block with the largest sum.  A first kernel of one block lists the experts by classes of falling rows in a
// workspace; blocks of the second take tiles from one queue per XCD, each with a contiguous eighth of every class (tiles
// that run together share rows through its L2), and from the other XCDs' queues when theirs is empty.  Who computes a tile
// does not change it.  4096 tokens, Zipf, top 8 of 128 experts of 1536 x 2048, fp32: 393 us where the experts' order takes 432 (the
// same with even experts: 421 and 428).
#pragma once
#include "ft_device.h"
#include "ft_products.h"

namespace ftk {

constexpr int kClasses = 8, kQueues = 8;
constexpr int kPlanThreads = 1024;

// An expert's rows.
struct alignas(16) PlanPart {
  int expert, row0, rows, pad;
};

struct Plan {
  int32_t ctr[kQueues][16];     // tiles taken from each queue, a cache line each
  int32_t parts, pad[3];
  int32_t first[kClasses + 4];  // first tile of each class; first[kClasses]: number of tiles
  PlanPart part[1];             // up to E, by class
};
constexpr size_t plan_bytes(int E) { return sizeof(Plan) + (size_t)E * sizeof(PlanPart); }

__device__ __forceinline__ bool group_of(const RowGroups& s, int e, int& slot, int& row0, int& cnt) {
  slot = s.slot_of ? s.slot_of[e] : e;
  row0 = min(max(s.offsets[e], 0), s.P);
  cnt = max(min(max(s.offsets[e + 1], 0), s.P) - row0, 0);
  return (uint32_t)slot < s.n_slots;
}

// Classes of experts with more than 2048, 1024, ... 64 rows, and the rest; `tiles` of each.
static __global__ __launch_bounds__(kPlanThreads) void plan_kernel(RowGroups s, int tiles, Plan* plan) {
  constexpr int W = kPlanThreads / 64;
  __shared__ int s_parts[kClasses][W + 1];
  const int e = threadIdx.x, lane = e & 63, wv = e >> 6;
  if (e < kQueues) plan->ctr[e][0] = 0;
  int cls = -1, slot, row0 = 0, cnt = 0;
  if (e < s.E && group_of(s, e, slot, row0, cnt)) {
    cls = 0;
    for (int c = 2048; c >= 64 && cnt <= c; c >>= 1) ++cls;
  }
  int at[kClasses];  // experts of each class up to and with this one, in its wave
#pragma unroll
  for (int c = 0; c < kClasses; ++c) {
    at[c] = wave_incl_scan(cls == c);
    if (lane == 63) s_parts[c][wv] = at[c];
  }
  __syncthreads();
  if (wv == 0) {  // lane c: the waves' sums of a class, then the classes' own
    const int c = min(lane, kClasses - 1);
    int p = 0;
    for (int w = 0; w < W; ++w) {
      const int v = s_parts[c][w];
      if (lane < kClasses) s_parts[c][w] = p;
      p += v;
    }
    const int before = wave_incl_scan(lane < kClasses ? p : 0) - (lane < kClasses ? p : 0);
    if (lane < kClasses) s_parts[c][W] = before;
    if (lane <= kClasses) plan->first[lane] = before * tiles;
    if (lane == kClasses) plan->parts = before;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kClasses; ++c)
    if (cls == c) {
      const int p = s_parts[c][W] + s_parts[c][wv] + at[c] - 1;
      plan->part[p] = PlanPart{e, row0, cnt, 0};
    }
}

// A block's view of a plan.
struct PlanQueue {
  Plan* plan;
  int* first;  // first tile of each class, in LDS
  int queue, tried;

  // Thread 0: asks for a tile of the current queue; the answer may be used later.
  __device__ __forceinline__ int ask() { return __hip_atomic_fetch_add(&plan->ctr[queue][0], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
  // This queue's share of class c: its first tile and their number.
  __device__ __forceinline__ int share(int c, int& lo) const {
    const long long n = first[c + 1] - first[c];
    lo = first[c] + (int)(n * queue / kQueues);
    return first[c] + (int)(n * (queue + 1) / kQueues) - lo;
  }
  // Thread 0: the tile that the answer stands for, or -1 when every queue is empty.
  __device__ __forceinline__ int take(int answer) {
    for (;;) {
      int all = 0, lo;
      for (int c = 0; c < kClasses; ++c) all += share(c, lo);
      if (answer < all)
        for (int c = 0;; ++c) {
          const int len = share(c, lo);
          if (answer < len) return lo + answer;
          answer -= len;
        }
      if (++tried == kQueues) return -1;
      queue = (queue + 1) % kQueues;
      answer = ask();
    }
  }
};

// run(part, local, next) for every tile that this block takes.  The next tile is asked for before one is computed, and run
// calls next() between its last load and its first store: the answer is not waited for behind the stores.
template <class Run>
__device__ __forceinline__ void run_plan(Plan* plan, int tiles, Run run) {
  __shared__ int s_item[2], s_first[kClasses + 1];
  PlanQueue q{plan, s_first, (int)(blockIdx.x % kQueues), 0};
  if (threadIdx.x <= kClasses) s_first[threadIdx.x] = plan->first[threadIdx.x];
  __syncthreads();
  if (threadIdx.x == 0) s_item[0] = q.take(q.ask());
  __syncthreads();
  for (int turn = 0;; turn ^= 1) {
    const int item = __builtin_amdgcn_readfirstlane(s_item[turn]);
    if (item < 0) return;
    int answer = 0;
    if (threadIdx.x == 0) answer = q.ask();
    const PlanPart* part = plan->part + item / tiles;
    run(PlanPart{__builtin_amdgcn_readfirstlane(part->expert), __builtin_amdgcn_readfirstlane(part->row0), __builtin_amdgcn_readfirstlane(part->rows), 0},
        item % tiles, [&] {
          if (threadIdx.x == 0) s_item[turn ^ 1] = q.take(answer);
        });
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

}  // namespace ftk
