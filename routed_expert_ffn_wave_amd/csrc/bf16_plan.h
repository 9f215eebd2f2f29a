// Order of the tiles of a large product: expensive ones first, from queues.
//
// Tiles differ by up to five times in time (64 to 256 rows; matrix gradients by their expert's rows), and a block takes a few of
// them, so that a fixed share of the list leaves most of the GPU waiting for the block with the largest sum.  A first kernel of
// one block lists the tiles by classes of falling cost in a workspace; blocks of the second take them from one queue
// per XCD, each with a contiguous eighth of every class (tiles that run together share rows and matrices through their L2),
// and from the other XCDs' queues when theirs is empty.  Who computes a tile does not change it.
// 4096 tokens, Zipf, top 8 of 128 experts of 1536 x 2048, fixed shares / queues: see the kernels.
#pragma once
#include "ft_device.h"
#include "ft_products.h"

namespace ftk {

constexpr int kClasses = 8, kQueues = 8;
constexpr int kPlanThreads = 1024;

// A run of tiles of one expert and class: rows first .. first + rows - 1 of the expert's, from row0 on.
struct alignas(16) PlanPart {
  int slot, row0, rows, item0;  // slot: of the matrix (matrix gradients: the expert); item0: its first tile's number
};

struct Plan {
  int32_t ctr[kQueues][16];     // tiles taken from each queue, a cache line each
  int32_t parts, pad[3];
  int32_t first[kClasses + 4];  // first tile of each class; first[kClasses]: number of tiles
  PlanPart part[1];             // up to 2 E, by class
};
constexpr size_t plan_bytes(int E) { return sizeof(Plan) + (size_t)2 * E * sizeof(PlanPart); }

__device__ __forceinline__ bool group_of(const RowGroups& s, int e, int& slot, int& row0, int& cnt) {
  slot = s.slot_of ? s.slot_of[e] : e;
  row0 = min(max(s.offsets[e], 0), s.P);
  cnt = max(min(max(s.offsets[e + 1], 0), s.P) - row0, 0);
  return (uint32_t)slot < s.n_slots;
}

// parts_of(slot, e, row0, cnt, cls, tiles, part): up to two parts of an expert that has a slot; cls -1: none.
template <class PartsOf>
__device__ __forceinline__ void make_plan(const RowGroups& s, Plan* plan, PartsOf parts_of) {
  constexpr int W = kPlanThreads / 64;
  __shared__ int s_tiles[kClasses][W + 1], s_parts[kClasses][W + 1];
  const int e = threadIdx.x, lane = e & 63, wv = e >> 6;
  if (e < kQueues) plan->ctr[e][0] = 0;
  int cls[2] = {-1, -1}, tiles[2] = {0, 0};
  PlanPart part[2] = {};
  int slot, row0, cnt;
  if (e < s.E && group_of(s, e, slot, row0, cnt)) parts_of(slot, e, row0, cnt, cls, tiles, part);
  int ti[kClasses], pi[kClasses];  // sums up to and with this thread's, by class
#pragma unroll
  for (int c = 0; c < kClasses; ++c) {
    ti[c] = wave_incl_scan((cls[0] == c ? tiles[0] : 0) + (cls[1] == c ? tiles[1] : 0));
    pi[c] = wave_incl_scan((cls[0] == c) + (cls[1] == c));
    if (lane == 63) s_tiles[c][wv] = ti[c], s_parts[c][wv] = pi[c];
  }
  __syncthreads();
  if (wv == 0) {  // lane c: the waves' sums of a class, then the classes' own
    const int c = min(lane, kClasses - 1);
    int t = 0, p = 0;
    for (int w = 0; w < W; ++w) {
      const int vt = s_tiles[c][w], vp = s_parts[c][w];
      if (lane < kClasses) s_tiles[c][w] = t, s_parts[c][w] = p;
      t += vt, p += vp;
    }
    const int tt = wave_incl_scan(lane < kClasses ? t : 0) - (lane < kClasses ? t : 0);
    const int pp = wave_incl_scan(lane < kClasses ? p : 0) - (lane < kClasses ? p : 0);
    if (lane < kClasses) s_tiles[c][W] = tt, s_parts[c][W] = pp;
    if (lane <= kClasses) plan->first[lane] = tt;
    if (lane == kClasses) plan->parts = pp;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kClasses; ++c) {
    int t = s_tiles[c][W] + s_tiles[c][wv] + ti[c], p = s_parts[c][W] + s_parts[c][wv] + pi[c];
#pragma unroll
    for (int q = 1; q >= 0; --q)
      if (cls[q] == c) {
        t -= tiles[q], --p;
        part[q].item0 = t;
        plan->part[p] = part[q];
      }
  }
}

// A block's view of a plan; in LDS: the first tile of all parts (2 E ints) and of the classes.
struct PlanQueue {
  Plan* plan;
  int* item0;
  int* first;
  int queue, tried;

  __device__ __forceinline__ void open(Plan* p, int* lds, int* lds_first) {
    plan = p, item0 = lds, first = lds_first;
    queue = blockIdx.x % kQueues, tried = 0;
    for (int i = threadIdx.x; i < p->parts; i += blockDim.x) item0[i] = p->part[i].item0;
    if (threadIdx.x <= kClasses) first[threadIdx.x] = p->first[threadIdx.x];
  }
  // Thread 0: asks for a tile of the current queue; the answer may be used later.
  __device__ __forceinline__ int ask() { return __hip_atomic_fetch_add(&plan->ctr[queue][0], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
  // This queue's share of class c: its first tile and their number.
  __device__ __forceinline__ int share(int c, int& lo) const {
    const long long n = first[c + 1] - first[c];
    lo = first[c] + (int)(n * queue / kQueues);
    return first[c] + (int)(n * (queue + 1) / kQueues) - lo;
  }
  // Thread 0: the tile that the answer stands for, or -1 when every queue is empty.  Answers go to the two ends of a queue in
  // turn: tiles bound by the matrix cores and tiles bound by memory run beside each other.
  __device__ __forceinline__ int take(int answer) {
    for (;;) {
      int all = 0, lo;
      for (int c = 0; c < kClasses; ++c) all += share(c, lo);
      if (answer < all) {
        int q = answer;
        for (int c = 0;; ++c) {
          const int len = share(c, lo);
          if (q < len) return lo + q;
          q -= len;
        }
      }
      if (++tried == kQueues) return -1;
      queue = (queue + 1) % kQueues;
      answer = ask();
    }
  }
  // The part that holds a tile.
  __device__ __forceinline__ int find(int item) const {
    int lo = 0, hi = plan->parts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (item0[mid] <= item)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

// run(part, local, next) for every tile that this block takes.  The next tile is asked for before one is computed, and run
// calls next() between its last load and its first store: the answer is not waited for behind the stores.
template <class Run>
__device__ __forceinline__ void run_plan(Plan* plan, int* lds, Run run) {
  __shared__ int s_item[2], s_first[kClasses + 1];
  PlanQueue q;
  q.open(plan, lds, s_first);
  __syncthreads();
  if (threadIdx.x == 0) s_item[0] = q.take(q.ask());
  __syncthreads();
  for (int turn = 0;; turn ^= 1) {
    const int item = __builtin_amdgcn_readfirstlane(s_item[turn]);
    if (item < 0) return;
    int answer = 0;
    if (threadIdx.x == 0) answer = q.ask();
    const PlanPart* part = plan->part + __builtin_amdgcn_readfirstlane(q.find(item));
    run(PlanPart{__builtin_amdgcn_readfirstlane(part->slot), __builtin_amdgcn_readfirstlane(part->row0), __builtin_amdgcn_readfirstlane(part->rows), 0},
        item - __builtin_amdgcn_readfirstlane(part->item0), [&] {
          if (threadIdx.x == 0) s_item[turn ^ 1] = q.take(answer);
        });
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

}  // namespace ftk
