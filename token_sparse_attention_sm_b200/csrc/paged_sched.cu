// paged_sched.cu -- the schedule of a paged attention call, from the lengths
// on the device.
//
// The rows of sequence b form nrb = ceil(n / TB) blocks, each reading up to
// u key tiles; with few blocks the key range of every block is cut into np
// pieces of `len` tiles whose partial results are merged.  The pieces of all
// blocks of a sequence share their boundaries, so the workers that run them
// at the same time read the same K and V tiles from L2.
//
// A piece length serves the whole batch.  32 warps weigh one candidate each
// (the longest range cut into 1 .. 192 pieces): pieces per head P =
// sum nrb * np, waves = ceil(P * Hkv / workers), cost = waves * (longest
// piece + a fixed part for starting a piece and, when cut, for writing and
// merging its partial: the caller's, in quarters of a tile).  The cheapest whose
// partials fit the workspace wins; ties go to fewer pieces.  One CTA; latency bound (it also sets the call's
// claim counter, which needs no value before a call).
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kScThreads = 1024;
constexpr int kCand = 32;
__constant__ int kPieces[kCand] = {1,  2,  3,  4,  5,  6,  7,  8,  9,  10, 11,  12,  13,  14,  15,  16,
                                   18, 20, 22, 24, 28, 32, 37, 42, 49, 56, 64, 74, 96, 112, 148, 192};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// blocks of a sequence's rows, and the most key tiles that one of them reads
__device__ __forceinline__ int sc_blocks(const PgArgs &a, int b, int TB, int KT, int *u,
                                         bool report) {
  int row0, n, kv;
  *u = 1;
  if (!pg_lengths(a, b, &row0, &n, &kv)) {
    if (report) raise_flag(a.status, FLAG_INDEX);
    return 0;
  }
  const int nrb = ceil_div(n, TB);
  if (nrb > 0) {
    // the last block sees the most keys; a window bounds every block
    int x = pg_tiles(kv - n + (nrb - 1) * TB, kv - 1, a.window, a.sinks, KT).units();
    if (a.window > 0 && nrb > 1)
      x = min(ceil_div(kv, KT), ceil_div(min(a.sinks, kv), KT) +
                                    (int)(((long long)a.window + TB - 2) / KT) + 2);
    *u = max(x, 1);
  }
  return nrb;
}

// Every warp walks the batch itself, so the candidates meet at one barrier.
__global__ void __launch_bounds__(kScThreads) paged_schedule_kernel(const PgArgs a, int TB, int KT,
                                                                    int workers, int whole_cost,
                                                                    int cut_cost) {
  __shared__ unsigned long long s_cost[kCand];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) a.head->next = (uint32_t)workers;  // a worker's first item is its own number
  // the first 32 sequences' blocks and tiles stay in registers
  int umax = 1, u0 = 1;
  const int nrb0 = lane < a.B ? sc_blocks(a, lane, TB, KT, &u0, warp == 0) : 0;
  if (nrb0) umax = max(umax, u0);
  for (int b = lane + 32; b < a.B; b += 32) {
    int u;
    if (sc_blocks(a, b, TB, KT, &u, warp == 0)) umax = max(umax, u);
  }
  auto blocks = [&](int b, int *u) {
    if (b < 32) {
      *u = u0;
      return nrb0;
    }
    return sc_blocks(a, b, TB, KT, u, false);
  };
  umax = __reduce_max_sync(0xffffffffu, umax);
  {
    // this warp's candidate
    const int C = ceil_div(umax, kPieces[warp]);
    long long pieces = 0, slots = 0;
    int longest = 1, cut = 0;
    for (int b = lane; b < a.B; b += 32) {
      int u;
      const int nrb = blocks(b, &u);
      if (!nrb) continue;
      const int np = ceil_div(u, C);
      pieces += (long long)nrb * np;
      if (np > 1) slots += (long long)nrb * np, cut = 1;
      longest = max(longest, ceil_div(u, np));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      pieces += __shfl_xor_sync(0xffffffffu, pieces, o);
      slots += __shfl_xor_sync(0xffffffffu, slots, o);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    cut = __reduce_or_sync(0xffffffffu, cut);
    if (lane == 0) {
      const unsigned long long waves =
          ((unsigned long long)pieces * a.Hkv + workers - 1) / workers;
      s_cost[warp] = slots <= a.slot_cap
                         ? waves * (unsigned)(4 * longest + (cut ? cut_cost : whole_cost))
                         : ~0ull;
    }
  }
  __syncthreads();
  if (warp > 0) return;
  // the cheapest (one piece needs no slot: always possible)
  unsigned long long cost = s_cost[lane];
  int best = lane;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long c = __shfl_xor_sync(0xffffffffu, cost, o);
    const int i = __shfl_xor_sync(0xffffffffu, best, o);
    if (c < cost || (c == cost && i < best)) cost = c, best = i;
  }
  const int C = ceil_div(umax, kPieces[best]);
  // exclusive prefix sums of items and slots
  int bx = 0, by = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int np = 1, len = 1, items = 0, slots = 0;
    if (b < a.B) {
      int u;
      const int nrb = blocks(b, &u);
      np = ceil_div(u, C);
      len = ceil_div(u, np);
      items = nrb * np;
      slots = np > 1 ? items : 0;
    }
    int x = items, y = slots;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int px = __shfl_up_sync(0xffffffffu, x, o), py = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += px, y += py;
    }
    if (b < a.B) a.seqs[b] = PgSeq{bx + x - items, by + y - slots, np, len};
    bx += __shfl_sync(0xffffffffu, x, 31);
    by += __shfl_sync(0xffffffffu, y, 31);
  }
  if (lane == 0) a.seqs[a.B] = PgSeq{bx, by, 1, 1};
}

}  // namespace

cudaError_t launch_paged_schedule(const PagedShape &, const PgArgs &a, int tb, int kt, int grid,
                                  int whole_cost, int cut_cost, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kScThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  cfg.attrs = attrs;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  return cudaLaunchKernelEx(&cfg, paged_schedule_kernel, a, tb, kt, grid, whole_cost,
                            cut_cost);
}

}  // namespace sd
