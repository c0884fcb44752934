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
// merging its partial).  The cheapest whose partials fit the workspace wins;
// ties go to fewer pieces.  One CTA; latency bound (it also resets the call's
// counters, so nothing in the workspace has to be zero before a call).
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kScThreads = 1024;
constexpr int kCand = 32;
__constant__ int kPieces[kCand] = {1,  2,  3,  4,  5,  6,  7,  8,  9,  10, 11,  12,  13,  14,  15,  16,
                                   18, 20, 22, 24, 28, 32, 37, 42, 49, 56, 64, 74, 96, 112, 148, 192};
// in key tiles: what a piece costs besides its tiles, whole and cut
constexpr int kPieceCost = 2, kCutCost = 8;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__global__ void __launch_bounds__(kScThreads) paged_schedule_kernel(const PgArgs a, int TB, int KT,
                                                                    int workers) {
  __shared__ int s_nrb[kPagedMaxB], s_u[kPagedMaxB];
  __shared__ int s_max, s_best;
  __shared__ unsigned long long s_cost[kCand];
  __shared__ int s_w[kScThreads / 32][2], s_carry[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) {
    s_max = 1;
    s_carry[0] = s_carry[1] = 0;
    a.head->next = 0;
  }
  __syncthreads();
  int most = 1;
  for (int b = tid; b < a.B; b += kScThreads) {
    int row0, n, kv, nrb = 0, u = 1;
    if (pg_lengths(a, b, &row0, &n, &kv)) {
      nrb = ceil_div(n, TB);
      if (nrb > 0) {
        // the last block sees the most keys; a window bounds every block
        const PgTiles last = pg_tiles(kv - n + (nrb - 1) * TB, kv - 1, a.window, a.sinks, KT);
        u = last.units();
        if (a.window > 0 && nrb > 1)
          u = min(ceil_div(kv, KT), ceil_div(min(a.sinks, kv), KT) +
                                        (int)(((long long)a.window + TB - 2) / KT) + 2);
        u = max(u, 1);
      }
    } else {
      raise_flag(a.status, FLAG_INDEX);
    }
    s_nrb[b] = nrb;
    s_u[b] = u;
    if (nrb) most = max(most, u);
  }
  atomicMax(&s_max, most);
  __syncthreads();
  const int umax = s_max;
  {
    // this warp's candidate
    const int C = ceil_div(umax, kPieces[warp]);
    long long pieces = 0, slots = 0;
    int longest = 1, cut = 0;
    for (int b = lane; b < a.B; b += 32) {
      const int np = ceil_div(s_u[b], C);
      if (!s_nrb[b]) continue;
      pieces += (long long)s_nrb[b] * np;
      if (np > 1) slots += (long long)s_nrb[b] * np, cut = 1;
      longest = max(longest, ceil_div(s_u[b], np));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      pieces += __shfl_xor_sync(0xffffffffu, pieces, o);
      slots += __shfl_xor_sync(0xffffffffu, slots, o);
      longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
      cut |= __shfl_xor_sync(0xffffffffu, cut, o);
    }
    if (lane == 0) {
      const unsigned long long waves =
          ((unsigned long long)pieces * a.Hkv + workers - 1) / workers;
      s_cost[warp] = slots <= a.slot_cap
                         ? waves * (unsigned)(longest + (cut ? kCutCost : kPieceCost))
                         : ~0ull;
    }
  }
  __syncthreads();
  if (tid == 0) {
    int best = 0;  // one piece needs no slot: always possible
    for (int i = 1; i < kCand; ++i)
      if (s_cost[i] < s_cost[best]) best = i;
    s_best = ceil_div(umax, kPieces[best]);
  }
  __syncthreads();
  const int C = s_best;
  // exclusive prefix sums of items and slots, kScThreads sequences at a time
  for (int b0 = 0; b0 < a.B; b0 += kScThreads) {
    const int b = b0 + tid;
    int np = 1, len = 1, items = 0, slots = 0;
    if (b < a.B) {
      np = ceil_div(s_u[b], C);
      len = ceil_div(s_u[b], np);
      items = s_nrb[b] * np;
      slots = np > 1 ? items : 0;
    }
    int x = items, y = slots;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int px = __shfl_up_sync(0xffffffffu, x, o), py = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += px, y += py;
    }
    if (lane == 31) s_w[warp][0] = x, s_w[warp][1] = y;
    __syncthreads();
    int bx = s_carry[0], by = s_carry[1];
    for (int w = 0; w < warp; ++w) bx += s_w[w][0], by += s_w[w][1];
    if (b < a.B) a.seqs[b] = PgSeq{bx + x - items, by + y - slots, np, len};
    __syncthreads();
    if (tid == kScThreads - 1) s_carry[0] = bx + x, s_carry[1] = by + y;
    __syncthreads();
  }
  if (tid == 0) a.seqs[a.B] = PgSeq{s_carry[0], s_carry[1], 1, 1};
  for (int i = tid; i < a.slot_cap * a.Hkv; i += kScThreads) a.arrive[i] = 0u;
}

}  // namespace

cudaError_t launch_paged_schedule(const PagedShape &, const PgArgs &a, int tb, int kt, int grid,
                                  cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kScThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  cfg.attrs = attrs;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  return cudaLaunchKernelEx(&cfg, paged_schedule_kernel, a, tb, kt, grid);
}

}  // namespace sd
