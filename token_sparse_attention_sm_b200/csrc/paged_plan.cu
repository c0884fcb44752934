// paged_plan.cu -- the block tables and slot map of one batch step, from the
// requests' lengths.
//
// Sequence b with lens[b] = c cached tokens and n = new_lens[b] new ones needs
// ceil((c+n)/page) - ceil(c/page) more pages; the pages of the batch are taken
// from the end of the free list, sequences in order, blocks in order.  New
// token i of sequence b is row q_start[b] + i, stands at position c + i and
// goes to slot page_id * page + position % page.
//
// Two exclusive prefix sums over the batch (rows, pages) give everything; the
// rest is a search per token and independent loads, so the kernel is bound by
// latency.  One cluster: every CTA computes the sums itself (B <= 4096, in
// shared memory), one cluster barrier separates the last read of lens and
// free_count from the first write, so the results may replace them in place,
// and the CTAs share the writes.  A batch that does not fit (rows, pages or
// table columns) is refused as a whole: nothing is taken or appended.
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kPlThreads = 512;
constexpr int kPlCluster = 16;  // CTAs of the largest cluster (opt-in size)
constexpr int kPlRows = 4;      // rows a thread has in flight

struct PlanArgs {
  const int *new_lens, *lens, *free_pages, *free_count;
  int *table, *kv_lens, *q_start, *positions, *slots, *free_left;
  int B, T, page, pages, blocks, F;
  uint32_t *status;
};

// last b with pre[b] <= x
__device__ __forceinline__ int find_seq(const int *pre, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlThreads) paged_plan_kernel(const PlanArgs a) {
  extern __shared__ int sm[];
  int *rows = sm, *take = rows + a.B + 1, *past = take + a.B + 1;
  __shared__ long long s_w[kPlThreads / 32][2], s_carry[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int CL = (int)gridDim.x, rank = (int)blockIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) s_carry[0] = s_carry[1] = 0;
  __syncthreads();
  const int fc = *a.free_count;
  bool bad = false, full = false;
  for (int b0 = 0; b0 < a.B; b0 += kPlThreads) {
    const int b = b0 + tid;
    long long n = 0, need = 0;
    if (b < a.B) {
      const int nn = a.new_lens[b], c = a.lens[b];
      const long long end = (long long)nn + c;
      if (nn < 0 || c < 0) {
        bad = true;
      } else if (end > (long long)a.blocks * a.page) {
        full = true;
      } else {
        n = nn;
        need = (end + a.page - 1) / a.page - ((long long)c + a.page - 1) / a.page;
      }
      past[b] = c;
    }
    long long x = n, y = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long px = __shfl_up_sync(0xffffffffu, x, o);
      const long long py = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += px, y += py;
    }
    if (lane == 31) s_w[warp][0] = x, s_w[warp][1] = y;
    __syncthreads();
    long long bx = s_carry[0], by = s_carry[1];
    for (int w = 0; w < warp; ++w) bx += s_w[w][0], by += s_w[w][1];
    if (b < a.B) {
      rows[b] = (int)(bx + x - n);
      take[b] = (int)(by + y - need);
    }
    __syncthreads();
    if (tid == kPlThreads - 1) s_carry[0] = bx + x, s_carry[1] = by + y;
    __syncthreads();
  }
  bad = __syncthreads_or(bad || fc < 0 || fc > a.F);
  full = __syncthreads_or(full) || s_carry[0] > a.T || s_carry[1] > fc;
  const bool ok = !bad && !full;
  const int sum_rows = ok ? (int)s_carry[0] : 0, sum_take = ok ? (int)s_carry[1] : 0;
  if (tid == 0) {
    rows[a.B] = sum_rows;
    take[a.B] = sum_take;
    if (rank == 0 && bad) raise_flag(a.status, FLAG_INDEX);
    if (rank == 0 && full) raise_flag(a.status, FLAG_CAPACITY);
  }
  if (CL > 1) cluster_sync_all();
  else __syncthreads();

  const int t0 = rank * kPlThreads + tid, step = CL * kPlThreads;
  for (int b = t0; b < a.B; b += step) {
    a.kv_lens[b] = past[b] + (ok ? rows[b + 1] - rows[b] : 0);
    a.q_start[b] = ok ? rows[b] : 0;
  }
  if (t0 == 0) {
    a.q_start[a.B] = sum_rows;
    *a.free_left = fc - sum_take;
  }
  auto taken = [&](int i) {  // the i-th page taken, -1 if the list holds no page there
    const int p = a.free_pages[fc - 1 - i];
    if (p >= 0 && p < a.pages) return p;
    raise_flag(a.status, FLAG_INDEX);
    return -1;
  };
  for (int i = t0; i < sum_take; i += step) {
    const int b = find_seq(take, a.B, i);
    const int old = (int)(((long long)past[b] + a.page - 1) / a.page);
    a.table[(size_t)b * a.blocks + old + i - take[b]] = taken(i);
  }
  // four rows at a time, so that their searches and loads overlap
  for (int tt = t0; tt < a.T; tt += kPlRows * step) {
    int pos[kPlRows], slot[kPlRows];
    const int *src[kPlRows];
#pragma unroll
    for (int i = 0; i < kPlRows; ++i) {
      const int t = tt + i * step;
      pos[i] = -1;
      src[i] = nullptr;
      if (t < sum_rows) {
        const int b = find_seq(rows, a.B, t);
        pos[i] = past[b] + t - rows[b];
        const uint32_t blk = (uint32_t)pos[i] / a.page;
        const uint32_t old = ((uint32_t)past[b] + a.page - 1) / a.page;
        src[i] = blk < old ? a.table + (size_t)b * a.blocks + blk
                           : a.free_pages + (fc - 1 - (take[b] + (int)(blk - old)));
      }
    }
#pragma unroll
    for (int i = 0; i < kPlRows; ++i) slot[i] = src[i] ? *src[i] : -1;
#pragma unroll
    for (int i = 0; i < kPlRows; ++i) {
      const int t = tt + i * step;
      if (t >= a.T) break;
      if (src[i]) {
        if (slot[i] >= 0 && slot[i] < a.pages) {
          slot[i] = slot[i] * a.page + (int)((uint32_t)pos[i] % a.page);
        } else {
          raise_flag(a.status, FLAG_INDEX);
          slot[i] = -1;
        }
      }
      a.positions[t] = pos[i];
      a.slots[t] = slot[i];
    }
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedShape &s, const int *new_lens, const int *lens,
                              int *table, const int *free_pages, int F, const int *free_count,
                              int *kv_lens, int *q_start, int *positions, int *slots,
                              int *free_left, uint32_t *status, cudaStream_t st) {
  PlanArgs a{new_lens, lens,  free_pages, free_count, table, kv_lens, q_start, positions,
             slots,    free_left, s.B,    s.T,        s.page, s.pages, s.blocks, F, status};
  const size_t smem = (size_t)(3 * s.B + 2) * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (3 * kPagedMaxB + 2) * (int)sizeof(int));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  DeviceInfo di;
  if ((e = device_info(&di)) != cudaSuccess) return e;
  // one CTA while its threads take at most four rows each
  const int most = di.select_cluster >= kPlCluster ? kPlCluster : 8;
  const int cl = s.T <= kPlRows * kPlThreads ? 1 : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cl, 1, 1);
  cfg.blockDim = dim3(kPlThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  cfg.attrs = attrs;
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = (unsigned)cl;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  cfg.numAttrs = 1;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace sd
