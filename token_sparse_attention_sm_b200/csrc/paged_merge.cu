// paged_merge.cu -- joins the pieces of cut key ranges: with a block's row r and
// its pieces' partials (O_p, m_p, l_p), m = max m_p, o = sum 2^(m_p - m) O_p /
// sum 2^(m_p - m) l_p.
//
// Bound by latency: a range cut for all SMs has a dozen partials per row, in L2.
// A kernel of its own spreads them over the SMs, a share of a block's rows for
// each of its pieces, so that every CTA reads about one partial's worth; the last
// of a block's pieces to arrive took them all before (52 us after 38 us of work
// for 32 tokens over 32K, 8 KV heads; 52 us in all now).  A call without cut
// ranges pays 1 us for the launch.
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kMgThreads = 512;

// T: type of out; TB: tokens of a block
template <int D, typename T>
__global__ void __launch_bounds__(kMgThreads, 2) paged_merge_kernel(const PgArgs a, int TB) {
  grid_dep_wait();
  grid_dep_launch();
  const long long total = (long long)a.seqs[a.B].slot * a.Hkv;
  for (long long x = blockIdx.x; x < total; x += gridDim.x) {
    const int slot = (int)(x / a.Hkv), h = (int)(x % a.Hkv);
    PgSeq sq;
    const int b = pg_find(a.seqs, a.B, slot, &PgSeq::slot, &sq);
    int row0, n, kv;
    pg_lengths(a, b, &row0, &n, &kv);
    const int rb = (slot - sq.slot) / sq.np, piece = (slot - sq.slot) % sq.np;
    const int t0 = rb * TB, rows = (min(n, t0 + TB) - t0) * a.G;
    const int r0 = rows * piece / sq.np, r1 = rows * (piece + 1) / sq.np;
    pg_merge<D, 2>(a, (size_t)(slot - piece) * a.Hkv + h, sq.np, r0, r1 - r0, (int)threadIdx.x,
                   kMgThreads,
                   [&](int r) {
                     const int t = a.by_G(r);
                     return (size_t)(row0 + t0 + t) * a.Hq + h * a.G + r - t * a.G;
                   },
                   static_cast<T *>(a.out));
  }
}

template <int D, typename T>
cudaError_t run(const PgArgs &a, int tb, cudaStream_t st) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  // all that fit the SMs together
  const int most = a.slot_cap * a.Hkv, fit = 2 * di.sm_count;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < fit ? most : fit), 1, 1);
  cfg.blockDim = dim3(kMgThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  cfg.attrs = attrs;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, T>, a, tb);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_merge(const PagedShape &s, const PgArgs &a, int tb, cudaStream_t st) {
  if (s.dtype == SPARSE_DTYPE_F32)
    return s.d == 64 ? run<64, float>(a, tb, st) : run<128, float>(a, tb, st);
  return s.d == 64 ? run<64, __nv_bfloat16>(a, tb, st) : run<128, __nv_bfloat16>(a, tb, st);
}

}  // namespace sd
