// paged_append.cu -- the new tokens' key and value rows into their pages:
// K[slot / page, h, slot % page, :] = k_new[t, h, :], V likewise; a row with
// slot -1 (padding) writes nothing.
//
// A copy, bound by HBM: a warp moves up to 2 KB of a token's K and as much of
// its V, all eight 16-byte loads of a lane in flight before the first store.
// The source may be a column range of wider rows (a fused projection).
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kApThreads = 256;
constexpr int kApUnroll = 4;
constexpr int kApSeg = 32 * kApUnroll;  // 16-byte pieces a warp moves of each cache

// CPR: 16-byte pieces of a head's row
template <int CPR>
__global__ void __launch_bounds__(kApThreads)
    paged_append_kernel(uint4 *__restrict__ K, uint4 *__restrict__ V,
                        const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
                        long long k_stride, long long v_stride, const int *__restrict__ slots,
                        int T, int Hkv, int page, int pages, int nseg, uint32_t *status) {
  grid_dep_wait();
  grid_dep_launch();
  const long long w = ((long long)blockIdx.x * kApThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / nseg), seg = (int)(w % nseg);
  if (t >= T) return;
  const int slot = slots[t];
  if (slot == -1) return;
  if (slot < 0 || slot / page >= pages) {
    if (lane == 0 && seg == 0) raise_flag(status, FLAG_INDEX);
    return;
  }
  const size_t dst0 = ((size_t)(slot / page) * Hkv * page + slot % page) * CPR;
  const size_t head = (size_t)page * CPR;  // pieces between the heads of a page
  const int n = Hkv * CPR, i0 = seg * kApSeg + lane;
  uint4 k[kApUnroll], v[kApUnroll];
#pragma unroll
  for (int u = 0; u < kApUnroll; ++u) {
    const int i = i0 + u * 32;
    if (i < n) {
      k[u] = __ldcs(k_new + (size_t)t * k_stride + i);
      v[u] = __ldcs(v_new + (size_t)t * v_stride + i);
    }
  }
#pragma unroll
  for (int u = 0; u < kApUnroll; ++u) {
    const int i = i0 + u * 32;
    if (i < n) {
      const size_t dst = dst0 + (size_t)(i / CPR) * head + i % CPR;
      K[dst] = k[u];
      V[dst] = v[u];
    }
  }
}

template <int CPR>
cudaError_t run(const PagedShape &s, void *K, void *V, const void *k_new, const void *v_new,
                long long k_stride, long long v_stride, const int *slots, uint32_t *status,
                cudaStream_t st) {
  const int nseg = (s.Hkv * CPR + kApSeg - 1) / kApSeg;
  const long long warps = (long long)s.T * nseg, per = kApThreads / 32;
  const long long blocks = (warps + per - 1) / per;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(kApThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  cfg.attrs = attrs;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  const int per16 = 16 / s.esize();
  cudaError_t e = cudaLaunchKernelEx(
      &cfg, paged_append_kernel<CPR>, static_cast<uint4 *>(K), static_cast<uint4 *>(V),
      static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), k_stride / per16,
      v_stride / per16, slots, s.T, s.Hkv, s.page, s.pages, nseg, status);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_append(const PagedShape &s, void *K, void *V, const void *k_new,
                                const void *v_new, long long k_stride, long long v_stride,
                                const int *slots, uint32_t *status, cudaStream_t st) {
  switch (s.d * s.esize() / 16) {
    case 8: return run<8>(s, K, V, k_new, v_new, k_stride, v_stride, slots, status, st);
    case 16: return run<16>(s, K, V, k_new, v_new, k_stride, v_stride, slots, status, st);
    default: return run<32>(s, K, V, k_new, v_new, k_stride, v_stride, slots, status, st);
  }
}

}  // namespace sd
