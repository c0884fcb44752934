// paged_tma.cu -- encoding of the tensor maps in paged_tma.h, through the
// driver entry point that the runtime hands out (no link against libcuda).
#include "paged_tma.h"

#include "paged.h"

#include <mutex>

namespace sd {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

cudaError_t encode(CUtensorMap *map, int dtype, int rank, const void *base, const cuuint64_t *dims,
                   const cuuint64_t *strides, const cuuint32_t *box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  const CUresult r =
      fn(map, dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box,
         step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t pg_cache_map(CUtensorMap *map, const void *cache, const PagedShape &s,
                         const PgTile &t) {
  const cuuint64_t row = (cuuint64_t)s.d * s.esize(), cb = row / 128, head = row * s.page;
  const cuuint64_t ph = (cuuint64_t)s.pages * s.Hkv;
  const cuuint32_t per = 128 / s.esize();  // elements of a 128-byte row
  if (t.whole) {  // (element, token, column block, -, page * Hkv + head)
    const cuuint64_t dims[5] = {per, (cuuint64_t)s.page, cb, 1, ph};
    const cuuint64_t strides[4] = {row, 128, head, head};
    const cuuint32_t box[5] = {per, (cuuint32_t)t.part, (cuuint32_t)cb, 1, 1};
    return encode(map, s.dtype, 5, cache, dims, strides, box);
  }
  // (element, token of 8, column block, group of 8 tokens, page * Hkv + head)
  const cuuint64_t dims[5] = {per, 8, cb, (cuuint64_t)s.page / 8, ph};
  const cuuint64_t strides[4] = {row, 128, 8 * row, head};
  const cuuint32_t box[5] = {per, 8, (cuuint32_t)cb, (cuuint32_t)t.part / 8, 1};
  return encode(map, s.dtype, 5, cache, dims, strides, box);
}

cudaError_t pg_query_map(CUtensorMap *map, const void *q, int d, int Hq, int T,
                         long long q_stride, int heads, int tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  return encode(map, 1, 3, q, dims, strides, box);
}

}  // namespace sd
