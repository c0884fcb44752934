// paged_tma.h -- tensor maps over a paged cache (bf16): tiles of `rows`
// tokens by 64 elements (128 bytes), 128-byte swizzled, addressed as
// (element, token of the page, page * Hkv + head).  Coordinates past the
// pool, and tokens past a page's end, read zeros.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace sd {

// rows of a tile's parts that lie in one page: parts of a KT-key tile never
// straddle pages (single-page tables: the tile itself, clipped at the end)
inline int pg_part_rows(int page, int blocks, int KT) {
  if (blocks == 1) return KT;
  int r = KT;
  while (page % r) r >>= 1;
  return r;
}

cudaError_t pg_cache_map(CUtensorMap *map, const void *cache, int d, int page,
                         long long pages_heads, int rows);
// q [T, Hq, d] (tokens q_stride elements apart) as (element, head, token),
// tiles of 64 elements x `heads` x `tokens`.
cudaError_t pg_query_map(CUtensorMap *map, const void *q, int d, int Hq, int T,
                         long long q_stride, int heads, int tokens);

}  // namespace sd
