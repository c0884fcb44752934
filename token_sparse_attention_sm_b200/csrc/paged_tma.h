// paged_tma.h -- tensor maps over a paged cache.  One copy brings the
// part of a key tile that lies in one page, all d columns, in 128-byte rows of
// 64 bf16 or 32 fp32 elements, 128-byte swizzled.  Two shared-memory layouts:
//  * the whole tile is one part: [column block][key][128 B];
//  * several parts: [8 keys][column block][key of the 8][128 B], so that the
//    parts, one after another, make the same uniform layout.
// (One copy per part and column block, as a plain 2-D tile would need, is
// bound by issuing the copies when pages are short: 16-token pages at d = 128
// streamed at 5.2 TB/s, 32-token ones at 6.8.)  Coordinates past the pool, and
// tokens past a single page's end, read zeros.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sd {

// rows of a tile's parts that lie in one page: parts of a KT-key tile never
// straddle pages (single-page tables: the tile itself, clipped at the end)
inline int pg_part_rows(int page, int blocks, int KT) {
  if (blocks == 1) return KT;
  int r = KT;
  while (page % r) r >>= 1;
  return r;
}

// Byte strides of a tile's layout in shared memory: between groups of 8 keys,
// between column blocks.
struct PgTile {
  int part;  // keys of a part
  int whole; // the tile is one part
  int group, col;
};
inline PgTile pg_tile(int page, int blocks, int row_bytes, int KT) {
  const int part = pg_part_rows(page, blocks, KT);
  if (part == KT) return PgTile{part, 1, 1024, KT * 128};
  return PgTile{part, 0, row_bytes / 128 * 1024, 1024};
}

struct PagedShape;
cudaError_t pg_cache_map(CUtensorMap *map, const void *cache, const PagedShape &s,
                         const PgTile &t);
// q [T, Hq, d] in bf16 (tokens q_stride elements apart) as (element, head, token),
// tiles of 64 elements x `heads` x `tokens`.
cudaError_t pg_query_map(CUtensorMap *map, const void *q, int d, int Hq, int T,
                         long long q_stride, int heads, int tokens);

#ifdef __CUDACC__
// The part of a tile that starts at token y of page-and-head z.
__device__ __forceinline__ void pg_tma_part(uint32_t dst, const CUtensorMap *map, const PgTile &t,
                                            int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %2, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(0), "r"(t.whole ? y : 0), "r"(t.whole ? 0 : y >> 3), "r"(z),
      "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void pg_prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
#endif

}  // namespace sd
