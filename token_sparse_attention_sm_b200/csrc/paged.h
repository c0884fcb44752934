// paged.h -- host side of the paged-cache operators, shared between their
// translation units.
#pragma once

#include "internal.h"

namespace sd {

struct PgArgs;

// A caller's paged shape after the checks every entry point shares.
struct PagedShape {
  int B, T, Hq, Hkv, d, dtype, page, pages, blocks, max_new;
  int G() const { return Hq / Hkv; }
  int esize() const { return dtype == 0 ? 4 : 2; }
};
constexpr int kPagedMaxB = 4096;  // sequences a call may have

// Workspace of the attention: the schedule, then the partials.
struct PagedLayout {
  size_t head_off, seqs_off, part_off, total;
  int slot_cap, part_rows;
};

// Runs that the decode kernel may cut its work into (two partials each).
constexpr int kPagedMaxRuns = 192;
constexpr int kPagedTops = 12;

// bf16, at most 16 query rows per (sequence, KV head) (paged_decode.cu).
cudaError_t launch_paged_decode(const PagedShape &s, const PgArgs &a, cudaStream_t st);
// bf16, any number of rows (paged_chunk.cu): tcgen05.
cudaError_t launch_paged_chunk(const PagedShape &s, const PgArgs &a, cudaStream_t st);
// fp32, at most 16 rows (paged_decode_f32.cu), any number (paged_chunk_f32.cu).
cudaError_t launch_paged_decode_f32(const PagedShape &s, const PgArgs &a, cudaStream_t st);
cudaError_t launch_paged_chunk_f32(const PagedShape &s, const PgArgs &a, cudaStream_t st);
// The work items' schedule for row blocks of `tb` tokens, key tiles of `kt`
// keys and `grid` workers; what a piece costs besides its tiles, whole or cut, in
// quarters of a tile (paged_sched.cu).
cudaError_t launch_paged_schedule(const PagedShape &s, const PgArgs &a, int tb, int kt, int grid,
                                  int whole_cost, int cut_cost, cudaStream_t st);
// Joins the partials of the cut ranges (paged_merge.cu), row blocks of `tb` tokens.
cudaError_t launch_paged_merge(const PagedShape &s, const PgArgs &a, int tb, cudaStream_t st);

}  // namespace sd
