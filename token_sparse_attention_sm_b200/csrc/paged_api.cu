// paged_api.cu -- the C entry points of the paged-cache operators: argument
// checks on the host (an error returns before anything is enqueued), then the
// kernels on the caller's stream.
//
// Workspace: the 4 KB header with the device status word first and the decode
// runs' arrival counters (zero between calls) from bytes 128 and 3328, the area
// that the routing calls keep zero between calls (skipped, so that a workspace
// may serve both), then the schedule and the partial results, which every call writes
// before reading.
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

constexpr size_t kPagedHeader = 4096, kRunsOff = 3328, kTopsOff = 128, kGroupsOff = 192;
static_assert(kTopsOff + kPagedTops * sizeof(uint32_t) <= kGroupsOff &&
                  kGroupsOff + kPagedMaxRuns * sizeof(uint32_t) <= 1024 &&
                  kRunsOff + kPagedMaxRuns * sizeof(uint32_t) <= kPagedHeader,
              "the counters fit around the routing scan's");
constexpr size_t kPagedScratch = kPagedHeader + (size_t)256 * kHistBins * sizeof(uint32_t);
constexpr int kPartialSlots = 592;  // four pieces for each of 148 SMs
static_assert(kPartialSlots >= 2 * kPagedMaxRuns, "two partials per decode run");

sparse_status_t check_paged(const sparse_paged_shape_t *p, PagedShape *s) {
  if (!p) return SPARSE_ERR_INVALID_ARG;
  *s = PagedShape{p->B,    p->T,         p->Hq,        p->Hkv,        p->d,
                  p->dtype, p->page_size, p->num_pages, p->max_blocks, p->max_new};
  if (s->B < 1 || s->T < 0 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 || s->page < 1 ||
      s->pages < 1 || s->blocks < 1 || s->max_new < 0)
    return SPARSE_ERR_INVALID_ARG;
  if (s->Hq % s->Hkv != 0) return SPARSE_ERR_INVALID_ARG;
  if (s->d != 64 && s->d != 128) return SPARSE_ERR_UNSUPPORTED;
  if (s->dtype != SPARSE_DTYPE_F32 && s->dtype != SPARSE_DTYPE_BF16)
    return SPARSE_ERR_UNSUPPORTED;
  if (s->G() > 16 || s->B > kPagedMaxB || s->Hkv > 65535) return SPARSE_ERR_UNSUPPORTED;
  if (s->page % 16 != 0 && s->blocks != 1) return SPARSE_ERR_UNSUPPORTED;
  if ((long long)s->pages * s->page > 0x7fffffffll ||
      (long long)s->pages * s->Hkv > 0x7fffffffll ||
      (long long)s->blocks * s->page > (1ll << 30) || s->T > (1 << 24) ||
      // the 32-key tiles that the longest batch has, in 31 bits
      (long long)s->B * s->Hkv * ((long long)s->blocks * s->page / 32 + 32) > 0x7fffffffll)
    return SPARSE_ERR_UNSUPPORTED;
  if (s->max_new == 0 || s->max_new > s->T) s->max_new = s->T;
  return SPARSE_OK;
}

PagedLayout layout(const PagedShape &s) {
  PagedLayout l;
  l.slot_cap = (kPartialSlots + s.Hkv - 1) / s.Hkv;
  const long long rows = (long long)s.max_new * s.G();
  l.part_rows = (int)(rows < 256 ? rows : 256);
  l.head_off = kPagedScratch;
  l.seqs_off = l.head_off + up256(sizeof(PgHead));
  // partials: slot_cap * Hkv >= kPartialSlots >= 2 * kPagedMaxRuns
  l.part_off = l.seqs_off + up256((size_t)(s.B + 1) * sizeof(PgSeq));
  l.total = l.part_off + up256((size_t)l.slot_cap * s.Hkv * l.part_rows * (s.d + 2) *
                               sizeof(float));
  return l;
}

// the status area of calls whose workspaces are temporaries
__device__ __align__(256) unsigned char g_static_status[kPagedHeader];

sparse_status_t status_of(cudaError_t e) {
  return e == cudaSuccess ? SPARSE_OK : SPARSE_ERR_CUDA;
}

}  // namespace

cudaError_t launch_paged_plan(const PagedShape &s, const int *new_lens, const int *lens,
                              int *table, const int *free_pages, int F, const int *free_count,
                              int *kv_lens, int *q_start, int *positions, int *slots,
                              int *free_left, uint32_t *status, cudaStream_t st);
cudaError_t launch_paged_append(const PagedShape &s, void *K, void *V, const void *k_new,
                                const void *v_new, long long k_stride, long long v_stride,
                                const int *slots, uint32_t *status, cudaStream_t st);

}  // namespace sd

using sd::PagedShape;

extern "C" {

sparse_status_t sparse_paged_workspace_size(const sparse_paged_shape_t *shape, size_t *bytes) {
  PagedShape s;
  sparse_status_t r = sd::check_paged(shape, &s);
  if (r != SPARSE_OK) return r;
  if (!bytes) return SPARSE_ERR_INVALID_ARG;
  *bytes = sd::layout(s).total;
  return SPARSE_OK;
}

sparse_status_t sparse_paged_plan(const sparse_paged_shape_t *shape, const int32_t *new_lens,
                                  const int32_t *lens, int32_t *block_table,
                                  const int32_t *free_pages, int32_t free_cap,
                                  const int32_t *free_count, int32_t *kv_lens, int32_t *q_start,
                                  int32_t *positions, int32_t *slots, int32_t *free_left, void *ws,
                                  size_t ws_bytes, void *stream) {
  PagedShape s;
  sparse_status_t r = sd::check_paged(shape, &s);
  if (r != SPARSE_OK) return r;
  if (!new_lens || !lens || !block_table || !free_count || !kv_lens || !q_start || !free_left ||
      free_cap < 0 || (free_cap > 0 && !free_pages) || (s.T > 0 && (!positions || !slots)))
    return SPARSE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)new_lens, (const void *)lens, (const void *)block_table,
                        (const void *)free_pages, (const void *)free_count, (const void *)kv_lens,
                        (const void *)q_start, (const void *)positions, (const void *)slots,
                        (const void *)free_left})
    if (!sd::aligned(p, 4)) return SPARSE_ERR_INVALID_ARG;
  if (!ws || !sd::aligned(ws, 256)) return SPARSE_ERR_INVALID_ARG;
  if (ws_bytes < sd::kPagedHeader) return SPARSE_ERR_WORKSPACE;
  return sd::status_of(sd::launch_paged_plan(
      s, new_lens, lens, block_table, free_pages, free_cap, free_count, kv_lens, q_start,
      positions, slots, free_left, static_cast<uint32_t *>(ws), static_cast<cudaStream_t>(stream)));
}

sparse_status_t sparse_paged_append(const sparse_paged_shape_t *shape, void *K, void *V,
                                    const void *k_new, int64_t k_stride, const void *v_new,
                                    int64_t v_stride, const int32_t *slots, void *ws,
                                    size_t ws_bytes, void *stream) {
  PagedShape s;
  sparse_status_t r = sd::check_paged(shape, &s);
  if (r != SPARSE_OK) return r;
  if (s.T < 1 || !K || !V || !k_new || !v_new || !slots) return SPARSE_ERR_INVALID_ARG;
  const int64_t row = (int64_t)s.Hkv * s.d, per16 = 16 / s.esize();
  for (const int64_t st : {k_stride, v_stride})
    if (st % per16 != 0 || (st < row && s.T > 1)) return SPARSE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)K, (const void *)V, k_new, v_new})
    if (!sd::aligned(p, 16)) return SPARSE_ERR_INVALID_ARG;
  if (!sd::aligned(slots, 4) || !ws || !sd::aligned(ws, 256)) return SPARSE_ERR_INVALID_ARG;
  if (ws_bytes < sd::kPagedHeader) return SPARSE_ERR_WORKSPACE;
  return sd::status_of(sd::launch_paged_append(s, K, V, k_new, v_new, k_stride, v_stride, slots,
                                               static_cast<uint32_t *>(ws),
                                               static_cast<cudaStream_t>(stream)));
}

sparse_status_t sparse_paged_attn(const sparse_paged_shape_t *shape, const void *q,
                                  int64_t q_stride, const void *K, const void *V,
                                  const int32_t *block_table, const int32_t *q_start,
                                  const int32_t *kv_lens, int32_t window, int32_t sinks, void *out,
                                  float *lse, void *ws, size_t ws_bytes, void *stream) {
  return sparse_paged_attn_status(shape, q, q_stride, K, V, block_table, q_start, kv_lens, window,
                                  sinks, out, lse, ws, ws_bytes, static_cast<uint32_t *>(ws),
                                  stream);
}

sparse_status_t sparse_paged_attn_status(const sparse_paged_shape_t *shape, const void *q,
                                         int64_t q_stride, const void *K, const void *V,
                                         const int32_t *block_table, const int32_t *q_start,
                                         const int32_t *kv_lens, int32_t window, int32_t sinks,
                                         void *out, float *lse, void *ws, size_t ws_bytes,
                                         uint32_t *status, void *stream) {
  PagedShape s;
  sparse_status_t r = sd::check_paged(shape, &s);
  if (r != SPARSE_OK) return r;
  if (s.T < 1 || !q || !K || !V || !block_table || !q_start || !kv_lens || !out || window < 0 ||
      sinks < 0)
    return SPARSE_ERR_INVALID_ARG;
  const int64_t row = (int64_t)s.Hq * s.d, per16 = 16 / s.esize();
  if (q_stride % per16 != 0 || (q_stride < row && s.T > 1)) return SPARSE_ERR_INVALID_ARG;
  for (const void *p : {q, K, V, (const void *)out})
    if (!sd::aligned(p, 16)) return SPARSE_ERR_INVALID_ARG;
  for (const void *p : {(const void *)block_table, (const void *)q_start, (const void *)kv_lens,
                        (const void *)lse})
    if (!sd::aligned(p, 4)) return SPARSE_ERR_INVALID_ARG;
  if (!ws || !sd::aligned(ws, 256) || !status || !sd::aligned(status, 4))
    return SPARSE_ERR_INVALID_ARG;
  const sd::PagedLayout l = sd::layout(s);
  if (ws_bytes < l.total) return SPARSE_ERR_WORKSPACE;
  // results written while other blocks still read: never over the inputs
  const size_t es = (size_t)s.esize(), o_bytes = (size_t)s.T * row * es;
  const size_t q_bytes = ((size_t)(s.T - 1) * q_stride + row) * es;
  const size_t c_bytes = (size_t)s.pages * s.Hkv * s.page * s.d * es;
  const size_t l_bytes = lse ? (size_t)s.T * s.Hq * sizeof(float) : 0;
  if (sd::overlap(out, o_bytes, q, q_bytes) || sd::overlap(out, o_bytes, K, c_bytes) ||
      sd::overlap(out, o_bytes, V, c_bytes))
    return SPARSE_ERR_INVALID_ARG;
  if (lse && (sd::overlap(lse, l_bytes, q, q_bytes) || sd::overlap(lse, l_bytes, K, c_bytes) ||
              sd::overlap(lse, l_bytes, V, c_bytes) || sd::overlap(lse, l_bytes, out, o_bytes)))
    return SPARSE_ERR_INVALID_ARG;
  char *w = static_cast<char *>(ws);
  sd::PgArgs a;
  a.q = q;
  a.K = K;
  a.V = V;
  a.table = block_table;
  a.q_start = q_start;
  a.kv_lens = kv_lens;
  a.out = out;
  a.lse = lse;
  a.q_stride = q_stride;
  a.B = s.B;
  a.T = s.T;
  a.Hq = s.Hq;
  a.Hkv = s.Hkv;
  a.G = s.G();
  a.by_G = sd::pg_divisor((uint32_t)a.G);
  a.by_page = sd::pg_divisor((uint32_t)s.page);
  a.page = s.page;
  a.pages = s.pages;
  a.blocks = s.blocks;
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;  // without a window every earlier key is seen
  a.max_new = s.max_new;
  a.scale_log2 = (float)(1.4426950408889634 / (s.d == 64 ? 8.0 : 11.313708498984761));
  a.status = status;
  a.head = reinterpret_cast<sd::PgHead *>(w + l.head_off);
  a.seqs = reinterpret_cast<sd::PgSeq *>(w + l.seqs_off);
  a.runs = reinterpret_cast<uint32_t *>(w + sd::kRunsOff);
  a.groups = reinterpret_cast<uint32_t *>(w + sd::kGroupsOff);
  a.tops = reinterpret_cast<uint32_t *>(w + sd::kTopsOff);
  a.part = reinterpret_cast<float *>(w + l.part_off);
  a.slot_cap = l.slot_cap;
  a.part_rows = l.part_rows;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // few rows per cache row: bound by memory; many: by arithmetic
  const bool few = s.max_new * s.G() <= 16;
  if (s.dtype == SPARSE_DTYPE_F32)
    return sd::status_of(few ? sd::launch_paged_decode_f32(s, a, st)
                             : sd::launch_paged_chunk_f32(s, a, st));
  return sd::status_of(few ? sd::launch_paged_decode(s, a, st) : sd::launch_paged_chunk(s, a, st));
}

sparse_status_t sparse_paged_static_status(void **ws) {
  if (!ws) return SPARSE_ERR_INVALID_ARG;
  // the lookup may load the library's code: allowed while this thread captures
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return SPARSE_ERR_CUDA;
  e = cudaGetSymbolAddress(ws, sd::g_static_status);
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  return sd::status_of(e == cudaSuccess ? back : e);
}

}  // extern "C"
