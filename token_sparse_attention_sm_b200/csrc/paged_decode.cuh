// paged_decode.cuh -- the frame of the decode kernels: paged attention of up to
// 16 query rows per (sequence, KV head), a decode step (one token, G query
// heads) or a few tokens of each sequence.
//
// Bound by HBM: every key and value row is read once for the G heads that
// share it.  The work is the list of key tiles of all (sequence, head) pairs,
// cut into equal runs, one per SM, whatever the sequences' lengths; a run that
// starts or ends inside a pair's list leaves a partial (O, max, sum), and the
// last of the pair's runs to arrive merges them in run order (so the result
// does not depend on which one that is).
//
// A CTA is two or four producer warps and some consumer warps.  The producers
// stream the run's K and V tiles through a ring of shared-memory stages with
// TMA (one copy per page and tile, 128-byte swizzle), across pair boundaries,
// so the ring never drains.  Each consumer warp takes every kWarps-th tile with
// its own running maximum, sum and O (sharing a tile between the warps made a
// tile's chain of latencies the limit at d = 64).
//
// The arithmetic of a tile is the class C (one object per consumer warp):
//   Elem, kD, kKeys (keys of a tile), kRows, kWarps, kPairs (pairs of producer
//   warps), kThreads, kTile (bytes of a K or V tile), kStages, kRing, kOS and
//   kOBytes (floats between rows of O, bytes of all warps'), kScratch, kSmem;
//   begin(): the segment's queries; tile(): one tile; join(): the warp's O, max
//   and sum for the segment, unnormalised, into shared memory.
#pragma once

#include "paged.h"
#include "paged.cuh"
#include "paged_tma.h"

namespace sd {
namespace {

constexpr int kDcMerge = 8;      // partials merged at a time
constexpr int kDcGroup = 16;     // runs of a pair merged at once
static_assert(kPagedMaxRuns / kDcGroup <= kPagedTops, "a counter per stretch of kDcGroup runs");

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ void pg_store4(float *dst, const float4 &v, float f) {
  *reinterpret_cast<float4 *>(dst) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void pg_store4(__nv_bfloat16 *dst, const float4 &v, float f) {
  *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(v.x * f, v.y * f), pack2(v.z * f, v.w * f));
}

// Where a run starts: sequence, KV head, tile of the pair.
struct DcStart {
  int total, run;  // tiles of the call (the host bounds them below 2^31), tiles per run
  int align;       // a pair's tiles are counted in multiples of this
  int b, h, u;
};

__device__ __forceinline__ int dc_units(const PgTiles &t) { return max(t.units(), 1); }
__device__ __forceinline__ int dc_round(int units, int align) {
  return align == 1 ? units : (units + align - 1) / align * align;
}
// tiles of a (sequence, head) pair; 0: the sequence has no new tokens
template <int KT>
__device__ __forceinline__ int dc_pair(const PgArgs &a, int b, bool report) {
  int row0, n, kv;
  if (!pg_lengths(a, b, &row0, &n, &kv)) {
    if (report) raise_flag(a.status, FLAG_INDEX);
    return 0;
  }
  return n == 0 ? 0 : dc_units(pg_tiles(kv - n, kv - 1, a.window, a.sinks, KT));
}

// Runs are equal shares of the call's tiles, which balances any batch, unless
// whole multiples of 4, 8 or 16 tiles of single pairs fit the grid: a small
// call is a matter of latency, and runs that never cross a pair then have
// fewer steps one after another (one token each over eight heads of 16 tokens:
// 26 us in runs of four pairs).
constexpr int kDcAligns = 4;  // 1, 4, 8, 16: 1 or 2 << i

// Every CTA finds its own run: thread i sums a stretch of the batch, a block
// scan gives the total and the stretch's first tile, and the thread whose
// stretch holds the run's first tile walks to it.  (A kernel of its own for
// this cost a launch and 4 us of a one-request call.)
template <int kThreads, int KT>
__device__ __forceinline__ void dc_schedule(const PgArgs &a, DcStart *st,
                                            int (*sums)[kDcAligns]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int mine[kDcAligns] = {}, x[kDcAligns];
  for (int b = b0; b < b1; ++b) {
    const int u = dc_pair<KT>(a, b, blockIdx.x == 0);
#pragma unroll
    for (int i = 0; i < kDcAligns; ++i)
      mine[i] += a.Hkv * dc_round(u, i == 0 ? 1 : 2 << i);
  }
#pragma unroll
  for (int i = 0; i < kDcAligns; ++i) {
    x[i] = mine[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += p;
    }
    if (lane == 31) sums[warp][i] = x[i];
  }
  __syncthreads();
  int pick = 0;
  int total = 0, run = 0, base = 0, part = 0;
#pragma unroll
  for (int i = kDcAligns - 1; i >= 0; --i) {
    int t = 0, bs = x[i] - mine[i];
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) bs += sums[w][i];
      t += sums[w][i];
    }
    const int al = 2 << i;
    if (i == 0 || t <= (int)gridDim.x * al) {
      if (i > 0 || pick == 0) {
        pick = i;
        total = t;
        base = bs;
        part = mine[i];
        run = i > 0 ? al : (int)((t + gridDim.x - 1) / gridDim.x);
      }
    }
  }
  const int align = pick > 0 ? 2 << pick : 1;
  const long long x0 = (long long)blockIdx.x * run;  // may pass the total
  if (tid == 0) st->total = total, st->run = run, st->align = align;
  if (part > 0 && base <= x0 && x0 < base + part) {
    for (int b = b0; b < b1; ++b) {
      const int each = dc_round(dc_pair<KT>(a, b, false), align);
      const int t = a.Hkv * each;
      if (x0 < base + t) {
        const int off = (int)x0 - base;
        st->b = b;
        st->h = off / each;
        st->u = off % each;
        break;
      }
      base += t;
    }
  }
  __syncthreads();
}

// One (sequence, KV head) pair's part of a run.
struct DcSeg {
  int b, h, row0, n, kv, units, u0, u1;  // units: rounded up where runs are aligned
  bool cut;                              // not the whole pair
  int p_first, limit, low;  // first row's position; keys the rows see: j < limit and (j >= low or a sink)
  PgTiles t;
};

// Walks a run's segments: every warp of the CTA takes the same walk.
template <int KT>
struct DcWalk {
  int left, item;  // tiles left in the run; the pair's first tile in the call's list
  int b, h, u, align;
  __device__ bool next(const PgArgs &a, DcSeg *s) {
    if (left <= 0) return false;
    int row0, n, kv;
    // sequences without tiles (the last one with some ends the list)
    while (!pg_lengths(a, b, &row0, &n, &kv) || n == 0)
      if (++b >= a.B) return false;
    s->b = b;
    s->h = h;
    s->row0 = row0;
    s->n = n;
    s->kv = kv;
    s->p_first = kv - n;
    s->limit = kv;
    s->low = pg_window_low(kv - n, a.window);
    s->t = pg_tiles(kv - n, kv - 1, a.window, a.sinks, KT);
    const int units = dc_units(s->t);
    s->units = dc_round(units, align);
    s->u0 = u;
    const int end = min(s->units, u + left);
    left -= end - u;
    s->cut = end - u < s->units;
    s->u1 = min(end, units);
    return true;
  }
  // past the segment just taken
  __device__ void advance(const PgArgs &a, const DcSeg &s) {
    item += s.units;
    u = 0;
    if (++h == a.Hkv) {
      h = 0;
      ++b;
    }
  }
};

template <int N>
__device__ __forceinline__ void consumers_sync_n() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    paged_decode_kernel(const __grid_constant__ PgArgs a, const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ CUtensorMap mapV, const PgTile tl) {
  constexpr int D = C::kD, KT = C::kKeys;
  using T = typename C::Elem;
  extern __shared__ unsigned char raw[];
  const uint32_t raw_s = smem_u32(raw);
  const uint32_t base = (raw_s + 1023u) & ~1023u;
  unsigned char *gen = raw + (base - raw_s);
  float *os = reinterpret_cast<float *>(gen + C::kRing);          // [warp][row][kOS]
  unsigned char *small = gen + C::kRing + C::kOBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(small);
  uint64_t *empty = full + C::kStages;
  uint32_t *okmask = reinterpret_cast<uint32_t *>(empty + C::kStages);
  float *ml = reinterpret_cast<float *>(okmask + C::kStages);     // [warp][row][2]
  uint32_t *flag = reinterpret_cast<uint32_t *>(ml + C::kWarps * C::kRows * 2);
  __shared__ DcStart s0;
  __shared__ int warp_sums[C::kThreads / 32][kDcAligns];
  unsigned char *scratch = small + 1024;                          // C::kScratch
  static_assert(C::kStages * 20 + C::kWarps * C::kRows * 8 + 4 <= 1024, "small area");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 2);   // K and V
      mbar_init(&empty[i], 1);  // the warp that takes the tile
    }
    fence_mbar_init();
    pg_prefetch_map(&mapK);
    pg_prefetch_map(&mapV);
  }
  // the arguments through the constant cache once, while the kernel before may
  // still run: a first touch later would stall the one chain there is
  __shared__ volatile uint32_t touched[sizeof(PgArgs) / 4];
  if (tid < (int)(sizeof(PgArgs) / 4)) touched[tid] = reinterpret_cast<const uint32_t *>(&a)[tid];
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  dc_schedule<C::kThreads, KT>(a, &s0, warp_sums);
  const int run = s0.run;
  if ((long long)blockIdx.x * run >= s0.total) return;
  const int x0 = blockIdx.x * run;
  DcWalk<KT> walk{min(run, s0.total - x0), x0 - s0.u, s0.b, s0.h, s0.u, s0.align};
  DcSeg seg;
  const int page = a.page, part_rows = tl.part;
  const int nparts = KT / part_rows, part_log = 31 - __clz(part_rows);

  if (warp >= C::kWarps) {
    // ---- producers: K and V, of every tile or of the even and the odd ones ---------
    const bool isV = (warp - C::kWarps) & 1;
    const int odd = (warp - C::kWarps) >> 1;
    const CUtensorMap *map = isV ? &mapV : &mapK;
    const int per = 32 / nparts;  // tiles whose table entries the lanes hold
    int stage = odd, at = 0, last = -1;  // at: tiles of the run before the one considered
    uint32_t phase = 0;
    bool alive = true;
    while (alive && walk.next(a, &seg)) {
      const int *table = a.table + (size_t)seg.b * a.blocks;
      // lane i: where part i % nparts of tile ub + i / nparts is (token of its
      // page, page * Hkv + head); past the pool (zeros) if it is not read
      int y, z;
      bool bad;
      auto fetch = [&](int ub) {
        const int u = ub + lane / nparts;
        int yy = 0, zz = a.pages * a.Hkv;
        bool bb = false;
        if (u < seg.u1) {
          const int j0 = seg.t.tile(u) * KT + (lane % nparts) * part_rows;
          // some row sees one of the part's keys
          if (j0 < seg.limit && (j0 + part_rows > seg.low || j0 < a.sinks)) {
            const int blk = a.by_page(j0), e = table[blk];
            if (e >= 0 && e < a.pages) {
              yy = j0 - blk * page;
              zz = e * a.Hkv + seg.h;
            } else {
              if (!isV) raise_flag(a.status, FLAG_INDEX);
              bb = true;
            }
          }
        }
        y = yy;
        z = zz;
        bad = bb;
      };
      fetch(seg.u0);
      for (int ub = seg.u0; ub < seg.u1 && alive; ub += per) {
        const int cy = y, cz = z;
        const uint32_t cbad = __ballot_sync(0xffffffffu, bad);
        fetch(ub + per);
        for (int u = ub; u < min(seg.u1, ub + per); ++u, ++at) {
          if (at % C::kPairs != odd) continue;
          const int src = (u - ub) * nparts + lane % nparts;
          const int ty = __shfl_sync(0xffffffffu, cy, src);
          const int tz = __shfl_sync(0xffffffffu, cz, src);
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, a.status))) {
            alive = false;
            break;
          }
          if (lane == 0) {
            if (!isV) okmask[stage] = ~(cbad >> ((u - ub) * nparts));
            mbar_arrive_expect_tx(&full[stage], C::kTile);
          }
          __syncwarp();
          if (lane < nparts)
            pg_tma_part(base + (2 * stage + isV) * C::kTile + lane * part_rows * (D * (int)sizeof(T)), map, tl,
                        ty, tz, &full[stage]);
          __syncwarp();
          last = at;
          stage += C::kPairs;
          if (stage >= C::kStages) stage -= C::kStages, phase ^= 1u;
        }
      }
      walk.advance(a, seg);
    }
    // this warp's copies have landed before it leaves, whatever happened
    for (int i = last; i >= max(0, last - C::kStages + 1); i -= C::kPairs)
      mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, a.status);
    return;
  }

  // ---- consumers -----------------------------------------------------------------
  auto consumers_sync = [] { consumers_sync_n<32 * C::kWarps>(); };
  const int G = a.G;
  T *out = static_cast<T *>(a.out);
  C math;
  // this warp's next tile of the run, and its stage
  int mine = warp, seg0 = 0;
  int stage = warp;
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out: no further waiting, the results are void
  while (walk.next(a, &seg)) {
    const int rows = seg.n * G;
    math.begin(a, seg, rows, scratch, consumers_sync);
    // the pair's first and last run (divided here, where the tile is waited for)
    const int first = walk.item / run, last_run = (walk.item + seg.units - 1) / run;
    // the last row's window is the tightest
    const int low_last = pg_window_low(seg.kv - 1, a.window);
    const int seg1 = seg0 + seg.u1 - seg.u0;
    for (; mine < seg1; mine += C::kWarps) {
      const int key0 = seg.t.tile(seg.u0 + mine - seg0) * KT;
      if (!dead && !mbar_wait(&full[stage], phase, a.status)) dead = true;
      const uint32_t all_parts = (1u << nparts) - 1u, ok = okmask[stage] & all_parts;
      const uint32_t ks = base + stage * 2 * C::kTile, vs = ks + C::kTile;
      // every row sees every key of the tile
      const bool whole = ok == all_parts && key0 + KT - 1 <= seg.p_first &&
                         (key0 >= low_last || key0 + KT <= a.sinks);
      if (key0 + KT > seg.limit || (key0 < seg.low && key0 + KT > a.sinks)) {
        // V rows that no row sees may hold anything: clear them
#pragma unroll
        for (int i = 0; i < KT / 32; ++i) {
          const int r = i * 32 + lane, j = key0 + r;
          if (j >= seg.limit || (j < seg.low && j >= a.sinks)) {
#pragma unroll
            for (int c = 0; c < D * (int)sizeof(T) / 16; ++c)  // 16-byte pieces, rotated: lanes hit other banks
              asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                               vs + (r >> 3) * tl.group + (c >> 3) * tl.col + (r & 7) * 128 +
                               ((c + lane) & 7) * 16),
                           "r"(0u)
                           : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      math.tile(a, tl, ks, vs, key0, whole, ok, part_log);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      stage += C::kWarps;
      if (stage >= C::kStages) stage -= C::kStages, phase ^= 1u;
    }
    seg0 = seg1;

    // ---- the warps' parts of the segment, joined in shared memory ---------
    math.join(os + warp * C::kRows * C::kOS, ml + warp * C::kRows * 2);
    consumers_sync();
    const size_t per = (size_t)a.part_rows * D;
    float2 *pml = reinterpret_cast<float2 *>(a.part + (size_t)a.slot_cap * a.Hkv * per);
    const size_t slot = 2 * (size_t)blockIdx.x + (seg.u0 == 0 ? 1 : 0);
    auto store = [&](int r, int c, float4 acc, float mm, float ll) {
      const float inv = pg_inverse(ll);
      const size_t at = (size_t)(seg.row0 + a.by_G(r)) * a.Hq + seg.h * G + r - a.by_G(r) * G;
      pg_store4(out + at * D + c * 4, acc, inv);
      if (a.lse && c == 0) a.lse[at] = pg_lse(mm, ll);
    };
    for (int i = tid; i < rows * (D / 4); i += 32 * C::kWarps) {
      const int r = i / (D / 4), c = i % (D / 4);
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) mm = fmaxf(mm, ml[(w * C::kRows + r) * 2]);
      const float us = mm == -INFINITY ? 0.f : mm;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float f = exp2f(ml[(w * C::kRows + r) * 2] - us);
        ll += ml[(w * C::kRows + r) * 2 + 1] * f;
        const float4 v =
            *reinterpret_cast<const float4 *>(os + (w * C::kRows + r) * C::kOS + c * 4);
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
      if (!seg.cut) {
        store(r, c, acc, mm, ll);
      } else {
        *reinterpret_cast<float4 *>(a.part + slot * per + (size_t)r * D + c * 4) = acc;
        if (c == 0) pml[slot * a.part_rows + r] = make_float2(mm, ll);
      }
    }
    if (seg.cut) {
      // Partials are merged by the last run to arrive, in run order; of more
      // than kDcGroup runs by groups first (each group's last to arrive), then
      // the groups: no one CTA reads them all.  A counter wraps to zero with
      // the last arrival, so the counters stay clear between calls.
      auto arrive_last = [&](uint32_t *ctr, int count) {
        __threadfence();
        consumers_sync();
        if (tid == 0) *flag = atomicInc(ctr, (uint32_t)count - 1) == (uint32_t)count - 1;
        consumers_sync();
        const bool l = *flag != 0;
        if (l) __threadfence();
        return l;
      };
      // merges the partials of runs w0, w0 + step, .. (n of them); the result
      // is the pair's output, or replaces the first one
      auto merge = [&](int w0, int step, int n, bool final) {
        for (int i = tid; i < C::kRows * (D / 4); i += 32 * C::kWarps) {
          const int r = i / (D / 4), c = i % (D / 4);
          if (r >= rows) break;
          float mm = -INFINITY, ll = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < n; k += kDcMerge) {
            // several at a time, all loads in flight together
            float2 e[kDcMerge];
            float4 v[kDcMerge];
            float top = mm;
#pragma unroll
            for (int j = 0; j < kDcMerge; ++j) {
              const int w = w0 + min(k + j, n - 1) * step;
              const size_t s = 2 * (size_t)w + (w == first);
              e[j] = __ldcg(&pml[s * a.part_rows + r]);
              v[j] = __ldcg(
                  reinterpret_cast<const float4 *>(a.part + s * per + (size_t)r * D + c * 4));
              if (k + j >= n) e[j] = make_float2(-INFINITY, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kDcMerge; ++j) top = fmaxf(top, e[j].x);
            const float us = top == -INFINITY ? 0.f : top, corr = exp2f(mm - us);
            mm = top;
            ll *= corr;
            acc.x *= corr;
            acc.y *= corr;
            acc.z *= corr;
            acc.w *= corr;
#pragma unroll
            for (int j = 0; j < kDcMerge; ++j) {
              const float f = exp2f(e[j].x - us);
              ll += e[j].y * f;
              acc.x += v[j].x * f;
              acc.y += v[j].y * f;
              acc.z += v[j].z * f;
              acc.w += v[j].w * f;
            }
          }
          if (final) {
            store(r, c, acc, mm, ll);
          } else {
            // every reader of this element of the first partial is this thread,
            // but its (max, sum) has D / 4 readers: they meet below
            const size_t s = 2 * (size_t)w0 + (w0 == first);
            *reinterpret_cast<float4 *>(a.part + s * per + (size_t)r * D + c * 4) = acc;
            if (c == 0) ml[r * 2] = mm, ml[r * 2 + 1] = ll;
          }
        }
        if (!final) {
          consumers_sync();
          const size_t s = 2 * (size_t)w0 + (w0 == first);
          if (tid < rows) pml[s * a.part_rows + tid] = make_float2(ml[tid * 2], ml[tid * 2 + 1]);
        }
      };
      const int count = last_run - first + 1;
      if (count <= kDcGroup) {
        if (arrive_last(&a.runs[first], count)) merge(first, 1, count, true);
      } else {
        const int g = ((int)blockIdx.x - first) / kDcGroup, w0 = first + g * kDcGroup;
        const int n = min(kDcGroup, count - g * kDcGroup);
        // (a group's first run may be the next pair's first: other counters)
        if (arrive_last(g == 0 ? &a.runs[w0] : &a.groups[w0], n)) {
          merge(w0, 1, n, false);
          const int groups = (count + kDcGroup - 1) / kDcGroup;
          // pairs of more than kDcGroup runs start in different stretches of as many
          if (arrive_last(&a.tops[first / kDcGroup], groups)) merge(first, kDcGroup, groups, true);
        }
      }
    }
    consumers_sync();
    walk.advance(a, seg);
  }
}

template <typename C>
cudaError_t dc_run(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  auto kern = paged_decode_kernel<C>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const PgTile tile = pg_tile(s.page, s.blocks, C::kD * (int)sizeof(typename C::Elem), C::kKeys);
  CUtensorMap mk, mv;
  e = pg_cache_map(&mk, a.K, s, tile);
  if (e == cudaSuccess) e = pg_cache_map(&mv, a.V, s, tile);
  if (e != cudaSuccess) return e;
  const int grid = di.sm_count < kPagedMaxRuns ? di.sm_count : kPagedMaxRuns;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, kern, a, mk, mv, tile);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace
}  // namespace sd
