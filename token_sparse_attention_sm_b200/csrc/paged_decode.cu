// paged_decode.cu -- paged attention in bf16 for up to 16 query rows per
// (sequence, KV head): a decode step (one token, G query heads), or a few
// tokens of each sequence.
//
// Bound by HBM: every key and value row is read once for the G heads that
// share it, 4 G flop per two bytes.  The work is the list of 64-key tiles of
// all (sequence, head) pairs, cut into equal runs, one per SM, whatever the
// sequences' lengths; a run that starts or ends inside a pair's list leaves a
// partial (O, max, sum), and the last of the pair's runs to arrive merges them
// in run order (so the result does not depend on which one that is).
//
// A CTA is one producer warp and four consumer warps.  The producer streams
// the run's tiles through a ring of shared-memory stages with TMA (one copy
// per page fragment and 64 columns, 128-byte swizzle), across pair
// boundaries, so the ring never drains.  Each consumer warp takes 16 keys of a
// tile with its own running maximum, sum and O: S = Q K^T and O += P V on
// mma.sync m16n8k16 -- 16 rows are all there is, a quarter of the smallest
// tcgen05 tile, and nothing has to leave the registers between the two
// products.  P is split in two bf16 parts (P_hi + P_lo: 16 significant bits),
// which costs nothing where memory is the limit.
#include "paged.h"
#include "paged.cuh"
#include "paged_tma.h"

namespace sd {
namespace {

constexpr int kDcKeys = 64;      // keys per tile
constexpr int kDcWarps = 4;      // consumer warps, 16 keys each
constexpr int kDcThreads = 32 * (kDcWarps + 1);
constexpr int kDcRows = 16;
constexpr int kDcMinRun = 2;     // tiles a run has at least

template <int D>
struct DcCfg {
  static constexpr int kTile = kDcKeys * D * 2;           // K or V of a tile
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kOS = D + 8;                        // floats between rows of O
  static constexpr int kOBytes = kDcWarps * kDcRows * kOS * 4;
  static constexpr int kSmem = kRing + kOBytes + 1024 + 1024;  // + small, alignment
};

// where a run starts: sequence, KV head, tile of the pair
struct DcStart {
  int b, h, u, pad;
};
struct DcHead {
  long long total;  // tiles of the call
  long long run;    // tiles per run
};

__device__ __forceinline__ int dc_units(const PgTiles &t) { return max(t.units(), 1); }

__global__ void __launch_bounds__(1024) paged_decode_schedule_kernel(const PgArgs a, int workers) {
  __shared__ long long s_pre[kPagedMaxB + 1];
  __shared__ long long s_w[32], s_carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) s_carry = 0;
  __syncthreads();
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + tid;
    long long u = 0;
    if (b < a.B) {
      int row0, n, kv;
      if (!pg_lengths(a, b, &row0, &n, &kv)) raise_flag(a.status, FLAG_INDEX);
      else if (n > 0)
        u = (long long)a.Hkv * dc_units(pg_tiles(kv - n, kv - 1, a.window, a.sinks, kDcKeys));
    }
    long long x = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long p = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += p;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    long long base = s_carry;
    for (int w = 0; w < warp; ++w) base += s_w[w];
    if (b < a.B) s_pre[b] = base + x - u;
    __syncthreads();
    if (tid == 1023) s_carry = base + x;
    __syncthreads();
  }
  const long long total = s_carry;
  long long run = (total + workers - 1) / workers;
  if (run < kDcMinRun) run = kDcMinRun;
  DcHead *hd = reinterpret_cast<DcHead *>(a.head);
  if (tid == 0) {
    s_pre[a.B] = total;
    *hd = DcHead{total, run};
  }
  DcStart *st = reinterpret_cast<DcStart *>(a.seqs);
  for (int w = tid; w < workers; w += 1024) {
    const long long x = w * run;
    if (x < total) {
      int lo = 0, hi = a.B - 1;  // the last sequence whose tiles start at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_pre[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      const long long end = lo + 1 < a.B ? s_pre[lo + 1] : total;
      const long long per = (end - s_pre[lo]) / a.Hkv, off = x - s_pre[lo];
      st[w] = DcStart{lo, (int)(off / per), (int)(off % per), 0};
    }
    a.arrive[w] = 0u;
  }
}

// One (sequence, KV head) pair's part of a run.
struct DcSeg {
  int b, h, row0, n, kv, units, u0, u1;
  int p_first, limit, low;  // first row's position; keys the rows see: j < limit and (j >= low or a sink)
  PgTiles t;
};

// Walks a run's segments: every warp of the CTA takes the same walk.
struct DcWalk {
  long long left, item;  // tiles left in the run; the pair's first tile in the call's list
  int b, h, u;
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
    s->t = pg_tiles(kv - n, kv - 1, a.window, a.sinks, kDcKeys);
    s->units = dc_units(s->t);
    s->u0 = u;
    s->u1 = (int)min((long long)s->units, u + left);
    left -= s->u1 - u;
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

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                     uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kDcWarps) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kDcThreads, 1)
    paged_decode_kernel(const PgArgs a, const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ CUtensorMap mapV, int part_rows) {
  using C = DcCfg<D>;
  constexpr int CB = D / 64;  // 64-column blocks of a row
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
  uint32_t *flag = reinterpret_cast<uint32_t *>(ml + kDcWarps * kDcRows * 2);
  static_assert(C::kStages * 20 + kDcWarps * kDcRows * 8 + 4 <= 1024, "small area");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kDcWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const DcHead hd = *reinterpret_cast<const DcHead *>(a.head);
  const long long x0 = (long long)blockIdx.x * hd.run;
  if (x0 >= hd.total) return;
  const DcStart s0 = reinterpret_cast<const DcStart *>(a.seqs)[blockIdx.x];
  DcWalk walk{min(hd.run, hd.total - x0), x0 - s0.u, s0.b, s0.h, s0.u};
  DcSeg seg;
  const int page = a.page;
  const int nparts = kDcKeys / part_rows;

  if (warp == kDcWarps) {
    // ---- producer ------------------------------------------------------------
    const int per = 32 / nparts;  // tiles whose table entries the lanes hold
    int stage = 0;
    uint32_t phase = 0;
    while (walk.next(a, &seg)) {
      const int *table = a.table + (size_t)seg.b * a.blocks;
      // lane i: entry of part i % nparts of tile ub + i / nparts; -1: not read
      auto fetch = [&](int ub) {
        const int u = ub + lane / nparts;
        int e = -1;
        if (lane < per * nparts && u < seg.u1) {
          const int j0 = seg.t.tile(u) * kDcKeys + (lane % nparts) * part_rows;
          // some row sees one of the part's keys
          if (j0 < seg.limit && (j0 + part_rows > seg.low || j0 < a.sinks)) {
            e = table[j0 / page];
            if (e < 0 || e >= a.pages) {
              raise_flag(a.status, FLAG_INDEX);
              e = -2;
            }
          }
        }
        return e;
      };
      int next = fetch(seg.u0);
      for (int ub = seg.u0; ub < seg.u1; ub += per) {
        const int cur = next;
        next = fetch(ub + per);
        for (int u = ub; u < min(seg.u1, ub + per); ++u) {
          const int e = __shfl_sync(0xffffffffu, cur, (u - ub) * nparts + lane % nparts);
          const uint32_t bad = __ballot_sync(0xffffffffu, lane < nparts && e == -2);
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, a.status))) return;
          if (lane == 0) {
            okmask[stage] = ~bad;
            mbar_arrive_expect_tx(&full[stage], 2 * C::kTile);
          }
          __syncwarp();
          if (lane < nparts) {
            const int j0 = seg.t.tile(u) * kDcKeys + lane * part_rows;
            const int y = e >= 0 ? j0 % page : 0;
            const int z = e >= 0 ? e * a.Hkv + seg.h : a.pages * a.Hkv;  // past the pool: zeros
            const uint32_t k = base + stage * 2 * C::kTile + lane * part_rows * 128;
#pragma unroll
            for (int c = 0; c < CB; ++c)
              tma3(k + c * (kDcKeys * 128), &mapK, c * 64, y, z, &full[stage]);
#pragma unroll
            for (int c = 0; c < CB; ++c)
              tma3(k + C::kTile + c * (kDcKeys * 128), &mapV, c * 64, y, z, &full[stage]);
          }
          __syncwarp();
          if (++stage == C::kStages) stage = 0, phase ^= 1u;
        }
      }
      walk.advance(a, seg);
    }
    return;
  }

  // ---- consumers -----------------------------------------------------------------
  const int G = a.Hq / a.Hkv;
  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
  const int g8 = lane >> 2, t4 = lane & 3;
  int stage = 0;
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out: no further waiting, the results are void
  while (walk.next(a, &seg)) {
    const int rows = seg.n * G;
    uint32_t qf[D / 16][4];
    int pos[2], low[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g8 + i * 8;
      pos[i] = r < rows ? seg.p_first + r / G : -1;
      low[i] = pg_window_low(pos[i], a.window);
      const uint32_t *src =
          r < rows ? reinterpret_cast<const uint32_t *>(
                         q + (size_t)(seg.row0 + r / G) * a.q_stride +
                         (size_t)(seg.h * G + r % G) * D)
                   : nullptr;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][i] = src ? src[s * 8 + t4] : 0u;
        qf[s][i + 2] = src ? src[s * 8 + t4 + 4] : 0u;
      }
    }
    // the last row's window is the tightest
    const int low_last = pg_window_low(seg.kv - 1, a.window);
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int u = seg.u0; u < seg.u1; ++u) {
      const int key0 = seg.t.tile(u) * kDcKeys;
      if (!dead && !mbar_wait(&full[stage], phase, a.status)) dead = true;
      const uint32_t ok = okmask[stage];
      const uint32_t ks = base + stage * 2 * C::kTile, vs = ks + C::kTile;
      const bool bad_page = (ok & ((1u << nparts) - 1u)) != ((1u << nparts) - 1u);
      // every row sees every key of the tile
      const bool whole = !bad_page && key0 + kDcKeys - 1 <= seg.p_first &&
                         (key0 >= low_last || key0 + kDcKeys <= a.sinks);
      if (key0 + kDcKeys > seg.limit || (key0 < seg.low && key0 + kDcKeys > a.sinks)) {
        // V rows that no row sees may hold anything: clear this warp's
        const int r = warp * 16 + (lane >> 1), j = key0 + r;
        if (j >= seg.limit || (j < seg.low && j >= a.sinks)) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const int ch = (lane & 1) * (D / 16) + c;  // 16-byte piece; the swizzle permutes a row
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                             vs + (ch >> 3) * (kDcKeys * 128) + r * 128 + (ch & 7) * 16),
                         "r"(0u)
                         : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
      {
        const int r = warp * 16 + ((lane >> 4) << 3) + (lane & 7);
        const uint32_t row = ks + r * 128;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const int ch = 2 * s + ((lane >> 3) & 1);
          uint32_t kf[4];
          ldsm4(row + (ch >> 3) * (kDcKeys * 128) + (((ch & 7) ^ (r & 7)) << 4), kf);
          mma16816(sc[0], qf[s], kf[0], kf[1]);
          mma16816(sc[1], qf[s], kf[2], kf[3]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] *= a.scale_log2;
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = warp * 16 + nt * 8 + t4 * 2 + (e & 1), j = key0 + r;
            const bool see = j <= pos[e >> 1] && (j >= low[e >> 1] || j < a.sinks) &&
                             ((ok >> (r / part_rows)) & 1u);
            if (!see) sc[nt][e] = -INFINITY;
          }
      }
      float mx[2], use[2];
      bool up = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1]));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        mx[i] = fmaxf(mx[i], m[i]);
        use[i] = mx[i] == -INFINITY ? 0.f : mx[i];
        up |= mx[i] > m[i];
      }
      if (__any_sync(0xffffffffu, up)) {
        const float c0 = exp2f(m[0] - use[0]), c1 = exp2f(m[1] - use[1]);
        l[0] *= c0;
        l[1] *= c1;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= c0;
          o[i][1] *= c0;
          o[i][2] *= c1;
          o[i][3] *= c1;
        }
        m[0] = mx[0];
        m[1] = mx[1];
      }
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = pg_exp2(sc[nt][2 * i] - use[i]), p1 = pg_exp2(sc[nt][2 * i + 1] - use[i]);
          l[i] += p0 + p1;
          const uint32_t hi = pack2(p0, p1);
          ph[nt * 2 + i] = hi;
          pl[nt * 2 + i] = pack2(p0 - __uint_as_float(hi << 16),
                                 p1 - __uint_as_float(hi & 0xffff0000u));
        }
      {
        const int r = warp * 16 + (lane & 15);
        const uint32_t row = vs + r * 128;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const int ch = 2 * s + (lane >> 4);
          uint32_t vf[4];
          ldsm4t(row + (ch >> 3) * (kDcKeys * 128) + (((ch & 7) ^ (r & 7)) << 4), vf);
          mma16816(o[2 * s], ph, vf[0], vf[1]);
          mma16816(o[2 * s + 1], ph, vf[2], vf[3]);
          mma16816(o[2 * s], pl, vf[0], vf[1]);
          mma16816(o[2 * s + 1], pl, vf[2], vf[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == C::kStages) stage = 0, phase ^= 1u;
    }

    // ---- the four warps' parts of the segment, joined in shared memory ---------
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = g8 + i * 8;
      if (t4 == 0) {
        ml[(warp * kDcRows + r) * 2] = m[i];
        ml[(warp * kDcRows + r) * 2 + 1] = l[i];
      }
      float *dst = os + (warp * kDcRows + r) * C::kOS + t4 * 2;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2 *>(dst + c * 8) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
    }
    consumers_sync();
    const bool cut = seg.u1 - seg.u0 < seg.units;
    const int first = (int)(walk.item / hd.run);  // the pair's first and last run
    const int last_run = (int)((walk.item + seg.units - 1) / hd.run);
    const size_t per = (size_t)a.part_rows * D;
    float2 *pml = reinterpret_cast<float2 *>(a.part + (size_t)a.slot_cap * a.Hkv * per);
    const size_t slot = 2 * (size_t)blockIdx.x + (seg.u0 == 0 ? 1 : 0);
    auto store = [&](int r, int c, float4 acc, float mm, float ll) {
      const float inv = ll > 0.f ? 1.f / ll : 0.f;
      const size_t at = (size_t)(seg.row0 + r / G) * a.Hq + seg.h * G + r % G;
      uint2 pk;
      pk.x = pack2(acc.x * inv, acc.y * inv);
      pk.y = pack2(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2 *>(out + at * D + c * 4) = pk;
      if (a.lse && c == 0)
        a.lse[at] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
    };
    for (int i = tid; i < rows * (D / 4); i += 32 * kDcWarps) {
      const int r = i / (D / 4), c = i % (D / 4);
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDcWarps; ++w) mm = fmaxf(mm, ml[(w * kDcRows + r) * 2]);
      const float us = mm == -INFINITY ? 0.f : mm;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kDcWarps; ++w) {
        const float f = exp2f(ml[(w * kDcRows + r) * 2] - us);
        ll += ml[(w * kDcRows + r) * 2 + 1] * f;
        const float4 v =
            *reinterpret_cast<const float4 *>(os + (w * kDcRows + r) * C::kOS + c * 4);
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
      if (!cut) {
        store(r, c, acc, mm, ll);
      } else {
        *reinterpret_cast<float4 *>(a.part + slot * per + (size_t)r * D + c * 4) = acc;
        if (c == 0) pml[slot * a.part_rows + r] = make_float2(mm, ll);
      }
    }
    if (cut) {
      __threadfence();
      consumers_sync();
      if (tid == 0) *flag = atomicAdd(&a.arrive[first], 1u) == (uint32_t)(last_run - first);
      consumers_sync();
      if (*flag) {
        // this was the pair's last run to arrive: merge all of them, in order
        __threadfence();
        for (int i = tid; i < rows * (D / 4); i += 32 * kDcWarps) {
          const int r = i / (D / 4), c = i % (D / 4);
          float mm = -INFINITY;
#pragma unroll 8
          for (int w = first; w <= last_run; ++w)
            mm = fmaxf(mm, __ldcg(&pml[(2 * (size_t)w + (w == first)) * a.part_rows + r].x));
          const float us = mm == -INFINITY ? 0.f : mm;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float ll = 0.f;
#pragma unroll 8
          for (int w = first; w <= last_run; ++w) {
            const size_t s = 2 * (size_t)w + (w == first);
            const float2 e = __ldcg(&pml[s * a.part_rows + r]);
            const float4 v = __ldcg(
                reinterpret_cast<const float4 *>(a.part + s * per + (size_t)r * D + c * 4));
            const float f = exp2f(e.x - us);
            ll += e.y * f;
            acc.x += v.x * f;
            acc.y += v.y * f;
            acc.z += v.z * f;
            acc.w += v.w * f;
          }
          store(r, c, acc, mm, ll);
        }
      }
    }
    consumers_sync();
    walk.advance(a, seg);
  }
}

template <int D>
cudaError_t run(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  using C = DcCfg<D>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  auto kern = paged_decode_kernel<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int part = pg_part_rows(s.page, s.blocks, kDcKeys);
  CUtensorMap mk, mv;
  e = pg_cache_map(&mk, a.K, D, s.page, (long long)s.pages * s.Hkv, part);
  if (e == cudaSuccess) e = pg_cache_map(&mv, a.V, D, s.page, (long long)s.pages * s.Hkv, part);
  if (e != cudaSuccess) return e;
  const int grid = di.sm_count < kPagedMaxRuns ? di.sm_count : kPagedMaxRuns;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, paged_decode_schedule_kernel, a, grid);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kDcThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, kern, a, mk, mv, part);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_decode(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.d == 64 ? run<64>(s, a, st) : run<128>(s, a, st);
}

}  // namespace sd
