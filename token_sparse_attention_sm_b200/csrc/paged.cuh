// paged.cuh -- what the kernels over a paged K/V cache share: the arguments,
// which keys a block of query rows sees, and the schedule of a call (how the
// rows of a ragged batch are cut into work items), which one small kernel
// derives on the device from the sequences' lengths.
//
// A new token i of sequence b stands at position p = kv_len[b] - n[b] + i and
// sees key j when 0 <= j <= p and, under a window w, j > p - w or j < sinks.
// Query rows of one KV head are (token, query head of the group) pairs,
// token-major: row r of a block of TB tokens is token r / G, head r % G, so
// the G heads that share a KV head share every key tile read.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "common.cuh"

namespace sd {

// One sequence's part of the schedule, written by the schedule kernel.
struct PgSeq {
  int base;  // work items (per KV head) before this sequence
  int slot;  // partial slots (per KV head) before this sequence
  int np;    // pieces its key range is cut into (1: no partials)
  int len;   // key tiles per piece
};
// The schedule in the workspace: header, then PgSeq[B + 1] (the last one
// holds the totals).
struct PgHead {
  uint32_t next;  // claim counter of the work items after each worker's first
  uint32_t pad[15];
};

// Division of n in [0, 2^31) by a divisor the host knows: the multiplier is
// floor(2^(31+s) / d) + 1 with 2^(s-1) < d <= 2^s, whose error stays below one
// part in 2^31 of the quotient's unit.
struct PgDiv {
  uint32_t mul;
  int shift;  // s - 1; -1: d = 1
  __device__ __forceinline__ int operator()(int n) const {
    return shift < 0 ? n : (int)(__umulhi((uint32_t)n, mul) >> shift);
  }
};
inline PgDiv pg_divisor(uint32_t d) {
  int s = 0;
  while ((1u << s) < d) ++s;
  return s == 0 ? PgDiv{0, -1} : PgDiv{(uint32_t)(((1ull << (31 + s)) / d) + 1), s - 1};
}

struct PgArgs {
  const void *q, *K, *V;
  const int *table, *q_start, *kv_lens;
  void *out;
  float *lse;
  long long q_stride;  // elements between the tokens of q
  int G;            // Hq / Hkv
  PgDiv by_G, by_page;
  int B, T, Hq, Hkv, page, pages, blocks, window, sinks, max_new;
  float scale_log2;
  uint32_t *status;
  // schedule and partials (workspace)
  PgHead *head;
  PgSeq *seqs;
  // decode: arrivals, zero between calls
  uint32_t *runs;    // [kPagedMaxRuns] of a pair's runs, or its first group's, at its first run
  uint32_t *groups;  // [kPagedMaxRuns] of another group's runs, at the group's first run
  uint32_t *tops;    // [kPagedTops] of a pair's groups
  float *part;       // [slot_cap * Hkv][part_rows][d] then [..][part_rows] (max, sum)
  int slot_cap;      // partial slots per KV head
  int part_rows;
};

// pairs of fp32 values in one 64-bit register, and packed arithmetic on them
__device__ __forceinline__ uint64_t pg_u2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pg_f2(float lo, float hi) {
  return pg_u2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ void pg_split(uint64_t x, float *lo, float *hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x));
  *lo = __uint_as_float(a);
  *hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t pg_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pg_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pg_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x by the hardware approximation (relative error about 2^-22; results
// below 2^-126 flush to zero, which a softmax weight does not notice).
__device__ __forceinline__ float pg_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a row's sum of weights l makes of its O, and its lse (m: its reference
// in log2 units).  l is 0 when the row sees nothing; a score that is NaN or
// +inf leaves l NaN, and that stays in both.
__device__ __forceinline__ float pg_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float pg_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// The key tiles a block of tokens [t0, t1) of a sequence reads: tiles
// [0, sink_tiles) and [lo, hi), KT keys each.
struct PgTiles {
  int sink_tiles, lo, hi;
  __device__ int units() const { return sink_tiles + hi - lo; }
  __device__ int tile(int u) const { return u < sink_tiles ? u : u - sink_tiles + lo; }
};

// bits 0 .. n-1 of a word
__device__ __forceinline__ uint32_t pg_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// The first key that the window leaves a row at position p (0: no window).
__device__ __forceinline__ int pg_window_low(int p, int window) {
  const long long lo = (long long)p - window + 1;
  return window > 0 && lo > 0 ? (int)lo : 0;
}

__device__ __forceinline__ PgTiles pg_tiles(int p_first, int p_last, int window, int sinks,
                                            int KT) {
  PgTiles t;
  const int hi = max(p_last + 1, 0);
  const int lo = pg_window_low(p_first, window);
  t.hi = (hi + KT - 1) / KT;
  t.lo = min(lo / KT, t.hi);
  t.sink_tiles = min((min(sinks, hi) + KT - 1) / KT, t.lo);
  return t;
}

// A sequence's lengths as given, or false if they make no sense (the schedule
// kernel reports that).
__device__ __forceinline__ bool pg_lengths(const PgArgs &a, int b, int *row0, int *n, int *kv) {
  const int s = a.q_start[b], e = a.q_start[b + 1], c = a.kv_lens[b];
  *row0 = s;
  *n = e - s;
  *kv = c;
  return s >= 0 && e >= s && e <= a.T && c >= 0 && e - s <= a.max_new &&
         (long long)c <= (long long)a.blocks * a.page;
}

// The sequence (and its schedule entry) that work item (`of` = &PgSeq::base) or
// partial slot (&PgSeq::slot) x of a head is in: the last one that starts at x or
// before.  One warp, 32 probes a round.
__device__ __forceinline__ int pg_find(const PgSeq *seqs, int B, int x, int PgSeq::*of,
                                       PgSeq *out) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // seqs[lo] starts at x or before, seqs[lo + n] after it
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = min(lo + lane * step, lo + n);
    const bool le = seqs[at].*of <= x && at < lo + n;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = __popc(m) - 1;
    const int nlo = lo + k * step;
    n = min(step, lo + n - nlo);
    lo = nlo;
  }
  *out = seqs[lo];
  return lo;
}

// Merges the np partials of `rows` rows from row0 on, in piece order, by nt
// threads; out and lse get the result.  slot0 is the first piece's partial,
// the others follow a.Hkv apart; at(row) is a row's place in out [T, Hq].
// Several elements and pieces are loaded together: row by row, one piece after
// another, this was a tail of 80 us (13 pieces of 64 rows).
// E: elements a thread has in flight.
template <int D, int E, typename T, typename At>
__device__ __forceinline__ void pg_merge(const PgArgs &a, size_t slot0, int np, int row0, int rows,
                                         int tid, int nt, At at, T *out) {
  constexpr int P = 4;  // pieces at a time
  const size_t per = (size_t)a.part_rows * D;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part + (size_t)a.slot_cap * a.Hkv * per);
  const int total = rows * (D / 4);
  for (int i0 = tid; i0 < total; i0 += E * nt) {
    float m[E], l[E];
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.f;
      acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int p0 = 0; p0 < np; p0 += P) {
      float2 x[E][P];
      float4 v[E][P];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = min(i0 + e * nt, total - 1), row = row0 + i / (D / 4), c = i % (D / 4);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const size_t s = slot0 + (size_t)min(p0 + p, np - 1) * a.Hkv;
          x[e][p] = __ldcg(&ml[s * a.part_rows + row]);
          v[e][p] = __ldcg(
              reinterpret_cast<const float4 *>(a.part + s * per + (size_t)row * D + c * 4));
          if (p0 + p >= np) x[e][p] = make_float2(-INFINITY, 0.f);
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float top = m[e];
#pragma unroll
        for (int p = 0; p < P; ++p) top = fmaxf(top, x[e][p].x);
        const float use = top == -INFINITY ? 0.f : top, corr = exp2f(m[e] - use);
        m[e] = top;
        l[e] *= corr;
        acc[e].x *= corr;
        acc[e].y *= corr;
        acc[e].z *= corr;
        acc[e].w *= corr;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float f = exp2f(x[e][p].x - use);
          l[e] += x[e][p].y * f;
          acc[e].x += v[e][p].x * f;
          acc[e].y += v[e][p].y * f;
          acc[e].z += v[e][p].z * f;
          acc[e].w += v[e][p].w * f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = i0 + e * nt;
      if (i >= total) break;
      const size_t o = at(row0 + i / (D / 4));
      const int c = i % (D / 4);
      const float inv = pg_inverse(l[e]);
      alignas(16) T r[4] = {DT<T>::from_f(acc[e].x * inv), DT<T>::from_f(acc[e].y * inv),
                DT<T>::from_f(acc[e].z * inv), DT<T>::from_f(acc[e].w * inv)};
      using Vec = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
      *reinterpret_cast<Vec *>(out + o * D + c * 4) = *reinterpret_cast<const Vec *>(r);
      if (a.lse && c == 0) a.lse[o] = pg_lse(m[e], l[e]);
    }
  }
}

}  // namespace sd
