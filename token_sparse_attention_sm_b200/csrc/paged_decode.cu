// paged_decode.cu -- the decode kernels' arithmetic in bf16, on mma.sync
// m16n8k16 in the transposed form S^T = K Q^T, O^T += V^T P^T: the queries are
// the instruction's 8 columns, so up to 8 rows cost half of what padding them
// to the 16 (or 128) rows of the other operand would, P^T only changes lanes
// (an 8x8 transpose) between the two products, and nothing leaves the
// registers.  P is split in two bf16 parts (P_hi + P_lo: 16 significant bits),
// which costs little where memory is the limit.
//
// Measured: 16 ragged sequences of up to 65,536 tokens over 8 KV heads at
// d = 128, 380-390 us, 6.8-6.9 TB/s of K and V (the copy rate, reads and writes,
// is 6.6); one sequence of 131,072 tokens, 88-90 us.
#include "paged_decode.cuh"

namespace sd {
namespace {

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
// the transpose of an 8x8 block of 16-bit values held by the warp (lane: row
// lane / 4, columns 2 (lane % 4), + 1)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// NT: groups of 8 query rows
template <int D, int NT>
struct DcMma {
  using Elem = __nv_bfloat16;
  static constexpr int kD = D, kKeys = 64;
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = kKeys * D * 2;  // K or V of a tile
  static constexpr int kWarps = NT == 1 ? 6 : 4;  // consumer warps
  // pairs of producer warps: d = 64 tiles are half as long and as many copies
  // (16-token pages at d = 64: 34.2 -> 30.2 us for 64 windows of 4,095 tokens;
  // at d = 128 the registers of two more warps cost more than they bring)
  static constexpr int kPairs = D == 64 || NT == 2 ? 2 : 1;
  static constexpr int kThreads = 32 * (kWarps + 2 * kPairs);
  // a multiple of the consumer warps: a stage's tiles all belong to one warp,
  // which has then seen every phase of the stage's barrier before the next (a
  // parity wait is only sound one phase ahead)
  static constexpr int kStages = (D == 128 ? 1 : 2) * kWarps;
  static_assert(kStages % kPairs == 0, "and to one pair of producers");
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kOS = D + 4;              // floats between rows of O
  static constexpr int kOBytes = kWarps * kRows * kOS * 4;
  static constexpr int kScratch = 0;
  static constexpr int kSmem = kRing + kOBytes + kScratch + 1024 + 1024;  // + small, alignment
  static_assert(kSmem <= 227 * 1024, "fits an SM");

  // Q as the B operand: query 8 nt + g8, elements 16 s + 2 t4, + 8
  uint32_t qf[NT][D / 16][2];
  int pos[NT][2], low[NT][2];  // of queries 8 nt + 2 t4, + 1
  // O^T: row 16 dt + g8 (+ 8) of V's columns, queries 8 nt + 2 t4, + 1
  float o[D / 16][NT][4], m[NT][2], l[NT][2];

  template <typename Sync>
  __device__ __forceinline__ void begin(const PgArgs &a, const DcSeg &seg, int rows,
                                        unsigned char *, Sync) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3, G = a.G;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + t4 * 2 + e;
        pos[nt][e] = r < rows ? seg.p_first + a.by_G(r) : -1;
        low[nt][e] = pg_window_low(pos[nt][e], a.window);
      }
      const int r = nt * 8 + g8;
      const uint32_t *src =
          r < rows ? reinterpret_cast<const uint32_t *>(
                         q + (size_t)(seg.row0 + a.by_G(r)) * a.q_stride +
                         (size_t)(seg.h * G + r - a.by_G(r) * G) * D)
                   : nullptr;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[nt][s][0] = src ? src[s * 8 + t4] : 0u;
        qf[nt][s][1] = src ? src[s * 8 + t4 + 4] : 0u;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const PgArgs &a, const PgTile &tl, uint32_t ks, uint32_t vs,
                                       int key0, bool whole, uint32_t ok, int part_log) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2;
    // S^T = K Q^T: keys 16 mt + g8 (+ 8), queries 8 nt + 2 t4, + 1
    constexpr int MT = kKeys / 16;
    float sc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        sc[i][nt][0] = sc[i][nt][1] = sc[i][nt][2] = sc[i][nt][3] = 0.f;
    {
      const uint32_t row = ks + ((lane >> 3) & 1) * tl.group + (lane & 7) * 128;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const int ch = 2 * s + (lane >> 4);
        const uint32_t at = row + (ch >> 3) * tl.col + (((ch & 7) ^ (lane & 7)) << 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t kf[4];
          ldsm4(at + mt * 2 * tl.group, kf);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(sc[mt][nt], kf, qf[nt][s][0], qf[nt][s][1]);
        }
      }
    }
    if (!whole) {
      // the keys a row sees, a bit each
      uint32_t pages[2];
#pragma unroll
      for (int w = 0; w < 2; ++w)
        pages[w] = ((ok >> ((32 * w) >> part_log)) & 1u ? 0xffffu : 0u) |
                   ((ok >> ((32 * w + 16) >> part_log)) & 1u ? 0xffff0000u : 0u);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int hi = pos[nt][e] - key0, lo = low[nt][e] - key0, sk = a.sinks - key0;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t see = pg_below(hi + 1 - 32 * w) &
                           (~pg_below(lo - 32 * w) | pg_below(sk - 32 * w)) & pages[w];
            see >>= g8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((see >> (8 * i)) & 1u)) sc[2 * w + (i >> 1)][nt][(i & 1) * 2 + e] = -INFINITY;
          }
        }
    }
    float use[NT][2];
    bool up = false;
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) x = fmaxf(x, fmaxf(sc[mt][nt][e], sc[mt][nt][2 + e]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        mx[nt][e] = fmaxf(x * a.scale_log2, m[nt][e]);
        use[nt][e] = mx[nt][e] == -INFINITY ? 0.f : mx[nt][e];
        up |= mx[nt][e] > m[nt][e];
      }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float c0 = exp2f(m[nt][0] - use[nt][0]), c1 = exp2f(m[nt][1] - use[nt][1]);
        l[nt][0] *= c0;
        l[nt][1] *= c1;
        m[nt][0] = mx[nt][0];
        m[nt][1] = mx[nt][1];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][nt][0] *= c0;
          o[i][nt][1] *= c1;
          o[i][nt][2] *= c0;
          o[i][nt][3] *= c1;
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // P^T of 16 keys as the B operand: 8x8 blocks transposed between lanes
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = pg_exp2(fmaf(sc[mt][nt][2 * i], a.scale_log2, -use[nt][0]));
          const float p1 = pg_exp2(fmaf(sc[mt][nt][2 * i + 1], a.scale_log2, -use[nt][1]));
          l[nt][0] += p0;
          l[nt][1] += p1;
          const uint32_t hi = pack2(p0, p1);
          ph[nt][i] = transpose8(hi);
          pl[nt][i] = transpose8(pack2(p0 - __uint_as_float(hi << 16),
                                       p1 - __uint_as_float(hi & 0xffff0000u)));
        }
      // O^T += V^T P^T
      const uint32_t row = vs + (2 * mt + (lane >> 4)) * tl.group + (lane & 7) * 128;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        const int ch = 2 * dt + ((lane >> 3) & 1);
        uint32_t vf[4];
        ldsm4t(row + (ch >> 3) * tl.col + (((ch & 7) ^ (lane & 7)) << 4), vf);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[dt][nt], vf, ph[nt][0], ph[nt][1]);
          mma16816(o[dt][nt], vf, pl[nt][0], pl[nt][1]);
        }
      }
    }
  }

  // rows 0 .. kRows-1 of this warp
  __device__ __forceinline__ void join(float *os, float *ml) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = nt * 8 + t4 * 2 + e;
        if (g8 == 0) {
          ml[r * 2] = m[nt][e];
          ml[r * 2 + 1] = sum;
        }
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          os[r * kOS + dt * 16 + g8] = o[dt][nt][e];
          os[r * kOS + dt * 16 + g8 + 8] = o[dt][nt][2 + e];
        }
      }
  }
};

template <int D>
cudaError_t pick(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.max_new * s.G() <= 8 ? dc_run<DcMma<D, 1>>(s, a, st) : dc_run<DcMma<D, 2>>(s, a, st);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.d == 64 ? pick<64>(s, a, st) : pick<128>(s, a, st);
}

}  // namespace sd
