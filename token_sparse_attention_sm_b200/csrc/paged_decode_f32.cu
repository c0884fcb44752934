// paged_decode_f32.cu -- the decode kernels' arithmetic in fp32, on the CUDA
// cores.  A warp has a tile of 32 keys to itself: for S a lane is a key (its
// row read in 16-byte pieces, the queries' pieces broadcast), for O a lane is
// four columns (at d = 64 half the lanes take every other key), with P passed
// through a line of shared memory per row.  At R rows a tile costs 2 * 32 * d *
// R / 32 multiply-adds per lane, below the time HBM needs for it up to 8 rows,
// about equal at 16.  A row's reference maximum moves only when the maximum has
// left it by more than 2^8 (the weights and sums are fp32), so most tiles need
// a vote instead of a reduction.
//
// Measured: one sequence of 32,768 tokens over 8 KV heads at d = 128, 54 us
// (4.9 TB/s);
// 16 ragged sequences of up to 8,192 over 2 at d = 64, 24 us.
#include "paged_decode.cuh"

namespace sd {
namespace {

// R: query rows kept
template <int D, int R>
struct DcFma {
  using Elem = float;
  static constexpr int kD = D, kKeys = 32, kRows = R;
  static constexpr int kWarps = R == 4 ? 6 : R == 8 ? 5 : 4;
  static constexpr int kPairs = 1;
  static constexpr int kThreads = 32 * (kWarps + 2 * kPairs);
  static constexpr int kTile = kKeys * D * 4;
  static constexpr int kStages = (D == 128 ? 1 : 2) * kWarps;  // a stage belongs to one warp
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kOS = D + 4;
  static constexpr int kOBytes = kWarps * kRows * kOS * 4;
  static constexpr int kScratch = R * D * 4 + kWarps * R * kKeys * 4;  // Q; P of a tile per warp
  static constexpr int kSmem = kRing + kOBytes + kScratch + 1024 + 1024;
  static_assert(kSmem <= 227 * 1024, "fits an SM");
  static constexpr float kLag = 8.f;

  float4 o[R];
  float m[R], l[R];
  int p_first, rows;
  const float *q;
  float *p;

  template <typename Sync>
  __device__ __forceinline__ void begin(const PgArgs &a, const DcSeg &seg, int n_rows,
                                        unsigned char *scratch, Sync sync) {
    float *qs = reinterpret_cast<float *>(scratch);
    q = qs;
    p = qs + R * D + (threadIdx.x >> 5) * R * kKeys;
    p_first = seg.p_first;
    rows = n_rows;
    const float *src = static_cast<const float *>(a.q);
    for (int i = threadIdx.x; i < R * (D / 4); i += 32 * kWarps) {
      const int r = i / (D / 4), c = i % (D / 4), tok = a.by_G(r);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = *reinterpret_cast<const float4 *>(src + (size_t)(seg.row0 + tok) * a.q_stride +
                                              (size_t)(seg.h * a.G + r - tok * a.G) * D + c * 4);
      reinterpret_cast<float4 *>(qs)[i] = v;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    sync();  // Q is there; the segment before has been merged
  }

  __device__ __forceinline__ void tile(const PgArgs &a, const PgTile &tl, uint32_t ks, uint32_t vs,
                                       int key0, bool whole, uint32_t ok, int part_log) {
    const int lane = threadIdx.x & 31;
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 0.f;
    {
      const uint32_t row = ks + (lane >> 3) * tl.group + (lane & 7) * 128;
#pragma unroll
      for (int cb = 0; cb < D / 32; ++cb)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 k = lds4(row + cb * tl.col + ((c ^ (lane & 7)) << 4));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float4 x = *reinterpret_cast<const float4 *>(q + r * D + cb * 32 + c * 4);
            s[r] = fmaf(x.x, k.x, s[r]);
            s[r] = fmaf(x.y, k.y, s[r]);
            s[r] = fmaf(x.z, k.z, s[r]);
            s[r] = fmaf(x.w, k.w, s[r]);
          }
        }
    }
    bool raise = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] *= a.scale_log2;
      if (!whole) {
        const int j = key0 + lane, pos = r < rows ? p_first + a.by_G(r) : -1;
        const bool see = j <= pos && (j >= pg_window_low(pos, a.window) || j < a.sinks) &&
                         ((ok >> (lane >> part_log)) & 1u);
        if (!see) s[r] = -INFINITY;
      }
      raise |= s[r] > m[r] + kLag || (m[r] == -INFINITY && s[r] > m[r]);
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float top = fmaxf(m[r], warp_max(s[r]));
        const float corr = top == -INFINITY ? 1.f : exp2f(m[r] - top);
        m[r] = top;
        l[r] *= corr;
        o[r].x *= corr;
        o[r].y *= corr;
        o[r].z *= corr;
        o[r].w *= corr;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float w = exp2f(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
      l[r] += w;
      p[r * kKeys + lane] = w;
    }
    __syncwarp();
    // lanes' columns: 4 * (lane % (D / 4)); at d = 64 the upper half of the
    // warp has the odd groups of four keys
    constexpr int L = D / 4;
    const int col = lane % L, odd = lane / L;
    const uint32_t at = vs + (col >> 3) * tl.col;
#pragma unroll
    for (int k0 = 0; k0 < kKeys; k0 += 4 * (32 / L)) {
      const int kb = k0 + 4 * odd;
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = kb + i;
        v[i] = lds4(at + (key >> 3) * tl.group + (key & 7) * 128 +
                    (((col & 7) ^ (key & 7)) << 4));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 w = *reinterpret_cast<const float4 *>(p + r * kKeys + kb);
        fma4(o[r], w.x, v[0]);
        fma4(o[r], w.y, v[1]);
        fma4(o[r], w.z, v[2]);
        fma4(o[r], w.w, v[3]);
      }
    }
    __syncwarp();  // P is used up
  }

  __device__ __forceinline__ void join(float *os, float *ml) {
    const int lane = threadIdx.x & 31;
    constexpr int L = D / 4;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float sum = warp_sum(l[r]);
      if (L < 32) {
        o[r].x += __shfl_xor_sync(0xffffffffu, o[r].x, 16);
        o[r].y += __shfl_xor_sync(0xffffffffu, o[r].y, 16);
        o[r].z += __shfl_xor_sync(0xffffffffu, o[r].z, 16);
        o[r].w += __shfl_xor_sync(0xffffffffu, o[r].w, 16);
      }
      if (lane < L) *reinterpret_cast<float4 *>(os + r * kOS + lane * 4) = o[r];
      if (lane == 0) {
        ml[r * 2] = m[r];
        ml[r * 2 + 1] = sum;
      }
    }
  }

  static __device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
  }
  static __device__ __forceinline__ void fma4(float4 &o, float w, const float4 &v) {
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
};

template <int D>
cudaError_t pick(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  const int rows = s.max_new * s.G();
  if (rows <= 4) return dc_run<DcFma<D, 4>>(s, a, st);
  return rows <= 8 ? dc_run<DcFma<D, 8>>(s, a, st) : dc_run<DcFma<D, 16>>(s, a, st);
}

}  // namespace

cudaError_t launch_paged_decode_f32(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.d == 64 ? pick<64>(s, a, st) : pick<128>(s, a, st);
}

}  // namespace sd
