// paged_chunk_f32.cu -- paged attention in fp32 for blocks of many query rows:
// o_i = sum_j softmax(z_i)_j v_j, z_ij = <q_i, k_j> / sqrt(d) over the keys row i
// sees, one pass over the keys with a running maximum m and sum l (when a tile
// raises m, o and l are scaled by exp2(m_old - m_new)).
//
// Both products run on mma.sync m16n8k8 with every fp32 operand split in two
// tf32 parts, x = hi + lo (hi: x rounded to 11 significant bits, lo: the
// exact rest, of which the instruction keeps 11): a b ~ hi hi + hi lo + lo hi is
// off by about 2^-22 |a b|.  The instruction's own sums are cut, not rounded, so
// chains of them are kept short: the mixed products have accumulators of their
// own, and a tile's share of O starts from zero and is added to O (one chain
// over all keys was off by 3.9e-6 relative, this 4.2e-7).  Bound by those
// instructions, three for each product: a 256-token chunk of 8,192 at d = 128,
// 32 query heads over 8, takes 817 us (41 TFLOP/s; 1,265 with register-tiled
// multiply-adds), a 250-token chunk of 4,096 at d = 64, 8 over 2, 70 us.
//
// A worker (CTA) claims items of the schedule: a block of 128 query rows of one
// (sequence, KV head), 16 per warp, and a piece of its 64-key tiles.  K and V
// alternate: while one is used the other arrives (cp.async), in fp32 rows padded
// by 16 bytes, which leaves ldmatrix and the 16-byte reads free of bank
// conflicts.  The weights go from the accumulators of S straight into the
// operand of the second product: its inner index runs over the keys in the
// order 0 2 4 6 1 3 5 7, which is how a lane already holds them.  A piece of a
// cut range writes (O, m, l) to its slot, which the merge kernel joins in piece
// order.
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kCfKeys = 64;  // keys per tile
constexpr int kCfRows = 128;
constexpr int kCfThreads = 256;

template <int D>
struct CfCfg {
  static constexpr int kStride = D + 4;  // floats between rows
  static constexpr int kSmem = (kCfRows + 2 * kCfKeys) * kStride * 4 + 64 + kCfKeys;
};

__device__ __forceinline__ void cf_cp16(void *dst, const void *src, bool pred) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(pred ? 16u : 0u)
               : "memory");
}
__device__ __forceinline__ void cf_ldsm4(const float *p, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p))
               : "memory");
}
// x = hi + lo, hi x rounded to 11 significant bits (halves away from zero).
// Rounded, not cut: a cut leaves lo with the sign of x, and the lo lo that is
// dropped then adds up over the sum.  An addition and a mask; the conversion instruction would run on the slow special-function unit.
__device__ __forceinline__ void cf_split(float x, uint32_t *hi, uint32_t *lo) {
  *hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  *lo = __float_as_uint(x - __uint_as_float(*hi));
}
__device__ __forceinline__ void cf_mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// big + small += a b, a split already: hi hi in big, the two mixed products in
// small
__device__ __forceinline__ void cf_mma3(float *big, float *small, const uint32_t *ah,
                                        const uint32_t *al, float b0, float b1) {
  uint32_t h0, l0, h1, l1;
  cf_split(b0, &h0, &l0);
  cf_split(b1, &h1, &l1);
  cf_mma(small, ah, l0, l1);
  cf_mma(small, al, h0, h1);
  cf_mma(big, ah, h0, h1);
}

// Keys [key0, key0 + 64) of the sequence, those in [0, limit) that any row of
// the block sees (j >= low or j < sinks), into dst; zeros for the others and for
// pages outside the pool.  kok (nullable): which were read; *bad is set when one
// that should have been was not.
template <int D>
__device__ __forceinline__ void cf_load(float *dst, unsigned char *kok, int *bad,
                                        const float *cache, const PgArgs &a, const int *table,
                                        int h, int key0, int limit, int low) {
  constexpr int CPR = D / 4;  // 16-byte pieces of a row
  for (int p = threadIdx.x; p < kCfKeys * CPR; p += kCfThreads) {
    const int r = p / CPR, c = p % CPR, j = key0 + r;
    bool ok = j < limit && (j >= low || j < a.sinks);
    size_t off = 0;
    if (ok) {
      const int blk = a.by_page(j), pg = table[blk];
      ok = pg >= 0 && pg < a.pages;
      if (ok) {
        off = (((size_t)pg * a.Hkv + h) * a.page + j - blk * a.page) * D + c * 4;
      } else if (kok && c == 0) {
        raise_flag(a.status, FLAG_INDEX);
        *bad = 1;
      }
    }
    if (kok && c == 0) kok[r] = ok;
    cf_cp16(dst + r * CfCfg<D>::kStride + c * 4, cache + off, ok);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kCfThreads, 1)
    paged_chunk_f32_kernel(const __grid_constant__ PgArgs a) {
  constexpr int S = CfCfg<D>::kStride;
  extern __shared__ float cf_smem[];
  float *Qs = cf_smem, *Ks = Qs + kCfRows * S, *Vs = Ks + kCfKeys * S;
  int *box = reinterpret_cast<int *>(Vs + kCfKeys * S);  // the claimed item; arrival; bad pages
  unsigned char *kok = reinterpret_cast<unsigned char *>(box + 16);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int G = a.G, TB = kCfRows / G;
  const float *q = static_cast<const float *>(a.q), *K = static_cast<const float *>(a.K),
              *V = static_cast<const float *>(a.V);
  float *out = static_cast<float *>(a.out);
  if (tid == 0) box[1] = 0;
  grid_dep_wait();
  grid_dep_launch();
  const int per_head = a.seqs[a.B].base;

  for (bool first_item = true;; first_item = false) {
    if (tid == 0)
      box[0] = first_item ? (int)blockIdx.x : (int)min(atomicAdd(&a.head->next, 1u), 0x7fffffffu);
    __syncthreads();
    const long long item = box[0];
    __syncthreads();
    if (item >= (long long)per_head * a.Hkv) break;
    const int h = (int)(item / per_head), x = (int)(item % per_head);
    PgSeq sq;
    const int b = pg_find(a.seqs, a.B, x, &PgSeq::base, &sq);
    int row0, n, kv;
    pg_lengths(a, b, &row0, &n, &kv);
    const int nrb = (n + TB - 1) / TB;
    // piece-major, the longest ranges first
    const int piece = (x - sq.base) / nrb, rb = nrb - 1 - (x - sq.base) % nrb;
    const int t0 = rb * TB, t1 = min(n, t0 + TB), rows = (t1 - t0) * G;
    const int p_first = kv - n + t0, p_last = kv - n + t1 - 1;
    const PgTiles tiles = pg_tiles(p_first, p_last, a.window, a.sinks, kCfKeys);
    const int u0 = piece * sq.len, u1 = min(tiles.units(), u0 + sq.len);
    const int limit = p_last + 1, low = pg_window_low(p_first, a.window);
    const int low_last = pg_window_low(p_last, a.window);
    const int *table = a.table + (size_t)b * a.blocks;
    if (u0 < u1) cf_load<D>(Ks, kok, box + 1, K, a, table, h, tiles.tile(u0) * kCfKeys, limit, low);
    auto place = [&](int r) {  // of row r of the block, in q and out
      return (size_t)(row0 + t0 + a.by_G(r)) * a.Hq + h * G + r - a.by_G(r) * G;
    };
    for (int p = tid; p < kCfRows * (D / 4); p += kCfThreads) {
      const int r = p / (D / 4), c = p % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = *reinterpret_cast<const float4 *>(q + (size_t)(row0 + t0 + a.by_G(r)) * a.q_stride +
                                              (size_t)(h * G + r - a.by_G(r) * G) * D + c * 4);
      *reinterpret_cast<float4 *>(Qs + r * S + c * 4) = v;
    }
    // this lane's rows: g8 and g8 + 8 of the warp's 16
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
    int pos[2], lowr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = warp * 16 + g8 + 8 * i;
      pos[i] = r < rows ? p_first + a.by_G(r) : -1;
      lowr[i] = pg_window_low(pos[i], a.window);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const bool live = warp * 16 < rows;  // warps without rows only help with the copies

    for (int u = u0; u < u1; ++u) {
      const int key0 = tiles.tile(u) * kCfKeys;
      cf_load<D>(Vs, nullptr, nullptr, V, a, table, h, key0, limit, low);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      float s[kCfKeys / 8][4];
      if (live) {
#pragma unroll
        for (int i = 0; i < kCfKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
        float low4[kCfKeys / 8][4] = {};
        const float *qrow = Qs + (warp * 16 + (lane & 15)) * S + (lane >> 4) * 4;
        const float *krow = Ks + (((lane >> 4) << 3) + (lane & 7)) * S + ((lane >> 3) & 1) * 4;
#pragma unroll 2
        for (int k = 0; k < D; k += 8) {
          uint32_t x4[4], ah[4], al[4];
          cf_ldsm4(qrow + k, x4);
#pragma unroll
          for (int i = 0; i < 4; ++i) cf_split(__uint_as_float(x4[i]), &ah[i], &al[i]);
#pragma unroll
          for (int nt = 0; nt < kCfKeys / 16; ++nt) {
            uint32_t kf[4];
            cf_ldsm4(krow + nt * 16 * S + k, kf);
            cf_mma3(s[2 * nt], low4[2 * nt], ah, al, __uint_as_float(kf[0]), __uint_as_float(kf[1]));
            cf_mma3(s[2 * nt + 1], low4[2 * nt + 1], ah, al, __uint_as_float(kf[2]),
                    __uint_as_float(kf[3]));
          }
        }
#pragma unroll
        for (int nt = 0; nt < kCfKeys / 8; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] += low4[nt][e];
        const bool whole = key0 + kCfKeys - 1 <= p_first &&
                           (key0 >= low_last || key0 + kCfKeys <= a.sinks) &&
                           *(volatile int *)(box + 1) == 0;
        if (!whole) {
#pragma unroll
          for (int nt = 0; nt < kCfKeys / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = nt * 8 + t4 * 2 + (e & 1), j = key0 + r, i = e >> 1;
              const bool see =
                  j <= pos[i] && (j >= lowr[i] || j < a.sinks) && kok[r];
              if (!see) s[nt][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < kCfKeys / 8; ++nt)
            mx = fmaxf(mx, fmaxf(s[nt][2 * i], s[nt][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx = fmaxf(mx * a.scale_log2, m[i]);
          const float use = mx == -INFINITY ? 0.f : mx, corr = exp2f(m[i] - use);
          m[i] = mx;
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < kCfKeys / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p = pg_exp2(fmaf(s[nt][2 * i + e], a.scale_log2, -use));
              sum += p;
              s[nt][2 * i + e] = p;
            }
          l[i] = l[i] * corr + sum;
          if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              o[c][2 * i] *= corr;
              o[c][2 * i + 1] *= corr;
            }
          }
        }
      }
      __syncthreads();  // K is used up
      if (u + 1 < u1)
        cf_load<D>(Ks, kok, box + 1, K, a, table, h, tiles.tile(u + 1) * kCfKeys, limit, low);
      else
        asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();  // V has landed
      if (live) {
        // keys 8 kt + 2 t4, + 1; columns 32 cb + 4 g8 + j are column g8 of the
        // instruction for accumulator 4 cb + j
        const float *vrow = Vs + t4 * 2 * S + g8 * 4;
        uint32_t ah[kCfKeys / 8][4], al[kCfKeys / 8][4];
#pragma unroll
        for (int kt = 0; kt < kCfKeys / 8; ++kt) {
          cf_split(s[kt][0], &ah[kt][0], &al[kt][0]);
          cf_split(s[kt][2], &ah[kt][1], &al[kt][1]);
          cf_split(s[kt][1], &ah[kt][2], &al[kt][2]);
          cf_split(s[kt][3], &ah[kt][3], &al[kt][3]);
        }
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          float big[4][4] = {}, small[4][4] = {};
#pragma unroll
          for (int kt = 0; kt < kCfKeys / 8; ++kt) {
            const float4 v0 = *reinterpret_cast<const float4 *>(vrow + kt * 8 * S + cb * 32);
            const float4 v1 = *reinterpret_cast<const float4 *>(vrow + (kt * 8 + 1) * S + cb * 32);
            cf_mma3(big[0], small[0], ah[kt], al[kt], v0.x, v1.x);
            cf_mma3(big[1], small[1], ah[kt], al[kt], v0.y, v1.y);
            cf_mma3(big[2], small[2], ah[kt], al[kt], v0.z, v1.z);
            cf_mma3(big[3], small[3], ah[kt], al[kt], v0.w, v1.w);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[cb * 4 + j][e] += big[j][e] + small[j][e];
        }
      }
      __syncthreads();  // V is used up
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    const size_t per = (size_t)a.part_rows * D;
    const size_t mine = (size_t)(sq.slot + rb * sq.np + piece) * a.Hkv + h;  // its partial
    float2 *ml = reinterpret_cast<float2 *>(a.part + (size_t)a.slot_cap * a.Hkv * per);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = warp * 16 + g8 + 8 * i;
      if (r >= rows) continue;
      const bool whole = sq.np == 1;
      const float f = whole ? pg_inverse(l[i]) : 1.f;
      float *dst = whole ? out + place(r) * D : a.part + mine * per + (size_t)r * D;
#pragma unroll
      for (int cb = 0; cb < D / 32; ++cb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4 *>(dst + cb * 32 + t4 * 8 + e * 4) =
              make_float4(o[cb * 4][2 * i + e] * f, o[cb * 4 + 1][2 * i + e] * f,
                          o[cb * 4 + 2][2 * i + e] * f, o[cb * 4 + 3][2 * i + e] * f);
      if (t4 == 0) {
        if (!whole) ml[mine * a.part_rows + r] = make_float2(m[i], l[i]);
        else if (a.lse) a.lse[place(r)] = pg_lse(m[i], l[i]);
      }
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t run(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  using C = CfCfg<D>;
  auto kern = paged_chunk_f32_kernel<D>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = di.sm_count;  // two CTAs an SM would halve the registers (78 us at d = 64)
  // a tile takes 6 (d = 64) or 12 us, starting a piece or merging one a few
  if ((e = launch_paged_schedule(s, a, kCfRows / s.G(), kCfKeys, grid, 1, 4, st)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kCfThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  cfg.attrs = attrs;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  if ((e = cudaLaunchKernelEx(&cfg, kern, a)) != cudaSuccess) return e;
  return launch_paged_merge(s, a, kCfRows / s.G(), st);
}

}  // namespace

cudaError_t launch_paged_chunk_f32(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.d == 64 ? run<64>(s, a, st) : run<128>(s, a, st);
}

}  // namespace sd
