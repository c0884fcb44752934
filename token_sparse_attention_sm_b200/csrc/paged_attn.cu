// paged_attn.cu -- attention of new tokens over a paged fp32 cache on the CUDA
// cores: o_i = sum_j softmax(z_i)_j v_j, z_ij = <q_i, k_j> / sqrt(d) over the
// keys row i sees, one pass over the keys with a running maximum m and sum l
// (when a tile raises m, o and l are scaled by exp2(m_old - m_new)).
//
// A worker (CTA) claims items of the schedule: a block of RB query rows of
// one (sequence, KV head) and a piece of its key tiles.  Each tile of 64 keys
// is copied into shared memory, K for S = Q K^T and V for O += P V
// in turn, the next tile's K arriving while V is used and the other way round.
// Thread (ty, tx) holds rows ty*RT .. and keys tx + TX*j of S, then columns of
// O; a row's TX threads are in one warp, so its maximum and sum are warp
// shuffles.  A piece of a cut range writes (O, m, l) to its slot; the last
// piece of the block to arrive merges them in piece order.
#include "paged.h"
#include "paged.cuh"

namespace sd {
namespace {

constexpr int kKT = 64;  // keys per tile

template <int D, int RB>
struct SimtCfg {
  static constexpr int TX = 16;
  static constexpr int RT = 8;             // rows per thread
  static constexpr int kThreads = RB / RT * TX;
  static constexpr int NK = kKT / TX;      // keys per thread
  static constexpr int NC = D / TX;        // columns per thread
  static constexpr int PS = kKT;           // row stride of P, in floats
  static constexpr int kBlocks = D == 64 ? 3 : 2;  // per SM: shared memory's limit
  static constexpr int kFloats = RB * D + 2 * kKT * D + RB * PS;
  static constexpr int kSmem = kFloats * 4 + 64 + kKT;  // + the claimed item, key flags
  static_assert(NC % 4 == 0, "16-byte reads of V");
};

__device__ __forceinline__ void cp16(void *dst, const void *src, bool pred) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(pred ? 16u : 0u)
               : "memory");
}

// keys [key0, key0 + 64) of the sequence, those in [0, limit) that any row of
// the block sees (j >= low or j < sinks), into dst as fp32 rows; zeros for
// the others and for pages outside the pool.  SWIZZLE: 16-byte pieces permuted by
// row, so that a column of 8 rows is free of bank conflicts.  kok (nullable): which were read.
template <int D, bool SWIZZLE, int THREADS>
__device__ __forceinline__ void load_tile(float *dst, unsigned char *kok, const float *cache,
                                          const PgArgs &a, const int *table, int h, int key0,
                                          int limit, int low) {
  constexpr int PER = 4;  // elements of a 16-byte piece
  constexpr int CPR = D / PER;
  for (int p = threadIdx.x; p < kKT * CPR; p += THREADS) {
    const int r = p / CPR, c = p % CPR;
    const int j = key0 + r;
    bool ok = j < limit && (j >= low || j < a.sinks);
    size_t off = 0;
    if (ok) {
      const int blk = a.by_page(j), pg = table[blk];
      ok = pg >= 0 && pg < a.pages;
      if (ok) off = (((size_t)pg * a.Hkv + h) * a.page + j - blk * a.page) * D + c * PER;
      else if (c == 0) raise_flag(a.status, FLAG_INDEX);
    }
    if (kok && c == 0) kok[r] = ok;
    cp16(dst + r * D + (SWIZZLE ? c ^ (r & 7) : c) * PER, cache + off, ok);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int D, int RB>
__global__ void __launch_bounds__(SimtCfg<D, RB>::kThreads, SimtCfg<D, RB>::kBlocks)
    paged_attn_simt_kernel(const PgArgs a) {
  using C = SimtCfg<D, RB>;
  constexpr int TX = C::TX, RT = C::RT, NK = C::NK, NC = C::NC, PS = C::PS;
  constexpr int THREADS = C::kThreads;
  extern __shared__ float sm[];
  float *Qs = sm, *Ks = Qs + RB * D, *Vs = Ks + kKT * D, *Ps = Vs + kKT * D;
  int *box = reinterpret_cast<int *>(Ps + RB * PS);
  unsigned char *kok = reinterpret_cast<unsigned char *>(box + 16);
  const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
  const int G = a.G, TB = RB / G;
  const float *q = static_cast<const float *>(a.q), *K = static_cast<const float *>(a.K),
              *V = static_cast<const float *>(a.V);
  float *out = static_cast<float *>(a.out);
  grid_dep_wait();
  grid_dep_launch();
  const int per_head = a.seqs[a.B].base;

  for (;;) {
    if (tid == 0) box[0] = (int)min(atomicAdd(&a.head->next, 1u), 0x7fffffffu);
    __syncthreads();
    const long long item = box[0];
    __syncthreads();
    if (item >= (long long)per_head * a.Hkv) break;
    const int h = (int)(item / per_head), x = (int)(item % per_head);
    PgSeq sq;
    const int b = pg_find(a.seqs, a.B, x, &sq);
    int row0, n, kv;
    pg_lengths(a, b, &row0, &n, &kv);
    const int nrb = (n + TB - 1) / TB;
    // piece-major, the longest ranges first
    const int piece = (x - sq.base) / nrb, rb = nrb - 1 - (x - sq.base) % nrb;
    const int t0 = rb * TB, t1 = min(n, t0 + TB), rows = (t1 - t0) * G;
    const int p_first = kv - n + t0, p_last = kv - n + t1 - 1;
    const PgTiles tiles = pg_tiles(p_first, p_last, a.window, a.sinks, kKT);
    const int u0 = piece * sq.len, u1 = min(tiles.units(), u0 + sq.len);
    const int limit = p_last + 1, low = pg_window_low(p_first, a.window);
    const int *table = a.table + (size_t)b * a.blocks;

    for (int p = tid; p < RB * (D / 4); p += THREADS) {
      const int r = p / (D / 4), c = p % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const float *src = q + (size_t)(row0 + t0 + a.by_G(r)) * a.q_stride + (h * G + r - a.by_G(r) * G) * D + c * 4;
        v = *reinterpret_cast<const float4 *>(src);
      }
      *reinterpret_cast<float4 *>(Qs + r * D + c * 4) = v;
    }
    float m[RT], l[RT];
    uint64_t o[RT][NC / 2];  // pairs of columns
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) o[i][c] = 0ull;
    }
    int pos[RT], lowr[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = ty * RT + i;
      pos[i] = r < rows ? p_first + a.by_G(r) : -1;
      lowr[i] = pg_window_low(pos[i], a.window);
    }
    if (u0 < u1)
      load_tile<D, true, THREADS>(Ks, kok, K, a, table, h, tiles.tile(u0) * kKT, limit, low);
    for (int u = u0; u < u1; ++u) {
      const int key0 = tiles.tile(u) * kKT;
      load_tile<D, false, THREADS>(Vs, nullptr, V, a, table, h, key0, limit, low);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      // S, even and odd elements of the rows in the two halves of a pair
      uint64_t s2[RT][NK];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NK; ++j) s2[i][j] = 0ull;
#pragma unroll 4
      for (int k = 0; k < D; k += 4) {
        ulonglong2 qv[RT], kv4[NK];
#pragma unroll
        for (int i = 0; i < RT; ++i)
          qv[i] = *reinterpret_cast<const ulonglong2 *>(Qs + (ty * RT + i) * D + k);
#pragma unroll
        for (int j = 0; j < NK; ++j)
          kv4[j] = *reinterpret_cast<const ulonglong2 *>(Ks + (tx + TX * j) * D +
                                                         (k ^ ((tx & 7) << 2)));
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < NK; ++j) {
            s2[i][j] = pg_fma2(qv[i].x, kv4[j].x, s2[i][j]);
            s2[i][j] = pg_fma2(qv[i].y, kv4[j].y, s2[i][j]);
          }
      }
      float s[RT][NK];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          float even, odd;
          pg_split(s2[i][j], &even, &odd);
          s[i][j] = even + odd;
        }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const int key = key0 + tx + TX * j;
          const bool see =
              key <= pos[i] && (key >= lowr[i] || key < a.sinks) && kok[tx + TX * j];
          s[i][j] = see ? s[i][j] * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int w = TX / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float use = mx == -INFINITY ? 0.f : mx;
        const float corr = exp2f(m[i] - use);
        m[i] = mx;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const float p = pg_exp2(s[i][j] - use);
          sum += p;
          Ps[(ty * RT + i) * PS + tx + TX * j] = p;
        }
        l[i] = l[i] * corr + sum;
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) o[i][c] = pg_mul2(o[i][c], pg_f2(corr, corr));
      }
      __syncthreads();  // K is used up, P complete
      if (u + 1 < u1)
        load_tile<D, true, THREADS>(Ks, kok, K, a, table, h, tiles.tile(u + 1) * kKT, limit, low);
      else
        asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();  // V has landed
#pragma unroll 2
      for (int k = 0; k < kKT; k += 4) {
        float4 pv[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i)
          pv[i] = *reinterpret_cast<const float4 *>(Ps + (ty * RT + i) * PS + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint64_t v[NC / 2];
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(
                Vs + (k + kk) * D + (c / 4) * (TX * 4) + tx * 4);
            v[c / 2] = x.x;
            v[c / 2 + 1] = x.y;
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float p = kk == 0 ? pv[i].x : kk == 1 ? pv[i].y : kk == 2 ? pv[i].z : pv[i].w;
            const uint64_t pp = pg_f2(p, p);
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) o[i][c] = pg_fma2(pp, v[c], o[i][c]);
          }
        }
      }
      __syncthreads();  // V and P are used up
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the row's sum over its threads
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int w = TX / 2; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);

    if (sq.np == 1) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int r = ty * RT + i;
        if (r >= rows) continue;
        const size_t tok = (size_t)(row0 + t0 + a.by_G(r)), hq = h * G + r - a.by_G(r) * G;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          ulonglong2 x;
          x.x = pg_mul2(o[i][c / 2], pg_f2(inv, inv));
          x.y = pg_mul2(o[i][c / 2 + 1], pg_f2(inv, inv));
          *reinterpret_cast<ulonglong2 *>(out + (tok * a.Hq + hq) * D + (c / 4) * (TX * 4) +
                                          tx * 4) = x;
        }
        if (a.lse && tx == 0)
          a.lse[tok * a.Hq + hq] =
              l[i] > 0.f ? (m[i] + log2f(l[i])) * 0.69314718055994531f : -INFINITY;
      }
    } else {
      const size_t first = (size_t)(sq.slot + rb * sq.np) * a.Hkv;  // slots (piece, head)
      const size_t per = (size_t)a.part_rows * D;
      float2 *ml = reinterpret_cast<float2 *>(a.part + (size_t)a.slot_cap * a.Hkv * per);
      const size_t mine = first + (size_t)piece * a.Hkv + h;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int r = ty * RT + i;
        if (r >= rows) continue;
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          ulonglong2 x;
          x.x = o[i][c / 2];
          x.y = o[i][c / 2 + 1];
          *reinterpret_cast<ulonglong2 *>(a.part + mine * per + (size_t)r * D +
                                          (c / 4) * (TX * 4) + tx * 4) = x;
        }
        if (tx == 0) ml[mine * a.part_rows + r] = make_float2(m[i], l[i]);
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) box[0] = atomicAdd(&a.arrive[first + h], 1u) == (uint32_t)(sq.np - 1);
      __syncthreads();
      const bool last = box[0] != 0;
      __syncthreads();
      if (last) {
        __threadfence();
        pg_merge<D, 4>(a, first + h, sq.np, 0, rows, tid, THREADS,
                    [&](int r) {
                      return (size_t)(row0 + t0 + a.by_G(r)) * a.Hq + h * G + r - a.by_G(r) * G;
                    },
                    out);
      }
    }
    __syncthreads();
  }
}

template <int D, int RB>
cudaError_t run(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  using C = SimtCfg<D, RB>;
  auto kern = paged_attn_simt_kernel<D, RB>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  int per_sm = 1;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, C::kThreads, C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = di.sm_count * (per_sm < 1 ? 1 : per_sm);
  if ((e = launch_paged_schedule(s, a, RB / s.G(), kKT, grid, st)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attrs[1];
  cfg.attrs = attrs;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, kern, a);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_attn_simt(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.d == 64 ? run<64, 64>(s, a, st) : run<128, 64>(s, a, st);
}

}  // namespace sd
