// paged_chunk.cu -- paged attention in bf16 for blocks of many query rows (a
// prompt's chunk; any batch whose sequences may have more than 16 rows per KV
// head): S = Q K^T and O += P V on the 5th-generation tensor cores.
//
// One persistent CTA per SM claims items of the schedule: a block of up to
// 256 query rows of one (sequence, KV head) -- two tiles of 128, row r of a
// tile being token r / G, head r % G -- and a piece of its 128-key tiles.
// Both row tiles use every K and V tile, which halves what one reads from L2
// (at 128 rows the tile loads alone would ask for more than L2 gives).
//
// Roles (384 threads):
//  * two TMA warps, one of which claims the items and copies Q, stream K and V
//    tiles through one ring (one copy per page and tile, 128-byte swizzle);
//  * a warp per row tile issues its MMAs: S_t = Q_t K^T (M = N = 128) and
//    O_t += P_t V, P_t read from tensor memory;
//  * four softmax warps per row tile, one row per thread: S from tensor
//    memory, the row's maximum, P = exp2(S scale - m) rounded to bf16 over the
//    dead S, in two halves so that the product starts on the first, and O
//    scaled when the maximum moves.
// A row tile is one chain, scores - softmax - product - scores; the two tiles'
// chains run side by side, and each has its own issuing warp so that neither
// waits behind the other's waits.  Tensor memory: S_0, S_1, O_0, O_1 (512
// columns at d = 128).  (Two 64-key S buffers per row tile took the turn-round
// out of the chain but cost more: M = 128, N = 64 reads as much of Q for half
// the work, 725 against 904 TFLOP/s on a 2,048-token chunk of 32K.)
//
// The reference m of a row is only raised when the running maximum has left it
// by more than 2^8: weights then reach 256 instead of 1, the sums stay fp32,
// the division at the end cancels m, and O is almost never rescaled.
// P is rounded to bf16 (at most 2^-8 of a weight, independent errors that the
// sum over keys averages; the result is rounded to bf16 anyway); its sum is
// taken before the rounding.
//
// A step of 128 keys takes about 4,100 cycles for two row tiles, of which the
// MMAs need 2,000 and the exponentials 2,048: the chains' latencies are the
// limit, 895-908 TFLOP/s on full blocks (d = 128).  Taking a quarter of the
// exponentials on the FMA pipe, sixteen softmax warps with half a row each, or
// interleaving the softmax by 32 keys all came out slower (887, 889, 886).
//
// Every wait is bounded; when one runs out the kernel raises TIMEOUT, all
// roles leave their loops, the tensor memory is freed and the kernel returns.
#include "paged.h"
#include "paged.cuh"
#include "paged_tma.h"

namespace sd {
namespace {

constexpr int kChKeys = 128;
constexpr int kChSoftWarps = 8;
constexpr int kChThreads = 384;  // three warpgroups: two of softmax warps; MMA and copies
// registers a thread: 168 at launch, moved from the third warpgroup to the
// softmax ones (2 * 128 * 216 + 128 * 72 = 384 * 168)
constexpr int kChSoftRegs = 216, kChOtherRegs = 72;
constexpr int kChMmaWarp = kChSoftWarps, kChTmaWarp = kChSoftWarps + 2;  // row tiles' MMA; K, V
constexpr float kChLag = 8.f;  // log2 units the maximum may run ahead of its reference

template <int D>
struct ChCfg {
  static constexpr int CB = D / 64;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kTile = kChKeys * D * 2;  // K or V of a tile: one ring slot
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kQOff = 0, kRingOff = 2 * kQTile;
  static constexpr int kSmallOff = kRingOff + kSlots * kTile;
  static constexpr int kShareOff = kSmallOff + 1024;  // (max, sum) of 128 rows
  static constexpr int kSmem = kShareOff + 1024 + 1024;  // + alignment slack
  static_assert(kSmem <= 227 * 1024, "fits an SM");
};

// A block of one row tile only has its key tiles shared out between the two
// chains (even and odd ones, both with the first row tile's queries) if there
// are this many, and their results joined at the end.
constexpr int kChAlternate = 4;

// One work item, as the TMA warp found it.
struct ChItem {
  int b, h, row0, t0, rows;            // rows: query rows of the block
  int p_first, p_last, low;            // positions of its first and last token; lowest key of a window
  int u0, u1;                          // the piece's tiles
  int sink_tiles, lo;
  int np, piece, first;                // partial slots: (first + piece) * Hkv + h
  int valid;                           // 0: no more items
};

struct ChSmall {
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_ready[2][2], pv_done[2], o_empty[2], wg[2], pair;  // p_ready: half a tile each
  uint64_t item_full[2], item_empty[2];
  ChItem item[2];
  uint32_t ok[8];
  uint32_t tmem, abort, last[2];
};
static_assert(sizeof(ChSmall) <= 1024, "small area");

// ---- tcgen05 ------------------------------------------------------------------
__device__ __forceinline__ void ch_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void ch_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void ch_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void ch_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void ch_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void ch_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// shared-memory matrix descriptor, 128-byte swizzle (sm_100 version)
__device__ __forceinline__ uint64_t ch_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, bf16 operands, fp32 accumulator, M = 128
__host__ __device__ constexpr uint32_t ch_idesc(int N, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void ch_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A in tensor memory: lane = row, two bf16 per column
__device__ __forceinline__ void ch_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void ch_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void ch_tma(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                       uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint4 lds128_at(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ch_join(uint32_t x, float fx, uint32_t y, float fy) {
  return __float_as_uint(__uint_as_float(x) * fx + __uint_as_float(y) * fy);
}
// one lane of a converged warp, always the same
__device__ __forceinline__ bool ch_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
// a value that is the same in all lanes of a converged warp
template <typename T>
__device__ __forceinline__ T ch_uniform(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}
__device__ __forceinline__ uint32_t ch_pack(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// Wait for a phase; false once any wait of the CTA has run out.
__device__ __forceinline__ bool ch_wait(uint64_t *bar, uint32_t parity, ChSmall *sm,
                                        uint32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  volatile uint32_t *abort = &sm->abort;
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      raise_flag(status, FLAG_TIMEOUT);
      *abort = 1u;
      return false;
    }
  }
  return true;
}

// ALT: blocks of one row tile use both chains
template <int D, bool ALT>
__global__ void __launch_bounds__(kChThreads, 1)
    paged_chunk_kernel(const PgArgs a, const __grid_constant__ CUtensorMap mapQ,
                       const __grid_constant__ CUtensorMap mapK,
                       const __grid_constant__ CUtensorMap mapV, const PgTile tl) {
  using C = ChCfg<D>;
  extern __shared__ unsigned char raw[];
  const uint32_t raw_s = smem_u32(raw);
  const uint32_t base = (raw_s + 1023u) & ~1023u;
  ChSmall *sm = reinterpret_cast<ChSmall *>(raw + (base - raw_s) + C::kSmallOff);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.G, TPT = 128 / G, TB = 2 * TPT;  // tokens per row tile, per block

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm->tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    sm->abort = 0;
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], 2);  // both row tiles
    }
    mbar_init(&sm->q_full, 1);
    mbar_init(&sm->q_empty, 2);
    mbar_init(&sm->pair, kChSoftWarps);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm->s_full[t], 1);
      mbar_init(&sm->p_ready[t][0], 4);
      mbar_init(&sm->p_ready[t][1], 4);
      mbar_init(&sm->pv_done[t], 1);
      mbar_init(&sm->o_empty[t], 4);
      mbar_init(&sm->wg[t], 4);
      mbar_init(&sm->item_full[t], 1);
      mbar_init(&sm->item_empty[t], kChSoftWarps + 3);
    }
    fence_mbar_init();
    pg_prefetch_map(&mapQ);
    pg_prefetch_map(&mapK);
    pg_prefetch_map(&mapV);
  }
  ch_fence_before();
  __syncthreads();
  ch_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = sm->tmem;

  if (warp >= kChSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChOtherRegs));
    if (warp == kChTmaWarp || warp == kChTmaWarp + 1) {
      // ---- TMA warps: items, Q and K; V ---------------------------------------------
      const bool isV = warp != kChTmaWarp;
      const CUtensorMap *map = isV ? &mapV : &mapK;
      const int per_head = a.seqs[a.B].base;
      const long long total = (long long)per_head * a.Hkv;
      const int nparts = kChKeys / tl.part, per = 32 / nparts;
      int slot = isV, unit = 0, q_count = 0;  // K and V take the ring's slots in turn
      uint32_t phase = 0;
      bool alive = true;
      for (int it = 0; alive; ++it) {
        ChItem &I = sm->item[it & 1];
        if (isV) {
          if (!__all_sync(0xffffffffu,
                          ch_wait(&sm->item_full[it & 1], (it >> 1) & 1, sm, a.status)))
            break;
        } else {
          uint32_t x = blockIdx.x;
          if (lane == 0 && it > 0) x = atomicAdd(&a.head->next, 1u);
          x = __shfl_sync(0xffffffffu, x, 0);
          if (!__all_sync(0xffffffffu,
                          ch_wait(&sm->item_empty[it & 1], ((it >> 1) & 1) ^ 1, sm, a.status)))
            break;
          const bool valid = x < total;
          if (valid) {
            const int y = (int)(x % (uint32_t)per_head);
            PgSeq sq;
            const int b = pg_find(a.seqs, a.B, y, &sq);
            if (lane == 0) {
              int row0, n, kv;
              pg_lengths(a, b, &row0, &n, &kv);
              const int nrb = (n + TB - 1) / TB;
              // piece-major, the blocks with the longest ranges first
              const int piece = (y - sq.base) / nrb, rb = nrb - 1 - (y - sq.base) % nrb;
              const int t0 = rb * TB, t1 = min(n, t0 + TB);
              const int p_first = kv - n + t0, p_last = kv - n + t1 - 1;
              const PgTiles t = pg_tiles(p_first, p_last, a.window, a.sinks, kChKeys);
              I.b = b;
              I.h = (int)(x / (uint32_t)per_head);
              I.row0 = row0;
              I.t0 = t0;
              I.rows = (t1 - t0) * G;
              I.p_first = p_first;
              I.p_last = p_last;
              I.low = pg_window_low(p_first, a.window);
              I.sink_tiles = t.sink_tiles;
              I.lo = t.lo;
              I.u0 = min(piece * sq.len, t.units());
              I.u1 = min(t.units(), I.u0 + sq.len);
              I.np = sq.np;
              I.piece = piece;
              I.first = sq.slot + rb * sq.np;
            }
          }
          if (lane == 0) {
            I.valid = valid;
            mbar_arrive(&sm->item_full[it & 1]);
          }
          __syncwarp();
        }
        const int valid = I.valid, u0 = I.u0, u1 = I.u1, h = I.h, low = I.low;
        const int limit = I.p_last + 1, sink_tiles = I.sink_tiles, lo = I.lo, b = I.b;
        const int rows = I.rows, q_row = I.row0 + I.t0;
        __syncwarp();
        if (isV && lane == 0) mbar_arrive(&sm->item_empty[it & 1]);
        if (!valid) break;
        if (u0 >= u1) continue;
        if (!isV) {  // Q: the block's one or two row tiles
          if (!__all_sync(0xffffffffu, ch_wait(&sm->q_empty, (q_count & 1) ^ 1, sm, a.status)))
            break;
          ++q_count;
          if (lane == 0) {
            const int tiles = rows > TPT * G ? 2 : 1;
            mbar_arrive_expect_tx(&sm->q_full, tiles * C::CB * TPT * G * 128);
            for (int t = 0; t < tiles; ++t)
              for (int c = 0; c < C::CB; ++c)
                ch_tma(base + C::kQOff + t * C::kQTile + c * (128 * 128), &mapQ, c * 64, h * G,
                       q_row + t * TPT, &sm->q_full);
          }
          __syncwarp();
        }
        const int *table = a.table + (size_t)b * a.blocks;
        // lane i: where part i % nparts of tile ub + i / nparts is (token of its
        // page, page * Hkv + head); past the pool (zeros) if it is not read
        int y, z;
        bool bad;
        auto fetch = [&](int ub) {
          const int u = ub + lane / nparts;
          int yy = 0, zz = a.pages * a.Hkv;
          bool bb = false;
          if (u < u1) {
            const int j0 = (u < sink_tiles ? u : u - sink_tiles + lo) * kChKeys +
                           (lane % nparts) * tl.part;
            if (j0 < limit && (j0 + tl.part > low || j0 < a.sinks)) {
              const int blk = a.by_page(j0), e = table[blk];
              if (e >= 0 && e < a.pages) {
                yy = j0 - blk * a.page;
                zz = e * a.Hkv + h;
              } else {
                if (isV) raise_flag(a.status, FLAG_INDEX);
                bb = true;
              }
            }
          }
          y = yy;
          z = zz;
          bad = bb;
        };
        fetch(u0);
        for (int ub = u0; ub < u1 && alive; ub += per) {
          const int cy = y, cz = z;
          const uint32_t cbad = __ballot_sync(0xffffffffu, bad);
          fetch(ub + per);
          for (int u = ub; u < min(u1, ub + per); ++u) {
            const int src = (u - ub) * nparts + lane % nparts;
            const int ty = __shfl_sync(0xffffffffu, cy, src);
            const int tz = __shfl_sync(0xffffffffu, cz, src);
            if (!__all_sync(0xffffffffu, ch_wait(&sm->empty[slot], phase ^ 1u, sm, a.status))) {
              alive = false;
              break;
            }
            if (lane == 0) {
              if (isV) {  // one bit per 16 keys; the softmax waits for V before it looks
                uint32_t ok16 = 0;
                const uint32_t bits = cbad >> ((u - ub) * nparts);
                for (int i = 0; i < kChKeys / 16; ++i)
                  ok16 |= (~(bits >> (i * 16 / tl.part)) & 1u) << i;
                sm->ok[unit & 7] = ok16;
              }
              mbar_arrive_expect_tx(&sm->full[slot], C::kTile);
            }
            __syncwarp();
            if (lane < nparts)
              pg_tma_part(base + C::kRingOff + slot * C::kTile + lane * tl.part * (D * 2), map, tl,
                          ty, tz, &sm->full[slot]);
            __syncwarp();
            slot += 2;
            if (slot >= C::kSlots) slot -= C::kSlots, phase ^= 1u;
            ++unit;
          }
        }
      }
      // this warp's copies have landed before it leaves, whatever happened (the
      // last kSlots positions of the ring: an older slot has moved on)
      for (int at = 2 * unit - 2 + isV; at >= max(0, 2 * unit - C::kSlots); at -= 2)
        mbar_wait(&sm->full[at % C::kSlots], (at / C::kSlots) & 1, a.status);
    } else {
      // ---- MMA warps, one per row tile: all lanes walk, one issues ---------------------
      // (The walk stays uniform and the issue under elect.sync, so the operands
      // live in uniform registers: issued from a divergent lane 0, with each
      // descriptor moved over on its own, an instruction took about 100 cycles.)
      const int t = warp - kChMmaWarp;
      constexpr uint32_t idS = ch_idesc(kChKeys, false), idPV = ch_idesc(D, true);
      const bool lead = ch_elect();
      const uint32_t tS = ch_uniform(tmem + t * 128), tO = ch_uniform(tmem + 256 + t * 128);
      const uint64_t q_own = ch_desc(ch_uniform(base + C::kQOff + t * C::kQTile), 16, 1024);
      const uint64_t q_first = ch_desc(ch_uniform(base + C::kQOff), 16, 1024);
      const uint32_t ring = ch_uniform(base + C::kRingOff);
      const uint32_t kcol = tl.col / 16, vstep = 2 * tl.group / 16;  // 16-byte units
      int slot = 0;  // ring position of the next tile
      uint32_t phase = 0, q_count = 0, pv_cnt = 0, o_cnt = 0;
      auto step = [&]() {
        if (++slot == C::kSlots) slot = 0, phase ^= 1u;
      };
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ch_wait(bar, parity & 1u, sm, a.status)) != 0;
      };
      // S of the K tile in the ring's next slot, which it frees
      auto scores = [&](uint64_t q, bool last) {
        const uint64_t k = ch_desc(ch_uniform(ring + slot * C::kTile), 16, tl.group);
        if (lead) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            ch_mma_ss(tS, q + ((s >> 2) * (128 * 128) + (s & 3) * 32) / 16,
                      k + (s >> 2) * kcol + (s & 3) * 2, idS, s > 0);
          ch_commit(&sm->s_full[t]);
          ch_commit(&sm->empty[slot]);
          if (last) ch_commit(&sm->q_empty);
        }
        __syncwarp();
        step();
      };
      bool ok = true;
      for (int it = 0; ok; ++it) {
        if (!(ok = wait(&sm->item_full[it & 1], it >> 1))) break;
        const ChItem &I = sm->item[it & 1];
        const int valid = ch_uniform(I.valid), n = ch_uniform(I.u1 - I.u0);
        const bool two = ch_uniform(I.rows) > TPT * G;  // row tiles
        __syncwarp();
        if (lead) mbar_arrive(&sm->item_empty[it & 1]);
        if (!valid) break;
        if (n <= 0) continue;
        const bool alt = ALT && !two && n >= kChAlternate;
        if (!(ok = wait(&sm->q_full, q_count++))) break;
        // a ring slot that only the other row tile's chain uses
        auto skip = [&]() {
          ok = wait(&sm->full[slot], phase);
          if (lead) mbar_arrive(&sm->empty[slot]);
          __syncwarp();
          step();
        };
        if (t == 1 && !two && !alt) {
          for (int j = 0; j < 2 * n && ok; ++j) skip();
          if (lead) mbar_arrive(&sm->q_empty);
          __syncwarp();
          continue;
        }
        // turns: this chain has every other key tile, from its own number on
        auto chain = [&](auto turns) {
          constexpr bool kTurns = decltype(turns)::value;
          const uint64_t q = kTurns ? q_first : q_own;
          if (kTurns && t == 1) {
            skip();
            if (ok) skip();
            if (!ok) return;
          }
          // (the last P of the item before was used up: its end was waited for)
          if (!(ok = wait(&sm->full[slot], phase))) return;
          ch_fence_after();
          // (in turns, the queries' space is freed by the first chain's scores and,
          // once it has served to join the results, by the softmax)
          const bool frees_q = !(kTurns && t == 1);
          scores(q, frees_q && (kTurns ? n <= 2 : n == 1));
          for (int j = kTurns ? t : 0; j < n; j += kTurns ? 2 : 1) {
            if (!(ok = wait(&sm->full[slot], phase))) return;
            if (j == (kTurns ? t : 0) && o_cnt++ > 0)  // O of the item before was read
              if (!(ok = wait(&sm->o_empty[t], o_cnt - 2))) return;
            const uint64_t v = ch_desc(ch_uniform(ring + slot * C::kTile), tl.col, tl.group);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!(ok = wait(&sm->p_ready[t][h], pv_cnt))) return;
              ch_fence_after();
              if (lead) {
#pragma unroll
                for (int kk = h * 4; kk < h * 4 + 4; ++kk)
                  ch_mma_ts(tO, tS + kk * 8, v + kk * vstep, idPV,
                            kk > 0 ? 1u : (uint32_t)(j > (kTurns ? t : 0)));
              }
              __syncwarp();
            }
            if (lead) {
              ch_commit(&sm->pv_done[t]);
              ch_commit(&sm->empty[slot]);
            }
            __syncwarp();
            step();
            if (kTurns && j + 1 < n) {
              skip();
              if (ok) skip();
              if (!ok) return;
            }
            const int next = j + (kTurns ? 2 : 1);
            if (next < n && !(ok = wait(&sm->full[slot], phase))) return;
            // S overwrites the P that the product just issued reads
            if (!(ok = wait(&sm->pv_done[t], pv_cnt++))) return;
            if (next < n) {
              ch_fence_after();
              scores(q, frees_q && next + (kTurns ? 2 : 1) >= n);
            }
          }
        };
        if constexpr (ALT) {
          if (alt) chain(std::true_type{});
          else chain(std::false_type{});
        } else {
          chain(std::false_type{});
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChSoftRegs));
    // ---- softmax warps: tile t, one row per thread -----------------------------------
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + 256 + t * 128;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    int ring = 0;  // ring position of the next K tile, and the phase of its round
    uint32_t phase = 0, s_cnt = 0, wg_cnt = 0;
    int unit = 0;
    bool ok = true;
    constexpr uint32_t all_ok = (1u << (kChKeys / 16)) - 1u;
    auto step = [&]() {
      if (++ring == C::kSlots) ring = 0, phase ^= 1u;
    };
    // (max, sum) of a row from the other chain; the space of the second row
    // tile's queries, for its O
    float2 *share = reinterpret_cast<float2 *>(raw + (base - raw_s) + C::kShareOff);
    uint32_t pair_cnt = 0;
    auto pair_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->pair);
      const bool w = ch_wait(&sm->pair, pair_cnt & 1, sm, a.status);
      ++pair_cnt;
      return __all_sync(0xffffffffu, w) != 0;
    };
    // the four warps of the tile meet (bounded)
    auto wg_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->wg[t]);
      const bool w = ch_wait(&sm->wg[t], wg_cnt & 1, sm, a.status);
      ++wg_cnt;
      return w;
    };
    for (int it = 0;; ++it) {
      if (!ch_wait(&sm->item_full[it & 1], (it >> 1) & 1, sm, a.status)) break;
      const ChItem &I = sm->item[it & 1];  // until this warp's arrival below
      auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->item_empty[it & 1]);
      };
      if (!I.valid) break;
      const int n = max(0, I.u1 - I.u0), tile_rows = TPT * G;
      const bool alt = ALT && I.rows <= tile_rows && n >= kChAlternate;
      if (t == 1 && I.rows <= tile_rows && !alt) {  // nothing here: keep count of the ring
        for (int j = 0; j < n; ++j) step(), step();
        unit += n;
        done();
        continue;
      }
      const int rt = alt ? 0 : t;           // row tile
      const int br = rt * tile_rows + r;  // row of the block
      const bool live = r < tile_rows && br < I.rows;
      const int pos = live ? I.p_first + a.by_G(br) : -1;
      const int low = pg_window_low(pos, a.window);
      const int pf = I.p_first + rt * TPT, pl = min(I.p_last, pf + TPT - 1);  // the tile's tokens
      const int low_last = pg_window_low(pl, a.window);
      float m = -INFINITY, l = 0.f;
      bool begun = false;  // a tile of this item has been through this chain
      for (int j = 0; j < n; ++j) {
        if (alt && (j & 1) != t) {
          step(), step();
          ++unit;
          continue;
        }
        const int u = I.u0 + j;
        const int key0 = (u < I.sink_tiles ? u : u - I.sink_tiles + I.lo) * kChKeys;
        step();
        const int vslot = ring;
        const uint32_t vphase = phase;
        step();
        ok = ch_wait(&sm->s_full[t], s_cnt & 1, sm, a.status);
        ++s_cnt;
        // also orders this after the TMA warp's note on the tile's pages
        if (ok) ok = ch_wait(&sm->full[vslot], vphase, sm, a.status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ch_fence_after();
        const uint32_t good = sm->ok[unit & 7];
        ++unit;
        if (key0 + kChKeys > I.p_last + 1 || (key0 < I.low && key0 + kChKeys > a.sinks)) {
          // V rows that no row of the block sees may hold anything: clear them
          // (each tile's warps before its own product; both write zeros)
          const int key = key0 + r;
          if (key > I.p_last || (key < I.low && key >= a.sinks)) {
            const uint32_t v =
                base + C::kRingOff + vslot * C::kTile + (r >> 3) * tl.group + (r & 7) * 128;
#pragma unroll
            for (int c = 0; c < C::CB; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                                 v + c * tl.col + ((i + r) & 7) * 16),
                             "r"(0u)
                             : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        const bool whole = key0 + kChKeys - 1 <= pf &&
                           (key0 >= low_last || key0 + kChKeys <= a.sinks) && good == all_ok;
        uint32_t s[128], p[32];
        uint64_t sum2[2];
        const uint64_t scale2 = pg_f2(a.scale_log2, a.scale_log2);
        // weights of keys 64 c .. 64 c + 63 against the reference m
        auto weights = [&](int c, bool fresh) {
          const float use = m == -INFINITY ? 0.f : m;
          const uint64_t neg2 = pg_f2(-use, -use);
          if (fresh) sum2[0] = sum2[1] = 0ull;  // pairs of zeros
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int k = c * 64 + i * 2;
            float p0, p1;
            pg_split(pg_fma2(pg_u2(s[k], s[k + 1]), scale2, neg2), &p0, &p1);
            p0 = pg_exp2(p0);
            p1 = pg_exp2(p1);
            sum2[i & 1] = pg_add2(sum2[i & 1], pg_f2(p0, p1));
            p[i] = ch_pack(p0, p1);
          }
        };
        // four accumulators, each block's maximum while the next one is read
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        ch_ld32(tS, s);
        ch_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) ch_ld32(tS + (c + 1) * 32, s + (c + 1) * 32);
          if (!whole) {
            // the row's keys of the block, a bit each
            const int hi = pos - key0, lo = low - key0, sk = a.sinks - key0;
            const uint32_t pages = ((good >> (2 * c)) & 1u ? 0xffffu : 0u) |
                                   ((good >> (2 * c)) & 2u ? 0xffff0000u : 0u);
            const uint32_t see = pg_below(hi + 1 - 32 * c) &
                                 (~pg_below(lo - 32 * c) | pg_below(sk - 32 * c)) & pages;
            // (most blocks of an edge tile are seen whole by all of the warp's rows)
            if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1u)) s[c * 32 + i] = 0xff800000u;
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(s[c * 32 + i]));
          if (c < 3) ch_wait_ld();
        }
        // the first half's weights do not wait for the maximum: the reference
        // rarely moves, and if it does they are taken again (after the first
        // tile, which always sets it)
        if (begun) weights(0, true);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
        const bool raise = mx > m + kChLag || (m == -INFINITY && mx > m);
        if (!begun || __any_sync(0xffffffffu, raise)) {
          const float mn = raise ? mx : m;
          const float corr = raise ? exp2f(m - mn) : 1.f;  // 0 for the first tile
          m = mn;
          l *= corr;
          if (begun) {
            // the product before has finished: S of this tile came after it
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              ch_ld32(tO + c * 32, p);
              ch_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) p[i] = __float_as_uint(__uint_as_float(p[i]) * corr);
              ch_st32(tO + c * 32, p);
            }
          }
          weights(0, true);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 1) weights(1, false);
          ch_st32(tS + c * 32, p);
          ch_wait_st();
          ch_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->p_ready[t][c]);
        }
        begun = true;
        float a0, a1;
        pg_split(pg_add2(sum2[0], sum2[1]), &a0, &a1);
        l += a0 + a1;
      }
      if (!ok) break;
      // ---- the piece's result ----------------------------------------------------------
      if (n > 0) {
        // every product of the item is done when its last one is
        ok = ch_wait(&sm->pv_done[t], (s_cnt - 1) & 1, sm, a.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        ch_fence_after();
      }
      // In turns: the second chain hands its O over in two halves of the columns,
      // through the space of the second row tile's queries.
      float own = 1.f, other = 0.f;  // factors of the two chains' O
      const uint32_t xrow = base + C::kQOff + C::kQTile + r * (D * 2);
      auto xaddr = [&](int i) { return xrow + ((i + r) & (D / 8 - 1)) * 16; };  // 16-byte pieces
      if (alt && t == 1) {
        share[r] = make_float2(m, l);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half == 1 && !(ok = pair_sync())) break;  // the first half has been read
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            ch_ld32(tO + half * (D / 2) + c * 32, o);
            ch_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(xaddr(c * 8 + i)),
                           "r"(o[4 * i]), "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                           : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          if (!(ok = pair_sync())) break;  // this half is there
        }
        if (!ok) break;
        ch_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->o_empty[t]);
        if (!(ok = pair_sync())) break;  // both have been read
        done();
        continue;
      }
      if (alt) {
        if (!(ok = pair_sync())) break;  // the other's first half is there
        const float2 e = share[r];
        const float top = fmaxf(m, e.x), use = top == -INFINITY ? 0.f : top;
        own = exp2f(m - use);
        other = exp2f(e.x - use);
        m = top;
        l = l * own + e.y * other;
      }
      const size_t at =
          (size_t)(I.row0 + I.t0 + a.by_G(br)) * a.Hq + I.h * G + br - a.by_G(br) * G;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const size_t per = (size_t)a.part_rows * D;
      const size_t first = (size_t)I.first * a.Hkv + I.h;
      const size_t mine = first + (size_t)I.piece * a.Hkv;
      float2 *ml = reinterpret_cast<float2 *>(a.part + (size_t)a.slot_cap * a.Hkv * per);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          ch_ld32(tO + c * 32, o);
          ch_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (alt) {
          if (c == D / 64) {  // the other's second half
            if (!(ok = pair_sync()) || !(ok = pair_sync())) break;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = lds128_at(xaddr((c & (D / 64 - 1)) * 8 + i));
            o[4 * i] = ch_join(o[4 * i], own, x.x, other);
            o[4 * i + 1] = ch_join(o[4 * i + 1], own, x.y, other);
            o[4 * i + 2] = ch_join(o[4 * i + 2], own, x.z, other);
            o[4 * i + 3] = ch_join(o[4 * i + 3], own, x.w, other);
          }
        }
        if (live) {
          if (I.np == 1) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 pk;
              uint32_t *w = &pk.x;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = ch_pack(__uint_as_float(o[i + 2 * e]) * inv,
                               __uint_as_float(o[i + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4 *>(out + at * D + c * 32 + i) = pk;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4 *>(a.part + mine * per + (size_t)br * D + c * 32 + i) =
                  make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
      }
      if (!ok) break;
      if (alt) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (!(ok = pair_sync())) break;  // read: the queries' space is free
        if (r == 0) mbar_arrive(&sm->q_empty);
      }
      ch_fence_before();
      __syncwarp();
      if (lane == 0 && n > 0) mbar_arrive(&sm->o_empty[t]);
      if (I.np == 1) {
        if (live && a.lse)
          a.lse[at] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        done();
        continue;
      }
      if (live) ml[mine * a.part_rows + br] = make_float2(m, l);
      __threadfence();
      if (!(ok = wg_sync())) break;
      if (tid % 128 == 0)
        sm->last[t] = atomicAdd(&a.arrive[first + (size_t)t * a.Hkv], 1u) == (uint32_t)(I.np - 1);
      if (!(ok = wg_sync())) break;
      if (sm->last[t]) {
        // the block's last piece to arrive merges them all
        __threadfence();
        pg_merge<D, 4>(a, first, I.np, t * tile_rows, min(I.rows - t * tile_rows, tile_rows), r, 128,
                    [&](int row) {
                      return (size_t)(I.row0 + I.t0 + a.by_G(row)) * a.Hq + I.h * G + row -
                             a.by_G(row) * G;
                    },
                    out);
      }
      if (!(ok = wg_sync())) break;  // sm->last is read before the next item's
      done();
    }
  }
  ch_fence_before();
  __syncthreads();
  ch_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

template <int D, bool ALT>
cudaError_t run(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  using C = ChCfg<D>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  auto kern = paged_chunk_kernel<D, ALT>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const PgTile tile = pg_tile(s.page, s.blocks, D * 2, kChKeys);
  const int TPT = 128 / s.G();
  CUtensorMap mq, mk, mv;
  e = pg_query_map(&mq, a.q, D, s.Hq, s.T, a.q_stride, s.G(), TPT);
  if (e == cudaSuccess) e = pg_cache_map(&mk, a.K, s, tile);
  if (e == cudaSuccess) e = pg_cache_map(&mv, a.V, s, tile);
  if (e != cudaSuccess) return e;
  // starting a piece takes about as long as two tiles, a partial's way out and
  // back another three
  if ((e = launch_paged_schedule(s, a, 2 * TPT, kChKeys, di.sm_count, 8, 20, st)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[1];
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.gridDim = dim3((unsigned)di.sm_count, 1, 1);
  cfg.blockDim = dim3(kChThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.numAttrs = 0;
  add_pdl_attr(cfg, attrs);
  e = cudaLaunchKernelEx(&cfg, kern, a, mq, mk, mv, tile);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  // Blocks of one row tile leave half of the kernel idle unless the two chains
  // take turns at the key tiles, but the code for that slows full blocks down by
  // 4 % (2,048-token chunk of 32K: 1,200 against 1,250 us).  So it goes by the
  // batch's average: with it, one 1,000-token chunk among 31 decoding sequences
  // takes 207 instead of 215 us, a 646-token one among ten 53 instead of 65.
  const bool alt = (long long)s.T * s.G() <= 256ll * s.B;
  if (s.d == 64) return alt ? run<64, true>(s, a, st) : run<64, false>(s, a, st);
  return alt ? run<128, true>(s, a, st) : run<128, false>(s, a, st);
}

}  // namespace sd
