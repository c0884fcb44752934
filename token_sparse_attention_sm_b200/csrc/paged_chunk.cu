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
//  * a warp per row tile issues its MMAs: S_t = Q_t K^T (M = 128, N = 64) and
//    O_t += P_t V, P_t read from tensor memory;
//  * four softmax warps per row tile, one row per thread: S from tensor
//    memory, P = exp2(S scale - m) rounded to bf16 over the dead S, the row's
//    maximum meanwhile, and O scaled when m has to move.
// K and V tiles have 128 keys, S tiles 64: a row tile has two S buffers, so the
// scores of the next keys are made while the softmax of these is at work, and
// each row tile has its own issuing warp, so that neither waits behind the
// other's waits.  Tensor memory: two S buffers and O per row tile (512 columns
// at d = 128).  M = 128, N = 64 reads 6 KB of shared memory for 32 cycles of
// products, 48 cycles; S tiles of 128 keys, one buffer each, need 64 for 64 but
// make every row tile one chain, scores - softmax - product - scores: 888 TFLOP/s
// against 1,107 (a 2,048-token chunk of 32K, 32 query heads over 8, d = 128; now
// 1,100-1,130 in short runs at 1,965 MHz, 980-1,000 once the power cap has brought
// the clock to 1,710-1,750 MHz).  Its 256 items on 148 SMs leave 13 % of them idle.
// Handing P over in two halves costs more in the softmax than the earlier
// product gains (921).
//
// The reference m of a row is only raised when the running maximum has left it
// by more than 2^8: weights then reach 256 instead of 1, the sums stay fp32,
// the division at the end cancels m, and O is almost never rescaled.
// P is rounded to bf16 once, where the decode kernel keeps two parts: a second
// product per tile would lengthen the unit that bounds this kernel by 40 %.
// Its sum is taken before the rounding.  The errors of single weights are
// independent and about as large as the rounding of the result, so the result
// is off by 0.0022-0.0024 of its norm where that rounding alone makes 0.0017.
//
// Every wait is bounded; when one runs out the kernel raises TIMEOUT, all
// roles leave their loops, each waits for what it still has in flight (copies,
// products, loads), the tensor memory is freed and the kernel returns.
#include "paged.h"
#include "paged.cuh"
#include "paged_tma.h"

namespace sd {
namespace {

constexpr int kChKeys = 128;  // keys of a K or V tile
constexpr int kChHalf = 64;   // keys of an S tile
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
  static constexpr int kSmem = kSmallOff + 1024 + 1024;  // small area, alignment slack
};

// One work item, as the TMA warp found it.
struct ChItem {
  int b, h, row0, t0, rows;            // rows: query rows of the block
  int p_first, p_last, low;            // positions of its first and last token; lowest key of a window
  int u0, u1, halves;                  // the piece's tiles, and the 64-key halves to run
  int sink_tiles, lo;
  int np, slot;                        // pieces of the range; its partial: slot * Hkv + h
  int valid;                           // 0: no more items
};

struct ChSmall {
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty;
  // [row tile][S buffer]: a buffer's phases alternate strictly, so a parity
  // wait is never two phases off
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2][2];
  uint64_t o_empty[2];
  uint64_t item_full[2], item_empty[2];
  ChItem item[2];
  uint32_t ok[8];
  uint32_t tmem, abort;
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

// max(a, b, c) of fp32 values
__device__ __forceinline__ float ch_max3(float a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
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

template <int D>
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
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm->s_full[t][i], 1);
        mbar_init(&sm->p_ready[t][i], 4);
        mbar_init(&sm->pv_done[t][i], 1);
      }
      mbar_init(&sm->o_empty[t], 4);
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
            const int b = pg_find(a.seqs, a.B, y, &PgSeq::base, &sq);
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
              // no row sees the second half of a tile that ends a range early
              I.halves = 2 * (I.u1 - I.u0);
              if (I.u1 > I.u0 && I.u1 == t.units() &&
                  t.tile(I.u1 - 1) * kChKeys + kChHalf > p_last)
                --I.halves;
              I.np = sq.np;
              I.slot = sq.slot + rb * sq.np + piece;
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
      if (q_count > 0) mbar_wait(&sm->q_full, (q_count - 1) & 1, a.status);
    } else {
      // ---- MMA warps, one per row tile: all lanes walk, one issues ---------------------
      // (The walk stays uniform and the issue under elect.sync, so the operands
      // live in uniform registers: issued from a divergent lane 0, with each
      // descriptor moved over on its own, an instruction took about 100 cycles.)
      const int t = warp - kChMmaWarp;
      constexpr uint32_t idS = ch_idesc(kChHalf, false), idPV = ch_idesc(D, true);
      const bool lead = ch_elect();
      const uint32_t tS = ch_uniform(tmem + t * 128), tO = ch_uniform(tmem + 256 + t * 128);
      const uint64_t q = ch_desc(ch_uniform(base + C::kQOff + t * C::kQTile), 16, 1024);
      const uint32_t ring = ch_uniform(base + C::kRingOff);
      // in 16-byte units: between column blocks, 16 and 64 keys
      const uint32_t kcol = tl.col / 16, vstep = 2 * tl.group / 16, half = 8 * tl.group / 16;
      int slot = 0;  // ring position of the next tile
      uint32_t phase = 0, q_count = 0, o_cnt = 0;
      uint32_t s_cnt = 0, p_cnt = 0;  // halves whose scores, whose product were issued
      auto step = [&]() {
        if (++slot == C::kSlots) slot = 0, phase ^= 1u;
      };
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ch_wait(bar, parity & 1u, sm, a.status)) != 0;
      };
      bool ok = true;
      for (int it = 0; ok; ++it) {
        if (!(ok = wait(&sm->item_full[it & 1], it >> 1))) break;
        const ChItem &I = sm->item[it & 1];
        const int valid = ch_uniform(I.valid), n = ch_uniform(I.halves);
        const bool mine = t == 0 || ch_uniform(I.rows) > TPT * G;
        __syncwarp();
        if (lead) mbar_arrive(&sm->item_empty[it & 1]);
        if (!valid) break;
        if (n <= 0) continue;
        if (!(ok = wait(&sm->q_full, q_count++))) break;
        if (!mine) {  // no rows in this tile: free what the other one uses
          for (int j = 0; j < (n + 1) / 2 * 2 && ok; ++j) {
            ok = wait(&sm->full[slot], phase);
            if (lead) mbar_arrive(&sm->empty[slot]);
            step();
          }
          if (lead) mbar_arrive(&sm->q_empty);
          __syncwarp();
          continue;
        }
        int kslot = 0, vslot = 0;
        // scores of half i into the buffer whose turn it is; the last half of a
        // K tile frees it
        auto scores = [&](int i) {
          if ((i & 1) == 0) {
            kslot = slot;
            if (!(ok = wait(&sm->full[slot], phase))) return;
            step();
          }
          const uint32_t buf = s_cnt & 1;
          // the P that the buffer held is used up
          if (s_cnt >= 2 && !(ok = wait(&sm->pv_done[t][buf], (s_cnt >> 1) - 1))) return;
          ch_fence_after();
          const uint64_t k =
              ch_desc(ch_uniform(ring + kslot * C::kTile), 16, tl.group) + (i & 1) * half;
          if (lead) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              ch_mma_ss(tS + buf * 64, q + ((s >> 2) * (128 * 128) + (s & 3) * 32) / 16,
                        k + (s >> 2) * kcol + (s & 3) * 2, idS, s > 0);
            ch_commit(&sm->s_full[t][buf]);
            if ((i & 1) || i == n - 1) ch_commit(&sm->empty[kslot]);
            if (i == n - 1) ch_commit(&sm->q_empty);
          }
          __syncwarp();
          ++s_cnt;
        };
        scores(0);
        for (int i = 0; i < n && ok; ++i) {
          if ((i & 1) == 0) {  // V follows its K in the ring
            vslot = slot;
            if (!(ok = wait(&sm->full[slot], phase))) break;
            step();
          }
          // the next scores run while the softmax of these is at work
          if (i + 1 < n) {
            scores(i + 1);
            if (!ok) break;
          }
          const uint32_t buf = p_cnt & 1;
          if (i == 0 && o_cnt++ > 0)  // O of the item before has been read
            if (!(ok = wait(&sm->o_empty[t], o_cnt - 2))) break;
          if (!(ok = wait(&sm->p_ready[t][buf], p_cnt >> 1))) break;
          ch_fence_after();
          const uint64_t v =
              ch_desc(ch_uniform(ring + vslot * C::kTile), tl.col, tl.group) + (i & 1) * half;
          if (lead) {
#pragma unroll
            for (int kk = 0; kk < kChHalf / 16; ++kk)
              ch_mma_ts(tO, tS + buf * 64 + kk * 8, v + kk * vstep, idPV,
                        kk > 0 ? 1u : (uint32_t)(i > 0));
            ch_commit(&sm->pv_done[t][buf]);
            if ((i & 1) || i == n - 1) ch_commit(&sm->empty[vslot]);
          }
          __syncwarp();
          ++p_cnt;
        }
      }
      // and its products, before their tensor memory is freed
      if (s_cnt > 0)
        mbar_wait(&sm->s_full[t][(s_cnt - 1) & 1], ((s_cnt - 1) >> 1) & 1, a.status);
      if (p_cnt > 0)
        mbar_wait(&sm->pv_done[t][(p_cnt - 1) & 1], ((p_cnt - 1) >> 1) & 1, a.status);
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
    uint32_t phase = 0, s_cnt = 0;
    int unit = 0;
    bool ok = true;
    constexpr uint32_t all_ok = (1u << (kChHalf / 16)) - 1u;
    auto step = [&]() {
      if (++ring == C::kSlots) ring = 0, phase ^= 1u;
    };
    for (int it = 0;; ++it) {
      // the warp leaves together: its lanes meet again in the collectives below
      if (!__all_sync(0xffffffffu,
                      ch_wait(&sm->item_full[it & 1], (it >> 1) & 1, sm, a.status)))
        break;
      const ChItem &I = sm->item[it & 1];  // until this warp's arrival below
      auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->item_empty[it & 1]);
      };
      if (!I.valid) break;
      const int n = max(0, I.halves), tile_rows = TPT * G;
      if (t == 1 && I.rows <= tile_rows) {  // no second row tile: keep count of the ring
        for (int j = 0; j < n; j += 2) {
          step(), step();
          ++unit;
        }
        done();
        continue;
      }
      const int br = t * tile_rows + r;  // row of the block
      const bool live = r < tile_rows && br < I.rows;
      const int pos = live ? I.p_first + a.by_G(br) : -1;
      const int low = pg_window_low(pos, a.window);
      const int pf = I.p_first + t * TPT, pl = min(I.p_last, pf + TPT - 1);  // the tile's tokens
      const int low_last = pg_window_low(pl, a.window);
      float m = -INFINITY, l = 0.f;
      const int u0 = I.u0, sink_tiles = I.sink_tiles, hi_first = I.lo - I.sink_tiles;
      const int last_key = I.p_last, first_low = I.low;
      int vslot = 0, key0 = 0;
      uint32_t good8 = 0;
      for (int j0 = 0; j0 < n && ok; j0 += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = j0 + h;
          if (j >= n) break;
          if (h == 0) {
            const int u = u0 + (j0 >> 1);
            key0 = (u < sink_tiles ? u : u + hi_first) * kChKeys;
          } else {
            key0 += kChHalf;
          }
          const uint32_t buf = s_cnt & 1, tB = tS + buf * 64;
          ok = ch_wait(&sm->s_full[t][buf], (s_cnt >> 1) & 1, sm, a.status);
          ch_fence_after();
          uint32_t s[kChHalf], p[32];
          ch_ld32(tB, s);
          ch_ld32(tB + 32, s + 32);
          if (h == 0) {
            step();
            vslot = ring;
            // also orders this after the V warp's note on the tile's pages
            if (ok) ok = ch_wait(&sm->full[vslot], phase, sm, a.status);
            step();
            good8 = sm->ok[unit++ & 7];
          }
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          const uint32_t good = (good8 >> (4 * h)) & all_ok;
          if (key0 + kChHalf > last_key + 1 || (key0 < first_low && key0 + kChHalf > a.sinks)) {
            // V rows that no row of the block sees may hold anything: clear them
            // (each tile's warps before its own product; both write zeros)
            const int key = key0 + (r >> 1);
            if (key > last_key || (key < first_low && key >= a.sinks)) {
              const int vr = h * kChHalf + (r >> 1);
              const uint32_t v =
                  base + C::kRingOff + vslot * C::kTile + (vr >> 3) * tl.group + (vr & 7) * 128;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {  // 16-byte pieces, half a row
                const int c = (r & 1) * (D / 16) + ((i + (r >> 1)) & (D / 16 - 1));
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                                 v + (c >> 3) * tl.col + (c & 7) * 16),
                             "r"(0u)
                             : "memory");
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          const bool whole = key0 + kChHalf - 1 <= pf &&
                             (key0 >= low_last || key0 + kChHalf <= a.sinks) && good == all_ok;
          ch_wait_ld();
          if (!whole) {
            // the row's keys, a bit each
            const int hi = pos - key0, lo = low - key0, sk = a.sinks - key0;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t pages = ((good >> (2 * w)) & 1u ? 0xffffu : 0u) |
                                     ((good >> (2 * w)) & 2u ? 0xffff0000u : 0u);
              const uint32_t see = pg_below(hi + 1 - 32 * w) &
                                   (~pg_below(lo - 32 * w) | pg_below(sk - 32 * w)) & pages;
              // (most blocks of an edge tile are seen whole by all of the warp's rows)
              if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!((see >> i) & 1u)) s[w * 32 + i] = 0xff800000u;
              }
            }
          }
          auto top = [&]() {
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kChHalf; i += 2)
              mx4[(i >> 1) & 3] = ch_max3(mx4[(i >> 1) & 3], s[i], s[i + 1]);
            return fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
          };
          uint64_t sum2[2];
          auto weights = [&]() {
            const float use = m == -INFINITY ? 0.f : m;
            const uint64_t scale2 = pg_f2(a.scale_log2, a.scale_log2), neg2 = pg_f2(-use, -use);
            sum2[0] = sum2[1] = 0ull;  // pairs of zeros
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float p0, p1;
              pg_split(pg_fma2(pg_u2(s[2 * i], s[2 * i + 1]), scale2, neg2), &p0, &p1);
              p0 = pg_exp2(p0);
              p1 = pg_exp2(p1);
              sum2[i & 1] = pg_add2(sum2[i & 1], pg_f2(p0, p1));
              p[i] = ch_pack(p0, p1);
            }
          };
          // The weights do not wait for the maximum: the reference rarely moves,
          // and if it does they are taken again (the first half sets it first).
          if (j == 0) m = top();
          weights();
          const float mx = top();
          const bool raise = mx > m + kChLag || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, raise)) {
            const float mn = raise ? mx : m;
            const float corr = raise ? exp2f(m - mn) : 1.f;  // 0 when m was none yet
            m = mn;
            l *= corr;
            if (j > 0) {
              // the product before this one has to finish (the one before that
              // did before this buffer's scores were issued)
              const uint32_t before = s_cnt - 1;
              ok = ch_wait(&sm->pv_done[t][before & 1], (before >> 1) & 1, sm, a.status);
              if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
              }
              ch_fence_after();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                ch_ld32(tO + c * 32, p);
                ch_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) p[i] = __float_as_uint(__uint_as_float(p[i]) * corr);
                ch_st32(tO + c * 32, p);
              }
            }
            weights();
          }
          ch_st32(tB, p);
          float a0, a1;
          pg_split(pg_add2(sum2[0], sum2[1]), &a0, &a1);
          l += a0 + a1;
          ch_wait_st();
          ch_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->p_ready[t][buf]);
          ++s_cnt;
        }
      }
      if (!ok) break;
      // ---- the piece's result ----------------------------------------------------------
      if (n > 0) {
        // every product of the item is done when its last one is
        const uint32_t last = s_cnt - 1;
        ok = ch_wait(&sm->pv_done[t][last & 1], (last >> 1) & 1, sm, a.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        ch_fence_after();
      }
      const size_t at = (size_t)(I.row0 + I.t0 + a.by_G(br)) * a.Hq + I.h * G + br - a.by_G(br) * G;
      const float inv = pg_inverse(l);
      const size_t per = (size_t)a.part_rows * D;
      const size_t mine = (size_t)I.slot * a.Hkv + I.h;
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
      ch_fence_before();
      __syncwarp();
      if (lane == 0 && n > 0) mbar_arrive(&sm->o_empty[t]);
      if (I.np == 1) {
        if (live && a.lse) a.lse[at] = pg_lse(m, l);
        done();
        continue;
      }
      if (live) ml[mine * a.part_rows + br] = make_float2(m, l);
      done();
    }
    ch_wait_ld();
    ch_wait_st();
  }
  ch_fence_before();
  __syncthreads();
  ch_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

template <int D>
cudaError_t run(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  using C = ChCfg<D>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  auto kern = paged_chunk_kernel<D>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const PgTile tile = pg_tile(s.page, s.blocks, D * 2, kChKeys);
  const int TPT = 128 / s.G();
  CUtensorMap mq, mk, mv;
  e = pg_query_map(&mq, a.q, D, s.Hq, s.T, a.q_stride, s.G(), TPT);
  if (e == cudaSuccess) e = pg_cache_map(&mk, a.K, s, tile);
  if (e == cudaSuccess) e = pg_cache_map(&mv, a.V, s, tile);
  if (e != cudaSuccess) return e;
  // starting a piece takes about as long as two and a half tiles, a partial's
  // way out and back nearly four more (2 and 5 in all: 94 us against 85 for 32
  // tokens each of 8 sequences of 8K)
  if ((e = launch_paged_schedule(s, a, 2 * TPT, kChKeys, di.sm_count, 10, 25, st)) != cudaSuccess)
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
  if ((e = cudaLaunchKernelEx(&cfg, kern, a, mq, mk, mv, tile)) != cudaSuccess) return e;
  return launch_paged_merge(s, a, 2 * TPT, st);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedShape &s, const PgArgs &a, cudaStream_t st) {
  return s.d == 64 ? run<64>(s, a, st) : run<128>(s, a, st);
}

}  // namespace sd
