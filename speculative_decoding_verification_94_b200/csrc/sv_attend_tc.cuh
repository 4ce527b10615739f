// sv_attend_tc.cuh -- bf16 attention of many rows (long drafts, candidate
// trees) on the fifth-generation tensor cores.  D is 64 or 128; the tensor maps
// fill the columns past a smaller head size with zeros.
//
// Products.  A tile is 128 keys.  S = Q K^T is one 128 x 128 product (128
// lanes of tensor memory), O += P V one of 128 x D; their operands come from
// shared memory (TMA, 128-byte swizzle), the weights P from tensor memory.
// The lanes are the rows of a row tile of RT = 32, 64 or 128; with fewer than
// 128 rows they are repeated, and copy c of a row takes the weights of the
// c-th part of the keys only, so that all four warps of a warp group work on
// the softmax of every tile; the copies add up at the end.
//
// Weights.  A weight enters the product as the sum of two bf16, its rounding
// and the rest's, which keeps it to 2^-16, as in the kernel of few rows: the
// output's error is then its own rounding (0.0017 of its size; 0.0021 with one
// bf16).  128 rows take two products for it (16 instructions a tile instead of
// 8).  Repeated rows take none: copies c and c ^ 1 of a row are partners that
// share a maximum, and the rests of one's part go to the other's lanes, which
// had zeros there.  The partner computes those weights from its own lanes of S
// (two copies tell each other their maxima, of four each looks at both parts).
//
// Bound.  One SM's share of HBM brings the 64 KB of a tile in 1.5 us.  An
// instruction of the products (16 of the summed index) took 95 cycles whether
// it was 64 or 128 wide, so a tile's 16 take 0.8 us (24 with 128 rows: 1.2 us),
// and a softmax of 128 rows 0.9 us without the rests.  With the products and the
// softmax taken out, the copies alone needed 109 us for 130,000 keys of 8 heads
// (40 rows).  What the rests cost: 67.3 -> 68.3 us with 28 rows (32 requests of
// 700 to 9000 keys), 100 -> 107 us with 40 (130,000 keys), 49 -> 59 us with 256
// (8 requests of 2000 to 8000 keys), 191 -> 235 us with 128 (64 requests), there
// mostly in the softmax.  What was slower: second products for all numbers of
// rows (74 and 117 us with 28 and 40); S in halves of 64 keys (32 instructions a
// tile); with 128 rows, half of a tile's second product under the other half's
// softmax (244 us).
//
// Roles.  Two warps issue the copies (keys, values), one the products, as
// their operands arrive, one fills the rows behind a request's own.  Two warp
// groups take the even and the odd tiles, each with its own S, P, O, maximum
// and sum, so that one's softmax runs under the other's products, and neither
// waits for the other.  O stays in tensor memory; it is rescaled only when the
// maximum grows by more than 2^8 (a weight may then be up to 2^8, which costs
// no precision: the sum is fp32).  P is stored over S.
//
// Every wait has a time limit; a block whose wait runs out gives NaN for its
// segments, sets SV_DEV_TIMEOUT and goes on to the end.
#pragma once

#include <cuda.h>

#include "sv_attend.cuh"
#include "sv_attend_mma.cuh"
#include "sv_device.cuh"

namespace sv {

constexpr int kTcU = 128;            // keys of a tile
// A segment's beginning and end, in tiles: about 5 us with 32 rows, 10 us with 128.
// (With 2, 3 and 5 instead, 8 requests of 28 rows took 31 us instead of 25, the
// 32 requests of 28 rows 74 us instead of 68; with 5, 6 and 12 as now.)
__host__ __device__ constexpr int tc_ov(int rt) { return rt == 128 ? 9 : rt == 64 ? 5 : 4; }
constexpr int kTcSoftmax = 256;      // threads of the two warp groups
constexpr int kTcThreads = 384;      // + two copy warps, product warp, one for the rest
constexpr int kTcStages = 3;

template <int D>
struct TcCfg {
  static constexpr int kTile = kTcU * D * 2;               // bytes of keys (or values)
  static constexpr int kHalf = kTcU * 128;                 // 64 columns of a tile: 128-byte rows
  static constexpr int kOffK = kTcU * D * 2;               // after Q
  static constexpr int kOffV = kOffK + kTcStages * kTile;
  static constexpr int kOffEnd = kOffV + kTcStages * kTile;
  static constexpr int kOffMl = kOffEnd;                   // [2][128] (m, l)
  static constexpr int kOffBar = kOffMl + 2048;
  static constexpr int kOffMisc = kOffBar + 256;
  static constexpr int kOffShare = kOffMisc + 64;
  static constexpr int kSmem = kOffShare + kShareBytes;
  // output columns added at a time, through the space of Q
  static constexpr int kCols = D == 128 ? 32 : 16;
};

// ---------------------------------------------------------------------------
// PTX of the tensor cores and the tensor maps.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok;
}
// D = A B (+ D): A and B in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool add) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.u32 P, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, P;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// A in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          bool add) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.u32 P, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, P;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tc_ld(uint32_t a, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
               "%10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                 "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, "
               "%8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
               "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(
                   r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_ld(uint32_t a, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
               "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, "
               "%26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                 "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                 "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                 "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                 "=r"(r[30]), "=r"(r[31])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, "
               "%8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
               "%24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
               "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
               "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
               "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
               "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(a)
               : "memory");
}
// Waits for the loads so far; the values of `r` are not there before.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// A box of the cache: 64 columns x box rows of one page and head.
__device__ __forceinline__ void tma_page(void* dst, const CUtensorMap* map, int col, int token,
                                         int head, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(col), "r"(token), "r"(head), "r"(page)
      : "memory");
}
// The largest of three; NaN only if all are.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Named barrier of the softmax threads.
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

// Shared-memory operand with 128-byte swizzle: 8 rows of 128 bytes are one
// 1024-byte atom; `lead` is the distance of 64-element blocks along the
// contiguous dimension where that dimension is not the summed one.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32, M = 128; b_cols: B is contiguous along N.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_cols) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_cols ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

struct TcParams {
  AttendParams a;
  int box;  // rows of a copy box: keys of a page within a tile
  unsigned long long wait_ns;  // limit of a wait
  int stall;  // test: the values of the first tile of all are never copied
};

// Wait for phase `parity` of a barrier, giving up after `limit_ns`.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity,
                                        unsigned long long limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

template <int D, int RT>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_tc_kernel(const TcParams tp, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using C = TcCfg<D>;
  constexpr int kCopies = 128 / RT;          // copies of a row among the lanes
  constexpr int kKeys = kTcU / kCopies;      // keys of a copy
  constexpr int kParts = kCopies == 1 ? 2 : 1;  // of the weights, one product after the other
  extern __shared__ __align__(1024) unsigned char smem[];
  const AttendParams& p = tp.a;
  const unsigned long long wait_ns = tp.wait_ns;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* s_q = smem;
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t *k_full = bars, *k_empty = bars + 3, *v_full = bars + 6, *v_empty = bars + 9,
           *s_full = bars + 12, *p_ready = bars + 14, *pv_done = bars + 16, *q_full = bars + 18,
           *q_first = bars + 19, *tops = bars + 20;  // tops: RT 64 only
  int* misc = reinterpret_cast<int*>(smem + C::kOffMisc);
  volatile int* s_abort = misc;      // a wait ran out
  int* s_bad = misc + 1;             // the segment's keys are on a bad page
  int* s_fix = misc + 2;             // a new token's value is not finite
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + 4);

  if (tid == 0) {
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + i, 128);
      mbar_init(pv_done + i, 1);
      mbar_init(tops + i, 128);
    }
    mbar_init(q_full, kTcSoftmax);
    mbar_init(q_first, kTcSoftmax);
    fence_mbar_init();
    misc[0] = misc[1] = misc[2] = 0;
    att_clear_note(p);
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  pdl_launch_dependents();
  AttCursor<kTcU, RT, tc_ov(RT)> cur;
  const AttShare s = att_share<kTcThreads>(p, cur, smem + C::kOffShare);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == 8 || warp == 10) {
    // ---------------- copies: keys (warp 8) and values (warp 10) ---------------
    // apart, because keys are done with two tiles before values are
    const bool keys = warp == 8;
    const int boxes = kTcU / tp.box;              // <= 16 per 64 columns
    constexpr int kHalves = D / 64;
    const int bi = lane & 15, half = lane >> 4;
    const bool mine = bi < boxes && half < kHalves;
    uint64_t *fulls = keys ? k_full : v_full, *empties = keys ? k_empty : v_empty;
    unsigned char* ring = smem + (keys ? C::kOffK : C::kOffV) + half * C::kHalf + bi * tp.box * 128;
    auto page_of = [&]() {  // out of the pool: zeros are copied
      const int pos = cur.tile * kTcU + bi * tp.box;
      if (cur.v >= s.u1 || !mine || pos >= cur.kv + cur.q) return p.num_pages;
      const int id = __ldg(p.table + (long long)cur.b * p.max_pages + fast_div(pos, p.div_page));
      return id >= 0 && id < p.num_pages ? id : p.num_pages;
    };
    int page = page_of();
    int slot = 0, round = 0;
    bool ok = true;
    while (cur.v < s.u1) {
      const int h = cur.seg / cur.mt;
      const int pos = cur.tile * kTcU + bi * tp.box;
      const int token = pos - fast_div(pos, p.div_page) * p.page;
      const int id = page;
      cur.step(p, 1);
      page = page_of();
      if (round) ok = __all_sync(0xffffffffu, tc_wait(empties + slot, (round - 1) & 1, wait_ns));
      // q is on its way with the first tile; the others would come before it
      if (slot == 1 && round == 0)
        ok = __all_sync(0xffffffffu, tc_wait(q_first, 0, wait_ns));
      if (!ok) break;
      const bool skip = tp.stall && !keys && slot == 0 && round == 0 &&
                        (int)blockIdx.x == s.block_of(tc_ov(RT));
      if (lane == 0 && !skip) mbar_arrive_expect_tx(fulls + slot, C::kTile);
      __syncwarp();
      if (mine && !skip) {
        unsigned char* dst = ring + slot * C::kTile;
        if (keys)
          tma_page(dst, &kmap, half * 64, token, h, id, fulls + slot);
        else
          tma_page(dst, &vmap, half * 64, token, h, id, fulls + slot);
      }
      if (++slot == kTcStages) slot = 0, ++round;
    }
    if (!ok) {  // the copies under way end before the block does
      *s_abort = 1;
      kv_flag(p.status, SV_DEV_TIMEOUT);
      for (int i = 0; i < kTcStages; ++i)
        tc_wait(fulls + i, (round - (i >= slot)) & 1, wait_ns);
    }
  } else if (warp == 9) {
    // ------------------------------ products ------------------------------
    {
      constexpr uint32_t kIdQk = tc_idesc(kTcU, false), kIdPv = tc_idesc(D, true);
      const uint32_t qa = smem_u32(s_q);
      int kg = 0, vg = 0;      // tiles whose keys, values have been used
      int streams[2] = {0, 0};  // tiles of each warp group
      int segs = 0;
      bool ok = true;
      while (cur.v < s.u1 && ok) {
        const int left = cur.tiles - cur.tile;
        const int cnt = s.u1 - cur.v < left ? (int)(s.u1 - cur.v) : left;
        if (lane == 0) {  // one thread issues
          ok = tc_wait(q_full, segs & 1, wait_ns);
          tc_fence_after();
          // whichever product has its operands: S of tile nq (its warp group's
          // last P is used up), or P V of tile np
          int nq = 0, np = 0;
          uint64_t t0 = 0;  // the clock is far away: read once in many idle rounds
          uint32_t spins = 0;
          while (ok && np < cnt) {
            bool idle = true;
            if (np < nq) {
              const int w = np & 1, slot = vg % kTcStages;
              if (mbar_test(p_ready + w, streams[w] & 1) &&
                  mbar_test(v_full + slot, (vg / kTcStages) & 1)) {
                tc_fence_after();
                const uint32_t va = smem_u32(smem + C::kOffV + slot * C::kTile);
                const uint32_t pa = tmem + w * 128, o = tmem + 256 + w * 128;
#pragma unroll
                for (int part = 0; part < kParts; ++part)
#pragma unroll
                  for (int ks = 0; ks < kTcU / 16; ++ks)
                    tc_mma_ts(o, pa + (ks / 2) * 32 + part * 16 + (ks & 1) * 8,
                              tc_desc(va + ks * 2048, C::kHalf), kIdPv, np >= 2 || part || ks);
                tc_commit(pv_done + w);
                tc_commit(v_empty + slot);
                ++streams[w];
                ++vg;
                ++np;
                idle = false;
              }
            }
            if (nq < cnt && nq < np + 2) {
              const int w = nq & 1, slot = kg % kTcStages;
              if (mbar_test(k_full + slot, (kg / kTcStages) & 1)) {
                tc_fence_after();
                const uint32_t ka = smem_u32(smem + C::kOffK + slot * C::kTile);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint32_t o = (ks / 4) * C::kHalf + (ks % 4) * 32;
                  tc_mma_ss(tmem + w * 128, tc_desc(qa + o, 16), tc_desc(ka + o, 16), kIdQk,
                            ks > 0);
                }
                tc_commit(s_full + w);
                tc_commit(k_empty + slot);
                ++kg;
                ++nq;
                idle = false;
              }
            }
            if (!idle) {
              spins = 0;
            } else if ((++spins & 1023) == 0) {
              const uint64_t now = globaltimer_ns();
              if (spins == 1024) t0 = now;
              if (now - t0 > wait_ns) {
                ok = false;
                break;
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++segs;
        cur.step(p, cnt);
      }
      if (!ok && lane == 0) {
        *s_abort = 1;
        kv_flag(p.status, SV_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    att_fill_padding<__nv_bfloat16>(p, 11, 1);
  } else {
    // ------------------------------- softmax -------------------------------
    const int w = warp >> 2, quad = warp & 3;
    const int lr = quad * 32 + lane;              // lane of tensor memory
    const int row = lr % RT, copy = lr / RT;      // copy is the same for a warp
    const uint32_t lane_at = (uint32_t)(quad * 32) << 16;
    const uint32_t s_at = tmem + lane_at + w * 128, o_at = tmem + lane_at + 256 + w * 128;
    int tiles_done = 0;                           // of this warp group
    int tile_g = 0;                               // of the block
    bool dead = false;
    // q: neighbouring threads load neighbouring 16 bytes; a row goes to each of
    // its copies
    constexpr int kPieces16 = D / 8, kPer = RT * kPieces16 / kTcSoftmax;
    uint4 qx[kPer];
    auto load_q = [&](const AttCursor<kTcU, RT, tc_ov(RT)>& c) {
      const int h = c.seg / c.mt, first = (c.seg - h * c.mt) * RT;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int qr = first + (tid + j * kTcSoftmax) / kPieces16;
        const bool on = qr < c.q * p.g;
        const int i = on ? fast_div(qr, p.div_g) : 0, gi = on ? qr - i * p.g : 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(p.q) + c.b * p.q_b + i * p.q_t +
            (long long)(h * p.g + gi) * p.d);
        qx[j] = on && tid % kPieces16 * 8 < p.d ? __ldg(src + tid % kPieces16)
                                                : make_uint4(0, 0, 0, 0);
      }
    };
    // ahead of its segment where that takes few registers
    constexpr bool kQAhead = RT < 128;
    if (kQAhead && cur.v < s.u1) load_q(cur);
    while (cur.v < s.u1) {
      const int h = cur.seg / cur.mt, row0 = (cur.seg % cur.mt) * RT;
      const int rows = min(RT, cur.q * p.g - row0);
      const int tile0 = cur.tile, left = cur.tiles - cur.tile;
      const int cnt = s.u1 - cur.v < left ? (int)(s.u1 - cur.v) : left;
      const int kv = cur.kv, len = cur.kv + cur.q;
      const int32_t* par = p.parents ? p.parents + (long long)cur.b * p.n : nullptr;
      const int32_t* trow = p.table + (long long)cur.b * p.max_pages;
      // the rows of q
      if (!kQAhead) load_q(cur);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int c = tid % kPieces16, r = (tid + j * kTcSoftmax) / kPieces16;
#pragma unroll
        for (int copy = 0; copy < kCopies; ++copy)  // RT is a multiple of the 8 rows of an atom
          *reinterpret_cast<uint4*>(s_q + (c / 8) * C::kHalf + (copy * RT + r) * 128 +
                                    (((c % 8) ^ (r & 7)) << 4)) = qx[j];
      }
      // the pages of these tiles: loaded here, looked at when the tiles are done
      const int page0 = fast_div(tile0 * kTcU, p.div_page);
      const int pages = fast_div(min((tile0 + cnt) * kTcU, len) - 1, p.div_page) + 1 - page0;
      const int id0 = tid < pages ? __ldg(trow + page0 + tid) : 0;
      const int id1 = tid + kTcSoftmax < pages ? __ldg(trow + page0 + tid + kTcSoftmax) : 0;
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(q_full);
      if (tile_g == 0) mbar_arrive(q_first);
      // where the next segment is; its rows of q are brought to L2
      AttCursor<kTcU, RT, tc_ov(RT)> next = cur;
      next.step(p, cnt);
      if (!kQAhead && next.v < s.u1) {
        const int h2 = next.seg / next.mt;
        const int qr = (next.seg - h2 * next.mt) * RT + (tid & (RT - 1));
        if (qr < next.q * p.g && tid / RT * 64 < p.d) {
          const int i = fast_div(qr, p.div_g), gi = qr - i * p.g;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(
              static_cast<const __nv_bfloat16*>(p.q) + next.b * p.q_b + i * p.q_t +
              (long long)(h2 * p.g + gi) * p.d + tid / RT * 64));
        }
      }
      const int qi = min(fast_div(row0 + row, p.div_g), cur.q - 1);
      float m = -INFINITY, l = 0.f;
      bool tree_ok = true;
      for (int k = w; k < cnt; k += 2) {
        if (!dead) dead = !__all_sync(0xffffffffu, tc_wait(s_full + w, tiles_done & 1, wait_ns));
        if (dead) {
          *s_abort = 1;
          break;
        }
        tc_fence_after();
        // S is read twice, 32 columns at a time, for the maximum and for the
        // weights (but for the last two chunks, which are still there: the
        // weights begin with them); registers are not plenty, which is also why
        // 128 rows store theirs 16 keys at a time (64 requests x 16 tokens x 8
        // heads: 259 us in order and with 32, 241, 235).
        // The chunks of this copy, then those of its partner, whose weights'
        // rests go to this copy's lanes.
        constexpr int kOwn = kKeys / 32, kChunks = kCopies > 1 ? 2 * kOwn : kOwn;
        constexpr int kSeen = kCopies == 2 ? kOwn : kChunks;  // looked at for the maximum
        auto chunk = [&](int c) { return c < kOwn ? copy * kOwn + c : (copy ^ 1) * kOwn + c - kOwn; };
        const bool tail = (tile0 + k + 1) * kTcU > kv;
        auto seen = [&](int c) {  // which of chunk c's keys this row sees
          const int pos0 = (tile0 + k) * kTcU + chunk(c) * 32;
          return pos0 + 32 > kv ? att_tail_bits<32>(par, qi, pos0, kv, tree_ok) : 0xffffffffu;
        };
        auto hide = [&](int c, uint32_t (&x)[32]) {
          if (tail) {
            const uint32_t bits = seen(c);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1u)) x[e] = 0xff800000u;
          }
        };
        // chunk c is looked at while chunk c + 1 is on its way
        uint32_t x[2][32];
        float top = -INFINITY;
        tc_ld(s_at + chunk(0) * 32, x[0]);
        if (kSeen > 2) tc_ld(s_at + chunk(1) * 32, x[1]);
#pragma unroll
        for (int c = 0; c < kSeen; ++c) {
          tc_wait_ld(x[c & 1]);
          if (kSeen == 2 && c == 0) tc_ld(s_at + chunk(1) * 32, x[1]);
          if (kSeen > 2 && c == 2) tc_ld(s_at + chunk(3) * 32, x[1]);
          hide(c, x[c & 1]);
          float t2[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            t2[(e >> 1) & 3] = max3(t2[(e >> 1) & 3], __uint_as_float(x[c & 1][e]),
                                    __uint_as_float(x[c & 1][e + 1]));
          top = fmaxf(fmaxf(t2[0], t2[1]), fmaxf(t2[2], t2[3]));
          if (kSeen > 2 && c == 0) tc_ld(s_at + chunk(2) * 32, x[0]);
        }
        if constexpr (kSeen < kChunks) {
          // the partner's maximum, from shared memory; a place is written again
          // two tiles on, when everyone has passed the next one's barrier
          float* both = reinterpret_cast<float*>(s_ml + w * 128) + (tiles_done & 1);
          both[2 * lr] = top;
          mbar_arrive(tops + w);
          dead = !__all_sync(0xffffffffu, tc_wait(tops + w, tiles_done & 1, wait_ns));
          if (dead) {
            *s_abort = 1;
            break;
          }
          top = fmaxf(top, both[2 * (lr ^ RT)]);
        }
        top *= p.scale_log2;  // scale > 0 here
        // a new maximum only when weights would pass 2^8
        const bool grow = top > m + 8.f || (m == -INFINITY && top != -INFINITY);
        if (__any_sync(0xffffffffu, grow) && k >= 2) {
          dead = !__all_sync(0xffffffffu, tc_wait(pv_done + w, (tiles_done - 1) & 1, wait_ns));
          if (dead) {
            *s_abort = 1;
            break;
          }
          tc_fence_after();
          const float a = grow ? pow2(m - top) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t y[32];
            tc_ld(o_at + c, y);
            tc_wait_ld(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
            tc_st(o_at + c, y);
          }
        }
        if (grow) {
          l *= pow2(m - top);
          m = top;
        }
        const float ms = m == -INFINITY ? 0.f : m;
        const unsigned long long cc = f2_pack(p.scale_log2, p.scale_log2), mm = f2_pack(-ms, -ms);
        unsigned long long sum[2] = {0, 0};
        // P over S: bf16 pairs in the first half of their keys' columns; the
        // rests in the second half, or in the partner's lanes
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = (i + kSeen - 2) % kChunks;  // the last two looked at are still there
          if (i >= 2) {
            tc_wait_ld(x[c & 1]);
            hide(c, x[c & 1]);
          }
          if constexpr (kCopies == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t y[8], rest[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float a, b;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c & 1][16 * h + 2 * e]),
                                         __uint_as_float(x[c & 1][16 * h + 2 * e + 1])),
                                 cc, mm),
                          a, b);
                a = pow2(a);
                b = pow2(b);
                sum[e & 1] = f2_add(sum[e & 1], f2_pack(a, b));
                y[e] = pack_bf16(a, b);
                float ra, rb;
                f2_unpack(f2_fma(f2_pack(bf16_lo(y[e]), bf16_hi(y[e])), f2_pack(-1.f, -1.f),
                                 f2_pack(a, b)),
                          ra, rb);
                rest[e] = pack_bf16(ra, rb);
              }
              tc_st(s_at + chunk(c) * 32 + 8 * h, y);
              tc_st(s_at + chunk(c) * 32 + 16 + 8 * h, rest);
            }
          } else {
          uint32_t y[16], rest[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c & 1][2 * e]),
                                     __uint_as_float(x[c & 1][2 * e + 1])),
                             cc, mm),
                      a, b);
            a = pow2(a);
            b = pow2(b);
            if (c < kOwn) sum[e & 1] = f2_add(sum[e & 1], f2_pack(a, b));
            y[e] = pack_bf16(a, b);
            if (c >= kOwn) {
              float ra, rb;
              f2_unpack(f2_fma(f2_pack(bf16_lo(y[e]), bf16_hi(y[e])), f2_pack(-1.f, -1.f),
                               f2_pack(a, b)),
                        ra, rb);
              rest[e] = pack_bf16(ra, rb);
            }
          }
          tc_st(s_at + chunk(c) * 32, c < kOwn ? y : rest);
          }
          if (i + 2 < kChunks) tc_ld(s_at + chunk((c + 2) % kChunks) * 32, x[c & 1]);
        }
        if constexpr (kCopies > 2) {  // the other copies' keys
          const uint32_t zero[16] = {};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if ((c / kOwn) / 2 != copy / 2) tc_st(s_at + c * 32, zero);
        }
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        if (tail) {
          // Values past the end become zeros, and so do new tokens' values
          // that are not finite: as 0 x inf they would reach rows that do not
          // see them; they are added to those that do at the end.
          const int g = tile_g + k, slot = g % kTcStages;
          dead = !__all_sync(0xffffffffu,
                             tc_wait(v_full + slot, (g / kTcStages) & 1, wait_ns));
          if (dead) {
            *s_abort = 1;
            break;
          }
          // Pages past the end were copied as zeros already.
          const int pos0v = (tile0 + k) * kTcU;
          const long long page_end =
              (long long)(fast_div(len - 1, p.div_page) + 1) * p.page - pos0v;
          const int end = page_end < kTcU ? (int)page_end : kTcU;
          constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;
          for (int r = max((cur.q > 1 ? kv : len) - pos0v, 0) + quad * kRowsPer + lane / kChunks;
               r < end; r += 4 * kRowsPer) {
            const int c = lane % kChunks;
            uint4* at = reinterpret_cast<uint4*>(smem + C::kOffV + slot * C::kTile +
                                                 (c / 8) * C::kHalf + r * 128 + (c % 8) * 16);
            uint32_t y[4] = {0, 0, 0, 0};
            if (pos0v + r < len) {
              const uint4 v = *at;
              y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
              bool any = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                any |= bf16x2_not_finite(y[e]);
                if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u;
                if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0xffffu;
              }
              if (!any) continue;
              *s_fix = 1;
            }
            *at = make_uint4(y[0], y[1], y[2], y[3]);
          }
          fence_async_smem();
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready + w);
        ++tiles_done;
      }
      const bool used = w < cnt;
      if (kQAhead && next.v < s.u1) load_q(next);
      if (used && !dead) {
        dead = !__all_sync(0xffffffffu, tc_wait(pv_done + w, (tiles_done - 1) & 1, wait_ns));
        if (dead) *s_abort = 1;
      }
      tc_fence_after();
      tile_g += cnt;
      // ---- the row's parts together --------------------------------------------
      if (!tree_ok) {
        l = __int_as_float(0x7fc00000);
        if (row < rows) kv_flag(p.status, SV_DEV_BAD_TREE);
      }
      s_ml[w * 128 + lr] = make_float2(m, l);
      bool off = (unsigned)id0 >= (unsigned)p.num_pages || (unsigned)id1 >= (unsigned)p.num_pages;
      for (int j = tid + 2 * kTcSoftmax; j < pages; j += kTcSoftmax)
        off |= (unsigned)__ldg(trow + page0 + j) >= (unsigned)p.num_pages;
      if (off) *s_bad = 1;
      softmax_sync();
      const bool gone = __any_sync(0xffffffffu, *s_abort != 0);
      const bool bad = *s_bad != 0, fix = *s_fix != 0;
      if (gone) dead = true;
      if (bad && tid == 0) kv_flag(p.status, SV_DEV_BAD_INDEX);
      auto row_stats = [&](int r, float& top, float& sum) {
        top = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * kCopies; ++j)
          top = fmaxf(top, s_ml[(j / kCopies) * 128 + (j % kCopies) * RT + r].x);
#pragma unroll
        for (int j = 0; j < 2 * kCopies; ++j) {
          const float2 ml = s_ml[(j / kCopies) * 128 + (j % kCopies) * RT + r];
          sum += top == -INFINITY ? ml.y : pow2(ml.x - top) * ml.y;
        }
        if (bad || gone) sum = __int_as_float(0x7fc00000);
      };
      float top, sum;
      row_stats(row, top, sum);
      const float f = top == -INFINITY ? 0.f : pow2(m - top);
      const bool whole = tile0 == 0 && cnt == cur.tiles;
      float* part = att_part<D, RT>(p, blockIdx.x, tile0 == 0);
      float* stage = reinterpret_cast<float*>(s_q);  // [2][128][kCols]
      constexpr int kPieces = C::kCols / 4;
      // a thread adds the same piece of the same rows in every round
      constexpr int kRowStep = kTcSoftmax / kPieces, kMine = (RT + kRowStep - 1) / kRowStep;
      const int piece = tid % kPieces, r_first = tid / kPieces;
      float inv[kMine];
      long long out_at[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = r_first + i * kRowStep;
        inv[i] = 0.f;
        out_at[i] = 0;
        if (r < rows) {
          float rt, rs;
          row_stats(r, rt, rs);
          inv[i] = 1.f / rs;
          out_at[i] = whole ? att_out_row(p, cur.b, h, row0 + r) * p.d : (long long)r * D;
        }
      }
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += C::kCols) {
        float4* dst = reinterpret_cast<float4*>(stage + (w * 128 + lr) * C::kCols);
        if (used && !gone) {
          if constexpr (C::kCols == 32) {
            uint32_t y[32];
            tc_ld(o_at + c0, y);
            tc_wait_ld(y);
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
              dst[j ^ (lr & (kPieces - 1))] = make_float4(
                  __uint_as_float(y[4 * j]) * f, __uint_as_float(y[4 * j + 1]) * f,
                  __uint_as_float(y[4 * j + 2]) * f, __uint_as_float(y[4 * j + 3]) * f);
          } else {
            uint32_t y[16];
            tc_ld(o_at + c0, y);
            tc_wait_ld(y);
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
              dst[j ^ (lr & (kPieces - 1))] = make_float4(
                  __uint_as_float(y[4 * j]) * f, __uint_as_float(y[4 * j + 1]) * f,
                  __uint_as_float(y[4 * j + 2]) * f, __uint_as_float(y[4 * j + 3]) * f);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kPieces; ++j) dst[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        softmax_sync();
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
          const int r = r_first + n * kRowStep, j = piece;
          if (r >= rows) continue;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 2 * kCopies; ++q) {
            const int at = (q / kCopies) * 128 + (q % kCopies) * RT + r;
            const float4 b = reinterpret_cast<const float4*>(
                stage + at * C::kCols)[j ^ (at & (kPieces - 1))];
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
          }
          const int col = c0 + j * 4;
          if (whole && col >= p.d) continue;
          if (fix && col < p.d) {
            const int i = fast_div(row0 + r, p.div_g);
            for (int t = max(0, tile0 * kTcU - kv); t < cur.q; ++t) {
              const int pos = kv + t;
              if (pos >= (tile0 + cnt) * kTcU) break;
              int up = i;
              if (!par) {
                up = t <= i ? t : -1;
              } else {
                while (up > t) {
                  const int above = par[up];
                  up = above < up ? above : -1;  // a bad parent ends the walk
                }
              }
              if (up != t) continue;
              const int pi = pos / p.page, id = trow[pi];
              if (id < 0 || id >= p.num_pages) continue;
              const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + id * p.c_page +
                                       (long long)(pos - pi * p.page) * p.c_token + h * p.c_head +
                                       col;
              const float y0 = __bfloat162float(v[0]), y1 = __bfloat162float(v[1]);
              const float y2 = __bfloat162float(v[2]), y3 = __bfloat162float(v[3]);
              if (not_finite(y0)) a.x += y0;
              if (not_finite(y1)) a.y += y1;
              if (not_finite(y2)) a.z += y2;
              if (not_finite(y3)) a.w += y3;
            }
          }
          if (whole) {
            uint2 y;
            y.x = pack_bf16(a.x * inv[n], a.y * inv[n]);
            y.y = pack_bf16(a.z * inv[n], a.w * inv[n]);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + out_at[n] + col) = y;
          } else {
            __stcg(reinterpret_cast<float4*>(part + out_at[n] + col), a);
          }
        }
        softmax_sync();
      }
      if (w == 0 && lr < rows) {
        if (whole) {
          if (p.lse) p.lse[att_out_row(p, cur.b, h, row0 + lr)] = (top + log2f(sum)) * kLn2;
        } else {
          __stcg(part + RT * D + lr, top);
          __stcg(part + RT * D + RT + lr, sum);
        }
      }
      if (!whole && tile0 == 0 && tid == 0)
        att_note(p, s, cur.b, h, row0, rows, cur.v + cur.tiles);
      tc_fence_before();
      if (tid == 0) *s_bad = *s_fix = 0;
      softmax_sync();  // before the next segment's q and flags
      cur = next;
    }
    if (dead && lane == 0) kv_flag(p.status, SV_DEV_TIMEOUT);
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace sv
