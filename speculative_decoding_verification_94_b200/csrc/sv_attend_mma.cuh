// sv_attend_mma.cuh -- bf16 attention of few rows: one new token or a short
// chain, up to 16 rows (new tokens x query heads per key head) at a time, and
// up to 32 where the tensor-memory kernel does not take the call (pages that no
// tile is a multiple of, unaligned q, a scale that is not positive).  D is 64 or
// 128; the columns past a smaller head size are zeros that are never loaded.
//
// With so few rows each key and value byte is used about once, so the bound
// is the read of the cache: 4 D bytes of HBM per key against 4 D rows
// operations.  What counts is bytes in flight without pauses.  Four
// warps of a block take 16 keys each of a 64-key tile and work on their own:
// every warp has its own ring of tiles, filled by its own asynchronous
// copies, its own running softmax and its own output, so no barrier stands in
// the stream; the copies of the next segment are under way while a segment
// ends.  Only there do the warps meet, to add their outputs.
//
// Matrix products are m16n8k16: 16 rows of q against 8 keys, then the weights
// (in registers as the first product left them) against the values.
// The weights enter the second product as the sum of two bf16 numbers, which
// keeps them to 2^-16, as in the kernel of many rows: with one bf16 the
// output's error grows from 0.0017 (its own rounding) to 0.0021 of its size.
//
// Measured: 256 requests of 100 to 4000 tokens, 8 key heads, 4 rows: 2.19 GB
// in 331 to 339 us under ncu, 6.5 to 6.6 TB/s (of reads alone; a copy of as many
// bytes read and written runs at 6.55), 376 us a call among others.  At 16 rows
// and 32 requests of 700 to 9000 tokens this kernel and the tensor-memory one
// both take 65 us, at 28 rows 106 against 68 us; with 256 requests of 100 to 300
// tokens 53 against 82 us at 16 rows.
#pragma once

#include "sv_attend.cuh"

namespace sv {

// What a segment costs beside its tiles, in tiles (256 requests of 100 to 4000
// tokens, calls back to back: 358 us with 0, 338 with 1, 332 with 2 and with 4).
constexpr int kMmaOv = 2;
constexpr int kMmaThreads = 128, kMmaWarps = 4, kMmaKeys = 16, kMmaU = kMmaWarps * kMmaKeys;

template <int D, int MT>
struct MmaCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kPlane = kMmaKeys * kRowBytes;      // keys (or values) of a warp's step
  static constexpr int kStage = 2 * kPlane;
  static constexpr int kStages = D == 128 ? 3 : 6;         // 24 KB a warp
  static constexpr int kCols = 64 / MT;                    // output columns added at a time
  static constexpr int kRing = kMmaWarps * kStages * kStage;
  static constexpr int kMerge = kMmaWarps * kRows * kCols * 4;
  // of its own: nothing holds a warp back between the division of the work and
  // its first results, while others may still read their part of it
  static constexpr int kShare = kRing + kMerge;
  static constexpr int kSmem = kShare + kShareBytes;  // two blocks an SM
};

// 16 bytes, or zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two fp32 as bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ bool bf16x2_not_finite(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
// 2^x, two units in the last place; 0 for -inf.
__device__ __forceinline__ float pow2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The keys of [pos0, pos0 + COUNT) that token i sees, as bits, in a tile that
// reaches past the committed length.
template <int COUNT>
__device__ __forceinline__ uint32_t att_tail_bits(const int32_t* par, int i, int pos0, int kv,
                                                  bool& tree_ok) {
  const uint32_t all = COUNT == 32 ? 0xffffffffu : (1u << (COUNT & 31)) - 1u;
  const int lo = pos0 - kv;  // the tile's first key as a new token
  if (!par) {
    const int c = i + 1 - lo;
    return c >= COUNT ? all : c <= 0 ? 0u : (1u << c) - 1u;
  }
  if (lo >= 0) return att_tree_bits(par, i, lo, COUNT, tree_ok);
  return ((1u << -lo) - 1u) | (att_tree_bits(par, i, 0, COUNT + lo, tree_ok) << -lo);
}

template <int D, int MT>
__global__ void __launch_bounds__(kMmaThreads, 2) attend_mma_kernel(const AttendParams p) {
  using C = MmaCfg<D, MT>;
  constexpr int kRows = C::kRows, kStages = C::kStages;
  constexpr int kChunks = D / 8;              // 16-byte chunks of a row
  constexpr int kPerCopy = 32 / kChunks;      // rows that a warp's 32 lanes copy at once
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem + warp * kStages * C::kStage;
  float* merge = reinterpret_cast<float*>(smem + C::kRing);
  float2* s_ml = reinterpret_cast<float2*>(merge);  // [warp][row] (m, l), before the outputs
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(p.k);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(p.v);

  if (tid == 0) att_clear_note(p);
  pdl_launch_dependents();
  AttCursor<kMmaU, kRows, kMmaOv> cur;
  const AttShare s = att_share<kMmaThreads>(p, cur, smem + C::kShare);

  // ---- the copies: they run kStages - 1 tiles ahead of the products ---------
  AttCursor<kMmaU, kRows, kMmaOv> ahead = cur;
  uint32_t bad_stages = 0;
  // page of this lane's key in the tile to be copied next; -1: past the end
  auto page_of = [&]() {
    const int pos = ahead.tile * kMmaU + warp * kMmaKeys + (lane & 15);
    if (ahead.v >= s.u1 || pos >= ahead.kv + ahead.q) return -1;
    const int id = __ldg(p.table + (long long)ahead.b * p.max_pages + fast_div(pos, p.div_page));
    return id >= 0 && id < p.num_pages ? id : -2;
  };
  int page = page_of();
  auto copy_next = [&](int stage) {
    if (ahead.v < s.u1) {
      const int h = ahead.seg / ahead.mt;
      const int pos = ahead.tile * kMmaU + warp * kMmaKeys + (lane & 15);
      long long at = -1;
      if (page >= 0)
        at = page * p.c_page +
             (long long)(pos - fast_div(pos, p.div_page) * p.page) * p.c_token + h * p.c_head;
      const bool bad = __any_sync(0xffffffffu, page == -2);
      bad_stages = (bad_stages & ~(1u << stage)) | ((uint32_t)bad << stage);
      const uint32_t dst = smem_u32(ring + stage * C::kStage);
      const int c = lane % kChunks;
#pragma unroll
      for (int j = 0; j < kMmaKeys / kPerCopy; ++j) {
        const int row = j * kPerCopy + lane / kChunks;
        const long long o = __shfl_sync(0xffffffffu, at, row);
        const bool on = o >= 0 && c * 8 < p.d;
        const long long src = on ? o + c * 8 : 0;
        const uint32_t to = dst + row * C::kRowBytes + ((c ^ (row & 7)) << 4);
        cp_async16(to, kc + src, on);
        cp_async16(to + C::kPlane, vc + src, on);
      }
      ahead.step(p, 1);
      page = page_of();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) copy_next(j);
  int stage = 0;

  while (cur.v < s.u1) {
    const int h = cur.seg / cur.mt, row0 = (cur.seg % cur.mt) * kRows;
    const int rows = min(kRows, cur.q * p.g - row0);
    const int tile0 = cur.tile, left = cur.tiles - cur.tile;
    const int cnt = s.u1 - cur.v < left ? (int)(s.u1 - cur.v) : left;
    const int kv = cur.kv, len = cur.kv + cur.q;
    const int32_t* par = p.parents ? p.parents + (long long)cur.b * p.n : nullptr;

    // q fragments of the segment's rows
    uint32_t qa[MT][D / 16][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = row0 + mt * 16 + half * 8 + (lane >> 2);
        const bool on = r - row0 < rows;
        const int i = on ? fast_div(r, p.div_g) : 0, gi = on ? r - i * p.g : 0;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            static_cast<const __nv_bfloat16*>(p.q) + cur.b * p.q_b + i * p.q_t +
            (long long)(h * p.g + gi) * p.d + (lane & 3) * 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qa[mt][ks][half] = on && ks * 16 < p.d ? __ldg(src + ks * 8) : 0u;
          qa[mt][ks][half + 2] = on && ks * 16 + 8 < p.d ? __ldg(src + ks * 8 + 4) : 0u;
        }
      }
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    bool tree_ok = true, bad = false;

    for (int t = tile0; t < tile0 + cnt; ++t) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      unsigned char* kt = ring + stage * C::kStage;
      const uint32_t ka = smem_u32(kt), va = ka + C::kPlane;
      bad |= (bad_stages >> stage) & 1u;
      // scores
      float z[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[mt][0][e] = z[mt][1][e] = 0.f;
      {
        const int row = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t base = ka + row * C::kRowBytes;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b[4];
          ldmatrix4(base + (((2 * ks + ((lane >> 3) & 1)) ^ (row & 7)) << 4), b);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(z[mt][0], qa[mt][ks], b[0], b[1]);
            mma_bf16(z[mt][1], qa[mt][ks], b[2], b[3]);
          }
        }
      }
      const int pos0 = t * kMmaU + warp * kMmaKeys;
      const bool tail = pos0 + kMmaKeys > kv;
      uint32_t seen[MT][2];
      float alpha[MT][2];
      bool grew = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x[4] = {z[mt][0][2 * half], z[mt][0][2 * half + 1], z[mt][1][2 * half],
                        z[mt][1][2 * half + 1]};
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= p.scale_log2;
          seen[mt][half] = 0xffffu;
          if (tail) {
            const int r = row0 + mt * 16 + half * 8 + (lane >> 2);
            const int i = min(fast_div(r, p.div_g), cur.q - 1);
            const uint32_t bits = att_tail_bits<kMmaKeys>(par, i, pos0, kv, tree_ok);
            seen[mt][half] = bits;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(bits >> ((e >> 1) * 8 + (lane & 3) * 2 + (e & 1)) & 1u)) x[e] = -INFINITY;
          }
          float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float mn = fmaxf(m[mt][half], top);
          const float ms = mn == -INFINITY ? 0.f : mn;
          alpha[mt][half] = pow2(m[mt][half] - ms);
          grew |= mn != m[mt][half];
          m[mt][half] = mn;
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = pow2(x[e] - ms);
            sum += x[e];
          }
          l[mt][half] = l[mt][half] * alpha[mt][half] + sum;
          z[mt][0][2 * half] = x[0];
          z[mt][0][2 * half + 1] = x[1];
          z[mt][1][2 * half] = x[2];
          z[mt][1][2 * half + 1] = x[3];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < D / 8; ++nt) {
            o[mt][nt][0] *= alpha[mt][0];
            o[mt][nt][1] *= alpha[mt][0];
            o[mt][nt][2] *= alpha[mt][1];
            o[mt][nt][3] *= alpha[mt][1];
          }
      }
      // New tokens' values that are not finite would reach, as 0 x inf, rows
      // that do not see them: they are added to the rows that do, and leave
      // the product as zeros.
      if (tail && cur.q > 1) {
        bool found = false;
        for (int e = lane; e < kMmaKeys * kChunks; e += 32) {
          const int row = e / kChunks;
          if (pos0 + row < kv || pos0 + row >= len) continue;
          const uint4 x = *reinterpret_cast<const uint4*>(kt + C::kPlane + e * 16);
          found |= bf16x2_not_finite(x.x) || bf16x2_not_finite(x.y) || bf16x2_not_finite(x.z) ||
                   bf16x2_not_finite(x.w);
        }
        if (__any_sync(0xffffffffu, found)) {
          for (int row = 0; row < kMmaKeys; ++row) {
            if (pos0 + row < kv || pos0 + row >= len) continue;
#pragma unroll
            for (int nt = 0; nt < D / 8; ++nt) {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(
                  kt + C::kPlane + row * C::kRowBytes + ((nt ^ (row & 7)) << 4) + (lane & 3) * 4);
              const float v0 = bf16_lo(x), v1 = bf16_hi(x);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  if (seen[mt][half] >> row & 1u) {
                    if (not_finite(v0)) o[mt][nt][2 * half] += v0;
                    if (not_finite(v1)) o[mt][nt][2 * half + 1] += v1;
                  }
            }
          }
          __syncwarp();
          for (int e = lane; e < kMmaKeys * D; e += 32) {
            const int row = e / D;
            if (pos0 + row < kv || pos0 + row >= len) continue;
            uint16_t* x = reinterpret_cast<uint16_t*>(kt + C::kPlane) + e;
            if ((*x & 0x7f80u) == 0x7f80u) *x = 0;
          }
          __syncwarp();
        }
      }
      // weights x values
      uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (row g, keys 0-7), (g + 8, 0-7), (g, 8-15), (g + 8, 8-15)
          const float a = z[mt][j >> 1][2 * (j & 1)], b = z[mt][j >> 1][2 * (j & 1) + 1];
          ph[mt][j] = pack_bf16(a, b);
          pl[mt][j] = pack_bf16(a - bf16_lo(ph[mt][j]), b - bf16_hi(ph[mt][j]));
        }
      {
        const int row = lane & 15;
        const uint32_t base = va + row * C::kRowBytes;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t b[4];
          ldmatrix4_t(base + (((2 * j + (lane >> 4)) ^ (row & 7)) << 4), b);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16(o[mt][2 * j], ph[mt], b[0], b[1]);
            mma_bf16(o[mt][2 * j + 1], ph[mt], b[2], b[3]);
            mma_bf16(o[mt][2 * j], pl[mt], b[0], b[1]);
            mma_bf16(o[mt][2 * j + 1], pl[mt], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      copy_next(stage == 0 ? kStages - 1 : stage - 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- the warps' results together -------------------------------------------
    const float nan = __int_as_float(0x7fc00000);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x = l[mt][half];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const int r = mt * 16 + half * 8 + (lane >> 2);
        if (!tree_ok && r < rows) kv_flag(p.status, SV_DEV_BAD_TREE);
        if (bad || !tree_ok) x = nan;
        if ((lane & 3) == 0) s_ml[warp * kRows + r] = make_float2(m[mt][half], x);
      }
    if (bad && lane == 0) kv_flag(p.status, SV_DEV_BAD_INDEX);
    __syncthreads();
    float f[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + (lane >> 2);
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s_ml[w * kRows + r].x);
        f[mt][half] = top == -INFINITY ? 0.f : pow2(m[mt][half] - top);
      }
    // columns kCols at a time through shared memory; a thread then holds
    // eight columns of one row
    constexpr int kThreadsPerRow = C::kCols / 8;
    const int orow = tid / kThreadsPerRow, ocol = (tid % kThreadsPerRow) * 8;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s_ml[w * kRows + orow].x);
#pragma unroll
    for (int w = 0; w < kMmaWarps; ++w) {
      const float2 ml = s_ml[w * kRows + orow];
      sum += top == -INFINITY ? ml.y : pow2(ml.x - top) * ml.y;
    }
    const bool whole = tile0 == 0 && cnt == cur.tiles;
    float* part = att_part<D, kRows>(p, blockIdx.x, tile0 == 0);
    const long long orow_at = att_out_row(p, cur.b, h, row0 + min(orow, rows - 1));
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += C::kCols) {
      __syncthreads();  // s_ml, then the last columns, are read
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < C::kCols / 8; ++nt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = mt * 16 + half * 8 + (lane >> 2);
            const int col = (nt * 8 + (lane & 3) * 2) ^ ((r & 3) << 3);
            *reinterpret_cast<float2*>(merge + (warp * kRows + r) * C::kCols + col) =
                make_float2(o[mt][c0 / 8 + nt][2 * half] * f[mt][half],
                            o[mt][c0 / 8 + nt][2 * half + 1] * f[mt][half]);
          }
      __syncthreads();
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kMmaWarps; ++w) {
        const float4* src = reinterpret_cast<const float4*>(
            merge + (w * kRows + orow) * C::kCols + (ocol ^ ((orow & 3) << 3)));
        const float4 a = src[0], b = src[1];
        x[0] += a.x, x[1] += a.y, x[2] += a.z, x[3] += a.w;
        x[4] += b.x, x[5] += b.y, x[6] += b.z, x[7] += b.w;
      }
      if (orow < rows) {
        if (whole) {
          const float inv = 1.f / sum;
          uint4 y;
          y.x = pack_bf16(x[0] * inv, x[1] * inv);
          y.y = pack_bf16(x[2] * inv, x[3] * inv);
          y.z = pack_bf16(x[4] * inv, x[5] * inv);
          y.w = pack_bf16(x[6] * inv, x[7] * inv);
          if (c0 + ocol < p.d)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow_at * p.d + c0 +
                                      ocol) = y;
        } else {
          float4* dst = reinterpret_cast<float4*>(part + orow * D + c0 + ocol);
          __stcg(dst, make_float4(x[0], x[1], x[2], x[3]));
          __stcg(dst + 1, make_float4(x[4], x[5], x[6], x[7]));
        }
      }
    }
    if (ocol == 0 && orow < rows) {
      if (whole) {
        if (p.lse) p.lse[orow_at] = (top + log2f(sum)) * kLn2;
      } else {
        __stcg(part + kRows * D + orow, top);
        __stcg(part + kRows * D + kRows + orow, sum);
      }
    }
    if (!whole && tile0 == 0 && tid == 0)
      att_note(p, s, cur.b, h, row0, rows, cur.v + cur.tiles);
    __syncthreads();  // merge is free again
    cur.step(p, cnt);
  }
  cp_async_wait<0>();
  att_fill_padding<__nv_bfloat16>(p, 0, kMmaWarps);
}

}  // namespace sv
