// sv_attend_tf32.cuh -- fp32 attention of more than 8 rows, 16 at a time, for
// head sizes up to 128 (D is 64 or 128, the columns past the head size are
// zeros).
//
// From 16 rows on the fp32 pipe is the bound by far (32 requests of 4000 keys,
// 16 rows: 680 us against 160 us for the read; this kernel 291).  Here the
// products go through the tensor cores in tf32, which has 11 bits: each operand
// is the sum of two tf32 numbers, x = h + l, and a product is three, h h' + h l' + l h'.
// Weights and q round h to nearest (|l| <= 2^-11 |x|), keys and values cut
// it off (|l| <= 2^-10 |x|, one instruction, and nothing overflows); l rounds
// to nearest.  What that leaves out of a product is at most 2^-21 + 2^-21 +
// 2^-22 of it, 20 half steps of fp32, where the sum over the head size
// already has d of them.
//
// The frame is that of the other kernels of few rows: four warps with their own
// rings of 8-key steps.  q lies in shared memory in its two parts.  A warp's
// first product is m16n8k8 over the head size; its weights are, in registers,
// the second product's operand if the summation index t stands for key 2t
// and t + 4 for key 2t + 1, which is how the values are loaded.
#pragma once

#include "sv_attend.cuh"
#include "sv_attend_f32.cuh"
#include "sv_attend_mma.cuh"

namespace sv {

template <int D>
struct Tf32Cfg {
  static constexpr int kRows = 16;
  static constexpr int kRowBytes = 4 * D;
  static constexpr int kPlane = kF32Keys * kRowBytes;
  static constexpr int kStage = 2 * kPlane;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kCols = 64;  // output columns added at a time
  static constexpr int kRing = kF32Warps * kStages * kStage;
  static constexpr int kQ = kRows * kRowBytes;  // one part of q
  static constexpr int kMerge = kF32Warps * kRows * kCols * 4;  // over q, when it is used up
  static constexpr int kSmem = kRing + (2 * kQ > kMerge ? 2 * kQ : kMerge);
};

__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void split_tf32(float x, uint32_t& h, uint32_t& l) {
  h = to_tf32(x);
  l = to_tf32(x - __uint_as_float(h));
}
// As split_tf32, for any finite x: what would round up past the largest number
// is cut off, by at most 2^-11 of it there too.
__device__ __forceinline__ void split_tf32_any(float x, uint32_t& h, uint32_t& l) {
  h = to_tf32(x);
  if (not_finite(__uint_as_float(h))) h = __float_as_uint(x) & 0xffffe000u;
  l = to_tf32(x - __uint_as_float(h));
}
__device__ __forceinline__ void cut_tf32(float x, uint32_t& h, uint32_t& l) {
  h = __float_as_uint(x) & 0xffffe000u;
  l = to_tf32(x - __uint_as_float(h));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A B alone.  The tensor core cuts its sums off, which adds up over thousands
// of steps (60,000 keys: an error of 1.7e-5 of the output, 7.5e-7 without): a
// step's product, and every four of a score, are added by fp32 additions.
__device__ __forceinline__ void mma_tf32_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int D>
__global__ void __launch_bounds__(kF32Threads, 2) attend_tf32_kernel(const AttendParams p) {
  using C = Tf32Cfg<D>;
  constexpr int kRows = 16, kStages = C::kStages;
  constexpr int kChunks = D / 4;          // 16-byte chunks of a row
  constexpr int kPerCopy = 32 / kChunks;  // rows copied by one instruction
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem + warp * kStages * C::kStage;
  unsigned char* s_q = smem + C::kRing;  // first parts, then rests; rows swizzled as in the ring
  float* merge = reinterpret_cast<float*>(s_q);
  float2* s_ml = reinterpret_cast<float2*>(merge);  // [warp][row] (m, l), before the outputs
  const float* kc = static_cast<const float*>(p.k);
  const float* vc = static_cast<const float*>(p.v);

  if (tid == 0) att_clear_note(p);
  pdl_launch_dependents();
  AttCursor<kF32U, kRows, kF32Ov> cur;
  const AttShare s = att_share<kF32Threads>(p, cur, merge);

  // ---- the copies ---------------------------------------------------------
  AttCursor<kF32U, kRows, kF32Ov> ahead = cur;
  uint32_t bad_stages = 0;
  auto page_of = [&]() {  // -1: past the end, -2: not in the pool
    const int pos = ahead.tile * kF32U + warp * kF32Keys + (lane & 7);
    if (ahead.v >= s.u1 || pos >= ahead.kv + ahead.q) return -1;
    const int id = __ldg(p.table + (long long)ahead.b * p.max_pages + fast_div(pos, p.div_page));
    return id >= 0 && id < p.num_pages ? id : -2;
  };
  int page = page_of();
  auto copy_next = [&](int stage) {
    if (ahead.v < s.u1) {
      const int h = ahead.seg / ahead.mt;
      const int pos = ahead.tile * kF32U + warp * kF32Keys + (lane & 7);
      long long at = -1;
      if (page >= 0)
        at = page * p.c_page +
             (long long)(pos - fast_div(pos, p.div_page) * p.page) * p.c_token + h * p.c_head;
      const bool bad = __any_sync(0xffffffffu, page == -2);
      bad_stages = (bad_stages & ~(1u << stage)) | ((uint32_t)bad << stage);
      const uint32_t dst = smem_u32(ring + stage * C::kStage);
      const int c = lane % kChunks;
#pragma unroll
      for (int j = 0; j < kF32Keys / kPerCopy; ++j) {
        const int row = j * kPerCopy + lane / kChunks;
        const long long o = __shfl_sync(0xffffffffu, at, row);
        const bool on = o >= 0 && c * 4 < p.d;
        const long long src = on ? o + c * 4 : 0;
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
    __syncthreads();  // the last segment's outputs are read
    for (int e = tid; e < kRows * D; e += kF32Threads) {
      const int r = e / D, d = e % D;
      float x = 0.f;
      if (r < rows && d < p.d) {
        const int i = fast_div(row0 + r, p.div_g), gi = (row0 + r) - i * p.g;
        x = static_cast<const float*>(p.q)[cur.b * p.q_b + i * p.q_t +
                                           (long long)(h * p.g + gi) * p.d + d];
      }
      uint32_t hi, lo;
      split_tf32_any(x, hi, lo);
      uint32_t* at = reinterpret_cast<uint32_t*>(s_q + r * C::kRowBytes +
                                                 (((d >> 2) ^ (r & 7)) << 4)) + (d & 3);
      at[0] = hi;
      at[C::kQ / 4] = lo;
    }
    __syncthreads();
    float o[1][D / 8][4], m[1][2], l[1][2];
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][nt][e] = 0.f;
    m[0][0] = m[0][1] = -INFINITY;
    l[0][0] = l[0][1] = 0.f;
    bool tree_ok = true, bad = false;

    for (int t = tile0; t < tile0 + cnt; ++t) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      unsigned char* kt = ring + stage * C::kStage;
      const uint32_t ka = smem_u32(kt);
      bad |= (bad_stages >> stage) & 1u;
      // scores: rows lane / 4 and + 8, keys 2 (lane % 4) and + 1
      float z[4] = {0.f, 0.f, 0.f, 0.f}, zl[4] = {0.f, 0.f, 0.f, 0.f}, z4[4];
      {
        const uint32_t krow = ka + (lane & 7) * C::kRowBytes;
        const int qr = lane & 15;
        const uint32_t qrow = smem_u32(s_q) + qr * C::kRowBytes;
#pragma unroll
        for (int ks = 0; ks < D / 8; ks += 2) {
          uint32_t kf[4];  // chunks 2 ks .. 2 ks + 3 of 8 keys
          ldmatrix4(krow + (((2 * ks + (lane >> 3)) ^ (lane & 7)) << 4), kf);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t qh[4], ql[4], h0, l0, h1, l1;
            const uint32_t at = qrow + (((2 * (ks + j) + (lane >> 4)) ^ (qr & 7)) << 4);
            ldmatrix4(at, qh);
            ldmatrix4(at + C::kQ, ql);
            cut_tf32(__uint_as_float(kf[2 * j]), h0, l0);
            cut_tf32(__uint_as_float(kf[2 * j + 1]), h1, l1);
            if (ks % 4 == 0 && j == 0)
              mma_tf32_first(z4, qh, h0, h1);
            else
              mma_tf32(z4, qh, h0, h1);
            mma_tf32(zl, qh, l0, l1);
            mma_tf32(zl, ql, h0, h1);
          }
          if (ks % 4 == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += z4[e];
          }
        }
      }
      const int pos0 = t * kF32U + warp * kF32Keys;
      const bool tail = pos0 + kF32Keys > kv;
      uint32_t seen[2];
      float alpha[2], w[4];
      bool grew = false;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[2] = {(z[2 * half] + zl[2 * half]) * p.scale_log2,
                      (z[2 * half + 1] + zl[2 * half + 1]) * p.scale_log2};
        seen[half] = 0xffu;
        if (tail) {
          const int i =
              min(fast_div(row0 + half * 8 + (lane >> 2), p.div_g), cur.q - 1);
          const uint32_t bits = att_tail_bits<kF32Keys>(par, i, pos0, kv, tree_ok);
          seen[half] = bits;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!(bits >> ((lane & 3) * 2 + e) & 1u)) x[e] = -INFINITY;
        }
        float top = fmaxf(x[0], x[1]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[0][half], top);
        const float ms = mn == -INFINITY ? 0.f : mn;
        alpha[half] = exp2f(m[0][half] - ms);
        grew |= mn != m[0][half];
        m[0][half] = mn;
        w[2 * half] = exp2f(x[0] - ms);
        w[2 * half + 1] = exp2f(x[1] - ms);
        l[0][half] = l[0][half] * alpha[half] + (w[2 * half] + w[2 * half + 1]);
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) {
          o[0][nt][0] *= alpha[0];
          o[0][nt][1] *= alpha[0];
          o[0][nt][2] *= alpha[1];
          o[0][nt][3] *= alpha[1];
        }
      }
      // New tokens' values that are not finite would reach, as 0 x inf, rows
      // that do not see them: they are added to the rows that do, and leave
      // the product as zeros.
      if (tail && cur.q > 1) {
        bool found = false;
        for (int e = lane; e < kF32Keys * D; e += 32) {
          const int r = e / D;
          if (pos0 + r >= kv && pos0 + r < len)
            found |= not_finite(reinterpret_cast<const float*>(kt + C::kPlane)[e]);
        }
        if (__any_sync(0xffffffffu, found)) {
          for (int r = 0; r < kF32Keys; ++r) {
            if (pos0 + r < kv || pos0 + r >= len) continue;
#pragma unroll
            for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int d = nt * 8 + (lane & 3) * 2 + e;
                const float v = reinterpret_cast<const float*>(
                    kt + C::kPlane + r * C::kRowBytes + (((d >> 2) ^ (r & 7)) << 4))[d & 3];
                if (!not_finite(v)) continue;
                if (seen[0] >> r & 1u) o[0][nt][e] += v;
                if (seen[1] >> r & 1u) o[0][nt][2 + e] += v;
              }
          }
          __syncwarp();
          for (int e = lane; e < kF32Keys * D; e += 32) {
            const int r = e / D;
            float* x = reinterpret_cast<float*>(kt + C::kPlane) + e;
            if (pos0 + r >= kv && pos0 + r < len && not_finite(*x)) *x = 0.f;
          }
          __syncwarp();
        }
      }
      // weights x values
      {
        // (row g, key 2t), (g + 8, 2t), (g, 2t + 1), (g + 8, 2t + 1)
        uint32_t ph[4], pl[4];
        split_tf32(w[0], ph[0], pl[0]);
        split_tf32(w[2], ph[1], pl[1]);
        split_tf32(w[1], ph[2], pl[2]);
        split_tf32(w[3], ph[3], pl[3]);
        const int k0 = (lane & 3) * 2, g = lane >> 2;
        const float* v0 = reinterpret_cast<const float*>(kt + C::kPlane + k0 * C::kRowBytes);
        const float* v1 = v0 + D;
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt) {
          const int c = nt * 2 + (g >> 2);
          uint32_t h0, l0, h1, l1;
          cut_tf32(v0[((c ^ k0) << 2) + (g & 3)], h0, l0);
          cut_tf32(v1[((c ^ (k0 + 1)) << 2) + (g & 3)], h1, l1);
          float c4[4];
          mma_tf32_first(c4, pl, h0, h1);
          mma_tf32(c4, ph, l0, l1);
          mma_tf32(c4, ph, h0, h1);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[0][nt][e] += c4[e];
        }
      }
      __syncwarp();
      copy_next(stage == 0 ? kStages - 1 : stage - 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- the warps' results together -------------------------------------------
    const float nan = __int_as_float(0x7fc00000);
    __syncthreads();  // q is read
#pragma unroll
    for (int mt = 0; mt < 1; ++mt)
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
    float f[1][2];
#pragma unroll
    for (int mt = 0; mt < 1; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + (lane >> 2);
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w) top = fmaxf(top, s_ml[w * kRows + r].x);
        f[mt][half] = top == -INFINITY ? 0.f : exp2f(m[mt][half] - top);
      }
    // columns kCols at a time through shared memory; a thread then holds
    // eight columns of one row
    constexpr int kThreadsPerRow = C::kCols / 8;
    const int orow = tid / kThreadsPerRow, ocol = (tid % kThreadsPerRow) * 8;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kF32Warps; ++w) top = fmaxf(top, s_ml[w * kRows + orow].x);
#pragma unroll
    for (int w = 0; w < kF32Warps; ++w) {
      const float2 ml = s_ml[w * kRows + orow];
      sum += top == -INFINITY ? ml.y : exp2f(ml.x - top) * ml.y;
    }
    const bool whole = tile0 == 0 && cnt == cur.tiles;
    float* part = att_part<D, 16>(p, blockIdx.x, tile0 == 0);
    const long long orow_at = att_out_row(p, cur.b, h, row0 + min(orow, rows - 1));
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += C::kCols) {
      __syncthreads();  // s_ml, then the last columns, are read
#pragma unroll
      for (int mt = 0; mt < 1; ++mt)
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
      for (int w = 0; w < kF32Warps; ++w) {
        const float4* src = reinterpret_cast<const float4*>(
            merge + (w * kRows + orow) * C::kCols + (ocol ^ ((orow & 3) << 3)));
        const float4 a = src[0], b = src[1];
        x[0] += a.x, x[1] += a.y, x[2] += a.z, x[3] += a.w;
        x[4] += b.x, x[5] += b.y, x[6] += b.z, x[7] += b.w;
      }
      if (orow < rows) {
        if (whole) {
          const float inv = 1.f / sum;
          float4* dst =
              reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow_at * p.d + c0 + ocol);
          if (c0 + ocol < p.d) dst[0] = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
          if (c0 + ocol + 4 < p.d)
            dst[1] = make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
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
    cur.step(p, cnt);
  }
  cp_async_wait<0>();
  att_fill_padding<float>(p, 0, kF32Warps);
}

}  // namespace sv
