// sv_attend_f32.cuh -- fp32 attention of head sizes up to 128 (D is 64 or 128, the
// columns past the head size are zeros), up to 8 rows.
//
// A key costs 4 D rows operations against 8 D bytes: up to 4 rows the read of
// the cache is the bound (32 requests of 4000 keys, 8 key heads, 4 rows: 1.05 GB
// in 204 us, 5.1 TB/s), then the fp32 pipe (8 rows: 338 us).  The frame is that
// of the bf16 kernel of few rows: four warps, each with its own ring of 8-key
// steps, its own softmax and output.  Scores: four lanes share a key, each
// takes every fourth 16 bytes of the row; their sums are exchanged so that
// each of the four ends with a quarter of the rows.  Outputs: a lane holds
// D / 32 columns of all rows.  Products are packed pairs (one instruction for
// two of them); the weights lie twice in shared memory, so that pairs of them
// come out of it as they are used.
#pragma once

#include "sv_attend.cuh"
#include "sv_attend_mma.cuh"

namespace sv {

constexpr int kF32Threads = 128, kF32Warps = 4, kF32Keys = 8, kF32U = kF32Warps * kF32Keys;
constexpr int kF32Ov = 2;

template <int D, int RT>
struct F32Cfg {
  static constexpr int kRowBytes = 4 * D;
  static constexpr int kPlane = kF32Keys * kRowBytes;
  static constexpr int kStage = 2 * kPlane;
  static constexpr int kStages = D == 128 ? 3 : 6;  // 24 KB a warp
  static constexpr int kRing = kF32Warps * kStages * kStage;
  // q [RT][D] while tiles run; afterwards the warps' outputs, kOutRows rows at a time
  static constexpr int kOutRows = 4;
  static constexpr int kShared = (RT > 16 ? RT : 16) * D * 4;
  static constexpr int kP = kF32Warps * RT * kF32Keys * 8;  // weights, twice
  static constexpr int kSmem = kRing + kShared + kP + kF32Warps * RT * 8;
};

__device__ __forceinline__ void lds2(uint32_t a, unsigned long long& x, unsigned long long& y) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a) : "memory");
}
__device__ __forceinline__ unsigned long long lds1(uint32_t a) {
  unsigned long long x;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(x) : "r"(a) : "memory");
  return x;
}

template <int D, int RT>
__global__ void __launch_bounds__(kF32Threads, 2) attend_f32_kernel(const AttendParams p) {
  using C = F32Cfg<D, RT>;
  constexpr int kStages = C::kStages;
  constexpr int kRL = RT / 4;                  // rows of a lane in the softmax
  constexpr int kChunks = D / 4;               // 16-byte chunks of a row
  constexpr int kPerCopy = 32 / kChunks;       // rows copied by one instruction
  constexpr int kV = D / 32;                   // columns of a lane
  constexpr int kV2 = kV / 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int key = lane >> 2, quarter = lane & 3;
  unsigned char* ring = smem + warp * kStages * C::kStage;
  float* s_q = reinterpret_cast<float*>(smem + C::kRing);
  float2* s_p = reinterpret_cast<float2*>(smem + C::kRing + C::kShared) + warp * RT * kF32Keys;
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kRing + C::kShared + C::kP);  // [warp][row]
  const float* kc = static_cast<const float*>(p.k);
  const float* vc = static_cast<const float*>(p.v);

  if (tid == 0) att_clear_note(p);
  pdl_launch_dependents();
  AttCursor<kF32U, RT, kF32Ov> cur;
  const AttShare s = att_share<kF32Threads>(p, cur, s_q);

  // ---- the copies ---------------------------------------------------------
  AttCursor<kF32U, RT, kF32Ov> ahead = cur;
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
        const uint32_t to = dst + row * C::kRowBytes + ((c ^ ((row & 1) << 2)) << 4);
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
    const int h = cur.seg / cur.mt, row0 = (cur.seg % cur.mt) * RT;
    const int rows = min(RT, cur.q * p.g - row0);
    const int tile0 = cur.tile, left = cur.tiles - cur.tile;
    const int cnt = s.u1 - cur.v < left ? (int)(s.u1 - cur.v) : left;
    const int kv = cur.kv, len = cur.kv + cur.q;
    const int32_t* par = p.parents ? p.parents + (long long)cur.b * p.n : nullptr;
    __syncthreads();  // the last segment's outputs are read
    for (int e = tid; e < RT * D; e += kF32Threads) {
      const int r = e / D, d = e % D;
      float x = 0.f;
      if (r < rows && d < p.d) {
        const int i = fast_div(row0 + r, p.div_g), gi = (row0 + r) - i * p.g;
        x = static_cast<const float*>(p.q)[cur.b * p.q_b + i * p.q_t +
                                           (long long)(h * p.g + gi) * p.d + d];
      }
      s_q[e] = x;
    }
    __syncthreads();
    unsigned long long acc[RT][kV2];
    float m[kRL], l[kRL];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < kV2; ++e) acc[r][e] = 0;
#pragma unroll
    for (int i = 0; i < kRL; ++i) m[i] = -INFINITY, l[i] = 0.f;
    bool tree_ok = true, bad = false;

    for (int t = tile0; t < tile0 + cnt; ++t) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint32_t ka = smem_u32(ring + stage * C::kStage), va = ka + C::kPlane;
      bad |= (bad_stages >> stage) & 1u;
      // scores of this lane's key over its quarter of the columns
      unsigned long long z2[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) z2[r] = 0;
      {
        const uint32_t krow = ka + key * C::kRowBytes, qrow = smem_u32(s_q) + quarter * 16;
        const int flip = (key & 1) << 2;
#pragma unroll
        for (int i = 0; i < kChunks / 4; ++i) {
          unsigned long long k0, k1;
          lds2(krow + (((i * 4 + quarter) ^ flip) << 4), k0, k1);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            unsigned long long q0, q1;
            lds2(qrow + r * C::kRowBytes + i * 64, q0, q1);
            z2[r] = f2_fma(q0, k0, z2[r]);
            z2[r] = f2_fma(q1, k1, z2[r]);
          }
        }
      }
      // the four lanes of a key exchange, each keeps a quarter of the rows
      float x[kRL];
      {
        float z[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float a, b;
          f2_unpack(z2[r], a, b);
          z[r] = a + b;
        }
        float y[RT / 2];
        const bool up = quarter & 2, right = quarter & 1;
#pragma unroll
        for (int r = 0; r < RT / 2; ++r) {
          const float give = up ? z[r] : z[r + RT / 2];
          y[r] = (up ? z[r + RT / 2] : z[r]) + __shfl_xor_sync(0xffffffffu, give, 2);
        }
#pragma unroll
        for (int r = 0; r < kRL; ++r) {
          const float give = right ? y[r] : y[r + kRL];
          x[r] = (right ? y[r + kRL] : y[r]) + __shfl_xor_sync(0xffffffffu, give, 1);
        }
      }
      const int pos0 = t * kF32U + warp * kF32Keys;
      const bool tail = pos0 + kF32Keys > kv;
      float alpha[kRL];
      bool grew = false;
#pragma unroll
      for (int i = 0; i < kRL; ++i) {
        x[i] *= p.scale_log2;
        bool off = false;
        if (tail) {
          const int tok = min(fast_div(row0 + quarter * kRL + i, p.div_g), cur.q - 1);
          off = !(att_tail_bits<kF32Keys>(par, tok, pos0, kv, tree_ok) >> key & 1u);
          if (off) x[i] = -INFINITY;
        }
        float top = x[i];
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float mn = fmaxf(m[i], top);
        const float ms = mn == -INFINITY ? 0.f : mn;
        alpha[i] = exp2f(m[i] - ms);
        grew |= mn != m[i];
        m[i] = mn;
        x[i] = exp2f(x[i] - ms);
        if (tail) x[i] = att_mark_seen(x[i], off);
        l[i] = l[i] * alpha[i] + x[i];
        s_p[(quarter * kRL + i) * kF32Keys + key] = make_float2(x[i], x[i]);
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float a = __shfl_sync(0xffffffffu, alpha[r % kRL], r / kRL);
          const unsigned long long a2 = f2_pack(a, a);
#pragma unroll
          for (int e = 0; e < kV2; ++e) acc[r][e] = f2_fma(acc[r][e], a2, 0ull);
        }
      }
      __syncwarp();
      const uint32_t pa = smem_u32(s_p);
#pragma unroll
      for (int a = 0; a < kF32Keys / 2; ++a) {
        unsigned long long v0[kV2], v1[kV2];
        const uint32_t r0 = va + 2 * a * C::kRowBytes, r1 = r0 + C::kRowBytes;
        if constexpr (kV == 4) {
          lds2(r0 + (lane << 4), v0[0], v0[1]);
          lds2(r1 + ((lane ^ 4) << 4), v1[0], v1[1]);
        } else {
          v0[0] = lds1(r0 + lane * 8);
          v1[0] = lds1(r1 + ((lane >> 1 ^ 4) << 4) + (lane & 1) * 8);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          unsigned long long p0, p1;
          lds2(pa + (r * kF32Keys + 2 * a) * 8, p0, p1);
          if (!tail) {
#pragma unroll
            for (int e = 0; e < kV2; ++e) {
              acc[r][e] = f2_fma(p0, v0[e], acc[r][e]);
              acc[r][e] = f2_fma(p1, v1[e], acc[r][e]);
            }
          } else {
            // keys that only some rows see leave the others (weight +0) as
            // they are, whatever their values hold
#pragma unroll
            for (int e = 0; e < kV2; ++e) {
              if (p0 != 0) acc[r][e] = f2_fma(p0, v0[e], acc[r][e]);
              if (p1 != 0) acc[r][e] = f2_fma(p1, v1[e], acc[r][e]);
            }
          }
        }
      }
      __syncwarp();
      copy_next(stage == 0 ? kStages - 1 : stage - 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- the warps' results together -------------------------------------------
    const float nan = __int_as_float(0x7fc00000);
    tree_ok = __all_sync(0xffffffffu, tree_ok);
#pragma unroll
    for (int i = 0; i < kRL; ++i) {
      float y = l[i];
      y += __shfl_xor_sync(0xffffffffu, y, 4);
      y += __shfl_xor_sync(0xffffffffu, y, 8);
      y += __shfl_xor_sync(0xffffffffu, y, 16);
      if (bad || !tree_ok) y = nan;
      if (key == 0) s_ml[warp * RT + quarter * kRL + i] = make_float2(m[i], y);
    }
    if (lane == 0 && bad) kv_flag(p.status, SV_DEV_BAD_INDEX);
    if (lane == 0 && !tree_ok) kv_flag(p.status, SV_DEV_BAD_TREE);
    __syncthreads();  // also: q is read
    const bool whole = tile0 == 0 && cnt == cur.tiles;
    float* part = att_part<D, RT>(p, blockIdx.x, tile0 == 0);
    constexpr int kVecs = D / 4;
#pragma unroll
    for (int g0 = 0; g0 < RT; g0 += C::kOutRows) {
      if (g0 >= rows) break;
      if (g0) __syncthreads();
#pragma unroll
      for (int r = 0; r < C::kOutRows; ++r) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w) top = fmaxf(top, s_ml[w * RT + g0 + r].x);
        const float f = top == -INFINITY ? 0.f : exp2f(s_ml[warp * RT + g0 + r].x - top);
        const unsigned long long ff = f2_pack(f, f);
        unsigned long long* dst = reinterpret_cast<unsigned long long*>(
            s_q + (warp * C::kOutRows + r) * D + lane * kV);
#pragma unroll
        for (int e = 0; e < kV2; ++e) dst[e] = f2_fma(acc[g0 + r][e], ff, 0ull);
      }
      __syncthreads();
      for (int it = tid; it < C::kOutRows * kVecs; it += kF32Threads) {
        const int r = it / kVecs, c = it % kVecs, row = g0 + r;
        if (row >= rows) continue;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w) {
          const float4 b = reinterpret_cast<const float4*>(s_q + (w * C::kOutRows + r) * D)[c];
          a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
          top = fmaxf(top, s_ml[w * RT + row].x);
        }
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w) {
          const float2 ml = s_ml[w * RT + row];
          sum += top == -INFINITY ? ml.y : exp2f(ml.x - top) * ml.y;
        }
        if (whole) {
          const long long o = att_out_row(p, cur.b, h, row0 + row);
          if (c * 4 < p.d)
            reinterpret_cast<float4*>(static_cast<float*>(p.out) + o * p.d)[c] =
                make_float4(a.x / sum, a.y / sum, a.z / sum, a.w / sum);
          if (c == 0 && p.lse) p.lse[o] = (top + log2f(sum)) * kLn2;
        } else {
          __stcg(reinterpret_cast<float4*>(part + row * D) + c, a);
          if (c == 0) {
            __stcg(part + RT * D + row, top);
            __stcg(part + RT * D + RT + row, sum);
          }
        }
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
