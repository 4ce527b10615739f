// sv_attend.cuh -- attention of a step's new tokens over the paged cache:
// the division of the work, the join of split sequences, and the general
// kernel (any type, head size, stride and alignment).
//
// For a request with a committed tokens and m new ones (a chain or a tree),
// the row of token i and query head x attends to the keys
//   S_i = [0, a) + {a + j : j is i or an ancestor of i},
//   o = sum_{j in S_i} e^{z_j - lse} v_j,  z_j = scale q . k_j,
//   lse = log sum_{j in S_i} e^{z_j}.
// The rows of all new tokens and of the query heads that share a key head are
// computed together, so a key is read once for all of them.  The softmax is
// the running one: a maximum m, a sum l of e^{z - m} and the unnormalised
// output, all in fp32, rescaled when m grows; parts of a sequence computed
// apart join by the same rescaling.  Exponentials are powers of two of
// z log2 e.
//
// Division.  The lengths live on the device, so the grid does not know them.
// A unit is one tile of keys of one (request, key head, row tile); the units
// of all requests in order are cut into as many equal runs as there are
// blocks.  A block therefore holds at most two segments that it shares with
// other blocks, its first and its last; their partial results (output, m, l)
// go to the scratch buffer, and a second launch joins them in block order.  (The
// last block to finish a segment joined them at first: 128 rows of a few
// parts, or 40 rows of 19, are 0.4 MB to read and clear, 10 to 27 us on one
// SM and 3 us over all of them.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sv_device.cuh"
#include "sv_internal.h"
#include "sv_kv_pages.cuh"

namespace sv {

// A segment that starts in a block and ends in block c1 (c1 < 0: none).
struct AttShared {
  int b, h, row0, rows, c1, pad[3];
};

struct AttendParams {
  const void* q;
  const void *k, *v;
  const int32_t *table, *kv_len, *q_len, *parents;
  void* out;
  float* lse;
  int B, n, hkv, g, d, page, num_pages, max_pages;
  long long q_b, q_t;                 // strides of q, elements
  long long c_page, c_token, c_head;  // strides of the cache, elements
  float scale_log2;
  FastDiv div_g, div_page;
  AttShared* shared;  // [grid] the shared segment that starts in block i
  float* partial;            // [grid][2] partial results
  int32_t* status;
};

constexpr int kAttMaxBlocks = 296;  // two blocks on each of 148 SMs
constexpr long long kAttMaxLen = 0x7fffff00;  // a tile past the end still has int positions
constexpr float kLn2 = 0.69314718055994530942f;

// A row tile's partial result: o [rows][DP], then m [rows], l [rows].
__host__ __device__ constexpr int att_partial_floats(int rows, int dp) { return rows * (dp + 2); }

__device__ __forceinline__ float warp_add(float x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Lengths of a request: false if they are out of range (the request fails).
__device__ __forceinline__ bool att_lens(const AttendParams& p, int b, int& kv, int& q) {
  q = p.q_len ? p.q_len[b] : p.n;
  kv = p.kv_len[b];
  if (q == 0) return true;
  return q > 0 && q <= p.n && kv >= 0 && (long long)kv + q <= (long long)p.max_pages * p.page &&
         (long long)kv + q <= kAttMaxLen;
}

// The walk over units: requests, then segments (key head, row tile), then
// tiles of U keys.  A segment counts OV units more than its tiles, which
// stand before its first tile: what it costs to begin and end one, so that
// blocks with many short segments get fewer tiles.
template <int U, int RT, int OV>
struct AttCursor {
  int b, seg, tile, tiles, mt, kv, q;
  long long v;  // the tile's unit
  __device__ __forceinline__ long long load(const AttendParams& p) {  // units of request b
    tiles = mt = 0;
    if (b >= p.B || !att_lens(p, b, kv, q) || q == 0) return 0;
    tiles = (int)(((long long)kv + q + U - 1) / U);
    mt = (q * p.g + RT - 1) / RT;
    return (long long)(tiles + OV) * mt * p.hkv;
  }
  __device__ __forceinline__ void place(long long unit, long long off) {  // off: in the request
    seg = (int)(off / (tiles + OV));
    const int r = (int)(off - (long long)seg * (tiles + OV)) - OV;
    tile = r < 0 ? 0 : r;
    v = unit + (tile - r);
  }
  // `count` tiles on, within the segment or to the next one.  All lanes of a
  // warp come here together: past a request's last segment they look at 32
  // requests at a time, since a batch may be idle but for a few.
  __device__ __forceinline__ void step(const AttendParams& p, int count) {
    tile += count;
    v += count;
    if (tile < tiles) return;
    v += OV;
    tile = 0;
    if (++seg < mt * p.hkv) return;
    seg = 0;
    while (b < p.B) {
      const int at = b + 1 + (threadIdx.x & 31);
      int kv1, q1;
      const bool has = at < p.B && att_lens(p, at, kv1, q1) && q1 > 0;
      const uint32_t found = __ballot_sync(0xffffffffu, has);
      if (found) {
        b += __ffs(found);
        load(p);
        return;
      }
      b += 32;
    }
  }
};

struct AttShare {
  long long total, u0, u1;  // all units; this block's run
  int blocks;               // blocks with work
  __device__ __forceinline__ long long start(int c) const { return total * c / blocks; }
  __device__ __forceinline__ int block_of(long long u) const {
    return (int)(((u + 1) * blocks - 1) / total);
  }
};

// Every block sums the units of all requests and finds its own run.  `scratch`
// is kShareBytes of shared memory, read until every thread has returned: it is
// written again after a barrier or not at all.
constexpr int kShareBytes = 128;
template <int THREADS, int U, int RT, int OV>
__device__ __forceinline__ AttShare att_share(const AttendParams& p, AttCursor<U, RT, OV>& cur,
                                              void* scratch) {
  static_assert(8 * (THREADS / 32 + 2) <= kShareBytes, "");
  long long* s_sum = static_cast<long long*>(scratch);
  long long& s_off = s_sum[THREADS / 32];
  int& s_b = *reinterpret_cast<int*>(s_sum + THREADS / 32 + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = tid * per;
  long long sum = 0;
  for (int j = 0; j < per; ++j) {
    cur.b = b0 + j;
    sum += cur.load(p);
  }
  long long inc = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += a;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) inc += s_sum[w];
    total += s_sum[w];
  }
  AttShare s;
  s.total = total;
  s.blocks = total < (long long)gridDim.x ? (int)total : (int)gridDim.x;
  s.u0 = s.u1 = 0;
  if ((int)blockIdx.x < s.blocks) {
    s.u0 = s.start(blockIdx.x);
    s.u1 = s.start(blockIdx.x + 1);
    long long at = inc - sum;
    if (s.u0 >= at && s.u0 < inc) {
      for (int j = 0; j < per; ++j) {
        cur.b = b0 + j;
        const long long u = cur.load(p);
        if (s.u0 < at + u) {
          s_b = cur.b;
          s_off = s.u0 - at;
          break;
        }
        at += u;
      }
    }
  }
  __syncthreads();
  cur.v = s.u1;
  if (s.u0 < s.u1) {
    cur.b = s_b;
    cur.load(p);
    cur.place(s.u0, s_off);
  }
  return s;
}

// Does the row of token i attend to the key at position pos >= kv?  Chains:
// pos - kv <= i.  Trees: the keys of one tile as bits, found by walking up
// from i; false in `ok` for a parent that is not an earlier node or -1.
__device__ __forceinline__ uint32_t att_tree_bits(const int32_t* parents, int i, int lo, int count,
                                                  bool& ok) {
  uint32_t bits = 0;
  int a = i;
  while (a >= lo) {
    if (a - lo < count) bits |= 1u << (a - lo);
    const int up = parents[a];
    if (up >= a || up < -1) {
      ok = false;
      break;
    }
    a = up;
  }
  return bits;
}

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// In a tile that only some rows see all of, a weight of +0 says that the row
// does not attend to the key; one that has underflowed becomes -0.
__device__ __forceinline__ float att_mark_seen(float w, bool off) {
  return w == 0.f && !off ? -0.f : w;
}
__device__ __forceinline__ bool not_finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u;
}

// Output row of tile row r: token and query head.
__device__ __forceinline__ long long att_out_row(const AttendParams& p, int b, int h, int r) {
  const int i = fast_div(r, p.div_g);
  return ((long long)b * p.n + i) * ((long long)p.hkv * p.g) + (long long)h * p.g + (r - i * p.g);
}

// Tokens that no row was computed for: zeros and lse -inf for those behind a
// request's own, NaN for a failed request.
// Warps [w0, w0 + warps) of every block take part.
template <class T>
__device__ __forceinline__ void att_fill_padding(const AttendParams& p, int w0, int warps) {
  const int hq = p.hkv * p.g, lane = threadIdx.x & 31;
  const long long tokens = (long long)p.B * p.n;
  const long long step = (long long)gridDim.x * warps;
  const long long mine = (long long)blockIdx.x * warps + (threadIdx.x >> 5) - w0;
  // a lane looks at a token, the warp fills those that need it
  for (long long t0 = mine; t0 < tokens; t0 += 32 * step) {
    const long long t = t0 + lane * step;
    int what = 0;
    if (t < tokens) {
      const int b = (int)(t / p.n), i = (int)(t - (long long)b * p.n);
      int kv, q;
      if (!att_lens(p, b, kv, q)) {
        what = 2;
        if (i == 0) kv_flag(p.status, SV_DEV_BAD_LEN);
      } else if (i >= q) {
        what = 1;
      }
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, what != 0); left; left &= left - 1) {
      const int j = __ffs(left) - 1;
      const bool bad = __shfl_sync(0xffffffffu, what, j) == 2;
      const long long at = (t0 + j * step) * hq;
      const float nan = __int_as_float(0x7fc00000);
      const T z = from_f32<T>(bad ? nan : 0.f);
      T* o = static_cast<T*>(p.out) + at * p.d;
      for (int e = lane; e < hq * p.d; e += 32) o[e] = z;
      if (p.lse)
        for (int e = lane; e < hq; e += 32) p.lse[at + e] = bad ? nan : -INFINITY;
    }
  }
}

// The place of a block's part of a segment it shares; the block in which the
// segment starts keeps it in its second place and notes the segment.
template <int DP, int RT>
__device__ __forceinline__ float* att_part(const AttendParams& p, int block, bool starts) {
  return p.partial + ((long long)block * 2 + starts) * att_partial_floats(RT, DP);
}
__device__ __forceinline__ void att_note(const AttendParams& p, const AttShare& s, int b, int h,
                                         int row0, int rows, long long seg_u1) {
  p.shared[blockIdx.x] = AttShared{b, h, row0, rows, s.block_of(seg_u1 - 1), {0, 0, 0}};
}
// Before any note, by one thread of every block.
__device__ __forceinline__ void att_clear_note(const AttendParams& p) {
  p.shared[blockIdx.x].c1 = -1;
}

// Joins the parts of shared segments: block x takes the segment that starts
// in block x of the first launch.  kSplit warps share a row's parts; lanes
// hold the parts' weights, then the row's values, eight parts in flight.
constexpr int kJoinThreads = 128;
template <class T, int DP, int RT>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendParams p) {
  constexpr int kSplit = RT >= 128 ? 1 : RT == 64 ? 2 : 4;  // RT 4 to 32: 4
  constexpr int kRowsHere = 4 / kSplit;
  constexpr int kV = DP / 32;  // values of a lane
  constexpr int kBatch = 8;
  __shared__ float s_m[4], s_l[4], s_o[4][DP];
  pdl_wait();
  const AttShared g = p.shared[blockIdx.x];
  if (g.c1 < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % kSplit;
  const int r = blockIdx.y * kRowsHere + warp / kSplit;
  const int parts = g.c1 - (int)blockIdx.x + 1;
  if (blockIdx.y * kRowsHere >= g.rows) return;
  const bool on = r < g.rows;
  auto part = [&](int j) { return att_part<DP, RT>(p, blockIdx.x + j, j == 0); };
  float m = -INFINITY, l = 0.f, acc[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] = 0.f;
  if (on) {
    for (int j = lane * kSplit + sub; j < parts; j += 32 * kSplit)
      m = fmaxf(m, part(j)[RT * DP + r]);
    m = warp_max(m);
    const float ms = m == -INFINITY ? 0.f : m;
    for (int j0 = sub; j0 < parts; j0 += 32 * kSplit) {
      const int j = j0 + lane * kSplit;
      float w = 0.f;
      if (j < parts) {
        const float* t = part(j) + RT * DP + r;
        w = exp2f(t[0] - ms);
        l += w * t[RT];
      }
      const int count = min(32, (parts - j0 + kSplit - 1) / kSplit);
      for (int i0 = 0; i0 < count; i0 += kBatch) {
        float x[kBatch][kV];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float* t = part(j0 + min(i0 + i, count - 1) * kSplit) + r * DP + lane * kV;
#pragma unroll
          for (int e = 0; e < kV; e += 2) {
            if constexpr (kV == 2) {
              const float2 y = *reinterpret_cast<const float2*>(t);
              x[i][0] = y.x, x[i][1] = y.y;
            } else if (e % 4 == 0) {
              const float4 y = *reinterpret_cast<const float4*>(t + e);
              x[i][e] = y.x, x[i][e + 1] = y.y, x[i][e + 2] = y.z, x[i][e + 3] = y.w;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
          if (i0 + i < count) {
#pragma unroll
            for (int e = 0; e < kV; ++e) acc[e] += wi * x[i][e];
          }
        }
      }
    }
    l = warp_add(l);
  }
  if constexpr (kSplit > 1) {
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < kV; ++e) s_o[warp][lane * kV + e] = acc[e];
    __syncthreads();
    if (sub != 0 || !on) return;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) top = fmaxf(top, s_m[warp + i]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) {
      if (sub + i >= parts) break;  // a warp without parts
      const float f = top == -INFINITY ? 1.f : exp2f(s_m[warp + i] - top);
      l += f * s_l[warp + i];
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] += f * s_o[warp + i][lane * kV + e];
    }
    m = top;
  }
  if (!on) return;
  const long long row = att_out_row(p, g.b, g.h, g.row0 + r);
  T* out = static_cast<T*>(p.out) + row * p.d;
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < kV; ++e)
    if (lane * kV + e < p.d) out[lane * kV + e] = from_f32<T>(acc[e] * inv);
  if (lane == 0 && p.lse) p.lse[row] = (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------------------
// The general kernel: fp32 arithmetic throughout, so fp32 caches keep their
// precision.  32 keys a tile, staged in shared memory as fp32; a lane holds a
// key and a warp four of the 16 rows while scores are formed, then a thread
// holds a column of the output.
// ---------------------------------------------------------------------------
constexpr int kGenThreads = 128, kGenU = 32, kGenR = 16, kGenOv = 1;

template <int DP>
struct GenSmem {
  float k[kGenU][DP + 4];  // +4: a lane per row reads 16 bytes without conflicts
  float v[kGenU][DP];
  float q[kGenR][DP];
  float p[kGenR][kGenU];
  float alpha[kGenR], m[kGenR], l[kGenR];
  const unsigned char* row_k[kGenU];
  const unsigned char* row_v[kGenU];
  int bad;
  alignas(16) unsigned char share[kShareBytes];
};

template <class T, int DP, bool VEC>
__global__ void __launch_bounds__(kGenThreads) attend_general_kernel(const AttendParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  GenSmem<DP>& sm = *reinterpret_cast<GenSmem<DP>*>(smem_raw);
  constexpr int kRG = DP == 64 ? 2 : 1;            // thread groups over the rows
  constexpr int kRows = kGenR / kRG;               // rows of a thread
  constexpr int kCols = DP == 256 ? 2 : 1;         // columns of a thread
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = tid % (kGenThreads / kRG), rg = tid / (kGenThreads / kRG) * kRows;
  if (tid == 0) att_clear_note(p);
  pdl_launch_dependents();
  AttCursor<kGenU, kGenR, kGenOv> cur;
  const AttShare s = att_share<kGenThreads>(p, cur, sm.share);
  const T* kc = static_cast<const T*>(p.k);
  const T* vc = static_cast<const T*>(p.v);
  while (cur.v < s.u1) {
    const int h = cur.seg / cur.mt, row0 = (cur.seg % cur.mt) * kGenR;
    const int rows = min(kGenR, cur.q * p.g - row0);
    const int tile0 = cur.tile, left = cur.tiles - cur.tile;
    const int cnt = s.u1 - cur.v < left ? (int)(s.u1 - cur.v) : left;
    const int len = cur.kv + cur.q;
    const int32_t* trow = p.table + (long long)cur.b * p.max_pages;
    const int32_t* par = p.parents ? p.parents + (long long)cur.b * p.n : nullptr;
    __syncthreads();
    if (tid == 0) sm.bad = 0;
    for (int e = tid; e < kGenR * DP; e += kGenThreads) {
      const int r = e / DP, d = e % DP;
      float x = 0.f;
      if (r < rows && d < p.d) {
        const int i = fast_div(row0 + r, p.div_g), gi = (row0 + r) - i * p.g;
        x = to_f32<T>(static_cast<const T*>(p.q)[cur.b * p.q_b + i * p.q_t +
                                                 (long long)(h * p.g + gi) * p.d + d]);
      }
      sm.q[r][d] = x;
    }
    float m[4], l[4], acc[kRows * kCols];
    bool tree_ok = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = -INFINITY, l[j] = 0.f;
#pragma unroll
    for (int j = 0; j < kRows * kCols; ++j) acc[j] = 0.f;
    for (int t = tile0; t < tile0 + cnt; ++t) {
      const int pos0 = t * kGenU;
      __syncthreads();
      if (tid < kGenU) {
        const int pos = pos0 + tid;
        const unsigned char *rk = nullptr, *rv = nullptr;
        if (pos < len) {
          const int pi = fast_div(pos, p.div_page);
          const int id = trow[pi];
          if (id >= 0 && id < p.num_pages) {
            const long long at =
                id * p.c_page + (long long)(pos - pi * p.page) * p.c_token + h * p.c_head;
            rk = reinterpret_cast<const unsigned char*>(kc + at);
            rv = reinterpret_cast<const unsigned char*>(vc + at);
          } else {
            sm.bad = 1;
          }
        }
        sm.row_k[tid] = rk;
        sm.row_v[tid] = rv;
      }
      __syncthreads();
      if constexpr (VEC) {
        constexpr int kPer = 16 / sizeof(T), kCh = DP / kPer;
        const int nch = p.d / kPer;
#pragma unroll 4
        for (int e = tid; e < kGenU * kCh * 2; e += kGenThreads) {
          const int w = e / (kGenU * kCh), f = e % (kGenU * kCh);
          const int r = f / kCh, c = f % kCh;
          const unsigned char* src = w ? sm.row_v[r] : sm.row_k[r];
          uint4 x = make_uint4(0, 0, 0, 0);
          if (src && c < nch) x = __ldcs(reinterpret_cast<const uint4*>(src) + c);
          float* dst = (w ? sm.v[r] : sm.k[r]) + c * kPer;
          if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<uint4*>(dst) = x;
          } else {
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              dst[2 * j] = __uint_as_float(y[j] << 16);
              dst[2 * j + 1] = __uint_as_float(y[j] & 0xffff0000u);
            }
          }
        }
      } else {
        for (int e = tid; e < kGenU * DP * 2; e += kGenThreads) {
          const int w = e / (kGenU * DP), f = e % (kGenU * DP);
          const int r = f / DP, d = f % DP;
          const T* src = reinterpret_cast<const T*>(w ? sm.row_v[r] : sm.row_k[r]);
          (w ? sm.v[r] : sm.k[r])[d] = (src && d < p.d) ? to_f32<T>(src[d]) : 0.f;
        }
      }
      __syncthreads();
      // scores: lane = key, rows warp, warp + 4, ...
      float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int d = 0; d < DP; d += 4) {
        const float4 kk = *reinterpret_cast<const float4*>(&sm.k[lane][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 qq = *reinterpret_cast<const float4*>(&sm.q[warp + 4 * j][d]);
          z[j] = fmaf(qq.x, kk.x, z[j]);
          z[j] = fmaf(qq.y, kk.y, z[j]);
          z[j] = fmaf(qq.z, kk.z, z[j]);
          z[j] = fmaf(qq.w, kk.w, z[j]);
        }
      }
      const int pos = pos0 + lane;
      const bool tail = pos0 + kGenU > cur.kv;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = warp + 4 * j;
        float x = z[j] * p.scale_log2;
        bool off = false;
        if (tail) {
          const int i = min(fast_div(row0 + r, p.div_g), cur.q - 1);
          bool on = pos < cur.kv || (pos < len && pos - cur.kv <= i);
          if (par && pos0 + kGenU > cur.kv) {
            const int lo = pos0 - cur.kv;  // node of the tile's first key
            const uint32_t bits = lo >= 0 ? att_tree_bits(par, i, lo, kGenU, tree_ok)
                                          : att_tree_bits(par, i, 0, kGenU + lo, tree_ok) << -lo;
            on = pos < cur.kv || (bits >> lane & 1u);
          }
          off = !on;
          if (off) x = -INFINITY;
        }
        const float mn = fmaxf(m[j], warp_max(x));
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m[j] - ms);
        float pr = exp2f(x - ms);
        if (tail) pr = att_mark_seen(pr, off);
        m[j] = mn;
        l[j] = l[j] * a + pr;
        sm.p[r][lane] = pr;
        if (lane == 0) sm.alpha[r] = a;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float a = sm.alpha[rg + r];
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[r * kCols + c] *= a;
      }
      if (!tail) {
#pragma unroll 2
        for (int key = 0; key < kGenU; key += 4) {
          float vv[4][kCols];
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int c = 0; c < kCols; ++c) vv[x][c] = sm.v[key + x][col + c * kGenThreads];
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const float4 pp = *reinterpret_cast<const float4*>(&sm.p[rg + r][key]);
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              float& o = acc[r * kCols + c];
              o = fmaf(pp.x, vv[0][c], o);
              o = fmaf(pp.y, vv[1][c], o);
              o = fmaf(pp.z, vv[2][c], o);
              o = fmaf(pp.w, vv[3][c], o);
            }
          }
        }
      } else {
        // keys that only some rows see leave the others (weight +0) as they
        // are, whatever their values hold
        for (int key = 0; key < kGenU; ++key)
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const float pr = sm.p[rg + r][key];
            const bool on = __float_as_uint(pr) != 0;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              float& o = acc[r * kCols + c];
              o = on ? fmaf(pr, sm.v[key][col + c * kGenThreads], o) : o;
            }
          }
      }
    }
    // this segment's result
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = warp_add(l[j]);
      if (!tree_ok) {
        x = __int_as_float(0x7fc00000);
        if (lane == 0 && warp + 4 * j < rows) kv_flag(p.status, SV_DEV_BAD_TREE);
      }
      if (lane == 0) sm.m[warp + 4 * j] = m[j], sm.l[warp + 4 * j] = x;
    }
    __syncthreads();
    const bool bad = sm.bad != 0;
    if (bad && tid == 0) kv_flag(p.status, SV_DEV_BAD_INDEX);
    const float nan = __int_as_float(0x7fc00000);
    if (tile0 == 0 && cnt == cur.tiles) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (rg + r >= rows) continue;
        const float ll = bad ? nan : sm.l[rg + r];
        const long long o = att_out_row(p, cur.b, h, row0 + rg + r);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int d = col + c * kGenThreads;
          if (d < p.d) static_cast<T*>(p.out)[o * p.d + d] = from_f32<T>(acc[r * kCols + c] / ll);
        }
        if (col == 0 && p.lse) p.lse[o] = (sm.m[rg + r] + log2f(ll)) * kLn2;
      }
    } else {
      float* t = att_part<DP, kGenR>(p, blockIdx.x, tile0 == 0);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (rg + r < rows) __stcg(t + (rg + r) * DP + col + c * kGenThreads, acc[r * kCols + c]);
      if (tid < rows) {
        __stcg(t + kGenR * DP + tid, sm.m[tid]);
        __stcg(t + kGenR * DP + kGenR + tid, bad ? nan : sm.l[tid]);
      }
      if (tid == 0 && tile0 == 0)
        att_note(p, s, cur.b, h, row0, rows, cur.v + cur.tiles);
    }
    cur.step(p, cnt);
  }
  att_fill_padding<T>(p, 0, kGenThreads / 32);
}

}  // namespace sv
