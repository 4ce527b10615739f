// sv_kv_pages.cuh -- bookkeeping of the paged key-value cache: the plan of a
// step (commit, page roll-back, page allocation, slot map), the append of new
// tokens' keys and values, and the commit of an accepted tree path.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

__device__ __forceinline__ void kv_flag(int32_t* status, int bit) {
  if (status) atomicOr(status, bit);
}

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
struct PlanParams {
  const int32_t *kv_len, *written, *accepted, *release, *new_len, *pages, *free_count;
  int B, max_new, page, num_pages, max_pages;
  FastDiv div_page, div_new;
  int32_t *table, *free_pages;
  int32_t *kv_len_out, *pages_out, *free_count_out, *q_len;
  int64_t* slot_map;
  int32_t* positions;
  int32_t* status;
  int write_slots;  // 1: this launch writes the slots, 0: kv_plan_slots_kernel does
};

constexpr int kPlanMaxThreads = 1024;
constexpr int kPlanMaxB = 8192;  // six ints of each request stay in shared memory
// Slots that one block writes about as fast as a second launch would start.
constexpr long long kPlanInlineSlots = 8192;

inline size_t plan_smem(int B) { return (size_t)B * 6 * sizeof(int32_t); }

// Threads of the block: one for each request or for every four slots, since
// the time of a small plan is that of its barriers and of three loads one after
// another (B = 32, events around one call: 8.2 us with 128 threads, 10.2 us with
// 1024; 5.8 us a call among others); all of them for steps with prompts, which
// move thousands of pages.
inline int plan_threads(int B, long long slots) {
  if (slots > kPlanInlineSlots) return kPlanMaxThreads;
  const long long want = B > slots / 4 ? B : slots / 4;
  return want <= 128 ? 128 : want <= 256 ? 256 : want <= 512 ? 512 : kPlanMaxThreads;
}

// Slot of position `pos` through a request's table row; -1 for a page id
// outside the pool.
__device__ __forceinline__ long long plan_slot(const PlanParams& p, const int32_t* row, int pos) {
  const int pi = fast_div(pos, p.div_page);
  const int id = row[pi];
  if (id < 0 || id >= p.num_pages) {
    kv_flag(p.status, SV_DEV_BAD_INDEX);
    return -1;
  }
  return (long long)id * p.page + (pos - pi * p.page);
}

// One block.  The sums over requests (pages given back, pages wanted) are
// sequential in the request order, so they are a scan in one block; what
// follows is at most a few pages per request.  All inputs are read before the
// first output is written, so an output may be the array of its input.
__global__ void __launch_bounds__(kPlanMaxThreads) kv_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_base = sm;             // committed length
  int32_t* s_new = s_base + p.B;    // new tokens; -1: failed, nothing of it changes
  int32_t* s_held = s_new + p.B;    // pages held before
  int32_t* s_need = s_held + p.B;   // pages held afterwards
  int32_t* s_give = s_need + p.B;   // pages that the requests before give back
  int32_t* s_take = s_give + p.B;   // and take
  __shared__ long long warp_give[32], warp_take[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  int count = *p.free_count;
  // ---- lengths, and pages wanted or given back --------------------------
  long long cap = (long long)p.max_pages * p.page;
  if (cap > 0x7fffffffLL - p.page) cap = 0x7fffffffLL - p.page;  // positions are int32
  long long give_all = 0;
  for (int b = tid; b < p.B; b += threads) {
    const int len = p.kv_len[b], held = p.pages[b];
    const int rel = p.release ? p.release[b] : 0;
    const int w = p.written ? p.written[b] : 0;
    const int acc = p.accepted ? p.accepted[b] : w - 1;
    const int nl = rel ? 0 : p.new_len[b];
    long long base = len;
    if (w > 0 && acc >= 0) base += acc + 1;
    bool ok = len >= 0 && w >= 0 && (w == 0 || acc < w) && held >= 0 && held <= p.max_pages &&
              nl >= 0 && nl <= p.max_new;
    if (rel) base = 0;
    ok = ok && base + nl <= cap && fast_div((int)base + p.page - 1, p.div_page) <= held;
    int need = held;
    if (ok) {
      need = fast_div((int)base + nl + p.page - 1, p.div_page);
    } else {
      kv_flag(p.status, SV_DEV_BAD_LEN);
      base = len;
    }
    s_base[b] = (int)base;
    s_new[b] = ok ? nl : -1;
    s_held[b] = held;
    s_need[b] = need;
    if (need < held) give_all += held - need;
  }
  if (count < 0 || count > p.num_pages) {
    if (tid == 0) kv_flag(p.status, SV_DEV_BAD_LEN);
    count = count < 0 ? 0 : p.num_pages;
  }
  // all pages given back
  for (int o = 16; o; o >>= 1) give_all += __shfl_xor_sync(0xffffffffu, give_all, o);
  if (lane == 0) warp_give[warp] = give_all;
  __syncthreads();
  give_all = lane < warps ? warp_give[lane] : 0;
  for (int o = 16; o; o >>= 1) give_all += __shfl_xor_sync(0xffffffffu, give_all, o);
  const long long top = (long long)count + give_all;
  const long long top_ok = top < p.num_pages ? top : p.num_pages;
  if (top > p.num_pages && tid == 0) kv_flag(p.status, SV_DEV_BAD_LEN);
  // ---- exclusive scans over the requests ----------------------------------
  // Requests are served in order until one finds too few pages; `taken` is
  // what those before it took.
  long long run_give = 0, run_take = 0, taken = 0;
  for (int b0 = 0; b0 < p.B; b0 += threads) {
    const int b = b0 + tid;
    int give = 0, take = 0;
    if (b < p.B) {
      const int dlt = s_need[b] - s_held[b];
      give = dlt < 0 ? -dlt : 0;
      take = dlt > 0 ? dlt : 0;
    }
    long long ig = give, it = take;
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, ig, o);
      const long long c = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) ig += a, it += c;
    }
    __syncthreads();  // the sums of the last round are read
    if (lane == 31) warp_give[warp] = ig, warp_take[warp] = it;
    __syncthreads();
    long long wg = lane < warps ? warp_give[lane] : 0, wt = lane < warps ? warp_take[lane] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, wg, o);
      const long long c = __shfl_up_sync(0xffffffffu, wt, o);
      if (lane >= o) wg += a, wt += c;
    }
    const long long before_g = __shfl_sync(0xffffffffu, wg, warp ? warp - 1 : 0);
    const long long before_t = __shfl_sync(0xffffffffu, wt, warp ? warp - 1 : 0);
    ig += run_give + (warp ? before_g : 0);
    it += run_take + (warp ? before_t : 0);
    run_give += __shfl_sync(0xffffffffu, wg, 31);
    run_take += __shfl_sync(0xffffffffu, wt, 31);
    if (b < p.B) {
      s_give[b] = (int)(ig - give);
      s_take[b] = (int)(it - take);
      if (take) {
        if (it <= top_ok) {
          taken = it;
        } else {  // the pool ends before this request's pages
          kv_flag(p.status, SV_DEV_NO_PAGES);
          s_need[b] = s_held[b];
          s_new[b] = 0;
        }
      }
    }
  }
  for (int o = 16; o; o >>= 1) {
    const long long a = __shfl_xor_sync(0xffffffffu, taken, o);
    taken = a > taken ? a : taken;
  }
  __syncthreads();
  if (lane == 0) warp_take[warp] = taken;
  // The request that page i of those given (taken) belongs to: the last one
  // with no more than i before it.
  auto owner = [&](const int32_t* before, int i) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  };
  __syncthreads();
  // ---- pages given back go onto the stack ----------------------------------
  if (give_all) {
    for (int i0 = tid; i0 < (int)give_all; i0 += 4 * threads) {
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * threads;
        if (i >= (int)give_all) break;
        const int b = owner(s_give, i);
        id[j] = p.table[(long long)b * p.max_pages + s_need[b] + (i - s_give[b])];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * threads;
        if (i >= (int)give_all) break;
        if (id[j] < 0 || id[j] >= p.num_pages) kv_flag(p.status, SV_DEV_BAD_INDEX);
        if ((long long)count + i < p.num_pages) p.free_pages[count + i] = id[j];
      }
    }
    __syncthreads();
  }
  // ---- and the new ones come off its top --------------------------------------
  taken = lane < warps ? warp_take[lane] : 0;
  for (int o = 16; o; o >>= 1) {
    const long long a = __shfl_xor_sync(0xffffffffu, taken, o);
    taken = a > taken ? a : taken;
  }
  for (int i0 = tid; i0 < (int)taken; i0 += 4 * threads) {
    int id[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * threads < (int)taken) id[j] = p.free_pages[top_ok - 1 - (i0 + j * threads)];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * threads;
      if (i >= (int)taken) break;
      const int b = owner(s_take, i);
      if (id[j] < 0 || id[j] >= p.num_pages) kv_flag(p.status, SV_DEV_BAD_INDEX);
      p.table[(long long)b * p.max_pages + s_held[b] + (i - s_take[b])] = id[j];
    }
  }
  for (int b = tid; b < p.B; b += threads) {
    p.kv_len_out[b] = s_base[b];
    p.pages_out[b] = s_need[b];
    p.q_len[b] = s_new[b] < 0 ? 0 : s_new[b];
  }
  if (tid == 0) *p.free_count_out = (int)(top_ok - taken);
  if (!p.write_slots) return;
  __syncthreads();
  const int total = p.B * p.max_new;
  for (int e = tid; e < total; e += threads) {
    const int b = fast_div(e, p.div_new), i = e - b * p.max_new;
    const bool on = i < s_new[b];
    const int pos = s_base[b] + i;
    p.slot_map[e] = on ? plan_slot(p, p.table + (long long)b * p.max_pages, pos) : -1;
    if (p.positions) p.positions[e] = on ? pos : -1;
  }
}

// Slots of a step with many new tokens (prompts): four of a request for each
// thread, two at a time, so that the stores are 16 bytes wide.
constexpr int kSlotThreads = 256, kSlotPer = 4;
__global__ void __launch_bounds__(kSlotThreads) kv_plan_slots_kernel(const PlanParams p) {
  pdl_wait();  // the plan
  const int b = blockIdx.y;
  const int q = p.q_len[b], base = p.kv_len_out[b];
  const int32_t* row = p.table + (long long)b * p.max_pages;
  const long long line = (long long)b * p.max_new;
  const bool wide = (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0 &&
                    (reinterpret_cast<uintptr_t>(p.positions) & 7) == 0;
#pragma unroll
  for (int t = 0; t < kSlotPer / 2; ++t) {
    const int i = 2 * (blockIdx.x * (kSlotThreads * kSlotPer / 2) + t * kSlotThreads + threadIdx.x);
    if (i >= p.max_new) break;
    long long s[2] = {-1, -1};
    int x[2] = {-1, -1};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (i + j < q) {
        x[j] = base + i + j;
        s[j] = plan_slot(p, row, x[j]);
      }
    if (wide && i + 1 < p.max_new && ((line + i) & 1) == 0) {
      *reinterpret_cast<longlong2*>(p.slot_map + line + i) = make_longlong2(s[0], s[1]);
      if (p.positions) *reinterpret_cast<int2*>(p.positions + line + i) = make_int2(x[0], x[1]);
    } else {
      for (int j = 0; j < 2 && i + j < p.max_new; ++j) {
        p.slot_map[line + i + j] = s[j];
        if (p.positions) p.positions[line + i + j] = x[j];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
struct AppendParams {
  const unsigned char *k, *v;
  unsigned char *kc, *vc;
  long long in_b, in_t;                // strides of k and v, bytes
  long long c_page, c_token, c_head;   // strides of the cache, bytes
  const int64_t* slot_map;
  int B, n, heads, page, num_pages;
  int head_chunks;  // head_dim bytes / sizeof(VEC); all of a token's where its heads are dense
  int per_warp;     // tokens of a warp
  FastDiv div_n, div_page, div_chunks;
  int32_t* status;
};

// A warp copies the key and value rows of `per_warp` tokens, whose slots it
// loads at once: a pure copy, one read and one write of each byte, bound by
// HBM (46,000 tokens of 8 heads of 128 in bf16: 378 MB in 65 us, 5.8 TB/s;
// with each load stored before the next, 71 us).  VEC is the widest unit that
// every address is a multiple of.
template <class VEC>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int tokens = p.B * p.n;
  const long long slots = (long long)p.num_pages * p.page;
  const int chunks = p.heads * p.head_chunks;
  const long long first =
      ((long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * p.per_warp;
  const long long last = first + p.per_warp < tokens ? first + p.per_warp : tokens;
  for (long long t0 = first; t0 < last; t0 += 32) {
    const int here = last - t0 < 32 ? (int)(last - t0) : 32;
    long long src = 0, dst = -1;
    if (lane < here) {
      const long long slot = p.slot_map[t0 + lane];
      if (slot >= slots) {
        kv_flag(p.status, SV_DEV_BAD_INDEX);
      } else if (slot >= 0) {
        long long pg;
        if (slot <= 0x7fffffffLL)
          pg = fast_div((int)slot, p.div_page);
        else
          pg = slot / p.page;
        const int b = fast_div((int)(t0 + lane), p.div_n), i = (int)(t0 + lane) - b * p.n;
        src = b * p.in_b + i * p.in_t;
        dst = pg * p.c_page + (slot - pg * p.page) * p.c_token;
      }
    }
    for (int j = 0; j < here; ++j) {
      const long long to = __shfl_sync(0xffffffffu, dst, j);
      if (to < 0) continue;
      const long long from = __shfl_sync(0xffffffffu, src, j);
      const VEC* ks = reinterpret_cast<const VEC*>(p.k + from);
      const VEC* vs = reinterpret_cast<const VEC*>(p.v + from);
      constexpr int kBatch = 4;  // loads before the first store, of keys and of values
      for (int c0 = lane; c0 < chunks; c0 += 32 * kBatch) {
        VEC a[kBatch], z[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
          if (c0 + 32 * x < chunks) a[x] = ks[c0 + 32 * x], z[x] = vs[c0 + 32 * x];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int c = c0 + 32 * x;
          if (c >= chunks) break;
          const int h = fast_div(c, p.div_chunks), r = c - h * p.head_chunks;
          const long long at = to + h * p.c_head + (long long)r * sizeof(VEC);
          *reinterpret_cast<VEC*>(p.kc + at) = a[x];
          *reinterpret_cast<VEC*>(p.vc + at) = z[x];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Commit of an accepted tree path
// ---------------------------------------------------------------------------
struct CommitParams {
  unsigned char *kc, *vc;
  long long c_layer, c_page, c_token, c_head;  // bytes
  const int32_t *table, *kv_len, *q_len, *nodes, *accepted;
  int B, width, layers, heads, page, num_pages, max_pages;
  int head_chunks;
  FastDiv div_page, div_chunks, div_head;  // chunks: of a token; head: of a head
  int32_t* status;
};

constexpr int kCommitThreads = 256;
constexpr int kCommitMaxWidth = 1024;

// Path entry i moves from the slot of node_i to the slot of position i.  The
// nodes ascend, so node_i >= i and no destination is the source of a later
// entry; a destination may be the source of an earlier one.  A thread that
// moves all entries of its own 16 bytes in path order therefore needs no
// barrier, and may read several entries ahead before it writes them.  Bound by
// the latency of path, table and rows, one after another: 256 requests, 28
// layers, 59 MB in 20 us (with two of these 16 bytes to a thread, and half
// the blocks, 32 us).
template <class VEC>
__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const CommitParams p) {
  __shared__ long long s_src[kCommitMaxWidth], s_dst[kCommitMaxWidth];
  const int b = blockIdx.y;
  const int32_t* nodes = p.nodes + (long long)b * p.width;
  const int32_t* row = p.table + (long long)b * p.max_pages;
  // the path's loads do not wait for one another
  const int a = p.accepted[b], base = p.kv_len[b];
  const int wrote = p.q_len ? p.q_len[b] : 0x7fffffff;
  int nd = threadIdx.x < p.width ? nodes[threadIdx.x] : 0;
  int before = threadIdx.x > 0 && threadIdx.x < p.width ? nodes[threadIdx.x - 1] : -1;
  // The root is in its place already; -1: failed verification; a request that
  // the step left out may have given its pages to another.
  if (a < 1 || wrote == 0) return;
  int bad = 0;
  if (a >= p.width || base < 0 || wrote < 0) {
    bad = SV_DEV_BAD_LEN;
  } else {
    for (int i = threadIdx.x; i <= a; i += kCommitThreads) {
      if (i >= kCommitThreads) nd = nodes[i], before = nodes[i - 1];
      const long long at[2] = {(long long)base + nd, (long long)base + i};
      if (nd < i || (i == 0 && nd != 0) || before >= nd || nd >= wrote) {
        bad |= SV_DEV_BAD_TREE;
        continue;
      }
      if (at[0] >= (long long)p.max_pages * p.page || at[0] > 0x7fffffffLL) {
        bad |= SV_DEV_BAD_LEN;
        continue;
      }
      for (int j = 0; j < 2; ++j) {
        const int pi = fast_div((int)at[j], p.div_page), off = (int)at[j] - pi * p.page;
        const int id = row[pi];
        if (id < 0 || id >= p.num_pages) {
          bad |= SV_DEV_BAD_INDEX;
          continue;
        }
        (j ? s_dst : s_src)[i] = id * p.c_page + off * p.c_token;
      }
    }
  }
  if (bad) kv_flag(p.status, bad);
  if (__syncthreads_or(bad)) return;  // a bad path moves nothing
  const int chunks = p.heads * p.head_chunks;
  const int items = 2 * p.layers * chunks;
  constexpr int kAhead = 8;
  for (int e = blockIdx.x * kCommitThreads + threadIdx.x; e < items;
       e += gridDim.x * kCommitThreads) {
    const int lk = fast_div(e, p.div_chunks), c = e - lk * chunks;
    const int h = fast_div(c, p.div_head), r = c - h * p.head_chunks;
    unsigned char* cache = (lk & 1 ? p.vc : p.kc) + (lk >> 1) * p.c_layer + h * p.c_head +
                           (long long)r * sizeof(VEC);
    for (int i0 = 1; i0 <= a; i0 += kAhead) {
      VEC t[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j <= a && s_src[i0 + j] != s_dst[i0 + j])
          t[j] = *reinterpret_cast<const VEC*>(cache + s_src[i0 + j]);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j <= a && s_src[i0 + j] != s_dst[i0 + j])
          *reinterpret_cast<VEC*>(cache + s_dst[i0 + j]) = t[j];
    }
  }
}

}  // namespace sv
