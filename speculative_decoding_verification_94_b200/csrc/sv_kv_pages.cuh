// sv_kv_pages.cuh -- bookkeeping of the paged key-value cache: the plan of a
// step (commit, page roll-back, page allocation, slot map), the append of new
// tokens' keys and values, and the commit of an accepted tree path.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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
  int32_t *table, *free_pages;
  int32_t *kv_len_out, *pages_out, *free_count_out, *q_len;
  int64_t* slot_map;
  int32_t* positions;
  int32_t* status;
  int write_slots;  // 1: this launch writes the slots, 0: plan_slots_kernel does
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxB = 8192;  // five ints of each request stay in shared memory
// Slots that one block writes about as fast as a second launch would start.
constexpr long long kPlanInlineSlots = 8192;

inline size_t plan_smem(int B) { return (size_t)B * 5 * sizeof(int32_t); }

// Slot of position `pos` through a request's table row; -1 for a page id
// outside the pool.
__device__ __forceinline__ long long plan_slot(const int32_t* row, int pos, int page,
                                               int num_pages, int32_t* status) {
  const int pi = pos / page;
  const int id = row[pi];
  if (id < 0 || id >= num_pages) {
    kv_flag(status, SV_DEV_BAD_INDEX);
    return -1;
  }
  return (long long)id * page + (pos - pi * page);
}

// One block.  The sums over requests (pages given back, pages wanted) are
// sequential in the request order, so they are a scan in one block; what
// follows is at most a few pages per request.  All inputs are read before the
// first output is written, so an output may be the array of its input.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_base = sm;             // committed length
  int32_t* s_new = s_base + p.B;    // new tokens, 0 where nothing was granted
  int32_t* s_held = s_new + p.B;    // pages held before (after phase 2: unchanged)
  int32_t* s_need = s_held + p.B;   // pages held afterwards
  int32_t* s_off = s_need + p.B;    // first page on the stack given / taken (from the top)
  __shared__ long long warp_give[32], warp_take[32];
  __shared__ long long run_give, run_take, s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int count = *p.free_count;
  if (count < 0 || count > p.num_pages) {
    if (tid == 0) kv_flag(p.status, SV_DEV_BAD_LEN);
    count = count < 0 ? 0 : p.num_pages;
  }
  // ---- lengths, and pages wanted or given back --------------------------
  long long cap = (long long)p.max_pages * p.page;
  if (cap > 0x7fffffffLL) cap = 0x7fffffffLL;  // positions are int32
  long long give_all = 0;
  for (int b = tid; b < p.B; b += kPlanThreads) {
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
    ok = ok && base + nl <= cap && (base + p.page - 1) / p.page <= held;
    int need = held;
    if (ok) {
      need = (int)((base + nl + p.page - 1) / p.page);
    } else {
      kv_flag(p.status, SV_DEV_BAD_LEN);
      base = len;
    }
    s_base[b] = (int)base;
    s_new[b] = ok ? nl : -1;  // -1: failed, nothing of it changes
    s_held[b] = held;
    s_need[b] = need;
    if (need < held) give_all += held - need;
  }
  if (tid == 0) run_give = run_take = s_taken = 0;
  // total given back: warp sums, then all warps
  for (int o = 16; o; o >>= 1) give_all += __shfl_xor_sync(0xffffffffu, give_all, o);
  if (lane == 0) warp_give[warp] = give_all;
  __syncthreads();
  give_all = 0;
  for (int w = 0; w < 32; ++w) give_all += warp_give[w];
  __syncthreads();
  const long long top = (long long)count + give_all;
  const long long top_ok = top < p.num_pages ? top : p.num_pages;
  if (top > p.num_pages && tid == 0) kv_flag(p.status, SV_DEV_BAD_LEN);
  // ---- exclusive scans over the requests ----------------------------------
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
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
    if (lane == 31) warp_give[warp] = ig, warp_take[warp] = it;
    __syncthreads();
    for (int w = 0; w < warp; ++w) ig += warp_give[w], it += warp_take[w];
    ig += run_give;
    it += run_take;
    __syncthreads();
    if (tid == kPlanThreads - 1) run_give = ig, run_take = it;
    if (b < p.B) {
      if (give) {
        s_off[b] = (int)(ig - give);
      } else if (take) {
        if (it <= top_ok) {
          s_off[b] = (int)(it - take);
          atomicMax(&s_taken, it);
        } else {  // the pool ends before this request's pages
          kv_flag(p.status, SV_DEV_NO_PAGES);
          s_need[b] = s_held[b];
          s_new[b] = 0;
        }
      }
    }
    __syncthreads();
  }
  // ---- pages given back go onto the stack ----------------------------------
  for (int b = warp; b < p.B; b += 32) {
    const int held = s_held[b], need = s_need[b];
    const int32_t* row = p.table + (long long)b * p.max_pages;
    for (int j = need + lane; j < held; j += 32) {
      const long long at = (long long)count + s_off[b] + (j - need);
      if (at < p.num_pages) p.free_pages[at] = row[j];
    }
  }
  __syncthreads();
  // ---- and the new ones come off its top --------------------------------------
  for (int b = warp; b < p.B; b += 32) {
    const int held = s_held[b], need = s_need[b];
    int32_t* row = p.table + (long long)b * p.max_pages;
    for (int j = held + lane; j < need; j += 32) {
      const int id = p.free_pages[top_ok - 1 - s_off[b] - (j - held)];
      if (id < 0 || id >= p.num_pages) kv_flag(p.status, SV_DEV_BAD_INDEX);
      row[j] = id;
    }
  }
  for (int b = tid; b < p.B; b += kPlanThreads) {
    p.kv_len_out[b] = s_base[b];
    p.pages_out[b] = s_need[b];
    p.q_len[b] = s_new[b] < 0 ? 0 : s_new[b];
  }
  if (tid == 0) *p.free_count_out = (int)(top_ok - s_taken);
  if (!p.write_slots) return;
  __syncthreads();
  const int total = p.B * p.max_new;
  for (int e = tid; e < total; e += kPlanThreads) {
    const int b = e / p.max_new, i = e - b * p.max_new;
    const bool on = i < s_new[b];
    const int pos = s_base[b] + i;
    p.slot_map[e] = on ? plan_slot(p.table + (long long)b * p.max_pages, pos, p.page, p.num_pages,
                                   p.status)
                       : -1;
    if (p.positions) p.positions[e] = on ? pos : -1;
  }
}

// Slots of a step with many new tokens (prompts): one block per 1024 tokens of
// a request, two at a time per thread, so that the stores are 16 bytes wide.
constexpr int kSlotThreads = 256, kSlotPer = 4;
__global__ void __launch_bounds__(kSlotThreads) kv_plan_slots_kernel(const PlanParams p) {
  const int b = blockIdx.y;
  const int q = p.q_len[b], base = p.kv_len_out[b];
  const int32_t* row = p.table + (long long)b * p.max_pages;
  const long long line = (long long)b * p.max_new;
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
        s[j] = plan_slot(row, x[j], p.page, p.num_pages, p.status);
      }
    if (i + 1 < p.max_new && ((line + i) & 1) == 0 &&
        (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0 &&
        (reinterpret_cast<uintptr_t>(p.positions) & 7) == 0) {
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
  int head_chunks;  // head_dim bytes / sizeof(VEC)
  int32_t* status;
};

// A warp copies the key row and the value row of one token: a pure copy, one
// read and one write of each byte, bound by HBM.  VEC is the widest unit that
// every address is a multiple of.
template <class VEC>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long tokens = (long long)p.B * p.n;
  const long long slots = (long long)p.num_pages * p.page;
  const int chunks = p.heads * p.head_chunks;
  for (long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < tokens;
       t += warps) {
    const long long slot = p.slot_map[t];
    if (slot < 0) continue;
    if (slot >= slots) {
      if (lane == 0) kv_flag(p.status, SV_DEV_BAD_INDEX);
      continue;
    }
    const long long pg = slot / p.page, off = slot - pg * p.page;
    const long long b = t / p.n, i = t - b * p.n;
    const long long src = b * p.in_b + i * p.in_t;
    const long long dst = pg * p.c_page + off * p.c_token;
    const VEC* ks = reinterpret_cast<const VEC*>(p.k + src);
    const VEC* vs = reinterpret_cast<const VEC*>(p.v + src);
#pragma unroll 4
    for (int c = lane; c < chunks; c += 32) {
      const int h = c / p.head_chunks, r = c - h * p.head_chunks;
      const VEC a = ks[c], z = vs[c];
      const long long at = dst + h * p.c_head + (long long)r * sizeof(VEC);
      *reinterpret_cast<VEC*>(p.kc + at) = a;
      *reinterpret_cast<VEC*>(p.vc + at) = z;
    }
  }
}

// ---------------------------------------------------------------------------
// Commit of an accepted tree path
// ---------------------------------------------------------------------------
struct CommitParams {
  unsigned char *kc, *vc;
  long long c_layer, c_page, c_token, c_head;  // bytes
  const int32_t *table, *kv_len, *nodes, *accepted;
  int B, width, layers, heads, page, num_pages, max_pages;
  int head_chunks;
  int32_t* status;
};

constexpr int kCommitThreads = 256;
constexpr int kCommitMaxWidth = 1024;

// Path entry i moves from the slot of node_i to the slot of position i.  The
// nodes ascend, so node_i >= i and no destination is the source of a later
// entry; a destination may be the source of an earlier one.  A thread that
// moves all entries of its own 16 bytes in path order therefore needs no
// barrier, and may read several entries ahead before it writes them.
template <class VEC>
__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const CommitParams p) {
  __shared__ long long s_src[kCommitMaxWidth], s_dst[kCommitMaxWidth];
  const int b = blockIdx.y;
  const int a = p.accepted[b];
  if (a < 1) return;  // the root is in its place already; -1: failed verification
  const int base = p.kv_len[b];
  const int32_t* nodes = p.nodes + (long long)b * p.width;
  const int32_t* row = p.table + (long long)b * p.max_pages;
  int bad = 0;
  if (a >= p.width || base < 0) {
    bad = SV_DEV_BAD_LEN;
  } else {
    for (int i = threadIdx.x; i <= a; i += kCommitThreads) {
      const int nd = nodes[i];
      const long long at[2] = {(long long)base + nd, (long long)base + i};
      if (nd < i || (i == 0 && nd != 0) || (i > 0 && nodes[i - 1] >= nd)) {
        bad |= SV_DEV_BAD_TREE;
        continue;
      }
      if (at[0] >= (long long)p.max_pages * p.page) {
        bad |= SV_DEV_BAD_LEN;
        continue;
      }
      for (int j = 0; j < 2; ++j) {
        const int pi = (int)(at[j] / p.page), off = (int)(at[j] - (long long)pi * p.page);
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
  const long long items = 2LL * p.layers * chunks;
  const long long e = (long long)blockIdx.x * kCommitThreads + threadIdx.x;
  if (e >= items) return;
  const int c = (int)(e % chunks);
  const long long lk = e / chunks;
  const int h = c / p.head_chunks, r = c - h * p.head_chunks;
  unsigned char* cache = (lk & 1 ? p.vc : p.kc) + (lk >> 1) * p.c_layer + h * p.c_head +
                         (long long)r * sizeof(VEC);
  constexpr int kAhead = 8;
  for (int i0 = 1; i0 <= a; i0 += kAhead) {
    VEC t[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j <= a) t[j] = *reinterpret_cast<const VEC*>(cache + s_src[i0 + j]);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j <= a && s_src[i0 + j] != s_dst[i0 + j])
        *reinterpret_cast<VEC*>(cache + s_dst[i0 + j]) = t[j];
  }
}

}  // namespace sv
