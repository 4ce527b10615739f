// sv_kv.cu -- the paged key-value cache calls of the C ABI: argument checks,
// choice of kernel and launches.  No entry point synchronises or allocates.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "sv_attend.cuh"
#include "sv_attend_f32.cuh"
#include "sv_attend_mma.cuh"
#include "sv_attend_tc.cuh"
#include "sv_attend_tf32.cuh"
#include "sv_kv_pages.cuh"

namespace sv {
namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool aligned_or_null(const void* p, size_t a) { return aligned(p, a); }
inline int esize(sv_dtype d) { return d == SV_BF16 ? 2 : 4; }
inline sv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

// The widest power of two up to 16 that divides every value.
int common_width(std::initializer_list<long long> v) {
  int w = 16;
  for (long long x : v)
    while (x % w) w /= 2;
  return w;
}
long long addr(const void* p) { return (long long)(reinterpret_cast<uintptr_t>(p) % 16); }

// Type, sizes, and strides under which no two tokens' rows overlap.
sv_status check_cache(const sv_kv_cache* c, int layers = 1, long long layer_stride = 0) {
  if (!c || (c->dtype != SV_F32 && c->dtype != SV_BF16)) return SV_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1)
    return SV_ERR_INVALID_ARG;
  if (c->head_dim > 256) return SV_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !aligned(c->k, esize(c->dtype)) || !aligned(c->v, esize(c->dtype)))
    return SV_ERR_INVALID_ARG;
  struct Dim {
    long long stride, extent;
  } d[4] = {{c->page_stride, c->num_pages}, {c->token_stride, c->page_size},
            {c->head_stride, c->heads}, {layer_stride, layers}};
  for (auto& x : d)
    if (x.stride < 0 || x.stride > (1LL << 44)) return SV_ERR_INVALID_ARG;
  std::sort(d, d + 4, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  double span = c->head_dim;  // elements from the first to the last of the dimensions so far
  for (auto& x : d) {
    if (x.extent == 1) continue;
    if ((double)x.stride < span) return SV_ERR_INVALID_ARG;
    span += (double)x.stride * (double)(x.extent - 1);
  }
  if (span > 1e18) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

// Up to 48 KB of shared memory, the kernel's own (static) included, need no
// permission; no kernel here has more than kStaticSmem of its own.
constexpr int kStaticSmem = 16 * 1024;
static_assert(2 * sizeof(long long) * kCommitMaxWidth <= kStaticSmem, "");
template <class K, class Prm>
cudaError_t launch(K kernel, const Prm& prm, dim3 grid, int threads, int smem, cudaStream_t s) {
  cudaError_t e = smem > 48 * 1024 - kStaticSmem
                      ? ensure_kernel_attrs(reinterpret_cast<const void*>(kernel), smem, false)
                      : cudaSuccess;
  if (e != cudaSuccess) return e;
  if ((e = launch_mark_before(s)) != cudaSuccess) return e;
  kernel<<<grid, threads, smem, s>>>(prm);
  return launch_mark_after(s, cudaGetLastError());
}

// A launch that follows another of the same call: its blocks may be on the
// device before the first ends; the kernel waits for it.
template <class K, class Prm>
cudaError_t launch_after(K kernel, const Prm& prm, dim3 grid, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = launch_mark_before(s);
  if (e != cudaSuccess) return e;
  return launch_mark_after(s, cudaLaunchKernelEx(&cfg, kernel, prm));
}

// ---------------------------------------------------------------------------
// Attention: grid and scratch
// ---------------------------------------------------------------------------
int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

constexpr size_t kSharedBytes = (sizeof(AttShared) * kAttMaxBlocks + 255) / 256 * 256;

// Rows of a row tile, which set the size of a partial result.  16 also covers
// the general kernel, which any bf16 call may need for its strides.
int tile_rows(int rows, int head_dim, sv_dtype dt) {
  if (dt != SV_BF16 || head_dim > 128 || rows <= 16) return 16;
  return rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

size_t attend_scratch(int rows, int head_dim, sv_dtype dt) {
  const int tile = tile_rows(rows, head_dim, dt);
  return kSharedBytes +
         (size_t)kAttMaxBlocks * 2 * att_partial_floats(tile, padded_dim(head_dim)) * 4;
}

// The second launch.
template <class T, int DP, int RT>
cudaError_t launch_join(const AttendParams& p, int grid, cudaStream_t s) {
  constexpr int kRowsHere = RT >= 128 ? 4 : RT == 64 ? 2 : 1;
  const int rows = std::min(RT, p.n * p.g);
  return launch_after(attend_join_kernel<T, DP, RT>, p,
                      dim3((unsigned)grid, (unsigned)((rows + kRowsHere - 1) / kRowsHere)),
                      kJoinThreads, s);
}

template <class T, int DP, int RT, class K>
cudaError_t launch_attend(K kernel, AttendParams& p, int threads, int smem, cudaStream_t s) {
  const void* kp = reinterpret_cast<const void*>(kernel);
  cudaError_t e = ensure_kernel_attrs(kp, smem, false);
  if (e != cudaSuccess) return e;
  int per_sm = 0, sms = 0;
  if ((e = blocks_per_sm(kp, threads, smem, &per_sm)) != cudaSuccess) return e;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int grid = std::min(per_sm * sms, kAttMaxBlocks);
  if ((e = launch(kernel, p, dim3((unsigned)grid), threads, smem, s)) != cudaSuccess) return e;
  return launch_join<T, DP, RT>(p, grid, s);
}

template <class T, bool VEC>
cudaError_t launch_general(AttendParams& p, cudaStream_t s) {
  switch (padded_dim(p.d)) {
    case 64:
      return launch_attend<T, 64, kGenR>(attend_general_kernel<T, 64, VEC>, p, kGenThreads,
                                           sizeof(GenSmem<64>), s);
    case 128:
      return launch_attend<T, 128, kGenR>(attend_general_kernel<T, 128, VEC>, p, kGenThreads,
                                           sizeof(GenSmem<128>), s);
    default:
      return launch_attend<T, 256, kGenR>(attend_general_kernel<T, 256, VEC>, p, kGenThreads,
                                           sizeof(GenSmem<256>), s);
  }
}

// ---------------------------------------------------------------------------
// The tensor-memory kernel: tensor maps over the cache
// ---------------------------------------------------------------------------
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Copies take up to 16 boxes of whole pages, or of 128 rows of a page.
int tc_box(int page) {
  if (page >= kTcU) return page % kTcU == 0 ? kTcU : 0;
  return page >= 8 && kTcU % page == 0 ? page : 0;
}

bool tc_map(const AttendParams& p, const void* base, int box, CUtensorMap* map) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page, (cuuint64_t)p.hkv,
                              (cuuint64_t)p.num_pages};
  // a dimension of one has no stride of its own
  const cuuint64_t strides[3] = {
      (cuuint64_t)(p.page > 1 ? p.c_token : p.d) * 2, (cuuint64_t)(p.hkv > 1 ? p.c_head : p.d) * 2,
      (cuuint64_t)(p.num_pages > 1 ? p.c_page : p.d) * 2};
  for (cuuint64_t x : strides)
    if (x >= (1ull << 40)) return false;
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
             boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RT>
cudaError_t launch_tc(const TcParams& tp, const CUtensorMap& km, const CUtensorMap& vm,
                      cudaStream_t s) {
  auto kernel = attend_tc_kernel<D, RT>;
  cudaError_t e =
      ensure_kernel_attrs(reinterpret_cast<const void*>(kernel), TcCfg<D>::kSmem, false);
  if (e != cudaSuccess) return e;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  if ((e = launch_mark_before(s)) != cudaSuccess) return e;
  const int grid = std::min(sms, kAttMaxBlocks);
  kernel<<<(unsigned)grid, kTcThreads, TcCfg<D>::kSmem, s>>>(tp, km, vm);
  if ((e = launch_mark_after(s, cudaGetLastError())) != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, D, RT>(tp.a, grid, s);
}

template <int D>
cudaError_t launch_tc(const TcParams& tp, const CUtensorMap& km, const CUtensorMap& vm,
                      cudaStream_t s) {
  const int rows = tp.a.n * tp.a.g;
  if (rows <= 32) return launch_tc<D, 32>(tp, km, vm, s);
  if (rows <= 64) return launch_tc<D, 64>(tp, km, vm, s);
  return launch_tc<D, 128>(tp, km, vm, s);
}

template <int D>
cudaError_t launch_mma(AttendParams& p, cudaStream_t s) {
  // a second row tile of 16 only where there are rows for it
  if (p.n * p.g <= 16)
    return launch_attend<__nv_bfloat16, D, 16>(attend_mma_kernel<D, 1>, p, kMmaThreads,
                                               MmaCfg<D, 1>::kSmem, s);
  return launch_attend<__nv_bfloat16, D, 32>(attend_mma_kernel<D, 2>, p, kMmaThreads,
                                             MmaCfg<D, 2>::kSmem, s);
}

template <int D>
cudaError_t launch_f32(AttendParams& p, cudaStream_t s) {
  const int rows = p.n * p.g;
  if (rows <= 4)
    return launch_attend<float, D, 4>(attend_f32_kernel<D, 4>, p, kF32Threads, F32Cfg<D, 4>::kSmem,
                                      s);
  if (rows <= 8)
    return launch_attend<float, D, 8>(attend_f32_kernel<D, 8>, p, kF32Threads, F32Cfg<D, 8>::kSmem,
                                      s);
  return launch_attend<float, D, 16>(attend_tf32_kernel<D>, p, kF32Threads, Tf32Cfg<D>::kSmem, s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

sv_status sv_kv_plan(const int32_t* kv_len, const int32_t* written, const int32_t* accepted_len,
                     const int32_t* release, const int32_t* new_len, int B, int max_new,
                     int page_size, int num_pages, int32_t* block_table, int max_pages,
                     const int32_t* pages, int32_t* free_pages, const int32_t* free_count,
                     int32_t* kv_len_out, int32_t* pages_out, int32_t* free_count_out,
                     int32_t* q_len, int64_t* slot_map, int32_t* positions, int32_t* device_status,
                     void* stream) {
  if (B < 0 || max_new < 1 || page_size < 1 || num_pages < 1 || max_pages < 1)
    return SV_ERR_INVALID_ARG;
  if (B == 0) {  // no request changes the stack
    if (!free_count || !free_count_out || !aligned(free_count, 4) || !aligned(free_count_out, 4))
      return SV_ERR_INVALID_ARG;
    if (free_count == free_count_out) return SV_OK;
    return cuda_status(cudaMemcpyAsync(free_count_out, free_count, 4, cudaMemcpyDeviceToDevice,
                                       reinterpret_cast<cudaStream_t>(stream)));
  }
  const void* need[] = {kv_len, new_len,    block_table, pages,          free_pages,
                        free_count, kv_len_out, pages_out,   free_count_out, q_len};
  for (const void* x : need)
    if (!x || !aligned(x, 4)) return SV_ERR_INVALID_ARG;
  const void* may[] = {written, accepted_len, release, positions, device_status};
  for (const void* x : may)
    if (!aligned_or_null(x, 4)) return SV_ERR_INVALID_ARG;
  if (!slot_map || !aligned(slot_map, 8)) return SV_ERR_INVALID_ARG;
  if (accepted_len && !written) return SV_ERR_INVALID_ARG;
  if (B > kPlanMaxB || (long long)B * max_pages > 0x7fffffffLL ||
      (long long)B * max_new > 0x7fffffffLL)
    return SV_ERR_UNSUPPORTED;
  if (page_size > (1 << 30) || max_new > (1 << 30)) return SV_ERR_UNSUPPORTED;
  PlanParams p = {};
  p.kv_len = kv_len;
  p.written = written;
  p.accepted = accepted_len;
  p.release = release;
  p.new_len = new_len;
  p.pages = pages;
  p.free_count = free_count;
  p.B = B;
  p.max_new = max_new;
  p.page = page_size;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.div_page = make_fastdiv(page_size);
  p.div_new = make_fastdiv(max_new);
  p.table = block_table;
  p.free_pages = free_pages;
  p.kv_len_out = kv_len_out;
  p.pages_out = pages_out;
  p.free_count_out = free_count_out;
  p.q_len = q_len;
  p.slot_map = slot_map;
  p.positions = positions;
  p.status = device_status;
  const long long slots = (long long)B * max_new;
  p.write_slots = slots <= kPlanInlineSlots;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch(kv_plan_kernel, p, dim3(1), plan_threads(B, slots),
                         (int)plan_smem(B), s);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  if (!p.write_slots) {
    constexpr int kPerBlock = kSlotThreads * kSlotPer;
    e = launch_after(kv_plan_slots_kernel, p,
                     dim3((unsigned)((max_new + kPerBlock - 1) / kPerBlock), (unsigned)B),
                     kSlotThreads, s);
  }
  return cuda_status(e);
}

sv_status sv_kv_append(const sv_kv_cache* cache, const void* k, const void* v, int B, int n,
                       int64_t batch_stride, int64_t token_stride, const int64_t* slot_map,
                       int32_t* device_status, void* stream) {
  if (B < 0 || n < 1) return SV_ERR_INVALID_ARG;
  const sv_status st = check_cache(cache);
  if (st != SV_OK) return st;
  if (batch_stride < 0 || token_stride < 0) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  const int es = esize(cache->dtype);
  if (!k || !v || !slot_map || !aligned(k, es) || !aligned(v, es) || !aligned(slot_map, 8) ||
      !aligned_or_null(device_status, 4))
    return SV_ERR_INVALID_ARG;
  if (batch_stride > (1LL << 40) || token_stride > (1LL << 40)) return SV_ERR_INVALID_ARG;
  AppendParams p = {};
  p.k = static_cast<const unsigned char*>(k);
  p.v = static_cast<const unsigned char*>(v);
  p.kc = static_cast<unsigned char*>(cache->k);
  p.vc = static_cast<unsigned char*>(cache->v);
  p.in_b = batch_stride * es;
  p.in_t = token_stride * es;
  p.c_page = cache->page_stride * es;
  p.c_token = cache->token_stride * es;
  p.c_head = cache->head_stride * es;
  p.slot_map = slot_map;
  p.B = B;
  p.n = n;
  p.heads = cache->heads;
  p.page = cache->page_size;
  p.num_pages = cache->num_pages;
  p.status = device_status;
  if ((long long)B * n > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  const long long row = (long long)cache->head_dim * es;
  const int w = common_width({addr(k), addr(v), addr(cache->k), addr(cache->v), p.in_b, p.in_t,
                              p.c_page, p.c_token, p.c_head, row});
  if (row / w * p.heads > 0x3fffffffLL) return SV_ERR_UNSUPPORTED;  // counted in int
  p.head_chunks = (int)(row / w);
  if (p.heads > 1 && p.c_head == row) {  // a token's heads are one row
    p.head_chunks *= p.heads;
    p.heads = 1;
  }
  p.div_n = make_fastdiv(n);
  p.div_page = make_fastdiv(cache->page_size);
  p.div_chunks = make_fastdiv(p.head_chunks);
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) return SV_ERR_CUDA;
  // as many warps as are on the device at once, each with a run of tokens
  const long long tokens = (long long)B * n, most = (long long)sms * 64;
  p.per_warp = (int)((tokens + most - 1) / most);
  const long long warps = (tokens + p.per_warp - 1) / p.per_warp;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (w) {
    case 16: return cuda_status(launch(kv_append_kernel<uint4>, p, dim3(grid), 256, 0, s));
    case 8: return cuda_status(launch(kv_append_kernel<uint2>, p, dim3(grid), 256, 0, s));
    case 4: return cuda_status(launch(kv_append_kernel<uint32_t>, p, dim3(grid), 256, 0, s));
    default: return cuda_status(launch(kv_append_kernel<uint16_t>, p, dim3(grid), 256, 0, s));
  }
}

size_t sv_kv_attend_scratch_size(int B, int n, int q_heads, int heads, int head_dim,
                                   sv_dtype dtype) {
  if (B < 0 || n < 1 || heads < 1 || q_heads < 1 || head_dim < 1 || head_dim > 256 ||
      (dtype != SV_F32 && dtype != SV_BF16))
    return 0;
  if (n > 1024 || q_heads % heads) return 0;
  return attend_scratch(n * (q_heads / heads), head_dim, dtype);
}

sv_status sv_kv_attend(const sv_kv_cache* cache, const void* q, int64_t batch_stride,
                       int64_t token_stride, int B, int n, int q_heads, const int32_t* block_table,
                       int max_pages, const int32_t* kv_len, const int32_t* q_len,
                       const int32_t* parents, float scale, void* out, float* lse, void* scratch,
                       size_t scratch_bytes, int32_t* device_status, void* stream) {
  if (B < 0 || n < 1 || n > 1024 || q_heads < 1 || max_pages < 1) return SV_ERR_INVALID_ARG;
  const sv_status st = check_cache(cache);
  if (st != SV_OK) return st;
  if (q_heads % cache->heads) return SV_ERR_INVALID_ARG;
  if (!isfinite(scale) || !isfinite(scale * 1.4426950408889634f)) return SV_ERR_INVALID_ARG;
  if (batch_stride < 0 || token_stride < 0 || batch_stride > (1LL << 40) ||
      token_stride > (1LL << 40))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  const int es = esize(cache->dtype);
  if (!q || !out || out == q || !block_table || !kv_len || !aligned(q, es) || !aligned(out, es) ||
      !aligned(block_table, 4) || !aligned(kv_len, 4) || !aligned_or_null(q_len, 4) ||
      !aligned_or_null(parents, 4) || !aligned_or_null(lse, 4) ||
      !aligned_or_null(device_status, 4))
    return SV_ERR_INVALID_ARG;
  if (q_heads > (1 << 16) || (long long)B * n > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  if (!scratch || !aligned(scratch, 16) ||
      scratch_bytes <
          attend_scratch(n * (q_heads / cache->heads), cache->head_dim, cache->dtype))
    return SV_ERR_WORKSPACE;
  AttendParams p = {};
  p.q = q;
  p.k = cache->k;
  p.v = cache->v;
  p.table = block_table;
  p.kv_len = kv_len;
  p.q_len = q_len;
  p.parents = parents;
  p.out = out;
  p.lse = lse;
  p.B = B;
  p.n = n;
  p.hkv = cache->heads;
  p.g = q_heads / cache->heads;
  p.d = cache->head_dim;
  p.page = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages;
  p.q_b = batch_stride;
  p.q_t = token_stride;
  p.c_page = cache->page_stride;
  p.c_token = cache->token_stride;
  p.c_head = cache->head_stride;
  p.div_g = make_fastdiv(p.g);
  p.div_page = make_fastdiv(p.page);
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.shared = static_cast<AttShared*>(scratch);
  p.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(scratch) + kSharedBytes);
  p.status = device_status;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = common_width({addr(cache->k), addr(cache->v), p.c_page * es, p.c_token * es,
                                 p.c_head * es, (long long)p.d * es}) == 16;
  // The matrix kernels take 16-byte rows of the cache and of out, and q in pairs.
  const bool pairs = common_width({addr(q), p.q_b * es, p.q_t * es}) >= 4 &&
                     aligned(out, 16);
  cudaError_t e;
  // 16 rows: where the two kernels of bf16 take the same time (65 us each for 32
  // requests of 700 to 9000 tokens); at 8 rows 59 us each, at 28 rows 106 us
  // against 70, and with short contexts the kernel of few rows wins up to 16.
  const int box = tc_box(p.page);
  CUtensorMap km, vm;
  if (cache->dtype == SV_BF16 && vec && aligned(out, 16) && p.d <= 128 && p.n * p.g > 16 && box &&
      scale > 0.f &&
      common_width({addr(q), p.q_b * es, p.q_t * es}) == 16 && tc_map(p, p.k, box, &km) &&
      tc_map(p, p.v, box, &vm)) {
    const long long wait = knob(SV_KNOB_WAIT_NS);
    const TcParams tp = {p, box, wait > 0 ? (unsigned long long)wait : kWaitLimitNs,
                         knob(SV_KNOB_STALL) != 0};
    e = p.d > 64 ? launch_tc<128>(tp, km, vm, s) : launch_tc<64>(tp, km, vm, s);
  } else if (cache->dtype == SV_BF16 && vec && pairs && p.d > 64 && p.d <= 128)
    e = launch_mma<128>(p, s);
  else if (cache->dtype == SV_BF16 && vec && pairs && p.d <= 64)
    e = launch_mma<64>(p, s);
  else if (cache->dtype == SV_F32 && vec && aligned(out, 16) && p.d <= 128)
    e = p.d > 64 ? launch_f32<128>(p, s) : launch_f32<64>(p, s);
  else if (cache->dtype == SV_BF16)
    e = vec ? launch_general<__nv_bfloat16, true>(p, s)
            : launch_general<__nv_bfloat16, false>(p, s);
  else
    e = vec ? launch_general<float, true>(p, s) : launch_general<float, false>(p, s);
  return cuda_status(e);
}

sv_status sv_kv_commit(const sv_kv_cache* cache, int layers, int64_t layer_stride, int B,
                       const int32_t* block_table, int max_pages, const int32_t* kv_len,
                       const int32_t* accepted_nodes, int width, const int32_t* accepted_len,
                       int32_t* device_status, void* stream) {
  return sv_kv_commit_ragged(cache, layers, layer_stride, B, block_table, max_pages, kv_len,
                             nullptr, accepted_nodes, width, accepted_len, device_status, stream);
}

sv_status sv_kv_commit_ragged(const sv_kv_cache* cache, int layers, int64_t layer_stride, int B,
                              const int32_t* block_table, int max_pages, const int32_t* kv_len,
                              const int32_t* q_len, const int32_t* accepted_nodes, int width,
                              const int32_t* accepted_len, int32_t* device_status,
                              void* stream) {
  if (B < 0 || layers < 1 || layer_stride < 0 || max_pages < 1 || width < 1)
    return SV_ERR_INVALID_ARG;
  const sv_status st = check_cache(cache, layers, layer_stride);
  if (st != SV_OK) return st;
  if (width > kCommitMaxWidth || B > 65535) return SV_ERR_UNSUPPORTED;
  if (B == 0) return SV_OK;
  if (!block_table || !kv_len || !accepted_nodes || !accepted_len || !aligned(block_table, 4) ||
      !aligned(kv_len, 4) || !aligned(accepted_nodes, 4) || !aligned(accepted_len, 4) ||
      !aligned_or_null(q_len, 4) || !aligned_or_null(device_status, 4))
    return SV_ERR_INVALID_ARG;
  const int es = esize(cache->dtype);
  CommitParams p = {};
  p.kc = static_cast<unsigned char*>(cache->k);
  p.vc = static_cast<unsigned char*>(cache->v);
  p.c_layer = layer_stride * es;
  p.c_page = cache->page_stride * es;
  p.c_token = cache->token_stride * es;
  p.c_head = cache->head_stride * es;
  p.table = block_table;
  p.kv_len = kv_len;
  p.q_len = q_len;
  p.nodes = accepted_nodes;
  p.accepted = accepted_len;
  p.B = B;
  p.width = width;
  p.layers = layers;
  p.heads = cache->heads;
  p.page = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_pages = max_pages;
  p.status = device_status;
  const long long row = (long long)cache->head_dim * es;
  const int w = common_width(
      {addr(cache->k), addr(cache->v), p.c_layer, p.c_page, p.c_token, p.c_head, row});
  const long long per_token = row / w * p.heads;
  if (per_token > 0x3fffffffLL || 2LL * layers * per_token > 0x3fffffffLL ||  // counted in int
      cache->page_size > (1 << 30))
    return SV_ERR_UNSUPPORTED;
  const long long items = 2LL * layers * per_token;
  p.head_chunks = (int)(row / w);
  if (p.heads > 1 && p.c_head == row) {  // a token's heads are one row
    p.head_chunks *= p.heads;
    p.heads = 1;
  }
  p.div_page = make_fastdiv(cache->page_size);
  p.div_chunks = make_fastdiv(p.heads * p.head_chunks);
  p.div_head = make_fastdiv(p.head_chunks);
  const long long blocks = (items + kCommitThreads - 1) / kCommitThreads;
  const dim3 grid((unsigned)blocks, (unsigned)B);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (w) {
    case 16: return cuda_status(launch(kv_commit_kernel<uint4>, p, grid, kCommitThreads, 0, s));
    case 8: return cuda_status(launch(kv_commit_kernel<uint2>, p, grid, kCommitThreads, 0, s));
    case 4: return cuda_status(launch(kv_commit_kernel<uint32_t>, p, grid, kCommitThreads, 0, s));
    default: return cuda_status(launch(kv_commit_kernel<uint16_t>, p, grid, kCommitThreads, 0, s));
  }
}

}  // extern "C"
