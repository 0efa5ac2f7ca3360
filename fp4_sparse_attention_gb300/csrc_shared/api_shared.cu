// api_shared.cu -- the C ABI of the calls for requests that share a prefix
// (include/fp4idx.h): host-side argument checks and launches.  Nothing here
// reads device memory or synchronises.
#include <cstring>

#include "fp4idx.h"
#include "internal.h"
#include "shared.h"

namespace fp4idx {
namespace {

#define FAIL(status, ...)        \
  do {                           \
    set_last_error(__VA_ARGS__); \
    return status;               \
  } while (0)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fp4idx_status_t cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FP4IDX_OK;
  FAIL(FP4IDX_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// int32 arrays that a call cannot do without.
template <class... P>
fp4idx_status_t check_arrays(const char* names, P... ptrs) {
  for (const int32_t* ptr : {static_cast<const int32_t*>(ptrs)...})
    if (!ptr || !aligned(ptr, 4)) FAIL(FP4IDX_EINVAL, "%s are required, 4-byte aligned", names);
  return FP4IDX_OK;
}

fp4idx_status_t check_pool(int32_t num_reqs, int32_t page_size, int64_t num_pages, int64_t table_stride) {
  if (num_reqs < 1 || num_pages < 1 || table_stride < 1)
    FAIL(FP4IDX_EINVAL, "num_reqs, num_pages and table_stride >= 1 required");
  if (page_size != 64 && page_size != 128)
    FAIL(FP4IDX_EUNSUPPORTED, "page_size %d: only 64 and 128 are supported", page_size);
  if (num_pages > INT32_MAX / page_size) FAIL(FP4IDX_EUNSUPPORTED, "num_pages * page_size must be below 2^31");
  if (table_stride > INT32_MAX) FAIL(FP4IDX_EUNSUPPORTED, "table_stride must be below 2^31");
  return FP4IDX_OK;
}

fp4idx_status_t check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return FP4IDX_OK;
  if (!workspace || bytes < need)
    FAIL(FP4IDX_EWORKSPACE, "workspace of %zu bytes is smaller than %zu", workspace ? bytes : size_t{0}, need);
  if (!aligned(workspace, 16)) FAIL(FP4IDX_EINVAL, "workspace must be 16-byte aligned");
  return FP4IDX_OK;
}

// What the attention calls check, and what the groups add.
fp4idx_status_t check_shared(const fp4idx_shared_attention_t* s) {
  if (!s) FAIL(FP4IDX_EINVAL, "shared is NULL");
  const fp4idx_attention_t* a = &s->attention;
  if (!a->v) FAIL(FP4IDX_EUNSUPPORTED, "v is NULL: a shared prefix is supported for K/V caches only");
  if (a->indices) FAIL(FP4IDX_EINVAL, "indices: a shared prefix is attended to whole");
  const fp4idx_status_t st = check_attention(a, false);
  if (st != FP4IDX_OK) return st;
  if (s->num_groups < 1 || s->max_group_rows < 1) FAIL(FP4IDX_EINVAL, "num_groups and max_group_rows >= 1 required");
  if (!s->group_offsets || !s->prefix_len || !aligned(s->group_offsets, 4) || !aligned(s->prefix_len, 4))
    FAIL(FP4IDX_EINVAL, "group_offsets and prefix_len are required, 4-byte aligned");
  if (s->num_groups > 1 << 20 || s->max_group_rows > 1 << 20)
    FAIL(FP4IDX_EUNSUPPORTED, "up to 2^20 groups and 2^20 rows a group are supported");
  return FP4IDX_OK;
}

SharedParams shared_params(const fp4idx_shared_attention_t* s) {
  SharedParams p;
  std::memset(&p, 0, sizeof(p));
  p.a = attention_params(&s->attention);
  p.group_offsets = s->group_offsets;
  p.prefix_len = s->prefix_len;
  p.num_groups = s->num_groups;
  p.max_group_rows = s->max_group_rows;
  return p;
}

fp4idx_status_t shared_maps(const fp4idx_attention_t* a, SharedMaps* maps) {
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(a->num_kv_heads) * a->page_size, kPagedDim / 64,
                              static_cast<cuuint64_t>(a->num_pages)};
  const cuuint64_t strides[3] = {kPagedDim * 2, 128, static_cast<cuuint64_t>(a->page_stride) * 2};
  const cuuint32_t k_box[4] = {64, 64, 1, 1}, v_box[4] = {64, 64, 2, 1}, part_box[4] = {64, 16, 1, 1};
  fp4idx_status_t s = call_tensor_map16(&maps->k, a->k, 4, dims, strides, k_box);
  if (s == FP4IDX_OK) s = call_tensor_map16(&maps->v, a->v, 4, dims, strides, v_box);
  return s != FP4IDX_OK ? s : call_tensor_map16(&maps->v_part, a->v, 4, dims, strides, part_box);
}

PoolParams pool_params(int32_t num_reqs, int32_t page_size, int64_t num_pages, const int32_t* block_table,
                       int64_t table_stride, uint32_t* err) {
  PoolParams p;
  std::memset(&p, 0, sizeof(p));
  p.num_reqs = num_reqs;
  p.page_shift = page_size == 128 ? 7 : 6;
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.table_stride = table_stride;
  p.width = static_cast<int32_t>(table_stride);
  p.err = err;
  return p;
}

}  // namespace
}  // namespace fp4idx

using namespace fp4idx;

extern "C" {

size_t fp4idx_shared_attention_workspace_bytes(const fp4idx_shared_attention_t* shared) {
  set_last_error("%s", "");
  if (check_shared(shared) != FP4IDX_OK) return 0;
  SharedParams p = shared_params(shared);
  int sms = 0;
  if (shared->attention.num_rows == 0 || call_device(&sms, &p.a.err) != FP4IDX_OK || !plan_shared(&p, sms)) return 0;
  return shared_workspace(p);
}

fp4idx_status_t fp4idx_shared_prefix_attention(const fp4idx_shared_attention_t* shared, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  set_last_error("%s", "");
  fp4idx_status_t s = check_shared(shared);
  if (s != FP4IDX_OK) return s;
  if (shared->attention.num_rows == 0) return FP4IDX_OK;
  SharedParams p = shared_params(shared);
  int sms = 0;
  if ((s = call_device(&sms, &p.a.err)) != FP4IDX_OK) return s;
  if (!plan_shared(&p, sms))
    FAIL(FP4IDX_EUNSUPPORTED, "more than 2^20 blocks of 256 (row, head) pairs over all groups, or 2^31 key tiles");
  if ((s = check_workspace(workspace, workspace_bytes, shared_workspace(p))) != FP4IDX_OK) return s;
  SharedMaps maps;
  if ((s = shared_maps(&shared->attention, &maps)) != FP4IDX_OK) return s;
  return cuda_status(launch_shared(p, maps, shared->attention.dtype, workspace, static_cast<cudaStream_t>(stream)),
                     "shared-prefix attention launch");
}

fp4idx_status_t fp4idx_fork_requests(const int32_t* parent, const int32_t* child, const int32_t* fork_len,
                                     int32_t num_forks, int32_t num_reqs, int32_t page_size, int64_t num_pages,
                                     const int32_t* free_pages, int32_t num_free, int32_t* cached_len,
                                     int32_t* block_table, int64_t table_stride, int32_t* copy_src,
                                     int32_t* copy_dst, int32_t* pages_taken, void* stream) {
  set_last_error("%s", "");
  fp4idx_status_t s = check_pool(num_reqs, page_size, num_pages, table_stride);
  if (s != FP4IDX_OK) return s;
  if (num_forks < 0 || num_free < 0) FAIL(FP4IDX_EINVAL, "num_forks and num_free >= 0 required");
  if ((s = check_arrays("cached_len, block_table and pages_taken", cached_len, block_table, pages_taken)) != FP4IDX_OK) return s;
  if (num_forks > 0 && (s = check_arrays("parent, child, copy_src and copy_dst", parent, child, copy_src, copy_dst)) != FP4IDX_OK)
    return s;
  if (num_free > 0 && (s = check_arrays("free_pages", free_pages)) != FP4IDX_OK) return s;
  if (!aligned(fork_len, 4)) FAIL(FP4IDX_EINVAL, "fork_len must be 4-byte aligned");
  ForkParams p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  if ((s = call_device(&sms, &p.err)) != FP4IDX_OK) return s;
  p.parent = parent;
  p.child = child;
  p.fork_len = fork_len;
  p.num_forks = num_forks;
  p.num_reqs = num_reqs;
  p.page_size = page_size;
  p.page_shift = page_size == 128 ? 7 : 6;
  p.num_pages = num_pages;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.cached_len = cached_len;
  p.block_table = block_table;
  p.table_stride = table_stride;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.pages_taken = pages_taken;
  return cuda_status(launch_fork(p, static_cast<cudaStream_t>(stream)), "fork launch");
}

fp4idx_status_t fp4idx_copy_pages(const fp4idx_page_span_t* spans, int32_t num_spans, int64_t num_pages,
                                  const int32_t* src, const int32_t* dst, int32_t num_copies, const int32_t* count,
                                  void* stream) {
  set_last_error("%s", "");
  if (!spans || num_spans < 1 || num_pages < 1 || num_copies < 0)
    FAIL(FP4IDX_EINVAL, "spans, num_spans >= 1, num_pages >= 1 and num_copies >= 0 required");
  if (num_spans > kMaxSpans) FAIL(FP4IDX_EUNSUPPORTED, "num_spans %d: up to %d", num_spans, kMaxSpans);
  if (num_pages > INT32_MAX) FAIL(FP4IDX_EUNSUPPORTED, "num_pages below 2^31 supported");
  CopyParams p;
  std::memset(&p, 0, sizeof(p));
  int64_t pieces = 0;
  for (int i = 0; i < num_spans; ++i) {
    const fp4idx_page_span_t& x = spans[i];
    if (!x.base || !aligned(x.base, 16) || x.page_bytes < 16 || x.page_bytes % 16 || x.page_stride % 16 ||
        x.page_stride < x.page_bytes)
      FAIL(FP4IDX_EINVAL, "span %d: base, page_stride and page_bytes must be multiples of 16 and page_stride >= page_bytes >= 16", i);
    if (x.page_bytes > int64_t{1} << 32) FAIL(FP4IDX_EUNSUPPORTED, "span %d: pages of up to 4 GB", i);
    p.span[i].base = static_cast<uint4*>(x.base);
    p.span[i].page_stride = x.page_stride / 16;
    p.span[i].units = static_cast<int32_t>(x.page_bytes / 16);
    pieces += p.span[i].units;
  }
  if (pieces > INT32_MAX) FAIL(FP4IDX_EUNSUPPORTED, "pages of more than 2^31 16-byte pieces in all spans");
  if (num_copies == 0) return FP4IDX_OK;
  fp4idx_status_t s = check_arrays("src and dst", src, dst);
  if (s != FP4IDX_OK) return s;
  if (!aligned(count, 4)) FAIL(FP4IDX_EINVAL, "count must be 4-byte aligned");
  int sms = 0;
  if ((s = call_device(&sms, &p.err)) != FP4IDX_OK) return s;
  p.src = src;
  p.dst = dst;
  p.count = count;
  p.num_copies = num_copies;
  p.num_spans = num_spans;
  p.num_pages = num_pages;
  return cuda_status(launch_copy_pages(p, sms, static_cast<cudaStream_t>(stream)), "page copy launch");
}

size_t fp4idx_pages_workspace_bytes(int64_t num_pages, int32_t num_reqs, int64_t table_stride) {
  set_last_error("%s", "");
  return num_pages < 1 || num_pages > INT32_MAX || num_reqs < 1 || table_stride < 1 ? 0 : pool_workspace(num_pages, num_reqs, table_stride);
}

fp4idx_status_t fp4idx_release_pages(const int32_t* requests, const int32_t* keep_len, int32_t num_released,
                                     int32_t num_reqs, int32_t page_size, int64_t num_pages, int32_t* cached_len,
                                     const int32_t* block_table, int64_t table_stride, int32_t* free_pages,
                                     int32_t* num_free, void* workspace, size_t workspace_bytes, void* stream) {
  set_last_error("%s", "");
  fp4idx_status_t s = check_pool(num_reqs, page_size, num_pages, table_stride);
  if (s != FP4IDX_OK) return s;
  if (num_released < 0) FAIL(FP4IDX_EINVAL, "num_released >= 0 required");
  if ((s = check_arrays("cached_len, block_table, free_pages and num_free", cached_len, block_table, free_pages, num_free)) !=
      FP4IDX_OK)
    return s;
  if (num_released > 0 && (s = check_arrays("requests", requests)) != FP4IDX_OK) return s;
  if (!aligned(keep_len, 4)) FAIL(FP4IDX_EINVAL, "keep_len must be 4-byte aligned");
  if ((s = check_workspace(workspace, workspace_bytes, pool_workspace(num_pages, num_reqs, table_stride))) != FP4IDX_OK) return s;
  int sms = 0;
  uint32_t* err = nullptr;
  if ((s = call_device(&sms, &err)) != FP4IDX_OK) return s;
  PoolParams p = pool_params(num_reqs, page_size, num_pages, block_table, table_stride, err);
  p.requests = requests;
  p.keep_len = keep_len;
  p.num_released = num_released;
  p.cached_len = cached_len;
  p.free_pages = free_pages;
  p.num_free = num_free;
  return cuda_status(launch_release(p, sms, workspace, static_cast<cudaStream_t>(stream)), "release launch");
}

fp4idx_status_t fp4idx_compact_pages(const int32_t* cached_len, int32_t num_reqs, int32_t page_size, int64_t num_pages,
                                     const int32_t* block_table, int64_t table_stride, int32_t width, int32_t* new_table,
                                     int64_t new_stride, int32_t max_moves, int32_t* copy_src, int32_t* copy_dst,
                                     int32_t* num_moves, int32_t* extent, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  set_last_error("%s", "");
  fp4idx_status_t s = check_pool(num_reqs, page_size, num_pages, table_stride);
  if (s != FP4IDX_OK) return s;
  if (width < 1 || width > table_stride || width > new_stride)
    FAIL(FP4IDX_EINVAL, "width must be at least 1 and at most table_stride and new_stride");
  if (new_table == block_table && new_stride != table_stride)
    FAIL(FP4IDX_EINVAL, "a table rewritten in place keeps its stride");
  if (max_moves < 0) FAIL(FP4IDX_EINVAL, "max_moves >= 0 required");
  if ((s = check_arrays("cached_len, block_table, new_table, num_moves and extent", cached_len, block_table, new_table, num_moves,
                        extent)) != FP4IDX_OK)
    return s;
  if (max_moves > 0 && (s = check_arrays("copy_src and copy_dst", copy_src, copy_dst)) != FP4IDX_OK) return s;
  if ((s = check_workspace(workspace, workspace_bytes, pool_workspace(num_pages, num_reqs, table_stride))) != FP4IDX_OK) return s;
  int sms = 0;
  uint32_t* err = nullptr;
  if ((s = call_device(&sms, &err)) != FP4IDX_OK) return s;
  PoolParams p = pool_params(num_reqs, page_size, num_pages, block_table, table_stride, err);
  p.cached_len = const_cast<int32_t*>(cached_len);
  p.width = width;
  p.new_table = new_table;
  p.new_stride = new_stride;
  p.max_moves = max_moves;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.num_moves = num_moves;
  p.extent = extent;
  return cuda_status(launch_compact(p, sms, workspace, static_cast<cudaStream_t>(stream)), "compaction launch");
}

}  // extern "C"
