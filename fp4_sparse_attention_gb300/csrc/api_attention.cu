// api_attention.cu -- the C ABI of the attention calls, the 16-bit cache
// writers and the step tables (include/fp4idx.h): host-side argument checks
// and launches.  Nothing here reads device memory or synchronises.
#include <cfloat>
#include <cmath>
#include <cstring>

#include "attention.h"
#include "fp4idx.h"
#include "internal.h"

namespace fp4idx {
namespace {

#define FAIL(status, ...)        \
  do {                           \
    set_last_error(__VA_ARGS__); \
    return status;               \
  } while (0)

constexpr float kLog2e = 1.44269504088896341f;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fp4idx_status_t cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FP4IDX_OK;
  FAIL(FP4IDX_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Arguments of either attention call.
fp4idx_status_t check_attention(const fp4idx_attention_t* a, bool latent) {
  if (!a) FAIL(FP4IDX_EINVAL, "attention is NULL");
  if (a->dtype != FP4IDX_BF16 && a->dtype != FP4IDX_FP16)
    FAIL(FP4IDX_EINVAL, "dtype %d is neither BF16 (0) nor FP16 (1)", a->dtype);
  if (a->num_seqs < 1 || a->num_rows < 0) FAIL(FP4IDX_EINVAL, "num_seqs >= 1 and num_rows >= 0 required");
  if (a->num_heads < 1 || a->num_kv_heads < 1 || a->num_heads % a->num_kv_heads != 0)
    FAIL(FP4IDX_EINVAL, "num_heads (%d) must be a positive multiple of num_kv_heads (%d)", a->num_heads,
         a->num_kv_heads);
  if (a->num_heads > 1024) FAIL(FP4IDX_EUNSUPPORTED, "num_heads %d: supported up to 1024", a->num_heads);
  if (latent && a->num_kv_heads != 1)
    FAIL(FP4IDX_EINVAL, "latent attention has one shared latent (num_kv_heads = %d)", a->num_kv_heads);
  if (latent && a->v) FAIL(FP4IDX_EINVAL, "latent attention takes no v: the values are the cache's first 512");
  if (a->page_size != 64 && a->page_size != 128)
    FAIL(FP4IDX_EUNSUPPORTED, "page_size %d: only 64 and 128 are supported", a->page_size);
  if (a->num_pages < 1) FAIL(FP4IDX_EINVAL, "num_pages must be >= 1");
  if (a->num_pages >= INT32_MAX || a->page_stride >= int64_t{1} << 39 ||
      static_cast<int64_t>(a->num_kv_heads) * a->page_size > INT32_MAX)
    FAIL(FP4IDX_EUNSUPPORTED, "num_pages below 2^31 - 1 and page_stride below 2^39 are supported");
  if (a->max_seqlen_q < 1 || a->max_seqlen_k < 0)
    FAIL(FP4IDX_EINVAL, "max_seqlen_q >= 1 and max_seqlen_k >= 0 required");
  if (a->max_seqlen_k > 1 << 30) FAIL(FP4IDX_EUNSUPPORTED, "max_seqlen_k %d: up to 2^30", a->max_seqlen_k);
  // (a call without rows may come with the null pointers of empty tensors)
  if ((a->num_rows > 0 && (!a->q || !a->out)) || !a->k || (!latent && !a->v) || !a->cu_seqlens_q || !a->cu_seqlens_k ||
      !a->block_table)
    FAIL(FP4IDX_EINVAL, "q, k, v (paged), cu_seqlens_q, cu_seqlens_k, block_table and out are required");
  const int dk = latent ? kLatentDim + kRopeDim : kPagedDim, dv = latent ? kLatentDim : kPagedDim;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 16))
    FAIL(FP4IDX_EINVAL, "q, k, v and out must be 16-byte aligned");
  if (!aligned(a->lse, 4) || !aligned(a->indices, 4)) FAIL(FP4IDX_EINVAL, "lse and indices must be 4-byte aligned");
  if (a->q_head_stride < dk || a->q_head_stride % 8 != 0)
    FAIL(FP4IDX_EINVAL, "q_head_stride %lld must be a multiple of 8 and >= %d",
         static_cast<long long>(a->q_head_stride), dk);
  if (a->q_row_stride < dk || a->q_row_stride % 8 != 0)
    FAIL(FP4IDX_EINVAL, "q_row_stride %lld must be a multiple of 8 and >= %d", static_cast<long long>(a->q_row_stride), dk);
  // a row holds its heads, or a head its rows (products computed by head)
  if (a->num_heads > 1 && a->num_rows > 1 && a->q_head_stride > (a->q_row_stride - dk) / (a->num_heads - 1) &&
      a->q_row_stride > (a->q_head_stride - dk) / (a->num_rows - 1))
    FAIL(FP4IDX_EINVAL, "q_row_stride %lld and q_head_stride %lld: the queries of %d rows and %d heads overlap",
         static_cast<long long>(a->q_row_stride), static_cast<long long>(a->q_head_stride), a->num_rows, a->num_heads);
  if (a->out_row_stride < static_cast<int64_t>(a->num_heads) * dv || a->out_row_stride % 8 != 0)
    FAIL(FP4IDX_EINVAL, "out_row_stride %lld must be a multiple of 8 and >= num_heads * %d",
         static_cast<long long>(a->out_row_stride), dv);
  if (a->page_stride < static_cast<int64_t>(a->num_kv_heads) * a->page_size * dk || a->page_stride % 8 != 0)
    FAIL(FP4IDX_EINVAL, "page_stride %lld must be a multiple of 8 and >= one page's content",
         static_cast<long long>(a->page_stride));
  if (!a->page_offsets) {
    const int64_t need = (static_cast<int64_t>(a->max_seqlen_k) + a->page_size - 1) / a->page_size;
    if (a->table_stride < need)
      FAIL(FP4IDX_EINVAL, "table_stride %lld < pages of max_seqlen_k (%lld)", static_cast<long long>(a->table_stride),
           static_cast<long long>(need));
  }
  if (a->qo_offset && !a->causal) FAIL(FP4IDX_EINVAL, "qo_offset is only allowed with causal != 0");
  if (!std::isfinite(a->scale * kLog2e)) FAIL(FP4IDX_EINVAL, "scale must be finite");
  if (a->indices && a->num_indices < 1) FAIL(FP4IDX_EINVAL, "num_indices must be >= 1 with indices");
  if (a->indices && a->num_indices > (1 << 20)) FAIL(FP4IDX_EUNSUPPORTED, "num_indices %d: up to 2^20", a->num_indices);
  return FP4IDX_OK;
}

AttnParams attention_params(const fp4idx_attention_t* a) {
  AttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_row_stride = a->q_row_stride;
  p.q_head_stride = a->q_head_stride;
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.page_stride = a->page_stride;
  p.num_pages = a->num_pages;
  p.cu_seqlens_q = a->cu_seqlens_q;
  p.cu_seqlens_k = a->cu_seqlens_k;
  p.block_table = a->block_table;
  p.page_offsets = a->page_offsets;
  p.table_stride = a->table_stride;
  p.visible_len = a->visible_len;
  p.qo_offset = a->qo_offset;
  p.causal = a->causal;
  p.page_size = a->page_size;
  p.page_shift = a->page_size == 128 ? 7 : 6;
  p.num_seqs = a->num_seqs;
  p.num_rows = a->num_rows;
  p.num_heads = a->num_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.group = a->num_heads / a->num_kv_heads;
  p.max_seqlen_q = a->max_seqlen_q;
  p.max_seqlen_k = a->max_seqlen_k;
  p.indices = a->indices;
  p.num_indices = a->indices ? a->num_indices : 0;
  // scale 0 becomes the smallest normal number: every finite score still is 0
  // to fp32, and a masked one stays -inf (not 0 * -inf)
  p.scale_log2 = std::fmax(std::fabs(a->scale) * kLog2e, FLT_MIN);
  p.negate = a->scale < 0.0f;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_row_stride = a->out_row_stride;
  p.lse = a->lse;
  return p;
}

// Tensor maps of the caches (selected latent rows are copied without one).
fp4idx_status_t cache_maps(const fp4idx_attention_t* a, bool latent, AttnMaps* maps) {
  std::memset(maps, 0, sizeof(*maps));
  if (latent && a->indices) return FP4IDX_OK;
  const cuuint64_t dk = latent ? kLatentDim + kRopeDim : kPagedDim;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(a->num_kv_heads) * a->page_size, dk / 64,
                              static_cast<cuuint64_t>(a->num_pages)};
  const cuuint64_t strides[3] = {dk * 2, 128, static_cast<cuuint64_t>(a->page_stride) * 2};
  const cuuint32_t box[4] = {64, 64, static_cast<cuuint32_t>(latent ? kLatentBoxPieces : kPagedBoxPieces), 1};
  fp4idx_status_t s = call_tensor_map16(&maps->k, a->k, 4, dims, strides, box);
  if (s != FP4IDX_OK || latent) return s;
  return call_tensor_map16(&maps->v, a->v, 4, dims, strides, box);
}

fp4idx_status_t attention_any(const fp4idx_attention_t* a, bool latent, void* workspace, size_t workspace_bytes,
                              void* stream) {
  set_last_error("%s", "");
  fp4idx_status_t s = check_attention(a, latent);
  if (s != FP4IDX_OK) return s;
  if (a->num_rows == 0) return FP4IDX_OK;
  AttnParams p = attention_params(a);
  int sms = 0;
  if ((s = call_device(&sms, &p.err)) != FP4IDX_OK) return s;
  if (!plan_attention(&p, sms)) FAIL(FP4IDX_EUNSUPPORTED, "more than 2^31 key tiles or 2^20 rows per request");
  const size_t need = attention_workspace(p);
  if (!workspace || workspace_bytes < need)
    FAIL(FP4IDX_EWORKSPACE, "workspace of %zu bytes is smaller than %zu", workspace ? workspace_bytes : size_t{0}, need);
  if (!aligned(workspace, 16)) FAIL(FP4IDX_EINVAL, "workspace must be 16-byte aligned");
  AttnMaps maps;
  if ((s = cache_maps(a, latent, &maps)) != FP4IDX_OK) return s;
  return cuda_status(launch_attention(p, maps, a->dtype, workspace, static_cast<cudaStream_t>(stream)), "attention launch");
}

// Arguments that both cache writers share.
fp4idx_status_t check_store(const int32_t* slots, int32_t num_tokens, int32_t heads, int32_t page_size,
                            int64_t num_pages, int64_t page_stride, int64_t page_elems) {
  if (!slots || !aligned(slots, 4)) FAIL(FP4IDX_EINVAL, "slots is NULL or not 4-byte aligned");
  if (num_tokens < 0 || heads < 1 || num_pages < 1)
    FAIL(FP4IDX_EINVAL, "num_tokens >= 0, num_kv_heads >= 1 and num_pages >= 1 required");
  if (heads > 1024) FAIL(FP4IDX_EUNSUPPORTED, "num_kv_heads %d: supported up to 1024", heads);
  if (page_size != 64 && page_size != 128)
    FAIL(FP4IDX_EUNSUPPORTED, "page_size %d: only 64 and 128 are supported", page_size);
  if (page_stride < page_elems || page_stride % 8 != 0)
    FAIL(FP4IDX_EINVAL, "page_stride %lld must be a multiple of 8 and >= one page's content",
         static_cast<long long>(page_stride));
  return FP4IDX_OK;
}

bool bad_source(const void* p, int64_t stride, int64_t least) {
  return !p || !aligned(p, 16) || stride < least || stride % 8 != 0;
}

fp4idx_status_t store_rows(StoreRowsParams* p, const int32_t* slots, int32_t num_tokens, int32_t heads,
                           int32_t page_size, int64_t num_pages, int64_t page_stride, void* stream) {
  if (num_tokens == 0) return FP4IDX_OK;
  const int64_t pieces = static_cast<int64_t>(num_tokens) * heads * (p->part[0].units + p->part[1].units);
  if (pieces > UINT32_MAX - 256) FAIL(FP4IDX_EUNSUPPORTED, "more than 2^32 16-byte pieces in a call");
  int sms = 0;
  fp4idx_status_t s = call_device(&sms, &p->err);
  if (s != FP4IDX_OK) return s;
  p->slots = slots;
  p->num_tokens = num_tokens;
  p->heads = heads;
  p->page_size = page_size;
  p->page_shift = page_size == 128 ? 7 : 6;
  p->num_pages = num_pages;
  p->page_stride = page_stride;
  return cuda_status(launch_store_rows(*p, sms, static_cast<cudaStream_t>(stream)), "store launch");
}

}  // namespace
}  // namespace fp4idx

using namespace fp4idx;

extern "C" {

size_t fp4idx_attention_workspace_bytes(const fp4idx_attention_t* attention) {
  set_last_error("%s", "");
  if (check_attention(attention, attention && attention->v == nullptr) != FP4IDX_OK) return 0;
  AttnParams p = attention_params(attention);
  int sms = 0;
  if (attention->num_rows == 0 || call_device(&sms, &p.err) != FP4IDX_OK || !plan_attention(&p, sms)) return 0;
  return attention_workspace(p);
}

fp4idx_status_t fp4idx_latent_attention(const fp4idx_attention_t* attention, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  return attention_any(attention, true, workspace, workspace_bytes, stream);
}

fp4idx_status_t fp4idx_paged_attention(const fp4idx_attention_t* attention, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return attention_any(attention, false, workspace, workspace_bytes, stream);
}

fp4idx_status_t fp4idx_store_latent(const void* latent, int64_t latent_stride, const void* rope, int64_t rope_stride,
                                    const int32_t* slots, int32_t num_tokens, int32_t page_size, int64_t num_pages,
                                    int64_t page_stride, void* cache, void* stream) {
  set_last_error("%s", "");
  constexpr int kRow = kLatentDim + kRopeDim;
  if (bad_source(latent, latent_stride, kLatentDim) || bad_source(rope, rope_stride, kRopeDim) || !cache ||
      !aligned(cache, 16))
    FAIL(FP4IDX_EINVAL, "latent, rope and cache must be 16-byte aligned, with token strides that are multiples of 8 "
                        "and hold 512 and 64 elements");
  fp4idx_status_t s = check_store(slots, num_tokens, 1, page_size, num_pages, page_stride,
                                  static_cast<int64_t>(page_size) * kRow);
  if (s != FP4IDX_OK) return s;
  StoreRowsParams p;
  std::memset(&p, 0, sizeof(p));
  p.part[0] = {static_cast<const uint16_t*>(latent), latent_stride, 0, static_cast<uint16_t*>(cache), 0, kRow,
               kLatentDim / 8};
  p.part[1] = {static_cast<const uint16_t*>(rope), rope_stride, 0, static_cast<uint16_t*>(cache) + kLatentDim, 0, kRow,
               kRopeDim / 8};
  return store_rows(&p, slots, num_tokens, 1, page_size, num_pages, page_stride, stream);
}

fp4idx_status_t fp4idx_store_kv(const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                                const int32_t* slots, int32_t num_tokens, int32_t num_kv_heads, int32_t page_size,
                                int64_t num_pages, int64_t page_stride, void* k, void* v, void* stream) {
  set_last_error("%s", "");
  const int64_t row = static_cast<int64_t>(num_kv_heads) * kPagedDim;
  if (bad_source(k_new, k_stride, row) || bad_source(v_new, v_stride, row) || !k || !v || !aligned(k, 16) ||
      !aligned(v, 16))
    FAIL(FP4IDX_EINVAL, "k_new, v_new, k and v must be 16-byte aligned, with token strides that are multiples of 8 "
                        "and hold num_kv_heads * 128 elements");
  fp4idx_status_t s = check_store(slots, num_tokens, num_kv_heads, page_size, num_pages, page_stride,
                                  static_cast<int64_t>(page_size) * row);
  if (s != FP4IDX_OK) return s;
  StoreRowsParams p;
  std::memset(&p, 0, sizeof(p));
  const int64_t head = static_cast<int64_t>(page_size) * kPagedDim;
  p.part[0] = {static_cast<const uint16_t*>(k_new), k_stride, kPagedDim, static_cast<uint16_t*>(k), head, kPagedDim,
               kPagedDim / 8};
  p.part[1] = {static_cast<const uint16_t*>(v_new), v_stride, kPagedDim, static_cast<uint16_t*>(v), head, kPagedDim,
               kPagedDim / 8};
  return store_rows(&p, slots, num_tokens, num_kv_heads, page_size, num_pages, page_stride, stream);
}

fp4idx_status_t fp4idx_build_tables(const int32_t* cached_len, const int32_t* new_len, int32_t num_reqs,
                                    int32_t num_rows, int32_t page_size, int64_t num_pages,
                                    const int32_t* free_pages, int32_t num_free, int32_t* block_table,
                                    int64_t table_stride, int32_t* cu_seqlens_q, int32_t* cu_seqlens_k,
                                    int32_t* visible_len, int32_t* slots, int32_t* pages_taken, void* stream) {
  set_last_error("%s", "");
  if (!cached_len || !new_len || !block_table || !cu_seqlens_q || !cu_seqlens_k || !pages_taken)
    FAIL(FP4IDX_EINVAL, "cached_len, new_len, block_table, cu_seqlens_q, cu_seqlens_k and pages_taken are required");
  if (num_reqs < 1 || num_rows < 0 || num_free < 0 || num_pages < 1 || table_stride < 1)
    FAIL(FP4IDX_EINVAL, "num_reqs, num_pages and table_stride >= 1, num_rows and num_free >= 0 required");
  if ((num_rows > 0 && (!visible_len || !slots)) || (num_free > 0 && !free_pages))
    FAIL(FP4IDX_EINVAL, "visible_len and slots (with rows) and free_pages (with free pages) are required");
  for (const void* ptr : {static_cast<const void*>(cached_len), static_cast<const void*>(new_len),
                          static_cast<const void*>(free_pages), static_cast<const void*>(block_table),
                          static_cast<const void*>(cu_seqlens_q), static_cast<const void*>(cu_seqlens_k),
                          static_cast<const void*>(visible_len), static_cast<const void*>(slots),
                          static_cast<const void*>(pages_taken)})
    if (!aligned(ptr, 4)) FAIL(FP4IDX_EINVAL, "every array must be 4-byte aligned");
  if (page_size != 64 && page_size != 128)
    FAIL(FP4IDX_EUNSUPPORTED, "page_size %d: only 64 and 128 are supported", page_size);
  if (num_pages > INT32_MAX / page_size) FAIL(FP4IDX_EUNSUPPORTED, "num_pages * page_size must be below 2^31");
  TablesParams p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  fp4idx_status_t s = call_device(&sms, &p.err);
  if (s != FP4IDX_OK) return s;
  p.cached_len = cached_len;
  p.new_len = new_len;
  p.num_reqs = num_reqs;
  p.num_rows = num_rows;
  p.page_size = page_size;
  p.page_shift = page_size == 128 ? 7 : 6;
  p.num_pages = num_pages;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.block_table = block_table;
  p.table_stride = table_stride;
  p.cu_seqlens_q = cu_seqlens_q;
  p.cu_seqlens_k = cu_seqlens_k;
  p.visible_len = visible_len;
  p.slots = slots;
  p.pages_taken = pages_taken;
  return cuda_status(launch_tables(p, sms, static_cast<cudaStream_t>(stream)), "table launch");
}

}  // extern "C"
