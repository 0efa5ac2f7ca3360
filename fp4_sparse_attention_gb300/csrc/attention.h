// attention.h -- parameters shared by the attention host layer
// (api_attention.cu) and its kernels.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4idx.h"

namespace fp4idx {

constexpr uint32_t kErrLengths = 0x8u;  // FP4IDX_ERR_LENGTHS

constexpr int kLatentDim = 512;  // shared latent values of a token (keys and values)
constexpr int kRopeDim = 64;     // rotary values of a token (keys only)
constexpr int kPagedDim = 128;   // head size of the paged K/V cache
constexpr int kSelectBlock = 128;  // keys of one selectable block

struct AttnParams {
  const uint16_t* q;
  int64_t q_row_stride, q_head_stride;  // elements
  const uint16_t* k;
  const uint16_t* v;                    // paged; the latent cache holds both in k
  int64_t page_stride;                  // elements
  int64_t num_pages;
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  const int32_t* block_table;
  const int32_t* page_offsets;
  int64_t table_stride;
  const int32_t* visible_len;
  const int32_t* qo_offset;
  int32_t causal;
  int32_t page_size, page_shift;
  int32_t num_seqs, num_rows, num_heads, num_kv_heads;
  int32_t group;                        // num_heads / num_kv_heads
  uint64_t group_mul;                   // division by it (plan_attention)
  int32_t max_seqlen_q, max_seqlen_k;
  const int32_t* indices;               // nullptr: whole prefix
  int32_t num_indices;
  float scale_log2;                     // |scale| * log2(e): scores in powers of two
  int32_t negate;                       // scale < 0: the product is of -q
  uint16_t* out;
  int64_t out_row_stride;
  float* lse;
  uint32_t* err;
  // work split (plan_attention)
  int32_t members;      // CTAs of a group: they share an item's keys and split its query rows
  int32_t chunk_groups; // row-chunk groups of one (request, K/V head)
  int32_t groups;       // CTA groups of the grid
  int32_t items;        // (request or row) x K/V head x chunk group
  int32_t two_queries;  // paged, at most 32 rows a CTA: two segments' queries are held
  int32_t whole_items;  // runs are whole items: no partial sums
  int32_t list_tiles;   // key tiles of an item with a selection (0: whole prefix)
  // workspace
  void* info;           // [groups] GroupInfo: the first item of each group's run
  float2* stats;        // [groups][2][members][64]: reference maximum and sum of a partial row
  float* partial;       // [groups][2][members][64][dv]: its unnormalised output
};

// 128-byte-swizzled tensor maps {64 values, (K/V head, offset), piece of 64
// values, page}: boxes of 64 keys of one page and kBoxPieces pieces.
struct AttnMaps {
  CUtensorMap k, v;
};
constexpr int kLatentBoxPieces = 3, kPagedBoxPieces = 2;

constexpr int kChunkRows = 64;  // query rows ((row, head) pairs) of one CTA

// Rows copied into a paged cache by slot: up to two sources, each a run of
// `units` 16-byte pieces per (token, head).
struct StoreRowsPart {
  const uint16_t* src;   // (token, head) at src + token*token_stride + head*head_stride (elements)
  int64_t token_stride, head_stride;
  uint16_t* dst;         // (page, head, offset) at dst + page*page_stride + head*dst_head_stride + offset*dst_row
  int64_t dst_head_stride;
  int32_t dst_row;       // elements
  int32_t units;         // 16-byte pieces per (token, head)
};
struct StoreRowsParams {
  StoreRowsPart part[2];
  const int32_t* slots;
  int32_t num_tokens, heads;
  int32_t page_size, page_shift;
  int64_t num_pages, page_stride;
  uint32_t per_token;  // 16-byte pieces of a token (launch_store_rows)
  int32_t slice;       // tokens between a thread's tokens
  uint32_t* err;
};

struct TablesParams {
  const int32_t* cached_len;
  const int32_t* new_len;
  int32_t num_reqs, num_rows;
  int32_t page_size, page_shift;
  int64_t num_pages;
  const int32_t* free_pages;
  int32_t num_free;
  int32_t* block_table;
  int64_t table_stride;
  int32_t* cu_seqlens_q;
  int32_t* cu_seqlens_k;
  int32_t* visible_len;
  int32_t* slots;
  int32_t* pages_taken;
  int32_t reqs_per_cta;
  int32_t shares;       // parts of a request's first rows (launch_tables)
  uint32_t* err;
};

// SM count and error word of the current device (api.cu).
fp4idx_status_t call_device(int* sms, uint32_t** err);
// Tensor map of 16-bit elements, innermost box of 64 (128 bytes, 128-byte
// swizzle), zeros outside (api.cu).  strides in bytes.
fp4idx_status_t call_tensor_map16(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                                  const cuuint64_t* strides, const cuuint32_t* box);

// Fills the work split of p; false if it does not fit the counters.
bool plan_attention(AttnParams* p, int sms);
size_t attention_workspace(const AttnParams& p);
cudaError_t launch_attention(AttnParams p, const AttnMaps& maps, int dtype, void* workspace, cudaStream_t stream);
cudaError_t launch_store_rows(StoreRowsParams p, int sms, cudaStream_t stream);
cudaError_t launch_tables(TablesParams p, int sms, cudaStream_t stream);

#ifdef __CUDACC__
// ---------------------------------------------------------------- device helpers
// Request of row t: the last b with cu_seqlens_q[b] <= t (num_seqs >= 1).
__device__ __forceinline__ int attn_request(const AttnParams& p, int t) {
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu_seqlens_q + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// Positions row t of request b sees: [0, the result).  A row behind the last
// request's (a selection's item; attn_request gives it that request) sees none.
__device__ __forceinline__ int attn_visible(const AttnParams& p, int b, int t) {
  const int end = p.indices ? __ldg(p.cu_seqlens_q + b + 1) : INT32_MAX;
  const int k_len = min(max(0, __ldg(p.cu_seqlens_k + b + 1) - __ldg(p.cu_seqlens_k + b)), p.max_seqlen_k);
  int64_t vis = k_len;
  if (p.visible_len) {
    vis = __ldg(p.visible_len + t);
  } else if (p.causal) {
    const int q0 = __ldg(p.cu_seqlens_q + b), q_len = __ldg(p.cu_seqlens_q + b + 1) - q0;
    const int64_t off = p.qo_offset ? static_cast<int64_t>(__ldg(p.qo_offset + b))
                                    : static_cast<int64_t>(k_len) - q_len;
    vis = static_cast<int64_t>(t - q0) + off + 1;
  }
  vis = vis < 0 || t >= end ? 0 : vis;
  return static_cast<int>(vis > k_len ? k_len : vis);
}
__device__ __forceinline__ int64_t attn_table_base(const AttnParams& p, int b) {
  return p.page_offsets ? static_cast<int64_t>(__ldg(p.page_offsets + b)) : static_cast<int64_t>(b) * p.table_stride;
}
#endif

}  // namespace fp4idx
