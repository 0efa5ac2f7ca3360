// shared.h -- parameters shared by the host layer (api_shared.cu) and the
// kernels of requests that share a prefix.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "fp4idx.h"

namespace fp4idx {

constexpr uint32_t kErrRequests = 0x10u;  // FP4IDX_ERR_REQUESTS

struct ForkParams {
  const int32_t* parent;
  const int32_t* child;
  const int32_t* fork_len;  // or nullptr
  int32_t num_forks, num_reqs;
  int32_t page_size, page_shift;
  int64_t num_pages;
  const int32_t* free_pages;
  int32_t num_free;
  int32_t* cached_len;
  int32_t* block_table;
  int64_t table_stride;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* pages_taken;
  uint32_t* err;
};

constexpr int kMaxSpans = 256;
struct CopyParams {
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;  // or nullptr
  int32_t num_copies;
  int32_t num_spans;
  int64_t num_pages;
  int32_t pieces;         // of a page of all spans (launch_copy_pages)
  uint32_t* err;
  struct Span {
    uint4* base;
    int64_t page_stride;  // 16-byte units, as below
    int32_t units;        // of a page
    int32_t first_piece;
  } span[kMaxSpans];
};

// Pages in use, marked in a bitmap from the held table entries.
struct PoolParams {
  const int32_t* requests;   // release: requests cut to keep_len
  const int32_t* keep_len;
  int32_t num_released;
  int32_t num_reqs;
  int32_t page_shift;
  int64_t num_pages;
  int32_t* cached_len;       // written by a release only
  const int32_t* block_table;
  int64_t table_stride;
  int32_t width;             // entries of a row
  uint32_t* bitmap;          // workspace: a bit per page, in whole words
  int32_t* rank;             // workspace: pages in use before each four words
  // release
  int32_t* free_pages;
  int32_t* num_free;
  // compaction
  int32_t* new_table;
  int64_t new_stride;
  int32_t max_moves;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* num_moves;
  int32_t* extent;
  uint32_t* err;
};

// Attention of groups of requests that share a prefix.
struct SharedParams {
  AttnParams a;                  // its work split is not used
  const int32_t* group_offsets;
  const int32_t* prefix_len;
  int32_t num_groups;
  int32_t max_group_rows;
  // work split (plan_shared)
  int32_t blocks_per_group;
  int32_t ctas;
};

// The caches as {64 values, (K/V head, offset), piece of 64 values, page}: boxes of
// 64 keys of one page, a piece of the keys and both of the values, and of 16 keys,
// a piece of the values.
struct SharedMaps {
  CUtensorMap k, v, v_part;
};

// Fills the work split; false if it does not fit the counters.
bool plan_shared(SharedParams* p, int sms);
size_t shared_workspace(const SharedParams& p);
cudaError_t launch_shared(SharedParams p, const SharedMaps& maps, int dtype, void* workspace, cudaStream_t stream);

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream);
cudaError_t launch_copy_pages(CopyParams p, int sms, cudaStream_t stream);
size_t pool_workspace(int64_t num_pages, int32_t num_reqs, int64_t table_stride);  // 0: none needed
cudaError_t launch_release(PoolParams p, int sms, void* workspace, cudaStream_t stream);
cudaError_t launch_compact(PoolParams p, int sms, void* workspace, cudaStream_t stream);

}  // namespace fp4idx
