// store_rows.cu -- writers of the 16-bit paged caches: rows copied by slot
// (fp4idx_store_latent: a token's latent and rotary values into one cache
// row; fp4idx_store_kv: K and V rows of every KV head).
//
// One thread per 16-byte piece of one (token, head) row, pieces of a row in
// consecutive threads, so both sides are coalesced.  Nothing is computed:
// bound by memory for many tokens, by the launch for few.
#include <cstring>

#include "attention.h"
#include "ptx.cuh"

namespace fp4idx {
namespace {

constexpr int kStoreThreads = 256;

__global__ void __launch_bounds__(kStoreThreads) store_rows_kernel(const StoreRowsParams p) {
  pdl_wait();  // tokens and slots may come from the kernel before this one
  pdl_launch_dependents();
  const uint32_t u0 = p.part[0].units, units = u0 + p.part[1].units;
  const uint32_t per_token = units * p.heads;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x;
  const int64_t tok = i / per_token;
  if (tok >= p.num_tokens) return;
  const uint32_t rest = static_cast<uint32_t>(i - tok * per_token);
  const uint32_t head = rest / units;
  uint32_t unit = rest - head * units;
  const int32_t slot = __ldg(p.slots + tok);
  if (slot < 0) return;
  const int64_t page = slot >> p.page_shift;
  if (page >= p.num_pages) {
    if (rest == 0) atomicOr(p.err, kErrPageRange);
    return;
  }
  const StoreRowsPart& w = unit < u0 ? p.part[0] : p.part[1];
  if (unit >= u0) unit -= u0;
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(w.src + tok * w.token_stride + head * w.head_stride) + unit);
  uint16_t* row = w.dst + page * p.page_stride + head * w.dst_head_stride +
                  static_cast<int64_t>(slot & (p.page_size - 1)) * w.dst_row;
  reinterpret_cast<uint4*>(row)[unit] = v;
}

}  // namespace

cudaError_t launch_store_rows(const StoreRowsParams& p, cudaStream_t stream) {
  const int64_t pieces = static_cast<int64_t>(p.num_tokens) * p.heads * (p.part[0].units + p.part[1].units);
  if (pieces == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>((pieces + kStoreThreads - 1) / kStoreThreads));
  cfg.blockDim = dim3(kStoreThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, store_rows_kernel, p);
}

}  // namespace fp4idx
