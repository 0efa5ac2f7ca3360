// store_rows.cu -- writers of the 16-bit paged caches: rows copied by slot
// (fp4idx_store_latent: a token's latent and rotary values into one cache
// row; fp4idx_store_kv: K and V rows of every KV head).
//
// A thread owns one 16-byte piece of the (token, head) rows and takes it of
// kTokens tokens, all loads before the first store; the pieces of a row are in
// consecutive threads, so both sides are coalesced.  Nothing is computed:
// bound by memory for many tokens (32,768 tokens of K and V, 4 heads: 21.6 us,
// 6.2 TB/s read and written, 91 % of a copy), by the launch for few (64 latent
// rows: 6.0 us with the call).
#include <cstring>

#include "attention.h"
#include "ptx.cuh"

namespace fp4idx {
namespace {

constexpr int kStoreThreads = 256;

template <int kTokens>
__global__ void __launch_bounds__(kStoreThreads) store_rows_kernel(const StoreRowsParams p) {
  pdl_wait();  // tokens and slots may come from the kernel before this one
  pdl_launch_dependents();
  const uint32_t u0 = p.part[0].units, units = u0 + p.part[1].units;
  const uint32_t i = blockIdx.x * kStoreThreads + threadIdx.x;  // piece of one token of the first slice
  const uint32_t tok0 = i / p.per_token;
  if (tok0 >= static_cast<uint32_t>(p.slice)) return;
  const uint32_t rest = i - tok0 * p.per_token;
  const uint32_t head = rest / units;
  uint32_t unit = rest - head * units;
  const StoreRowsPart& w = unit < u0 ? p.part[0] : p.part[1];
  if (unit >= u0) unit -= u0;
  const uint16_t* src = w.src + head * w.head_stride + unit * 8;
  uint16_t* dst = w.dst + head * w.dst_head_stride + unit * 8;
  // tokens tok0, tok0 + slice, ...
  int32_t slot[kTokens];
  uint4 v[kTokens];
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    const int64_t tok = tok0 + static_cast<int64_t>(n) * p.slice;
    slot[n] = tok < p.num_tokens ? __ldg(p.slots + tok) : -1;
    if (tok < p.num_tokens) v[n] = __ldg(reinterpret_cast<const uint4*>(src + tok * w.token_stride));
  }
#pragma unroll
  for (int n = 0; n < kTokens; ++n) {
    if (slot[n] < 0) continue;
    const int64_t page = slot[n] >> p.page_shift;
    if (page >= p.num_pages) {
      if (rest == 0) atomicOr(p.err, kErrPageRange);
      continue;
    }
    *reinterpret_cast<uint4*>(dst + page * p.page_stride + static_cast<int64_t>(slot[n] & (p.page_size - 1)) * w.dst_row) = v[n];
  }
}

template <int kTokens>
cudaError_t launch(StoreRowsParams p, cudaStream_t stream) {
  p.slice = (p.num_tokens + kTokens - 1) / kTokens;
  const int64_t threads = static_cast<int64_t>(p.slice) * p.per_token;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>((threads + kStoreThreads - 1) / kStoreThreads));
  cfg.blockDim = dim3(kStoreThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, store_rows_kernel<kTokens>, p);
}

}  // namespace

cudaError_t launch_store_rows(StoreRowsParams p, int sms, cudaStream_t stream) {
  p.per_token = static_cast<uint32_t>(p.heads) * (p.part[0].units + p.part[1].units);
  if (p.num_tokens == 0) return cudaSuccess;
  // Four pieces a thread once they fill the GPU several times over: 32,768 tokens
  // of K and V take 21.5 us so and 28.7 with one piece a thread; fewer tokens
  // need the threads.
  const int64_t pieces = static_cast<int64_t>(p.num_tokens) * p.per_token;
  return pieces >= static_cast<int64_t>(sms) * 2048 * 8 ? launch<4>(p, stream) : launch<1>(p, stream);
}

}  // namespace fp4idx
