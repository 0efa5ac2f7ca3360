// attention.cu -- attention over the 16-bit paged caches (fp4idx_latent_attention,
// fp4idx_paged_attention): one CTA per (row, head), one key per thread for the
// scores and one or four output dimensions per thread for the weighted sum, with a
// running maximum and sum over tiles of 128 keys.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "ptx.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 128;

template <int DTYPE>
__device__ __forceinline__ float to_float(uint16_t w) {
  if constexpr (DTYPE == FP4IDX_BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
  return __half2float(__ushort_as_half(w));
}
template <int DTYPE>
__device__ __forceinline__ uint16_t from_float(float x) {
  if constexpr (DTYPE == FP4IDX_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return __half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < kThreads / 32; ++i) r = is_max ? fmaxf(r, red[i]) : r + red[i];
  return r;
}

template <int DTYPE, bool LATENT>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttnParams p) {
  constexpr int DK = LATENT ? kLatentDim + kRopeDim : kPagedDim;
  constexpr int DV = LATENT ? kLatentDim : kPagedDim;
  __shared__ float q[DK];
  __shared__ float weight[kThreads];
  __shared__ int64_t row_at[kThreads];
  __shared__ float red[kThreads / 32];
  const int t = blockIdx.x, h = blockIdx.y, hk = h / p.group, tid = threadIdx.x;
  const int b = attn_request(p, t);
  const int vis = attn_visible(p, b, t);
  const int64_t base = attn_table_base(p, b);
  for (int d = tid; d < DK; d += kThreads)
    q[d] = to_float<DTYPE>(p.q[t * p.q_row_stride + h * p.q_head_stride + d]);
  __syncthreads();
  int64_t n = vis;
  const int32_t* list = nullptr;
  if (p.indices) {
    n = static_cast<int64_t>(p.num_indices) * (LATENT ? 1 : kSelectBlock);
    list = p.indices + (LATENT ? static_cast<int64_t>(t) : static_cast<int64_t>(hk) * p.num_rows + t) * p.num_indices;
  }
  float m = -INFINITY, l = 0.0f, acc[DV / kThreads] = {};
  for (int64_t j0 = 0; j0 < n; j0 += kThreads) {
    const int64_t j = j0 + tid;
    int64_t pos = -1;
    if (j < n) pos = !list ? j : LATENT ? __ldg(list + j) : static_cast<int64_t>(__ldg(list + j / kSelectBlock)) * kSelectBlock + j % kSelectBlock;
    int64_t at = -1;
    if (pos >= 0 && pos < vis) {
      const int64_t page = __ldg(p.block_table + base + (pos >> p.page_shift));
      if (page >= 0 && page < p.num_pages)
        at = page * p.page_stride +
             (static_cast<int64_t>(LATENT ? 0 : hk) * p.page_size + (pos & (p.page_size - 1))) * DK;
      else
        atomicOr(p.err, kErrPageRange);
    }
    float s = -INFINITY;
    if (at >= 0) {
      s = 0.0f;
      for (int d = 0; d < DK; ++d) s = fmaf(q[d], to_float<DTYPE>(p.k[at + d]), s);
      s *= p.scale_log2;
    }
    const float top = fmaxf(m, block_reduce(s, true, red));
    const float ref = top == -INFINITY ? 0.0f : top;
    const float w = exp2f(s - ref), keep = exp2f(m - ref);
    l = l * keep + block_reduce(w, false, red);
    m = top;
    weight[tid] = w;
    row_at[tid] = at;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < DV / kThreads; ++i) acc[i] *= keep;
    for (int u = 0; u < kThreads; ++u) {
      if (row_at[u] < 0) continue;
      const uint16_t* row = (LATENT ? p.k : p.v) + row_at[u];
#pragma unroll
      for (int i = 0; i < DV / kThreads; ++i) acc[i] = fmaf(weight[u], to_float<DTYPE>(row[i * kThreads + tid]), acc[i]);
    }
    __syncthreads();
  }
  const float inv = l > 0.0f ? 1.0f / l : l;  // no keys: 0; NaN stays
  for (int i = 0; i < DV / kThreads; ++i)
    p.out[t * p.out_row_stride + static_cast<int64_t>(h) * DV + i * kThreads + tid] = from_float<DTYPE>(l == 0.0f ? 0.0f : acc[i] * inv);
  if (p.lse && tid == 0)
    p.lse[static_cast<int64_t>(t) * p.num_heads + h] = (m + log2f(l)) * 0.693147180559945309f;
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, int dtype, cudaStream_t stream) {
  const dim3 grid(p.num_rows, p.num_heads);
  const bool latent = p.v == nullptr;
  if (dtype == FP4IDX_BF16)
    latent ? attention_kernel<FP4IDX_BF16, true><<<grid, kThreads, 0, stream>>>(p)
           : attention_kernel<FP4IDX_BF16, false><<<grid, kThreads, 0, stream>>>(p);
  else
    latent ? attention_kernel<FP4IDX_FP16, true><<<grid, kThreads, 0, stream>>>(p)
           : attention_kernel<FP4IDX_FP16, false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fp4idx
