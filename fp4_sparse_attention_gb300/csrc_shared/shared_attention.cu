// shared_attention.cu -- grouped-query attention of requests that share a
// prefix (fp4idx_shared_prefix_attention).
//
//   s(r, j) = scale * q[r] . k[j],   out[r] = sum_j exp(s - lse) v[j]
//
// The simplest form: a CTA takes a row and a K/V head, a warp the heads of that
// group in turn; a lane holds four of the 128 dimensions and the keys are
// walked with a running maximum and sum, all in fp32.
#include <cstring>

#include "attn_ptx.cuh"
#include "shared.h"

namespace fp4idx {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

template <int DTYPE>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (DTYPE == FP4IDX_BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  float2 r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}\n" : "=f"(r.x), "=f"(r.y) : "r"(v));
  return r;
}
template <int DTYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (DTYPE == FP4IDX_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads) shared_kernel(const __grid_constant__ SharedParams sp) {
  pdl_wait();
  pdl_launch_dependents();
  const AttnParams& p = sp.a;
  const int t = blockIdx.x, hk = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = attn_request(p, t);
  // the request's group: the last one that starts at or before it
  int g = 0, hi = sp.num_groups - 1;
  while (g < hi) {
    const int mid = (g + hi + 1) >> 1;
    if (__ldg(sp.group_offsets + mid) <= b) g = mid; else hi = mid - 1;
  }
  const int first = max(0, __ldg(sp.group_offsets + g));
  const bool in = first <= b && b < __ldg(sp.group_offsets + g + 1) && t < __ldg(p.cu_seqlens_q + b + 1);
  int vis = 0, prefix = 0;
  if (in) {
    vis = attn_visible(p, b, t);
    const int k_len = __ldg(p.cu_seqlens_k + first + 1) - __ldg(p.cu_seqlens_k + first);
    prefix = max(0, min(__ldg(sp.prefix_len + g), min(k_len, p.max_seqlen_k)));
  }
  const int64_t own = in ? attn_table_base(p, b) : 0, shared = in ? attn_table_base(p, first) : 0;
  for (int i = warp; i < p.group; i += kWarps) {
    const int h = hk * p.group + i;
    const uint2 qv = *reinterpret_cast<const uint2*>(p.q + t * p.q_row_stride + h * p.q_head_stride + lane * 4);
    const float2 q0 = unpack2<DTYPE>(qv.x), q1 = unpack2<DTYPE>(qv.y);
    const float sign = p.negate ? -p.scale_log2 : p.scale_log2;
    float m = -INFINITY, l = 0.0f, o[4] = {};
    for (int j = 0; j < vis; ++j) {
      const int page = __ldg(p.block_table + (j < prefix ? shared : own) + (j >> p.page_shift));
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.err, kErrPageRange);
        continue;
      }
      const int64_t at = page * p.page_stride + (static_cast<int64_t>(hk) * p.page_size + (j & (p.page_size - 1))) * kPagedDim + lane * 4;
      const uint2 kv = __ldg(reinterpret_cast<const uint2*>(p.k + at)), vv = __ldg(reinterpret_cast<const uint2*>(p.v + at));
      const float2 k0 = unpack2<DTYPE>(kv.x), k1 = unpack2<DTYPE>(kv.y), v0 = unpack2<DTYPE>(vv.x), v1 = unpack2<DTYPE>(vv.y);
      float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= sign;
      const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.0f : top, keep = ex2(m - ref), w = ex2(s - ref);
      m = top;
      l = l * keep + w;
      o[0] = o[0] * keep + w * v0.x;
      o[1] = o[1] * keep + w * v0.y;
      o[2] = o[2] * keep + w * v1.x;
      o[3] = o[3] * keep + w * v1.y;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(p.out + t * p.out_row_stride + h * kPagedDim + lane * 4) =
        make_uint2(pack2<DTYPE>(o[0] * inv, o[1] * inv), pack2<DTYPE>(o[2] * inv, o[3] * inv));
    if (p.lse && lane == 0)
      p.lse[static_cast<int64_t>(t) * p.num_heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
  }
}

}  // namespace

bool plan_shared(SharedParams*, int) { return true; }
size_t shared_workspace(const SharedParams&) { return 16; }

cudaError_t launch_shared(SharedParams p, const AttnMaps&, int dtype, void*, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(p.a.num_rows, p.a.num_kv_heads);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return dtype == FP4IDX_BF16 ? cudaLaunchKernelEx(&cfg, shared_kernel<FP4IDX_BF16>, p)
                              : cudaLaunchKernelEx(&cfg, shared_kernel<FP4IDX_FP16>, p);
}

}  // namespace fp4idx
