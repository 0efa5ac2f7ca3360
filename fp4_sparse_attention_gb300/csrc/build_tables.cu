// build_tables.cu -- metadata of one step from its request lengths
// (fp4idx_build_tables): prefix sums of rows and keys, the new pages of every
// request entered in the block table, and each row's slot and visible length.
//
// One launch and no workspace: a CTA owns `reqs_per_cta` consecutive
// requests and first sums the three running counts (rows, keys, new pages)
// of every request before its own -- a coalesced read of two words a
// request, L2-resident after the first CTA -- instead of waiting for another
// CTA's prefix; then it scans its own requests.  blockIdx.y splits the rows
// of each request, so one long prompt does not sit in one CTA.  The page of
// a new row is computed from the free list, not read back from the table,
// so no CTA waits for another's writes.  Bound by the launch and a chain of
// three dependent loads: 4.2 us on the device for 64 requests of one row, 7.5
// for 2,048 requests of 0 to 255 rows.
#include <cstring>

#include "attention.h"
#include "ptx.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxReqs = 1024;  // requests of one CTA (shared memory)

struct ReqCounts {
  int32_t cached, fresh, has, need;  // tokens held, new rows, pages held, pages needed
};

__device__ __forceinline__ ReqCounts req_counts(const TablesParams& p, int b, bool* bad) {
  ReqCounts r;
  const int32_t c = __ldg(p.cached_len + b), n = __ldg(p.new_len + b);
  *bad |= (c | n) < 0;
  r.cached = max(c, 0);
  r.fresh = max(n, 0);
  const int64_t ps = p.page_size;
  r.has = static_cast<int32_t>((r.cached + ps - 1) >> p.page_shift);
  r.need = static_cast<int32_t>((static_cast<int64_t>(r.cached) + r.fresh + ps - 1) >> p.page_shift);
  return r;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Saturates: a sum past 2^31 - 1 is outside the contract, not undefined.
__device__ __forceinline__ int32_t sat32(int64_t v) { return v > INT32_MAX ? INT32_MAX : static_cast<int32_t>(v); }

__global__ void __launch_bounds__(kThreads) build_tables_kernel(const TablesParams p) {
  __shared__ int64_t part[3][kWarps];
  __shared__ int64_t first_row[kMaxReqs + 1];   // rows before each of this CTA's requests
  __shared__ int64_t first_page[kMaxReqs + 1];  // new pages before it
  pdl_wait();  // the lengths may come from the kernel before this one
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int b0 = blockIdx.x * p.reqs_per_cta;
  const int nb = min(p.reqs_per_cta, p.num_reqs - b0);
  bool bad = false;
  // counts of every request before b0
  int64_t rows = 0, keys = 0, pages = 0;
  for (int b = tid; b < b0; b += kThreads) {
    const ReqCounts r = req_counts(p, b, &bad);
    rows += r.fresh;
    keys += static_cast<int64_t>(r.cached) + r.fresh;
    pages += r.need - r.has;
  }
  rows = warp_sum(rows);
  keys = warp_sum(keys);
  pages = warp_sum(pages);
  if (lane == 0) {
    part[0][wid] = rows;
    part[1][wid] = keys;
    part[2][wid] = pages;
  }
  __syncthreads();
  // one warp scans this CTA's requests, 32 at a time
  if (wid == 0) {
    rows = keys = pages = 0;
    for (int w = 0; w < kWarps; ++w) {
      rows += part[0][w];
      keys += part[1][w];
      pages += part[2][w];
    }
    for (int i0 = 0; i0 < nb; i0 += 32) {
      ReqCounts r = {0, 0, 0, 0};
      if (i0 + lane < nb) r = req_counts(p, b0 + i0 + lane, &bad);
      int64_t a = r.fresh, k = static_cast<int64_t>(r.cached) + r.fresh, g = r.need - r.has;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t a1 = __shfl_up_sync(0xffffffffu, a, o), k1 = __shfl_up_sync(0xffffffffu, k, o),
                      g1 = __shfl_up_sync(0xffffffffu, g, o);
        if (lane >= o) {
          a += a1;
          k += k1;
          g += g1;
        }
      }
      if (i0 + lane < nb) {
        first_row[i0 + lane] = rows + a - r.fresh;
        first_page[i0 + lane] = pages + g - (r.need - r.has);
        if (blockIdx.y == 0) {
          p.cu_seqlens_q[b0 + i0 + lane + 1] = sat32(rows + a);
          p.cu_seqlens_k[b0 + i0 + lane + 1] = sat32(keys + k);
        }
      }
      rows += __shfl_sync(0xffffffffu, a, 31);
      keys += __shfl_sync(0xffffffffu, k, 31);
      pages += __shfl_sync(0xffffffffu, g, 31);
    }
    if (lane == 0) {
      first_row[nb] = rows;
      first_page[nb] = pages;
      if (blockIdx.y == 0 && b0 == 0) p.cu_seqlens_q[0] = p.cu_seqlens_k[0] = 0;
      if (blockIdx.y == 0 && b0 + nb == p.num_reqs) {
        p.pages_taken[0] = sat32(pages < p.num_free ? pages : p.num_free);
        bad |= rows > p.num_rows || pages > p.num_free;
      }
    }
  }
  __syncthreads();
  // rows past the requests' sum
  if (b0 + nb == p.num_reqs) {
    for (int64_t t = first_row[nb] + blockIdx.y * kThreads + tid; t < p.num_rows; t += gridDim.y * kThreads) {
      p.visible_len[t] = 0;
      p.slots[t] = -1;
    }
  }
  bool range = false;
  for (int i = wid; i < nb; i += kWarps) {  // a warp per request
    const int b = b0 + i;
    const ReqCounts r = req_counts(p, b, &bad);
    int32_t* row = p.block_table + static_cast<int64_t>(b) * p.table_stride;
    const int64_t page0 = first_page[i];
    if (blockIdx.y == 0) {
      for (int j = r.has + lane; j < r.need; j += 32) {
        const int64_t f = page0 + (j - r.has);
        if (j < p.table_stride) row[j] = f < p.num_free ? __ldg(p.free_pages + f) : -1; else bad = true;
      }
    }
    const int64_t t0 = first_row[i];
    for (int64_t n = blockIdx.y * 32 + lane; n < r.fresh; n += gridDim.y * 32) {
      if (t0 + n >= p.num_rows) break;
      const int64_t pos = r.cached + n;
      const int64_t j = pos >> p.page_shift;
      int32_t page = -1;
      if (j >= p.table_stride) {
        bad = true;
      } else if (j < r.has) {  // the last page held
        page = row[j];
        range |= page < 0 || page >= p.num_pages;
      } else {
        const int64_t f = page0 + (j - r.has);
        if (f < p.num_free) {
          page = __ldg(p.free_pages + f);
          range |= page < 0 || page >= p.num_pages;
        }
      }
      p.visible_len[t0 + n] = sat32(pos + 1);
      p.slots[t0 + n] = page < 0 || page >= p.num_pages
                            ? -1
                            : page * p.page_size + static_cast<int32_t>(pos & (p.page_size - 1));
    }
  }
  if (bad) atomicOr(p.err, kErrLengths);
  if (range) atomicOr(p.err, kErrPageRange);
}

}  // namespace

cudaError_t launch_tables(TablesParams p, int sms, cudaStream_t stream) {
  // Eight requests a CTA (one per warp) until four CTAs per SM; above that
  // the CTAs take more requests instead, since every CTA sums all requests
  // before its own.
  int per = (p.num_reqs + 4 * sms - 1) / (4 * sms);
  per = per < 8 ? 8 : (per + 7) / 8 * 8;
  p.reqs_per_cta = per > kMaxReqs ? kMaxReqs : per;
  const int ctas = (p.num_reqs + p.reqs_per_cta - 1) / p.reqs_per_cta;
  // rows split so that a CTA's warp writes about 256 rows of an even split
  const int64_t even = (static_cast<int64_t>(p.num_rows) + p.num_reqs - 1) / p.num_reqs;
  int64_t split = (even + 255) / 256;
  split = split < 1 ? 1 : (split > 64 ? 64 : split);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(split));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, build_tables_kernel, p);
}

}  // namespace fp4idx
