// build_tables.cu -- metadata of one step from its request lengths
// (fp4idx_build_tables): prefix sums of rows and keys, the new pages of every
// request entered in the block table, and each row's slot and visible length.
//
// One launch and no workspace: a CTA owns `reqs_per_cta` consecutive
// requests and first sums the three running counts (rows, keys, new pages)
// of every request before its own -- a coalesced read of two words a
// request, L2-resident after the first CTA -- instead of waiting for another
// CTA's prefix; then it scans its own requests.  A warp writes up to 256 rows
// of a request, and blockIdx.y splits the rows of each by their mean.  What a
// request has beyond that (one long prompt among decodes) is written by all
// warps of all its CTAs, some of which may be there for it alone and return at
// once where no request is that long.  The page of a new row is computed from
// the free list, not read back from the table, so no CTA waits for another's
// writes.  Bound by the launch and a chain of three dependent loads.  Per call
// in a graph of such calls: 2.5 us for 64 requests of one row, 4.3 for 2,048
// requests of 0 to 255 rows, 12.1 for 2,047 of one row and one of 32,768 (141
// when one warp wrote a request's rows).
#include <cstring>

#include "attention.h"
#include "ptx.cuh"

namespace fp4idx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxReqs = 1024;  // requests of one CTA (shared memory)
constexpr int kWarpRows = 256;  // rows that a warp writes at a time (at most five pages)

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
  __shared__ bool any_long;                     // one of its requests has more than `most` rows
  pdl_wait();  // the lengths may come from the kernel before this one
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int b0 = blockIdx.x * p.reqs_per_cta;
  const int nb = min(p.reqs_per_cta, p.num_reqs - b0);
  bool bad = false;
  // CTAs beyond the shares are there for the rows of requests of more than `most`
  const int shares = p.shares, y = blockIdx.y, most = shares * kWarpRows;
  if (y >= shares) {
    bool more = false;
    for (int i = tid; i < nb; i += kThreads) more |= __ldg(p.new_len + b0 + i) > most;
    if (!__syncthreads_or(more)) return;
  }
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
    bool more = false;
    rows = keys = pages = 0;
    for (int w = 0; w < kWarps; ++w) {
      rows += part[0][w];
      keys += part[1][w];
      pages += part[2][w];
    }
    for (int i0 = 0; i0 < nb; i0 += 32) {
      ReqCounts r = {0, 0, 0, 0};
      if (i0 + lane < nb) r = req_counts(p, b0 + i0 + lane, &bad);
      more |= r.fresh > most;
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
    more = __any_sync(0xffffffffu, more);
    if (lane == 0) {
      any_long = more;
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
  if (b0 + nb == p.num_reqs && y < shares) {
    for (int64_t t = first_row[nb] + y * kThreads + tid; t < p.num_rows; t += shares * kThreads) {
      p.visible_len[t] = 0;
      p.slots[t] = -1;
    }
  }
  bool range = false;
  // New pages from, from + step, ... of request b0 + i, below logical page `end`.
  const auto write_entries = [&](int i, const ReqCounts& r, int from, int end, int step) {
    int32_t* entries = p.block_table + static_cast<int64_t>(b0 + i) * p.table_stride;
    for (int64_t j = r.has + from; j < end && j < p.table_stride; j += step) {
      const int64_t f = first_page[i] + (j - r.has);
      entries[j] = f < p.num_free ? __ldg(p.free_pages + f) : -1;
    }
  };
  // Rows [from, end) of request b0 + i by one warp, kWarpRows at a time and then
  // `step` rows on.  A lane looks up one of the pages that these lie in.  (32
  // bits: tokens held and rows are below 2^31 each, steps far below.)
  const auto write_rows = [&](int i, const ReqCounts& r, uint32_t from, uint32_t end, uint32_t step) {
    const int32_t* entries = p.block_table + static_cast<int64_t>(b0 + i) * p.table_stride;
    const int64_t page0 = first_page[i] - r.has;  // logical page j gets free page page0 + j
    const int64_t left = p.num_free - first_page[i], t0 = first_row[i], room = p.num_rows - t0;
    const uint32_t has = r.has, need = r.need;
    // the first `known` pages have an entry to come from: held, or in the free list, and inside the row
    uint32_t known = left >= need - has ? need : has + static_cast<uint32_t>(left > 0 ? left : 0);
    if (known > p.table_stride) known = static_cast<uint32_t>(p.table_stride);
    if (end > room) end = static_cast<uint32_t>(room > 0 ? room : 0);
    for (; from < end; from += step) {
      const uint32_t first = (static_cast<uint32_t>(r.cached) + from) >> p.page_shift, j = first + lane;
      int32_t page = -1;
      if (j < known) page = j < has ? entries[j] : __ldg(p.free_pages + page0 + j);
      const bool in = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_pages);
      const int32_t slot0 = in ? page * p.page_size : -1;
      const uint32_t stop = min(end, from + kWarpRows);
      range |= !in && j < known && j <= ((static_cast<uint32_t>(r.cached) + stop - 1) >> p.page_shift);
#pragma unroll 4
      for (uint32_t n0 = from; n0 < stop; n0 += 32) {
        const uint32_t n = n0 + lane, pos = static_cast<uint32_t>(r.cached) + n;
        const int32_t base = __shfl_sync(0xffffffffu, slot0, (pos >> p.page_shift) - first);
        if (n < stop) {
          p.visible_len[t0 + n] = static_cast<int32_t>(min(pos + 1, static_cast<uint32_t>(INT32_MAX)));
          p.slots[t0 + n] = base < 0 ? -1 : base + static_cast<int32_t>(pos & (p.page_size - 1));
        }
      }
    }
  };
  for (int i = y < shares ? wid : nb; i < nb; i += kWarps) {  // a warp per request
    const ReqCounts r = req_counts(p, b0 + i, &bad);
    bad |= r.fresh > 0 && r.need > p.table_stride;
    write_entries(i, r, y * 32 + lane, min(r.need, r.has + most / 32), shares * 32);
    write_rows(i, r, y * kWarpRows, min(r.fresh, most), shares * kWarpRows);
  }
  if (any_long) {  // what long requests have beyond that, by every warp
    for (int i = 0; i < nb; ++i) {
      const ReqCounts r = req_counts(p, b0 + i, &bad);
      if (r.fresh <= most) continue;
      write_entries(i, r, most / 32 + y * kThreads + tid, r.need, gridDim.y * kThreads);
      write_rows(i, r, most + (y * kWarps + wid) * kWarpRows, r.fresh, gridDim.y * kWarps * kWarpRows);
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
  // rows split so that a warp writes about 256 rows of an even split
  const int64_t even = (static_cast<int64_t>(p.num_rows) + p.num_reqs - 1) / p.num_reqs;
  const int64_t shares = (even + kWarpRows - 1) / kWarpRows;
  p.shares = static_cast<int32_t>(shares < 1 ? 1 : (shares > 64 ? 64 : shares));
  // and, in case one request has most of them, so that each of its warps writes
  // about 1,024, as long as the CTAs stay few: with more than two a SM the next
  // kernel's no longer find room beside them (6,000 requests of two rows 5.8 us,
  // 7.7 with a second CTA per eight requests).
  const int64_t alone = (static_cast<int64_t>(p.num_rows) + 4 * kWarps * kWarpRows - 1) / (4 * kWarps * kWarpRows);
  const int64_t room = 2 * sms / ctas;
  int64_t split = alone < room ? alone : room;
  split = split < p.shares ? p.shares : (split > 64 ? 64 : split);
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
