// pages.cu -- page operations of requests that share pages
// (fp4idx_fork_requests, fp4idx_copy_pages, fp4idx_release_pages,
// fp4idx_compact_pages).
//
// Which pages are in use is not counted anywhere: it is the set that the held
// table entries name, found by marking a bitmap.  With u(p) = 1 for a page in
// use and rank(p) = sum of u below p, a free page is entry p - rank(p) of the
// free list, and with n pages in use a page p >= n that is in use is move
// n - 1 - rank(p), the free page p < n the target of move p - rank(p).
#include <algorithm>
#include <cstring>

#include "ptx.cuh"
#include "shared.h"

namespace fp4idx {
namespace {

template <class... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- fork
constexpr int kForkThreads = 256, kForkWarps = kForkThreads / 32;

struct Fork {
  int32_t parent, child, len, full;
  bool valid, part, range;  // inside the table and its row; ends inside a page; a number past the table
};
__device__ __forceinline__ Fork fork_of(const ForkParams& p, int i) {
  Fork f;
  f.parent = __ldg(p.parent + i);
  f.child = __ldg(p.child + i);
  f.valid = f.parent >= 0 && f.child >= 0;
  f.range = f.valid && (f.parent >= p.num_reqs || f.child >= p.num_reqs);
  f.valid = f.valid && !f.range;
  f.len = f.valid ? max(0, p.cached_len[f.parent]) : 0;
  if (p.fork_len && f.valid) f.len = min(f.len, max(0, __ldg(p.fork_len + i)));
  f.full = f.len >> p.page_shift;
  f.part = (f.len & (p.page_size - 1)) != 0;
  return f;
}

// A warp writes a fork's table row.  Every CTA first passes over all forks, a
// thread each: it counts the unfinished pages of the ones before its own and
// looks for one that names an own child.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const ForkParams p) {
  __shared__ int32_t child[kForkWarps];
  __shared__ int bad[kForkWarps];
  __shared__ int part_sum[kForkWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int i0 = blockIdx.x * kForkWarps, i = i0 + wid;
  Fork f = {};
  if (i < p.num_forks) f = fork_of(p, i);
  const bool fits = f.full + f.part <= p.table_stride;
  if (lane == 0) {
    child[wid] = i < p.num_forks && f.valid ? f.child : -1;
    bad[wid] = 0;
  }
  __syncthreads();
  int32_t mine[kForkWarps];
#pragma unroll
  for (int k = 0; k < kForkWarps; ++k) mine[k] = child[k];
  int parts = 0;  // unfinished pages of forks before i0
  const bool last = i0 + kForkWarps >= p.num_forks;
  for (int j = tid; j < p.num_forks; j += kForkThreads) {
    const int32_t from = __ldg(p.parent + j), to = __ldg(p.child + j);
    const bool valid = from >= 0 && to >= 0 && from < p.num_reqs && to < p.num_reqs;
    if (!valid) continue;
#pragma unroll
    for (int k = 0; k < kForkWarps; ++k)
      if (from == mine[k] || (to == mine[k] && j < i0 + k)) bad[k] = 1;
    if (j < i0) {
      const Fork g = fork_of(p, j);
      parts += g.part && g.full + 1 <= p.table_stride;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) parts += __shfl_xor_sync(0xffffffffu, parts, o);
  if (lane == 0) part_sum[wid] = parts;
  __syncthreads();
  parts = 0;
#pragma unroll
  for (int w = 0; w < kForkWarps; ++w) parts += part_sum[w];
  __syncthreads();
  const bool takes = f.valid && fits && f.part;
  if (lane == 0) part_sum[wid] = takes;
  __syncthreads();
  int before = parts, all = parts;
#pragma unroll
  for (int w = 0; w < kForkWarps; ++w) {
    if (w < wid) before += part_sum[w];
    all += part_sum[w];
  }
  if (last && tid == 0) p.pages_taken[0] = min(all, p.num_free);
  if (i >= p.num_forks) return;
  int32_t src = -1, dst = -1;
  uint32_t err = f.range ? kErrRequests : 0;
  if (f.valid && !fits) err |= kErrLengths;
  if (f.valid && bad[wid]) err |= kErrRequests;
  if (f.valid && fits && !bad[wid]) {
    const int32_t* from = p.block_table + static_cast<int64_t>(f.parent) * p.table_stride;
    int32_t* to = p.block_table + static_cast<int64_t>(f.child) * p.table_stride;
    for (int j = lane; j < f.full; j += 32) to[j] = from[j];
    if (f.part) {
      if (before < p.num_free) dst = __ldg(p.free_pages + before);
      else err |= kErrLengths;
      if (lane == 0) to[f.full] = dst;
      src = from[f.full];
      if (src < 0 || src >= p.num_pages) {
        err |= kErrPageRange;
        src = -1;
      }
      if (src < 0 || dst < 0) src = dst = -1;
    }
    if (lane == 0) p.cached_len[f.child] = f.len;
  }
  if (lane == 0) {
    p.copy_src[i] = src;
    p.copy_dst[i] = dst;
    if (err) atomicOr(p.err, err);
  }
}

// ---------------------------------------------------------------- copy
// A warp copies a piece of one page of one span: up to 4 KB, eight 16-byte
// loads a lane before the first store.
constexpr int kCopyThreads = 256, kCopyWarps = kCopyThreads / 32;
constexpr int kCopyLoads = 8, kPieceUnits = 32 * kCopyLoads;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n = p.count ? min(max(0, __ldg(p.count)), p.num_copies) : p.num_copies;
  const int64_t work = static_cast<int64_t>(n) * p.pieces;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); w < work;
       w += static_cast<int64_t>(gridDim.x) * kCopyWarps) {
    const int i = static_cast<int>(w / p.pieces), piece = static_cast<int>(w - static_cast<int64_t>(i) * p.pieces);
    const int32_t from = __ldg(p.src + i), to = __ldg(p.dst + i);
    if (from < 0 || to < 0) continue;
    if (from >= p.num_pages || to >= p.num_pages) {
      if (piece == 0 && lane == 0) atomicOr(p.err, kErrPageRange);
      continue;
    }
    int s = 0, hi = p.num_spans - 1;
    while (s < hi) {
      const int mid = (s + hi + 1) >> 1;
      if (p.span[mid].first_piece <= piece) s = mid; else hi = mid - 1;
    }
    const CopyParams::Span& span = p.span[s];
    const int u0 = (piece - span.first_piece) * kPieceUnits + lane;
    const uint4* src = span.base + from * span.page_stride;
    uint4* dst = span.base + to * span.page_stride;
    uint4 v[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
      if (u0 + 32 * k < span.units) v[k] = src[u0 + 32 * k];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
      if (u0 + 32 * k < span.units) dst[u0 + 32 * k] = v[k];
  }
}

// ---------------------------------------------------------------- pool
constexpr int kPoolThreads = 256, kPoolWarps = kPoolThreads / 32;

__device__ __forceinline__ int pool_words(const PoolParams& p) { return static_cast<int>((p.num_pages + 31) >> 5); }
// Held entries of request b inside its row.
__device__ __forceinline__ int held_entries(const PoolParams& p, int b, bool* past) {
  const int len = max(0, p.cached_len[b]);
  const int64_t held = (static_cast<int64_t>(len) + (1 << p.page_shift) - 1) >> p.page_shift;
  *past |= held > p.width;
  return static_cast<int>(min(held, static_cast<int64_t>(p.width)));
}

__global__ void __launch_bounds__(kPoolThreads) pool_start_kernel(const PoolParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int at = blockIdx.x * kPoolThreads + threadIdx.x, step = gridDim.x * kPoolThreads;
  const int words = pool_words(p);
  for (int w = at; w < words; w += step) p.bitmap[w] = 0;
  for (int i = at; i < p.num_released; i += step) {
    const int32_t b = __ldg(p.requests + i);
    if (b < 0) continue;
    if (b >= p.num_reqs) {
      atomicOr(p.err, kErrRequests);
      continue;
    }
    atomicMin(p.cached_len + b, p.keep_len ? max(0, __ldg(p.keep_len + i)) : 0);
  }
}

// A warp marks up to 128 entries of a row.
__global__ void __launch_bounds__(kPoolThreads) pool_mark_kernel(const PoolParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  bool past = false, range = false;
  const int parts = (p.width + 127) / 128;
  const int64_t work = static_cast<int64_t>(p.num_reqs) * parts;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kPoolWarps + wid; w < work;
       w += static_cast<int64_t>(gridDim.x) * kPoolWarps) {
    const int b = static_cast<int>(w / parts), j0 = static_cast<int>(w - static_cast<int64_t>(b) * parts) * 128 + lane;
    const int n = held_entries(p, b, &past);
    const int32_t* row = p.block_table + b * p.table_stride;
    int32_t page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = j0 + 32 * k < n ? __ldg(row + j0 + 32 * k) : INT32_MIN;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (page[k] == INT32_MIN && j0 + 32 * k >= n) continue;
      if (page[k] < 0 || page[k] >= p.num_pages) range = true;
      else atomicOr(p.bitmap + (page[k] >> 5), 1u << (page[k] & 31));
    }
  }
  if (past) atomicOr(p.err, kErrLengths);
  if (range) atomicOr(p.err, kErrPageRange);
}

// Sum over the CTA of up to two counts; every thread gets them.
__device__ __forceinline__ int2 cta_sum(int2 v, int2* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int2 all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kPoolWarps; ++w) {
    all.x += part[w].x;
    all.y += part[w].y;
  }
  return all;
}

// The lists.  A CTA owns a run of words; it sums all words for the total and
// those before its own for its first rank.
template <bool COMPACT>
__global__ void __launch_bounds__(kPoolThreads) pool_list_kernel(const PoolParams p) {
  __shared__ int2 part[kPoolWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int words = pool_words(p);
  const int per = (words + gridDim.x - 1) / gridDim.x;
  const int w0 = min(words, static_cast<int>(blockIdx.x) * per), w1 = min(words, w0 + per);
  int2 sum = make_int2(0, 0);  // pages in use: all, before w0
  for (int w = tid; w < words; w += kPoolThreads) {
    const int c = __popc(p.bitmap[w]);
    sum.x += c;
    sum.y += w < w0 ? c : 0;
  }
  sum = cta_sum(sum, part);
  const int n = sum.x;
  int moves = 0, movers = 0;
  if (COMPACT) {
    int below = 0;  // pages in use below n
    for (int w = tid; w <= (n >> 5) && w < words; w += kPoolThreads) {
      const uint32_t bits = p.bitmap[w];
      below += __popc(w == (n >> 5) ? bits & ((1u << (n & 31)) - 1) : bits);
    }
    movers = n - cta_sum(make_int2(below, 0), part).x;
    moves = min(movers, p.max_moves);
  }
  int rank = sum.y;  // pages in use before this warp's words
  for (int base = w0; base < w1; base += kPoolThreads) {
    const int w = base + tid;
    const uint32_t bits = w < w1 ? p.bitmap[w] : 0;
    int incl = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) part[wid].x = incl;
    __syncthreads();
    int before = rank;
#pragma unroll
    for (int k = 0; k < kPoolWarps; ++k) {
      if (k < wid) before += part[k].x;
      rank += part[k].x;
    }
    before += incl - __popc(bits);
    if (COMPACT && w < w1) p.rank[w] = before;
    // a warp's 32 words, one at a time: lane = page of the word
    const int w_first = base + wid * 32;
    for (int k = 0; k < 32 && w_first + k < w1; ++k) {
      const uint32_t word = __shfl_sync(0xffffffffu, bits, k);
      const int upto = __shfl_sync(0xffffffffu, before, k) + __popc(word & ((1u << lane) - 1));
      const int64_t page = static_cast<int64_t>(w_first + k) * 32 + lane;
      const bool used = word >> lane & 1;
      if (page >= p.num_pages) continue;
      if (!COMPACT) {
        if (!used) p.free_pages[page - upto] = static_cast<int32_t>(page);
      } else if (used && page >= n) {
        const int m = n - 1 - upto;
        if (m < moves) p.copy_src[m] = static_cast<int32_t>(page);
        if (m == moves) p.extent[0] = static_cast<int32_t>(page) + 1;  // the highest one that stays
      } else if (!used && page < n && page - upto < moves) {
        p.copy_dst[page - upto] = static_cast<int32_t>(page);
      }
    }
  }
  // what lies behind the lists
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kPoolThreads + tid, step = static_cast<int64_t>(gridDim.x) * kPoolThreads;
  if (!COMPACT) {
    for (int64_t i = p.num_pages - n + at; i < p.num_pages; i += step) p.free_pages[i] = -1;
    if (at == 0) p.num_free[0] = static_cast<int32_t>(p.num_pages - n);
  } else {
    for (int64_t i = moves + at; i < p.max_moves; i += step) p.copy_src[i] = p.copy_dst[i] = -1;
    if (at == 0) {
      p.num_moves[0] = moves;
      if (moves == movers) p.extent[0] = n;
    }
  }
}

// Table rows with the moved pages' new places; n comes with the moves: the
// pages at or above n are the ones whose rank from the top is below `moves`.
__global__ void __launch_bounds__(kPoolThreads) pool_rewrite_kernel(const PoolParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int words = pool_words(p), moves = p.num_moves[0];
  const int n = p.rank[words - 1] + __popc(p.bitmap[words - 1]);
  const int parts = (p.width + 127) / 128;
  const int64_t work = static_cast<int64_t>(p.num_reqs) * parts;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kPoolWarps + wid; w < work;
       w += static_cast<int64_t>(gridDim.x) * kPoolWarps) {
    const int b = static_cast<int>(w / parts), j0 = static_cast<int>(w - static_cast<int64_t>(b) * parts) * 128 + lane;
    bool past = false;
    const int held = held_entries(p, b, &past);
    const int32_t* row = p.block_table + b * p.table_stride;
    int32_t* to = p.new_table + b * p.new_stride;
    int32_t page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = j0 + 32 * k < p.width ? row[j0 + 32 * k] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 32 * k;
      if (j >= p.width) continue;
      if (j < held && page[k] >= n && page[k] < p.num_pages) {
        const int word = page[k] >> 5;
        const int m = n - 1 - (p.rank[word] + __popc(p.bitmap[word] & ((1u << (page[k] & 31)) - 1)));
        if (m < moves) page[k] = p.copy_dst[m];
      }
      to[j] = page[k];
    }
  }
}

int64_t round16(int64_t n) { return (n + 15) & ~int64_t{15}; }

cudaError_t mark(PoolParams* p, int sms, void* workspace, cudaStream_t stream) {
  const int64_t words = (p->num_pages + 31) / 32;
  p->bitmap = static_cast<uint32_t*>(workspace);
  p->rank = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + round16(words * 4));
  const int64_t most = 8 * static_cast<int64_t>(sms);
  const int64_t first = std::max<int64_t>(1, (std::max<int64_t>(words, p->num_released) + kPoolThreads - 1) / kPoolThreads);
  cudaError_t e = launch_dependent(pool_start_kernel, dim3(static_cast<unsigned>(std::min(first, most))), kPoolThreads, stream, *p);
  if (e != cudaSuccess) return e;
  const int64_t parts = static_cast<int64_t>(p->num_reqs) * ((p->width + 127) / 128);
  const int64_t ctas = std::min(most, (parts + kPoolWarps - 1) / kPoolWarps);
  return launch_dependent(pool_mark_kernel, dim3(static_cast<unsigned>(ctas)), kPoolThreads, stream, *p);
}

unsigned list_ctas(const PoolParams& p, int sms) {
  const int64_t words = (p.num_pages + 31) / 32;
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(sms, words / 64)));
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const int ctas = std::max(1, (p.num_forks + kForkWarps - 1) / kForkWarps);
  return launch_dependent(fork_kernel, dim3(ctas), kForkThreads, stream, p);
}

cudaError_t launch_copy_pages(CopyParams p, int sms, cudaStream_t stream) {
  p.pieces = 0;
  for (int s = 0; s < p.num_spans; ++s) {
    p.span[s].first_piece = p.pieces;
    p.pieces += (p.span[s].units + kPieceUnits - 1) / kPieceUnits;
  }
  const int64_t work = static_cast<int64_t>(p.num_copies) * p.pieces;
  const int64_t ctas = std::min<int64_t>((work + kCopyWarps - 1) / kCopyWarps, 8 * static_cast<int64_t>(sms));
  return launch_dependent(copy_kernel, dim3(static_cast<unsigned>(ctas)), kCopyThreads, stream, p);
}

size_t pool_workspace(int64_t num_pages) {
  return static_cast<size_t>(2 * round16((num_pages + 31) / 32 * 4));
}

cudaError_t launch_release(PoolParams p, int sms, void* workspace, cudaStream_t stream) {
  cudaError_t e = mark(&p, sms, workspace, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(pool_list_kernel<false>, dim3(list_ctas(p, sms)), kPoolThreads, stream, p);
}

cudaError_t launch_compact(PoolParams p, int sms, void* workspace, cudaStream_t stream) {
  cudaError_t e = mark(&p, sms, workspace, stream);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(pool_list_kernel<true>, dim3(list_ctas(p, sms)), kPoolThreads, stream, p)) != cudaSuccess) return e;
  const int64_t parts = static_cast<int64_t>(p.num_reqs) * ((p.width + 127) / 128);
  const int64_t ctas = std::min<int64_t>(8 * sms, (parts + kPoolWarps - 1) / kPoolWarps);
  return launch_dependent(pool_rewrite_kernel, dim3(static_cast<unsigned>(ctas)), kPoolThreads, stream, p);
}

}  // namespace fp4idx
