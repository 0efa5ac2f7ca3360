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
// looks for one that names an own child.  That is forks^2 / 8 reads from L2, but
// no second launch and no wait for another CTA: bound by latency, 4 forks 2.9 us
// on the device, 1,984 forks of up to 512 pages 5.7 us.
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
  constexpr int kBatch = 4;  // loads of so many forks under way
  for (int j0 = tid; j0 < p.num_forks; j0 += kBatch * kForkThreads) {
    int32_t from[kBatch], to[kBatch], len[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int j = j0 + x * kForkThreads;
      from[x] = j < p.num_forks ? __ldg(p.parent + j) : -1;
      to[x] = j < p.num_forks ? __ldg(p.child + j) : -1;
      len[x] = p.fork_len && j < i0 ? max(0, __ldg(p.fork_len + j)) : INT32_MAX;
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int j = j0 + x * kForkThreads;
      const bool valid = from[x] >= 0 && to[x] >= 0 && from[x] < p.num_reqs && to[x] < p.num_reqs;
      len[x] = valid && j < i0 ? min(len[x], max(0, p.cached_len[from[x]])) : 0;
      if (!valid) from[x] = to[x] = -2;
#pragma unroll
      for (int k = 0; k < kForkWarps; ++k)
        if (from[x] == mine[k] || (to[x] == mine[k] && j < i0 + k)) bad[k] = 1;
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) parts += (len[x] & (p.page_size - 1)) != 0 && (len[x] >> p.page_shift) < p.table_stride;
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
    for (int j = lane; j < f.full; j += 8 * 32) {
      int32_t page[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) page[k] = j + 32 * k < f.full ? from[j + 32 * k] : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (j + 32 * k < f.full) to[j + 32 * k] = page[k];
    }
    if (f.part) {
      if (before < p.num_free) dst = max(-1, __ldg(p.free_pages + before));
      if (dst < 0) {
        err |= kErrLengths;
      } else if (dst >= p.num_pages) {
        err |= kErrPageRange;
        dst = -1;
      }
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
// loads a lane before the first store, so that an SM has 256 KB under way.  Bound
// by HBM: 1,500 pages of four layers' latent and index caches, 937 MB, 145.7 us,
// 6.43 TB/s, 96 % of a plain copy; 8 pages of one layer 2.4 us on the device.
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

// ---------------------------------------------------------------- pool, any size
// One launch clears the bitmap (and cuts the released requests), one marks, one
// ranks and lists, and for a compaction one rewrites the table.  Bound by the
// launches' latency and the marks' atomics: 2,048 requests of up to 512 pages in
// a pool of 482,000 (4 MB) 12.4 us for a release, 21 us for a compaction in a
// pool of 682,000, on the device.
constexpr int kPoolThreads = 256, kPoolWarps = kPoolThreads / 32;
constexpr int kListThreads = 1024, kListWarps = kListThreads / 32;
constexpr int kEntries = 8;  // table entries that a lane has under way
// Runs of 32 x kEntries entries of a row, which may be as wide as 32 bits allow.
// (An entry's number then stays below 2^31, too: a run begins at a multiple of 256.)
__host__ __device__ constexpr int row_runs(int32_t width) {
  return static_cast<int>((static_cast<int64_t>(width) + 32 * kEntries - 1) / (32 * kEntries));
}

// Words of the bitmap, by fours.
__host__ __device__ constexpr int64_t pool_words(int64_t num_pages) { return (num_pages + 127) / 128 * 4; }
__device__ __forceinline__ int popc4(uint4 v) { return __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w); }
// Held entries of a row of `len` tokens, inside the row.
__device__ __forceinline__ int held_entries(const PoolParams& p, int len, uint32_t* err) {
  const int64_t held = (static_cast<int64_t>(max(0, len)) + (1 << p.page_shift) - 1) >> p.page_shift;
  if (held > p.width) *err |= kErrLengths;
  return static_cast<int>(min(held, static_cast<int64_t>(p.width)));
}
// Marks entries j0, j0 + 32, ... of a row.
__device__ __forceinline__ void mark_entries(const PoolParams& p, const int32_t* row, int j0, int n, uint32_t* bits, uint32_t* err) {
  int32_t page[kEntries];
#pragma unroll
  for (int x = 0; x < kEntries; ++x) page[x] = j0 + 32 * x < n ? row[j0 + 32 * x] : 0;
#pragma unroll
  for (int x = 0; x < kEntries; ++x) {
    if (j0 + 32 * x >= n) continue;
    if (page[x] < 0 || page[x] >= p.num_pages) *err |= kErrPageRange;
    else atomicOr(bits + (page[x] >> 5), 1u << (page[x] & 31));
  }
}
// Entries of a row at their pages' new places; rank(page) = pages in use before it.
template <class Rank>
__device__ __forceinline__ void move_entries(const PoolParams& p, const int32_t* row, int32_t* to, int j0, int held, int n, int moves,
                                             const Rank& rank) {
  int32_t page[kEntries], move[kEntries];
#pragma unroll
  for (int x = 0; x < kEntries; ++x) page[x] = j0 + 32 * x < p.width ? row[j0 + 32 * x] : -1;
#pragma unroll
  for (int x = 0; x < kEntries; ++x)
    move[x] = j0 + 32 * x < held && page[x] >= n && page[x] < p.num_pages ? n - 1 - rank(page[x]) : moves;
#pragma unroll
  for (int x = 0; x < kEntries; ++x)
    if (move[x] < moves) page[x] = __ldcg(p.copy_dst + move[x]);
#pragma unroll
  for (int x = 0; x < kEntries; ++x)
    if (j0 + 32 * x < p.width) to[j0 + 32 * x] = page[x];
}
// The lists' share of four words of the bitmap, a lane a page; `rank` pages are
// in use before them.
template <bool COMPACT>
__device__ __forceinline__ void list_words(const PoolParams& p, const uint32_t* bits, int group, int rank, int n, int moves) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t word = bits[4 * group + x];
    const int64_t page = (static_cast<int64_t>(4) * group + x) * 32 + lane;
    const int r = rank + __popc(word & ((1u << lane) - 1));
    rank += __popc(word);
    if (page >= p.num_pages) continue;
    const bool used = word >> lane & 1;
    if (!COMPACT) {
      if (!used) p.free_pages[page - r] = static_cast<int32_t>(page);
    } else if (used && page >= n) {
      const int m = n - 1 - r;
      if (m < moves) p.copy_src[m] = static_cast<int32_t>(page);
      if (m == moves) p.extent[0] = static_cast<int32_t>(page) + 1;  // the highest one that stays
    } else if (!used && page < n && page - r < moves) {
      p.copy_dst[page - r] = static_cast<int32_t>(page);
    }
  }
}
// What lies behind the lists, and the counts; at, step: this thread of all.
template <bool COMPACT>
__device__ __forceinline__ void end_lists(const PoolParams& p, int n, int moves, int movers, int64_t at, int64_t step) {
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

__global__ void __launch_bounds__(kPoolThreads) pool_start_kernel(const PoolParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int at = blockIdx.x * kPoolThreads + threadIdx.x, step = gridDim.x * kPoolThreads;
  const int groups = static_cast<int>(pool_words(p.num_pages) / 4);
  for (int g = at; g < groups; g += step) reinterpret_cast<uint4*>(p.bitmap)[g] = make_uint4(0, 0, 0, 0);
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

// A warp marks, or rewrites, up to 256 entries of a row.
__global__ void __launch_bounds__(kPoolThreads) pool_mark_kernel(const PoolParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t err = 0;
  const int parts = row_runs(p.width);
  const int64_t work = static_cast<int64_t>(p.num_reqs) * parts;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kPoolWarps + wid; w < work;
       w += static_cast<int64_t>(gridDim.x) * kPoolWarps) {
    const int b = static_cast<int>(w / parts), j0 = static_cast<int>(w - static_cast<int64_t>(b) * parts) * 32 * kEntries + lane;
    mark_entries(p, p.block_table + b * p.table_stride, j0, held_entries(p, p.cached_len[b], &err), p.bitmap, &err);
  }
  if (err) atomicOr(p.err, err);
}

// Sum of two counts over the CTA.
__device__ __forceinline__ int2 list_sum(int2 v, int2* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int2 all = part[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    all.x += __shfl_xor_sync(0xffffffffu, all.x, o);
    all.y += __shfl_xor_sync(0xffffffffu, all.y, o);
  }
  return all;
}

// The lists.  A CTA owns a run of words; it sums all words for the total and
// those before its own for its first rank.
template <bool COMPACT>
__global__ void __launch_bounds__(kListThreads) pool_list_kernel(const PoolParams p) {
  __shared__ int2 part[kListWarps];
  __shared__ int ranks[kListThreads];
  static_assert(kListWarps == 32, "a lane a warp");
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int groups = static_cast<int>(pool_words(p.num_pages) / 4);
  const int per = (groups + gridDim.x - 1) / gridDim.x;
  const int g0 = min(groups, static_cast<int>(blockIdx.x) * per), g1 = min(groups, g0 + per);
  const uint4* fours = reinterpret_cast<const uint4*>(p.bitmap);
  int2 sum = make_int2(0, 0);  // pages in use: all, before g0
#pragma unroll 4
  for (int g = tid; g < groups; g += kListThreads) {
    const int c = popc4(fours[g]);
    sum.x += c;
    sum.y += g < g0 ? c : 0;
  }
  sum = list_sum(sum, part);
  const int n = sum.x;
  int moves = 0, movers = 0;
  if (COMPACT) {
    int below = 0;  // pages in use below n
#pragma unroll 4
    for (int w = tid; w < (n >> 5); w += kListThreads) below += __popc(p.bitmap[w]);
    if (tid == 0 && (n & 31)) below += __popc(p.bitmap[n >> 5] & ((1u << (n & 31)) - 1));
    movers = n - list_sum(make_int2(below, 0), part).x;
    moves = min(movers, p.max_moves);
  }
  int rank = sum.y;  // pages in use before the next groups
  for (int base = g0; base < g1; base += kListThreads) {
    const int g = base + tid, mine = g < g1 ? popc4(fours[g]) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) part[wid].x = incl;
    __syncthreads();
    int before = part[lane].x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    const int all = __shfl_sync(0xffffffffu, before, 31);
    before = wid > 0 ? __shfl_sync(0xffffffffu, before, wid - 1) : 0;
    ranks[tid] = rank + before + incl - mine;
    if (COMPACT && g < g1) p.rank[g] = ranks[tid];
    __syncthreads();
    for (int x = wid; x < kListThreads && base + x < g1; x += kListWarps) list_words<COMPACT>(p, p.bitmap, base + x, ranks[x], n, moves);
    rank += all;
  }
  end_lists<COMPACT>(p, n, moves, movers, static_cast<int64_t>(blockIdx.x) * kListThreads + tid, static_cast<int64_t>(gridDim.x) * kListThreads);
}

// Table rows with the moved pages' new places; n comes with the moves: the
// pages at or above n are the ones whose rank from the top is below `moves`.
__global__ void __launch_bounds__(kPoolThreads) pool_rewrite_kernel(const PoolParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int groups = static_cast<int>(pool_words(p.num_pages) / 4), moves = p.num_moves[0];
  const uint4* fours = reinterpret_cast<const uint4*>(p.bitmap);
  const int n = p.rank[groups - 1] + popc4(fours[groups - 1]);
  const auto rank = [&](int page) {
    const int w = page >> 5, x = w & 3;
    const uint4 v = fours[w >> 2];
    const uint32_t mine = x == 0 ? v.x : x == 1 ? v.y : x == 2 ? v.z : v.w;
    return p.rank[w >> 2] + (x > 0 ? __popc(v.x) : 0) + (x > 1 ? __popc(v.y) : 0) + (x > 2 ? __popc(v.z) : 0) +
           __popc(mine & ((1u << (page & 31)) - 1));
  };
  uint32_t err = 0;  // (the marks have reported it)
  const int parts = row_runs(p.width);
  const int64_t work = static_cast<int64_t>(p.num_reqs) * parts;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kPoolWarps + wid; w < work;
       w += static_cast<int64_t>(gridDim.x) * kPoolWarps) {
    const int b = static_cast<int>(w / parts), j0 = static_cast<int>(w - static_cast<int64_t>(b) * parts) * 32 * kEntries + lane;
    move_entries(p, p.block_table + b * p.table_stride, p.new_table + b * p.new_stride, j0, held_entries(p, p.cached_len[b], &err), n, moves, rank);
  }
}

// ---------------------------------------------------------------- pool, one cluster
// The same in one launch, for small pools: a cluster of CTAs marks its requests'
// entries, each in a bitmap of its own in shared memory; CTA r ORs everyone's
// slice r and hands it to everyone; then each CTA has the whole bitmap, ranks
// it, lists its slice and rewrites its requests' rows.  No workspace, nothing to
// clear in memory, two or three cluster barriers.  64 requests of up to 256 pages
// 4.9 us for a release; 32 of up to 16 pages 6.2 us for a compaction, on the
// device: latency.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;
// What one cluster takes: more is faster on all SMs, in more launches.  (256
// requests of up to 256 pages: release 7.1 us, 8.0 in three launches; compaction
// 15 us, 17 in four.  256 of up to 512: 8.7, 8.4; 17, 16.)
constexpr int kClusterPages = 1 << 17;
constexpr int kClusterRuns = 512;  // runs of 256 entries of a row
constexpr int kClusterCtas = 8;    // (four: 5.6 and 11.8 us for 64 requests of up to 256 pages, eight 5.3 and 10.1)

struct ClusterSmem {
  int2 part[kClusterWarps];
};
static_assert(sizeof(ClusterSmem) % 16 == 0, "the bitmap behind it is read by 16 bytes");
// bitmap, pages in use before each four words of it, lengths of the CTA's requests
size_t cluster_smem(int64_t num_pages, int reqs_of_cta) {
  return sizeof(ClusterSmem) + static_cast<size_t>(pool_words(num_pages)) * 5 + 4 * static_cast<size_t>(reqs_of_cta);
}
__device__ __forceinline__ uint4 dsmem_ld_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void dsmem_st_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <bool COMPACT>
__global__ void __launch_bounds__(kClusterThreads, 1) pool_cluster_kernel(const PoolParams p) {
  constexpr int ctas = kClusterCtas;
  extern __shared__ __align__(16) uint8_t raw[];
  ClusterSmem& sm = *reinterpret_cast<ClusterSmem*>(raw);
  const int words = static_cast<int>(pool_words(p.num_pages)), groups = words / 4;
  uint32_t* bits = reinterpret_cast<uint32_t*>(raw + sizeof(ClusterSmem));
  uint32_t* ranks = bits + words;
  int32_t* len = reinterpret_cast<int32_t*>(ranks + groups);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int me = blockIdx.x;  // one cluster: the rank
  const int reqs = (p.num_reqs - me + ctas - 1) / ctas;  // requests me, me + ctas, ...
  for (int g = tid; g < groups; g += kClusterThreads) reinterpret_cast<uint4*>(bits)[g] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_launch_dependents();
  uint32_t err = 0;
  // lengths, cut where a request is released
  for (int k = tid; k < reqs; k += kClusterThreads) len[k] = p.cached_len[me + k * ctas];
  __syncthreads();
  for (int i = tid; i < p.num_released; i += kClusterThreads) {
    const int32_t b = __ldg(p.requests + i);
    if (b >= p.num_reqs) err |= kErrRequests;
    else if (b >= 0 && b % ctas == me) atomicMin(len + b / ctas, p.keep_len ? max(0, __ldg(p.keep_len + i)) : 0);
  }
  __syncthreads();
  if (p.num_released > 0)
    for (int k = tid; k < reqs; k += kClusterThreads) p.cached_len[me + k * ctas] = len[k];
  // marks: a warp takes up to 256 entries of a row
  const int parts = row_runs(p.width);
  for (int w = wid; w < reqs * parts; w += kClusterWarps) {
    const int k = w / parts, j0 = (w - k * parts) * 32 * kEntries + lane;
    mark_entries(p, p.block_table + static_cast<int64_t>(me + k * ctas) * p.table_stride, j0, held_entries(p, len[k], &err), bits, &err);
  }
  __syncwarp();
  cluster_sync();
  // everyone's slice of mine, to everyone
  const int slice = (groups + ctas - 1) / ctas, g0 = min(groups, me * slice), g1 = min(groups, g0 + slice);
  for (int g = g0 + tid; g < g1; g += kClusterThreads) {
    uint4 v = make_uint4(0, 0, 0, 0);
    for (int c = 0; c < ctas; ++c) {
      const uint4 x = dsmem_ld_v4(dsmem_addr(bits + 4 * g, c));
      v = make_uint4(v.x | x.x, v.y | x.y, v.z | x.z, v.w | x.w);
    }
    for (int c = 0; c < ctas; ++c) dsmem_st_v4(dsmem_addr(bits + 4 * g, c), v);
  }
  __syncwarp();
  cluster_sync();
  // ranks of all groups of four words: a thread has a run of them
  int n = 0;
  {
    const int per = (groups + kClusterThreads - 1) / kClusterThreads, first = min(groups, tid * per), last = min(groups, first + per);
    int mine = 0;
    for (int g = first; g < last; ++g) {
      mine += popc4(reinterpret_cast<const uint4*>(bits)[g]);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.part[wid].x = incl;
    __syncthreads();
    if (wid == 0) {
      int all = sm.part[lane].x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += y;
      }
      sm.part[lane].y = all;
    }
    __syncthreads();
    n = sm.part[kClusterWarps - 1].y;
    int before = incl - mine + (wid > 0 ? sm.part[wid - 1].y : 0);
    for (int g = first; g < last; ++g) {
      ranks[g] = before;
      before += popc4(reinterpret_cast<const uint4*>(bits)[g]);
    }
    __syncthreads();
  }
  const auto rank_of = [&](int64_t page) {  // pages in use before it
    const int w = static_cast<int>(page >> 5), g = w >> 2;
    int r = ranks[g];
    for (int x = 4 * g; x < w; ++x) r += __popc(bits[x]);
    return r + __popc(bits[w] & ((1u << (page & 31)) - 1));
  };
  const int below = n < p.num_pages ? rank_of(n) : n, movers = n - below, moves = COMPACT ? min(movers, p.max_moves) : 0;
  for (int g = g0 + wid; g < g1; g += kClusterWarps) list_words<COMPACT>(p, bits, g, ranks[g], n, moves);
  end_lists<COMPACT>(p, n, moves, movers, static_cast<int64_t>(me) * kClusterThreads + tid, static_cast<int64_t>(ctas) * kClusterThreads);
  if (COMPACT) {
    __syncwarp();
    cluster_sync();  // the targets are written
    for (int w = wid; w < reqs * parts; w += kClusterWarps) {
      const int k = w / parts, j0 = (w - k * parts) * 32 * kEntries + lane;
      const int64_t b = me + static_cast<int64_t>(k) * ctas;
      move_entries(p, p.block_table + b * p.table_stride, p.new_table + b * p.new_stride, j0, held_entries(p, len[k], &err), n, moves, rank_of);
    }
  }
  if (err) atomicOr(p.err, err);
}

bool in_one_cluster(const PoolParams& p) {
  return p.num_pages <= kClusterPages && static_cast<int64_t>(p.num_reqs) * row_runs(p.width) <= kClusterRuns;
}

template <bool COMPACT>
cudaError_t launch_cluster(const PoolParams& p, cudaStream_t stream) {
  constexpr int ctas = kClusterCtas;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = cluster_smem(p.num_pages, (p.num_reqs + ctas - 1) / ctas);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pool_cluster_kernel<COMPACT>, p);
}

int64_t round16(int64_t n) { return (n + 15) & ~int64_t{15}; }

unsigned entry_ctas(const PoolParams& p, int sms) {
  const int64_t parts = static_cast<int64_t>(p.num_reqs) * row_runs(p.width);
  return static_cast<unsigned>(std::min<int64_t>(8 * static_cast<int64_t>(sms), (parts + kPoolWarps - 1) / kPoolWarps));
}

cudaError_t mark(PoolParams* p, int sms, void* workspace, cudaStream_t stream) {
  const int64_t words = pool_words(p->num_pages);
  p->bitmap = static_cast<uint32_t*>(workspace);
  p->rank = reinterpret_cast<int32_t*>(p->bitmap + words);
  const int64_t most = 8 * static_cast<int64_t>(sms);
  const int64_t first = std::max<int64_t>(1, (std::max<int64_t>(words / 4, p->num_released) + kPoolThreads - 1) / kPoolThreads);
  cudaError_t e = launch_dependent(pool_start_kernel, dim3(static_cast<unsigned>(std::min(first, most))), kPoolThreads, stream, *p);
  if (e != cudaSuccess) return e;
  return launch_dependent(pool_mark_kernel, dim3(entry_ctas(*p, sms)), kPoolThreads, stream, *p);
}

// A CTA sums the whole bitmap: one for each 64 groups of four words at most.
unsigned list_ctas(const PoolParams& p, int sms) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(sms, pool_words(p.num_pages) / 4 / 64)));
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

size_t pool_workspace(int64_t num_pages, int32_t num_reqs, int64_t table_stride) {
  PoolParams p = {};
  p.num_pages = num_pages;
  p.num_reqs = num_reqs;
  p.width = static_cast<int32_t>(std::min<int64_t>(table_stride, INT32_MAX));
  return in_one_cluster(p) ? 0 : static_cast<size_t>(round16(5 * pool_words(num_pages)));
}

cudaError_t launch_release(PoolParams p, int sms, void* workspace, cudaStream_t stream) {
  if (in_one_cluster(p)) return launch_cluster<false>(p, stream);
  cudaError_t e = mark(&p, sms, workspace, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(pool_list_kernel<false>, dim3(list_ctas(p, sms)), kListThreads, stream, p);
}

cudaError_t launch_compact(PoolParams p, int sms, void* workspace, cudaStream_t stream) {
  if (in_one_cluster(p)) return launch_cluster<true>(p, stream);
  cudaError_t e = mark(&p, sms, workspace, stream);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(pool_list_kernel<true>, dim3(list_ctas(p, sms)), kListThreads, stream, p)) != cudaSuccess) return e;
  return launch_dependent(pool_rewrite_kernel, dim3(entry_ctas(p, sms)), kPoolThreads, stream, p);
}

}  // namespace fp4idx
