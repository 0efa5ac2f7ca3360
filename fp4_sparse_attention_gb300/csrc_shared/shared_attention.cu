// shared_attention.cu -- grouped-query attention of requests that share a
// prefix (fp4idx_shared_prefix_attention) for sm_103a.
//
//   s(r, j) = scale * q[r] . k[j],   out[r] = sum_j exp(s - lse) v[j]
//
// A group's (row, head) pairs of one K/V head are taken 256 at a time: a block.
// Its keys are what each of its requests has behind the prefix, then the
// prefix itself, once, for all of its rows: one list of 128-key tiles.  The
// tiles of all blocks and K/V heads are concatenated and cut into equal runs,
// one per CTA; a block cut by a boundary leaves partial sums that join_kernel
// adds in a fixed order.
//
// A CTA holds two score accumulators, two outputs (128 rows x 128 columns each,
// all 512 TMEM columns) and a ring of five 32 KB stages, each a tile's keys or
// its values:
//
//   S [128 rows x 128 keys] = Q K^T      tcgen05, Q and K in shared memory
//   P = 2^(S - m)                        registers; 16 bits, over S's columns in TMEM
//   O [128 rows x 128]     += P V        tcgen05, P in TMEM, V in shared memory
//
// While one accumulator's rows go through the softmax, the tensor pipe works
// on the other's: with more than 128 pairs the two hold the block's halves and
// share each tile; with fewer they hold the same rows and take tiles in turn,
// and the end adds them up.  A softmax thread owns a row, so it needs no other
// thread's maximum, sum or factor.
//
// Roles: warps 0-3 and 4-7 softmax of the two accumulators, queries and output;
// warp 8 MMA issuer; warp 9 loader (TMA; 16-byte copies, which can leave zeros
// where a value may be anything, for the values of a run that ends inside);
// warp 10 planner, which looks up the tiles' pages ahead of all of them.
#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstring>

#include "attn_ptx.cuh"
#include "shared.h"

namespace fp4idx {
namespace {

constexpr int kTile = 128;                 // keys of a tile: two runs of 64, each inside one page
constexpr int kRows = 128;                 // rows of an accumulator
constexpr int kBlockPairs = 2 * kRows;
constexpr int kSoftmaxWarps = 4;           // of one accumulator
constexpr int kMmaWarp = 8, kLoadWarp = 9, kPlanWarp = 10;
constexpr int kThreads = 352;
constexpr int kStages = 5;
constexpr uint32_t kStage = 32768, kPiece = 128 * 128, kRun = 64 * 128;
constexpr uint32_t kQBytes = 2 * kPiece;   // 128 rows x 128 values
constexpr int kDescs = 16;                 // tiles that the planner may be ahead
constexpr uint32_t kTmemCols = 512, kOCol = 256;
constexpr int kGroupShift = 40;            // pair / group as (pair * ceil(2^40 / group)) >> 40 (attention.cu)
// A row's reference maximum is raised only when the true one is 2^8 above it, and
// in fp16 lies another 2^7 lower, so that shares down to 2^-32 are kept
// (attention.cu has the same two).
constexpr float kRaise = 8.0f;
template <int DTYPE>
constexpr float kBelow = DTYPE == FP4IDX_FP16 ? 7.0f : 0.0f;

// ---------------------------------------------------------------- plan
struct Block {
  int32_t row0;        // the group's first row
  int32_t pair0;       // the block's first pair of the group's
  int32_t pairs;
  int32_t tiles;
  int32_t span0, spans;
  int32_t pad[2];
};
// Keys [lo, hi) of one table row for the pairs [p0, p1) of a block: tiles from
// position pos0 (a multiple of 64, at most 63 below lo) on.
struct Span {
  int32_t req, pos0, lo, hi;
  int32_t start, tiles;  // tiles of the block before it; its own
  int32_t p0, p1;
};
// The first block of a CTA's run (for the join).
struct RunInfo {
  int32_t item, start, total;  // K/V head * blocks + block; first tile of it; tiles of all
  int32_t row0, pair0, pairs, hk, pad;
};

struct Plan {
  SharedParams sp;
  int32_t blocks;          // of one K/V head: num_groups x blocks_per_group
  int32_t blocks_per_group;
  int32_t ctas;
  Block* block;
  int32_t* block_tiles;
  Span* span;
  int32_t* row_vis;        // positions that each row sees
  RunInfo* info;
  float2* stats;           // [ctas][2][256] reference maximum and sum of a partial row
  float4* partial;         // [ctas][2][32][256]: its unnormalised output, four columns at a time
};

__device__ __forceinline__ int group_div(const AttnParams& p, int64_t x) {
  return static_cast<int>((static_cast<uint64_t>(x) * p.group_mul) >> kGroupShift);
}

// Requests [first, second) of a group.
__device__ __forceinline__ int2 group_requests(const SharedParams& sp, int g) {
  const int lo = min(max(__ldg(sp.group_offsets + g), 0), sp.a.num_seqs);
  return make_int2(lo, min(max(__ldg(sp.group_offsets + g + 1), lo), sp.a.num_seqs));
}

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;

// A warp plans a block: its spans, its tiles and what its rows see.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ Plan pl) {
  pdl_wait();
  pdl_launch_dependents();
  const SharedParams& sp = pl.sp;
  const AttnParams& p = sp.a;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (i >= pl.blocks) return;
  const int g = i / pl.blocks_per_group;
  const int2 reqs = group_requests(sp, g);
  Block blk = {};
  blk.row0 = max(0, __ldg(p.cu_seqlens_q + reqs.x));
  const int rows = min(max(min(__ldg(p.cu_seqlens_q + reqs.y), p.num_rows) - blk.row0, 0), sp.max_group_rows);
  const int64_t pair0 = static_cast<int64_t>(i - g * pl.blocks_per_group) * kBlockPairs;
  const int64_t pairs = min(static_cast<int64_t>(rows) * p.group - pair0, static_cast<int64_t>(kBlockPairs));
  if (pairs <= 0) {
    if (lane == 0) pl.block_tiles[i] = 0;
    return;
  }
  blk.pair0 = static_cast<int>(pair0);
  blk.pairs = static_cast<int>(pairs);
  const int r0 = blk.row0 + group_div(p, pair0), r1 = blk.row0 + group_div(p, pair0 + pairs - 1) + 1;  // its rows
  // the requests of its first and last row
  const auto request_of = [&](int t) {
    int lo = reqs.x, hi = reqs.y - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.cu_seqlens_q + mid) <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  const int a0 = request_of(r0), a1 = request_of(r1 - 1);
  const auto key_count = [&](int a) {
    return min(max(0, __ldg(p.cu_seqlens_k + a + 1) - __ldg(p.cu_seqlens_k + a)), p.max_seqlen_k);
  };
  const int prefix = max(0, min(__ldg(sp.prefix_len + g), key_count(reqs.x)));
  // (a block has 1 + its requests spans at most, and the next block's first
  // request is not before this one's last)
  blk.span0 = 2 * i + a0;
  Span* spans = pl.span + blk.span0;
  int top = 0;
  const auto add = [&](bool have, const Span& s) {
    const uint32_t some = __ballot_sync(0xffffffffu, have);
    int incl = have ? s.tiles : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (have) {
      Span w = s;
      w.start = blk.tiles + incl - s.tiles;
      spans[blk.spans + __popc(some & ((1u << lane) - 1))] = w;
    }
    blk.spans += __popc(some);
    blk.tiles += __shfl_sync(0xffffffffu, incl, 31);
  };
  for (int base = a0; base <= a1; base += 32) {
    const int a = base + lane;
    int from = 0, to = 0, k_len = 0, hi = 0;  // its rows of the block, its keys, the most that a row sees
    int64_t off = 0;                          // causal: row t sees t + off
    if (a <= a1) {
      const int q0 = __ldg(p.cu_seqlens_q + a), q1 = __ldg(p.cu_seqlens_q + a + 1);
      from = max(q0, r0);
      to = min(q1, r1);
      k_len = key_count(a);
      off = (p.qo_offset ? static_cast<int64_t>(__ldg(p.qo_offset + a)) : static_cast<int64_t>(k_len) - (q1 - q0)) + 1 - q0;
    }
    const auto sees = [&](int t, int n, int64_t o) {
      int64_t v = n;
      if (p.visible_len) v = __ldg(p.visible_len + t);
      else if (p.causal) v = t + o;
      return static_cast<int>(v < 0 ? 0 : v > n ? n : v);
    };
    if (a1 - base < 8) {  // few requests: all lanes on the rows of one
      for (int x = 0; x <= a1 - base; ++x) {
        const int f = __shfl_sync(0xffffffffu, from, x), e = __shfl_sync(0xffffffffu, to, x), n = __shfl_sync(0xffffffffu, k_len, x);
        const int64_t o = __shfl_sync(0xffffffffu, off, x);
        int most = 0;
        for (int t = f + lane; t < e; t += 32) {
          const int v = sees(t, n, o);
          pl.row_vis[t] = v;
          most = max(most, v);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == x) hi = most;
      }
    } else {
      for (int t = from; t < to; ++t) {
        const int v = sees(t, k_len, off);
        pl.row_vis[t] = v;
        hi = max(hi, v);
      }
    }
    top = max(top, hi);
    Span s;
    s.req = a;
    s.lo = prefix;
    s.pos0 = prefix & ~63;
    s.hi = hi;
    s.tiles = (hi - s.pos0 + kTile - 1) / kTile;
    s.p0 = static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(from - blk.row0) * p.group - pair0));
    s.p1 = static_cast<int>(min(pairs, static_cast<int64_t>(to - blk.row0) * p.group - pair0));
    add(from < to && hi > prefix, s);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  Span s = {};
  s.req = reqs.x;
  s.hi = min(prefix, top);
  s.tiles = (s.hi + kTile - 1) / kTile;
  if (s.tiles == 0 && blk.tiles == 0) s.tiles = 1;  // rows without keys are written, too
  s.p1 = blk.pairs;
  add(lane == 0 && s.tiles > 0, s);
  if (lane == 0) {
    pl.block[i] = blk;
    pl.block_tiles[i] = blk.tiles;
  }
}

// ---------------------------------------------------------------- main kernel
enum : int32_t { kSlot0 = 1, kSlot1 = 2, kFirst = 4, kLast = 8, kEnd = 16, kTail = 32, kTwo = 64, kWhole = 128 };

// One tile, and with its first one what a segment (a run of one block's tiles) is.
struct Desc {
  int32_t flags;
  int32_t page[2];       // of its runs; -1: no keys
  int32_t pos0, lo, hi;  // position of its first key; keys that count
  int32_t p0, p1;        // pairs of the block that they count for
  int32_t row0, pair0, pairs, hk;
  int32_t part;          // slot of its partial sums
  int32_t pad[3];
};

struct Control {
  uint64_t dfull[kDescs], dempty[kDescs];
  uint64_t kfull[kStages], kempty[kStages];
  uint64_t sfull[2], pfull[2], odone[2], ofree[2], qfull[2];
  uint64_t qfree, mfull, drain;
  Desc desc[kDescs];
  float2 other[kRows];   // the second accumulator's maximum and sum, when both hold the same rows
  int32_t warp_sum[kThreads / 32];
  int32_t run_hk, run_block, run_start, run_lo, run_hi, per_head;
  uint32_t tmem;
  int abort;
};
constexpr uint32_t kOff_Q = kStages * kStage, kOff_Ctl = kOff_Q + 2 * kQBytes;
constexpr uint32_t kSmem = kOff_Ctl + sizeof(Control);
static_assert(kSmem <= 232448, "227 KB per CTA");

__device__ __forceinline__ int run_begin(int total, int cta, int used) {
  return static_cast<int>(static_cast<int64_t>(total) * cta / used);
}
__device__ __forceinline__ int used_ctas(int total, int ctas) { return min(total, ctas); }

template <int DTYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (DTYPE == FP4IDX_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}
// Arrival on `bar` once this thread's copies so far have landed; it counts
// itself as one more pending arrival first.
__device__ __forceinline__ void cp_async_arrive_extra(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Rows that no group holds: zeros and -inf, a (row, head) pair of a CTA at a time.
__device__ __forceinline__ void clear_other_rows(const SharedParams& sp, int lane) {
  const AttnParams& p = sp.a;
  const int first = min(max(0, __ldg(p.cu_seqlens_q + group_requests(sp, 0).x)), p.num_rows);
  const int last = min(max(first, __ldg(p.cu_seqlens_q + group_requests(sp, sp.num_groups - 1).y)), p.num_rows);
  const int64_t rows = first + (p.num_rows - last), pairs = rows * p.num_heads;
#pragma unroll 1
  for (int64_t x = blockIdx.x; x < pairs; x += gridDim.x) {
    const int n = static_cast<int>(x / p.num_heads), h = static_cast<int>(x - static_cast<int64_t>(n) * p.num_heads);
    const int t = n < first ? n : n - first + last;
    uint2* out = reinterpret_cast<uint2*>(p.out + t * p.out_row_stride + static_cast<int64_t>(h) * kPagedDim);
    out[lane] = make_uint2(0, 0);
    if (p.lse && lane == 0) p.lse[static_cast<int64_t>(t) * p.num_heads + h] = -INFINITY;
  }
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 1) shared_kernel(const __grid_constant__ Plan pl, const __grid_constant__ AttnMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control& ctl = *reinterpret_cast<Control*>(smem + kOff_Ctl);
  const SharedParams& sp = pl.sp;
  const AttnParams& p = sp.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem);
  volatile int* abort_flag = &ctl.abort;

  if (base & 1023u) {  // the swizzled layouts need it; the runtime places the window there
    if (tid == 0) {
      pl.info[blockIdx.x].total = 0;
      atomicOr(p.err, kErrTimeout);
    }
    return;
  }
  if (tid == 0) {
    for (int k = 0; k < kDescs; ++k) {
      mbar_init(smem_u32(&ctl.dfull[k]), 1);
      mbar_init(smem_u32(&ctl.dempty[k]), 2 * kSoftmaxWarps + 2);
    }
    for (int k = 0; k < kStages; ++k) {
      mbar_init(smem_u32(&ctl.kfull[k]), 1);
      mbar_init(smem_u32(&ctl.kempty[k]), 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&ctl.sfull[k]), 1);
      mbar_init(smem_u32(&ctl.pfull[k]), kSoftmaxWarps);
      mbar_init(smem_u32(&ctl.odone[k]), 1);
      mbar_init(smem_u32(&ctl.ofree[k]), kSoftmaxWarps);
      mbar_init(smem_u32(&ctl.qfull[k]), kSoftmaxWarps);
    }
    mbar_init(smem_u32(&ctl.qfree), 1);
    mbar_init(smem_u32(&ctl.mfull), kSoftmaxWarps);
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc<kTmemCols>(smem_u32(&ctl.tmem));
  __syncthreads();
  pdl_wait();  // everything below reads what earlier kernels wrote

  // ---- this CTA's run of tiles and the block that it starts in
  {
    const int per = (pl.blocks + kThreads - 1) / kThreads;
    const int first = min(pl.blocks, tid * per), last = min(pl.blocks, first + per);
    int mine = 0;
    for (int i = first; i < last; ++i) mine += pl.block_tiles[i];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) ctl.warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine, per_head = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int v = ctl.warp_sum[w];
      before += w < warp ? v : 0;
      per_head += v;
    }
    const int total = per_head * p.num_kv_heads, used = used_ctas(total, pl.ctas), cta = blockIdx.x;
    const int lo = cta < used ? run_begin(total, cta, used) : 0, hi = cta < used ? run_begin(total, cta + 1, used) : 0;
    if (tid == 0) {
      ctl.run_lo = lo;
      ctl.run_hi = hi;
      ctl.per_head = per_head;
      pl.info[cta].total = total;
    }
    if (lo < hi) {
      const int hk = lo / per_head, at = lo - hk * per_head;
      if (before <= at && at < before + mine) {  // the thread whose blocks hold the first tile
        int i = first;
        while (before + pl.block_tiles[i] <= at) before += pl.block_tiles[i++];
        ctl.run_hk = hk;
        ctl.run_block = i;
        ctl.run_start = hk * per_head + before;
        const Block b = pl.block[i];
        RunInfo& info = pl.info[cta];
        info.item = hk * pl.blocks + i;
        info.start = hk * per_head + before;
        info.row0 = b.row0;
        info.pair0 = b.pair0;
        info.pairs = b.pairs;
        info.hk = hk;
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  pdl_launch_dependents();  // the join may take its place; it waits for this grid's end

  // Calls f(tile, n) for every tile of this CTA, in order, n counting them;
  // whole warps.  f returns whether to go on.
  const auto for_tiles = [&](auto&& f) {
    for (uint32_t n = 0;; ++n) {
      const uint32_t slot = n % kDescs;
      if (!warp_try(smem_u32(&ctl.dfull[slot]), (n / kDescs) & 1, abort_flag, p.err)) return false;
      const Desc& d = ctl.desc[slot];
      if (d.flags & kEnd) return true;
      const bool ok = f(d, n);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.dempty[slot]));
      if (!ok) return false;
    }
  };

  if (warp == kPlanWarp) {
    // ================================================================ planner
    uint32_t n = 0;  // tiles published
    bool ok = true;
    const int hi = ctl.run_hi, per_head = ctl.per_head;
    int at = ctl.run_lo, hk = ctl.run_hk, block = ctl.run_block, start = ctl.run_start;
    while (ok && at < hi) {
      const Block b = pl.block[block];
      const int from = at - start, to = min(b.tiles, hi - start);  // tiles of the block
      const bool two = b.pairs > kRows, whole = from == 0 && to == b.tiles;
      int done = from;
      for (int s0 = 0; ok && done < to && s0 < b.spans; s0 += 32) {
        Span mine = {};
        if (s0 + lane < b.spans) mine = pl.span[b.span0 + s0 + lane];
        const uint32_t some = __ballot_sync(0xffffffffu, s0 + lane < b.spans && mine.start < to && mine.start + mine.tiles > from);
        for (uint32_t left = some; ok && left; left &= left - 1) {
          const int x = __ffs(left) - 1;
          const int req = __shfl_sync(0xffffffffu, mine.req, x), s_start = __shfl_sync(0xffffffffu, mine.start, x);
          const int s_end = min(to, s_start + __shfl_sync(0xffffffffu, mine.tiles, x));
          const int pos0 = __shfl_sync(0xffffffffu, mine.pos0, x), k_lo = __shfl_sync(0xffffffffu, mine.lo, x);
          const int k_hi = __shfl_sync(0xffffffffu, mine.hi, x);
          const int p0 = __shfl_sync(0xffffffffu, mine.p0, x), p1 = __shfl_sync(0xffffffffu, mine.p1, x);
          const int64_t table = attn_table_base(p, req);
          for (; ok && done < s_end; ) {
            const int count = min(32, s_end - done);
            Desc d = {};
            const int tile = done + lane;
            bool range = false;
            d.pos0 = pos0 + (tile - s_start) * kTile;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int pos = d.pos0 + 64 * r;
              d.page[r] = -1;
              if (lane < count && pos < k_hi) {
                d.page[r] = __ldg(p.block_table + table + (pos >> p.page_shift));
                if (d.page[r] < 0 || d.page[r] >= p.num_pages) {
                  range = true;
                  d.page[r] = -1;
                }
              }
            }
            if (range) atomicOr(p.err, kErrPageRange);
            d.lo = k_lo;
            d.hi = k_hi;
            d.p0 = p0;
            d.p1 = p1;
            d.row0 = b.row0;
            d.pair0 = b.pair0;
            d.pairs = b.pairs;
            d.hk = hk;
            d.part = 2 * blockIdx.x + (from == 0);
            d.flags = two ? kTwo | (p0 < kRows ? kSlot0 : 0) | (p1 > kRows ? kSlot1 : 0) : ((tile - from) & 1 ? kSlot1 : kSlot0);
            d.flags |= (tile == from ? kFirst : 0) | (tile == to - 1 ? kLast : 0) | (whole ? kWhole : 0);
            // a run that ends inside: its values may hold anything behind the end
            if (k_hi > d.pos0 && k_hi < d.pos0 + kTile && (k_hi & 63)) d.flags |= kTail;
            for (int k = 0; ok && k < count; ++k, ++n) {
              const uint32_t slot = n % kDescs;
              ok = n < kDescs || warp_try(smem_u32(&ctl.dempty[slot]), (n / kDescs - 1) & 1, abort_flag, p.err);
              if (ok && lane == k) {
                ctl.desc[slot] = d;
                mbar_arrive(smem_u32(&ctl.dfull[slot]));
              }
            }
            done += count;
          }
        }
      }
      at = start + to;
      if (at >= hi) break;
      // the next block that has tiles
      start = at;
      for (;;) {
        if (start == (hk + 1) * per_head) {
          ++hk;
          block = -1;
        }
        ++block;
        const uint32_t some = __ballot_sync(0xffffffffu, block + lane < pl.blocks && pl.block_tiles[block + lane] > 0);
        if (some) {
          block += __ffs(some) - 1;
          break;
        }
        block += 31;
        if (block >= pl.blocks) {  // (not reached: the tiles counted are there)
          ok = false;
          break;
        }
      }
    }
    if (ok) {
      const uint32_t slot = n % kDescs;
      ok = n < kDescs || warp_try(smem_u32(&ctl.dempty[slot]), (n / kDescs - 1) & 1, abort_flag, p.err);
      if (ok && lane == 0) {
        ctl.desc[slot].flags = kEnd;
        mbar_arrive(smem_u32(&ctl.dfull[slot]));
      }
    }
    clear_other_rows(sp, lane);
  } else if (warp == kLoadWarp) {
    // ================================================================ loader
    uint32_t issued = 0;  // stages
    const bool ok = for_tiles([&](const Desc& d, uint32_t) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {  // keys, values
        const uint32_t st = issued % kStages, bar = smem_u32(&ctl.kfull[st]), dst = base + st * kStage;
        if (issued >= kStages && !warp_try(smem_u32(&ctl.kempty[st]), (issued / kStages - 1) & 1, abort_flag, p.err)) return false;
        const int32_t beyond = static_cast<int32_t>(p.num_pages);  // past the cache: zeros
        const auto page = [&](int r) { return d.page[r] < 0 ? beyond : d.page[r]; };
        const auto row = [&](int r) { return d.hk * p.page_size + ((d.pos0 + 64 * r) & (p.page_size - 1)); };
        if (v == 0) {
          if (lane == 0) mbar_arrive_expect_tx(bar, kStage);
          __syncwarp();
          if (lane < 4) {
            const int r = lane & 1, c = lane >> 1;
            tma_load_4d(dst + c * kPiece + r * kRun, &maps.k, 0, row(r), c, page(r), bar);
          }
        } else {
          // runs of the tile that end inside are copied, with zeros behind the end
          const int tail = d.flags & kTail ? (d.hi - d.pos0) >> 6 : -1;
          if (tail >= 0) {
            const int keys = d.page[tail] < 0 ? 0 : d.hi - d.pos0 - 64 * tail;
            const uint16_t* src = p.v + (d.page[tail] < 0 ? 0 : d.page[tail]) * p.page_stride + static_cast<int64_t>(row(tail)) * kPagedDim;
            const int u = lane & 7, c = (lane >> 3) & 1, k0 = lane >> 4;  // 16-byte unit, piece, key
#pragma unroll 4
            for (int k = k0; k < 64; k += 2)
              cp_async_16_or_zero(dst + tail * 2 * kRun + c * kRun + k * 128 + ((u ^ (k & 7)) << 4), src + (k < keys ? k : 0) * kPagedDim + c * 64 + u * 8, k < keys);
            cp_async_arrive_extra(bar);
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(bar, tail >= 0 ? kStage / 2 : kStage);
          __syncwarp();
          if (lane < 2 && lane != tail) tma_load_4d(dst + lane * 2 * kRun, &maps.v, 0, row(lane), 0, page(lane), bar);
        }
        ++issued;
      }
      return true;
    });
    cp_async_wait_all();
    if (!ok && lane == 0) {  // after a time-out: what was issued lands before the CTA can exit
      int never = 0;
      for (uint32_t x = issued; x > 0 && x + kStages > issued; --x)
        mbar_wait(smem_u32(&ctl.kfull[(x - 1) % kStages]), ((x - 1) / kStages) & 1, &never, p.err);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ================================================================ MMA issuer
    // Steps: the accumulators of each tile.  The score product of a step is
    // issued before the value product of the step before it, when that is the
    // other accumulator's; P lies over S, so one accumulator's products follow
    // one another in order.
    const uint32_t tm = uniform(tmem);
    const uint32_t s_idesc = uniform(idesc_f16(128, 128, DTYPE == FP4IDX_BF16, false, p.negate != 0));
    const uint32_t o_idesc = uniform(idesc_f16(128, 128, DTYPE == FP4IDX_BF16, false, false) | 1u << 16);
    struct Step {
      uint32_t tile, slot;
      bool two, last_of_tile, first, last, tail;  // first / last of the segment
    };
    uint32_t n = 0;          // tiles read
    uint32_t segs = 0;       // segments begun
    uint32_t steps[2] = {};  // value products issued
    uint32_t started = 0;    // accumulators with a product in this segment
    uint32_t left = 0;       // accumulators of the current tile to come
    int32_t flags = 0;
    bool ok = true;
    const auto next = [&](Step& s) {  // false: no more steps (or a wait that failed)
      if (left == 0) {
        const uint32_t slot = n % kDescs;
        if (!warp_try(smem_u32(&ctl.dfull[slot]), (n / kDescs) & 1, abort_flag, p.err)) {
          ok = false;
          return false;
        }
        flags = static_cast<int32_t>(uniform(static_cast<uint32_t>(ctl.desc[slot].flags)));
        if (flags & kEnd) return false;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.dempty[slot]));
        left = flags & (kSlot0 | kSlot1);
        s.first = flags & kFirst;
        ++n;
      } else {
        s.first = false;
      }
      s.tile = n - 1;
      s.slot = left & 1 ? 0 : 1;
      s.two = flags & kTwo;
      left &= left - 1;
      s.last_of_tile = left == 0;
      s.last = s.last_of_tile && (flags & kLast);
      s.tail = flags & kTail;
      return true;
    };
    const auto score = [&](const Step& s) {
      const uint32_t stage = 2 * s.tile, st = uniform(stage % kStages);
      if (s.first) {
        ok = ok && warp_try(smem_u32(&ctl.qfull[0]), segs & 1, abort_flag, p.err);
        ok = ok && warp_try(smem_u32(&ctl.qfull[1]), segs & 1, abort_flag, p.err);
        ++segs;
      }
      ok = ok && warp_try(smem_u32(&ctl.kfull[st]), (stage / kStages) & 1, abort_flag, p.err);
      if (!ok) return;
      tc_fence_after();
      const uint32_t slot = uniform(s.slot);
      if (elect_one()) {
        const uint64_t a = desc_sw128(base + kOff_Q + (s.two ? slot * kQBytes : 0), 16), b = desc_sw128(base + st * kStage, 16);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = (k >> 2) * (kPiece >> 4) + (k & 3) * 2;
          tc_mma_f16(tm + slot * kTile, a + at, b + at, s_idesc, k > 0);
        }
        tc_commit(smem_u32(&ctl.sfull[slot]));
        if (s.last_of_tile) tc_commit(smem_u32(&ctl.kempty[st]));
        if (s.last) tc_commit(smem_u32(&ctl.qfree));
      }
      __syncwarp();
    };
    const auto value = [&](const Step& s) {
      const uint32_t stage = 2 * s.tile + 1, st = uniform(stage % kStages);
      const uint32_t slot = uniform(s.slot);
      if (s.first) started = 0;
      const bool more = started >> slot & 1;
      ok = ok && warp_try(smem_u32(&ctl.kfull[st]), (stage / kStages) & 1, abort_flag, p.err);
      ok = ok && warp_try(smem_u32(&ctl.pfull[slot]), steps[slot] & 1, abort_flag, p.err);
      // The output of the segment before has been read (segs counts this one).
      // Its own warps have done so when P is there, so that this wait is never
      // for a phase further back than the last one; the other ones may not have.
      if (!more && segs > 1) ok = ok && warp_try(smem_u32(&ctl.ofree[slot]), segs & 1, abort_flag, p.err);
      if (!ok) return;
      if (s.tail) fence_proxy_async_smem();
      tc_fence_after();
      ++steps[slot];
      started |= 1u << slot;
      if (elect_one()) {
        const uint64_t b = desc_sw128(base + st * kStage, kRun);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_f16_tmem(tm + kOCol + slot * kTile, tm + slot * kTile + k * 8, b + (k >> 2) * (2 * kRun >> 4) + (k & 3) * 128, o_idesc,
                          k > 0 || more);
        if (s.last_of_tile) tc_commit(smem_u32(&ctl.kempty[st]));
        if (s.last) {
          tc_commit(smem_u32(&ctl.odone[0]));
          tc_commit(smem_u32(&ctl.odone[1]));
        }
      }
      __syncwarp();
    };
    Step now, then;
    bool have = next(now);
    if (have) score(now);
    while (ok && have) {
      const bool more = !now.last && next(then);
      const bool early = more && then.slot != now.slot;
      if (early) score(then);
      if (ok) value(now);
      if (now.last) {
        have = ok && next(now);
        if (have) score(now);
        continue;
      }
      if (ok && more && !early) score(then);
      now = then;
      have = more;
    }
    // no product is in flight when TMEM is freed
    if (elect_one()) tc_commit(smem_u32(&ctl.drain));
    __syncwarp();
    if (lane == 0) {
      int never = 0;
      mbar_wait(smem_u32(&ctl.drain), 0, &never, p.err);
    }
    __syncwarp();
  } else if (warp < 2 * kSoftmaxWarps) {
    // ================================================================ softmax
    const int slot = warp / kSoftmaxWarps, r = tid & (kRows - 1);  // accumulator, row of it
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_at = tmem + lanes + slot * kTile, o_at = tmem + lanes + kOCol + slot * kTile;
    uint32_t segs = 0, steps = 0;   // segments begun; tiles of this accumulator
    uint32_t merged = 0;            // segments whose two accumulators were added up
    int steps_of_seg = 0;
    int vis = 0, pair = 0;          // of this thread's row
    bool valid = false, ok = true;
    float m = -INFINITY;            // reference maximum, in powers of two
    float2 l[2] = {};
    for_tiles([&](const Desc& d, uint32_t) {
      const int off = d.flags & kTwo ? slot * kRows : 0;  // first pair of this accumulator
      if (d.flags & kFirst) {
        pair = d.pair0 + off + r;
        valid = off + r < d.pairs;
        const int t = d.row0 + group_div(p, pair);
        if (segs > 0) ok = warp_try(smem_u32(&ctl.qfree), (segs - 1) & 1, abort_flag, p.err);
        if (!ok) return false;
        if (valid) {
          vis = pl.row_vis[t];
          if (slot == 0 || (d.flags & kTwo)) {
            const int h = d.hk * p.group + pair - group_div(p, pair) * p.group;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + t * p.q_row_stride + h * p.q_head_stride);
            uint4 q[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) q[u] = __ldg(src + u);
            uint8_t* dst = smem + kOff_Q + slot * kQBytes + r * 128;
#pragma unroll
            for (int u = 0; u < 16; ++u) *reinterpret_cast<uint4*>(dst + (u >> 3) * kPiece + (((u & 7) ^ (r & 7)) << 4)) = q[u];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.qfull[slot]));
        ++segs;
        steps_of_seg = 0;
        m = -INFINITY;
        l[0] = l[1] = make_float2(0.0f, 0.0f);
      }
      if (d.flags >> slot & 1) {
        ok = warp_try(smem_u32(&ctl.sfull[slot]), steps & 1, abort_flag, p.err);
        if (!ok) return false;
        tc_fence_after();
        // columns [c_lo, c_lo + c_len) of this row count
        const bool mine = valid && off + r >= d.p0 && off + r < d.p1;
        int c_lo = max(0, d.lo - d.pos0), c_hi = mine ? min(min(vis, d.hi) - d.pos0, kTile) : 0;
        if (d.page[0] < 0) c_lo = max(c_lo, 64);
        if (d.page[1] < 0) c_hi = min(c_hi, 64);
        const int c_len = max(0, c_hi - c_lo);
        if (__any_sync(0xffffffffu, c_len > 0)) {
          uint32_t x[kTile];
          tmem_ld(s_at, x);
          tmem_wait_ld();
          reg_fence(x);
          if (__any_sync(0xffffffffu, c_len < kTile)) {
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (static_cast<uint32_t>(c - c_lo) >= static_cast<uint32_t>(c_len)) x[c] = 0xff800000u;  // -inf
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kTile; c += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              top[k] = fmaxf(fmaxf(top[k], __uint_as_float(x[c + 2 * k])), __uint_as_float(x[c + 2 * k + 1]));
          }
          const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2 - kBelow<DTYPE>;
          const bool raise = most > m + kRaise;
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? ex2(m - most) : 1.0f;
            if (raise) m = most;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              l[k].x *= f;
              l[k].y *= f;
            }
            if (steps_of_seg > 0) {  // (the score product followed the last value product, so that is complete)
#pragma unroll 1
              for (int c = 0; c < kPagedDim; c += 16) {
                uint32_t o[16];
                tmem_ld(o_at + c, o);
                tmem_wait_ld();
                reg_fence(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st_x16(o_at + c, o);
              }
            }
          }
          // weights, their sum in fp32, and P in 16 bits (the MMA's operand type:
          // each weight is rounded once, the sum is of unrounded ones)
          const float2 scale = make_float2(p.scale_log2, p.scale_log2);
          const float2 ref = m == -INFINITY ? make_float2(0.0f, 0.0f) : make_float2(-m, -m);
#pragma unroll
          for (int c = 0; c < kTile; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 a = fma2(make_float2(__uint_as_float(x[c + 2 * k]), __uint_as_float(x[c + 2 * k + 1])), scale, ref);
              a = make_float2(ex2(a.x), ex2(a.y));
              l[k & 1] = add2(l[k & 1], a);
              w[k] = pack2<DTYPE>(a.x, a.y);
            }
            tmem_st_x16(s_at + c / 2, w);
          }
        } else {  // none of the warp's rows sees a key of this tile
          uint32_t w[16] = {};
#pragma unroll
          for (int c = 0; c < kTile / 2; c += 16) tmem_st_x16(s_at + c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.pfull[slot]));
        ++steps;
        ++steps_of_seg;
      }
      if (d.flags & kLast) {
        // ---- output of the segment
        float sum = (l[0].x + l[1].x) + (l[0].y + l[1].y);
        const bool two = d.flags & kTwo;
        const uint32_t parity = (segs - 1) & 1;
        ok = warp_try(smem_u32(&ctl.odone[slot]), parity, abort_flag, p.err);
        if (!ok) return false;
        tc_fence_after();
        if (!two && slot == 1) {
          // the other accumulator's warps read this one's output, once they have
          // read that of the segment before
          ok = segs < 2 || warp_try(smem_u32(&ctl.ofree[1]), parity ^ 1, abort_flag, p.err);
          if (!ok) return false;
          ctl.other[r] = make_float2(m, sum);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.mfull));
          return true;
        }
        // out = f0 O (+ f1 O of the other accumulator)
        float f0 = steps_of_seg > 0 ? 1.0f : 0.0f, f1 = 0.0f;
        if (!two) {
          // (the commit that this warp has waited for covers both accumulators)
          ok = warp_try(smem_u32(&ctl.mfull), merged++ & 1, abort_flag, p.err);
          if (!ok) return false;
          const float2 b = ctl.other[r];
          const float most = fmaxf(m, b.x), at = most == -INFINITY ? 0.0f : most;
          f0 = ex2(m - at);  // (accumulator 0 takes a segment's first tile)
          f1 = ex2(b.x - at);
          sum = f0 * sum + f1 * b.y;
          m = most;
        }
        const bool both = !two && __any_sync(0xffffffffu, f1 != 0.0f);
        const int t = d.row0 + group_div(p, pair), h = d.hk * p.group + pair - group_div(p, pair) * p.group;
        const bool whole = d.flags & kWhole;
        if (whole) {
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          f0 = sum == 0.0f ? 0.0f : f0 * inv;
          f1 *= inv;
        }
        const int row = off + r;  // of the block
        uint4* out = reinterpret_cast<uint4*>(p.out + t * p.out_row_stride + static_cast<int64_t>(h) * kPagedDim);
        float4* part = pl.partial + static_cast<int64_t>(d.part) * (kPagedDim / 4) * kBlockPairs + row;
#pragma unroll 1
        for (int c = 0; c < kPagedDim; c += 32) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld(o_at + c, o);
          tmem_wait_ld();
          reg_fence(o);
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = f0 == 0.0f ? 0.0f : __uint_as_float(o[e]) * f0;
          if (both) {
            tmem_ld(o_at + kTile + c, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = f1 == 0.0f ? y[e] : fmaf(__uint_as_float(o[e]), f1, y[e]);
          }
          if (valid && whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              out[(c + e) / 8] = make_uint4(pack2<DTYPE>(y[e], y[e + 1]), pack2<DTYPE>(y[e + 2], y[e + 3]), pack2<DTYPE>(y[e + 4], y[e + 5]),
                                            pack2<DTYPE>(y[e + 6], y[e + 7]));
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) part[(c + e) / 4 * kBlockPairs] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        if (valid) {
          if (!whole) pl.stats[static_cast<int64_t>(d.part) * kBlockPairs + row] = make_float2(m, sum);
          else if (p.lse) p.lse[static_cast<int64_t>(t) * p.num_heads + h] = row_lse(m, sum);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctl.ofree[slot]));
          if (!two) mbar_arrive(smem_u32(&ctl.ofree[1]));
        }
      }
      return true;
    });
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem);
  }
}

// ---------------------------------------------------------------- join
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the partial sums of
// a block that crosses run boundaries, in the order of its tiles.  blockIdx.x
// counts run boundaries; the first one inside a block does its work.  A CTA
// takes 32 rows and 32 columns, a lane a row; its warps take parts in turn and
// are added in order.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinCols = 32;

template <int DTYPE>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Plan pl) {
  __shared__ float4 sums[kJoinWarps][kJoinCols / 4][32];
  __shared__ float2 part[kJoinWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const AttnParams& p = pl.sp.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x + 1;  // the boundary before CTA c's run
  const int total = pl.info[0].total, used = used_ctas(total, pl.ctas);
  const auto inside = [&](int x, int item) {
    return x > 0 && x < used && pl.info[x].item == item && pl.info[x].start < run_begin(total, x, used);
  };
  if (c >= used) return;
  const RunInfo info = pl.info[c];
  if (!inside(c, info.item) || inside(c - 1, info.item)) return;
  const int row = blockIdx.y * 32 + lane, cols = blockIdx.z * kJoinCols;
  if (static_cast<int>(blockIdx.y) * 32 >= info.pairs) return;
  int parts = 2;
  for (;;) {  // 32 boundaries at a time
    const uint32_t in = __ballot_sync(0xffffffffu, inside(c + parts - 1 + lane, info.item));
    const int n = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
    parts += n;
    if (n < 32) break;
  }
  float4 acc[kJoinCols / 4] = {};
  float m = -INFINITY, l = 0.0f;
#pragma unroll 2
  for (int i = warp; i < parts; i += kJoinWarps) {
    // part i is CTA c - 1 + i's; of the first one its last segment, of the others their first
    const int64_t at = 2 * (c - 1 + i) + (i == 0);
    const float2 s = pl.stats[at * kBlockPairs + row];
    float4 o[kJoinCols / 4];
#pragma unroll
    for (int v = 0; v < kJoinCols / 4; ++v) o[v] = pl.partial[(at * (kPagedDim / 4) + cols / 4 + v) * kBlockPairs + row];
    const float top = fmaxf(m, s.x), ref = top == -INFINITY ? 0.0f : top;
    const float keep = ex2(m - ref), w = ex2(s.x - ref);
    m = top;
    l = l * keep + w * s.y;
#pragma unroll
    for (int v = 0; v < kJoinCols / 4; ++v) {
      acc[v].x = acc[v].x * keep + w * o[v].x;
      acc[v].y = acc[v].y * keep + w * o[v].y;
      acc[v].z = acc[v].z * keep + w * o[v].z;
      acc[v].w = acc[v].w * keep + w * o[v].w;
    }
  }
#pragma unroll
  for (int v = 0; v < kJoinCols / 4; ++v) sums[warp][v][lane] = acc[v];
  part[warp][lane] = make_float2(m, l);
  __syncthreads();
  // warp v adds the warps' shares of four columns
  static_assert(kJoinWarps == kJoinCols / 4, "four columns a warp");
  m = part[0][lane].x;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, part[w][lane].x);
  const float ref = m == -INFINITY ? 0.0f : m;
  l = 0.0f;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float4 o = sums[w][warp][lane];
    const float f = ex2(part[w][lane].x - ref);
    l = fmaf(f, part[w][lane].y, l);
    y.x = fmaf(f, o.x, y.x);
    y.y = fmaf(f, o.y, y.y);
    y.z = fmaf(f, o.z, y.z);
    y.w = fmaf(f, o.w, y.w);
  }
  if (row >= info.pairs) return;
  const int pair = info.pair0 + row, t = info.row0 + group_div(p, pair);
  const int h = info.hk * p.group + pair - group_div(p, pair) * p.group;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2* out = reinterpret_cast<uint2*>(p.out + t * p.out_row_stride + static_cast<int64_t>(h) * kPagedDim + cols);
  out[warp] = make_uint2(pack2<DTYPE>(y.x * inv, y.y * inv), pack2<DTYPE>(y.z * inv, y.w * inv));
  if (p.lse && warp == 0 && blockIdx.z == 0) p.lse[static_cast<int64_t>(t) * p.num_heads + h] = row_lse(m, l);
}

// ---------------------------------------------------------------- host
int64_t round16(int64_t n) { return (n + 15) & ~int64_t{15}; }

// The workspace's parts; returns its size.
size_t lay_out(Plan* pl, char* w) {
  char* const begin = w;
  const auto take = [&](int64_t bytes) {
    char* const at = w;
    w += round16(bytes);
    return at;
  };
  const int64_t blocks = pl->blocks, rows = static_cast<int64_t>(pl->ctas) * 2 * kBlockPairs;
  pl->block = reinterpret_cast<Block*>(take(blocks * sizeof(Block)));
  pl->block_tiles = reinterpret_cast<int32_t*>(take(blocks * 4));
  pl->span = reinterpret_cast<Span*>(take((2 * blocks + pl->sp.a.num_seqs + 2) * sizeof(Span)));
  pl->row_vis = reinterpret_cast<int32_t*>(take(static_cast<int64_t>(pl->sp.a.num_rows) * 4));
  pl->info = reinterpret_cast<RunInfo*>(take(pl->ctas * sizeof(RunInfo)));
  pl->stats = reinterpret_cast<float2*>(take(rows * 8));
  pl->partial = reinterpret_cast<float4*>(take(rows * kPagedDim * 4));
  return static_cast<size_t>(w - begin);
}

Plan plan_of(const SharedParams& p) {
  Plan pl;
  std::memset(&pl, 0, sizeof(pl));
  pl.sp = p;
  pl.blocks_per_group = p.blocks_per_group;
  pl.blocks = p.num_groups * p.blocks_per_group;
  pl.ctas = p.ctas;
  return pl;
}

template <int DTYPE>
cudaError_t launch(const Plan& pl, const AttnMaps& maps, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory limit (a call costs 1 us)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(shared_kernel<DTYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>((pl.blocks + kPlanWarps - 1) / kPlanWarps));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, plan_kernel, pl)) != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(pl.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  if ((e = cudaLaunchKernelEx(&cfg, shared_kernel<DTYPE>, pl, maps)) != cudaSuccess) return e;
  if (pl.ctas < 2) return cudaSuccess;
  // rows that a block can have
  const int64_t pairs = static_cast<int64_t>(pl.sp.max_group_rows) * pl.sp.a.group;
  const unsigned rows = static_cast<unsigned>(std::min<int64_t>(pairs, kBlockPairs));
  cfg.gridDim = dim3(static_cast<unsigned>(pl.ctas - 1), (rows + 31) / 32, kPagedDim / kJoinCols);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<DTYPE>, pl);
}

}  // namespace

bool plan_shared(SharedParams* p, int sms) {
  AttnParams& a = p->a;
  a.group_mul = ((uint64_t{1} << kGroupShift) + a.group - 1) / a.group;
  p->max_group_rows = std::min(p->max_group_rows, a.num_rows);
  const int64_t pairs = static_cast<int64_t>(p->max_group_rows) * a.group;
  const int64_t per = (pairs + kBlockPairs - 1) / kBlockPairs, blocks = per * p->num_groups;
  if (blocks > 1 << 20) return false;
  // A span is what a block has of one request or of the prefix.
  const int64_t tiles = (static_cast<int64_t>(a.max_seqlen_k) + 63) / kTile + 1;
  const int64_t spans = 2 * blocks + a.num_seqs;
  if (tiles * spans > INT32_MAX / a.num_kv_heads) return false;
  p->blocks_per_group = static_cast<int32_t>(per);
  p->ctas = static_cast<int32_t>(std::min<int64_t>(sms, tiles * spans * a.num_kv_heads));
  return true;
}

size_t shared_workspace(const SharedParams& p) {
  Plan pl = plan_of(p);
  return lay_out(&pl, nullptr);
}

cudaError_t launch_shared(SharedParams p, const AttnMaps& maps, int dtype, void* workspace, cudaStream_t stream) {
  Plan pl = plan_of(p);
  lay_out(&pl, static_cast<char*>(workspace));
  return dtype == FP4IDX_BF16 ? launch<FP4IDX_BF16>(pl, maps, stream) : launch<FP4IDX_FP16>(pl, maps, stream);
}

}  // namespace fp4idx
