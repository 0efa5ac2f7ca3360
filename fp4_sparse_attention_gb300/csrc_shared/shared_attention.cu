// shared_attention.cu -- grouped-query attention of requests that share a
// prefix (fp4idx_shared_prefix_attention) for sm_103a.
//
//   s(r, j) = scale * q[r] . k[j],   out[r] = sum_j exp(s - lse) v[j]
//
// A group's (row, head) pairs of one K/V head are taken 256 at a time: a block.
// Its keys are what each of its requests has behind the prefix, then the
// prefix itself, once, for all of its rows: one list of 128-key tiles.  The
// tiles of all blocks and K/V heads are concatenated and cut into runs, one per
// CTA: equal ones, or, where that loses little, each block's own.  A block cut
// by a boundary leaves partial sums that join_kernel adds in a fixed order.
//
// A CTA holds two score accumulators, two outputs (128 rows x 128 columns each,
// all 512 TMEM columns) and a ring of five 32 KB stages, each a tile's keys or
// its values:
//
//   S [128 rows x 128 keys] = Q K^T      tcgen05, Q and K in shared memory
//   P = 2^(S - m)                        registers; 16 bits, over S's columns in TMEM (each 64 keys' over their own)
//   O [128 rows x 128]     += P V        tcgen05, P in TMEM, V in shared memory
//
// While one accumulator's rows go through the softmax, the tensor pipe works
// on the other's: with more than 128 pairs the two hold the block's halves and
// share each tile; with fewer they hold the same rows and take tiles in turn,
// and the end adds them up.  Two threads share a row, 64 keys of a tile each.
// They take a tile's weights relative to the reference of the tiles before and
// look at their sum: only where that is too large (or there is no reference
// yet) do they go over the scores for a maximum, so that a tile's scores are
// read once and all that the two have to agree on is that neither wants to.
//
// Roles: warps 0-7 and 8-15 softmax of the two accumulators, queries and output
// (four of a lane quarter, by halves of the keys); warps 16 and 17 issue the
// products of one accumulator each; warp 18 loader (TMA; 16-byte copies, which
// can leave zeros where a value may be anything, for the last values of a run
// that ends inside); warp 19 planner, which looks up the tiles' pages ahead of all
// of them and hands them out in chunks.
//
// Bounds and figures (bf16, cold caches).  A tile of a full block is 16.8 MFLOP for
// 64 KB: with every row of 256 pairs on the same keys the tensor pipe and the
// softmax beside it bound it (2,048 rows x 32/8 heads on 8,191 + 512..640 keys:
// 196 us, 1,459 TFLOP/s, 76 % of a burst of large library products, and 205 us
// where long runs of calls bring the clock to the power limit; a tile takes
// 2,700 cycles, of which its products need 2,180); with keys of a request's own or
// few rows a group HBM does (8 groups x 24 rows x 40/8 heads, 365 MB: 82.7 us,
// 6.4 TB/s while the runs last; no prefix, 64 requests x 8,192 keys, 1,075 MB:
// 172 us, 6.3 TB/s, 93 % of a copy, and 189 us as one group, whose 32 requests a
// block each have tiles of their own).  What a short call pays: 2 us plan, 2 us until a
// run is known, 2 us for the first pages and keys, 2 us output, 4-7 us join (2
// requests on 200 keys 13.9 us, 64 samples of 32,768 keys 53.4 us).
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
constexpr int kHalf = kTile / 2;           // keys of a tile, or columns of an output, that a softmax thread has
constexpr int kSoftmaxWarps = 8;           // of one accumulator
constexpr int kMmaWarp = 2 * kSoftmaxWarps, kLoadWarp = kMmaWarp + 2, kPlanWarp = kMmaWarp + 3;
constexpr int kThreads = 32 * (kPlanWarp + 1);
constexpr int kStages = 5;
constexpr uint32_t kStage = 32768, kPiece = 128 * 128, kRun = 64 * 128;
constexpr uint32_t kQBytes = 2 * kPiece;   // 128 rows x 128 values
constexpr int kChunks = 4, kChunkTiles = 12;  // chunks that the planner may be ahead, tiles of a chunk
constexpr uint32_t kTmemCols = 512, kOCol = 256;
constexpr int kGroupShift = 40;            // pair / group as (pair * ceil(2^40 / group)) >> 40 (attention.cu)
// A row's reference is its maximum when it is set, in fp16 2^7 less, so that
// shares down to 2^-32 are kept (attention.cu).  It is set anew when a tile's
// weights add up to more than the limit: in fp16 the type's range (the sum
// bounds each weight), in bf16 far below that of fp32.
template <int DTYPE>
constexpr float kBelow = DTYPE == FP4IDX_FP16 ? 7.0f : 0.0f;
template <int DTYPE>
constexpr float kLimit = DTYPE == FP4IDX_FP16 ? 32768.0f : 16777216.0f;

// ---------------------------------------------------------------- plan
struct Block {
  int32_t row0;        // the group's first row
  int32_t pair0;       // the block's first pair of the group's
  int32_t pairs;
  int32_t tiles;
  int32_t span0, spans;
  int32_t own_tiles, own_spans;  // without the prefix's
};
// Keys [lo, hi) of one table row for the pairs [p0, p1) of a block: tiles from
// position pos0 (a multiple of 64, at most 63 below lo) on.
struct Span {
  int32_t req, pos0, lo, hi;
  int32_t start, tiles;  // tiles of the block before it; its own
  int32_t p0, p1;
};
// Where a CTA's run begins (for the join).
struct RunInfo {
  int32_t item;    // K/V head * blocks + block, -1: it has no tiles
  int32_t inside;  // behind the block's first tile
  int32_t row0, pair0, pairs, hk;
  int32_t pad[2];
};

struct Plan {
  SharedParams sp;
  int32_t blocks;          // of one K/V head: num_groups x blocks_per_group
  int32_t blocks_per_group;
  int32_t ctas;
  int32_t few;             // up to 32 blocks, tiles that 32 bits can be multiplied in
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
__device__ __forceinline__ int2 group_requests(const int32_t* offsets, int g, int num_seqs) {
  const int lo = min(max(offsets[g], 0), num_seqs);
  return make_int2(lo, min(max(offsets[g + 1], lo), num_seqs));
}

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanReqs = 512, kPlanRows = 2048;  // requests (and groups), rows that a CTA's shared memory has room for

// A warp, or with many requests a group (WIDE) a CTA, plans a block: its spans,
// its tiles and what its rows see: a warp takes 32 requests at a time, 1.4 us.
// (128 requests in one block: 37.7 us with a warp, 34.8 with a CTA.)
template <bool WIDE>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ Plan pl) {
  __shared__ int sums[kPlanWarps][3];  // WIDE: spans, tiles, most positions that a row sees
  constexpr int warps = WIDE ? kPlanWarps : 1;
  pdl_wait();
  pdl_launch_dependents();
  const SharedParams& sp = pl.sp;
  const AttnParams& p = sp.a;
  // What a small call gives comes to shared memory in one round trip: read where
  // it is needed, it is a chain of five.  (48 requests: 0.8 us less; 16: 0.7; two,
  // whose arrays are a line each: 0.2 more.)
  __shared__ int32_t cu_q_s[kPlanReqs + 1], cu_k_s[kPlanReqs + 1], qo_s[kPlanReqs], groups_s[kPlanReqs + 1], prefix_s[kPlanReqs], seen_s[kPlanRows];
  const int32_t *cu_q = p.cu_seqlens_q, *cu_k = p.cu_seqlens_k, *qo = p.qo_offset, *groups = sp.group_offsets, *prefix_lens = sp.prefix_len;
  const int32_t* visible = p.visible_len;
  if (p.num_seqs <= kPlanReqs && sp.num_groups <= kPlanReqs) {
    const auto stage = [&](int32_t* to, const int32_t*& from, int n) {
      for (int x = threadIdx.x; x < n; x += kPlanThreads) cp_async_4(smem_u32(to + x), from + x);
      from = to;
    };
    stage(groups_s, groups, sp.num_groups + 1);
    stage(prefix_s, prefix_lens, sp.num_groups);
    stage(cu_q_s, cu_q, p.num_seqs + 1);
    stage(cu_k_s, cu_k, p.num_seqs + 1);
    if (qo) stage(qo_s, qo, p.num_seqs);
    if (visible && p.num_rows <= kPlanRows) stage(seen_s, visible, p.num_rows);
    cp_async_wait_all();
    __syncthreads();
  }
  const int lane = threadIdx.x & 31;
  const int warp = WIDE ? threadIdx.x >> 5 : 0, i = WIDE ? blockIdx.x : blockIdx.x * kPlanWarps + (threadIdx.x >> 5);
  if (i >= pl.blocks) return;
  const int g = i / pl.blocks_per_group;
  const int2 reqs = group_requests(groups, g, p.num_seqs);
  const int n_reqs = reqs.y - reqs.x;
  // (loads that need nothing from each other stand together)
  const int step = (n_reqs + 31) >> 5;
  const int probe = lane * step < n_reqs ? cu_q[reqs.x + lane * step] : INT32_MAX;
  const int first_row = cu_q[reqs.x], end_row = cu_q[reqs.y];
  const int prefix_len = prefix_lens[g];
  const auto key_count = [&](int a) {
    return min(max(0, cu_k[a + 1] - cu_k[a]), p.max_seqlen_k);
  };
  int keys = lane < n_reqs ? key_count(reqs.x + lane) : -1;  // of the group's first requests
  Block blk = {};
  blk.row0 = max(0, first_row);
  const int group_rows = max(min(end_row, p.num_rows) - blk.row0, 0), rows = min(group_rows, sp.max_group_rows);
  if (group_rows > rows && i == g * pl.blocks_per_group && warp == 0 && lane == 0) atomicOr(p.err, kErrLengths);
  const int64_t pair0 = static_cast<int64_t>(i - g * pl.blocks_per_group) * kBlockPairs;
  const int64_t pairs = min(static_cast<int64_t>(rows) * p.group - pair0, static_cast<int64_t>(kBlockPairs));
  if (pairs <= 0) {
    if (warp == 0 && lane == 0) {
      pl.block[i] = blk;
      pl.block_tiles[i] = 0;
    }
    return;
  }
  blk.pair0 = static_cast<int>(pair0);
  blk.pairs = static_cast<int>(pairs);
  const int r0 = blk.row0 + group_div(p, pair0), r1 = blk.row0 + group_div(p, pair0 + pairs - 1) + 1;  // its rows
  // the requests of its first and last row: the last ones that begin at or
  // before it, 32 tests at a time
  int a0 = reqs.x + max(0, __popc(__ballot_sync(0xffffffffu, probe <= r0)) - 1) * step;
  int a1 = reqs.x + max(0, __popc(__ballot_sync(0xffffffffu, probe <= r1 - 1)) - 1) * step;
  for (int n = step; n > 1;) {
    const int by = (n + 31) >> 5, at = lane * by;
    const int x0 = at < n && a0 + at < reqs.y ? cu_q[a0 + at] : INT32_MAX;
    const int x1 = at < n && a1 + at < reqs.y ? cu_q[a1 + at] : INT32_MAX;
    a0 += max(0, __popc(__ballot_sync(0xffffffffu, x0 <= r0)) - 1) * by;
    a1 += max(0, __popc(__ballot_sync(0xffffffffu, x1 <= r1 - 1)) - 1) * by;
    n = by;
  }
  // The prefix is read through the first request whose keys reach its end, or
  // else the first of the longest ones: requests that have ended, the group's
  // first one among them, leave it shared.
  const int wanted = max(0, min(prefix_len, p.max_seqlen_k));
  uint32_t reach = __ballot_sync(0xffffffffu, keys >= wanted);
  int through = reqs.x + __ffs(reach) - 1, prefix = wanted;
  if (reach == 0) {
    prefix = -1;
    for (int x = 0; reach == 0 && x < n_reqs; x += 32) {
      if (x > 0) keys = x + lane < n_reqs ? key_count(reqs.x + x + lane) : -1;
      const int most = min(wanted, __reduce_max_sync(0xffffffffu, keys));
      reach = __ballot_sync(0xffffffffu, keys >= wanted);
      if (most > prefix) {
        prefix = most;
        through = reqs.x + x + __ffs(__ballot_sync(0xffffffffu, keys >= most)) - 1;
      }
    }
  }
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
    int spans_before = 0, tiles_before = 0, all_spans = __popc(some), all_tiles = __shfl_sync(0xffffffffu, incl, 31);
    if constexpr (WIDE) {
      __syncthreads();
      if (lane == 0) {
        sums[warp][0] = all_spans;
        sums[warp][1] = all_tiles;
      }
      __syncthreads();
      all_spans = all_tiles = 0;
#pragma unroll
      for (int w = 0; w < warps; ++w) {
        if (w < warp) {
          spans_before += sums[w][0];
          tiles_before += sums[w][1];
        }
        all_spans += sums[w][0];
        all_tiles += sums[w][1];
      }
    }
    if (have) {
      Span w = s;
      w.start = blk.tiles + tiles_before + incl - s.tiles;
      spans[blk.spans + spans_before + __popc(some & ((1u << lane) - 1))] = w;
    }
    blk.spans += all_spans;
    blk.tiles += all_tiles;
  };
  for (int base0 = a0; base0 <= a1; base0 += 32 * warps) {
    const int base = base0 + 32 * warp, a = base + lane;
    int from = 0, to = 0, k_len = 0, hi = 0;  // its rows of the block, its keys, the most that a row sees
    int64_t off = 0;                          // causal: row t sees t + off
    if (a <= a1) {
      const int q0 = cu_q[a], q1 = cu_q[a + 1];
      from = max(q0, r0);
      to = min(q1, r1);
      k_len = key_count(a);
      off = (qo ? static_cast<int64_t>(qo[a]) : static_cast<int64_t>(k_len) - (q1 - q0)) + 1 - q0;
    }
    const auto sees = [&](int t, int n, int64_t o) {
      int64_t v = n;
      if (visible) v = visible[t];
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
  blk.own_tiles = blk.tiles;
  blk.own_spans = blk.spans;
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (WIDE) {
    if (lane == 0) sums[warp][2] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < warps; ++w) top = max(top, sums[w][2]);
  }
  Span s = {};
  s.req = through;
  s.hi = min(prefix, top);
  s.tiles = (s.hi + kTile - 1) / kTile;
  if (s.tiles == 0 && blk.tiles == 0) s.tiles = 1;  // rows without keys are written, too
  s.p1 = blk.pairs;
  add(warp == 0 && lane == 0 && s.tiles > 0, s);
  if (warp == 0 && lane == 0) {
    pl.block[i] = blk;
    pl.block_tiles[i] = blk.tiles;
  }
}

// ---------------------------------------------------------------- main kernel
enum : int32_t { kFirst = 1, kLast = 2, kEnd = 4, kTwo = 8, kWhole = 16, kHole0 = 32, kHole1 = 64, kTail = 128, kOdd = 256, kSlot0 = 512, kSlot1 = 1024 };

constexpr int32_t kAllLanes = kRows << 16;

// Up to kChunkTiles consecutive tiles of one span; a tile with a page that is
// not there, or a run that ends inside, is a chunk of its own.
struct Chunk {
  int32_t flags;         // kFirst / kLast: holds the first / last tile of a segment (a run of one block's tiles)
  int32_t tiles;
  int32_t pos0, lo, hi;  // position of the first key; keys that count
  int32_t p0, p1;        // pairs of the block that they count for
  int32_t row0, pair0, pairs, hk;
  int32_t part;          // slot of the segment's partial sums
  int32_t lanes[2];      // rows of each accumulator that they count for, from | to << 16, or kAllLanes
  int32_t page[kChunkTiles][2];  // -1: no keys
};

struct Control {
  uint64_t cfull[kChunks], cempty[kChunks];
  uint64_t kfull[kStages], kempty[kStages];
  uint64_t sfull[2], pfull[2], odone[2], qfull[2];
  uint64_t turn[2], mfull, mfree, drain;
  Chunk chunk[kChunks];
  float row[2][2][kRows];  // exchange between the threads of a row
  Block first;           // the block that this CTA's run begins in
  int32_t run_hk, run_block, run_start, run_lo, run_hi, per_head;
  uint32_t worst;
  uint32_t tmem;
  int abort;
};
constexpr uint32_t kOff_Q = kStages * kStage, kOff_Ctl = kOff_Q + 2 * kQBytes;
constexpr uint32_t kSmem = kOff_Ctl + sizeof(Control);
static_assert(kSmem <= 232448, "227 KB per CTA");

// A run of a block's own pays for up to this many tiles more than an equal run
// over all blocks: a run that crosses from one block to the next has queries to
// wait for and sums to write twice.
constexpr int kOwnRunTiles = 3;
// In equal runs of 16 tiles and more a block's begin counts like two tiles: its
// queries, and the output of the block before it.  (8 groups, 364 MB of keys and
// values: 83.3 us with nothing for it, 82.4 with one, 81.4 with two, 81.8 with
// four.)
constexpr uint32_t kBeginTiles = 2;
// A block's own CTAs: [S used / all, (S + t) used / all) of a block of t tiles
// behind S others, at least t used / all of them.  (32 bits: below kTiles32 tiles.)
constexpr int kTiles32 = 1 << 21;
static_assert(static_cast<uint64_t>(kTiles32) * 3 * 257 < uint64_t{1} << 32, "with as many spans, times the CTAs (a join's threads) and one");
struct Split {
  uint32_t worst, limit;  // tiles of a block's longest own run; what that may be
};
__device__ __forceinline__ Split split_of(uint32_t tiles, uint32_t all, uint32_t used) {
  const uint32_t least = tiles * used / all;
  return {tiles == 0 ? 0u : least == 0 ? UINT32_MAX : (tiles + least - 1) / least, (all + used - 1) / used + kOwnRunTiles};
}
// The last tile that may be the first of CTA cta's block.
__device__ __forceinline__ uint32_t own_probe(uint32_t cta, uint32_t all, uint32_t used) { return ((cta + 1) * all - 1) / used; }
// CTA cta's run of block b's tiles, which begin at `start`.  Where it is long the
// block's spans are counted, too, as if they were alike: each one's mask, end
// inside a page and new reference take as long as half a tile.  (64 requests of
// one key each behind 32,768: 50.2 us without, 43.7 with a half, 46.5 with a
// quarter.  In runs of two tiles it costs a tile: 17.0 us for 15.0.)
constexpr uint32_t kLongRun = 8;
__device__ __forceinline__ void own_run(const Block& b, uint32_t start, uint32_t cta, uint32_t all, uint32_t used, uint32_t* lo, uint32_t* hi) {
  const uint32_t tiles = b.tiles, c0 = start * used / all, n = (start + tiles) * used / all - c0;
  const bool weigh = tiles >= kLongRun * n;
  const uint32_t own_tiles = weigh ? b.own_tiles : 0, spans = weigh ? b.own_spans : 0, own = 2 * own_tiles + spans, units = 2 * tiles + spans;
  const float rate = __fdividef(static_cast<float>(own_tiles), static_cast<float>(own));
  const auto cut = [&](uint32_t k) {  // the tile that unit units * k / n lies in
    const uint32_t u = units * k / n;
    return start + (u < own ? static_cast<uint32_t>(static_cast<float>(u) * rate) : own_tiles + (u - own + 1) / 2);
  };
  *lo = cut(cta - c0);
  *hi = cut(cta + 1 - c0);
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
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}
// Arrival on `bar` once this thread's copies so far have landed; it counts
// itself as one more pending arrival first.
__device__ __forceinline__ void cp_async_arrive_extra(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// tc_mma_f16_tmem for lanes [from, to) of D; the others stay as they are.  A
// request's own tile is multiplied with the weights of all rows of an
// accumulator: the other requests' are zeros, but its values may be infinite or
// NaN, which concerns nobody else.  (With the zeros that their output then has
// to begin with, 64 samples take 53.9 for 53.2 us, 8 groups 82.1 for 80.5, 64
// requests of 8,192 keys without a prefix 189 for 182, rows of one request what
// they took.  Masks made once a tile and eight products in a row were no faster.)
__device__ __forceinline__ void tc_mma_f16_tmem_lanes(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate,
                                                      int from, int to) {
  uint32_t off[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int lo = min(max(from - 32 * w, 0), 32), hi = min(max(to - 32 * w, 0), 32);
    off[w] = ~(static_cast<uint32_t>((uint64_t{1} << hi) - 1) & ~static_cast<uint32_t>((uint64_t{1} << lo) - 1));
  }
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}

// Rows that no group holds: zeros and -inf, a (row, head) pair of a CTA at a time.
__device__ __forceinline__ void clear_other_rows(const SharedParams& sp, int lane) {
  const AttnParams& p = sp.a;
  const int first = min(max(0, __ldg(p.cu_seqlens_q + group_requests(sp.group_offsets, 0, p.num_seqs).x)), p.num_rows);
  const int last = min(max(first, __ldg(p.cu_seqlens_q + group_requests(sp.group_offsets, sp.num_groups - 1, p.num_seqs).y)), p.num_rows);
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
__global__ void __launch_bounds__(kThreads, 1) shared_kernel(const __grid_constant__ Plan pl, const __grid_constant__ SharedMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control& ctl = *reinterpret_cast<Control*>(smem + kOff_Ctl);
  const SharedParams& sp = pl.sp;
  const AttnParams& p = sp.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem);
  volatile int* abort_flag = &ctl.abort;

  if (base & 1023u) {  // the swizzled layouts need it; the runtime places the window there
    if (tid == 0) {
      pl.info[blockIdx.x].item = -1;
      atomicOr(p.err, kErrTimeout);
    }
    return;
  }
  if (tid == 0) {
    for (int k = 0; k < kChunks; ++k) {
      mbar_init(smem_u32(&ctl.cfull[k]), 1);
      mbar_init(smem_u32(&ctl.cempty[k]), kPlanWarp);
    }
    for (int k = 0; k < kStages; ++k) {
      mbar_init(smem_u32(&ctl.kfull[k]), 1);
      mbar_init(smem_u32(&ctl.kempty[k]), 2);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&ctl.sfull[k]), 1);
      mbar_init(smem_u32(&ctl.pfull[k]), kSoftmaxWarps);
      mbar_init(smem_u32(&ctl.odone[k]), 1);
      mbar_init(smem_u32(&ctl.turn[k]), 1);
      mbar_init(smem_u32(&ctl.qfull[k]), kSoftmaxWarps);
    }
    mbar_init(smem_u32(&ctl.mfull), kSoftmaxWarps);
    mbar_init(smem_u32(&ctl.mfree), kSoftmaxWarps);
    mbar_init(smem_u32(&ctl.drain), 2);
    ctl.abort = 0;
    ctl.run_lo = ctl.run_hi = ctl.worst = 0;
    fence_barrier_init();
  }
  if (tid == 32 * kLoadWarp) {
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.v_part);
  }
  if (warp == kMmaWarp) tmem_alloc<kTmemCols>(smem_u32(&ctl.tmem));
  __syncthreads();
  pdl_wait();  // everything below reads what earlier kernels wrote

  // ---- this CTA's run of tiles and the block that it begins in
  const auto begin_run = [&](const Block& b, int i, int hk, int start, int lo, int per_head) {
    ctl.first = b;
    ctl.run_hk = hk;
    ctl.run_block = i;
    ctl.run_start = start;
    ctl.run_lo = lo;
    ctl.per_head = per_head;
    RunInfo info = {};
    info.item = hk * pl.blocks + i;
    info.inside = lo > start;
    info.row0 = b.row0;
    info.pair0 = b.pair0;
    info.pairs = b.pairs;
    info.hk = hk;
    pl.info[blockIdx.x] = info;
  };
  if (pl.few) {
    // a block a lane of one warp
    if (warp == kPlanWarp) {
      Block own = {};
      if (lane < pl.blocks) own = pl.block[lane];
      const uint32_t mine = own.tiles, cta = blockIdx.x;
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t before = incl - mine, per_head = __shfl_sync(0xffffffffu, incl, 31), all = per_head * p.num_kv_heads;
      const uint32_t used = min(static_cast<uint32_t>(pl.ctas), (all + 1) / 2);
      if (cta >= used) {
        if (lane == 0) pl.info[cta].item = -1;
      } else {
        const Split split = split_of(mine, all, used);
        const bool own_runs = static_cast<uint32_t>(pl.blocks * p.num_kv_heads) <= used &&
                              __reduce_max_sync(0xffffffffu, split.worst) <= split.limit;
        if (own_runs) {
          const uint32_t x = own_probe(cta, all, used), h = x / per_head, at = x - h * per_head;
          if (before <= at && at < before + mine) {
            const uint32_t start = h * per_head + before;
            uint32_t lo, hi;
            own_run(own, start, cta, all, used, &lo, &hi);
            ctl.run_hi = hi;
            begin_run(own, lane, h, start, lo, per_head);
          }
        } else {
          const uint32_t cost = all >= 16 * used ? kBeginTiles : 0, some = __ballot_sync(0xffffffffu, mine > 0);
          const uint32_t u_mine = mine > 0 ? mine + cost : 0, u_before = before + cost * __popc(some & ((1u << lane) - 1));
          const uint32_t u_head = per_head + cost * __popc(some), u_all = u_head * p.num_kv_heads;
#pragma unroll
          for (int end = 0; end < 2; ++end) {
            const uint32_t x = u_all * (cta + end) / used, h = x / u_head, at = x - h * u_head;
            if (end && x == u_all) {
              if (lane == 0) ctl.run_hi = all;
            } else if (u_before <= at && at < u_before + u_mine) {
              const uint32_t start = h * per_head + before, tile = start + max(at - u_before, cost) - cost;
              if (end) ctl.run_hi = tile;
              else begin_run(own, lane, h, start, tile, per_head);
            }
          }
        }
      }
    }
  } else {
    int* warp_sum = reinterpret_cast<int*>(smem);  // (the ring is not in use yet)
    const int per = (pl.blocks + kThreads - 1) / kThreads;
    const int first = min(pl.blocks, tid * per), last = min(pl.blocks, first + per);
    Block own = {};
    int mine = 0;
    if (per == 1) {
      if (first < last) own = pl.block[first];
      mine = own.tiles;
    } else {
      for (int i = first; i < last; ++i) mine += pl.block_tiles[i];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine, per_head = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int v = warp_sum[w];
      before += w < warp ? v : 0;
      per_head += v;
    }
    const int heads = p.num_kv_heads, total = per_head * heads, cta = blockIdx.x;
    const int used = min(pl.ctas, (total + 1) / 2);  // (two tiles go through the two accumulators at a time)
    bool own_runs = per == 1 && static_cast<int64_t>(pl.blocks) * heads <= used && total < kTiles32;
    if (own_runs) {
      const Split split = split_of(mine, total, used);
      const uint32_t worst = __reduce_max_sync(0xffffffffu, split.worst);
      if (lane == 0 && worst > 0) atomicMax(&ctl.worst, worst);
      __syncthreads();
      own_runs = ctl.worst <= split.limit;
    }
    // the thread whose blocks hold the run's first tile
    int lo = 0, hi = 0, hk = -1;
    if (cta >= used) {
      if (tid == 0) pl.info[cta].item = -1;
    } else if (own_runs) {
      const int x = own_probe(cta, total, used), h = x / per_head, at = x - h * per_head;
      if (before <= at && at < before + mine) {
        uint32_t from, to;
        own_run(own, h * per_head + before, cta, total, used, &from, &to);
        hk = h;
        lo = from;
        hi = to;
      }
    } else {
      lo = static_cast<int>(static_cast<int64_t>(total) * cta / used);
      hi = static_cast<int>(static_cast<int64_t>(total) * (cta + 1) / used);
      const int h = lo / per_head, at = lo - h * per_head;
      if (before <= at && at < before + mine) hk = h;
    }
    if (hk >= 0) {
      int i = first;
      if (per > 1) {
        while (hk * per_head + before + pl.block_tiles[i] <= lo) before += pl.block_tiles[i++];
        own = pl.block[i];
      }
      ctl.run_hi = hi;
      begin_run(own, i, hk, hk * per_head + before, lo, per_head);
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  pdl_launch_dependents();  // the join may take its place; it waits for this grid's end

  if (warp == kPlanWarp) {
    // ================================================================ planner
    uint32_t n = 0;  // chunks published
    bool ok = true;
    const int hi = ctl.run_hi, per_head = ctl.per_head;
    int at = ctl.run_lo, hk = ctl.run_hk, block = ctl.run_block, start = ctl.run_start;
    Block b = ctl.first;
    while (ok && at < hi) {
      const int from = at - start, to = min(b.tiles, hi - start);  // tiles of the block
      const bool two = b.pairs > kRows;
      const int segment = (two ? kTwo : 0) | (from == 0 && to == b.tiles ? kWhole : 0);
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
          while (ok && done < s_end) {
            // a lane looks up a tile's pages
            const int most = min(32, s_end - done), pos = pos0 + (done + lane - s_start) * kTile;
            int32_t page[2] = {-1, -1};
            int odd = 0;  // what makes a tile a chunk of its own
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (lane >= most || pos + 64 * r >= k_hi) continue;
              page[r] = __ldg(p.block_table + table + ((pos + 64 * r) >> p.page_shift));
              if (page[r] < 0 || page[r] >= p.num_pages) {
                atomicOr(p.err, kErrPageRange);
                page[r] = -1;
                odd |= r ? kHole1 : kHole0;
              }
            }
            // a run that ends inside: its values may hold anything behind the end
            if (lane < most && k_hi > pos && k_hi < pos + kTile && (k_hi & 63)) odd |= kTail;
            const uint32_t odds = __ballot_sync(0xffffffffu, odd != 0);
            // chunks: up to kChunkTiles tiles, odd ones alone
            for (int first = 0; ok && first < most;) {
              const uint32_t ahead = odds >> first;
              int count = min(kChunkTiles, most - first);
              if (ahead) count = min(count, (ahead & 1) ? 1 : __ffs(ahead) - 1);
              const uint32_t slot = n % kChunks;
              ok = n < kChunks || warp_try(smem_u32(&ctl.cempty[slot]), (n / kChunks - 1) & 1, abort_flag, p.err);
              if (!ok) break;
              Chunk& c = ctl.chunk[slot];
              if (lane >= first && lane < first + count) {
                c.page[lane - first][0] = page[0];
                c.page[lane - first][1] = page[1];
              }
              if (lane == first) {
                const int tile = done + first;
                c.flags = segment | odd | (tile == from ? kFirst : 0) | (tile + count == to ? kLast : 0) | ((tile - from) & 1 ? kOdd : 0) |
                          (p0 < kRows ? kSlot0 : 0) | (p1 > kRows ? kSlot1 : 0);
                c.tiles = count;
                c.pos0 = pos;
                c.lo = k_lo;
                c.hi = k_hi;
                c.p0 = p0;
                c.p1 = p1;
                c.row0 = b.row0;
                c.pair0 = b.pair0;
                c.pairs = b.pairs;
                c.hk = hk;
                c.part = 2 * blockIdx.x + (from == 0);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int r0 = x * kRows, r1 = min(b.pairs, r0 + kRows);
                  c.lanes[x] = p0 <= r0 && p1 >= r1 ? kAllLanes : min(max(p0 - r0, 0), kRows) | min(max(p1 - r0, 0), kRows) << 16;
                }
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&ctl.cfull[slot]));
              ++n;
              first += count;
            }
            done += most;
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
      if (ok) b = pl.block[block];
    }
    if (ok) {
      const uint32_t slot = n % kChunks;
      ok = n < kChunks || warp_try(smem_u32(&ctl.cempty[slot]), (n / kChunks - 1) & 1, abort_flag, p.err);
      if (ok && lane == 0) {
        ctl.chunk[slot].flags = kEnd;
        mbar_arrive(smem_u32(&ctl.cfull[slot]));
      }
    }
    clear_other_rows(sp, lane);
  } else if (warp == kLoadWarp) {
    // ================================================================ loader
    uint32_t issued = 0;  // stages
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t slot = n % kChunks;
      ok = warp_try(smem_u32(&ctl.cfull[slot]), (n / kChunks) & 1, abort_flag, p.err);
      if (!ok) break;
      const Chunk& c = ctl.chunk[slot];
      if (c.flags & kEnd) break;
      const int tiles = c.tiles, pos0 = c.pos0, hi = c.hi, head = c.hk * p.page_size;
      const bool tails = c.flags & kTail;
      const int32_t beyond = static_cast<int32_t>(p.num_pages);  // past the cache: zeros
      for (int i = 0; ok && i < tiles; ++i) {
        const int pos = pos0 + i * kTile;
        const int r = lane & 1, row = head + ((pos + 64 * r) & (p.page_size - 1));  // lanes 0-3: run, piece
        const int32_t here = c.page[i][r], page = here < 0 ? beyond : here;
#pragma unroll
        for (int v = 0; v < 2; ++v) {  // keys, values
          const uint32_t st = issued % kStages, bar = smem_u32(&ctl.kfull[st]), dst = base + st * kStage;
          ok = issued < kStages || warp_try(smem_u32(&ctl.kempty[st]), (issued / kStages - 1) & 1, abort_flag, p.err);
          if (!ok) break;
          if (v == 0) {
            if (lane == 0) mbar_arrive_expect_tx(bar, kStage);
            __syncwarp();
            if (lane < 4) tma_load_4d(dst + (lane >> 1) * kPiece + r * kRun, &maps.k, 0, row, lane >> 1, page, bar);
          } else {
            // Of a run that ends inside 16 keys at a time, as the products take
            // them: the whole ones by TMA, the last by copies with zeros behind
            // the end.  (All 64 by copies kept the loader for 1,850 cycles: 15.0
            // for 13.7 us with two requests, 96.3 for 94.7 with 486 ends of requests.)
            int tail = tails ? (hi - pos) >> 6 : -1, whole = 0;
            if (tail >= 0) {
              const int32_t its = __shfl_sync(0xffffffffu, here, tail), at = __shfl_sync(0xffffffffu, row, tail);
              if (its < 0) {
                tail = -1;  // zeros, like any page that is not there
              } else {
                const int keys = hi - pos - 64 * tail;
                const uint32_t to = dst + tail * 2 * kRun;
                whole = keys >> 4;
                if (keys & 15) {
                  const int u = lane & 7, piece = (lane >> 3) & 1, k0 = 16 * whole + (lane >> 4);  // 16-byte unit; row
                  const uint16_t* src = p.v + its * p.page_stride + static_cast<int64_t>(at) * kPagedDim + piece * 64 + u * 8;
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const int k = k0 + 2 * j;
                    cp_async_16_or_zero(to + piece * kRun + k * 128 + ((u ^ (k & 7)) << 4), src + (k < keys ? k : 0) * kPagedDim, k < keys);
                  }
                  cp_async_arrive_extra(bar);
                  __syncwarp();
                }
                if (lane == 0) mbar_arrive_expect_tx(bar, kStage / 2 + whole * (16 * 2 * 128));
                __syncwarp();
                if (lane < 2 * whole)
                  tma_load_4d(to + (lane & 1) * kRun + (lane >> 1) * (16 * 128), &maps.v_part, 0, at + (lane >> 1) * 16, lane & 1, its, bar);
              }
            }
            if (tail < 0 && lane == 0) mbar_arrive_expect_tx(bar, kStage);
            __syncwarp();
            if (lane < 2 && lane != tail) tma_load_4d(dst + lane * 2 * kRun, &maps.v, 0, row, 0, page, bar);
          }
          ++issued;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.cempty[slot]));
    }
    cp_async_wait_all();
    if (!ok && lane == 0) {  // after a time-out: what was issued lands before the CTA can exit
      int never = 0;
      for (uint32_t x = issued; x > 0 && x + kStages > issued; --x)
        mbar_wait(smem_u32(&ctl.kfull[(x - 1) % kStages]), ((x - 1) / kStages) & 1, &never, p.err);
    }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // ================================================================ MMA issuers
    // A warp issues the products of one accumulator: a tile's value product and
    // the next tile's score product together.  The score product may overwrite P
    // where the value product before it reads it, since one thread's products
    // are carried out in order.  The two warps take turns, tile by tile: left
    // to themselves they fall into step, both accumulators in the softmax at one
    // time and both in the tensor pipe at the other (3,900 cycles a tile; in
    // turn, one's softmax runs beside the other's products).
    const uint32_t tm = uniform(tmem), acc = uniform(warp - kMmaWarp);
    const uint32_t s_idesc = uniform(idesc_f16(128, 128, DTYPE == FP4IDX_BF16, false, p.negate != 0));
    const uint32_t o_idesc = uniform(idesc_f16(128, 128, DTYPE == FP4IDX_BF16, false, false) | 1u << 16);
    const uint32_t s_tmem = tm + acc * kTile, o_tmem = tm + kOCol + acc * kTile;
    const uint32_t my_turn = smem_u32(&ctl.turn[acc]), its_turn = smem_u32(&ctl.turn[acc ^ 1]);
    const uint32_t p_bar = smem_u32(&ctl.pfull[acc]), s_bar = smem_u32(&ctl.sfull[acc]);
    uint32_t tile = 0, segs = 0, steps = 0;  // tiles and segments begun; value products issued
    uint32_t turns = 0;
    bool ok = true;
    // A tile whose value product is to come: its number, its values' stage,
    // whether copies filled it, its keys by 16 (what lies behind them may be
    // anything), the rows that it counts for and whether its product adds to the
    // output.
    bool open = false;
    uint32_t open_tile = 0, v_st = 0, v_use = 0, v_tail = 0, v_steps = 0, v_lanes = kAllLanes, more = 0;
    uint32_t begun = 0;                      // this accumulator's output has values of the segment, or zeros
    const auto values = [&] {
      const uint64_t v = desc_sw128(base + v_st * kStage, kRun);
      if (v_steps == 8 && v_lanes == kAllLanes) {  // (a test in front of each product instead took 2 % of a long prefill)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          tc_mma_f16_tmem(o_tmem, s_tmem + (x >> 2) * kHalf + (x & 3) * 8, v + (x >> 2) * (2 * kRun >> 4) + (x & 3) * 128, o_idesc, x > 0 ? 1u : more);
      } else {
#pragma unroll 1
        for (uint32_t x = 0; x < v_steps; ++x)
          tc_mma_f16_tmem_lanes(o_tmem, s_tmem + (x >> 2) * kHalf + (x & 3) * 8, v + (x >> 2) * (2 * kRun >> 4) + (x & 3) * 128, o_idesc,
                                x > 0 ? 1u : more, v_lanes & 0xffff, v_lanes >> 16);
      }
      tc_commit(smem_u32(&ctl.kempty[v_st]));
    };
    const auto wait_weights = [&] {  // of the open tile, and its values
      ok = ok && warp_try(smem_u32(&ctl.kfull[v_st]), v_use & 1, abort_flag, p.err);
      if (v_tail) fence_proxy_async_smem();
      ok = ok && warp_try(p_bar, steps & 1, abort_flag, p.err);
      ++steps;
      tc_fence_after();
    };
    // Waits for this warp's turn, and behind it for the weights: they come
    // latest when all runs smoothly.
    const auto wait_turn = [&](bool product) {
      if (acc == 1 || turns > 0) ok = ok && warp_try(my_turn, (turns - (acc ^ 1)) & 1, abort_flag, p.err);
      ++turns;  // (the other's first turn is behind this one's first)
      if (product) wait_weights();
      tc_fence_after();
    };
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t slot = n % kChunks;
      ok = warp_try(smem_u32(&ctl.cfull[slot]), (n / kChunks) & 1, abort_flag, p.err);
      if (!ok) break;
      const uint32_t flags = uniform(ctl.chunk[slot].flags), tiles = uniform(ctl.chunk[slot].tiles);
      const int chunk_keys = uniform(ctl.chunk[slot].hi - ctl.chunk[slot].pos0);
      const uint32_t lanes = uniform(ctl.chunk[slot].lanes[flags & kTwo ? acc : 0]);
      __syncwarp();
      if (flags & kEnd) break;
      if (lane == 0) mbar_arrive(smem_u32(&ctl.cempty[slot]));
      const bool two = flags & kTwo;
      if (flags & kFirst) {
        // (once a tile is for all of an accumulator's rows, the ones behind it are, too)
        begun = lanes != kAllLanes;
        ok = warp_try(smem_u32(&ctl.qfull[0]), segs & 1, abort_flag, p.err);
        if (acc == 1) ok = ok && warp_try(smem_u32(&ctl.qfull[1]), segs & 1, abort_flag, p.err);
        ++segs;
      }
      const uint64_t q = desc_sw128(base + kOff_Q + (two ? acc * kQBytes : 0), 16);
#pragma unroll 1
      for (uint32_t i = 0; ok && i < tiles; ++i, ++tile) {
        const bool mine = two ? flags & (acc ? kSlot1 : kSlot0) : (((flags & kOdd ? 1 : 0) + i) & 1) == acc;
        const uint32_t k_st = uniform(2 * tile % kStages), k_use = 2 * tile / kStages;
        const uint32_t next_v = uniform((2 * tile + 1) % kStages), next_use = (2 * tile + 1) / kStages;
        // A value product is issued with its accumulator's next score product,
        // unless the keys are what all wait for.
        if (open && !__any_sync(0xffffffffu, mbar_test_wait(smem_u32(&ctl.kfull[k_st]), k_use & 1))) {
          wait_weights();
          if (!ok) break;
          if (elect_one()) values();
          __syncwarp();
          open = false;
        }
        if (!mine) {
          // (nor so long that the loader runs out of stages)
          const bool close = open && tile - open_tile >= 2;
          wait_turn(close);
          if (!ok) break;
          if (elect_one()) {
            if (close) values();
            mbar_arrive(its_turn);
          }
          __syncwarp();
          if (close) open = false;
          // (its arrivals are for this use of the stages, so it waits for them)
          ok = warp_try(smem_u32(&ctl.kfull[k_st]), k_use & 1, abort_flag, p.err) &&
               warp_try(smem_u32(&ctl.kfull[next_v]), next_use & 1, abort_flag, p.err);
          if (lane == 0) {
            mbar_arrive(smem_u32(&ctl.kempty[k_st]));
            mbar_arrive(smem_u32(&ctl.kempty[next_v]));
          }
          continue;
        }
        ok = warp_try(smem_u32(&ctl.kfull[k_st]), k_use & 1, abort_flag, p.err);
        const bool was_open = open;
        wait_turn(was_open);
        if (!ok) break;
        if (elect_one()) {
          if (was_open) values();
          const uint64_t k = desc_sw128(base + k_st * kStage, 16);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int at = (x >> 2) * (kPiece >> 4) + (x & 3) * 2;
            tc_mma_f16(s_tmem, q + at, k + at, s_idesc, x > 0);
          }
          mbar_arrive(its_turn);
          tc_commit(s_bar);
          tc_commit(smem_u32(&ctl.kempty[k_st]));
        }
        __syncwarp();
        more = begun;
        begun = 1;
        open = true;
        open_tile = tile;
        v_st = next_v;
        v_use = next_use;
        v_tail = flags & kTail;
        v_lanes = lanes;
        v_steps = min(max(chunk_keys - static_cast<int>(i) * kTile + 15, 16) >> 4, 8);
      }
      if (ok && (flags & kLast)) {
        const bool was_open = open;
        wait_turn(was_open);
        if (!ok) break;
        if (elect_one()) {
          if (was_open) values();
          mbar_arrive(its_turn);
          tc_commit(smem_u32(&ctl.odone[acc]));
        }
        __syncwarp();
        open = false;
      }
    }
    // no product is in flight when TMEM is freed
    if (elect_one()) tc_commit(smem_u32(&ctl.drain));
    __syncwarp();
    if (lane == 0) {
      int never = 0;
      mbar_wait(smem_u32(&ctl.drain), 0, &never, p.err);
    }
    __syncwarp();
  } else {
    // ================================================================ softmax
    // After a failed wait a chunk's tiles are walked without waiting, so that
    // the named barriers still meet; nothing is written then.
    const int acc = warp / kSoftmaxWarps, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;  // accumulator, keys and columns of it, row
    const uint32_t pair_bar = 1 + acc * 4 + (warp & 3);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_at = tmem + lanes + acc * kTile + half * kHalf, o_at = tmem + lanes + kOCol + acc * kTile + half * kHalf;
    uint32_t segs = 0, steps = 0;   // segments begun; tiles of this accumulator
    uint32_t merged = 0;            // segments whose two accumulators were added up
    bool merging = false;           // the last one was
    int steps_of_seg = 0;
    int vis = 0;                    // of this thread's row
    bool valid = false, ok = true;
    float m = -INFINITY;            // the row's reference, in powers of two
    float l = 0.0f;                 // this thread's share of the sum
    // The 32 rows of this warp in its half of the queries' buffer: rows of 128
    // bytes, 16-byte units swizzled.
    uint8_t* const my_rows = smem + kOff_Q + acc * kQBytes + half * kPiece + (warp & 3) * 32 * 128;
    const auto unit_at = [](int row, int unit) { return (unit ^ (row & 7)) << 4; };
    // This warp's part of a segment's queries, and what its rows see.
    const auto load_queries = [&](int row0, int pair0, int pairs, int hk, bool two) {
      // (the products that read the queries before are done: this warp has
      // waited for its own, and through mfull for the other issuer's)
      const int off = two ? acc * kRows : 0, pair = pair0 + off + r, t = row0 + group_div(p, pair);
      valid = off + r < pairs;
      if (valid) vis = pl.row_vis[t];
      if (acc == 0 || two) {
        // eight lanes a row: a warp's load touches four lines (with a row a lane
        // it touched 32, and 256 rows took 7,000 cycles)
        const int h = hk * p.group + pair - group_div(p, pair) * p.group;
        const int64_t from = valid ? t * p.q_row_stride + h * p.q_head_stride : -1;
        uint4 q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t at = __shfl_sync(0xffffffffu, from, 4 * u + (lane >> 3));
          q[u] = at < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(p.q + at) + half * 8 + (lane & 7));
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) *reinterpret_cast<uint4*>(my_rows + (4 * u + (lane >> 3)) * 128 + unit_at(4 * u + (lane >> 3), lane & 7)) = q[u];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.qfull[acc]));
    };
    // (the first segment's without waiting for the planner)
    if (ctl.run_lo < ctl.run_hi) load_queries(ctl.first.row0, ctl.first.pair0, ctl.first.pairs, ctl.run_hk, ctl.first.pairs > kRows);
    for (uint32_t n = 0;; ++n) {
      const uint32_t slot = n % kChunks;
      ok = ok && warp_try(smem_u32(&ctl.cfull[slot]), (n / kChunks) & 1, abort_flag, p.err);
      if (bar_red_or(pair_bar, 64, !ok)) break;
      const Chunk& d = ctl.chunk[slot];
      const int flags = d.flags;
      if (flags & kEnd) break;
      const bool two = flags & kTwo;
      const int off = two ? acc * kRows : 0;  // first pair of this accumulator
      if (flags & kFirst) {
        if (segs > 0) load_queries(d.row0, d.pair0, d.pairs, d.hk, two);
        // the other accumulator's warps have read this one's output and sums
        if (acc == 1 && merging) ok = warp_try(smem_u32(&ctl.mfree), (merged - 1) & 1, abort_flag, p.err);
        // a product of some rows does not begin the others' output
        if (d.lanes[two ? acc : 0] != kAllLanes) {
          tc_fence_after();
          const uint32_t none[16] = {};
#pragma unroll
          for (int c = 0; c < kHalf; c += 16) tmem_st_x16(o_at + c, none);
        }
        ++segs;
        steps_of_seg = 0;
        m = -INFINITY;
        l = 0.0f;
      }
      const int tiles = d.tiles;
      const bool mine = valid && off + r >= d.p0 && off + r < d.p1;
      // keys [lo, hi) count for this row, relative to the chunk's first
      int lo = d.lo - d.pos0, hi = mine ? min(vis, d.hi) - d.pos0 : 0;
      if (flags & kHole0) lo = max(lo, kHalf);
      if (flags & kHole1) hi = min(hi, kHalf);
      const int turn = flags & kOdd ? 1 : 0;
      const bool active = !two || (flags & (acc ? kSlot1 : kSlot0));
#pragma unroll 1
      for (int i = two ? 0 : turn ^ acc; active && i < tiles; i += two ? 1 : 2) {
        // keys [k_lo, k_lo + k_len) of the tile count
        const int k_lo = max(0, lo - i * kTile), k_len = max(0, min(hi - i * kTile, kTile) - k_lo);
        const bool some = __any_sync(0xffffffffu, k_len > 0), full = __all_sync(0xffffffffu, k_len == kTile);
        bool raise = k_len > 0 && m == -INFINITY;  // (alike in the two threads of a row)
        bool again = __any_sync(0xffffffffu, raise);
        if (ok) ok = warp_try(smem_u32(&ctl.sfull[acc]), steps & 1, abort_flag, p.err);
        tc_fence_after();
        if (some) {
          const auto masked = [&](uint32_t (&x)[32], int c) {
            if (full) return;
            // a bit for each of the columns from c on; the empty asm keeps the
            // tests of all columns from being worked out (and spilled) at once
            const int at = half * kHalf + c, from = min(max(k_lo - at, 0), 32), to = min(max(k_lo + k_len - at, 0), 32);
            uint32_t bits = static_cast<uint32_t>((uint64_t{1} << to) - 1) & ~static_cast<uint32_t>((uint64_t{1} << from) - 1);
            asm volatile("" : "+r"(bits));
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(bits >> k & 1)) x[k] = 0xff800000u;  // -inf
          };
          uint32_t w[kHalf / 2];
          float sum = 0.0f;
#pragma unroll 1
          for (bool once = false;; once = true) {
            if (again) {  // a new reference
              float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
              for (int c = 0; c < kHalf; c += 32) {
                uint32_t x[32];
                tmem_ld(s_at + c, x);
                tmem_wait_ld();
                reg_fence(x);
                masked(x, c);
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                  top[k / 2 & 3] = fmaxf(fmaxf(top[k / 2 & 3], __uint_as_float(x[k])), __uint_as_float(x[k + 1]));
              }
              // the row's, and whether either of its threads asked for it
              const float mine_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.scale_log2 - kBelow<DTYPE>;
              bar_sync(pair_bar, 64);  // what was exchanged before has been read
              ctl.row[acc][half][r] = mine_top;
              bar_sync(pair_bar, 64);
              const float most = fmaxf(mine_top, ctl.row[acc][half ^ 1][r]);
              const float f = most > m ? ex2(m - most) : 1.0f;
              // a row without a reference has weights and an output of zero so far
              const bool grown = __any_sync(0xffffffffu, most > m && m != -INFINITY);
              if (most > m) m = most;
              l *= f;
              if (grown && steps_of_seg > 0) {  // (the score product came behind the last value product)
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 16) {
                  uint32_t o[16];
                  tmem_ld(o_at + c, o);
                  tmem_wait_ld();
                  reg_fence(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st_x16(o_at + c, o);
                }
                tmem_wait_st();
              }
            }
            // weights, their sum in fp32, and P in 16 bits (the MMA's operand type:
            // each weight is rounded once, the sum is of unrounded ones)
            const float2 scale = make_float2(p.scale_log2, p.scale_log2);
            const float2 ref = m == -INFINITY ? make_float2(0.0f, 0.0f) : make_float2(-m, -m);
            float2 part[2] = {};
#pragma unroll
            for (int c = 0; c < kHalf; c += 32) {
              uint32_t x[32];
              tmem_ld(s_at + c, x);
              tmem_wait_ld();
              reg_fence(x);
              masked(x, c);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float2 a = fma2(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), scale, ref);
                a = make_float2(ex2(a.x), ex2(a.y));
                part[k & 1] = add2(part[k & 1], a);
                w[c / 2 + k] = pack2<DTYPE>(a.x, a.y);
              }
            }
            sum = (part[0].x + part[1].x) + (part[0].y + part[1].y);
            again = !once && bar_red_or(pair_bar, 64, sum > kLimit<DTYPE>);
            if (!again) break;
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < kHalf / 2; c += 16) {
            uint32_t v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = w[c + k];
            tmem_st_x16(s_at + c, v);
          }
        } else {  // none of the warp's rows sees a key of this tile
          uint32_t w[16] = {};
#pragma unroll
          for (int c = 0; c < kHalf / 2; c += 16) tmem_st_x16(s_at + c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.pfull[acc]));
        ++steps;
        ++steps_of_seg;
      }
      if (flags & kLast) {
        // ---- output of the segment
        bar_sync(pair_bar, 64);  // what was exchanged before has been read
        ctl.row[acc][half][r] = l;
        bar_sync(pair_bar, 64);
        float sum = ctl.row[acc][0][r] + ctl.row[acc][1][r];
        if (ok) ok = warp_try(smem_u32(&ctl.odone[acc]), (segs - 1) & 1, abort_flag, p.err);
        tc_fence_after();
        merging = !two;
        if (merging && acc == 1) {  // the other accumulator's warps add this one up
          bar_sync(pair_bar, 64);
          ctl.row[1][half][r] = half ? sum : m;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.mfull));
        } else {
          // out = f0 O (+ f1 O of the other accumulator)
          float f0 = steps_of_seg > 0 ? 1.0f : 0.0f, f1 = 0.0f;
          if (merging) {
            if (ok) ok = warp_try(smem_u32(&ctl.mfull), merged & 1, abort_flag, p.err);
            tc_fence_after();
            const float m1 = ctl.row[1][0][r], l1 = ctl.row[1][1][r];
            const float top = fmaxf(m, m1), at = top == -INFINITY ? 0.0f : top;
            f0 = ex2(m - at);  // (accumulator 0 takes a segment's first tile)
            f1 = ex2(m1 - at);
            sum = f0 * sum + f1 * l1;
            m = top;
          }
          const bool both = merging && __any_sync(0xffffffffu, f1 != 0.0f);
          const int pair = d.pair0 + off + r, t = d.row0 + group_div(p, pair), h = d.hk * p.group + pair - group_div(p, pair) * p.group;
          const bool whole = flags & kWhole;
          if (whole) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            f0 = sum == 0.0f ? 0.0f : f0 * inv;
            f1 *= inv;
          }
          const int row = off + r;  // of the block
          const int64_t to = valid && ok ? t * p.out_row_stride + static_cast<int64_t>(h) * kPagedDim + half * kHalf : -1;
          float4* part = pl.partial + (static_cast<int64_t>(d.part) * (kPagedDim / 4) + half * (kHalf / 4)) * kBlockPairs + row;
#pragma unroll 1
          for (int c = 0; c < kHalf; c += 16) {
            uint32_t o[16];
            __syncwarp();
            tmem_ld(o_at + c, o);
            tmem_wait_ld();
            reg_fence(o);
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = f0 == 0.0f ? 0.0f : __uint_as_float(o[e]) * f0;
            if (both) {
              tmem_ld(o_at + kTile + c, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = f1 == 0.0f ? y[e] : fmaf(__uint_as_float(o[e]), f1, y[e]);
            }
            if (whole) {  // rounded, into the queries' place, which is free now
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                *reinterpret_cast<uint4*>(my_rows + lane * 128 + unit_at(lane, (c + e) / 8)) =
                    make_uint4(pack2<DTYPE>(y[e], y[e + 1]), pack2<DTYPE>(y[e + 2], y[e + 3]), pack2<DTYPE>(y[e + 4], y[e + 5]),
                               pack2<DTYPE>(y[e + 6], y[e + 7]));
            } else if (valid && ok) {
#pragma unroll
              for (int e = 0; e < 16; e += 4) part[(c + e) / 4 * kBlockPairs] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
          }
          if (whole) {  // and out, eight lanes a row
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int row_u = 4 * u + (lane >> 3);
              const int64_t at = __shfl_sync(0xffffffffu, to, row_u);
              const uint4 v = *reinterpret_cast<const uint4*>(my_rows + row_u * 128 + unit_at(row_u, lane & 7));
              if (at >= 0) *(reinterpret_cast<uint4*>(p.out + at) + (lane & 7)) = v;
            }
            __syncwarp();
          }
          if (valid && ok && half == 0) {
            if (!whole) pl.stats[static_cast<int64_t>(d.part) * kBlockPairs + row] = make_float2(m, sum);
            else if (p.lse) p.lse[static_cast<int64_t>(t) * p.num_heads + h] = row_lse(m, sum);
          }
          tc_fence_before();
          __syncwarp();
          if (merging && lane == 0) mbar_arrive(smem_u32(&ctl.mfree));
        }
        merged += merging;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.cempty[slot]));
    }
    tmem_wait_st();  // (zeros of an accumulator without a tile)
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
// a block that crosses run boundaries, in the order of its tiles.  A lane has a
// row.  With few parts (BY_ITEM false: blockIdx.x counts run boundaries, the
// first one inside a block does its work) a warp adds all of them for 32 columns;
// with many (BY_ITEM: blockIdx.x is the block of a K/V head) a CTA's warps take
// parts in turn for 16 columns, several parts' loads together, and are added in
// order.  Bound by the round trips to L2: with a part of 32 columns at a time a
// block of 25 parts took 42.0 us in all, in this way 37.2; in 16 columns calls of
// two or three parts only have more CTAs (82.1 for 81.6, 35.6 for 34.4 us).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

template <int DTYPE, bool BY_ITEM>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Plan pl) {
  constexpr int kCols = BY_ITEM ? 16 : 32, kFours = kCols / 4, kUnits = kCols / 8, kParts = BY_ITEM ? 4 : 1;
  __shared__ float4 sums[BY_ITEM ? kJoinWarps : 1][kFours][32];
  __shared__ float2 part[kJoinWarps][32];
  __shared__ uint4 staged[BY_ITEM ? 1 : kJoinWarps][32 * kUnits];
  __shared__ RunInfo its;
  __shared__ int first_cta;
  pdl_wait();
  pdl_launch_dependents();
  const AttnParams& p = pl.sp.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // a CTA of the first kernel per thread (plan_shared)
  RunInfo info = {};
  info.item = -1;
  if (tid < pl.ctas) info = pl.info[tid];
  const int item = BY_ITEM ? blockIdx.x : pl.info[blockIdx.x + 1].item;
  if (tid == 0) first_cta = INT32_MAX;
  __syncthreads();
  // the CTAs whose run begins inside the block: consecutive ones
  const bool inside = tid > 0 && info.item == item && info.inside;
  if (inside) atomicMin(&first_cta, tid);
  const int parts = 1 + __syncthreads_count(inside);
  const int c = first_cta;  // the first boundary; the part before it is the previous CTA's
  if (item < 0 || parts == 1 || (!BY_ITEM && c != static_cast<int>(blockIdx.x) + 1)) return;
  if (tid == c) its = info;
  __syncthreads();
  const int row = (BY_ITEM ? blockIdx.y : blockIdx.y * 2 + (warp >> 2)) * 32 + lane, cols = (BY_ITEM ? blockIdx.z : warp & 3) * kCols;
  if (row - lane >= its.pairs) return;  // (BY_ITEM: the whole CTA)
  float4 acc[kFours] = {};
  float m = -INFINITY, l = 0.0f;
  constexpr int step = BY_ITEM ? kJoinWarps : 1;
#pragma unroll (BY_ITEM ? 1 : 2)
  for (int i0 = BY_ITEM ? warp : 0; i0 < parts; i0 += kParts * step) {
    float2 s[kParts];
    float4 o[kParts][kFours];
#pragma unroll
    for (int b = 0; b < kParts; ++b) {
      // part i is CTA c - 1 + i's; of the first one its last segment, of the others
      // their first (behind the last part: the last one, which does not count)
      const int i = min(i0 + b * step, parts - 1);
      const int64_t at = 2 * (c - 1 + i) + (i == 0);
      s[b] = pl.stats[at * kBlockPairs + row];
#pragma unroll
      for (int v = 0; v < kFours; ++v) o[b][v] = pl.partial[(at * (kPagedDim / 4) + cols / 4 + v) * kBlockPairs + row];
    }
#pragma unroll
    for (int b = 0; b < kParts; ++b) {
      if (i0 + b * step >= parts) break;
      const float top = fmaxf(m, s[b].x), ref = top == -INFINITY ? 0.0f : top;
      const float keep = ex2(m - ref), w = ex2(s[b].x - ref);
      m = top;
      l = l * keep + w * s[b].y;
#pragma unroll
      for (int v = 0; v < kFours; ++v) {
        acc[v].x = acc[v].x * keep + w * o[b][v].x;
        acc[v].y = acc[v].y * keep + w * o[b][v].y;
        acc[v].z = acc[v].z * keep + w * o[b][v].z;
        acc[v].w = acc[v].w * keep + w * o[b][v].w;
      }
    }
  }
  if constexpr (BY_ITEM) {
#pragma unroll
    for (int v = 0; v < kFours; ++v) sums[warp][v][lane] = acc[v];
    part[warp][lane] = make_float2(m, l);
    __syncthreads();
    // warp v adds the warps' shares of four columns
    m = part[0][lane].x;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, part[w][lane].x);
    const float ref = m == -INFINITY ? 0.0f : m;
    l = 0.0f;
    acc[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float4 o = sums[w][warp % kFours][lane];
      const float f = ex2(part[w][lane].x - ref);
      l = fmaf(f, part[w][lane].y, l);
      acc[0].x = fmaf(f, o.x, acc[0].x);
      acc[0].y = fmaf(f, o.y, acc[0].y);
      acc[0].z = fmaf(f, o.z, acc[0].z);
      acc[0].w = fmaf(f, o.w, acc[0].w);
    }
  }
  // Out by whole 32-byte sectors: a warp's 32 rows x 64 bytes (BY_ITEM: the
  // CTA's 32 rows x 32).  (Eight bytes a lane, as they come, took twice as long
  // as all the rest.)
  const bool have = row < its.pairs;
  const int pair = its.pair0 + row, t = its.row0 + group_div(p, pair);
  const int h = its.hk * p.group + pair - group_div(p, pair) * p.group;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t to = have ? t * p.out_row_stride + static_cast<int64_t>(h) * kPagedDim + cols : -1;
  if (p.lse && have && cols == 0 && (!BY_ITEM || warp == 0)) p.lse[static_cast<int64_t>(t) * p.num_heads + h] = row_lse(m, l);
  uint4* const rows = staged[BY_ITEM ? 0 : warp];
  if constexpr (BY_ITEM) {
    if (warp < kFours)
      reinterpret_cast<uint2*>(rows)[lane * 4 + warp] = make_uint2(pack2<DTYPE>(acc[0].x * inv, acc[0].y * inv), pack2<DTYPE>(acc[0].z * inv, acc[0].w * inv));
    __syncthreads();
    if (warp > 0) return;
  } else {
#pragma unroll
    for (int v = 0; v < kFours; v += 2)
      rows[lane * kUnits + ((v / 2) ^ (lane >> 1 & 3))] =
          make_uint4(pack2<DTYPE>(acc[v].x * inv, acc[v].y * inv), pack2<DTYPE>(acc[v].z * inv, acc[v].w * inv),
                     pack2<DTYPE>(acc[v + 1].x * inv, acc[v + 1].y * inv), pack2<DTYPE>(acc[v + 1].z * inv, acc[v + 1].w * inv));
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int row_i = (i * 32 + lane) / kUnits, unit = lane % kUnits;
    const int64_t at = __shfl_sync(0xffffffffu, to, row_i);
    const uint4 v = rows[row_i * kUnits + (BY_ITEM ? unit : unit ^ (row_i >> 1 & 3))];
    if (at >= 0) *(reinterpret_cast<uint4*>(p.out + at) + unit) = v;
  }
}

// ---------------------------------------------------------------- host
int64_t round16(int64_t n) { return (n + 15) & ~int64_t{15}; }

// Tiles that a call can have over all K/V heads: a span is what a block has of
// one request or of the prefix.
int64_t most_tiles(const SharedParams& p) {
  const int64_t tiles = (static_cast<int64_t>(p.a.max_seqlen_k) + 63) / kTile + 1;
  const int64_t of_head = tiles * (2 * static_cast<int64_t>(p.blocks_per_group) * p.num_groups + p.a.num_seqs);
  return of_head > INT32_MAX ? of_head : of_head * p.a.num_kv_heads;
}

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
  pl.few = pl.blocks <= 32 && most_tiles(p) < kTiles32;
  return pl;
}

template <int DTYPE>
cudaError_t launch(const Plan& pl, const SharedMaps& maps, cudaStream_t stream) {
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
  // can a block have more than 32 requests with rows, and has a group as many on average?
  const bool wide = pl.sp.a.group < kBlockPairs / 32 && pl.sp.a.num_seqs > 32 * static_cast<int64_t>(pl.sp.num_groups);
  cfg.gridDim = dim3(static_cast<unsigned>(wide ? pl.blocks : (pl.blocks + kPlanWarps - 1) / kPlanWarps));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, wide ? plan_kernel<true> : plan_kernel<false>, pl)) != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(pl.ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  if ((e = cudaLaunchKernelEx(&cfg, shared_kernel<DTYPE>, pl, maps)) != cudaSuccess) return e;
  if (pl.ctas < 2) return cudaSuccess;
  // rows that a block can have, and more than four parts of each on average?
  const int64_t pairs = static_cast<int64_t>(pl.sp.max_group_rows) * pl.sp.a.group;
  const unsigned rows = static_cast<unsigned>(std::min<int64_t>(pairs, kBlockPairs));
  const int64_t items = static_cast<int64_t>(pl.blocks) * pl.sp.a.num_kv_heads;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  if (pl.ctas > 4 * items) {
    cfg.gridDim = dim3(static_cast<unsigned>(items), (rows + 31) / 32, kPagedDim / 16);
    return cudaLaunchKernelEx(&cfg, join_kernel<DTYPE, true>, pl);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(pl.ctas - 1), (rows + 63) / 64);
  return cudaLaunchKernelEx(&cfg, join_kernel<DTYPE, false>, pl);
}

}  // namespace

bool plan_shared(SharedParams* p, int sms) {
  AttnParams& a = p->a;
  a.group_mul = ((uint64_t{1} << kGroupShift) + a.group - 1) / a.group;
  p->max_group_rows = std::min(p->max_group_rows, a.num_rows);
  const int64_t pairs = static_cast<int64_t>(p->max_group_rows) * a.group;
  const int64_t per = (pairs + kBlockPairs - 1) / kBlockPairs, blocks = per * p->num_groups;
  if (blocks > 1 << 20) return false;
  p->blocks_per_group = static_cast<int32_t>(per);
  const int64_t tiles = most_tiles(*p);
  if (tiles > INT32_MAX) return false;
  // (the join looks at one CTA per thread)
  p->ctas = static_cast<int32_t>(std::min<int64_t>(std::min(sms, kJoinThreads), tiles));
  return true;
}

size_t shared_workspace(const SharedParams& p) {
  Plan pl = plan_of(p);
  return lay_out(&pl, nullptr);
}

cudaError_t launch_shared(SharedParams p, const SharedMaps& maps, int dtype, void* workspace, cudaStream_t stream) {
  Plan pl = plan_of(p);
  lay_out(&pl, static_cast<char*>(workspace));
  return dtype == FP4IDX_BF16 ? launch<FP4IDX_BF16>(pl, maps, stream) : launch<FP4IDX_FP16>(pl, maps, stream);
}

}  // namespace fp4idx
