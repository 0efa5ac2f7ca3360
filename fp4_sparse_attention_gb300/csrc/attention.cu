// attention.cu -- attention over the 16-bit paged caches for sm_103a
// (fp4idx_latent_attention, fp4idx_paged_attention).
//
//   s(r, j) = scale * q[r] . k[j],   out[r] = sum_j exp(s - lse) v[j]
//
// One CTA owns up to 64 query rows that share their keys -- the (row, head)
// pairs of one request and K/V head, or of one row when every row has its own
// selection -- and walks the keys in tiles, with a running maximum and sum:
//
//   S   [64 rows x TK keys]  = Q K^T     tcgen05, M = 64 rows, N = TK keys
//   P   = 2^(S - m)                      registers, rounded to 16 bits once
//   O^T [dv x 64 rows]      += V^T P^T   tcgen05, M = 128 of dv, N = rows
//
// The second product is transposed so that M is the value dimension: M = 64
// runs at half of the tensor pipe's rate, and O^T of 512 values x 64 rows
// takes 256 TMEM columns where O would take all 512.  Both operands of both
// products come from one copy of the keys in shared memory: a key's row lies
// in 128-byte swizzled pieces of 64 values, which is the K-major layout Q K^T
// wants and, read along the other axis, the MN-major layout V^T wants; for
// the latent cache K and V are even the same bytes.
//
// A latent tile takes 74 KB, so a ring of three leaves no room for 74 KB of
// queries: 512 of their 576 values lie in TMEM, half of them in each half of
// the lanes that M = 64 leaves free (two accumulators, added by the softmax),
// the rotary ones in shared memory, and the weights take the place of the
// tile's rotary piece, which only the score product reads.  With two stages
// (queries in shared memory) neither loads nor softmax could be hidden: a tile
// took 3,200 cycles, now 2,200, of which the products fill 1,900.
//
// Roles (one CTA per SM):
//   warps 0-3   softmax: TMEM S as row fragments (four lanes per row), mask,
//               running maximum, 2^x, P to shared memory; rescale of O^T when
//               a row's maximum grew by more than 2^8 (until then the older
//               maximum serves as the reference: weights stay below 2^8, in
//               fp16 2^15, and the result is the same up to rounding); the output.
//   warp 4, 5   MMA issuers of the score and the value products.
//   warps 6-    loaders: a 64-key run of one page by TMA; listed keys, and a
//               run that a request ends in, by 16-byte asynchronous copies
//               (zeros for keys that do not exist); key positions; queries.  A
//               gather of four rows by TMA (tile::gather4) moves 512 bytes an
//               instruction and reached 6.7-8.7 TB/s from L2 where the copies
//               reach 20.
//   last warp   planner: the segments (runs of one item's tiles) to come.
// A tile arrives and leaves in parts (latent: three times 192 of the 576
// values; paged: keys, values): the score product starts with the first part
// and a part is loaded again as soon as its last product is done.  A latent
// segment's queries pass through a place of the ring like a tile and are
// copied to TMEM from there, so they load while the segment before computes.
//
// Work split: the tiles of all items (request or row, K/V head, row chunk)
// are concatenated and cut into equal runs, one per CTA group, so long and
// short requests balance (lists and short prefixes also stay whole:
// plan_attention); the `members` CTAs of a group walk the same keys
// for different row chunks, close enough in time for the L2 to serve the
// second reader.  An item cut by a boundary leaves partial sums that
// join_kernel adds in a fixed order.
//
// Measured (bf16): latent, 16 rows x 128 heads over 30,001-119,999 keys 310 us
// at 2,070 MHz (1,387 MB, 4.5 TB/s), 333 in a loop at the power limit (1,807
// MHz); 1,024 rows x 128 heads over 2,048 listed keys each 609 us, 959 TFLOP/s:
// both bound by the products, M = 64 at half rate; paged, 64 rows x 32 heads
// over 8,191-32,768 keys 110 us (6.1 TB/s, 90 % of a copy), 64 rows x 16 listed
// blocks 48 us (5.3 TB/s); single rows 8-11 us (latency).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstring>

#include "attention.h"
#include "attn_ptx.cuh"

namespace fp4idx {
namespace {

constexpr int kSoftmaxWarps = 4, kScoreWarp = 4, kLoadWarp = kScoreWarp + 2;
constexpr int kTeamWarps = 4, kTeamThreads = 32 * kTeamWarps;  // loader teams take tiles in turn
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxMembers = 8;
// Pair number / group as (x * ceil(2^40 / group)) >> 40: exact, and inside 64
// bits, for group <= 1024 and up to 2^20 rows of a request.
constexpr int kGroupShift = 40;
constexpr int kMaxRowsOfRequest = 1 << 20;
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
// Whole prefix items are for runs of at most this many tiles (plan_attention).
constexpr int kWholeTiles = 12;
// A row's reference maximum is raised only when the true one is 2^8 above it.
constexpr float kRaise = 8.0f;
// fp16 weights below 2^-14 lose bits and below 2^-25 become 0, while the sum keeps
// them: the reference lies 2^7 below the maximum, so that weights use the type
// up to 2^(7 + 8) (65,504 is its largest) and only shares below 2^-32 are lost.
// bf16 has the range of fp32.
template <int DTYPE>
constexpr float kBelow = DTYPE == FP4IDX_FP16 ? 7.0f : 0.0f;

template <bool LATENT>
struct Cfg {
  static constexpr int kDk = LATENT ? kLatentDim + kRopeDim : kPagedDim;
  static constexpr int kDv = LATENT ? kLatentDim : kPagedDim;
  static constexpr int kTk = LATENT ? 64 : 128;                 // keys per tile
  static constexpr int kRuns = kTk / 64;                        // 64-key runs of a tile: each inside one page
  static constexpr int kStages = 3;
  static constexpr int kParts = LATENT ? 3 : 2;                 // parts of a stage that arrive and leave alone
  static constexpr int kPosPart = LATENT ? 0 : 1;               // the part whose barriers guard the positions: it leaves after the softmax
  static constexpr int kTeams = LATENT ? 2 : 1;
  static constexpr int kSegSlots = 4;                           // planned segments
  static constexpr int kPlanWarp = kLoadWarp + kTeams * kTeamWarps;  // the last one
  static constexpr int kThreads = 32 * (kPlanWarp + 1);
  static constexpr int kKc = kDk / 64;                          // 128-byte pieces of a key
  static constexpr int kPartPieces = LATENT ? kLatentBoxPieces : kPagedBoxPieces;  // pieces of a part, per run
  static constexpr uint32_t kPiece = 64 * 128;                  // one piece of a run's keys
  static constexpr uint32_t kPart = kRuns * kPartPieces * kPiece;
  static constexpr uint32_t kStage = kParts * kPart;
  static constexpr uint32_t kV = LATENT ? 0 : kPart;            // values inside a stage
  static constexpr int kQPieces = LATENT ? 8 : 0;               // 64-value pieces of the queries in TMEM; the others in shared memory
  static constexpr uint32_t kQ = (kKc - kQPieces) * kChunkRows * 128;
  // Latent weights take the place of the tile's rotary piece, which only the
  // score product reads.
  static constexpr uint32_t kP = LATENT ? 0 : kTk / 64 * kChunkRows * 128;
  static constexpr uint32_t kOff_Q = kStages * kStage;
  static constexpr uint32_t kOff_P = LATENT ? kQPieces * kPiece : kOff_Q + kQ;
  static constexpr uint32_t kOff_Ctl = kOff_Q + kQ + kP;
  // TMEM: O^T, 64 columns per 128 values; score buffers; latent queries
  static constexpr uint32_t kOCols = kDv / 128 * kChunkRows;
  static constexpr uint32_t kQCol = kOCols + 2 * kTk;
};
constexpr uint32_t kUpper = 16u << 16;  // the other 16 lanes of each TMEM quarter that M = 64 leaves free
static_assert(Cfg<true>::kQCol + Cfg<true>::kQPieces * 16 == kTmemCols && Cfg<false>::kQCol <= kTmemCols, "TMEM");

struct Item {
  int b, hk;
  int q0;        // first row of the request (or the row of a selection)
  int rows;      // (row, head) pairs: rows of the request x group
  int c0;        // first pair of the chunk group
};

// The part of an item that one CTA computes.
struct Segment {
  Item it;
  int c, rows;       // its pairs [c, c + rows) of the request; rows <= 0: nothing to do
  int max_vis;       // largest visible length among them
  int lo, hi;        // key tiles [lo, hi) of the item's `tiles`
  int tiles;
};

// A CTA's run of tiles [lo, hi) of the concatenation, which ends before item
// `end`; its first item starts at tile `start`.  With whole items a run is
// the items [item, end), counted from tile 0.
struct Run {
  int lo, hi, item, start, end;
};

// Segments are worked out by a warp of its own, ahead of the roles that read them.
template <bool LATENT>
struct Control {
  uint64_t kfull[Cfg<LATENT>::kStages][Cfg<LATENT>::kParts], kempty[Cfg<LATENT>::kStages][Cfg<LATENT>::kParts];
  uint64_t sfull[2], sempty[2], pfull, pvdone, qfull[2], qempty[2], oempty, drain;
  int64_t row_off[kChunkRows];                                 // output element of each row
  uint64_t seg_ready[Cfg<LATENT>::kSegSlots], seg_free[Cfg<LATENT>::kSegSlots];
  Segment seg[Cfg<LATENT>::kSegSlots];
  Run run;
  alignas(8) int32_t key_pos[Cfg<LATENT>::kStages][Cfg<LATENT>::kTk];  // logical position, -1: no key (read in pairs)
  alignas(4) uint8_t holes[Cfg<LATENT>::kStages][kTeamWarps];  // a loader warp found a key that does not exist
  alignas(16) float factor[kChunkRows], row_inv[kChunkRows];
  uint8_t grown[kSoftmaxWarps];                                // a warp's rows have factors below 1
  uint32_t tmem;
  int abort;
};

static_assert(offsetof(Control<true>, key_pos) % 8 == 0 && offsetof(Control<false>, key_pos) % 8 == 0, "int2 reads");
static_assert(offsetof(Control<true>, holes) % 4 == 0 && offsetof(Control<false>, holes) % 4 == 0, "one-word reads");

template <bool LATENT>
constexpr uint32_t smem_bytes() {
  return Cfg<LATENT>::kOff_Ctl + sizeof(Control<LATENT>);
}
static_assert(smem_bytes<true>() <= 232448 && smem_bytes<false>() <= 232448, "227 KB per CTA");

// ---------------------------------------------------------------- items
// x / group and x % group of a pair number (plan_attention bounds it).
__device__ __forceinline__ int group_div(const AttnParams& p, int x) {
  return static_cast<int>((static_cast<uint64_t>(x) * p.group_mul) >> kGroupShift);
}
__device__ __forceinline__ int group_mod(const AttnParams& p, int x) { return x - group_div(p, x) * p.group; }

__device__ __forceinline__ Item item_of(const AttnParams& p, int item) {
  Item it;
  int u = item;
  it.c0 = 0;
  if (p.chunk_groups > 1) {
    u = item / p.chunk_groups;
    it.c0 = (item - u * p.chunk_groups) * p.members * kChunkRows;
  }
  it.hk = 0;
  if (p.num_kv_heads > 1) {
    const int x = u;
    u = x / p.num_kv_heads;
    it.hk = x - u * p.num_kv_heads;
  }
  if (p.indices) {
    it.q0 = u;
    it.b = attn_request(p, u);
    it.rows = p.group;
  } else {
    it.b = u;
    it.q0 = __ldg(p.cu_seqlens_q + u);
    const int n = min(__ldg(p.cu_seqlens_q + u + 1), p.num_rows) - it.q0;
    it.rows = max(0, min(n, p.max_seqlen_q)) * p.group;
  }
  return it;
}

// Largest visible length of the rows that pairs [c, c + n) belong to; called
// by `step` threads with lane = 0..step-1, each giving its share.
__device__ __forceinline__ int pairs_max_visible(const AttnParams& p, const Item& it, int c, int n, int lane, int step) {
  const int first = it.q0 + group_div(p, c), last = it.q0 + group_div(p, c + n - 1);
  if (!p.visible_len) return attn_visible(p, it.b, last);  // grows with the row
  int v = 0;
#pragma unroll 1
  for (int t = first + lane; t <= last; t += step) v = max(v, attn_visible(p, it.b, t));
  return v;
}

// Key tiles of an item (0 without rows; at least one otherwise, so that a row
// without keys is written too).
template <int TK>
__device__ __forceinline__ int item_tiles(const AttnParams& p, const Item& it, int lane, int step) {
  const int n = min(it.rows - it.c0, p.members * kChunkRows);
  if (n <= 0) return 0;
  if (p.indices) return p.list_tiles;
  int v = pairs_max_visible(p, it, it.c0, n, lane, step);
  if (step > 1) v = __reduce_max_sync(0xffffffffu, v);
  return max(1, (v + TK - 1) / TK);
}

// First tile of a group's run: runs differ by one tile at most, and cut items
// of one length alike when there is a whole number of groups per item.  (32
// bits: plan_attention bounds the tiles; long concatenations put the longer
// runs first.)
__device__ __forceinline__ int run_start(int total, int group, int groups) {
  const uint32_t n = total, g = group, all = groups;
  if (n < (1u << 23)) return n * g / all;
  const uint32_t each = n / all;
  return g * each + min(g, n - each * all);
}
__device__ __forceinline__ int used_groups(const AttnParams& p, int total) { return min(total, p.groups); }

// Segment of the tiles [pos, hi) of the concatenation, of an item of `tiles`
// tiles that starts at `start`.
__device__ __forceinline__ Segment segment_of(const AttnParams& p, const Item& it, int tiles, int start, int pos, int hi,
                                              int member, int lane, int step) {
  Segment s;
  s.it = it;
  s.tiles = tiles;
  s.c = it.c0 + member * kChunkRows;
  s.rows = min(kChunkRows, it.rows - s.c);
  s.lo = pos - start;
  s.hi = min(hi, start + tiles) - start;
  s.max_vis = s.rows > 0 ? pairs_max_visible(p, it, s.c, s.rows, lane, step) : 0;
  if (step > 1) s.max_vis = __reduce_max_sync(0xffffffffu, s.max_vis);
  return s;
}

// Rows behind the requests' (a batch padded to a fixed row count) belong to no
// item of a prefix call: zeros and -inf, a (row, head) pair of a CTA at a time.
template <bool LATENT>
__device__ __forceinline__ void clear_rows_of_no_request(const AttnParams& p, int lane) {
  constexpr int kDv = LATENT ? kLatentDim : kPagedDim;
  const int claimed = max(0, __ldg(p.cu_seqlens_q + p.num_seqs));
  const int64_t pairs = static_cast<int64_t>(p.num_rows - min(claimed, p.num_rows)) * p.num_heads;
#pragma unroll 1
  for (int64_t x = blockIdx.x; x < pairs; x += gridDim.x) {
    const int t = claimed + static_cast<int>(x / p.num_heads), h = static_cast<int>(x % p.num_heads);
    uint4* out = reinterpret_cast<uint4*>(p.out + t * p.out_row_stride + h * kDv);
    for (int i = lane; i < kDv / 8; i += 32) out[i] = make_uint4(0, 0, 0, 0);
    if (p.lse && lane == 0) p.lse[static_cast<int64_t>(t) * p.num_heads + h] = -INFINITY;
  }
}

// Where a segment's queries go: with at most 32 rows a CTA the buffer holds two
// segments' queries (32 rows each), so the next ones load early.  (The product
// of the second half reads 64 rows from row 32 on: what lies behind its 32
// rows only reaches score rows that nobody reads.)
struct QuerySlot {
  uint32_t slot, use;  // half, and how often it was used before
};
__device__ __forceinline__ QuerySlot query_slot(const AttnParams& p, uint32_t seg) {
  return p.two_queries ? QuerySlot{seg & 1, seg >> 1} : QuerySlot{0, seg};
}
constexpr uint32_t kQueryHalf = 32 * 128;

// What the join needs to know of a group's first item.
struct GroupInfo {
  int item, start, total;  // total: tiles of all items (every group writes it)
  int q0, rows, c0, hk, pad;
};

// Calls f(segment) for every segment of this CTA, in order; whole warps.
// SOFTMAX: the role's warps leave together, since they meet at named barriers.
template <bool LATENT, bool SOFTMAX, class F>
__device__ __forceinline__ void for_segments(Control<LATENT>& ctl, uint32_t* err, F&& f) {
  if (ctl.run.lo >= ctl.run.hi) return;
  for (uint32_t k = 0;; ++k) {
    bool ok = warp_try(smem_u32(&ctl.seg_ready[k % Cfg<LATENT>::kSegSlots]), (k / Cfg<LATENT>::kSegSlots) & 1, &ctl.abort, err);
    if (SOFTMAX) ok = !bar_red_or(1, 32 * kSoftmaxWarps, !ok);
    if (!ok) return;
    const Segment s = ctl.seg[k % Cfg<LATENT>::kSegSlots];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ctl.seg_free[k % Cfg<LATENT>::kSegSlots]));
    if (s.rows <= 0) return;
    f(s, k);
  }
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
// One value dimension a lane (dimension q = lane / 4 of eight), 16 rows (v) ->
// all eight dimensions of rows q and q + 8: three exchanges between lanes whose
// q differs in one bit, each lane keeping the rows that have its bit.
template <int DTYPE>
__device__ __forceinline__ void rows_to_lanes(const float (&v)[16], int q, uint4 (&out)[2]) {
  const bool b0 = q & 1, b1 = q & 2, b2 = q & 4;
  uint32_t w[8];  // two dimensions of row 2 i + b0
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t even = pack2<DTYPE>(v[2 * i], v[2 * i + 2]), odd = pack2<DTYPE>(v[2 * i + 1], v[2 * i + 3]);
    const uint32_t mine = b0 ? odd : even, theirs = __shfl_xor_sync(0xffffffffu, b0 ? even : odd, 4);
    w[i] = __byte_perm(mine, theirs, b0 ? 0x1054 : 0x5410);
    w[i + 1] = __byte_perm(mine, theirs, b0 ? 0x3276 : 0x7632);
  }
  uint2 u[4];  // four dimensions of row 4 i + 2 b1 + b0
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t mine = b1 ? w[2 * i + 1] : w[2 * i], theirs = __shfl_xor_sync(0xffffffffu, b1 ? w[2 * i] : w[2 * i + 1], 8);
    u[i] = b1 ? make_uint2(theirs, mine) : make_uint2(mine, theirs);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 mine = b2 ? u[2 * i + 1] : u[2 * i], send = b2 ? u[2 * i] : u[2 * i + 1];
    const uint2 theirs = make_uint2(__shfl_xor_sync(0xffffffffu, send.x, 16), __shfl_xor_sync(0xffffffffu, send.y, 16));
    out[i] = b2 ? make_uint4(theirs.x, theirs.y, mine.x, mine.y) : make_uint4(mine.x, mine.y, theirs.x, theirs.y);
  }
}
// ln(sum) of a row with reference maximum m (in powers of two) and sum l.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// ---------------------------------------------------------------- kernel
template <int DTYPE, bool LATENT>
__global__ void __launch_bounds__(Cfg<LATENT>::kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p,
                                                                const __grid_constant__ AttnMaps maps) {
  using C = Cfg<LATENT>;
  constexpr int TK = C::kTk;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control<LATENT>& ctl = *reinterpret_cast<Control<LATENT>*>(smem + C::kOff_Ctl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem);
  volatile int* abort_flag = &ctl.abort;

  if (base & 1023u) {  // the swizzled layouts need it; the runtime places the window there
    if (tid == 0) {
      reinterpret_cast<GroupInfo*>(p.info)->total = 0;
      atomicOr(p.err, kErrTimeout);
    }
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      for (int j = 0; j < C::kParts; ++j) {
        mbar_init(smem_u32(&ctl.kfull[s][j]), kTeamWarps);
        mbar_init(smem_u32(&ctl.kempty[s][j]), 1);
      }
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ctl.sfull[s]), 1);
      mbar_init(smem_u32(&ctl.sempty[s]), kSoftmaxWarps);
      mbar_init(smem_u32(&ctl.qfull[s]), LATENT ? 1 : kTeamWarps);
      mbar_init(smem_u32(&ctl.qempty[s]), 1);
    }
    for (int k = 0; k < C::kSegSlots; ++k) {
      mbar_init(smem_u32(&ctl.seg_ready[k]), 1);
      mbar_init(smem_u32(&ctl.seg_free[k]), C::kPlanWarp);
    }
    mbar_init(smem_u32(&ctl.pfull), kSoftmaxWarps);
    mbar_init(smem_u32(&ctl.pvdone), 1);
    mbar_init(smem_u32(&ctl.oempty), kSoftmaxWarps);
    mbar_init(smem_u32(&ctl.drain), 2);
    ctl.abort = 0;
    fence_barrier_init();
  }
  if (warp == kScoreWarp) tmem_alloc<kTmemCols>(smem_u32(&ctl.tmem));
  __syncthreads();
  pdl_wait();  // everything below reads what earlier kernels wrote

  // ---- the run of tiles of this CTA's group and its first segment
  const int group = blockIdx.x / p.members, member = blockIdx.x - group * p.members;
  {
    int total, before = 0, mine = 0, first = 0;  // all tiles; those before this thread's items, of them
    int per = 1, tiles = 0;
    Item it;
    if (p.whole_items) {
      total = p.items;
      mine = tid == 0 ? total : 0;
    } else if (p.indices) {
      total = p.items * p.list_tiles;
      mine = tid == 0 ? total : 0;
    } else {
      // every thread sums a run of items (the key ring is not in use yet)
      int* warp_sum = reinterpret_cast<int*>(smem);
      per = (p.items + C::kThreads - 1) / C::kThreads;
      first = min(p.items, tid * per);
      const int last = min(p.items, first + per);
#pragma unroll 1
      for (int i = first; i < last; ++i) {
        it = item_of(p, i);
        tiles = item_tiles<TK>(p, it, 0, 1);
        mine += tiles;
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      before = incl - mine;
      total = 0;
#pragma unroll
      for (int w = 0; w < C::kThreads / 32; ++w) {
        const int v = warp_sum[w];
        before += w < warp ? v : 0;
        total += v;
      }
    }
    const int used = used_groups(p, total);
    const bool work = group < used;
    const int lo = work ? run_start(total, group, used) : 0, hi = work ? run_start(total, group + 1, used) : 0;
    GroupInfo& info = reinterpret_cast<GroupInfo*>(p.info)[group];
    if (tid == 0) {
      ctl.run.lo = p.whole_items ? 0 : lo;
      ctl.run.hi = p.whole_items ? (work ? INT32_MAX : 0) : hi;
      ctl.run.end = p.whole_items ? hi : p.items;
      if (member == 0) info.total = total;
    }
    if (work && before <= lo && lo < before + mine) {  // the thread whose items hold the first tile
      int item = first, from = lo, to = hi;
      if (p.whole_items) {
        item = lo;
        it = item_of(p, item);
        tiles = item_tiles<TK>(p, it, 0, 1);
        before = from = 0;
        to = INT32_MAX;
      } else if (p.indices) {
        item = static_cast<uint32_t>(lo) / static_cast<uint32_t>(p.list_tiles);
        it = item_of(p, item);
        tiles = p.list_tiles;
        before = item * tiles;
      } else if (per > 1) {  // walk its items again
        --item;
        int at = before;
        do {
          before = at;
          it = item_of(p, ++item);
          tiles = item_tiles<TK>(p, it, 0, 1);
          at += tiles;
        } while (at <= lo);
      }
      ctl.run.item = item;
      ctl.run.start = before;
      ctl.seg[0] = segment_of(p, it, tiles, before, from, to, member, 0, 1);
      if (ctl.seg[0].rows > 0) mbar_arrive(smem_u32(&ctl.seg_ready[0]));
      if (member == 0) {
        info.item = item;
        info.start = before;
        info.q0 = it.q0;
        info.rows = it.rows;
        info.c0 = it.c0;
        info.hk = it.hk;
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const uint32_t s_col = C::kOCols;  // score buffers behind O^T
  pdl_launch_dependents();           // the join may take its place; it waits for this grid's end

  if (warp == C::kPlanWarp) {
    // ================================================================ planner
    // The segments behind the first one, up to kSegSlots ahead: an item's lengths
    // are several dependent loads away.
    const int lo = ctl.run.lo, hi = ctl.run.hi, end = ctl.run.end;
    if (lo < hi) {
      int item = ctl.run.item, start = ctl.run.start, tiles = ctl.seg[0].tiles;
      Segment n;
      n.rows = ctl.seg[0].rows;
      bool done = false;
#pragma unroll 1
      for (uint32_t k = n.rows > 0 ? 1 : 0; !done; ++k) {
        do {
          start += tiles;
          n.rows = 0;
          done = start >= hi || ++item >= end;
          if (done) break;
          const Item it = item_of(p, item);
          tiles = item_tiles<TK>(p, it, lane, 32);
          if (tiles > 0) n = segment_of(p, it, tiles, start, start, hi, member, lane, 32);
        } while (n.rows <= 0);
        const uint32_t slot = k % C::kSegSlots;
        if (k >= C::kSegSlots && !warp_try(smem_u32(&ctl.seg_free[slot]), (k / C::kSegSlots - 1) & 1, abort_flag, p.err)) break;
        if (lane == 0) {
          ctl.seg[slot] = n;
          mbar_arrive(smem_u32(&ctl.seg_ready[slot]));
        }
        __syncwarp();
      }
    }
    if (!p.indices) clear_rows_of_no_request<LATENT>(p, lane);
  } else if (warp >= kLoadWarp) {
    // ================================================================ loaders
    // Every warp of a team arrives once per part, after its share is issued
    // (TMA, whose bytes the barrier counts) or has landed (copies).
    const int lw = warp - kLoadWarp, team = lw / kTeamWarps, tw = lw % kTeamWarps;
    const int lt = tid - 32 * kLoadWarp - team * kTeamThreads;
    const int u = lt & 7, key0 = lt >> 3;                   // 16-byte unit of a 128-byte piece; first key
    constexpr int kPass = kTeamThreads / 8;                 // keys the team copies at a time
    constexpr int kFind = LATENT ? 64 / kPass : C::kRuns;   // positions a thread looks up: runs, or its listed keys
    uint32_t g = 0;                                         // places of the ring before this segment
    uint32_t issued = 0;                                    // this team's last place, counted from 1
    bool ok = true;
    for_segments<LATENT, false>(ctl, p.err, [&](const Segment& s, uint32_t seg) {
      if (!ok) return;
      const int64_t table = attn_table_base(p, s.it.b);
      const int32_t* list = nullptr;
      if (p.indices)
        list = p.indices + (LATENT ? static_cast<int64_t>(s.it.q0)
                                   : static_cast<int64_t>(s.it.hk) * p.num_rows + s.it.q0) * p.num_indices;
      const bool rows_listed = LATENT && list;              // keys are single rows, not runs
      // position n of tile i, -1 for none; loaded two tiles ahead
      const auto find = [&](int i, int n) -> int32_t {
        if (i >= s.hi) return -1;
        int32_t q = -1;
        if (rows_listed) {
          const int64_t j = static_cast<int64_t>(i) * TK + n * kPass + key0;
          q = j < p.num_indices ? __ldg(list + j) : -1;
        } else if (n >= C::kRuns) {
        } else if (list) {  // a tile is one listed block
          const int32_t blk = __ldg(list + i);
          q = blk >= 0 && blk <= (INT32_MAX - kSelectBlock) / kSelectBlock ? blk * kSelectBlock + 64 * n : -1;
        } else {
          q = i * TK + 64 * n;
        }
        return q;
      };
      // its block-table entry; loaded one tile ahead
      const auto entry = [&](int32_t q) -> int32_t {
        return q >= 0 && q < s.max_vis ? __ldg(p.block_table + table + (q >> p.page_shift)) : -1;
      };
      int i = s.lo + static_cast<int>((team + C::kTeams - g % C::kTeams) % C::kTeams);  // the team's first tile
      const bool queries = LATENT && i == s.lo;                  // latent: place g of the ring takes the queries
      if (LATENT) i += queries ? C::kTeams - 1 : -1;
      int32_t now[kFind], page[kFind], next[kFind];
#pragma unroll
      for (int n = 0; n < kFind; ++n) {
        now[n] = find(i, n);
        next[n] = find(i + C::kTeams, n);
      }
#pragma unroll
      for (int n = 0; n < kFind; ++n) page[n] = entry(now[n]);
      // paged: the segment's queries, once the previous segment's products are done
      bool q_issued = LATENT, q_landed = LATENT;
      const QuerySlot qs = query_slot(p, seg);
      const auto load_queries = [&] {
        q_issued = true;
        ok = warp_try(smem_u32(&ctl.qempty[qs.slot]), (qs.use & 1) ^ 1, abort_flag, p.err);
        if (!ok) return;
#pragma unroll 1
        for (int r = key0; r < ((s.rows + 15) & ~15); r += kPass) {
          const bool have = r < s.rows;
          const int x = s.c + (have ? r : 0), t = s.it.q0 + group_div(p, x), h = s.it.hk * p.group + group_mod(p, x);
          const uint16_t* src = p.q + t * p.q_row_stride + h * p.q_head_stride + u * 8;
          const uint32_t dst = base + C::kOff_Q + qs.slot * kQueryHalf + r * 128 + ((u ^ (r & 7)) << 4);
#pragma unroll
          for (int c = 0; c < C::kKc; ++c) cp_async_16_or_zero(dst + c * (kChunkRows * 128), src + c * 64, have);
        }
        cp_async_commit();
      };
      const auto queries_landed = [&] {  // called once this warp's copies so far have landed
        if (lane == 0 && q_issued && !q_landed) mbar_arrive(smem_u32(&ctl.qfull[qs.slot]));
        q_landed = q_issued;
      };
      if constexpr (LATENT) {
        if (queries) {
          // Eight pieces the way the copy to TMEM wants them, 128 rows a piece:
          // 16 query rows of piece c, then the same rows of piece c + 4, for
          // each quarter of the lanes.  The rotary piece has a place of its own,
          // free when the previous segment's score products are done.
          const uint32_t st = g % C::kStages, ph = ((g / C::kStages) & 1) ^ 1;
          uint4 rot[kChunkRows / kPass];
#pragma unroll
          for (int n = 0; n < kChunkRows / kPass; ++n) {
            const int r = n * kPass + key0;
            const bool have = r < s.rows;
            const int x = s.c + (have ? r : 0), t = s.it.q0 + group_div(p, x), h = s.it.hk * p.group + group_mod(p, x);
            const uint16_t* src = p.q + t * p.q_row_stride + h * p.q_head_stride + u * 8;
            if (n == 0) {
#pragma unroll
              for (int j = 0; j < C::kParts; ++j)
                ok = ok && (g < C::kStages || warp_try(smem_u32(&ctl.kempty[st][j]), ph, abort_flag, p.err));
              if (!ok) return;
            }
            const uint32_t dst = base + st * C::kStage + ((r >> 4) * 4 + ((r >> 3) & 1)) * 1024 + (r & 7) * 128 + ((u ^ (r & 7)) << 4);
#pragma unroll
            for (int c = 0; c < C::kQPieces; ++c)
              cp_async_16_or_zero(dst + (c & 3) * (2 * C::kPiece) + (c >> 2) * 2048, src + c * 64, have);
            rot[n] = have ? __ldg(reinterpret_cast<const uint4*>(src + C::kQPieces * 64)) : make_uint4(0, 0, 0, 0);
          }
          cp_async_commit();
          // (The parity cannot pass for the segment before the last one: after a
          // segment of one tile the same team takes the queries and has waited for
          // that one; after a longer one this place was free only once the last
          // segment's queries were in TMEM, which they wait for.)
          ok = warp_try(smem_u32(&ctl.qempty[0]), (seg & 1) ^ 1, abort_flag, p.err);
          if (!ok) return;
#pragma unroll
          for (int n = 0; n < kChunkRows / kPass; ++n) {
            const int r = n * kPass + key0;
            *reinterpret_cast<uint4*>(smem + C::kOff_Q + r * 128 + ((u ^ (r & 7)) << 4)) = rot[n];
          }
          cp_async_wait_group<0>();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane < C::kParts) mbar_arrive(smem_u32(&ctl.kfull[st][lane]));
        }
      }
      for (; i < s.hi; i += C::kTeams) {
        const uint32_t x = g + LATENT + (i - s.lo), st = x % C::kStages, ph = ((x / C::kStages) & 1) ^ 1;
        const uint32_t stage = base + st * C::kStage;
        // what the table says: pages outside the cache hold no keys
        int32_t pos[kFind];
        bool hole = false, ends = false;                    // a key missing; a run that ends inside
#pragma unroll
        for (int n = 0; n < kFind; ++n) {
          pos[n] = now[n] < s.max_vis ? now[n] : -1;
          if (pos[n] >= 0 && (page[n] < 0 || page[n] >= p.num_pages)) {
            if (rows_listed ? u == 0 : lt == 0) atomicOr(p.err, kErrPageRange);
            pos[n] = -1;
          }
          hole |= pos[n] < 0 && (rows_listed || n < C::kRuns);
          if (!rows_listed) ends |= pos[n] >= 0 && s.max_vis - pos[n] < 64;
        }
        const bool boxes = !rows_listed && !ends, issuer = boxes && tw == 0;
        hole = __any_sync(0xffffffffu, hole || ends);
        const bool fresh = x < C::kStages;                  // a stage's first use: nothing to wait for
        if (issuer && !fresh) {
          // the bytes can be announced before the part is free, once its last load is complete
#pragma unroll
          for (int j = 0; j < C::kParts; ++j) {
            const uint32_t bar = smem_u32(&ctl.kfull[st][j]);
            if (warp_try(bar, ph, abort_flag, p.err) && lane == 0) mbar_arrive_expect_tx(bar, C::kPart);
          }
        }
        __syncwarp();
        int64_t from[TK / kPass];                           // cache element of this thread's keys, -1: zeros
        if (!boxes) {
#pragma unroll
          for (int n = 0; n < TK / kPass; ++n) {
            const int f = rows_listed ? n % kFind : n * kPass / 64;
            int32_t q = pos[f];
            if (!rows_listed && q >= 0) {
              q += (n * kPass + key0) & 63;
              if (q >= s.max_vis) q = -1;
            }
            from[n] = q < 0 ? -1
                            : page[f] * p.page_stride + (static_cast<int64_t>(s.it.hk) * p.page_size +
                                                         (q & (p.page_size - 1))) * C::kDk + u * 8;
          }
        }
#pragma unroll
        for (int j = 0; j < C::kParts; ++j) {
          ok = fresh || warp_try(smem_u32(&ctl.kempty[st][j]), ph, abort_flag, p.err);
          if (!ok) return;
          if (j == C::kPosPart && !issuer) {                // positions for the masks
            if (rows_listed) {
#pragma unroll
              for (int n = 0; n < kFind; ++n)
                if (u == 0) ctl.key_pos[st][n * kPass + key0] = pos[n];
            } else if (lt >= 32 && lt < 96) {
#pragma unroll
              for (int n = 0; n < C::kRuns; ++n) {
                const int k = lt - 32;
                ctl.key_pos[st][64 * n + k] = pos[n] >= 0 && pos[n] + k < s.max_vis ? pos[n] + k : -1;
              }
            }
            if (lane == 0) {
              if (!boxes) ctl.holes[st][tw] = hole;
              else if (tw == 1) *reinterpret_cast<uint32_t*>(ctl.holes[st]) = hole;
            }
            __syncwarp();
          }
          if (issuer) {
            issued = x + 1;
            if (lane < C::kRuns) {
              const int32_t q = C::kRuns == 2 && lane ? pos[kFind - 1] : pos[0];
              const int32_t pg = C::kRuns == 2 && lane ? page[kFind - 1] : page[0];
              tma_load_4d(stage + j * C::kPart + lane * C::kPartPieces * C::kPiece, !LATENT && j ? &maps.v : &maps.k, 0,
                          s.it.hk * p.page_size + (q & (p.page_size - 1)), LATENT ? j * C::kPartPieces : 0,
                          q < 0 ? static_cast<int32_t>(p.num_pages) : pg, smem_u32(&ctl.kfull[st][j]));  // past the cache: zeros
            }
          } else if (boxes) {
            if (lane == 0) mbar_arrive(smem_u32(&ctl.kfull[st][j]));
          } else {
            const uint16_t* cache = !LATENT && j ? p.v : p.k + (LATENT ? j * C::kPartPieces * 64 : 0);
#pragma unroll
            for (int n = 0; n < TK / kPass; ++n) {
              const int key = (n * kPass + key0) & 63, run = n * kPass / 64;
              const uint32_t dst = stage + j * C::kPart + run * C::kPartPieces * C::kPiece + key * 128 + ((u ^ (key & 7)) << 4);
              const uint16_t* src = cache + (from[n] < 0 ? 0 : from[n]);
#pragma unroll
              for (int c = 0; c < C::kPartPieces; ++c) cp_async_16_or_zero(dst + c * C::kPiece, src + c * 64, from[n] >= 0);
            }
            cp_async_commit();
          }
        }
        if (issuer && fresh && lane == 0) {  // the loads are on their way before their bytes are announced
#pragma unroll
          for (int j = 0; j < C::kParts; ++j) mbar_arrive_expect_tx(smem_u32(&ctl.kfull[st][j]), C::kPart);
        }
        if (!q_issued) {
          load_queries();
          if (!ok) return;
        }
        // look ahead while the loads are under way
#pragma unroll
        for (int n = 0; n < kFind; ++n) {
          now[n] = next[n];
          page[n] = entry(now[n]);
          next[n] = find(i + 2 * C::kTeams, n);
        }
        if (!boxes) {
          const bool all = !q_landed;  // queries behind the parts: one wait for both
#pragma unroll
          for (int j = 0; j < C::kParts; ++j) {
            if (all || j == C::kParts - 1) cp_async_wait_group<0>();
            else if (j == C::kParts - 2) cp_async_wait_group<1>();
            else cp_async_wait_group<2>();
            fence_proxy_async_smem();  // the products read the copies through the async proxy
            __syncwarp();
            if (j == 0) queries_landed();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.kfull[st][j]));
          }
        } else if (!q_landed) {
          cp_async_wait_group<0>();
          fence_proxy_async_smem();
          __syncwarp();
          queries_landed();
        }
      }
      g += LATENT + (s.hi - s.lo);
    });
    // after a time-out: this warp's copies land before the CTA can exit
    cp_async_wait_all();
    if (!ok && lane == 0) {
      int never = 0;
      for (uint32_t x = issued; x > 0 && x + C::kStages > issued; x -= min(x, static_cast<uint32_t>(C::kTeams)))
        for (int j = 0; j < C::kParts; ++j)
          mbar_wait(smem_u32(&ctl.kfull[(x - 1) % C::kStages][j]), ((x - 1) / C::kStages) & 1, &never, p.err);
    }
    __syncwarp();
  } else if (warp >= kScoreWarp) {
    // ================================================================ MMA issuers
    // One warp issues the score products, one the value products: the tensor
    // pipe's queue is short, and a warp spends about 100 cycles on each barrier
    // and 50 on each commit, which the other's products cover.  The whole warp
    // runs its loop; one elected lane issues (always the same one: a commit
    // covers its own thread's products).
    uint32_t g = 0;
    bool ok = true;
    const uint32_t tm = uniform(tmem);
    if (warp == kScoreWarp) {
      const uint32_t idesc = uniform(idesc_f16(64, 64, DTYPE == FP4IDX_BF16, false, p.negate != 0));
      const uint64_t q_desc = desc_sw128(base + C::kOff_Q, 16);
      for_segments<LATENT, false>(ctl, p.err, [&](const Segment& s, uint32_t seg) {
        if (!ok) return;
        const uint32_t n = uniform(s.hi - s.lo);
        const QuerySlot qs = query_slot(p, seg);
        const uint64_t qh_desc = q_desc + uniform(qs.slot * (kQueryHalf >> 4));
        const uint32_t first = g + (LATENT ? seg + 1 : 0);  // place of the first tile in the ring
        if constexpr (LATENT) {                             // the queries' place is the one before
          const uint32_t st = uniform((first - 1) % C::kStages), use = ((first - 1) / C::kStages) & 1;
#pragma unroll
          for (int j = 0; j < C::kParts; ++j) ok = ok && warp_try(smem_u32(&ctl.kfull[st][j]), use, abort_flag, p.err);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t from = desc_sw128(base + st * C::kStage, 16);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_cp_128x256b(tm + C::kQCol + c * 32 + k * 8, from + c * (2 * C::kPiece >> 4) + k * 2);
            tc_commit(smem_u32(&ctl.qfull[0]));
          }
          __syncwarp();
        } else {
          ok = warp_try(smem_u32(&ctl.qfull[qs.slot]), qs.use & 1, abort_flag, p.err);
        }
#pragma unroll 1
        for (uint32_t i = 0; ok && i < n; ++i) {
          const uint32_t x = g + i, buf = x & 1;
          const uint32_t st = uniform((first + i) % C::kStages), use = ((first + i) / C::kStages) & 1;
          const uint32_t d = tm + s_col + buf * TK;
          const uint64_t k_desc = desc_sw128(base + st * C::kStage, 16);
          ok = warp_try(smem_u32(&ctl.sempty[buf]), ((x >> 1) & 1) ^ 1, abort_flag, p.err);
#pragma unroll
          for (int j = 0; j < (LATENT ? C::kParts : 1); ++j) {
            ok = ok && warp_try(smem_u32(&ctl.kfull[st][j]), use, abort_flag, p.err);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int r = 0; r < C::kRuns; ++r)
#pragma unroll
                for (int c = 0; c < C::kPartPieces; ++c)
#pragma unroll
                  for (int k = 0; k < 4; ++k) {  // descriptor addresses count 16 bytes
                    const uint64_t b = k_desc + (j * C::kPart >> 4) + (r * C::kPartPieces + c) * (C::kPiece >> 4) + k * 2;
                    if constexpr (LATENT) {  // both halves of the queries, each into its own lanes
                      const int step = (j * C::kPartPieces + c) * 4 + k, half = step / (C::kQPieces * 2), at = step % (C::kQPieces * 2);
                      if (step < C::kQPieces * 4)
                        tc_mma_f16_tmem(d + half * kUpper, tm + C::kQCol + half * kUpper + at * 8, b, idesc, at > 0);
                      else
                        tc_mma_f16(d, q_desc + k * 2, b, idesc, 1);
                    } else {
                      tc_mma_f16(d + r * 64, qh_desc + c * (kChunkRows * 8) + k * 2, b, idesc, c + k > 0);
                    }
                  }
              if (!LATENT || j == C::kParts - 1) {
                if constexpr (!LATENT) tc_commit(smem_u32(&ctl.kempty[st][0]));  // the keys' last reader
                tc_commit(smem_u32(&ctl.sfull[buf]));
                if (i + 1 == n) tc_commit(smem_u32(&ctl.qempty[qs.slot]));
              }
            }
            __syncwarp();
          }
        }
        g += n;
      });
    } else {
      const uint64_t p_base = desc_sw128(base + C::kOff_P, 16);
      for_segments<LATENT, false>(ctl, p.err, [&](const Segment& s, uint32_t seg) {
        if (!ok) return;
        const uint32_t idesc = uniform(idesc_f16(128, (s.rows + 15) & ~15, DTYPE == FP4IDX_BF16, true, false));
        const uint32_t n = uniform(s.hi - s.lo);
        if constexpr (LATENT) {
          // The queries are in TMEM: their place of the ring is free, but only
          // released behind the value products of the places before it.  The
          // loader teams take places in turn, and the parity that a team waits
          // for tells two uses of a stage apart only if places come free in order.
          const uint32_t place = g + seg, st = uniform(place % C::kStages);
          ok = warp_try(smem_u32(&ctl.qfull[0]), seg & 1, abort_flag, p.err);
          if (!ok) return;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < C::kParts; ++j) tc_commit(smem_u32(&ctl.kempty[st][j]));
          }
          __syncwarp();
        }
        ok = warp_try(smem_u32(&ctl.oempty), (seg & 1) ^ 1, abort_flag, p.err);
#pragma unroll 1
        for (uint32_t i = 0; ok && i < n; ++i) {
          const uint32_t x = g + i, place = x + (LATENT ? seg + 1 : 0), st = uniform(place % C::kStages), more = i > 0;
          const uint64_t v_desc = desc_sw128(base + st * C::kStage + C::kV, C::kPiece);
          const uint64_t p_desc = p_base + (LATENT ? st * (C::kStage >> 4) : 0);
          if constexpr (!LATENT)
            ok = warp_try(smem_u32(&ctl.kfull[st][1]), (place / C::kStages) & 1, abort_flag, p.err);
          ok = ok && warp_try(smem_u32(&ctl.pfull), x & 1, abort_flag, p.err);
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int d = 0; d < C::kDv / 128; ++d) {
#pragma unroll
              for (int k = 0; k < TK / 16; ++k)
                tc_mma_f16(tm + d * kChunkRows, v_desc + (d * 2 + (k >> 2) * C::kPartPieces) * (C::kPiece >> 4) + (k & 3) * 128,
                           p_desc + (k >> 2) * (kChunkRows * 8) + (k & 3) * 2, idesc, k > 0 ? 1u : more);
              // 128 values are pieces 2d and 2d+1; part j of a latent tile is pieces 3j .. 3j+2
              if (LATENT && d > 0) tc_commit(smem_u32(&ctl.kempty[st][d - 1]));
            }
            if constexpr (!LATENT) tc_commit(smem_u32(&ctl.kempty[st][1]));
            tc_commit(smem_u32(&ctl.pvdone));
          }
          __syncwarp();
        }
        g += n;
      });
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
    // After a failed wait the loop runs on without waiting, so that the
    // named barriers below still meet; nothing is written then.
    uint32_t g = 0;
    bool ok = true;
    const int r0 = 16 * warp + (lane >> 2);                 // this thread's rows: r0 and r0 + 8
    const uint32_t quarter = static_cast<uint32_t>(warp) << 21;  // TMEM lanes 32 * warp
    for_segments<LATENT, true>(ctl, p.err, [&](const Segment& s, uint32_t seg) {
      // rows past the chunk's end have zero queries: their scores are harmless
      int vis[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + 8 * i;
        vis[i] = r < s.rows ? attn_visible(p, s.it.b, s.it.q0 + group_div(p, s.c + r)) : INT32_MAX;
      }
      // tiles that all of the warp's rows see whole (a selection's keys are all visible or holes)
      const int full_tiles = p.indices ? INT32_MAX : __reduce_min_sync(0xffffffffu, min(vis[0], vis[1])) / TK;
      const bool active = 16 * warp < s.rows;
      const int cols = (s.rows + 15) & ~15;                  // O^T columns in use
      float m[2] = {-INFINITY, -INFINITY};                   // reference maximum, in powers of two
      float2 l[2] = {};                                      // this thread's share of the sums
      for (int i = s.lo; i < s.hi; ++i, ++g) {
        const uint32_t buf = g & 1, place = g + (LATENT ? seg + 1 : 0), st = place % C::kStages;
        float x[TK / 2];
        bool raise = false;
        float f[2] = {1.0f, 1.0f};
        if (active) {
          if (ok) ok = warp_try(smem_u32(&ctl.sfull[buf]), (g >> 1) & 1, abort_flag, p.err);
          if (ok) ok = warp_try(smem_u32(&ctl.kfull[st][C::kPosPart]), (place / C::kStages) & 1, abort_flag, p.err);
          tc_fence_after();
          static_assert(kTeamWarps == 4, "holes of a stage are read as one word");
          const bool mask = i >= full_tiles || *reinterpret_cast<const uint32_t*>(ctl.holes[st]) != 0;
#pragma unroll
          for (int c = 0; c < TK / 64; ++c) {
            uint32_t r[32];
            tmem_ld_16x256b_x8(tmem + quarter + s_col + buf * TK + c * 64, r);
            if constexpr (LATENT) {  // the sums over the two halves of the query
              uint32_t upper[32];
              tmem_ld_16x256b_x8(tmem + quarter + kUpper + s_col + buf * TK, upper);
              tmem_wait_ld();
              reg_fence(r);
              reg_fence(upper);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r[e]) + __uint_as_float(upper[e]);
            } else {
              tmem_wait_ld();
              reg_fence(r);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(r[e]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl.sempty[buf]));
          if (mask) {
#pragma unroll
            for (int j = 0; j < TK / 8; ++j) {
              const int2 kp = *reinterpret_cast<const int2*>(&ctl.key_pos[st][8 * j + 2 * (lane & 3)]);
#pragma unroll
              for (int e = 0; e < 4; ++e)  // -1 (no key) is the largest unsigned value
                if (static_cast<uint32_t>(e & 1 ? kp.y : kp.x) >= static_cast<uint32_t>(vis[e >> 1])) x[4 * j + e] = -INFINITY;
            }
          }
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < TK / 8; ++j) {
            top[0] = fmaxf(top[0], fmaxf(x[4 * j], x[4 * j + 1]));
            top[1] = fmaxf(top[1], fmaxf(x[4 * j + 2], x[4 * j + 3]));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
            top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2)) * p.scale_log2 - kBelow<DTYPE>;
            if (top[e] > m[e] + kRaise) {
              f[e] = ex2(m[e] - top[e]);
              m[e] = top[e];
              raise = true;
            }
          }
        }
        if (!active && lane == 0) mbar_arrive(smem_u32(&ctl.sempty[buf]));
        const bool any = bar_red_or(1, 32 * kSoftmaxWarps, raise);
        uint32_t w[TK / 4];
        if (active) {
          // weights, their sum in fp32, and P in 16 bits (the MMA's operand
          // type: each weight is rounded once, the sum is of unrounded ones)
          const float2 scale = make_float2(p.scale_log2, p.scale_log2);
          const float2 ref0 = m[0] == -INFINITY ? make_float2(0.0f, 0.0f) : make_float2(-m[0], -m[0]);
          const float2 ref1 = m[1] == -INFINITY ? make_float2(0.0f, 0.0f) : make_float2(-m[1], -m[1]);
          l[0].x *= f[0];
          l[0].y *= f[0];
          l[1].x *= f[1];
          l[1].y *= f[1];
#pragma unroll
          for (int j = 0; j < TK / 8; ++j) {
            float2 a = fma2(make_float2(x[4 * j], x[4 * j + 1]), scale, ref0);
            float2 b = fma2(make_float2(x[4 * j + 2], x[4 * j + 3]), scale, ref1);
            a = make_float2(ex2(a.x), ex2(a.y));
            b = make_float2(ex2(b.x), ex2(b.y));
            l[0] = add2(l[0], a);
            l[1] = add2(l[1], b);
            w[2 * j] = pack2<DTYPE>(a.x, a.y);
            w[2 * j + 1] = pack2<DTYPE>(b.x, b.y);
          }
        }
        // the previous product has read P (paged) and updated O^T
        if (ok && g > 0) ok = warp_try(smem_u32(&ctl.pvdone), (g - 1) & 1, abort_flag, p.err);
        if (active) {
          uint8_t* prow = smem + C::kOff_P + (LATENT ? st * C::kStage : 0) + r0 * 128 + (lane & 3) * 4;
#pragma unroll
          for (int j = 0; j < TK / 8; ++j) {
            uint8_t* at = prow + (j >> 3) * (kChunkRows * 128) + (((j & 7) ^ (r0 & 7)) << 4);
            *reinterpret_cast<uint32_t*>(at) = w[2 * j];
            *reinterpret_cast<uint32_t*>(at + 8 * 128) = w[2 * j + 1];
          }
          fence_proxy_async_smem();
        }
        if (any && i > s.lo) {
          const bool grown = __any_sync(0xffffffffu, raise);
          if (lane == 0) ctl.grown[warp] = grown;
          if ((lane & 3) == 0) {
            ctl.factor[r0] = f[0];
            ctl.factor[r0 + 8] = f[1];
          }
          bar_sync(2, 32 * kSoftmaxWarps);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            if (!ctl.grown[c >> 4]) continue;
#pragma unroll 1
            for (int d = 0; d < C::kDv / 128; ++d) {
              const uint32_t at = tmem + quarter + d * kChunkRows + c;
              uint32_t r[16];
              __syncwarp();
              tmem_ld(at, r);
              tmem_wait_ld();
              reg_fence(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * ctl.factor[c + e]);
              tmem_st_x16(at, r);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.pfull));
      }
      // ---- output of the segment
      float sum[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] = l[e].x + l[e].y;
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      }
      const bool whole = s.lo == 0 && s.hi == s.tiles;
      const int64_t slot = (static_cast<int64_t>(group) * 2 + (s.lo == 0)) * p.members + member;
      if ((lane & 3) == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 8 * e;
          const int t = s.it.q0 + group_div(p, s.c + r), h = s.it.hk * p.group + group_mod(p, s.c + r);
          ctl.row_inv[r] = sum[e] == 0.0f ? 0.0f : 1.0f / sum[e];
          ctl.row_off[r] = t * p.out_row_stride + static_cast<int64_t>(h) * C::kDv;
          if (r < s.rows && ok) {
            if (!whole)
              p.stats[slot * kChunkRows + r] = make_float2(m[e], sum[e]);
            else if (p.lse)
              p.lse[static_cast<int64_t>(t) * p.num_heads + h] = row_lse(m[e], sum[e]);
          }
        }
      }
      if (ok) ok = warp_try(smem_u32(&ctl.pvdone), (g - 1) & 1, abort_flag, p.err);
      bar_sync(2, 32 * kSoftmaxWarps);
      tc_fence_after();
      if (LATENT && whole) {
        // Row fragments of 16 dimensions: this lane has dimension lane / 4 (and
        // that + 8) of rows 8 j + 2 (lane % 4) + {0, 1}; after an exchange, 16
        // dimensions of two rows.
        const int q = lane >> 2, mine = 2 * (lane & 3);
        int row[2];
        int64_t off[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          row[n] = 8 * (4 * n + (q >> 1)) + mine + (q & 1);
          off[n] = ctl.row_off[row[n]] + 32 * warp;
        }
        float2 inv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = *reinterpret_cast<const float2*>(&ctl.row_inv[8 * j + mine]);
#pragma unroll 1
        for (int i = 0; i < C::kDv / 64; ++i) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_16x256b_x8(tmem + quarter + (i >> 1) * kChunkRows + (i & 1) * kUpper, r);
          tmem_wait_ld();
          reg_fence(r);
          uint4 w[2][2];
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[2 * j] = __uint_as_float(r[4 * j + 2 * o]) * inv[j].x;
              v[2 * j + 1] = __uint_as_float(r[4 * j + 2 * o + 1]) * inv[j].y;
            }
            rows_to_lanes<DTYPE>(v, q, w[o]);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (ok && row[n] < s.rows) {
              uint4* to = reinterpret_cast<uint4*>(p.out + off[n] + (i >> 1) * 128 + (i & 1) * 16);
              to[0] = w[0][n];
              to[1] = w[1][n];
            }
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < C::kDv / 128 * cols; c += 16) {
          const int d = c / cols, col = c - d * cols;
          const int dv = d * 128 + tid;  // this thread's value dimension (tid < 128)
          uint32_t r[16];
          __syncwarp();
          tmem_ld(tmem + quarter + d * kChunkRows + col, r);
          tmem_wait_ld();
          reg_fence(r);
          if (!ok) continue;
          if (!LATENT && whole) {
            // neighbouring lanes swap rows so that each stores two values of one row
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int row = col + e + (lane & 1);
              const float a = __uint_as_float(r[e]) * ctl.row_inv[col + e];
              const float b = __uint_as_float(r[e + 1]) * ctl.row_inv[col + e + 1];
              const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
              const uint32_t v = lane & 1 ? pack2<DTYPE>(other, b) : pack2<DTYPE>(a, other);
              if (row < s.rows) *reinterpret_cast<uint32_t*>(p.out + ctl.row_off[row] + (dv & ~1)) = v;
            }
          } else {
            float* o = p.partial + (slot * kChunkRows + col) * C::kDv + dv;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (col + e < s.rows) o[e * C::kDv] = __uint_as_float(r[e]);
          }
        }
      }
      tc_fence_before();
      bar_sync(2, 32 * kSoftmaxWarps);  // row_inv and row_off are read before the next segment writes them
      if (lane == 0) mbar_arrive(smem_u32(&ctl.oempty));
    });
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem);
  }
}

// ---------------------------------------------------------------- join
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the partial sums of
// an item that crosses run boundaries, in the order of its keys.  The eight
// warps of a CTA take a row each when an item has few partials (BY_ITEM
// false: blockIdx.x counts run boundaries, the first boundary inside an item
// does its work), and share one row's partials when many meet (BY_ITEM:
// blockIdx.x is the item).

template <int DTYPE, bool LATENT, bool BY_ITEM>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<LATENT>;
  constexpr int kVec = C::kDv / 128;  // float4s per lane
  __shared__ float4 sum[BY_ITEM ? kJoinWarps : 1][C::kDv / 4];
  __shared__ float2 part[kJoinWarps];
  __shared__ int total_tiles;
  __shared__ int first_group;
  __shared__ GroupInfo shared_info;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, member = blockIdx.y, warp = tid >> 5, lane = tid & 31;
  // one group per thread (plan_attention); groups without work hold nothing but the total
  const GroupInfo* infos = reinterpret_cast<const GroupInfo*>(p.info);
  GroupInfo info = {};
  if (tid < p.groups) info = infos[tid];
  const int candidate = BY_ITEM ? blockIdx.x : infos[blockIdx.x + 1].item;
  if (tid == 0) {
    total_tiles = info.total;
    first_group = INT32_MAX;
  }
  __syncthreads();
  const int used = used_groups(p, total_tiles);
  // the groups whose run begins inside the item: consecutive ones
  const bool inside = tid > 0 && tid < used && info.item == candidate && info.start < run_start(total_tiles, tid, used);
  if (inside) atomicMin(&first_group, tid);
  const int parts = 1 + __syncthreads_count(inside);
  const int group = first_group;  // the first boundary; the part before it is the previous group's
  if (parts == 1 || (!BY_ITEM && group != static_cast<int>(blockIdx.x) + 1)) return;
  if (tid == group) shared_info = info;
  __syncthreads();
  const int c = shared_info.c0 + member * kChunkRows;
  const int r = BY_ITEM ? blockIdx.z : blockIdx.z * kJoinWarps + warp;
  if (r >= min(kChunkRows, shared_info.rows - c)) return;  // (BY_ITEM: the whole CTA)
  // this warp's partials, each added relative to the largest maximum so far
  float4 acc[kVec] = {};
  float m = -INFINITY, l = 0.0f;
#pragma unroll 4
  for (int i = BY_ITEM ? warp : 0; i < parts; i += BY_ITEM ? kJoinWarps : 1) {
    // part i is group - 1 + i; the first one is its group's last segment, the others their groups' first
    const int64_t row = ((static_cast<int64_t>(group - 1 + i) * 2 + (i == 0)) * p.members + member) * kChunkRows + r;
    const float2 s = p.stats[row];
    float4 o[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) o[v] = reinterpret_cast<const float4*>(p.partial + row * C::kDv)[v * 32 + lane];
    const float top = fmaxf(m, s.x), ref = top == -INFINITY ? 0.0f : top;
    const float keep = ex2(m - ref), w = ex2(s.x - ref);
    m = top;
    l = l * keep + w * s.y;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      acc[v].x = acc[v].x * keep + w * o[v].x;
      acc[v].y = acc[v].y * keep + w * o[v].y;
      acc[v].z = acc[v].z * keep + w * o[v].z;
      acc[v].w = acc[v].w * keep + w * o[v].w;
    }
  }
  if constexpr (BY_ITEM) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) sum[warp][v * 32 + lane] = acc[v];
    if (lane == 0) part[warp] = make_float2(m, l);
    __syncthreads();
    if (warp >= kVec) return;
    // warp v adds the warps' shares of its 128 values
    m = part[0].x;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, part[w].x);
    const float ref = m == -INFINITY ? 0.0f : m;
    l = 0.0f;
    acc[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float4 o = sum[w][warp * 32 + lane];
      const float f = ex2(part[w].x - ref);
      l = fmaf(f, part[w].y, l);
      acc[0].x = fmaf(f, o.x, acc[0].x);
      acc[0].y = fmaf(f, o.y, acc[0].y);
      acc[0].z = fmaf(f, o.z, acc[0].z);
      acc[0].w = fmaf(f, o.w, acc[0].w);
    }
  }
  const int t = shared_info.q0 + group_div(p, c + r);
  const int h = shared_info.hk * p.group + group_mod(p, c + r);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2* out = reinterpret_cast<uint2*>(p.out + t * p.out_row_stride + static_cast<int64_t>(h) * C::kDv);
#pragma unroll
  for (int v = 0; v < (BY_ITEM ? 1 : kVec); ++v)
    out[(BY_ITEM ? warp : v) * 32 + lane] =
        make_uint2(pack2<DTYPE>(acc[v].x * inv, acc[v].y * inv), pack2<DTYPE>(acc[v].z * inv, acc[v].w * inv));
  if (p.lse && lane == 0 && (!BY_ITEM || warp == 0))
    p.lse[static_cast<int64_t>(t) * p.num_heads + h] = row_lse(m, l);
}

template <int DTYPE, bool LATENT>
cudaError_t launch(const AttnParams& p, const AttnMaps& maps, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose kernel has its shared memory limit (a call costs 1 us)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(attention_kernel<DTYPE, LATENT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes<LATENT>());
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(p.groups * p.members));
  cfg.blockDim = dim3(Cfg<LATENT>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<LATENT>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, attention_kernel<DTYPE, LATENT>, p, maps)) != cudaSuccess) return e;
  if (p.groups < 2 || p.whole_items) return cudaSuccess;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  // rows that a CTA of the first kernel can hold
  const int64_t pairs = (p.indices ? 1 : static_cast<int64_t>(p.max_seqlen_q)) * p.group;
  const unsigned rows = static_cast<unsigned>(pairs < kChunkRows ? pairs : kChunkRows);
  if (p.groups > 4 * static_cast<int64_t>(p.items)) {  // more than four partials per row
    cfg.gridDim = dim3(static_cast<unsigned>(p.items), static_cast<unsigned>(p.members), rows);
    return cudaLaunchKernelEx(&cfg, join_kernel<DTYPE, LATENT, true>, p);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(p.groups - 1), static_cast<unsigned>(p.members), (rows + kJoinWarps - 1) / kJoinWarps);
  return cudaLaunchKernelEx(&cfg, join_kernel<DTYPE, LATENT, false>, p);
}

int64_t round16(int64_t n) { return (n + 15) & ~int64_t{15}; }

}  // namespace

bool plan_attention(AttnParams* p, int sms) {
  const bool latent = p->v == nullptr;
  const int64_t pairs = (p->indices ? 1 : static_cast<int64_t>(p->max_seqlen_q)) * p->group;
  const int64_t chunks = (pairs + kChunkRows - 1) / kChunkRows;
  p->members = static_cast<int32_t>(chunks < kMaxMembers ? chunks : kMaxMembers);
  const int64_t cg = (chunks + p->members - 1) / p->members;
  const int64_t items = static_cast<int64_t>(p->indices ? p->num_rows : p->num_seqs) * p->num_kv_heads * cg;
  if (items > INT32_MAX || p->max_seqlen_q > kMaxRowsOfRequest) return false;
  p->group_mul = ((uint64_t{1} << kGroupShift) + p->group - 1) / p->group;
  p->two_queries = !latent && pairs <= 32;
  p->chunk_groups = static_cast<int32_t>(cg);
  p->items = static_cast<int32_t>(items);
  const int tk = latent ? Cfg<true>::kTk : Cfg<false>::kTk;
  p->list_tiles = p->indices ? static_cast<int32_t>((static_cast<int64_t>(p->num_indices) * (latent ? 1 : kSelectBlock) + tk - 1) / tk) : 0;
  // no more groups than tiles can exist
  const int64_t per_item = p->indices ? p->list_tiles : (static_cast<int64_t>(p->max_seqlen_k) + tk - 1) / tk;
  const int64_t most = items * (per_item < 1 ? 1 : per_item);
  if (most > INT32_MAX) return false;
  int64_t groups = sms / p->members;
  if (groups > kJoinThreads) groups = kJoinThreads;  // the join looks at one group per thread
  // How are the items cut?  In tiles' time:
  //   whole items: no partial sums and no join;
  //   each item into an equal number of runs: partial sums and a join, which
  //     cost as much as two (latent) or three (paged) tiles;
  //   equal runs over all items: every group busy, but most CTAs also cross from
  //     one item to the next, five tiles in all.
  // Lists have one length, so that HBM, which feeds as many CTAs as `feeds`,
  // bounds each form from below.  (Rows of one request find much of their keys in
  // L2, but gain nothing by equal runs: 77 / 100 / 130 rows x 64 heads of one
  // 32,768-key request, 2,048 listed keys each, 55 / 57 / 57 us whole, 51 / 57 / 66
  // in equal runs.)  Of a prefix only the largest length is known here, and every
  // other item may be a single tile: whole items are taken up to kWholeTiles,
  // where one long item among single-tile ones costs no more than equal runs (152
  // items, one of 8 / 12 paged tiles 19.6 / 22.5 against 20.5 / 21.0 us, of 12
  // latent ones 28.6 against 28.6).  Longer ones are cut by the lengths that the
  // device finds: 38 requests x 4 K/V heads of 1,024-32,768 keys 119 us (whole
  // 209), one of 32,768 keys among 37 of 1,024 48 us (238), 152 requests x 64
  // latent heads of 1,024-65,536 keys 392 us (1,142), a prompt of 1,024 rows
  // among 18 decodes 1.4 ms (17.2).  Items of one length pay a join for it: 152 of
  // 16 paged tiles 45.3 us (43.0), of 16 latent ones 51.8 (49.2).
  // Measured, whole against cut: one request of 2 / 3 / 4 latent tiles 10.4 /
  // 11.5 / 12.6 against 10.4 / 10.5 / 10.6 us, of 3 / 4 / 5 paged tiles 8.4 / 9.1
  // / 9.9 against 9.7 / 9.4 / 9.2 us, 64 requests of 3 / 12 latent tiles 11.7 /
  // 23.1 against 13.9 / 22.8 us, 96 items of 8-32 paged tiles 36.2 against 32.2;
  // whole against equal runs: 160 items of 4 / 6 / 8 paged tiles 18.1 / 22.7 /
  // 27.2 against 19.6 / 23.2 / 25.8 us, 256 listed items of 16 49.3 against 53.5 us.
  const double feeds = !p->indices ? HUGE_VAL : latent ? 90 : 86;
  const double longest = per_item < 1 ? 1 : static_cast<double>(per_item);
  const int64_t rest = items % groups;
  const double hbm = longest * items / feeds;
  const double whole = longest * (static_cast<double>(items / groups) * std::max(1.0, groups / feeds) +
                                  (rest ? std::max(1.0, rest / feeds) : 0.0));
  const int64_t cuts = std::min(groups / items, per_item);
  const double cut = cuts > 1 ? std::max(static_cast<double>((per_item + cuts - 1) / cuts), hbm) + (latent ? 2 : 3) : HUGE_VAL;
  const double equal = std::max(longest * items / groups, hbm) + 5;
  p->whole_items = whole < cut && whole <= equal && (p->indices || whole <= kWholeTiles);
  if (!p->whole_items && cut <= equal) groups = cuts * items;
  const int64_t units = p->whole_items ? items : most;
  p->groups = static_cast<int32_t>(units < groups ? units : groups);
  return true;
}

size_t attention_workspace(const AttnParams& p) {
  const int64_t rows = static_cast<int64_t>(p.groups) * 2 * p.members * kChunkRows;
  const int64_t dv = p.v == nullptr ? kLatentDim : kPagedDim;
  return static_cast<size_t>(round16(p.groups * static_cast<int64_t>(sizeof(GroupInfo))) + round16(rows * 8) + rows * dv * 4);
}

cudaError_t launch_attention(AttnParams p, const AttnMaps& maps, int dtype, void* workspace, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.groups) * 2 * p.members * kChunkRows;
  char* w = static_cast<char*>(workspace);
  p.info = reinterpret_cast<int64_t*>(w);
  w += round16(p.groups * static_cast<int64_t>(sizeof(GroupInfo)));
  p.stats = reinterpret_cast<float2*>(w);
  w += round16(rows * 8);
  p.partial = reinterpret_cast<float*>(w);
  const bool latent = p.v == nullptr;
  if (dtype == FP4IDX_BF16)
    return latent ? launch<FP4IDX_BF16, true>(p, maps, stream) : launch<FP4IDX_BF16, false>(p, maps, stream);
  return latent ? launch<FP4IDX_FP16, true>(p, maps, stream) : launch<FP4IDX_FP16, false>(p, maps, stream);
}

}  // namespace fp4idx
