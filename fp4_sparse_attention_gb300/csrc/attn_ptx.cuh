// attn_ptx.cuh -- inline-PTX building blocks of the attention kernels beyond
// ptx.cuh: 16-bit tcgen05 MMAs, their descriptors, TMEM loads in the
// row-fragment shape and TMEM stores, zero-filling asynchronous copies.
#pragma once

#include "ptx.cuh"

namespace fp4idx {

// One lane of a converged warp.  MMAs are issued inside `if (elect_one())`
// by a warp that runs its role converged: their operands then stay in uniform
// registers.  Measured issue cost of a 64x64x16 MMA (which takes 31 cycles): 30
// cycles so, 39 with an election per MMA, 56 from a branch of one thread.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit operands, fp32 accumulator.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in TMEM: M = 64 rows in 16 lanes of each quarter, two k in a
// column.  A and D lie in the same lanes: the lower or the upper 16.  (As fast
// as from shared memory: M = 64 runs at half of the tensor pipe's rate, 31
// cycles for 64x64x16 either way.)
__device__ __forceinline__ void tc_mma_f16_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Whole-warp wait for the phase of `parity`: every lane executes the same
// try_wait, without a suspend hint.  Measured hand-over between two warps
// (half a round trip): 100 cycles; with a hint 130; through one lane 140, with
// a hint 380.  Bounded like mbar_wait.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
static __device__ __noinline__ bool warp_try_again(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  const uint64_t t0 = globaltimer();
  bool ok = false;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try(bar, parity);
    if (ok || *abort) return ok;
    if (globaltimer() - t0 > kWaitLimitNs) {
      if ((threadIdx.x & 31) == 0) atomicOr(err, kErrTimeout);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool warp_try(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  bool ok = mbar_try(bar, parity);
  if (!ok) ok = warp_try_again(bar, parity, abort, err);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Instruction descriptor of kind::f16 with an fp32 accumulator; both operands
// fp16 (bf16 false) or both bf16.  a_mn: A is stored with M contiguous;
// negate: the product of -A.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool bf16, bool a_mn, bool negate) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (negate ? 1u << 13 : 0u) | (a_mn ? 1u << 15 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Operand in 128-byte rows, 128-byte swizzle (1,024-byte atoms of 8 rows).
//   K-major: a row holds 64 consecutive k of one m/n; 8-row groups every
//   1,024 B; a 16-wide k step inside the row advances the address by 32 B.
//   MN-major: a row holds 64 consecutive m of one k; groups of 8 k every
//   1,024 B, the next 64 m every `mn_stride` bytes.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_stride >> 4) << 16;  // leading byte offset (unused when K-major)
  d |= static_cast<uint64_t>(1024 >> 4) << 32;       // stride byte offset
  d |= static_cast<uint64_t>(1) << 46;               // descriptor version (tcgen05)
  d |= static_cast<uint64_t>(2) << 61;               // 128-byte swizzle
  return d;
}

// 16 lanes x 64 columns as the four warps' row fragments: thread i receives
// columns 8j + 2(i%4) + {0,1} of lane i/4 in r[4j], r[4j+1] and of lane i/4 + 8
// in r[4j+2], r[4j+3].
#define FP4IDX_R8(i) "=r"(r[i + 0]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), \
                     "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : FP4IDX_R8(0), FP4IDX_R8(8), FP4IDX_R8(16), FP4IDX_R8(24)
      : "r"(taddr));
}
#undef FP4IDX_R8

// 32 lanes x 16 columns: thread i of the warp writes its lane's columns.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16-byte asynchronous copy, or 16 zero bytes (src is not read).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0) : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z,
                                            int32_t w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Named barrier of `count` threads that also ORs a predicate over them.
__device__ __forceinline__ bool bar_red_or(uint32_t id, uint32_t count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.or.pred q, %1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t count) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

}  // namespace fp4idx
