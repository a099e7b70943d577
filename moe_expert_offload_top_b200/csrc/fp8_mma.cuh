// tcgen05 / TMEM / TMA helpers of the fp8 product kernels (e4m3 x e4m3 -> f32).
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "sm100_sync.cuh"

namespace ftk {

FT_DEVICE void fp8_tma_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
FT_DEVICE void fp8_tma_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Four rows of a 2-D map whose box is one row high.
FT_DEVICE void fp8_tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int r0, int r1, int r2,
                               int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
      : "memory");
}

// mbar_wait by a converged warp, which stays one; true when every lane's wait succeeded.  The
// first try is apart from the loop: a phase that is over costs 75 cycles so (a loop around the
// try, even one left at once, 290).
FT_DEVICE bool warp_wait(uint64_t* b, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  if (__all_sync(0xFFFFFFFFu, mbar_try(b, parity))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait(b, parity, abort_flag, err, code));
}
// Both phases over: the two first tries overlap.
FT_DEVICE bool warp_wait2(uint64_t* b0, uint32_t parity0, uint64_t* b1, uint32_t parity1, volatile int* abort_flag,
                          int* err, int code) {
  const bool t0 = mbar_try(b0, parity0), t1 = mbar_try(b1, parity1);
  if (__all_sync(0xFFFFFFFFu, t0 && t1)) return true;
  const bool ok = mbar_wait(b0, parity0, abort_flag, err, code) && mbar_wait(b1, parity1, abort_flag, err, code);
  return __all_sync(0xFFFFFFFFu, ok);
}
// The wait of a test for the way out: on a barrier that nothing arrives on, for 1 ms.
FT_DEVICE void never_wait(uint64_t* b, volatile int* abort_flag, int* err, int code) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_wait(b, 0, abort_flag, err, code, 1000000ull);
  __syncwarp();
}
// One arrival for the warp, behind everything its lanes did before.
FT_DEVICE void warp_arrive(uint64_t* b) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(b);
}

// One lane of a converged warp.  The compiler then knows that what follows runs in one thread,
// and issues tcgen05 instructions with warp-uniform operands once instead of in a loop over lanes.
FT_DEVICE bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 B apart.
FT_DEVICE uint64_t fp8_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// Instruction descriptor: kind::f8f6f4, e4m3 x e4m3 -> f32, A and B K-major, M x N.
__host__ __device__ constexpr uint32_t fp8_idesc(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
FT_DEVICE void fp8_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
FT_DEVICE void fp8_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(smem_u32(bar)) : "memory");
}
FT_DEVICE void fp8_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
FT_DEVICE void fp8_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 or 32 accumulator columns of this thread's TMEM lane.  The registers hold nothing before
// tmem_wait on them, which therefore has to follow in the same pass of a loop: a copy that the
// compiler places between the two (at a loop's back edge, say) would read them too early.
FT_DEVICE void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
FT_DEVICE void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The loads so far have landed, r's among them: r passes through, so that its uses stay behind.
FT_DEVICE void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
               "+r"(r[15])
               :: "memory");
}
FT_DEVICE void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
               "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
               "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
               "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :: "memory");
}

// acc += v * s, rounded once.  volatile: stays behind the wait for the accumulator column v.
FT_DEVICE void fma_col(float& acc, uint32_t v, float s) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(v)), "f"(s));
}

}  // namespace ftk
