// sm_100a building blocks of the sequence operators beside sm100.cuh's: tiles of four-dimensional
// tensors, products issued by a whole warp, and a load from two places of tensor memory.
#pragma once

#include <cstdint>

#include "sm100.cuh"

namespace rehyat {
namespace sm100 {

// Four-dimensional tile load and store (column, row, head, sequence of a strided tensor), with the
// checks of the three-dimensional ones in debug-bounds builds: the inner coordinate a multiple of
// 8 elements below two 64-column boxes, row, head and sequence inside the tensor.
__device__ __forceinline__ bool coord_4d_ok(int site, int c0, int c1, int c2, int c3, int ext1,
                                            int ext2, int ext3) {
#ifdef REHYAT_DEBUG_BOUNDS
  return bounds_ok(site, c0 & 7, 0, 1) & bounds_ok(site, c0, 0, 128) &
         bounds_ok(site, c1, 0, ext1) & bounds_ok(site, c2, 0, ext2) & bounds_ok(site, c3, 0, ext3);
#else
  (void)site, (void)c0, (void)c1, (void)c2, (void)c3, (void)ext1, (void)ext2, (void)ext3;
  return true;
#endif
}
__device__ __forceinline__ void tma_load_4d_chk(int site, void* dst, const CUtensorMap* map,
                                                uint64_t* bar, int c0, int c1, int c2, int c3,
                                                int ext1, int ext2, int ext3) {
  if (!coord_4d_ok(site, c0, c1, c2, c3, ext1, ext2, ext3)) c0 = c1 = c2 = c3 = 0;
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_store_4d_chk(int site, const CUtensorMap* map, const void* src,
                                                 int c0, int c1, int c2, int c3, int ext1,
                                                 int ext2, int ext3) {
  if (!coord_4d_ok(site, c0, c1, c2, c3, ext1, ext2, ext3)) return;
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
      ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// mma_ss, mma_ts and mma_commit issued by the one lane whose `leader` is non-zero, without a branch:
// the whole warp computes the descriptors, so they can stay in uniform registers, which the
// instruction takes its operands from.  Inside an `if (lane == 0)` every operand is moved there one by
// one, about 130 clk a product instead of the 64 it runs.
__device__ __forceinline__ void mma_ss_by(uint32_t leader, uint32_t d_tmem, uint64_t a_desc,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts_by(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                          uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_commit_by(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e;
}

// Load 32 consecutive columns from each of two places with one wait.
__device__ __forceinline__ void tmem_ld32_pair(uint32_t taddr0, uint32_t taddr1,
                                               uint32_t (&r0)[32], uint32_t (&r1)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, "
      "%41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, "
      "%58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : REHYAT_R32(r0, 0), REHYAT_R32(r1, 0)
      : "r"(taddr0), "r"(taddr1)
      : "memory");
}

}  // namespace sm100
}  // namespace rehyat
