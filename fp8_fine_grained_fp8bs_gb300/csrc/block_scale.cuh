// Copies of block scales from shared to tensor memory, for the block-scaled
// MMAs (gemm_mx.cu, gemm_fp4.cu).
#pragma once

#include "common.cuh"

namespace fp8bs {
namespace {

// True in one thread of a converged warp.  The compiler knows the branch on
// it is taken by one thread with the warp's uniform values, so the operands
// of tensor-core and TMA instructions behind it stay in uniform registers:
// behind `lane == 0` each operand is moved there first, and the 4-bit GEMM's
// issuing thread (16 such instructions per stage) took twice the time its
// MMAs did (4096x7168x7168, E4M3x16: 150 us against 78).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(p));
  return p != 0;
}

// Shared-memory matrix descriptor of 32 rows x 16 bytes stored contiguously
// without swizzling (8-row core matrices 128 bytes apart), the source of
// tcgen05.cp.32x128b: start address, leading- and stride-dimension offsets
// (both 128 bytes), descriptor version 1 (bits 46-48), no swizzle.
__device__ __forceinline__ uint64_t sf_rows_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

// Copies 32 rows x 16 bytes from shared memory into four TMEM columns of
// every lane quarter: row i to lane 32q + i, bytes 4c..4c+3 to column c.
// Ordered with the issuing thread's MMAs (the same asynchronous pipe).
__device__ __forceinline__ void tmem_cp_rows(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// The same in both CTAs of a pair, each from its own shared memory into its
// own tensor memory (issued by the leader).
__device__ __forceinline__ void tmem_cp_rows_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

}  // namespace
}  // namespace fp8bs
