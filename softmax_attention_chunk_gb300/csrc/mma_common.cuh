// Warp MMAs of the streaming paged kernels (bf16 operands, fp32 accumulators) and their helpers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pathattn {

// C (16 x 8) += A (16 x 16) B (16 x 8).  Lane (g = lane / 4, t = lane % 4) holds A rows g, g + 8 at columns
// 2t, 2t+1 (a0, a1) and 2t+8, 2t+9 (a2, a3), B rows 2t, 2t+1 (b0) and 2t+8, 2t+9 (b1) of column g, and C rows
// g (c0, c1), g + 8 (c2, c3) at columns 2t, 2t+1.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same over 8 columns of A (a0, a1) and 8 rows of B (b0).
__device__ __forceinline__ void mma_bf16_k8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(b0));
}
// Transposes an 8 x 8 matrix of 16-bit elements held two per lane: in, lane (g, t) has row g at columns 2t, 2t+1;
// out, it has rows 2t, 2t+1 of column g.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// x as a bf16 pair and what the pair leaves (about 16 significant bits together).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b);
  lo = pack2(a - lo_f(hi), b - hi_f(hi));
}

}  // namespace pathattn
