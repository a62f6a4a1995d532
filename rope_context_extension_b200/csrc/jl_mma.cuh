// Warp-level matrix helpers of the decode kernels: ldmatrix, mma.sync m16n8k16
// (bf16 or fp16 operands, fp32 accumulators), and the rotation of packed bf16 pairs
// into hi + lo bf16 parts.
#pragma once

#include "jl_common.cuh"

namespace jl {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bf16x2 word -> packed fp32x2 (exact)
__device__ __forceinline__ uint64_t bf16x2_to_f2(uint32_t w) { return f2_pack(bf16lo_to_f32(w), bf16hi_to_f32(w)); }

// Packed pair v = (a, b) -> bf16x2 hi = round(a, b) and lo = round((a, b) - hi).
__device__ __forceinline__ void split_f2_bf16(uint64_t v, uint32_t& hi, uint32_t& lo) {
  float a, b;
  f2_unpack(v, a, b);
  hi = pack_bf16x2(a, b);
  const uint64_t r = f2_sub(v, bf16x2_to_f2(hi));
  float ra, rb;
  f2_unpack(r, ra, rb);
  lo = pack_bf16x2(ra, rb);
}

// Rotate the bf16 pairs (x, y) of two adjacent RoPE pairs by the factors
// f = (c0, c1, s0, s1) and return the results as hi / lo bf16 parts:
// x' = x c - y s, y' = y c + x s.
__device__ __forceinline__ void rot_split_bf16(uint32_t xw, uint32_t yw, const float4& f, uint32_t& xh, uint32_t& xl,
                                               uint32_t& yh, uint32_t& yl) {
  const uint64_t x = bf16x2_to_f2(xw), y = bf16x2_to_f2(yw);
  const uint64_t c = f2_pack(f.x, f.y), sn = f2_pack(f.z, f.w);
  const uint64_t xr = f2_sub(f2_mul(x, c), f2_mul(y, sn));
  const uint64_t yr = f2_fma(x, sn, f2_mul(y, c));
  split_f2_bf16(xr, xh, xl);
  split_f2_bf16(yr, yh, yl);
}

}  // namespace jl
