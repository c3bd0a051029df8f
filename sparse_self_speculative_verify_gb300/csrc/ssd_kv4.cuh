// ssd_kv4.cuh -- the 4-bit (NVFP4) paged cache: its layout, and the conversions of its codes.
//
// A row of d elements (one token's K or V of one head) is d / 16 groups of 16 consecutive elements.
// A group has one scale s in e4m3 and 16 codes in e2m1 (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6); element
// i stands for code_i * s * (the cache's k_scale or v_scale).  A (page, K|V, head) block holds the
// codes of its page_size tokens (d / 2 bytes each, the even element of a pair in the low nibble), then
// their scales (d / 16 bytes each).
//
// A code has 2 significant bits and a scale 4, so code * s has 6 and its exponent lies in
// [2^-10, 2688]: the product is exact in f16, and what the attention kernels feed to the tensor cores
// carries no rounding beyond the cache's own.
#pragma once

#include "ssd_common.cuh"

namespace ssd {

constexpr int kKv4Group = 16;    // elements per scale
constexpr int kKv4MinPage = 8;   // smallest page: its blocks and their scale parts stay 16-byte multiples
__host__ __device__ constexpr int kv4_code_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int kv4_scale_bytes(int d) { return d / kKv4Group; }
__host__ __device__ constexpr int kv4_row_bytes(int d) { return kv4_code_bytes(d) + kv4_scale_bytes(d); }

// Four bytes of codes -> four f16 pairs (low nibble in the low half), exact.
__device__ __forceinline__ void e2m1_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{ .reg .b8 b0, b1, b2, b3;\n"
      "  mov.b32 {b0, b1, b2, b3}, %4;\n"
      "  cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "  cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "  cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "  cvt.rn.f16x2.e2m1x2 %3, b3; }\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight fp32 values -> eight codes (value k in nibble k), to nearest with ties to the even code; what
// is above 6 becomes 6.
__device__ __forceinline__ uint32_t f32_to_e2m1(const float *v) {
  uint32_t r;
  asm("{ .reg .b8 b0, b1, b2, b3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "  mov.b32 %0, {b0, b1, b2, b3}; }\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Two e4m3 bytes (low byte first) -> f16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }\n" : "=r"(r) : "r"(two));
  return r;
}

// fp32 -> e4m3 byte, to nearest with ties to even, saturating at 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float v) {
  uint32_t r;
  asm("{ .reg .b16 h; cvt.rn.satfinite.e4m3x2.f32 h, %2, %1; cvt.u32.u16 %0, h; }\n" : "=r"(r) : "f"(v), "f"(0.f));
  return r & 0xffu;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// D += A(16x16 f16, row) * B(16x8 f16, col), fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(a));
  return r;
}

}  // namespace ssd
