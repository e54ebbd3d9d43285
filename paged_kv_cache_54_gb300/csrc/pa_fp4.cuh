// Device helpers of the four-bit cache format: e2m1 codes, two to a byte,
// with one e4m3 scale for every 16.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kFp4Group = 16;

// bytes of one token's row of one head: its codes, its scales, both
__host__ __device__ constexpr int fp4_code_bytes(int head_dim) { return head_dim / 2; }
__host__ __device__ constexpr int fp4_scale_bytes(int head_dim) { return head_dim / kFp4Group; }
__host__ __device__ constexpr int fp4_row_bytes(int head_dim) { return head_dim / 16 * 9; }

// Eight codes in one word -> four half2 (code 2i in the low half of o[i]).
// Every e2m1 value is an fp16 value, so this is exact.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Two e4m3 scales (low byte first) -> half2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t d;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(d) : "r"(two));
  return d;
}

// The product of a code (at most two significant bits, at most 6) and a
// group scale (four bits, at most 448) has at most six significant bits, is
// at most 2688 and a multiple of 2^-10: every one is an fp16 value, so this
// multiplication is exact.
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Power of two that a bf16 query row is multiplied by before it is rounded
// to fp16 (its scores' multiplier becomes scale / it): its largest magnitude,
// top, comes to lie in [2^13, 2^14), so that nothing overflows and what
// underflows is 2^-38 of the largest.  It stays small enough for the
// multiplier to be a normal number, at least 2^-101: a multiplier that
// underflowed to zero would turn masked scores into NaN.  (Where that limit
// holds, the scores are below 2^-50 whatever the keys are.)  1 for rows of
// zeros and rows with an infinity.
__device__ __forceinline__ float query_factor(float top, float scale) {
  if (!(top > 0.f && top < INFINITY)) return 1.f;
  int e, es = 0;
  frexpf(top, &e);
  if (fabsf(scale) < 1.f) frexpf(scale, &es);
  return ldexpf(1.f, min(min(14 - e, 126), es + 100));
}

// 32 bytes as one access where the address allows it (two of 16 otherwise):
// lanes then touch whole sectors of consecutive addresses.
struct Words32 {
  uint4 a, b;
};
__device__ __forceinline__ Words32 load32(const uint8_t *p, bool wide) {
  Words32 w;
  if (wide) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w.a.x), "=r"(w.a.y), "=r"(w.a.z), "=r"(w.a.w), "=r"(w.b.x), "=r"(w.b.y), "=r"(w.b.z), "=r"(w.b.w)
        : "l"(p));
  } else {
    w.a = __ldg(reinterpret_cast<const uint4 *>(p));
    w.b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
  return w;
}
__device__ __forceinline__ void store32(uint8_t *p, const Words32 &w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w.a.x), "r"(w.a.y),
                 "r"(w.a.z), "r"(w.a.w), "r"(w.b.x), "r"(w.b.y), "r"(w.b.z), "r"(w.b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = w.a;
    reinterpret_cast<uint4 *>(p)[1] = w.b;
  }
}

}  // namespace pa
