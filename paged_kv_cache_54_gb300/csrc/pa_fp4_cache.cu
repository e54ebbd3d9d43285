// Cache write in four bits.
//
// A thread takes one group of 16 dimensions of one row, of K and of V: the
// group's scale needs no other thread, 32 bytes of each are in flight, and the
// stores of a row's groups are consecutive 8-byte runs of codes.  Moving the
// rows bounds it (2 bytes in and 9/16 out an element) as long as an element
// costs few instructions: at the HBM rate an SM has about 14 of them for
// each (128 lanes x 1.9 GHz over 9 elements a clock).  Two divisions an
// element would be more than that, so:
//   - the quotient by a group's scale g uses one reciprocal a group.  With
//     r the correctly rounded 1 / g, q0 = y r and the exact remainder
//     e = y - q0 g (an fma), q0 + e r is the correctly rounded y / g
//     (Markstein, IBM J. Res. Dev. 34, 1990), so ties stay ties and the
//     conversion to e2m1 rounds them to even;
//   - the quotient by the head's scale the same way, and not at all when that
//     is 1;
//   - groups that those steps do not hold for (NaN, infinities, quotients out
//     of range) are found on the packed 16-bit values and go the long way.
// 65536 tokens of 8 heads, head_dim 128, per-head scales: 62 us (344 MB, 5.5
// TB/s; the bytes alone 51 us), 12 instructions an element, 70% of the issue
// slots.  More CTAs an SM with fewer registers took longer (five 9%, six 16%).
#include "pa_fp4.cuh"
#include "pa_fp4.h"

namespace pa {
namespace {

// a / b in the binary32 arithmetic above: r is 1 / b correctly rounded, and
// neither quotient nor remainder overflows or matters when it underflows.
__device__ __forceinline__ float divide(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(q, -b, a), r, q);
}
// The negated quotient of two values at once (packed arithmetic, each lane
// rounded as the scalar): b is the divisor twice, nr is -r twice.  A zero
// keeps its sign this way round: for a = -0 the steps are q = +0, e = +0 + -0
// = +0, -0 + +0 = +0, and for a = +0 they end in -0 (with the positive
// quotient the last sum would be +0 for both).
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint64_t negated_quotient(uint64_t a, uint64_t b, uint64_t nr) {
  uint64_t q, e, d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(a), "l"(nr));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q), "l"(b), "l"(a));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(e), "l"(nr), "l"(q));
  return d;
}

// e2m1 codes of -y / g of 16 values (g2 is g twice, nrg -1 / g twice)
__device__ __forceinline__ uint2 e2m1_codes(const uint64_t (&y)[8], uint64_t g2, uint64_t nrg) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("{\n\t.reg .b8 b;\n\t.reg .f32 x, y;\n\tmov.b64 {x, y}, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, y, x;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(c[i])
        : "l"(negated_quotient(y[i], g2, nrg)));
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

// e2m1 code of y / g in the low four bits: nearest, ties to even, +-6 beyond;
// 0 for NaN.  g > 0.
__device__ __forceinline__ uint32_t e2m1_code(float y, float g) {
  if (y != y) return 0u;
  const float q = __fdiv_rn(fabsf(y), g);
  const uint32_t m = (q > 0.25f) + (q >= 0.75f) + (q > 1.25f) + (q >= 1.75f) + (q > 2.5f) + (q >= 3.5f) + (q > 5.f);
  return m | (signbit(y) ? 8u : 0u);
}

// A group by divisions, NaN left out: any input.  Codes and scale byte.
template <int SRC>
__device__ __noinline__ uint3 quantise_any(uint4 a, uint4 b, float scale) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = half2_bits_to_float2<SRC>(w[i]);
    top = fmaxf(top, fmaxf(fabsf(__fdiv_rn(f.x, scale)), fabsf(__fdiv_rn(f.y, scale))));  // (fmaxf leaves NaN out)
  }
  const uint32_t g8 = __nv_cvt_float_to_fp8(__fdiv_rn(top, 6.f), __NV_SATFINITE, __NV_E4M3);
  const float g = byte2_to_float2<kE4M3>(g8).x;
  uint32_t c[2] = {0u, 0u};
  if (g8 != 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = half2_bits_to_float2<SRC>(w[i]);
      c[i >> 2] |= (e2m1_code(__fdiv_rn(f.x, scale), g) | e2m1_code(__fdiv_rn(f.y, scale), g) << 4) << (8 * (i & 3));
    }
  }
  return make_uint3(c[0], c[1], g8);
}

// largest magnitude of the 16 values, NaN if there is one
template <int SRC>
__device__ __forceinline__ float largest(const uint32_t (&w)[8]) {
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    if constexpr (SRC == kF16)
      asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(a));
    else
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(a));
  }
  const float2 f = half2_bits_to_float2<SRC>(m);
  return f.x != f.x ? f.x : f.y != f.y ? f.y : fmaxf(f.x, f.y);
}

// One group: 16 values (32 bytes) -> 8 bytes of codes and the e4m3 scale
// byte.  r is 1 / scale correctly rounded, `plain` whether scale lies
// within 2^-60 .. 2^60; table[c] is the value of scale code c and its
// reciprocal.
template <int SRC>
__device__ __forceinline__ uint3 quantise_group(uint4 a, uint4 b, float scale, float r, bool plain,
                                                const float2 *table) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const float top = largest<SRC>(w);
  if (!(plain && top <= 0x1p60f)) return quantise_any<SRC>(a, b, scale);  // (NaN too)
  // (the quotient of the largest is the largest quotient: rounding keeps order)
  const float ytop = scale == 1.f ? top : divide(top, scale, r);
  const uint32_t g8 = __nv_cvt_float_to_fp8(divide(ytop, 6.f, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
  if (g8 == 0) return make_uint3(0u, 0u, 0u);
  const float2 g = table[g8];
  const uint64_t g2 = twice(g.x), nrg = twice(-g.y), s2 = twice(scale), nrs = twice(-r);
  uint64_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = half2_bits_to_float2<SRC>(w[i]);
    asm("mov.b64 %0, {%1, %2};" : "=l"(y[i]) : "f"(f.x), "f"(f.y));
  }
  // (both quotients, or one and the codes' signs turned round)
  if (scale == 1.f) {
    const uint2 c = e2m1_codes(y, g2, nrg);
    return make_uint3(c.x ^ 0x88888888u, c.y ^ 0x88888888u, g8);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = negated_quotient(y[i], s2, nrs);
  const uint2 c = e2m1_codes(y, g2, nrg);
  return make_uint3(c.x, c.y, g8);
}

// GPR: groups of a row.  A thread keeps one head and group (idx of the
// kv_heads * GPR of a token) and walks the tokens t, t + step, ...: its scales
// and places are set up once, and no index is divided on the way.
template <int SRC, int GPR>
__global__ void __launch_bounds__(256) write_fp4_kernel(
    const uint8_t *__restrict__ key, const uint8_t *__restrict__ value, const int64_t *__restrict__ slots,
    int num_tokens, int step, bool wide, uint32_t kv_heads, int bs_shift, long long num_slots,
    uint8_t *__restrict__ k_cache, uint8_t *__restrict__ v_cache, float k_scale, float v_scale,
    const float *__restrict__ k_head_scales, const float *__restrict__ v_head_scales, int *err) {
  __shared__ float2 table[128];
  launch_dependents();  // no block table or length is written here
  if (threadIdx.x < 128) {
    const float g = byte2_to_float2<kE4M3>(threadIdx.x).x;
    table[threadIdx.x] = make_float2(g, __frcp_rn(g));
  }
  __syncthreads();
  const uint32_t code_bytes = 8u * GPR << bs_shift, tile = 9u * GPR << bs_shift, bs_mask = (1u << bs_shift) - 1;
  const long long per_token = static_cast<long long>(kv_heads) * GPR, places = per_token * step;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < places; i += gridDim.x * 256ll) {
    const int t0 = static_cast<int>(i / per_token);
    const uint32_t idx = static_cast<uint32_t>(i - t0 * per_token), h = idx / GPR, g = idx % GPR;
    float sk = k_scale, sv = v_scale;
    if (k_head_scales != nullptr) {
      sk = __ldg(k_head_scales + h);
      sv = __ldg(v_head_scales + h);
    }
    const float rk = __frcp_rn(sk), rv = __frcp_rn(sv);
    const bool pk = sk >= 0x1p-60f && sk <= 0x1p60f, pv = sv >= 0x1p-60f && sv <= 0x1p60f;
    const size_t head = static_cast<size_t>(h) * tile;
    // the next token's rows are loaded while this one's are quantised
    long long slot_n = __ldg(slots + t0);
    const size_t src0 = (static_cast<size_t>(t0) * per_token + idx) * 32;
    const size_t stride = static_cast<size_t>(step) * per_token * 32;
    const uint8_t *ks = key + src0, *vs = value + src0;
    Words32 k_n = load32(ks, wide), v_n = load32(vs, wide);
    for (long long t = t0; t < num_tokens; t += step) {
      const long long slot = slot_n;
      const Words32 k = k_n, v = v_n;
      if (t + step < num_tokens) {
        slot_n = __ldg(slots + t + step);
        ks += stride;
        vs += stride;
        k_n = load32(ks, wide);
        v_n = load32(vs, wide);
      }
      if (slot < 0) continue;  // padding row
      if (slot >= num_slots) {
        if (idx == 0) record_error(err, kErrSlot);
        continue;
      }
      const uint32_t off = static_cast<uint32_t>(slot) & bs_mask;
      const size_t base = static_cast<size_t>(slot >> bs_shift) * kv_heads * tile + head;
      const size_t at = base + off * (8 * GPR) + g * 8, sat = base + code_bytes + (g << bs_shift) + off;
      const uint3 ck = quantise_group<SRC>(k.a, k.b, sk, rk, pk, table);
      *reinterpret_cast<uint2 *>(k_cache + at) = make_uint2(ck.x, ck.y);
      k_cache[sat] = static_cast<uint8_t>(ck.z);
      const uint3 cv = quantise_group<SRC>(v.a, v.b, sv, rv, pv, table);
      *reinterpret_cast<uint2 *>(v_cache + at) = make_uint2(cv.x, cv.y);
      v_cache[sat] = static_cast<uint8_t>(cv.z);
    }
  }
}

template <int SRC, int GPR>
void launch_write(const void *key, const void *value, const int64_t *slots, int num_tokens, void *k_cache,
                  void *v_cache, const pa_cache_desc *c, int *err, cudaStream_t stream) {
  const int shift = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
  const long long num_slots = static_cast<long long>(c->num_blocks) * c->block_size;
  const long long per_token = static_cast<long long>(c->kv_heads) * GPR;
  const int blocks = grid_for(num_tokens * per_token, 256);
  const bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31u) == 0;
  long long step = blocks * 256ll / per_token;  // tokens that the grid holds at a time
  if (step < 1) step = 1;
  if (step > num_tokens) step = num_tokens;
  write_fp4_kernel<SRC, GPR><<<blocks, 256, 0, stream>>>(
      static_cast<const uint8_t *>(key), static_cast<const uint8_t *>(value), slots, num_tokens,
      static_cast<int>(step), wide, c->kv_heads, shift, num_slots, static_cast<uint8_t *>(k_cache),
      static_cast<uint8_t *>(v_cache), c->k_scale, c->v_scale, c->k_head_scales, c->v_head_scales, err);
}

}  // namespace

pa_status write_fp4(const void *key, const void *value, int src_dtype, const int64_t *slots, int num_tokens,
                    void *k_cache, void *v_cache, const pa_cache_desc *cache, int *err, cudaStream_t stream) {
  auto *go = src_dtype == PA_F16 ? (cache->head_dim == 64 ? launch_write<kF16, 4> : launch_write<kF16, 8>)
                                 : (cache->head_dim == 64 ? launch_write<kBF16, 4> : launch_write<kBF16, 8>);
  go(key, value, slots, num_tokens, k_cache, v_cache, cache, err, stream);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace pa
