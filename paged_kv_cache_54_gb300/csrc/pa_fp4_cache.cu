// Cache write in four bits: each thread takes one group of 16 dimensions of
// one row of K and of V, so that the group's scale needs no other thread.
#include "pa_fp4.cuh"
#include "pa_fp4.h"

namespace pa {
namespace {

// e2m1 code of y / g in the low four bits: nearest, ties to even, +-6 beyond;
// 0 for NaN.  g > 0.
__device__ __forceinline__ uint32_t e2m1_code(float y, float g) {
  if (y != y) return 0u;
  const float q = __fdiv_rn(fabsf(y), g);
  const uint32_t m = (q > 0.25f) + (q >= 0.75f) + (q > 1.25f) + (q >= 1.75f) + (q > 2.5f) + (q >= 3.5f) + (q > 5.f);
  return m | (signbit(y) ? 8u : 0u);
}

// One group: 16 values at `in` -> 8 bytes of codes and the e4m3 scale byte.
template <int SRC>
__device__ __forceinline__ uint32_t quantise_group(const uint8_t *in, float scale, uint2 &codes) {
  const uint4 a = __ldg(reinterpret_cast<const uint4 *>(in));
  const uint4 b = __ldg(reinterpret_cast<const uint4 *>(in) + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float y[16], top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = half2_bits_to_float2<SRC>(w[i]);
    y[2 * i] = __fdiv_rn(f.x, scale);
    y[2 * i + 1] = __fdiv_rn(f.y, scale);
    top = fmaxf(top, fmaxf(fabsf(y[2 * i]), fabsf(y[2 * i + 1])));  // fmaxf leaves NaN out
  }
  const uint32_t g8 = __nv_cvt_float_to_fp8(__fdiv_rn(top, 6.f), __NV_SATFINITE, __NV_E4M3);
  const float g = byte2_to_float2<kE4M3>(g8).x;
  codes = make_uint2(0u, 0u);
  if (g8 != 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      codes.x |= e2m1_code(y[i], g) << (4 * i);
      codes.y |= e2m1_code(y[8 + i], g) << (4 * i);
    }
  }
  return g8;
}

template <int SRC>
__global__ void __launch_bounds__(256) write_fp4_kernel(
    const uint8_t *__restrict__ key, const uint8_t *__restrict__ value, const int64_t *__restrict__ slots,
    int num_tokens, int kv_heads, int head_dim, int block_size, long long num_slots, uint8_t *__restrict__ k_cache,
    uint8_t *__restrict__ v_cache, float k_scale, float v_scale, const float *__restrict__ k_head_scales,
    const float *__restrict__ v_head_scales, int *err) {
  launch_dependents();  // no block table or length is written here
  const int gpr = head_dim / kFp4Group;  // groups of a row
  const int code_bytes = block_size * fp4_code_bytes(head_dim);
  const long long tile = code_bytes + block_size * gpr;
  const long long total = static_cast<long long>(num_tokens) * kv_heads * gpr;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int g = static_cast<int>(i % gpr);
    const long long th = i / gpr;
    const int h = static_cast<int>(th % kv_heads);
    const long long t = th / kv_heads;
    const long long slot = __ldg(slots + t);
    if (slot < 0) continue;  // padding row
    if (slot >= num_slots) {
      if (h == 0 && g == 0) record_error(err, kErrSlot);
      continue;
    }
    const long long blk = slot / block_size;
    const int off = static_cast<int>(slot - blk * block_size);
    const size_t base = (static_cast<size_t>(blk) * kv_heads + h) * tile;
    const size_t src = (static_cast<size_t>(th) * head_dim + g * kFp4Group) * 2;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float *head_scales = which == 0 ? k_head_scales : v_head_scales;
      const float scale = head_scales != nullptr ? __ldg(head_scales + h) : (which == 0 ? k_scale : v_scale);
      uint8_t *out = (which == 0 ? k_cache : v_cache) + base;
      uint2 codes;
      const uint32_t g8 = quantise_group<SRC>((which == 0 ? key : value) + src, scale, codes);
      *reinterpret_cast<uint2 *>(out + off * (head_dim / 2) + g * 8) = codes;
      out[code_bytes + g * block_size + off] = static_cast<uint8_t>(g8);
    }
  }
}

}  // namespace

pa_status write_fp4(const void *key, const void *value, int src_dtype, const int64_t *slots, int num_tokens,
                    void *k_cache, void *v_cache, const pa_cache_desc *cache, int *err, cudaStream_t stream) {
  const long long work = static_cast<long long>(num_tokens) * cache->kv_heads * (cache->head_dim / kFp4Group);
  const int threads = 256;
  auto *kern = src_dtype == PA_F16 ? write_fp4_kernel<kF16> : write_fp4_kernel<kBF16>;
  kern<<<grid_for(work, threads), threads, 0, stream>>>(
      static_cast<const uint8_t *>(key), static_cast<const uint8_t *>(value), slots, num_tokens, cache->kv_heads,
      cache->head_dim, cache->block_size, static_cast<long long>(cache->num_blocks) * cache->block_size,
      static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), cache->k_scale, cache->v_scale,
      cache->k_head_scales, cache->v_head_scales, err);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace pa
