// pa_gather_cache: rows of K and V read back from the paged caches as 16-bit
// values, the inverse of the cache write.  A thread moves eight values (16
// bytes of output) of K and of V.
#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {
namespace {

// eight values from `in` (their group's scale byte at `g8` for kFP4) -> 16-bit words
template <int KV, int DST>
__device__ __forceinline__ uint4 read8(const uint8_t *in, const uint8_t *g8, float scale) {
  if constexpr (KV == kF16 || KV == kBF16) {
    return __ldg(reinterpret_cast<const uint4 *>(in));
  } else {
    uint32_t o[4];
    if constexpr (KV == kFP4) {
      uint32_t h[4];
      e2m1x8_to_half2x4(__ldg(reinterpret_cast<const uint32_t *>(in)), h);
      const uint32_t g = __ldg(g8);
      const uint32_t g2 = e4m3x2_to_half2(g | (g << 8));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = half2_bits_to_float2<kF16>(hmul2_bits(h[i], g2));
        o[i] = pack2_rn<DST>(f.x * scale, f.y * scale);
      }
    } else {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(in));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = byte2_to_float2<KV>((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
        o[i] = pack2_rn<DST>(f.x * scale, f.y * scale);
      }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int KV, int DST>
__global__ void __launch_bounds__(256) gather_kernel(uint8_t *__restrict__ key, uint8_t *__restrict__ value,
                                                     const int64_t *__restrict__ slots, int num_tokens, int kv_heads,
                                                     int head_dim, int block_size, long long num_slots,
                                                     const uint8_t *__restrict__ k_cache,
                                                     const uint8_t *__restrict__ v_cache, float k_scale, float v_scale,
                                                     const float *__restrict__ k_head_scales,
                                                     const float *__restrict__ v_head_scales, int *err) {
  launch_dependents();  // no block table or length is written here
  const int cpr = head_dim / 8;  // 16-byte chunks of an output row
  const long long total = static_cast<long long>(num_tokens) * kv_heads * cpr;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int c = static_cast<int>(i % cpr);
    const long long th = i / cpr;
    const int h = static_cast<int>(th % kv_heads);
    const long long t = th / kv_heads;
    const long long slot = __ldg(slots + t);
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (slot >= num_slots) {
      if (h == 0 && c == 0) record_error(err, kErrSlot);
      continue;
    }
    if (slot >= 0) {
      const long long blk = slot / block_size;
      const int off = static_cast<int>(slot - blk * block_size);
      const size_t tile = static_cast<size_t>(blk) * kv_heads + h;
      const float sk = k_head_scales != nullptr ? __ldg(k_head_scales + h) : k_scale;
      const float sv = v_head_scales != nullptr ? __ldg(v_head_scales + h) : v_scale;
      if constexpr (KV == kFP4) {
        const size_t at = tile * (block_size * fp4_row_bytes(head_dim));
        const size_t g8 = at + block_size * fp4_code_bytes(head_dim) + (c / 2) * block_size + off;
        const size_t in = at + off * fp4_code_bytes(head_dim) + c * 4;
        k = read8<KV, DST>(k_cache + in, k_cache + g8, sk);
        v = read8<KV, DST>(v_cache + in, v_cache + g8, sv);
      } else {
        const size_t in = ((tile * block_size + off) * head_dim + c * 8) * elt_bytes(KV);
        k = read8<KV, DST>(k_cache + in, nullptr, sk);
        v = read8<KV, DST>(v_cache + in, nullptr, sv);
      }
    }
    reinterpret_cast<uint4 *>(key)[i] = k;
    reinterpret_cast<uint4 *>(value)[i] = v;
  }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_gather_cache(void *key, void *value, int32_t dst_dtype, const int64_t *slot_mapping,
                                     int32_t num_tokens, const void *k_cache, const void *v_cache,
                                     const pa_cache_desc *cache, int *device_error, pa_stream_t stream) {
  if (!valid_cache_desc(cache) || num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PA_ERR_INVALID;
  if (dst_dtype != PA_F16 && dst_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (!supported_cache_shape(cache)) return PA_ERR_UNSUPPORTED;
  const int kv = cache->dtype;
  if ((kv == PA_F16 || kv == PA_BF16) && kv != dst_dtype) return PA_ERR_UNSUPPORTED;
  const int threads = 256;
  const int blocks =
      grid_for(static_cast<long long>(num_tokens) * cache->kv_heads * (cache->head_dim / 8), threads);
  auto launch = [&](auto kern) {
    kern<<<blocks, threads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<uint8_t *>(key), static_cast<uint8_t *>(value), slot_mapping, num_tokens, cache->kv_heads,
        cache->head_dim, cache->block_size, static_cast<long long>(cache->num_blocks) * cache->block_size,
        static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache), cache->k_scale, cache->v_scale,
        cache->k_head_scales, cache->v_head_scales, device_error);
  };
  const bool f16 = dst_dtype == PA_F16;
  switch (kv) {
    case PA_F16: launch(gather_kernel<kF16, kF16>); break;
    case PA_BF16: launch(gather_kernel<kBF16, kBF16>); break;
    case PA_FP8_E4M3: launch(f16 ? gather_kernel<kE4M3, kF16> : gather_kernel<kE4M3, kBF16>); break;
    case PA_FP8_E5M2: launch(f16 ? gather_kernel<kE5M2, kF16> : gather_kernel<kE5M2, kBF16>); break;
    case PA_INT8: launch(f16 ? gather_kernel<kI8, kF16> : gather_kernel<kI8, kBF16>); break;
    case PA_FP4: launch(f16 ? gather_kernel<kFP4, kF16> : gather_kernel<kFP4, kBF16>); break;
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}
