// pa_gather_cache: rows of K and V read back from the paged caches as 16-bit
// values, the inverse of the cache write.  A thread moves 16 values (one
// group of a four-bit cache, 32 bytes of output) of K and of V, stored as one
// access where the address allows it (as two, a warp's stores cover every
// other half sector: 77 us against 56 for 65536 tokens of 8 heads, head_dim
// 128, from four bits).  Those 56 us are 344 MB read and written, 6.1 TB/s.
// In a launch by itself part of the rows stays in L2 and DRAM is at 64% of
// its peak for as long: the latency of slot, code and store one after the
// other (22 cycles an instruction at 58 warps an SM) bounds it as much as
// memory does.  With slots in random order, of the same sizes: 71 us from
// four bits, 72 from one byte (403 MB), 91 from 16 bits (537 MB).
#include "pa_fp4.cuh"
#include "pa_host.h"

namespace pa {
namespace {

// 16 values from `in` (for kFP4 with their scale byte at `g8`)
template <int KV, int DST>
__device__ __forceinline__ Words32 read16(const uint8_t *in, const uint8_t *g8, float scale) {
  if constexpr (KV == kF16 || KV == kBF16) {
    return {__ldg(reinterpret_cast<const uint4 *>(in)), __ldg(reinterpret_cast<const uint4 *>(in) + 1)};
  } else {
    uint32_t h[8], o[8];  // fp16 pairs, results
    if constexpr (KV == kFP4) {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(in));
      const uint32_t g = __ldg(g8);
      const uint32_t g2 = e4m3x2_to_half2(g * 0x0101u);
      uint32_t x[4], y[4];
      e2m1x8_to_half2x4(w.x, x);
      e2m1x8_to_half2x4(w.y, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = hmul2_bits(x[i], g2);
        h[4 + i] = hmul2_bits(y[i], g2);
      }
    } else {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(in));
      byte4_to_half2x2<KV>(w.x, h[0], h[1]);
      byte4_to_half2x2<KV>(w.y, h[2], h[3]);
      byte4_to_half2x2<KV>(w.z, h[4], h[5]);
      byte4_to_half2x2<KV>(w.w, h[6], h[7]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = half2_bits_to_float2<kF16>(h[i]);
      o[i] = pack2_rn<DST>(f.x * scale, f.y * scale);
    }
    return {make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7])};
  }
}

// IDX: the type that counts the groups of 16.
template <int KV, int DST, class IDX>
__global__ void __launch_bounds__(256) gather_kernel(uint8_t *__restrict__ key, uint8_t *__restrict__ value,
                                                     const int64_t *__restrict__ slots, IDX total, bool wide,
                                                     uint32_t kv_heads, int gpr_shift, int bs_shift, long long num_slots,
                                                     const uint8_t *__restrict__ k_cache,
                                                     const uint8_t *__restrict__ v_cache, float k_scale, float v_scale,
                                                     const float *__restrict__ k_head_scales,
                                                     const float *__restrict__ v_head_scales, int *err) {
  launch_dependents();  // no block table or length is written here
  for (IDX i = blockIdx.x * static_cast<IDX>(256) + threadIdx.x; i < total; i += static_cast<IDX>(gridDim.x) * 256) {
    const uint32_t g = static_cast<uint32_t>(i) & ((1u << gpr_shift) - 1);
    const IDX th = i >> gpr_shift, t = th / kv_heads;
    const uint32_t h = static_cast<uint32_t>(th - t * kv_heads);
    const long long slot = __ldg(slots + t);
    if (slot < -1 || slot >= num_slots) {  // (-1: a padding row)
      if (h == 0 && g == 0) record_error(err, kErrSlot);
      continue;
    }
    Words32 k = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}, v = k;
    if (slot >= 0) {
      const uint32_t off = static_cast<uint32_t>(slot) & ((1u << bs_shift) - 1);
      const size_t tile = static_cast<size_t>(slot >> bs_shift) * kv_heads + h;
      float sk = k_scale, sv = v_scale;
      if (k_head_scales != nullptr) {
        sk = __ldg(k_head_scales + h);
        sv = __ldg(v_head_scales + h);
      }
      if constexpr (KV == kFP4) {  // 8 bytes of codes a group, then the scales [group][token]
        const size_t at = tile * (9u << (gpr_shift + bs_shift));
        const size_t g8 = at + (8u << (gpr_shift + bs_shift)) + (g << bs_shift) + off;
        const size_t in = at + (off << (gpr_shift + 3)) + g * 8;
        k = read16<KV, DST>(k_cache + in, k_cache + g8, sk);
        v = read16<KV, DST>(v_cache + in, v_cache + g8, sv);
      } else {
        const size_t in = (((tile << bs_shift) + off) << gpr_shift | g) * (kFp4Group * elt_bytes(KV));
        k = read16<KV, DST>(k_cache + in, nullptr, sk);
        v = read16<KV, DST>(v_cache + in, nullptr, sv);
      }
    }
    store32(key + static_cast<size_t>(i) * 32, k, wide);
    store32(value + static_cast<size_t>(i) * 32, v, wide);
  }
}

template <int KV, int DST>
void launch_gather(void *key, void *value, const int64_t *slots, int num_tokens, const void *k_cache,
                   const void *v_cache, const pa_cache_desc *c, int *err, cudaStream_t stream) {
  const int gpr_shift = c->head_dim == 64 ? 2 : 3, bs_shift = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
  const long long groups = static_cast<long long>(num_tokens) * c->kv_heads << gpr_shift;
  const long long num_slots = static_cast<long long>(c->num_blocks) * c->block_size;
  const int blocks = grid_for(groups, 256);
  const bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31u) == 0;
  auto go = [&](auto kern, auto total) {
    kern<<<blocks, 256, 0, stream>>>(static_cast<uint8_t *>(key), static_cast<uint8_t *>(value), slots, total, wide,
                                     c->kv_heads, gpr_shift, bs_shift, num_slots, static_cast<const uint8_t *>(k_cache),
                                     static_cast<const uint8_t *>(v_cache), c->k_scale, c->v_scale, c->k_head_scales,
                                     c->v_head_scales, err);
  };
  // (32-bit indexes divide in a quarter of the instructions; the last step past the end must not wrap)
  if (groups < 0xf0000000ll)
    go(gather_kernel<KV, DST, uint32_t>, static_cast<uint32_t>(groups));
  else
    go(gather_kernel<KV, DST, uint64_t>, static_cast<uint64_t>(groups));
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
  const bool f16 = dst_dtype == PA_F16;
  decltype(&launch_gather<kF16, kF16>) go = nullptr;
  switch (kv) {
    case PA_F16: go = launch_gather<kF16, kF16>; break;
    case PA_BF16: go = launch_gather<kBF16, kBF16>; break;
    case PA_FP8_E4M3: go = f16 ? launch_gather<kE4M3, kF16> : launch_gather<kE4M3, kBF16>; break;
    case PA_FP8_E5M2: go = f16 ? launch_gather<kE5M2, kF16> : launch_gather<kE5M2, kBF16>; break;
    case PA_INT8: go = f16 ? launch_gather<kI8, kF16> : launch_gather<kI8, kBF16>; break;
    default: go = f16 ? launch_gather<kFP4, kF16> : launch_gather<kFP4, kBF16>; break;
  }
  go(key, value, slot_mapping, num_tokens, k_cache, v_cache, cache, device_error,
     reinterpret_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}
