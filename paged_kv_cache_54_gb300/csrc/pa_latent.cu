// pa_latent_write: new tokens' rows of the latent cache, and the cache's
// tensor-map view.
//
// A token's row is 72 pieces of 16 bytes, 64 of its latent vector and 8 of
// its rotary key; a thread copies four pieces, all loaded before the first is
// stored.  Bound by memory: 32768 tokens, 36 MB read and as much written, take
// 15.5 us from DRAM (10.8 at the measured copy rate: the slots' loads lie ahead
// of the rows', in each of two passes of the grid), 11 where the rows are in L2.
#include "pa_common.cuh"
#include "pa_latent.h"

namespace pa {

bool encode_latent_view(CUtensorMap *map, const void *cache, const pa_latent_desc *c, int columns, int groups) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t row = kLatentRow * 2;
  const cuuint64_t dims[4] = {64, 8, kLatentRow / 64,
                              static_cast<cuuint64_t>(c->num_blocks) * (c->block_size / 8)};
  const cuuint64_t strides[3] = {row, 128, row * 8};
  const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(columns), static_cast<cuuint32_t>(groups)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(cache), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kPieces = kLatentRow / 8;
constexpr int kLatentPieces = kLatentDim / 8;
constexpr int kWriteThreads = 256;
constexpr int kUnroll = 4;

template <typename INDEX>
__global__ void __launch_bounds__(kWriteThreads) latent_write_kernel(
    const uint16_t *__restrict__ latent, const uint16_t *__restrict__ rope, INDEX latent_stride, INDEX rope_stride,
    const int64_t *__restrict__ slots, INDEX pieces, long long num_slots, uint16_t *__restrict__ cache, int *err) {
  const INDEX threads = static_cast<INDEX>(gridDim.x) * kWriteThreads;
  const INDEX me = static_cast<INDEX>(blockIdx.x) * kWriteThreads + threadIdx.x;
  for (INDEX i0 = 0; i0 < pieces; i0 += threads * kUnroll) {
    uint4 x[kUnroll];
    uint16_t *to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const INDEX i = i0 + me + threads * u;
      to[u] = nullptr;
      if (i < pieces) {
        const INDEX t = i / kPieces;
        const int c = static_cast<int>(i - t * kPieces);
        const int64_t slot = __ldg(slots + t);
        if (slot >= 0 && slot < num_slots) {
          const uint16_t *from = c < kLatentPieces ? latent + t * latent_stride + c * 8
                                                   : rope + t * rope_stride + (c - kLatentPieces) * 8;
          x[u] = __ldcs(reinterpret_cast<const uint4 *>(from));
          to[u] = cache + slot * kLatentRow + c * 8;
        } else if (slot != -1 && c == 0) {
          record_error(err, kErrSlot);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (to[u] != nullptr) *reinterpret_cast<uint4 *>(to[u]) = x[u];
  }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_latent_write(const void *latent, const void *rope, int64_t latent_stride, int64_t rope_stride,
                                     int32_t src_dtype, const int64_t *slot_mapping, int32_t num_tokens, void *cache,
                                     const pa_latent_desc *desc, int *device_error, pa_stream_t stream) {
  if (!valid_latent_desc(desc) || num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!latent || !rope || !slot_mapping || !cache) return PA_ERR_INVALID;
  if (!aligned16(latent) || !aligned16(rope) || !aligned16(cache) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PA_ERR_INVALID;
  if (latent_stride < desc->latent_dim || rope_stride < desc->rope_dim || latent_stride % 8 || rope_stride % 8)
    return PA_ERR_INVALID;
  if (!supported_latent_desc(desc) || src_dtype != desc->dtype) return PA_ERR_UNSUPPORTED;
  const long long pieces = static_cast<long long>(num_tokens) * kPieces;
  const long long slots = static_cast<long long>(desc->num_blocks) * desc->block_size;
  const int blocks = grid_for((pieces + kUnroll - 1) / kUnroll, kWriteThreads);
  auto go = [&](auto kern, auto ls, auto rs, auto n) {
    kern<<<blocks, kWriteThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint16_t *>(latent), static_cast<const uint16_t *>(rope), ls, rs, slot_mapping, n, slots,
        static_cast<uint16_t *>(cache), device_error);
  };
  // 32-bit indexes where no product of them can pass 2^32 (the step past the end must not wrap either)
  const long long widest = latent_stride > rope_stride ? latent_stride : rope_stride;
  if (widest < 0x70000000ll / num_tokens && pieces < 0x70000000ll)
    go(latent_write_kernel<uint32_t>, static_cast<uint32_t>(latent_stride), static_cast<uint32_t>(rope_stride),
       static_cast<uint32_t>(pieces));
  else
    go(latent_write_kernel<uint64_t>, static_cast<uint64_t>(latent_stride), static_cast<uint64_t>(rope_stride),
       static_cast<uint64_t>(pieces));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}
