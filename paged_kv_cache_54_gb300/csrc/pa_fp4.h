// Entry points of the four-bit cache's kernels, called by the C entry points
// that serve every cache type.  The caller has checked the arguments.
#pragma once

#include "pa_decode_params.h"

namespace pa {

// pa_reshape_and_cache and pa_gather_cache over a PA_FP4 cache (pa_fp4_cache.cu)
pa_status write_fp4(const void *key, const void *value, int src_dtype, const int64_t *slots, int num_tokens,
                    void *k_cache, void *v_cache, const pa_cache_desc *cache, int *err, cudaStream_t stream);

// pa_decode over a PA_FP4 cache (pa_decode_fp4.cuh), a translation unit for
// each block size
pa_status dispatch_decode_fp4_b8(int q_dtype, int head_dim, int group, const DecodeParams &p, const DeviceInfo &dev,
                                 cudaStream_t stream);
pa_status dispatch_decode_fp4_b16(int q_dtype, int head_dim, int group, const DecodeParams &p, const DeviceInfo &dev,
                                  cudaStream_t stream);
pa_status dispatch_decode_fp4_b32(int q_dtype, int head_dim, int group, const DecodeParams &p, const DeviceInfo &dev,
                                  cudaStream_t stream);

}  // namespace pa
