// Four-bit decode instantiations for blocks of 32 tokens.
#include "pa_decode_fp4.cuh"

namespace pa {

pa_status dispatch_decode_fp4_b32(int q_dtype, int head_dim, int group, const DecodeParams &p, const DeviceInfo &dev,
                                 cudaStream_t stream) {
  return dispatch<32>(q_dtype, head_dim, group, p, dev, stream);
}

}  // namespace pa
