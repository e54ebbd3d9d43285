// Four-bit decode instantiations for blocks of 8 tokens.
#include "pa_decode_fp4.cuh"

namespace pa {

pa_status dispatch_decode_fp4_b8(int q_dtype, int head_dim, int group, const DecodeParams &p, const DeviceInfo &dev,
                                cudaStream_t stream) {
  return dispatch<8>(q_dtype, head_dim, group, p, dev, stream);
}

}  // namespace pa
