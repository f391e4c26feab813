// attention_d64.cu -- attention over the 8-bit K/V cache, head_dim 64 (see attention_kernel.cuh).

#include "attention_kernel.cuh"

namespace idx {

cudaError_t launch_attention_d64(const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 const AttentionArgs &a, int dtype, int sms, cudaStream_t stream) {
  return a.candidates != nullptr ? launch_rows<64, true, false>(k_map, v_map, a, dtype, sms, stream)
                                 : launch_rows<64, false, false>(k_map, v_map, a, dtype, sms, stream);
}

cudaError_t attention_d64_status(int32_t *value, bool clear) {
  return read_attention_status(value, clear);
}

}  // namespace idx
