// attention4_d128.cu -- attention over the 4-bit K/V cache, head_dim 128 (see attention_kernel.cuh).

#include "attention_kernel.cuh"

namespace idx {

cudaError_t launch_attention4_d128(const CUtensorMap &k_map, const CUtensorMap &v_map,
                                  const AttentionArgs &a, int dtype, int sms, cudaStream_t stream) {
  return a.candidates != nullptr ? launch_rows<128, true, true>(k_map, v_map, a, dtype, sms, stream)
                                 : launch_rows<128, false, true>(k_map, v_map, a, dtype, sms, stream);
}

cudaError_t attention4_d128_status(int32_t *value, bool clear) {
  return read_attention_status(value, clear);
}

}  // namespace idx
