// attention_d128.cu -- attention over the 8-bit K/V cache, head_dim 128 (see attention_kernel.cuh).

#include "attention_kernel.cuh"

namespace idx {

cudaError_t launch_attention_d128(const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 const AttentionArgs &a, int dtype, int sms, cudaStream_t stream) {
  return a.candidates != nullptr ? launch_rows<128, true, false>(k_map, v_map, a, dtype, sms, stream)
                                 : launch_rows<128, false, false>(k_map, v_map, a, dtype, sms, stream);
}

cudaError_t attention_d128_status(int32_t *value, bool clear) {
  return read_attention_status(value, clear);
}

int64_t attention_workspace(int batch, int next_n, int heads, int kv_heads, int dim, int sms) {
  int64_t most = 0;
  for (const bool four : {false, true})
    for (const bool f16 : {false, true})
      for (const bool select : {false, true}) {
        const AttnShape s = attn_shape(heads / kv_heads * (select ? 1 : next_n), f16,
                                       most_rows(dim, select, four));
        const int64_t groups =
            static_cast<int64_t>(select ? batch * next_n : batch) * kv_heads * s.chunks;
        const int64_t bytes = attn_slots_bytes(static_cast<int64_t>(sms) * ctas_for(s.r), s.r, dim) +
                              groups * static_cast<int64_t>(sizeof(GroupParts));
        if (bytes > most) most = bytes;
      }
  return most;
}

}  // namespace idx
