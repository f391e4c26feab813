// layer.h -- host-side interface of the operators around the indexer (rotary positions, the
// writers of the two 8-bit pools, attention over the K/V pool) to the C ABI layer.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

// How a row's head is rotated: pairs of elements [offset, offset + rot) turned by the angle whose
// (cos, sin) stand in table[position].  table == nullptr: no rotation.
struct Rotation {
  const float2 *table;  // [max_positions][rot / 2]
  int32_t max_positions;
  int32_t rot;          // even
  int32_t offset;
  int32_t interleaved;  // pairs (2i, 2i + 1) rather than (i, i + rot / 2)
};

// Which request a new token belongs to and where it stands in it.  starts == nullptr: every
// request has next_n tokens; otherwise request b's are tokens [starts[b], starts[b + 1]).  The
// last of them stands at seq_lens[b] - 1.
struct TokenMap {
  const int32_t *starts;
  const int32_t *seq_lens;
  int64_t sl_stride;
  const int32_t *block_tables;
  int64_t bt_stride;
  int32_t bt_width;
  int32_t batch;
  int32_t next_n;
  int32_t tokens;
};

struct RotaryArgs {
  const void *x;
  void *out;
  int64_t x_token, x_head, out_token, out_head;  // strides in elements
  const int32_t *positions;
  int64_t tokens;
  int32_t heads;
  int32_t dim;
  Rotation r;
  float sin_sign;  // -1: the inverse rotation
  int32_t copy;    // the elements outside the rotated part are copied too (out is not x)
};
cudaError_t launch_rotary(const RotaryArgs &a, int dtype, bool vectors, cudaStream_t stream);
cudaError_t launch_rotary_table(const double *inv_freq, double magnitude, int32_t positions,
                                int32_t half, float2 *table, cudaStream_t stream);

struct IndexArgs {
  const void *k;  // [tokens, dim]
  int64_t k_token;
  const void *q;  // nullable: [tokens, heads, dim]
  int64_t q_token, q_head;
  const float *weights;  // [tokens, heads]
  int64_t w_token;
  uint8_t *q_out;      // [tokens, heads, dim]
  float *weights_out;  // [tokens, heads]
  uint8_t *pool;
  int64_t num_blocks;
  int32_t block_size;
  int32_t heads;  // 0 without q
  int32_t dim;
  Rotation r;
  TokenMap m;
};
// pairs: rows and angles may be read two elements at a time.
cudaError_t launch_index_prepare(const IndexArgs &a, int dtype, bool pairs, cudaStream_t stream);

struct AppendArgs {
  const void *k, *v;  // [tokens, heads, dim]
  int64_t k_token, k_head, v_token, v_head;
  uint8_t *k_pool, *v_pool;    // [num_blocks, heads, block_size, dim]
  float *k_scales, *v_scales;  // [num_blocks, heads]
  int64_t num_blocks;
  int32_t block_size;
  int32_t heads;
  int32_t dim;
  Rotation r;
  TokenMap m;
};
cudaError_t launch_kv_append(const AppendArgs &a, int dtype, bool pairs, cudaStream_t stream);

struct AttentionArgs {
  const void *q;  // [batch, next_n, heads, dim]
  int64_t q_batch, q_token, q_head;
  const uint8_t *k_pool, *v_pool;
  const float *k_scales, *v_scales;
  int64_t num_blocks;
  const int32_t *block_tables;
  int64_t bt_stride;
  int32_t bt_width;
  const int32_t *seq_lens;
  int64_t sl_stride;
  const int2 *candidates;  // nullable: [batch * next_n][slots]
  int64_t cand_stride;     // pairs
  const int32_t *ranges;   // [2][batch * next_n]
  int32_t slots;
  int32_t batch, next_n, heads, kv_heads, dim, block_size;
  float scale;  // softmax scale
  void *out;    // [batch, next_n, heads, dim], contiguous
  float *lse;   // nullable: [batch, next_n, heads]
  float *workspace;
};
// sms * (CTAs on an SM) runs; the workspace is attention_workspace(...) bytes.  k_map, v_map: the
// pools as rows of dim bytes, in boxes of block_size rows (not read with candidates).
cudaError_t launch_attention_d64(const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 const AttentionArgs &a, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_attention_d128(const CUtensorMap &k_map, const CUtensorMap &v_map,
                                  const AttentionArgs &a, int dtype, int sms, cudaStream_t stream);
// The most that any call of these sizes needs (either dtype, with candidates or without).
int64_t attention_workspace(int batch, int next_n, int heads, int kv_heads, int dim, int sms);

// Device-side status words (IDX_DEV_* bits) of the translation units above.
cudaError_t rotary_status(int32_t *value, bool clear);
cudaError_t index_status(int32_t *value, bool clear);
cudaError_t append_status(int32_t *value, bool clear);
cudaError_t attention_d64_status(int32_t *value, bool clear);
cudaError_t attention_d128_status(int32_t *value, bool clear);

}  // namespace idx
