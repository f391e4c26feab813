// abi_layer.cu -- the extern "C" entry points of the operators around the indexer (the last part
// of include/idx.h): argument checks, status codes and launches.  No allocation, no
// synchronisation.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <utility>

#include "../../include/idx.h"
#include "internal.h"
#include "layer.h"

#define IDX_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

using idx::cuda_fail;
using idx::fail;

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int element_bytes(int32_t dtype) {
  return dtype == IDX_DTYPE_F32 ? 4 : dtype == IDX_DTYPE_F16 || dtype == IDX_DTYPE_BF16 ? 2 : 0;
}

// The rotation's arguments (table == NULL: none).
int check_rotation(const float *table, int32_t max_positions, int32_t rot_dim, int32_t rot_offset,
                   int32_t head_dim, idx::Rotation *r, int32_t interleaved) {
  *r = idx::Rotation{};
  if (table == nullptr) return IDX_OK;
  if (max_positions < 1 || rot_dim < 2 || rot_dim % 2 != 0 || rot_offset < 0 ||
      rot_offset > head_dim - rot_dim)
    return fail(IDX_INVALID_ARG,
                "max_positions >= 1, an even rot_dim >= 2 and rot_offset + rot_dim <= head_dim "
                "required");
  if (!aligned(table, 8)) return fail(IDX_INVALID_ARG, "table must be 8-byte aligned");
  r->table = reinterpret_cast<const float2 *>(table);
  r->max_positions = max_positions;
  r->rot = rot_dim;
  r->offset = rot_offset;
  r->interleaved = interleaved != 0;
  return IDX_OK;
}

// Whether the rotated part can be read in pieces of v elements (and its angles two at a time).
bool rotation_in_pieces(const idx::Rotation &r, int v) {
  return r.table == nullptr ||
         (r.offset % v == 0 && (r.rot / 2) % v == 0 && aligned(r.table, 16));
}

// The new tokens' map to requests, positions and pages.
int check_tokens(const int32_t *token_starts, int64_t tokens, const int32_t *seq_lens,
                 int64_t seq_lens_stride, int32_t batch, int32_t next_n,
                 const int32_t *block_tables, int64_t bt_row_stride, int32_t bt_width,
                 int32_t block_size, int64_t num_blocks, idx::TokenMap *m) {
  if (seq_lens == nullptr || block_tables == nullptr)
    return fail(IDX_INVALID_ARG, "seq_lens, block_tables: NULL");
  if (batch < 0 || tokens < 0 || tokens > INT32_MAX / 2 || seq_lens_stride < 1 || bt_width < 0 ||
      bt_row_stride < bt_width || num_blocks < 1)
    return fail(IDX_INVALID_ARG, "negative or inconsistent size or stride");
  if (token_starts == nullptr && (next_n < 1 || static_cast<int64_t>(batch) * next_n != tokens))
    return fail(IDX_INVALID_ARG, "without token_starts, tokens must be batch * next_n");
  if (block_size != 32 && block_size != 64 && block_size != 128)
    return fail(IDX_UNSUPPORTED, "this build supports block_size 32, 64 or 128");
  if (batch > idx::kMaxBatch) return fail(IDX_UNSUPPORTED, "batch above 4096");
  if (!aligned(seq_lens, 4) || !aligned(block_tables, 4) || !aligned(token_starts, 4))
    return fail(IDX_INVALID_ARG, "int32 arguments must be 4-byte aligned");
  m->starts = token_starts;
  m->seq_lens = seq_lens;
  m->sl_stride = seq_lens_stride;
  m->block_tables = block_tables;
  m->bt_stride = bt_row_stride;
  m->bt_width = bt_width;
  m->batch = batch;
  m->next_n = next_n;
  m->tokens = static_cast<int32_t>(tokens);
  return IDX_OK;
}

// Whether rows can be read in pieces of v elements of `size` bytes.
bool pieces(const void *p, int64_t s0, int64_t s1, int v, int size) {
  return aligned(p, v * size) && s0 % v == 0 && s1 % v == 0;
}

// Whether every pair lies in whole pieces of eight elements (and its angles can be read two at a time).
bool heads_in_pieces(const idx::Rotation &r) {
  return r.table == nullptr || (r.offset % 8 == 0 && r.rot % (r.interleaved ? 8 : 16) == 0 &&
                                aligned(r.table, 16));
}
bool dim_in_pieces(const idx::HeadsArgs &a) {
  return a.dim % 16 == 0 && a.dim <= 256 && heads_in_pieces(a.r);
}

// The 4-bit cache's pools.
int check_kv4(uint8_t *k_pool, uint8_t *v_pool, uint8_t *k_scales, float *v_scales, int32_t dtype,
              int32_t kv_heads, int32_t head_dim, idx::Kv4Args *a) {
  if (k_pool == nullptr || v_pool == nullptr || k_scales == nullptr || v_scales == nullptr)
    return fail(IDX_INVALID_ARG, "k_pool, v_pool, k_scales, v_scales: NULL");
  if (element_bytes(dtype) == 0)
    return fail(IDX_UNSUPPORTED, "dtype must be IDX_DTYPE_F32, _F16 or _BF16");
  if (head_dim != 64 && head_dim != 128)
    return fail(IDX_UNSUPPORTED, "this build supports head_dim 64 or 128");
  if (kv_heads < 1 || kv_heads > 4096) return fail(IDX_INVALID_ARG, "kv_heads must be 1 .. 4096");
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(v_scales, 4))
    return fail(IDX_INVALID_ARG, "k_pool and v_pool must be 16-byte aligned, v_scales 4-byte");
  a->k_pool = k_pool;
  a->v_pool = v_pool;
  a->k_scales = k_scales;
  a->v_scales = v_scales;
  a->heads = kv_heads;
  a->dim = head_dim;
  return IDX_OK;
}

// Heads to be rotated by one axis or several (pair_axis: host memory), or not (table == NULL).
int check_heads(int32_t dtype, int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
                const int32_t *positions, int64_t axis_stride, const uint8_t *pair_axis, int32_t axes,
                const float *table, int32_t max_positions, int32_t rot_dim, int32_t rot_offset,
                int32_t interleaved, idx::HeadsArgs *a) {
  if (element_bytes(dtype) == 0)
    return fail(IDX_UNSUPPORTED, "dtype must be IDX_DTYPE_F32, _F16 or _BF16");
  if (tokens < 0 || tokens > INT32_MAX || q_heads < 0 || k_heads < 0 || q_heads > 65536 ||
      k_heads > 65536 || head_dim < 1)
    return fail(IDX_INVALID_ARG, "negative or too large a size");
  if (head_dim > IDX_NORM_MAX_DIM)
    return fail(IDX_UNSUPPORTED, "head_dim above IDX_NORM_MAX_DIM");
  const int st = check_rotation(table, max_positions, rot_dim, rot_offset, head_dim, &a->r, interleaved);
  if (st != IDX_OK) return st;
  a->axes.count = 1;
  if (table != nullptr) {
    if (positions == nullptr || !aligned(positions, 4))
      return fail(IDX_INVALID_ARG, "a table needs positions, 4-byte aligned");
    if (axes < 1 || axes > IDX_ROTARY_MAX_AXES)
      return fail(IDX_INVALID_ARG, "axes must be 1 .. IDX_ROTARY_MAX_AXES");
    if (axes > 1) {
      if (pair_axis == nullptr || axis_stride < 0)
        return fail(IDX_INVALID_ARG, "several axes need pair_axis and a stride of 0 or more");
      for (int i = 0; i < rot_dim / 2; ++i) {
        if (pair_axis[i] >= axes) return fail(IDX_INVALID_ARG, "pair_axis must be below axes");
        a->axes.axis[i / 16] |= static_cast<uint32_t>(pair_axis[i]) << (2 * (i % 16));
      }
      a->axes.count = axes;
      a->axes.stride = axis_stride;
    }
  }
  a->positions = positions;
  a->tokens = tokens;
  a->heads[0] = q_heads;
  a->heads[1] = k_heads;
  a->dim = head_dim;
  a->sin_sign = 1.0f;
  return IDX_OK;
}

int check_norm(int32_t dtype, float eps, const void *q_weight, const void *k_weight,
               int32_t weight_dtype, idx::HeadsArgs *a) {
  if (!(eps >= 0.0f) || std::isinf(eps))
    return fail(IDX_INVALID_ARG, "eps must be finite, 0 or more");
  if (q_weight != nullptr || k_weight != nullptr) {
    if (weight_dtype != dtype && weight_dtype != IDX_DTYPE_F32)
      return fail(IDX_UNSUPPORTED, "weights must have the dtype of q and k, or float32");
    const int size = element_bytes(weight_dtype);
    if (!aligned(q_weight, size) || !aligned(k_weight, size))
      return fail(IDX_INVALID_ARG, "weights must be aligned to their elements");
    // (Without weights weight_dtype says nothing: any value will do.)
    a->weight_f32 = weight_dtype == IDX_DTYPE_F32;
    a->weight_pieces = aligned(q_weight, 8 * size) && aligned(k_weight, 8 * size);
  }
  a->norm = 1;
  a->eps = eps;
  a->weight[0] = q_weight;
  a->weight[1] = k_weight;
  return IDX_OK;
}

// Rows [tokens][heads][dim] of one operand; whole: still all of them in pieces of eight elements.
int set_rows(const void *p, int64_t token, int64_t head, int size, const void **to, int64_t *token_to,
             int64_t *head_to, bool *whole) {
  if (!aligned(p, size))
    return fail(IDX_INVALID_ARG, "rows must be aligned to their elements");
  *to = p;
  *token_to = token;
  *head_to = head;
  *whole = *whole && pieces(p, token, head, 8, size);
  return IDX_OK;
}

}  // namespace

IDX_EXPORT int idx_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                                      double original_positions, double beta_fast,
                                      double beta_slow, double *inv_freq, double *magnitude) {
  idx::clear_error();
  if (inv_freq == nullptr || magnitude == nullptr)
    return fail(IDX_INVALID_ARG, "inv_freq, magnitude: NULL");
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > IDX_ROTARY_MAX_DIM)
    return fail(IDX_INVALID_ARG, "rot_dim must be even, 2 .. IDX_ROTARY_MAX_DIM");
  if (!(base > 1.0) || std::isinf(base)) return fail(IDX_INVALID_ARG, "base must be above 1");
  if (scaling < IDX_ROTARY_NONE || scaling > IDX_ROTARY_YARN)
    return fail(IDX_INVALID_ARG, "unknown scaling");
  if (scaling != IDX_ROTARY_NONE && (!(factor >= 1.0) || std::isinf(factor)))
    return fail(IDX_INVALID_ARG, "factor must be at least 1");
  if (scaling == IDX_ROTARY_NTK && rot_dim < 4)
    return fail(IDX_INVALID_ARG, "the base is scaled by factor^(rot_dim / (rot_dim - 2)): rot_dim "
                                 "must be at least 4");
  if (scaling == IDX_ROTARY_YARN &&
      (!(original_positions > 0.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow)))
    return fail(IDX_INVALID_ARG, "original_positions > 0 and beta_fast >= beta_slow > 0 required");
  const int half = rot_dim / 2;
  *magnitude = 1.0;
  double b = base;
  if (scaling == IDX_ROTARY_NTK)
    b = base * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  double low = 0.0, high = 0.0;
  if (scaling == IDX_ROTARY_YARN) {
    // The pair that turns `beta` times over the original positions.
    const double pi = 3.14159265358979323846;
    const auto pair = [&](double beta) {
      return rot_dim * std::log(original_positions / (beta * 2.0 * pi)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair(beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair(beta_slow)), rot_dim - 1.0);
    if (!(high > low)) high = low + 0.001;
    *magnitude = 0.1 * std::log(factor) + 1.0;
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == IDX_ROTARY_LINEAR) {
      inv_freq[i] = f / factor;
    } else if (scaling == IDX_ROTARY_YARN) {
      const double ramp = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
      inv_freq[i] = f * (1.0 - ramp) + f / factor * ramp;
    } else {
      inv_freq[i] = f;
    }
  }
  return IDX_OK;
}

IDX_EXPORT int idx_rotary_table(const double *inv_freq, double magnitude, int32_t max_positions,
                                int32_t rot_dim, float *table, void *stream) {
  idx::clear_error();
  if (inv_freq == nullptr || table == nullptr)
    return fail(IDX_INVALID_ARG, "inv_freq, table: NULL");
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > IDX_ROTARY_MAX_DIM)
    return fail(IDX_INVALID_ARG, "rot_dim must be even, 2 .. IDX_ROTARY_MAX_DIM");
  if (max_positions < 0) return fail(IDX_INVALID_ARG, "max_positions must be >= 0");
  if (!aligned(table, 8)) return fail(IDX_INVALID_ARG, "table must be 8-byte aligned");
  if (max_positions == 0) return IDX_OK;
  const cudaError_t e =
      idx::launch_rotary_table(inv_freq, magnitude, max_positions, rot_dim / 2,
                               reinterpret_cast<float2 *>(table), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "rotary table launch");
}

IDX_EXPORT int idx_rotary(const void *x, int64_t x_token_stride, int64_t x_head_stride,
                          const int32_t *positions, int64_t tokens, int32_t num_heads,
                          int32_t head_dim, int32_t dtype, const float *table,
                          int32_t max_positions, int32_t rot_dim, int32_t rot_offset,
                          int32_t interleaved, int32_t inverse, void *out,
                          int64_t out_token_stride, int64_t out_head_stride, void *stream) {
  idx::clear_error();
  if (x == nullptr || positions == nullptr || table == nullptr || out == nullptr)
    return fail(IDX_INVALID_ARG, "x, positions, table, out: NULL");
  const int size = element_bytes(dtype);
  if (size == 0) return fail(IDX_UNSUPPORTED, "dtype must be IDX_DTYPE_F32, _F16 or _BF16");
  if (tokens < 0 || tokens > INT32_MAX || num_heads < 0 || head_dim < 1 || head_dim > (1 << 20) ||
      num_heads > (1 << 20))
    return fail(IDX_INVALID_ARG, "negative or too large a size");
  idx::RotaryArgs a{};
  const int st = check_rotation(table, max_positions, rot_dim, rot_offset, head_dim, &a.r,
                                interleaved);
  if (st != IDX_OK) return st;
  if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 4))
    return fail(IDX_INVALID_ARG, "x, out and positions must be aligned to their elements");
  if (tokens == 0 || num_heads == 0) return IDX_OK;
  a.x = x;
  a.out = out;
  a.x_token = x_token_stride;
  a.x_head = x_head_stride;
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.positions = positions;
  a.tokens = tokens;
  a.heads = num_heads;
  a.dim = head_dim;
  a.sin_sign = inverse ? -1.0f : 1.0f;
  a.copy = !(x == out && x_token_stride == out_token_stride && x_head_stride == out_head_stride);
  const int v = 16 / size;
  const bool vectors = pieces(x, x_token_stride, x_head_stride, v, size) &&
                       pieces(out, out_token_stride, out_head_stride, v, size) && head_dim % v == 0 &&
                       rotation_in_pieces(a.r, v);
  const cudaError_t e = idx::launch_rotary(a, dtype, vectors, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "rotary launch");
}

IDX_EXPORT int idx_index_prepare(
    const void *k, int64_t k_token_stride, const void *q, int64_t q_token_stride,
    int64_t q_head_stride, const float *weights, int64_t weights_token_stride, int32_t dtype,
    int64_t tokens, int32_t num_heads, int32_t head_dim, const float *table, int32_t max_positions,
    int32_t rot_dim, int32_t rot_offset, int32_t interleaved, const int32_t *token_starts,
    const int32_t *seq_lens, int64_t seq_lens_stride, int32_t batch, int32_t next_n,
    const int32_t *block_tables, int64_t bt_row_stride, int32_t bt_width, int32_t block_size,
    int64_t num_blocks, uint8_t *kv_fused, uint8_t *q_out, float *weights_out, void *stream) {
  idx::clear_error();
  if (k == nullptr || kv_fused == nullptr) return fail(IDX_INVALID_ARG, "k, kv_fused: NULL");
  if (q != nullptr && (weights == nullptr || q_out == nullptr || weights_out == nullptr))
    return fail(IDX_INVALID_ARG, "q needs weights, q_out and weights_out");
  const int size = element_bytes(dtype);
  if (size == 0) return fail(IDX_UNSUPPORTED, "dtype must be IDX_DTYPE_F32, _F16 or _BF16");
  idx::IndexArgs a{};
  int st = check_tokens(token_starts, tokens, seq_lens, seq_lens_stride, batch, next_n,
                        block_tables, bt_row_stride, bt_width, block_size, num_blocks, &a.m);
  if (st != IDX_OK) return st;
  if (head_dim != 64 && head_dim != 128 && head_dim != 192)
    return fail(IDX_UNSUPPORTED, "this build supports head_dim 64, 128 or 192");
  if (q != nullptr && (num_heads < 1 || num_heads > 4096))
    return fail(IDX_INVALID_ARG, "num_heads must be 1 .. 4096");
  st = check_rotation(table, max_positions, rot_dim, rot_offset, head_dim, &a.r, interleaved);
  if (st != IDX_OK) return st;
  if (!aligned(k, size) || !aligned(q, size) || !aligned(kv_fused, 16) || !aligned(q_out, 16) ||
      !aligned(weights, 4) || !aligned(weights_out, 4))
    return fail(IDX_INVALID_ARG,
                "kv_fused and q_out must be 16-byte aligned, the rest aligned to its elements");
  if (tokens == 0 || batch == 0) return IDX_OK;
  a.k = k;
  a.k_token = k_token_stride;
  a.q = q;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.weights = weights;
  a.w_token = weights_token_stride;
  a.q_out = q_out;
  a.weights_out = weights_out;
  a.pool = kv_fused;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.heads = q != nullptr ? num_heads : 0;
  a.dim = head_dim;
  const bool pairs = pieces(k, k_token_stride, 0, 2, size) &&
                     (q == nullptr || pieces(q, q_token_stride, q_head_stride, 2, size)) &&
                     rotation_in_pieces(a.r, 2);
  const cudaError_t e =
      idx::launch_index_prepare(a, dtype, pairs, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "index_prepare launch");
}

IDX_EXPORT int idx_kv_append(const void *k, int64_t k_token_stride, int64_t k_head_stride,
                             const void *v, int64_t v_token_stride, int64_t v_head_stride,
                             int32_t dtype, int64_t tokens, int32_t kv_heads, int32_t head_dim,
                             const float *table, int32_t max_positions, int32_t rot_dim,
                             int32_t rot_offset, int32_t interleaved, const int32_t *token_starts,
                             const int32_t *seq_lens, int64_t seq_lens_stride, int32_t batch,
                             int32_t next_n, const int32_t *block_tables, int64_t bt_row_stride,
                             int32_t bt_width, int32_t block_size, int64_t num_blocks,
                             uint8_t *k_pool, uint8_t *v_pool, float *k_scales, float *v_scales,
                             void *stream) {
  idx::clear_error();
  if (k == nullptr || v == nullptr || k_pool == nullptr || v_pool == nullptr ||
      k_scales == nullptr || v_scales == nullptr)
    return fail(IDX_INVALID_ARG, "k, v, k_pool, v_pool, k_scales, v_scales: NULL");
  const int size = element_bytes(dtype);
  if (size == 0) return fail(IDX_UNSUPPORTED, "dtype must be IDX_DTYPE_F32, _F16 or _BF16");
  idx::AppendArgs a{};
  int st = check_tokens(token_starts, tokens, seq_lens, seq_lens_stride, batch, next_n,
                        block_tables, bt_row_stride, bt_width, block_size, num_blocks, &a.m);
  if (st != IDX_OK) return st;
  if (head_dim != 64 && head_dim != 128)
    return fail(IDX_UNSUPPORTED, "this build supports head_dim 64 or 128");
  if (kv_heads < 1 || kv_heads > 4096)
    return fail(IDX_INVALID_ARG, "kv_heads must be 1 .. 4096");
  st = check_rotation(table, max_positions, rot_dim, rot_offset, head_dim, &a.r, interleaved);
  if (st != IDX_OK) return st;
  if (!aligned(k, size) || !aligned(v, size) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
      !aligned(k_scales, 4) || !aligned(v_scales, 4))
    return fail(IDX_INVALID_ARG,
                "k_pool and v_pool must be 16-byte aligned, the rest aligned to its elements");
  if (tokens == 0 || batch == 0) return IDX_OK;
  a.k = k;
  a.v = v;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.heads = kv_heads;
  a.dim = head_dim;
  const bool pairs = pieces(k, k_token_stride, k_head_stride, 2, size) &&
                     pieces(v, v_token_stride, v_head_stride, 2, size) && rotation_in_pieces(a.r, 2);
  const cudaError_t e = idx::launch_kv_append(a, dtype, pairs, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "kv_append launch");
}

IDX_EXPORT int64_t idx_attention_workspace_bytes(int32_t batch, int32_t next_n, int32_t num_heads,
                                                 int32_t kv_heads, int32_t head_dim,
                                                 int32_t num_sms) {
  // (What idx_attention_fp8 refuses has no size; a K/V head without query heads would divide by 0.)
  if (batch < 0 || batch > idx::kMaxBatch || next_n < 1 || next_n > 4 || kv_heads < 1 ||
      num_heads < 1 || num_heads > 4096 || num_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128) || num_sms < 0)
    return -1;
  int32_t sms = 0;
  if (idx::resolve_sms(num_sms, &sms) != IDX_OK) return -1;
  return idx::attention_workspace(batch, next_n, num_heads, kv_heads, head_dim, sms);
}

namespace {

// idx_attention_fp8 and (four) idx_attention_fp4.
int attention(
    bool four,
    const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
    int32_t dtype, const uint8_t *k_pool, const uint8_t *v_pool, const void *k_scales,
    const float *v_scales, int64_t num_blocks, int32_t block_size, const int32_t *block_tables,
    int64_t bt_row_stride, int32_t bt_width, const int32_t *seq_lens, int64_t seq_lens_stride,
    int32_t batch, int32_t next_n, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
    float softmax_scale, const int32_t *candidates, int32_t slots, const int32_t *ranges,
    int32_t num_sms, void *out, float *lse, void *workspace, int64_t workspace_bytes,
    void *stream) {
  if (q == nullptr || k_pool == nullptr || v_pool == nullptr || k_scales == nullptr ||
      v_scales == nullptr || block_tables == nullptr || seq_lens == nullptr || out == nullptr)
    return fail(IDX_INVALID_ARG, "q, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, "
                                 "out: NULL");
  if (candidates != nullptr && (ranges == nullptr || slots < 1))
    return fail(IDX_INVALID_ARG, "candidates need ranges and slots >= 1");
  if (batch < 0 || num_blocks < 1 || bt_width < 0 || bt_row_stride < bt_width ||
      seq_lens_stride < 1 || num_heads < 1 || kv_heads < 1 || next_n < 1)
    return fail(IDX_INVALID_ARG, "negative or inconsistent size or stride");
  if (num_heads % kv_heads != 0)
    return fail(IDX_INVALID_ARG, "num_heads must be a multiple of kv_heads");
  if (!std::isfinite(softmax_scale)) return fail(IDX_INVALID_ARG, "softmax_scale must be finite");
  if (dtype != IDX_DTYPE_F16 && dtype != IDX_DTYPE_BF16)
    return fail(IDX_UNSUPPORTED, "dtype must be IDX_DTYPE_F16 or IDX_DTYPE_BF16");
  if (next_n > 4) return fail(IDX_UNSUPPORTED, "next_n must be 1..4");
  if (batch > idx::kMaxBatch) return fail(IDX_UNSUPPORTED, "batch above 4096");
  if ((head_dim != 64 && head_dim != 128) ||
      (block_size != 32 && block_size != 64 && block_size != 128))
    return fail(IDX_UNSUPPORTED,
                "this build supports head_dim 64 or 128 and block_size 32, 64 or 128");
  if (num_heads > 4096) return fail(IDX_UNSUPPORTED, "num_heads above 4096");
  if (num_blocks > INT32_MAX / (static_cast<int64_t>(kv_heads) * block_size) - 1)
    return fail(IDX_INVALID_ARG, "num_blocks too large for 32-bit TMA row coordinates");
  if (!aligned(q, 16) || q_batch_stride % 8 != 0 || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0)
    return fail(IDX_INVALID_ARG, "q must be 16-byte aligned with strides that are multiples of 8");
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_tables, 4) ||
      !aligned(seq_lens, 4) || !aligned(candidates, 8) || !aligned(ranges, 4) ||
      !aligned(workspace, 256))
    return fail(IDX_INVALID_ARG, "pools and out must be 16-byte aligned, candidates 8-byte, "
                                 "workspace 256-byte, the rest 4-byte");
  if (four && (!aligned(k_pool, 32) || !aligned(v_pool, 32) || !aligned(k_scales, 16) ||
               !aligned(v_scales, 16)))
    return fail(IDX_INVALID_ARG, "4-bit pools must be 32-byte aligned, their scales 16-byte");
  int32_t ctas = 0;
  int st = idx::resolve_sms(num_sms, &ctas);
  if (st != IDX_OK) return st;
  const int64_t need =
      idx_attention_workspace_bytes(batch, next_n, num_heads, kv_heads, head_dim, ctas);
  if (workspace_bytes < need || (need > 0 && workspace == nullptr))
    return fail(IDX_INVALID_ARG, "workspace_bytes < idx_attention_workspace_bytes(...)");
  if (batch == 0) return IDX_OK;
  idx::AttentionArgs a{};
  a.q = q;
  a.q_batch = q_batch_stride;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.num_blocks = num_blocks;
  a.block_tables = block_tables;
  a.bt_stride = bt_row_stride;
  a.bt_width = bt_width;
  a.seq_lens = seq_lens;
  a.sl_stride = seq_lens_stride;
  a.candidates = reinterpret_cast<const int2 *>(candidates);
  a.cand_stride = slots;
  a.ranges = ranges;
  a.slots = slots;
  a.batch = batch;
  a.next_n = next_n;
  a.heads = num_heads;
  a.kv_heads = kv_heads;
  a.dim = head_dim;
  a.block_size = block_size;
  a.scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  a.workspace = static_cast<float *>(workspace);
  CUtensorMap k_map{}, v_map{};  // (with candidates the rows are gathered without them)
  if (candidates == nullptr) {
    // (Rows of 128 elements in four bits: two tokens' of 64.)
    const int tokens = four ? 128 / head_dim : 1;
    const uint64_t rows = static_cast<uint64_t>(num_blocks) * kv_heads * (block_size / tokens);
    const uint32_t box = static_cast<uint32_t>(block_size / tokens);
    for (const auto &m : {std::pair<CUtensorMap *, const uint8_t *>{&k_map, k_pool}, {&v_map, v_pool}}) {
      st = four ? idx::encode_rows4(m.first, m.second, rows, box)
                : idx::encode_rows(m.first, m.second, rows, static_cast<uint32_t>(head_dim), box);
      if (st != IDX_OK) return st;
    }
  }
  const auto launch = four ? (head_dim == 64 ? idx::launch_attention4_d64 : idx::launch_attention4_d128)
                           : (head_dim == 64 ? idx::launch_attention_d64 : idx::launch_attention_d128);
  const cudaError_t e = launch(k_map, v_map, a, dtype, ctas, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "attention launch");
}

}  // namespace

IDX_EXPORT int idx_attention_fp8(
    const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
    int32_t dtype, const uint8_t *k_pool, const uint8_t *v_pool, const float *k_scales,
    const float *v_scales, int64_t num_blocks, int32_t block_size, const int32_t *block_tables,
    int64_t bt_row_stride, int32_t bt_width, const int32_t *seq_lens, int64_t seq_lens_stride,
    int32_t batch, int32_t next_n, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
    float softmax_scale, const int32_t *candidates, int32_t slots, const int32_t *ranges,
    int32_t num_sms, void *out, float *lse, void *workspace, int64_t workspace_bytes,
    void *stream) {
  idx::clear_error();
  return attention(false, q, q_batch_stride, q_token_stride, q_head_stride, dtype, k_pool, v_pool, k_scales,
                   v_scales, num_blocks, block_size, block_tables, bt_row_stride, bt_width, seq_lens,
                   seq_lens_stride, batch, next_n, num_heads, kv_heads, head_dim, softmax_scale,
                   candidates, slots, ranges, num_sms, out, lse, workspace, workspace_bytes, stream);
}

IDX_EXPORT int idx_attention_fp4(
    const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
    int32_t dtype, const uint8_t *k_pool, const uint8_t *v_pool, const uint8_t *k_scales,
    const float *v_scales, int64_t num_blocks, int32_t block_size, const int32_t *block_tables,
    int64_t bt_row_stride, int32_t bt_width, const int32_t *seq_lens, int64_t seq_lens_stride,
    int32_t batch, int32_t next_n, int32_t num_heads, int32_t kv_heads, int32_t head_dim,
    float softmax_scale, const int32_t *candidates, int32_t slots, const int32_t *ranges,
    int32_t num_sms, void *out, float *lse, void *workspace, int64_t workspace_bytes,
    void *stream) {
  idx::clear_error();
  return attention(true, q, q_batch_stride, q_token_stride, q_head_stride, dtype, k_pool, v_pool, k_scales,
                   v_scales, num_blocks, block_size, block_tables, bt_row_stride, bt_width, seq_lens,
                   seq_lens_stride, batch, next_n, num_heads, kv_heads, head_dim, softmax_scale,
                   candidates, slots, ranges, num_sms, out, lse, workspace, workspace_bytes, stream);
}

IDX_EXPORT int idx_kv_append_fp4(const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                 const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                 int32_t dtype, int64_t tokens, int32_t kv_heads, int32_t head_dim,
                                 const float *table, int32_t max_positions, int32_t rot_dim,
                                 int32_t rot_offset, int32_t interleaved,
                                 const int32_t *token_starts, const int32_t *seq_lens,
                                 int64_t seq_lens_stride, int32_t batch, int32_t next_n,
                                 const int32_t *block_tables, int64_t bt_row_stride,
                                 int32_t bt_width, int32_t block_size, int64_t num_blocks,
                                 uint8_t *k_pool, uint8_t *v_pool, uint8_t *k_scales,
                                 float *v_scales, void *stream) {
  idx::clear_error();
  if (k == nullptr || v == nullptr) return fail(IDX_INVALID_ARG, "k, v: NULL");
  idx::Kv4Args a{};
  int st = check_kv4(k_pool, v_pool, k_scales, v_scales, dtype, kv_heads, head_dim, &a);
  if (st != IDX_OK) return st;
  st = check_tokens(token_starts, tokens, seq_lens, seq_lens_stride, batch, next_n, block_tables,
                    bt_row_stride, bt_width, block_size, num_blocks, &a.m);
  if (st != IDX_OK) return st;
  st = check_rotation(table, max_positions, rot_dim, rot_offset, head_dim, &a.r, interleaved);
  if (st != IDX_OK) return st;
  const int size = element_bytes(dtype);
  if (!aligned(k, size) || !aligned(v, size))
    return fail(IDX_INVALID_ARG, "k and v must be aligned to their elements");
  if (tokens == 0 || batch == 0) return IDX_OK;
  a.k = k;
  a.v = v;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  const bool k_pieces = pieces(k, k_token_stride, k_head_stride, 8, size);
  const bool all = k_pieces && pieces(v, v_token_stride, v_head_stride, 8, size);
  const cudaError_t e = idx::launch_kv4_append(a, dtype, all, k_pieces && heads_in_pieces(a.r),
                                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "kv_append_fp4 launch");
}

IDX_EXPORT int idx_kv_read_fp4(const uint8_t *k_pool, const uint8_t *v_pool, const uint8_t *k_scales,
                               const float *v_scales, int64_t num_blocks, int32_t block_size,
                               int32_t kv_heads, int32_t head_dim, const int32_t *token_starts,
                               int64_t tokens, const int32_t *seq_lens, int64_t seq_lens_stride,
                               int32_t batch, int32_t next_n, const int32_t *block_tables,
                               int64_t bt_row_stride, int32_t bt_width, int32_t clear, int32_t dtype,
                               void *k_out,
                               int64_t k_token_stride, int64_t k_head_stride, void *v_out,
                               int64_t v_token_stride, int64_t v_head_stride, void *stream) {
  idx::clear_error();
  if (k_out == nullptr || v_out == nullptr) return fail(IDX_INVALID_ARG, "k_out, v_out: NULL");
  idx::Kv4Args a{};
  int st = check_kv4(const_cast<uint8_t *>(k_pool), const_cast<uint8_t *>(v_pool),
                     const_cast<uint8_t *>(k_scales), const_cast<float *>(v_scales), dtype, kv_heads,
                     head_dim, &a);
  if (st != IDX_OK) return st;
  st = check_tokens(token_starts, tokens, seq_lens, seq_lens_stride, batch, next_n, block_tables,
                    bt_row_stride, bt_width, block_size, num_blocks, &a.m);
  if (st != IDX_OK) return st;
  const int size = element_bytes(dtype);
  if (!aligned(k_out, size) || !aligned(v_out, size))
    return fail(IDX_INVALID_ARG, "k_out and v_out must be aligned to their elements");
  if (tokens == 0) return IDX_OK;
  if (batch == 0) return fail(IDX_INVALID_ARG, "tokens of no request");
  a.k_out = k_out;
  a.v_out = v_out;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  const auto at_once = [&](int bytes) {
    return pieces(k_out, k_token_stride, k_head_stride, bytes / size, size) &&
           pieces(v_out, v_token_stride, v_head_stride, bytes / size, size);
  };
  const cudaError_t e = idx::launch_kv4_read(a, dtype, at_once(8 * size), at_once(32), clear != 0,
                                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "kv_read_fp4 launch");
}

IDX_EXPORT int idx_rotary_axes(const void *x, int64_t x_token_stride, int64_t x_head_stride,
                               const int32_t *positions, int64_t axis_stride,
                               const uint8_t *pair_axis, int32_t axes, int64_t tokens,
                               int32_t num_heads, int32_t head_dim, int32_t dtype,
                               const float *table, int32_t max_positions, int32_t rot_dim,
                               int32_t rot_offset, int32_t interleaved, int32_t inverse, void *out,
                               int64_t out_token_stride, int64_t out_head_stride, void *stream) {
  idx::clear_error();
  if (x == nullptr || table == nullptr || positions == nullptr || out == nullptr)
    return fail(IDX_INVALID_ARG, "x, positions, table, out: NULL");
  idx::HeadsArgs a{};
  int st = check_heads(dtype, tokens, num_heads, 0, head_dim, positions, axis_stride, pair_axis, axes,
                       table, max_positions, rot_dim, rot_offset, interleaved, &a);
  if (st != IDX_OK) return st;
  bool whole = true;
  st = set_rows(x, x_token_stride, x_head_stride, element_bytes(dtype), &a.x[0], &a.x_token[0],
                &a.x_head[0], &whole);
  if (st == IDX_OK)
    st = set_rows(out, out_token_stride, out_head_stride, element_bytes(dtype),
                  const_cast<const void **>(&a.out[0]), &a.out_token[0], &a.out_head[0], &whole);
  if (st != IDX_OK) return st;
  if (tokens == 0 || num_heads == 0) return IDX_OK;
  a.sin_sign = inverse ? -1.0f : 1.0f;
  const cudaError_t e = idx::launch_heads(a, dtype, whole && dim_in_pieces(a),
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "rotary launch");
}

IDX_EXPORT int idx_norm_rotary(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, int32_t k_heads, int32_t dtype, int64_t tokens,
    int32_t head_dim, const void *q_weight, const void *k_weight, int32_t weight_dtype, float eps,
    const int32_t *positions, int64_t axis_stride, const uint8_t *pair_axis, int32_t axes,
    const float *table, int32_t max_positions, int32_t rot_dim, int32_t rot_offset,
    int32_t interleaved, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
    void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride, void *stream) {
  idx::clear_error();
  if (q == nullptr || q_out == nullptr || (k_heads > 0 && (k == nullptr || k_out == nullptr)))
    return fail(IDX_INVALID_ARG, "q, q_out (with k_heads: k, k_out): NULL");
  idx::HeadsArgs a{};
  int st = check_heads(dtype, tokens, q_heads, k_heads, head_dim, positions, axis_stride, pair_axis,
                       axes, table, max_positions, rot_dim, rot_offset, interleaved, &a);
  if (st == IDX_OK) st = check_norm(dtype, eps, q_weight, k_weight, weight_dtype, &a);
  if (st != IDX_OK) return st;
  const int size = element_bytes(dtype);
  bool whole = true;
  st = set_rows(q, q_token_stride, q_head_stride, size, &a.x[0], &a.x_token[0], &a.x_head[0], &whole);
  if (st == IDX_OK)
    st = set_rows(q_out, q_out_token_stride, q_out_head_stride, size,
                  const_cast<const void **>(&a.out[0]), &a.out_token[0], &a.out_head[0], &whole);
  if (st == IDX_OK && k_heads > 0)
    st = set_rows(k, k_token_stride, k_head_stride, size, &a.x[1], &a.x_token[1], &a.x_head[1], &whole);
  if (st == IDX_OK && k_heads > 0)
    st = set_rows(k_out, k_out_token_stride, k_out_head_stride, size,
                  const_cast<const void **>(&a.out[1]), &a.out_token[1], &a.out_head[1], &whole);
  if (st != IDX_OK) return st;
  if (tokens == 0 || q_heads + k_heads == 0) return IDX_OK;
  const cudaError_t e = idx::launch_heads(a, dtype, whole && dim_in_pieces(a),
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "norm_rotary launch");
}

IDX_EXPORT int64_t idx_norm_rotary_workspace_bytes(int32_t head_dim) {
  idx::clear_error();
  if (head_dim < 1 || head_dim > IDX_NORM_MAX_DIM) return -1;
  int32_t sms = 0;
  if (idx::resolve_sms(0, &sms) != IDX_OK) return -1;
  return (idx::heads_blocks(sms) + 1ll) * head_dim * 4;
}

IDX_EXPORT int idx_norm_rotary_backward(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, int32_t k_heads, int32_t dtype, int64_t tokens,
    int32_t head_dim, const void *q_weight, const void *k_weight, int32_t weight_dtype, float eps,
    const int32_t *positions, int64_t axis_stride, const uint8_t *pair_axis, int32_t axes,
    const float *table, int32_t max_positions, int32_t rot_dim, int32_t rot_offset,
    int32_t interleaved, const void *q_out_grad, int64_t qg_token_stride, int64_t qg_head_stride,
    const void *k_out_grad, int64_t kg_token_stride, int64_t kg_head_stride, void *q_grad,
    void *k_grad, void *q_weight_grad, void *k_weight_grad, void *workspace,
    int64_t workspace_bytes, void *stream) {
  idx::clear_error();
  if (q == nullptr || q_out_grad == nullptr || q_grad == nullptr ||
      (k_heads > 0 && (k == nullptr || k_out_grad == nullptr || k_grad == nullptr)))
    return fail(IDX_INVALID_ARG, "q, q_out_grad, q_grad (with k_heads: k, k_out_grad, k_grad): NULL");
  idx::HeadsArgs a{};
  int st = check_heads(dtype, tokens, q_heads, k_heads, head_dim, positions, axis_stride, pair_axis,
                       axes, table, max_positions, rot_dim, rot_offset, interleaved, &a);
  if (st == IDX_OK) st = check_norm(dtype, eps, q_weight, k_weight, weight_dtype, &a);
  if (st != IDX_OK) return st;
  if ((q_weight_grad != nullptr && q_weight == nullptr) ||
      (k_weight_grad != nullptr && k_weight == nullptr))
    return fail(IDX_INVALID_ARG, "a weight's gradient without the weight");
  const int size = element_bytes(dtype), wsize = element_bytes(weight_dtype);
  if (!aligned(q_weight_grad, wsize ? wsize : 1) || !aligned(k_weight_grad, wsize ? wsize : 1))
    return fail(IDX_INVALID_ARG, "the weights' gradients must be aligned to their elements");
  bool whole = true;
  const int64_t qt = static_cast<int64_t>(q_heads) * head_dim, kt = static_cast<int64_t>(k_heads) * head_dim;
  st = set_rows(q, q_token_stride, q_head_stride, size, &a.x[0], &a.x_token[0], &a.x_head[0], &whole);
  if (st == IDX_OK)
    st = set_rows(q_out_grad, qg_token_stride, qg_head_stride, size, &a.dy[0], &a.dy_token[0],
                  &a.dy_head[0], &whole);
  if (st == IDX_OK)
    st = set_rows(q_grad, qt, head_dim, size, const_cast<const void **>(&a.out[0]), &a.out_token[0],
                  &a.out_head[0], &whole);
  if (st == IDX_OK && k_heads > 0)
    st = set_rows(k, k_token_stride, k_head_stride, size, &a.x[1], &a.x_token[1], &a.x_head[1], &whole);
  if (st == IDX_OK && k_heads > 0)
    st = set_rows(k_out_grad, kg_token_stride, kg_head_stride, size, &a.dy[1], &a.dy_token[1],
                  &a.dy_head[1], &whole);
  if (st == IDX_OK && k_heads > 0)
    st = set_rows(k_grad, kt, head_dim, size, const_cast<const void **>(&a.out[1]), &a.out_token[1],
                  &a.out_head[1], &whole);
  if (st != IDX_OK) return st;
  int32_t sms = 0;
  st = idx::resolve_sms(0, &sms);
  if (st != IDX_OK) return st;
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < (idx::heads_blocks(sms) + 1ll) * head_dim * 4)
    return fail(IDX_INVALID_ARG, "workspace (16-byte aligned) below "
                                 "idx_norm_rotary_workspace_bytes(...)");
  a.dweight[0] = q_weight_grad;
  a.dweight[1] = k_weight_grad;
  a.workspace = static_cast<float *>(workspace);
  a.sin_sign = -1.0f;
  const cudaError_t e = idx::launch_heads_backward(a, dtype, whole && dim_in_pieces(a), sms,
                                                   static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? IDX_OK : cuda_fail(e, "norm_rotary_backward launch");
}
