// index_prepare.cu -- the indexer's inputs in 8 bits: each row is rotated, divided by its scale
// max|x| / 448 and rounded to e4m3.  A key row goes to its page of the pool (the values, then the
// float32 scales of the page's tokens); a query row goes to q_out, and its scale, which is
// positive and so commutes with the ReLU of the logits, into the head's weight:
//   sum_h w_h relu(q_h . k) = sum_h (w_h s_h) relu((q_h / s_h) . k).

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace idx {

__device__ int g_index_status;

namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 7.8886090522101180541e-31f;  // 2^-100: a row of zeros has a scale too

// A warp takes four rows of one token (its query heads, then its key), eight lanes a row; lane j
// of the eight holds pieces j, j + 8, ... of V elements.
//
// What bounds the kernel is its instructions (some 260 a warp, two thirds of the issue slots) and
// the latency of finding a token's place, behind which only other warps help: 32 registers, 64
// warps an SM.  465 MB of prompts take 114 us (floor 69; at 40 registers 132).  Several rows a warp,
// rows read ahead into registers, and a token's place found once for a CTA each took more registers
// than they saved time (165 to 335 us).
template <typename T, int V, int D>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 8 : 5) k_index_prepare(const IndexArgs a, uint32_t units) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t unit = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= units) return;
  const int lane = threadIdx.x & 31, j = lane & 7;
  const uint32_t per_token = (a.heads + 4) / 4;  // four rows a unit, heads + 1 rows
  const int t = unit / per_token;
  const int row = (unit - t * per_token) * 4 + lane / 8;
  const bool is_k = row == a.heads;
  const Place p = place_of(a.m, t, lane);
  if (p.b < 0) return;
  const bool live = row <= a.heads;
  const T *x = is_k || !live
                   ? static_cast<const T *>(a.k) + t * a.k_token
                   : static_cast<const T *>(a.q) + t * a.q_token + row * a.q_head;
  const float2 *cs = nullptr;
  if (a.r.table != nullptr && p.pos >= 0) {
    if (p.pos < a.r.max_positions)
      cs = a.r.table + static_cast<int64_t>(p.pos) * (a.r.rot >> 1);
    else if (is_k && j == 0)
      atomicOr(&g_index_status, IDX_DEV_BAD_POSITION);
  }
  constexpr int kPieces = D / V / 8;
  float v[kPieces][V];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int d = (j + 8 * i) * V;
    turned<T, V>(load_piece<T, V>(x + d), x, d, a.r, cs, v[i]);
    amax = largest(v[i], amax);
  }
  if (is_inf(amax)) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) amax = largest_finite(v[i], amax);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // No division (46 instructions each): the scale is within a unit of the 24th bit of max|x| / 448,
  // and the quotients, by the scale's reciprocal, within three, before they are rounded to four bits.
  const float scale = fmaxf(amax, kTiny) * (1.0f / 448.0f);
  const float inv = __fdividef(1.0f, scale);
  if (!live) return;
  uint8_t *dst;
  if (is_k) {
    if (p.pos < 0) return;
    const int blk = p.pos / a.block_size, at = p.pos - blk * a.block_size;
    int id = -1;
    if (blk < a.m.bt_width) id = __ldg(a.m.block_tables + p.b * a.m.bt_stride + blk);
    if (id < 0 || id >= a.num_blocks) {
      if (j == 0) atomicOr(&g_index_status, IDX_DEV_BAD_PAGE);
      return;
    }
    uint8_t *page = a.pool + static_cast<int64_t>(id) * (a.block_size * (D + 4));
    dst = page + at * D;
    if (j == 0) reinterpret_cast<float *>(page + a.block_size * D)[at] = scale;
  } else {
    dst = a.q_out + (static_cast<int64_t>(t) * a.heads + row) * D;
    if (j == 0)
      a.weights_out[static_cast<int64_t>(t) * a.heads + row] =
          __ldg(a.weights + t * a.w_token + row) * scale;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) store_e4m3<V>(dst + (j + 8 * i) * V, v[i], inv);
}

template <typename T, int V>
cudaError_t launch(const IndexArgs &a, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.m.tokens) * ((a.heads + 4) / 4);
  if (units > UINT32_MAX / 2) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32)));
  const uint32_t n = static_cast<uint32_t>(units);
  switch (a.dim) {
    case 64: return launch_dependent(k_index_prepare<T, V, 64>, grid, dim3(kThreads), 0, stream, a, n);
    case 128: return launch_dependent(k_index_prepare<T, V, 128>, grid, dim3(kThreads), 0, stream, a, n);
    case 192: return launch_dependent(k_index_prepare<T, V, 192>, grid, dim3(kThreads), 0, stream, a, n);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_index_prepare(const IndexArgs &a, int dtype, bool vectors, cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32:
      return vectors ? launch<float, 4>(a, stream) : launch<float, 1>(a, stream);
    case IDX_DTYPE_F16:
      return vectors ? launch<__half, 8>(a, stream) : launch<__half, 1>(a, stream);
    default:
      return vectors ? launch<__nv_bfloat16, 8>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
  }
}

cudaError_t index_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_index_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_index_status, &zero, sizeof(int32_t));
}

}  // namespace idx
