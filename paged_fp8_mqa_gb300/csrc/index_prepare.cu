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

// x / scale, rounded, for a piece (inv: 1 / scale within a unit or two).  The remainder is taken the
// other way about, so that a zero keeps its sign.
template <int V>
__device__ __forceinline__ void quotients(float (&x)[V], float scale, float inv) {
  if constexpr (V == 2) {
    const float2 a = make_float2(x[0], x[1]), i2 = make_float2(inv, inv);
    const float2 q = __fmul2_rn(a, i2);
    const float2 r = __ffma2_rn(__ffma2_rn(q, make_float2(scale, scale), make_float2(-x[0], -x[1])),
                                make_float2(-inv, -inv), q);
    x[0] = r.x;
    x[1] = r.y;
  } else {
    const float q = x[0] * inv;
    x[0] = fmaf(fmaf(q, scale, -x[0]), -inv, q);
  }
}

// A row of D elements in a warp (see kPieces).
template <typename T, int V, int D>
struct Row {
  static constexpr int N = kPieces<V, D>;
  Piece<T, V> own[N];

  __device__ __forceinline__ void load(const T *x, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) own[i] = load_piece<T, V>(x + (lane + 32 * i) * V);
  }

  // Turns the row (still at x), writes its bytes to dst, if there is one, and returns its scale.
  __device__ __forceinline__ float finish(const T *x, int lane, const Turn<V> (&t)[N],
                                          uint8_t *dst) const {
    float v[N][V], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      turned<T, V>(own[i], x + (lane + 32 * i) * V, t[i], v[i]);
      amax = largest(v[i], amax);
    }
    amax = warp_max(amax);
    if (is_inf(amax)) {
      amax = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) amax = largest_finite(v[i], amax);
      amax = fmaxf(warp_max(amax), kTiny);
#pragma unroll
      for (int i = 0; i < N; ++i)  // (an infinity is held at the largest code, as this is)
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (is_inf(fabsf(v[i][j]))) v[i][j] = copysignf(amax, v[i][j]);
    }
    // The scale is within a unit of the 24th bit of max|x| / 448 (a product).  The codes are those of
    // the quotients by it as a division rounds them.  A division an element would be 46
    // instructions; the product with a reciprocal alone, three units off, put one code in 10^5 on
    // its neighbour.  One step of Markstein's mends it: the remainder x - q scale comes out of one
    // fused operation, and q + remainder * inv is within 2^-21 of a unit before it is rounded.
    const float scale = fmaxf(amax, kTiny) * (1.0f / 448.0f);
    const float inv = __fdividef(1.0f, scale);
    if (dst != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        quotients(v[i], scale, inv);
        store_e4m3<V>(dst + (lane + 32 * i) * V, v[i]);
      }
    }
    return scale;
  }
};

// Units [0, tokens * share): a warp takes HEADS query heads of one token, whose place and angles
// are found once for them; their loads are on their way before that, four rows at a time.  Units
// after that: a key each.
//
// 465 MB of prompts take 117 us (floor 69; 103 with a product in place of the rounded quotient): a
// warp a row and two elements a lane, so that a warp's loads of angles are whole lines and its lanes
// hold four registers of them for sixteen rows.  With eight lanes a row and 16-byte pieces, whose
// angles lie 64 bytes apart, it was 11 to 38 us more, at best with 32 registers and no row ahead.
template <typename T, int V, int D, int HEADS>
__global__ void __launch_bounds__(kThreads, 6) k_index_prepare(const IndexArgs a, uint32_t units,
                                                            uint32_t share) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t unit = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= units) return;
  const int lane = threadIdx.x & 31;
  const uint32_t q_units = static_cast<uint32_t>(a.m.tokens) * share;
  const bool is_k = unit >= q_units;
  const int t = is_k ? unit - q_units : unit / share;
  constexpr int N = kPieces<V, D>, BATCH = HEADS < 4 ? HEADS : 4;
  const int head = is_k ? 0 : static_cast<int>(unit - t * share) * HEADS;
  const int n = is_k ? 1 : min(HEADS, a.heads - head);
  const T *x = is_k ? static_cast<const T *>(a.k) + t * a.k_token
                    : static_cast<const T *>(a.q) + t * a.q_token + head * a.q_head;
  Row<T, V, D> row[BATCH];
#pragma unroll
  for (int i = 0; i < BATCH; ++i)
    if (i < n) row[i].load(x + i * a.q_head, lane);
  float weight = 0.0f;  // lane r: of head + r
  if (!is_k && lane < n) weight = __ldg(a.weights + t * a.w_token + head + lane);
  const Place p = place_of(a.m, t, lane);
  if (p.b < 0) return;
  const float2 *angles = nullptr;
  if (a.r.table != nullptr && p.pos >= 0) {
    if (p.pos < a.r.max_positions)
      angles = a.r.table + static_cast<int64_t>(p.pos) * (a.r.rot >> 1);
    else if (lane == 0)
      atomicOr(&g_index_status, IDX_DEV_BAD_POSITION);
  }
  Turn<V> turn[N];
#pragma unroll
  for (int i = 0; i < N; ++i) turn[i] = turn_of<V>(a.r, angles, (lane + 32 * i) * V);
  if (is_k) {
    uint8_t *dst = nullptr;
    float *scale_at = nullptr;
    if (p.pos >= 0) {
      const int blk = p.pos / a.block_size, at = p.pos - blk * a.block_size;
      int id = -1;
      if (blk < a.m.bt_width) id = __ldg(a.m.block_tables + p.b * a.m.bt_stride + blk);
      if (id >= 0 && id < a.num_blocks) {
        uint8_t *page = a.pool + static_cast<int64_t>(id) * (a.block_size * (D + 4));
        dst = page + at * D;
        scale_at = reinterpret_cast<float *>(page + a.block_size * D) + at;
      } else if (lane == 0) {
        atomicOr(&g_index_status, IDX_DEV_BAD_PAGE);
      }
    }
    const float scale = row[0].finish(x, lane, turn, dst);
    if (lane == 0 && scale_at != nullptr) *scale_at = scale;
    return;
  }
  const int64_t line = static_cast<int64_t>(t) * a.heads + head;
  uint8_t *dst = a.q_out + line * D;
  float mine = 0.0f;  // lane r: the scale of head + r
#pragma unroll
  for (int r0 = 0; r0 < HEADS; r0 += BATCH) {
    if (r0 >= n) break;
    if (r0 > 0) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (r0 + i < n) row[i].load(x + (r0 + i) * a.q_head, lane);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (r0 + i >= n) break;
      const float scale = row[i].finish(x + (r0 + i) * a.q_head, lane, turn, dst + (r0 + i) * D);
      if (lane == r0 + i) mine = scale;
    }
  }
  if (lane < n) a.weights_out[line + lane] = weight * mine;
}

template <typename T, int V, int D, int HEADS>
cudaError_t launch_heads(const IndexArgs &a, cudaStream_t stream) {
  const uint32_t share = (a.heads + HEADS - 1) / HEADS;
  const int64_t units = static_cast<int64_t>(a.m.tokens) * (share + 1);
  if (units > UINT32_MAX / 2) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32)));
  return launch_dependent(k_index_prepare<T, V, D, HEADS>, grid, dim3(kThreads), 0, stream, a,
                          static_cast<uint32_t>(units), share);
}

template <typename T, int V, int D>
cudaError_t launch_dim(const IndexArgs &a, cudaStream_t stream) {
  // Few rows: a warp for every two heads, for the latency; many: sixteen, for the angles' sake.
  if (static_cast<int64_t>(a.m.tokens) * a.heads > 32768) return launch_heads<T, V, D, 16>(a, stream);
  return launch_heads<T, V, D, 2>(a, stream);
}

template <typename T, int V>
cudaError_t launch(const IndexArgs &a, cudaStream_t stream) {
  switch (a.dim) {
    case 64: return launch_dim<T, V, 64>(a, stream);
    case 128: return launch_dim<T, V, 128>(a, stream);
    case 192: return launch_dim<T, V, 192>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_index_prepare(const IndexArgs &a, int dtype, bool pairs, cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32:
      return pairs ? launch<float, 2>(a, stream) : launch<float, 1>(a, stream);
    case IDX_DTYPE_F16:
      return pairs ? launch<__half, 2>(a, stream) : launch<__half, 1>(a, stream);
    default:
      return pairs ? launch<__nv_bfloat16, 2>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
  }
}

cudaError_t index_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_index_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_index_status, &zero, sizeof(int32_t));
}

}  // namespace idx
