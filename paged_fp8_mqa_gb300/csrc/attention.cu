// attention.cu -- attention over the 8-bit K/V cache: for row (b, t) and query head h with K/V
// head g = h / (heads / kv_heads),
//   z_p = scale * ks[page(p), g] * (q . k_p),  out = sum_p softmax(z)_p * vs[page(p), g] * v_p
// over the positions p <= seq_lens[b] - next_n + t, or over those of them that the select stored
// in the row's slots.  A row without positions gives zeros (and a log-sum of -inf).

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace idx {

__device__ int g_attention_status;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// One CTA a (row, query head): its warps walk the positions in turn, each with a running maximum
// and sum, and join at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_attention(const AttentionArgs a) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.x, h = blockIdx.y;
  const int b = r / a.next_n, t = r - b * a.next_n;
  const int g = h / (a.heads / a.kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = __ldg(a.seq_lens + b * a.sl_stride);
  const int extent = max(0, len - a.next_n + t + 1);
  int lo = 0, n = extent;
  if (a.candidates != nullptr) {
    lo = max(0, __ldg(a.ranges + r));
    n = max(0, min(__ldg(a.ranges + a.batch * a.next_n + r), a.slots) - lo);
  }
  const T *q = static_cast<const T *>(a.q) + b * a.q_batch + t * a.q_token + h * a.q_head;
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f32(q[lane * E + e]) * a.scale;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int i = warp; i < n; i += kWarps) {
    const int p = a.candidates ? a.candidates[r * a.cand_stride + lo + i].x : i;
    if (p < 0 || p >= extent) continue;
    const int blk = p / a.block_size, at = p - blk * a.block_size;
    const int id = blk < a.bt_width ? __ldg(a.block_tables + b * a.bt_stride + blk) : -1;
    if (id < 0 || id >= a.num_blocks) {
      if (lane == 0) atomicOr(&g_attention_status, IDX_DEV_BAD_PAGE);
      continue;
    }
    const int64_t page = static_cast<int64_t>(id) * a.kv_heads + g;
    const int64_t row = (page * a.block_size + at) * D + lane * E;
    float z = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 k2 = e4m3x2_to_f32(*reinterpret_cast<const uint16_t *>(a.k_pool + row + e));
      const float2 v2 = e4m3x2_to_f32(*reinterpret_cast<const uint16_t *>(a.v_pool + row + e));
      z += qv[e] * k2.x + qv[e + 1] * k2.y;
      v[e] = v2.x;
      v[e + 1] = v2.y;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= a.k_scales[page];
    const float vs = a.v_scales[page];
    const float mn = fmaxf(m, z);
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float c = expf(m - ref), w = expf(z - ref);
    m = mn;
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * vs * v[e];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float mm = -INFINITY, ll = 0.0f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
  const float ref = mm == -INFINITY ? 0.0f : mm;
  for (int w = 0; w < kWarps; ++w) ll += s_l[w] * expf(s_m[w] - ref);
  T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(r) * a.heads + h) * D;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x += s_o[w][d] * expf(s_m[w] - ref);
    out[d] = from_f32<T>(ll == 0.0f ? 0.0f : x / ll);
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[static_cast<int64_t>(r) * a.heads + h] = ll == 0.0f ? -INFINITY : mm + logf(ll);
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs &a, int dtype, int ctas, cudaStream_t stream) {
  (void)ctas;
  const dim3 grid(a.batch * a.next_n, a.heads);
  if (dtype == IDX_DTYPE_F16)
    return a.dim == 64
               ? launch_dependent(k_attention<__half, 64>, grid, dim3(kThreads), 0, stream, a)
               : launch_dependent(k_attention<__half, 128>, grid, dim3(kThreads), 0, stream, a);
  return a.dim == 64
             ? launch_dependent(k_attention<__nv_bfloat16, 64>, grid, dim3(kThreads), 0, stream, a)
             : launch_dependent(k_attention<__nv_bfloat16, 128>, grid, dim3(kThreads), 0, stream, a);
}

cudaError_t attention_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_attention_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(int32_t));
}

}  // namespace idx
