// rotary.cu -- rotary positions: x'[a] = x[a] cos - x[b] sin, x'[b] = x[b] cos + x[a] sin for the
// pairs (a, b) of the rotated part of each head, with (cos, sin) from a table of positions.  The
// inverse rotation (sin negated) is the gradient with respect to x.

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace idx {

__device__ int g_rotary_status;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 512;  // pairs of the widest table the builder takes

// A thread takes one item of a token's row -- V pairs, or V elements to copy -- and walks HEADS
// heads with it, so that the V (cos, sin) of the item are read once for all of them and HEADS
// loads are in flight at once.
template <typename T, int V, int HEADS>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotaryArgs a, uint32_t first_token,
                                                     uint32_t total) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
  if (id >= total) return;
  const int half = a.r.rot >> 1;
  const uint32_t turns = half / V;
  const uint32_t items = turns + (a.copy ? (a.dim - a.r.rot) / V : 0);
  const uint32_t groups = (a.heads + HEADS - 1) / HEADS;
  const uint32_t rest = id / items;
  const int item = id - rest * items;
  const uint32_t tok = rest / groups;
  const int h0 = (rest - tok * groups) * HEADS;
  const int64_t t = static_cast<int64_t>(first_token) + tok;
  const int n = min(HEADS, a.heads - h0);
  const T *x = static_cast<const T *>(a.x) + t * a.x_token + h0 * a.x_head;
  T *out = static_cast<T *>(a.out) + t * a.out_token + h0 * a.out_head;
  if (item >= static_cast<int>(turns)) {
    int d = (item - turns) * V;
    if (d >= a.r.offset) d += a.r.rot;
    Piece<T, V> v[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h < n) v[h] = load_piece<T, V>(x + h * a.x_head + d);
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h < n) store_piece<T, V>(out + h * a.out_head + d, v[h]);
    return;
  }
  // Interleaved pairs: the item's 2V consecutive elements hold its V pairs.
  const int da = a.r.offset + item * (a.r.interleaved ? 2 * V : V);
  const int db = da + (a.r.interleaved ? V : half);
  Piece<T, V> va[HEADS], vb[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h < n) {
      va[h] = load_piece<T, V>(x + h * a.x_head + da);
      vb[h] = load_piece<T, V>(x + h * a.x_head + db);
    }
  const int pos = __ldg(a.positions + t);
  float2 cs[V];
  if (static_cast<uint32_t>(pos) < static_cast<uint32_t>(a.r.max_positions)) {
    const float2 *row = a.r.table + static_cast<int64_t>(pos) * half + item * V;
    if constexpr (V == 1) {
      cs[0] = __ldg(row);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float4 two = __ldg(reinterpret_cast<const float4 *>(row) + j);
        cs[2 * j] = make_float2(two.x, two.y);
        cs[2 * j + 1] = make_float2(two.z, two.w);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) cs[j].y *= a.sin_sign;
  } else {
    // As it is, to the bit: a product with a sine of 0 would make an infinity's partner NaN.
    if (item == 0 && h0 == 0) atomicOr(&g_rotary_status, IDX_DEV_BAD_POSITION);
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
      if (h < n) {
        store_piece<T, V>(out + h * a.out_head + da, va[h]);
        store_piece<T, V>(out + h * a.out_head + db, vb[h]);
      }
    return;
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h >= n) break;
    if (V > 1 && a.r.interleaved) {
      // Both pieces hold whole pairs.
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float a0 = to_f32(va[h].e[2 * j]), b0 = to_f32(va[h].e[2 * j + 1]);
        const float a1 = to_f32(vb[h].e[2 * j]), b1 = to_f32(vb[h].e[2 * j + 1]);
        va[h].e[2 * j] = from_f32<T>(turn_a(a0, b0, cs[j]));
        va[h].e[2 * j + 1] = from_f32<T>(turn_b(a0, b0, cs[j]));
        vb[h].e[2 * j] = from_f32<T>(turn_a(a1, b1, cs[V / 2 + j]));
        vb[h].e[2 * j + 1] = from_f32<T>(turn_b(a1, b1, cs[V / 2 + j]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x0 = to_f32(va[h].e[j]), x1 = to_f32(vb[h].e[j]);
        va[h].e[j] = from_f32<T>(turn_a(x0, x1, cs[j]));
        vb[h].e[j] = from_f32<T>(turn_b(x0, x1, cs[j]));
      }
    }
    store_piece<T, V>(out + h * a.out_head + da, va[h]);
    store_piece<T, V>(out + h * a.out_head + db, vb[h]);
  }
}

struct Frequencies {
  double f[kMaxHalf];
};

// table[p][i] = magnitude * (cos, sin)(p * f[i]): the angle, its cosine and sine in 64 bits, one
// rounding to float32 (an angle of 10^5 radians in 32 bits is off by up to 0.004).
__global__ void __launch_bounds__(kThreads) k_rotary_table(const __grid_constant__ Frequencies f,
                                                           double magnitude, int32_t positions,
                                                           int32_t half, float2 *table) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t n = static_cast<int64_t>(positions) * half;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t p = i / half;
    double s, c;
    sincos(static_cast<double>(p) * f.f[i - p * half], &s, &c);
    table[i] = make_float2(static_cast<float>(magnitude * c), static_cast<float>(magnitude * s));
  }
}

template <typename T, int V>
cudaError_t launch(const RotaryArgs &a, cudaStream_t stream) {
  constexpr int kHeads = 2;
  const int64_t per_token =
      static_cast<int64_t>(a.r.rot / 2 / V + (a.copy ? (a.dim - a.r.rot) / V : 0)) *
      ((a.heads + kHeads - 1) / kHeads);
  if (per_token == 0) return cudaSuccess;
  // The thread index is 32 bits wide: more tokens than fit it go in several launches.
  const int64_t most = (INT64_C(1) << 31) / per_token;
  if (most == 0) return cudaErrorInvalidValue;
  for (int64_t t = 0; t < a.tokens; t += most) {
    const int64_t n = a.tokens - t < most ? a.tokens - t : most;
    const uint32_t total = static_cast<uint32_t>(n * per_token);
    const cudaError_t e = launch_dependent(
        k_rotary<T, V, kHeads>, dim3((total + kThreads - 1) / kThreads), dim3(kThreads), 0, stream,
        a, static_cast<uint32_t>(t), total);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, int dtype, bool vectors, cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32:
      return vectors ? launch<float, 4>(a, stream) : launch<float, 1>(a, stream);
    case IDX_DTYPE_F16:
      return vectors ? launch<__half, 8>(a, stream) : launch<__half, 1>(a, stream);
    default:
      return vectors ? launch<__nv_bfloat16, 8>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
  }
}

cudaError_t launch_rotary_table(const double *inv_freq, double magnitude, int32_t positions,
                                int32_t half, float2 *table, cudaStream_t stream) {
  if (half > kMaxHalf) return cudaErrorInvalidValue;
  Frequencies f;
  for (int i = 0; i < kMaxHalf; ++i) f.f[i] = i < half ? inv_freq[i] : 0.0;
  const int64_t n = static_cast<int64_t>(positions) * half;
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  return launch_dependent(k_rotary_table, dim3(static_cast<unsigned>(blocks < 4864 ? blocks : 4864)),
                          dim3(kThreads), 0, stream, f, magnitude, positions, half, table);
}

cudaError_t rotary_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_rotary_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_rotary_status, &zero, sizeof(int32_t));
}

}  // namespace idx
