// rows.cuh -- device helpers shared by the operators that read rows of a head: 16-byte pieces of
// float32 / float16 / bfloat16, the rotation of pairs, the e4m3 conversion and the place of a
// token in its request.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "layer.h"

namespace idx {

// The float32 value of one element.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V consecutive elements, as one load or store (V * sizeof(T) = 4, 8 or 16 bytes) or as one
// element (V = 1).
template <typename T, int V>
struct alignas(V * sizeof(T)) Piece {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T *p) {
  return *reinterpret_cast<const Piece<T, V> *>(p);
}

template <typename T, int V>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, V> &v) {
  *reinterpret_cast<Piece<T, V> *>(p) = v;
}

// The two products are rounded before the sum, so that a value does not depend on which of them
// the compiler would have fused.
__device__ __forceinline__ float turn_a(float a, float b, float2 cs) {
  return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turn_b(float a, float b, float2 cs) {
  return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// Elements [d, d + V) of the row at `x`, rotated by the angles at `cs` (one per pair; nullptr: as
// they are), in float32.  With V > 1 the caller has checked that offset, rot / 2 and d are
// multiples of V.
template <typename T, int V>
__device__ __forceinline__ void load_turned(const T *x, int d, const Rotation &r, const float2 *cs,
                                            float (&out)[V]) {
  const Piece<T, V> own = load_piece<T, V>(x + d);
  const int i = d - r.offset;
  if (cs == nullptr || i < 0 || i >= r.rot) {
#pragma unroll
    for (int j = 0; j < V; ++j) out[j] = to_f32(own.e[j]);
    return;
  }
  if (r.interleaved) {
    if constexpr (V == 1) {
      const float2 c = cs[i >> 1];
      const float other = to_f32(x[(i & 1) ? d - 1 : d + 1]);
      out[0] = (i & 1) ? turn_b(other, to_f32(own.e[0]), c) : turn_a(to_f32(own.e[0]), other, c);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 c = cs[(i >> 1) + j];
        const float a = to_f32(own.e[2 * j]), b = to_f32(own.e[2 * j + 1]);
        out[2 * j] = turn_a(a, b, c);
        out[2 * j + 1] = turn_b(a, b, c);
      }
    }
    return;
  }
  const int half = r.rot >> 1;
  const bool first = i < half;
  const Piece<T, V> other = load_piece<T, V>(x + (first ? d + half : d - half));
  const float2 *c = cs + (first ? i : i - half);
#pragma unroll
  for (int j = 0; j < V; ++j)
    out[j] = first ? turn_a(to_f32(own.e[j]), to_f32(other.e[j]), c[j])
                   : turn_b(to_f32(other.e[j]), to_f32(own.e[j]), c[j]);
}

// |x| for the largest magnitude of a row: 0 for what is not finite, which has no say in a scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __int_as_float(0x7F800000) ? a : 0.0f;
}

// Four floats as e4m3 bytes: to nearest even, values past +-448 (infinities too) to +-448, NaN to
// the NaN code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Two e4m3 bytes as floats (exact: every e4m3 value is a float16).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// The request that token t belongs to, found by the whole warp together (every lane passes the
// same t): 32 boundaries at a time.  Empty requests are passed over.
__device__ __forceinline__ int find_request(const int32_t *starts, int batch, int t, int lane) {
  int lo = 0, n = batch;  // the answer is the last b in [lo, lo + n) with starts[b] <= t
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + min(lane * step, n - 1);
    const unsigned below = __ballot_sync(0xffffffffu, __ldg(starts + at) <= t && lane * step < n);
    const int last = below == 0 ? 0 : 31 - __clz(below);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) break;
  }
  return lo;
}

struct Place {
  int b;    // request; -1: the token is past the last request's (padding)
  int pos;  // position in it; negative: the request is shorter than its new tokens
};

__device__ __forceinline__ Place place_of(const TokenMap &m, int t, int lane) {
  Place p;
  int end;  // the token one past the request's
  if (m.starts == nullptr) {
    p.b = t / m.next_n;
    end = (p.b + 1) * m.next_n;
  } else {
    p.b = find_request(m.starts, m.batch, t, lane);
    end = __ldg(m.starts + p.b + 1);
  }
  p.pos = __ldg(m.seq_lens + p.b * m.sl_stride) - (end - t);
  if (t >= end) p.b = p.pos = -1;
  return p;
}

}  // namespace idx
