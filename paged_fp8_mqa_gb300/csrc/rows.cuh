// rows.cuh -- device helpers shared by the operators that read rows of a head: 16-byte pieces of
// float32 / float16 / bfloat16, the rotation of pairs, the e4m3 conversion and the place of a
// token in its request.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

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

// A piece's values in float32.
template <typename T, int V>
__device__ __forceinline__ void piece_f32(const Piece<T, V> &p, float (&out)[V]) {
  if constexpr (V > 1 && sizeof(T) == 2) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&p);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        out[2 * j] = __uint_as_float(w[j] << 16);
        out[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(w + j));
        out[2 * j] = f.x;
        out[2 * j + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) out[j] = to_f32(p.e[j]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, V> &v) {
  *reinterpret_cast<Piece<T, V> *>(p) = v;
}

// A pair turned: x cos - y sin and y cos + x sin.  The two products are rounded before the sum, so
// that a value does not depend on which of them the compiler would have fused.
__device__ __forceinline__ float turn_a(float a, float b, float2 cs) {
  return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float turn_b(float a, float b, float2 cs) {
  return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// Rows of D elements in the hands of a warp: lane l holds pieces l, l + 32, ... of V elements (V = 2,
// or 1 where bases, strides or the rotated part are odd).  Two elements a lane, because a warp's
// loads of angles, which are as many floats as there are elements, are then whole lines.
template <int V, int D>
constexpr int kPieces = D / (32 * V);

// How a piece is turned: element j becomes own c[j] + other s[j], the pair's first element with the
// negated sine.  The others stand `apart` elements further in the row, or, with apart = 0, in the
// piece itself, swapped (interleaved, V = 2).
template <int V>
struct Turn {
  float c[V], s[V];
  int apart;
  bool on;  // false: the elements stay as they are
};

// The turn of elements [d, d + V) of a row whose angles are at `row` (nullptr: none).  With V = 2
// offset and rot / 2 are even and the angles 16-byte aligned (the caller has checked).
template <int V>
__device__ __forceinline__ Turn<V> turn_of(const Rotation &r, const float2 *row, int d) {
  Turn<V> t;
  const int i = d - r.offset, half = r.rot >> 1;
  t.on = row != nullptr && i >= 0 && i < r.rot;
  t.apart = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) t.c[j] = t.s[j] = 0.0f;
  if (!t.on) return t;
  const bool first = r.interleaved ? (i & 1) == 0 : i < half;
  if constexpr (V == 1) {
    const float2 cs = __ldg(row + (r.interleaved ? i >> 1 : first ? i : i - half));
    t.c[0] = cs.x;
    t.s[0] = first ? -cs.y : cs.y;
    t.apart = r.interleaved ? (first ? 1 : -1) : first ? half : -half;
  } else if (r.interleaved) {
    const float2 cs = __ldg(row + (i >> 1));
    t.c[0] = t.c[1] = cs.x;
    t.s[0] = -cs.y;
    t.s[1] = cs.y;
  } else {
    const float4 cs = __ldg(reinterpret_cast<const float4 *>(row + (first ? i : i - half)));
    t.c[0] = cs.x;
    t.c[1] = cs.z;
    t.s[0] = first ? -cs.y : cs.y;
    t.s[1] = first ? -cs.w : cs.w;
    t.apart = first ? half : -half;
  }
  return t;
}

// The piece `own` of V elements at x in float32, turned (the others are read from memory, where
// their lines are in L1 by then).
template <typename T, int V>
__device__ __forceinline__ void turned(const Piece<T, V> &own, const T *x, const Turn<V> &t,
                                       float (&out)[V]) {
  piece_f32<T, V>(own, out);
  if (!t.on) return;
  float other[V];
  if (V == 2 && t.apart == 0) {
    other[0] = out[V - 1];
    other[V - 1] = out[0];
  } else {
    piece_f32<T, V>(load_piece<T, V>(x + t.apart), other);
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    out[j] = __fadd_rn(__fmul_rn(out[j], t.c[j]), __fmul_rn(other[j], t.s[j]));
}

// The largest x of the warp's lanes (a NaN loses against a number).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The largest magnitude of N values; NaN has no say in it (fmaxf passes it over), infinities have.
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N], float so_far) {
#pragma unroll
  for (int j = 0; j < N; ++j) so_far = fmaxf(so_far, fabsf(v[j]));
  return so_far;
}
// The same without the infinities, for the rare case that there are some.
template <int N>
__device__ __forceinline__ float largest_finite(const float (&v)[N], float so_far) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float a = fabsf(v[j]);
    so_far = a < __int_as_float(0x7F800000) ? fmaxf(so_far, a) : so_far;
  }
  return so_far;
}
__device__ __forceinline__ bool is_inf(float x) { return x == __int_as_float(0x7F800000); }

// Four floats as e4m3 bytes: to nearest even, values past +-448 (infinities too) to +-448, NaN to
// the NaN code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}\n"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return out;
}

// Four floats as e5m2 bytes, to nearest even, and the low two as floats again (an e5m2 value is the
// float16 whose upper byte it is).
__device__ __forceinline__ uint32_t e5m2x4(float a, float b, float c, float d) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}\n"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return out;
}
__device__ __forceinline__ float2 e5m2x2_to_f32(uint32_t two) {
  const uint32_t h = __byte_perm(two, 0, 0x1404);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// V values as e4m3 bytes.
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *dst, const float (&v)[V]) {
  if constexpr (V == 1) {
    *dst = static_cast<uint8_t>(e4m3x4(v[0], 0.0f, 0.0f, 0.0f));
  } else {
    static_assert(V == 2, "one or two");
    *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(e4m3x4(v[0], v[1], 0.0f, 0.0f));
  }
}
// V values times inv.
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *dst, const float (&v)[V], float inv) {
  float scaled[V];
#pragma unroll
  for (int j = 0; j < V; ++j) scaled[j] = v[j] * inv;
  store_e4m3<V>(dst, scaled);
}

// The low two e4m3 bytes as floats (exact: every e4m3 value is a float16).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}\n"
      : "=r"(h)
      : "r"(two));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
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
  int b;    // request; -1: the token is no request's (padding)
  int pos;  // position in it; negative: the request is shorter than its new tokens
};

__device__ __forceinline__ Place place_of(const TokenMap &m, int t, int lane) {
  Place p;
  int begin, end;  // the request's rows
  if (m.starts == nullptr) {
    p.b = t / m.next_n;
    begin = p.b * m.next_n;
    end = begin + m.next_n;
  } else {
    p.b = find_request(m.starts, m.batch, t, lane);
    begin = __ldg(m.starts + p.b);
    end = __ldg(m.starts + p.b + 1);
  }
  p.pos = __ldg(m.seq_lens + p.b * m.sl_stride) - (end - t);
  if (t < begin || t >= end) p.b = p.pos = -1;
  return p;
}

}  // namespace idx
