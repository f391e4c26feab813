// pieces.cuh -- rows of a head in the hands of a few lanes: a lane holds two pieces of eight elements, chosen
// so that both elements of every rotated pair are its own, and works on them two at a time.
#pragma once

#include "rows.cuh"

namespace idx {

// A lane's two pieces of a head of D = 16 * (lanes at work) elements, and how they are turned.
struct Pieces {
  int at[2];       // their first elements
  bool on[2];      // rotated
  float2 cs[8];    // the angles of the lane's pairs
  uint32_t valid;  // bit k: pair k is turned (its position is in the table)
};

// Where lane l's pieces lie (which does not depend on the token), and the pairs of their angles 0 and 4.
// Interleaved (ADJ) pairs are neighbours in a piece; else element k of the first piece goes with element k
// of the second.  What is not rotated is shared out in the same way: the first half of its pieces first.
template <bool ADJ>
__device__ __forceinline__ void place_pieces(const Rotation &r, int dim, int l, Pieces &p,
                                             int (&pair)[2]) {
  const int off = r.offset, rot = r.table != nullptr ? r.rot : 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (ADJ) {
      p.at[s] = 8 * l + s * (dim >> 1);
      p.on[s] = p.at[s] >= off && p.at[s] < off + rot;
      pair[s] = (p.at[s] - off) >> 1;
    } else if (l < rot / 16) {
      p.at[s] = off + 8 * l + s * (rot >> 1);
      p.on[s] = true;
      pair[s] = 8 * l + 4 * s;
    } else {
      const int e = 8 * (l - rot / 16) + s * ((dim - rot) >> 1);
      p.at[s] = e < off ? e : e + rot;
      p.on[s] = false;
      pair[s] = 0;
    }
  }
}

// The lane's 16 elements in float32, the first elements of its eight pairs in v[0], the second in v[1],
// two a register pair.
template <bool ADJ, typename T>
__device__ __forceinline__ void unpack(const Piece<T, 8> (&p)[2], float2 (&v)[2][4]) {
  float f[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s) piece_f32<T, 8>(p[s], f[s]);
  if constexpr (ADJ) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float *g = f[j >> 1] + 4 * (j & 1) + s;
        v[s][j] = make_float2(g[0], g[2]);
      }
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[s][j] = make_float2(f[s][2 * j], f[s][2 * j + 1]);
  }
}

// Two floats as two elements.
template <typename T>
__device__ __forceinline__ void put_two(Piece<T, 8> &p, int at, float a, float b) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
    p.e[at] = two.x;
    p.e[at + 1] = two.y;
  } else if constexpr (std::is_same_v<T, __half>) {
    const __half2 two = __floats2half2_rn(a, b);
    p.e[at] = two.x;
    p.e[at + 1] = two.y;
  } else {
    p.e[at] = a;
    p.e[at + 1] = b;
  }
}

template <bool ADJ, typename T>
__device__ __forceinline__ void pack(const float2 (&v)[2][4], Piece<T, 8> (&p)[2]) {
  if constexpr (ADJ) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      put_two<T>(p[j >> 1], 4 * (j & 1), v[0][j].x, v[1][j].x);
      put_two<T>(p[j >> 1], 4 * (j & 1) + 2, v[0][j].y, v[1][j].y);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) put_two<T>(p[s], 2 * j, v[s][j].x, v[s][j].y);
  }
}

// Element (s, j, e) of the lane's 16 as they are unpacked: its place in the head.
template <bool ADJ>
__device__ __forceinline__ int element_at(const Pieces &p, int s, int j, int e) {
  return ADJ ? p.at[j >> 1] + 4 * (j & 1) + 2 * e + s : p.at[s] + 2 * j + e;
}

// The pairs' cosines and sines, two a register pair.
__device__ __forceinline__ void angles_of(const Pieces &p, float2 (&c)[4], float2 (&n)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = make_float2(p.cs[2 * j].x, p.cs[2 * j + 1].x);
    n[j] = make_float2(p.cs[2 * j].y, p.cs[2 * j + 1].y);
  }
}
__device__ __forceinline__ float2 minus(float2 x) { return make_float2(-x.x, -x.y); }

// v, the lane's 16 elements, turned: both products rounded before their sum.  A pair that is not turned
// stays to the bit (a product with a sine of 0 would make an infinity's partner NaN).
__device__ __forceinline__ void turn(uint32_t valid, const float2 (&c)[4], const float2 (&n)[4],
                                     float2 (&v)[2][4]) {
  if (valid == 0) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = v[0][j], y = v[1][j];
    v[0][j] = __ffma2_rn(__fmul2_rn(y, n[j]), make_float2(-1.0f, -1.0f), __fmul2_rn(x, c[j]));
    v[1][j] = __fadd2_rn(__fmul2_rn(y, c[j]), __fmul2_rn(x, n[j]));
    if (valid != 0xFFu) {
      if (!((valid >> (2 * j)) & 1u)) v[0][j].x = x.x, v[1][j].x = y.x;
      if (!((valid >> (2 * j + 1)) & 1u)) v[0][j].y = x.y, v[1][j].y = y.y;
    }
  }
}

// Eight elements at once, or one by one.
template <typename T>
__device__ __forceinline__ Piece<T, 8> load_whole(const T *p, bool whole) {
  if (whole) return load_piece<T, 8>(p);
  Piece<T, 8> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = p[j];
  return v;
}

}  // namespace idx
