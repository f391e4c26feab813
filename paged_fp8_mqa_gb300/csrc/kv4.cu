// kv4.cu -- the 4-bit K/V cache: new keys (rotated) and values into it, and what it holds back as dense
// rows.
//
// A code is E2M1: a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A key has a scale for each 32
// elements, a power of two (UE8M0), the least with which they are at most 6: what the tensor core's
// block scaling takes, so that the attention reads keys as they lie.  A value row has one float32
// scale, its largest magnitude over 6: it goes into the softmax's weight, and a scale that is not a
// power of two brings the largest element to the largest code (a binade more precision for half of
// all rows, in as many bytes as four of a key's scales).  A token's rows depend on nothing else in the
// cache, so a page is filled token by token without touching what it holds.

#include <cuda_runtime.h>

#include "internal.h"
#include "pieces.cuh"
#include "ptx.cuh"

namespace idx {

__device__ int g_kv4_status;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLeastMax = 1.2621774483536189e-29f;  // 2^-96: a value row's least largest magnitude
constexpr float kInf = __builtin_huge_valf();

// Eight floats as codes, the first in the lowest four bits; to nearest even, past +-6 to +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t out;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return out;
}

// Eight codes' values.
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(h + j));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// 2^(byte - 127); 0xFF is NaN.
__device__ __forceinline__ float ue8m0(uint32_t byte) {
  return byte == 0 ? 5.8774717541114375e-39f  // 2^-127, below the normal range
                   : byte == 255 ? __int_as_float(0x7FC00000) : __uint_as_float(byte << 23);
}

// The least power of two, 2^-100 or more, that brings amax (finite, >= 0) to at most 6 = 1.5 * 2^2:
// its exponent, off amax's bits.
__device__ __forceinline__ int key_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 2 + ((u & 0x7FFFFFu) > 0x400000u);
  return max(e, -100);
}

// Elements [d, d + 8) of a key, turned by the angles at `row`.  turns: the pairs lie in whole pieces,
// eight elements and as many angles at a time.
template <typename T>
__device__ __forceinline__ void turn8(float (&v)[8], const T *x, int d, const Rotation &r,
                                      const float2 *row, bool turns) {
  const int half = r.rot >> 1;
  if (turns) {
    const int i = d - r.offset;
    if (i < 0 || i >= r.rot) return;
    if (r.interleaved) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 cs = __ldg(reinterpret_cast<const float4 *>(row + (i >> 1) + j));
        const float2 one = make_float2(cs.x, cs.y), two = make_float2(cs.z, cs.w);
        const float a = v[2 * j], b = v[2 * j + 1], c = v[2 * j + 2], e = v[2 * j + 3];
        v[2 * j] = turn_a(a, b, one);
        v[2 * j + 1] = turn_b(a, b, one);
        v[2 * j + 2] = turn_a(c, e, two);
        v[2 * j + 3] = turn_b(c, e, two);
      }
    } else {
      const bool first = i < half;
      float o[8];
      piece_f32<T, 8>(load_piece<T, 8>(x + (first ? d + half : d - half)), o);
      const float4 *at = reinterpret_cast<const float4 *>(row + (first ? i : i - half));
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float4 cs = __ldg(at + j / 2);
        const float2 one = make_float2(cs.x, cs.y), two = make_float2(cs.z, cs.w);
        v[j] = first ? turn_a(v[j], o[j], one) : turn_b(o[j], v[j], one);
        v[j + 1] = first ? turn_a(v[j + 1], o[j + 1], two) : turn_b(o[j + 1], v[j + 1], two);
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = d + j - r.offset;
    if (i < 0 || i >= r.rot) continue;
    const bool first = r.interleaved ? (i & 1) == 0 : i < half;
    const int apart = r.interleaved ? 1 : half;
    const float2 cs = __ldg(row + (r.interleaved ? i >> 1 : first ? i : i - half));
    const float o = to_f32(x[d + j + (first ? apart : -apart)]);
    v[j] = first ? turn_a(v[j], o, cs) : turn_b(o, v[j], cs);
  }
}

// Where a warp's token stands in the cache; page < 0: nowhere (no request's, or flagged).
struct Spot {
  int pos;
  int64_t page;
};
__device__ __forceinline__ Spot spot_of(const Kv4Args &a, int t, int lane) {
  const Place p = place_of(a.m, t, lane);
  Spot s{p.pos, -1};
  if (p.b < 0 || p.pos < 0) return s;
  const int blk = p.pos / a.block_size;
  const int id = blk < a.m.bt_width ? __ldg(a.m.block_tables + p.b * a.m.bt_stride + blk) : -1;
  if (id >= 0 && id < a.num_blocks)
    s.page = id;
  else if (lane == 0)
    atomicOr(&g_kv4_status, IDX_DEV_BAD_PAGE);
  return s;
}

// The larger of two magnitudes; a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// The largest finite magnitude of four pairs, or NaN.
__device__ __forceinline__ float finite_or_nan(const float2 (&v)[4]) {
  float f[8];
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = v[j].x;
    f[2 * j + 1] = v[j].y;
    nan |= v[j].x != v[j].x || v[j].y != v[j].y;
  }
  return nan ? __int_as_float(0x7FC00000) : largest_finite(f, 0.0f);
}
__device__ __forceinline__ float largest_of(const float2 (&v)[4]) {
  float m = max_nan(fabsf(v[0].x), fabsf(v[0].y));
#pragma unroll
  for (int j = 1; j < 4; ++j) m = max_nan(m, max_nan(fabsf(v[j].x), fabsf(v[j].y)));
  return m;
}
__device__ __forceinline__ uint32_t codes_of(const float2 (&v)[4]) {
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  return e2m1x8(f);
}

// 6 v / amax of 16-bit elements (6 v is exact), correctly rounded by Markstein's correction: the quotient's
// remainder times the reciprocal (within 2^-22 of it) added, so that what lies halfway between two codes
// stays there, and nothing else comes to lie there (their quotients are 2^-18 from a border or on it).
__device__ __forceinline__ float2 six_over(float2 v, float2 minus_m, float2 inv) {
  const float2 x = __fmul2_rn(v, make_float2(6.0f, 6.0f)), q = __fmul2_rn(x, inv);
  return __ffma2_rn(__ffma2_rn(q, minus_m, x), inv, q);
}
// The same of any element, float32 ones too: 6 v is taken in two parts, and a quotient that is not a float is
// rounded to one with an odd last bit, so that it stays on its side of every border between codes
// (which are even floats, and may be as near as 2^-26).  Below the first border, 0.25, it may be off.
template <typename T>
__device__ __forceinline__ float six_over(float v, float m, float inv) {
  const float x = 6.0f * v;
  float q = x * inv;
  if constexpr (sizeof(T) == 2) return fmaf(fmaf(-q, m, x), inv, q);
  const float low = fmaf(6.0f, v, -x);
  q = fmaf(fmaf(-q, m, x) + low, inv, q);
  // The remainder's sign: both terms are exact, or as good as that where the first is the larger.
  const float rest = fmaf(-q, m, x) + low;
  const uint32_t bits = __float_as_uint(q);
  if (rest != 0.0f && (bits & 1u) == 0 && fabsf(q) >= 0.25f)
    q = __uint_as_float((rest > 0.0f) == (q > 0.0f) ? bits + 1u : bits - 1u);
  return q;
}
// x / 6, correctly rounded in the same way.
__device__ __forceinline__ float sixth(float x) {
  constexpr float k = 1.0f / 6.0f;
  const float q = x * k;
  return fmaf(fmaf(-q, 6.0f, x), k, q);
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Rows whose pairs lie in whole pieces and whose pieces, four lanes' together, are a key's groups of 32.  A
// warp takes one token and ROUNDS rounds of 512 / D of its heads, the keys' first, then the values', and
// asks for all of them before the token's place is known; the values are done before the keys, whose angles
// come meanwhile.
//
// 34,000 tokens of 8 heads of 128 (176 MB) take 45 us, 26 at the copy rate: an instruction-bound and a
// latency-bound half.  With eight elements a lane, whose partners another lane holds, and scalar arithmetic
// 80 us; two rounds a warp 48; several tokens a warp, one after the other, the next one's rows asked for
// ahead, 61 to 71 (fewer warps fit).  Float32 (315 MB) 70, 7 of them for the exact side of every border.
constexpr int kPieceThreads = 128;
template <typename T, int D, bool ADJ, int ROUNDS>
__global__ void __launch_bounds__(kPieceThreads, ROUNDS == 1 ? 1 : 5)
    k_kv4_append_pieces(const Kv4Args a) {
  constexpr int W = D / 16, AT_ONCE = 32 / W;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % W, group = lane / W;
  const int t = blockIdx.x * (kPieceThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.m.tokens) return;
  const int half = (a.heads + AT_ONCE - 1) / AT_ONCE;  // rounds of keys, and of values
  const int first = blockIdx.y * ROUNDS;
  Pieces p;
  int pair[2];
  place_pieces<ADJ>(a.r, D, l, p, pair);
  Piece<T, 8> own[ROUNDS][2];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    // (Past the last: that one again, so that no branch parts the loads.)
    const int r = min(first + i, 2 * half - 1);
    const bool is_k = r < half;
    const int h = min((is_k ? r : r - half) * AT_ONCE + group, a.heads - 1);
    const T *x = static_cast<const T *>(is_k ? a.k : a.v) + t * (is_k ? a.k_token : a.v_token) +
                 h * (is_k ? a.k_head : a.v_head);
    own[i][0] = load_piece<T, 8>(x + p.at[0]);
    own[i][1] = load_piece<T, 8>(x + p.at[1]);
  }
  const Spot s = spot_of(a, t, lane);
  if (s.page < 0) return;
  uint32_t valid = 0;
  float2 c[4], n[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = n[j] = make_float2(0.0f, 0.0f);
  if (a.r.table != nullptr && first < half) {
    if (s.pos < a.r.max_positions) {
      const float2 *row = a.r.table + static_cast<int64_t>(s.pos) * (a.r.rot >> 1);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (p.on[e]) {
          valid |= 0xFu << (4 * e);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 two = __ldg(reinterpret_cast<const float4 *>(row + pair[e] + 2 * j));
            c[2 * e + j] = make_float2(two.x, two.z);
            n[2 * e + j] = make_float2(two.y, two.w);
          }
        }
    } else if (lane == 0) {
      atomicOr(&g_kv4_status, IDX_DEV_BAD_POSITION);
    }
  }
  // The row of the lane's first head in this token's place.
  const int64_t row0 =
      (s.page * a.heads + group) * a.block_size + (s.pos & (a.block_size - 1));
#pragma unroll
  for (int i = ROUNDS - 1; i >= 0; --i) {
    const int r = first + i;
    const bool is_k = r < half;  // (the same for the whole warp)
    const int h0 = (is_k ? r : r - half) * AT_ONCE;
    const bool live = h0 + group < a.heads;
    const int64_t row = row0 + h0 * a.block_size;
    if (r >= 2 * half) continue;
    float2 v[2][4];
    if (is_k) {
      unpack<ADJ, T>(own[i], v);
      turn(valid, c, n, v);
      float2 u[2][4];  // the pieces' elements in order
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = v[0][2 * e + (j >> 1)], g = v[1][2 * e + (j >> 1)];
          u[e][j] = !ADJ ? v[e][j] : j & 1 ? make_float2(f.y, g.y) : make_float2(f.x, g.x);
        }
      float m[2] = {largest_of(u[0]), largest_of(u[1])};
      if (__any_sync(0xffffffffu, m[0] == kInf || m[1] == kInf))
        m[0] = finite_or_nan(u[0]), m[1] = finite_or_nan(u[1]);
      uint8_t *to = a.k_pool + row * (D / 2), *scale = a.k_scales + row * (D / 32);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[e] = max_nan(m[e], __shfl_xor_sync(0xffffffffu, m[e], 1));
        m[e] = max_nan(m[e], __shfl_xor_sync(0xffffffffu, m[e], 2));
        // (Of a NaN, whose bits are past an infinity's: 0xFF, and codes that mean nothing.)
        const int exponent = min(key_exponent(m[e]), 127);
        const float up = __uint_as_float(static_cast<uint32_t>(127 - exponent) << 23);
        const float2 up2 = make_float2(up, up);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[e][j] = __fmul2_rn(u[e][j], up2);
        const uint32_t codes = codes_of(u[e]);
        if (live) {
          *reinterpret_cast<uint32_t *>(to + p.at[e] / 2) = codes;
          if ((lane & 3) == 0) scale[p.at[e] / 32] = m[e] != m[e] ? 255 : static_cast<uint8_t>(exponent + 127);
        }
      }
    } else {
      unpack<false, T>(own[i], v);
      float m = max_nan(largest_of(v[0]), largest_of(v[1]));
      const bool odd = __any_sync(0xffffffffu, m > 1.2676506002282294e30f);  // past 2^100
      if (odd) m = max_nan(finite_or_nan(v[0]), finite_or_nan(v[1]));
#pragma unroll
      for (int o = 1; o < W; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool nan = m != m;
      m = fmaxf(m, kLeastMax);  // (of a NaN: kLeastMax; the row's scale says what it is)
      if (live && l == 0) a.v_scales[row] = nan ? __int_as_float(0x7FC00000) : sixth(m);
      if (odd) {
        // Infinities to the largest; rows past 2^100 2^64 down, so that six times them is finite.
        const float down = m > 1.2676506002282294e30f ? 5.421010862427522e-20f : 1.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[e][j].x = fminf(fmaxf(v[e][j].x, -m), m) * down;
            v[e][j].y = fminf(fmaxf(v[e][j].y, -m), m) * down;
          }
        m *= down;
      }
      const float inv = reciprocal(m);
      const float2 inv2 = make_float2(inv, inv), m2 = make_float2(-m, -m);
      uint8_t *to = a.v_pool + row * (D / 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 2)
            v[e][j] = six_over(v[e][j], m2, inv2);
          else
            v[e][j] = make_float2(six_over<T>(v[e][j].x, m, inv), six_over<T>(v[e][j].y, m, inv));
        }
        const uint32_t codes = codes_of(v[e]);
        if (live) *reinterpret_cast<uint32_t *>(to + p.at[e] / 2) = codes;
      }
    }
  }
}

// Any other rotated part, strides or alignment: a warp takes one token and ROUNDS times 32 * 8 / D of its
// 2 * heads rows (the keys, then the values), eight elements a lane, the partners read from memory.  32,768
// tokens of 8 heads of 128 take 71 us with 32 elements rotated in halves, 96 with 20 (k_kv4_append_pieces 45
// with 64 or 128).
template <typename T, int D, int ROUNDS>
__global__ void __launch_bounds__(kThreads) k_kv4_append(const Kv4Args a, bool pieces, bool turns) {
  constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.m.tokens) return;
  const int first = blockIdx.y * ROUNDS * AT_ONCE + lane / LANES, d = (lane % LANES) * 8;
  const auto row_at = [&](int n) {
    const bool is_k = n < a.heads;
    return static_cast<const T *>(is_k ? a.k : a.v) +
           t * (is_k ? a.k_token : a.v_token) + (is_k ? n * a.k_head : (n - a.heads) * a.v_head);
  };
  Piece<T, 8> own[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i)  // (past the last row: that one again, so that no branch parts the loads)
    own[i] = load_whole<T>(row_at(min(first + i * AT_ONCE, 2 * a.heads - 1)) + d, pieces);
  const Spot s = spot_of(a, t, lane);
  if (s.page < 0) return;
  const float2 *angles = nullptr;
  if (a.r.table != nullptr) {
    if (s.pos < a.r.max_positions)
      angles = a.r.table + static_cast<int64_t>(s.pos) * (a.r.rot >> 1);
    else if (lane == 0)
      atomicOr(&g_kv4_status, IDX_DEV_BAD_POSITION);
  }
  const int in_page = s.pos & (a.block_size - 1);
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int n = first + i * AT_ONCE;
    const bool live = n < 2 * a.heads, is_k = n < a.heads;
    float v[8], amax = 0.0f;
    piece_f32<T, 8>(own[i], v);
    if (live && is_k && angles != nullptr) turn8<T>(v, row_at(n), d, a.r, angles, turns);
    bool nan = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      nan |= v[j] != v[j];
      amax = fmaxf(amax, fabsf(v[j]));
    }
    // Over the 32 elements of a key's scale, or over a value row.  (The lanes of keys go through the
    // values' steps with them; they keep what they had.)
    uint32_t odd = nan;
    if (__any_sync(0xffffffffu, amax == kInf)) amax = largest_finite(v, 0.0f);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, amax, o);
      const uint32_t z = __shfl_xor_sync(0xffffffffu, odd, o);
      if (o < 4 || !is_k) {
        amax = fmaxf(amax, y);
        odd |= z;
      }
    }
    if (!live) continue;
    const int64_t row = (s.page * a.heads + (is_k ? n : n - a.heads)) * a.block_size + in_page;
    if (is_k) {
      const int e = key_exponent(amax);
      const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= up;
      if ((lane & 3) == 0)
        a.k_scales[row * (D / 32) + d / 32] = odd ? 255 : static_cast<uint8_t>(e + 127);
    } else {
      // The codes of 6 v / amax; rows past 2^100 are brought down first.
      amax = fmaxf(amax, kLeastMax);
      const float down = amax > 1.2676506002282294e30f ? 5.421010862427522e-20f : 1.0f;  // 2^-64
      const float m = amax * down, inv = __frcp_rn(m);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = six_over<T>(fminf(fmaxf(v[j], -amax), amax) * down, m, inv);
      if (d == 0) a.v_scales[row] = odd ? __int_as_float(0x7FC00000) : __fdiv_rn(amax, 6.0f);
    }
    *reinterpret_cast<uint32_t *>((is_k ? a.k_pool : a.v_pool) + row * (D / 2) + d / 2) = e2m1x8(v);
  }
}

// 16 elements of a row: in stores of 32 bytes (wide), of 16, or one by one.
enum Store { kByOne, kInPieces, kWide };
template <typename T>
__device__ __forceinline__ void store16(T *out, const Piece<T, 8> (&p)[2], int how) {
  if (how == kWide) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + j * (32 / sizeof(T))),
                   "r"(w[8 * j]), "r"(w[8 * j + 1]), "r"(w[8 * j + 2]), "r"(w[8 * j + 3]), "r"(w[8 * j + 4]),
                   "r"(w[8 * j + 5]), "r"(w[8 * j + 6]), "r"(w[8 * j + 7])
                   : "memory");
  } else if (how == kInPieces) {
    store_piece<T, 8>(out, p[0]);
    store_piece<T, 8>(out + 8, p[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) out[j] = p[j >> 3].e[j & 7];
  }
}

// The rows back: a warp takes one token and ROUNDS times 512 / D of its 2 * heads rows (the keys, then the
// values), 16 elements a lane, all its loads before its first store.  34,000 tokens of 8 heads of 128
// (176 MB) take 31 us, 26 at the copy rate; one round a warp 36, two 34, eight 33 (eight elements
// a lane in 16-byte stores 37).
template <typename T, int D, int ROUNDS>
__global__ void __launch_bounds__(kThreads) k_kv4_read(const Kv4Args a, int how, bool clear) {
  constexpr int LANES = D / 16, AT_ONCE = 32 / LANES;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LANES;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.m.tokens) return;
  const int first = blockIdx.y * ROUNDS * AT_ONCE + lane / LANES;
  const Spot s = spot_of(a, t, lane);
  if (s.page < 0 && !clear) return;
  uint2 codes[ROUNDS];
  float scale[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    codes[i] = make_uint2(0, 0);
    scale[i] = 0.0f;
  }
  if (s.page >= 0) {
    const int64_t row0 = s.page * a.heads * a.block_size + (s.pos & (a.block_size - 1));
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int n = min(first + i * AT_ONCE, 2 * a.heads - 1);
      const bool is_k = n < a.heads;
      const int64_t row = row0 + (is_k ? n : n - a.heads) * a.block_size;
      codes[i] = *reinterpret_cast<const uint2 *>((is_k ? a.k_pool : a.v_pool) + row * (D / 2) + l * 8);
      scale[i] = is_k ? ue8m0(a.k_scales[row * (D / 32) + l / 2]) : a.v_scales[row];
    }
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int n = first + i * AT_ONCE;
    if (n >= 2 * a.heads) return;
    const bool is_k = n < a.heads;
    Piece<T, 8> p[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v[8];
      e2m1x8_to_f32(e ? codes[i].y : codes[i].x, v);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 f = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(scale[i], scale[i]));
        put_two<T>(p[e], j, f.x, f.y);
      }
    }
    store16<T>(static_cast<T *>(is_k ? a.k_out : a.v_out) + t * (is_k ? a.k_token : a.v_token) +
                   (is_k ? n * a.k_head : (n - a.heads) * a.v_head) + l * 16,
               p, how);
  }
}

// Rounds a warp: four of more than 16384 tokens and rounds, else one (a small call is one chain of latencies,
// which more warps shorten).  8 heads of 128, us with one and with four: 1024 tokens' append 3.6 and 3.7, read
// 2.7 and 3.0; 4096 8.0 and 7.3, 5.6 and 5.9; 8192 15.4 and 13.0, 9.4 and 7.6; 32768 59 and 45, 35 and 31 (by the
// general writer 5.6 and 7.1, 16.5 and 14.1, 32 and 26, 124 and 96).
inline bool many(const Kv4Args &a, int at_once) {
  return static_cast<int64_t>(a.m.tokens) * ((2 * a.heads + at_once - 1) / at_once) > 16384;
}
inline dim3 grid_of(const Kv4Args &a, int rows) {
  return dim3(static_cast<unsigned>((a.m.tokens + kWarps - 1) / kWarps),
              static_cast<unsigned>((2 * a.heads + rows - 1) / rows));
}

template <typename T, int D, bool ADJ>
cudaError_t append_pieces(const Kv4Args &a, cudaStream_t stream) {
  constexpr int AT_ONCE = 512 / D;
  const int rounds = 2 * ((a.heads + AT_ONCE - 1) / AT_ONCE);
  constexpr int WARPS = kPieceThreads / 32;
  const auto grid = [&](int each) {
    return dim3(static_cast<unsigned>((a.m.tokens + WARPS - 1) / WARPS),
                static_cast<unsigned>((rounds + each - 1) / each));
  };
  // (As with many(): a small call is one chain of latencies.)
  return static_cast<int64_t>(a.m.tokens) * rounds > 16384
             ? launch_dependent(k_kv4_append_pieces<T, D, ADJ, 4>, grid(4), dim3(kPieceThreads), 0, stream, a)
             : launch_dependent(k_kv4_append_pieces<T, D, ADJ, 1>, grid(1), dim3(kPieceThreads), 0, stream, a);
}

template <typename T, int D>
cudaError_t append(const Kv4Args &a, bool pieces, bool turns, cudaStream_t stream) {
  constexpr int AT_ONCE = 256 / D;
  // Where four lanes' pieces are a key's groups of 32 (see place_pieces).
  const bool adjacent = a.r.table != nullptr && a.r.interleaved;
  if (pieces && turns &&
      (a.r.table == nullptr || adjacent ||
       (a.r.offset % 32 == 0 && a.r.rot % 64 == 0 && (D - a.r.rot) % 64 == 0)))
    return adjacent ? append_pieces<T, D, true>(a, stream) : append_pieces<T, D, false>(a, stream);
  return many(a, AT_ONCE)
             ? launch_dependent(k_kv4_append<T, D, 4>, grid_of(a, 4 * AT_ONCE), dim3(kThreads), 0,
                                stream, a, pieces, turns)
             : launch_dependent(k_kv4_append<T, D, 1>, grid_of(a, AT_ONCE), dim3(kThreads), 0, stream,
                                a, pieces, turns);
}

template <typename T, int D>
cudaError_t read(const Kv4Args &a, int how, bool clear, cudaStream_t stream) {
  constexpr int AT_ONCE = 512 / D;
  return many(a, AT_ONCE) ? launch_dependent(k_kv4_read<T, D, 4>, grid_of(a, 4 * AT_ONCE),
                                             dim3(kThreads), 0, stream, a, how, clear)
                          : launch_dependent(k_kv4_read<T, D, 1>, grid_of(a, AT_ONCE), dim3(kThreads),
                                             0, stream, a, how, clear);
}

template <typename T>
cudaError_t append_dim(const Kv4Args &a, bool pieces, bool turns, cudaStream_t stream) {
  return a.dim == 64 ? append<T, 64>(a, pieces, turns, stream) : append<T, 128>(a, pieces, turns, stream);
}
template <typename T>
cudaError_t read_dim(const Kv4Args &a, int how, bool clear, cudaStream_t stream) {
  return a.dim == 64 ? read<T, 64>(a, how, clear, stream) : read<T, 128>(a, how, clear, stream);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args &a, int dtype, bool pieces, bool turns,
                              cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32: return append_dim<float>(a, pieces, turns, stream);
    case IDX_DTYPE_F16: return append_dim<__half>(a, pieces, turns, stream);
    default: return append_dim<__nv_bfloat16>(a, pieces, turns, stream);
  }
}

cudaError_t launch_kv4_read(const Kv4Args &a, int dtype, bool pieces, bool wide, bool clear,
                            cudaStream_t stream) {
  const int how = wide ? kWide : pieces ? kInPieces : kByOne;
  switch (dtype) {
    case IDX_DTYPE_F32: return read_dim<float>(a, how, clear, stream);
    case IDX_DTYPE_F16: return read_dim<__half>(a, how, clear, stream);
    default: return read_dim<__nv_bfloat16>(a, how, clear, stream);
  }
}

cudaError_t kv4_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_kv4_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_kv4_status, &zero, sizeof(int32_t));
}

}  // namespace idx
