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
#include "ptx.cuh"
#include "rows.cuh"

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

template <typename T>
__device__ __forceinline__ Piece<T, 8> load8(const T *p, bool whole) {
  if (whole) return load_piece<T, 8>(p);
  Piece<T, 8> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.e[j] = p[j];
  return v;
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

// A warp takes one token and ROUNDS times 32 * 8 / D of its 2 * heads rows (the keys, then the values),
// eight elements a lane; all its rows are asked for at once, before the token's place is known.
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
    own[i] = load8<T>(row_at(min(first + i * AT_ONCE, 2 * a.heads - 1)) + d, pieces);
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
      // The codes of 6 v / amax, correctly rounded (the remainder times the reciprocal), so that what
      // lies halfway between two codes stays there; rows past 2^100 are brought down first.
      amax = fmaxf(amax, kLeastMax);
      const float down = amax > 1.2676506002282294e30f ? 5.421010862427522e-20f : 1.0f;  // 2^-64
      const float m = amax * down, inv = __frcp_rn(m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = 6.0f * (fminf(fmaxf(v[j], -amax), amax) * down);
        const float q = x * inv;
        v[j] = fmaf(fmaf(-q, m, x), inv, q);
      }
      if (d == 0) a.v_scales[row] = odd ? __int_as_float(0x7FC00000) : __fdiv_rn(amax, 6.0f);
    }
    *reinterpret_cast<uint32_t *>((is_k ? a.k_pool : a.v_pool) + row * (D / 2) + d / 2) = e2m1x8(v);
  }
}

// The rows back: a warp's token and rows as above.
template <typename T, int D, int ROUNDS>
__global__ void __launch_bounds__(kThreads) k_kv4_read(const Kv4Args a, bool pieces, bool clear) {
  constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.m.tokens) return;
  const int first = blockIdx.y * ROUNDS * AT_ONCE + lane / LANES, d = (lane % LANES) * 8;
  const Spot s = spot_of(a, t, lane);
  if (s.page < 0 && !clear) return;
  const int in_page = s.pos & (a.block_size - 1);
  uint32_t codes[ROUNDS];
  float scale[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int n = min(first + i * AT_ONCE, 2 * a.heads - 1);
    const bool is_k = n < a.heads;
    codes[i] = 0;
    scale[i] = 0.0f;
    if (s.page < 0) continue;
    const int64_t row = (s.page * a.heads + (is_k ? n : n - a.heads)) * a.block_size + in_page;
    codes[i] = *reinterpret_cast<const uint32_t *>((is_k ? a.k_pool : a.v_pool) + row * (D / 2) + d / 2);
    scale[i] = is_k ? ue8m0(a.k_scales[row * (D / 32) + d / 32]) : a.v_scales[row];
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int n = first + i * AT_ONCE;
    if (n >= 2 * a.heads) return;
    const bool is_k = n < a.heads;
    float v[8];
    e2m1x8_to_f32(codes[i], v);
    Piece<T, 8> p;
#pragma unroll
    for (int j = 0; j < 8; ++j) p.e[j] = from_f32<T>(v[j] * scale[i]);
    T *out = static_cast<T *>(is_k ? a.k_out : a.v_out) + t * (is_k ? a.k_token : a.v_token) +
             (is_k ? n * a.k_head : (n - a.heads) * a.v_head) + d;
    if (pieces) {
      store_piece<T, 8>(out, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = p.e[j];
    }
  }
}

// Rounds a warp: four while that leaves some thousands of warps, else one (a small call is one chain of
// latencies, which more warps shorten).
inline bool many(const Kv4Args &a, int at_once) {
  return static_cast<int64_t>(a.m.tokens) * ((2 * a.heads + at_once - 1) / at_once) > 16384;
}
inline dim3 grid_of(const Kv4Args &a, int rows) {
  return dim3(static_cast<unsigned>((a.m.tokens + kWarps - 1) / kWarps),
              static_cast<unsigned>((2 * a.heads + rows - 1) / rows));
}

template <typename T, int D>
cudaError_t append(const Kv4Args &a, bool pieces, bool turns, cudaStream_t stream) {
  constexpr int AT_ONCE = 256 / D;
  return many(a, AT_ONCE)
             ? launch_dependent(k_kv4_append<T, D, 4>, grid_of(a, 4 * AT_ONCE), dim3(kThreads), 0,
                                stream, a, pieces, turns)
             : launch_dependent(k_kv4_append<T, D, 1>, grid_of(a, AT_ONCE), dim3(kThreads), 0, stream,
                                a, pieces, turns);
}

template <typename T, int D>
cudaError_t read(const Kv4Args &a, bool pieces, bool clear, cudaStream_t stream) {
  constexpr int AT_ONCE = 256 / D;
  return many(a, AT_ONCE) ? launch_dependent(k_kv4_read<T, D, 4>, grid_of(a, 4 * AT_ONCE),
                                             dim3(kThreads), 0, stream, a, pieces, clear)
                          : launch_dependent(k_kv4_read<T, D, 1>, grid_of(a, AT_ONCE), dim3(kThreads),
                                             0, stream, a, pieces, clear);
}

template <typename T>
cudaError_t append_dim(const Kv4Args &a, bool pieces, bool turns, cudaStream_t stream) {
  return a.dim == 64 ? append<T, 64>(a, pieces, turns, stream) : append<T, 128>(a, pieces, turns, stream);
}
template <typename T>
cudaError_t read_dim(const Kv4Args &a, bool pieces, bool clear, cudaStream_t stream) {
  return a.dim == 64 ? read<T, 64>(a, pieces, clear, stream) : read<T, 128>(a, pieces, clear, stream);
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

cudaError_t launch_kv4_read(const Kv4Args &a, int dtype, bool pieces, bool clear,
                            cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32: return read_dim<float>(a, pieces, clear, stream);
    case IDX_DTYPE_F16: return read_dim<__half>(a, pieces, clear, stream);
    default: return read_dim<__nv_bfloat16>(a, pieces, clear, stream);
  }
}

cudaError_t kv4_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_kv4_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_kv4_status, &zero, sizeof(int32_t));
}

}  // namespace idx
