// kv_append.cu -- new keys (rotated) and values into the 8-bit K/V cache: e4m3 values with one
// float32 scale for each block of tokens and head.
//
// The scale of a block is the least power of two that brings the largest magnitude of what it
// holds to at most 448.  A block that already holds tokens keeps its scale while the new ones
// fit it; otherwise the scale grows and what is there is multiplied by old / new and rounded
// again.  Between powers of two that product only moves the exponent, so it is exact for every
// value that does not become subnormal, and a block that is filled token by token does not wear
// its values down by growing; e4m3 being a floating type, a scale up to twice the least costs the
// new values no precision above its subnormals either.

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace idx {

__device__ int g_append_status;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The least power of two, 2^-100 or more, that brings amax (finite, >= 0) to at most 448 =
// 1.75 * 2^8: read off amax's exponent and mantissa, without a rounding.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8;
  if ((u & 0x7FFFFFu) > 0x600000u) ++e;
  e = max(e, -100);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Block j of request b, and the new tokens it receives.
struct Unit {
  int b, j;
  int first;    // position of the first new token in it
  int count;    // 0: nothing to do
  int64_t tok;  // that token's row
};

// Positions [begin, len) of request b are new; unit u of the request is its u-th touched block.
__device__ __forceinline__ Unit unit_of(int b, int u, int begin, int len, int64_t tok0, int bs) {
  Unit r;
  const int from = max(begin, 0);
  r.b = b;
  r.j = from / bs + u;
  r.first = max(from, r.j * bs);
  r.count = max(0, min(len, (r.j + 1) * bs) - r.first);
  r.tok = tok0 + (r.first - begin);
  return r;
}

__device__ __forceinline__ int touched(int begin, int len, int bs) {
  const int from = max(begin, 0);
  return len > from ? (len - 1) / bs - from / bs + 1 : 0;
}

// The unit of CTA `u` among all requests' touched blocks, request by request; count 0 past the
// last.  Every CTA scans the lengths itself: one round trip and a block scan, instead of a launch.
__device__ Unit find_unit(const TokenMap &m, int u, int bs, int *s_warp, Unit *s_unit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (m.batch + kThreads - 1) / kThreads;
  const int lo = min(tid * per, m.batch), hi = min(lo + per, m.batch);
  int mine = 0;
  for (int b = lo; b < hi; ++b) {
    const int len = __ldg(m.seq_lens + b * m.sl_stride);
    const int n = __ldg(m.starts + b + 1) - __ldg(m.starts + b);
    mine += touched(len - n, len, bs);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid == 0) s_unit->count = 0;
  __syncthreads();
  int at = incl - mine;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  if (u >= at && u < at + mine) {
    for (int b = lo; b < hi; ++b) {
      const int len = __ldg(m.seq_lens + b * m.sl_stride);
      const int s = __ldg(m.starts + b);
      const int n = __ldg(m.starts + b + 1) - s;
      const int k = touched(len - n, len, bs);
      if (u < at + k) {
        *s_unit = unit_of(b, u - at, len - n, len, s, bs);
        break;
      }
      at += k;
    }
  }
  __syncthreads();
  return *s_unit;
}

__device__ __forceinline__ uint32_t rescale4(uint32_t four, float f) {
  const float2 lo = e4m3x2_to_f32(four), hi = e4m3x2_to_f32(four >> 16);
  return e4m3x4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}

// Elements [d, d + V) of the row at `x`, read as `own`, rotated by the angles at `cs` (one per
// pair; nullptr: as they are), in float32.  With V > 1 the caller has checked that offset, rot / 2
// and d are multiples of V.
template <typename T, int V>
__device__ __forceinline__ void turned_piece(const Piece<T, V> &own, const T *x, int d, const Rotation &r,
                                       const float2 *cs, float (&out)[V]) {
  piece_f32<T, V>(own, out);
  const int i = d - r.offset;
  if (cs == nullptr || i < 0 || i >= r.rot) return;
  if (r.interleaved) {
    if constexpr (V == 1) {
      const float2 c = cs[i >> 1];
      const float other = to_f32(x[(i & 1) ? d - 1 : d + 1]);
      out[0] = (i & 1) ? turn_b(other, out[0], c) : turn_a(out[0], other, c);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 c = cs[(i >> 1) + j];
        const float a = out[2 * j], b = out[2 * j + 1];
        out[2 * j] = turn_a(a, b, c);
        out[2 * j + 1] = turn_b(a, b, c);
      }
    }
    return;
  }
  const int half = r.rot >> 1;
  const bool first = i < half;
  float other[V];
  piece_f32<T, V>(load_piece<T, V>(x + (first ? d + half : d - half)), other);
  const float2 *c = cs + (first ? i : i - half);
  // own cos - other sin for the pair's first element, own cos + other sin for its second.
#pragma unroll
  for (int j = 0; j < V; ++j) out[j] = turn_b(first ? -other[j] : other[j], out[j], c[j]);
}

// One item: a block of one head of K or of V.  GROUP = 32: a warp of its own (a few new tokens);
// GROUP = kThreads: the whole CTA (long runs of tokens).  The new tokens are read once for the
// largest magnitude and, from L1, once more to be written.
template <typename T, int V, int D, int GROUP>
__device__ __forceinline__ void append_item(const AppendArgs &a, const Unit &u, int64_t page, int h,
                                            bool is_k, float *s_max) {
  const int tid = GROUP == 32 ? threadIdx.x & 31 : threadIdx.x;
  constexpr int kPer = D / V;  // pieces of a row
  const int64_t token = is_k ? a.k_token : a.v_token, head = is_k ? a.k_head : a.v_head;
  const T *x = static_cast<const T *>(is_k ? a.k : a.v) + u.tok * token + h * head;
  const int64_t at = page * a.heads + h;
  uint8_t *block = (is_k ? a.k_pool : a.v_pool) + at * a.block_size * D;
  float *scale_at = (is_k ? a.k_scales : a.v_scales) + at;
  const int off0 = u.first - u.j * a.block_size;
  const float was = off0 > 0 ? *scale_at : 0.0f;
  const bool turn = is_k && a.r.table != nullptr;
  const auto row = [&](int i) -> const float2 * {
    const int pos = u.first + i;
    if (!turn || pos >= a.r.max_positions) return nullptr;
    return a.r.table + static_cast<int64_t>(pos) * (a.r.rot >> 1);
  };
  if (turn && h == 0 && tid == 0 && u.first + u.count > a.r.max_positions)
    atomicOr(&g_append_status, IDX_DEV_BAD_POSITION);
  float amax = 0.0f;
  const int n = u.count * kPer;
#pragma unroll 4
  for (int i = tid; i < n; i += GROUP) {
    float v[V];
    const int tk = i / kPer, d = (i % kPer) * V;
    turned_piece<T, V>(load_piece<T, V>(x + tk * token + d), x + tk * token, d, a.r, row(tk), v);
    amax = largest_finite(v, amax);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if constexpr (GROUP != 32) {
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();  // (also: every thread has read the old scale)
#pragma unroll
    for (int w = 0; w < GROUP / 32; ++w) amax = fmaxf(amax, s_max[w]);
  } else {
    __syncwarp();
  }
  float scale = block_scale(amax);
  if (off0 > 0 && !(scale > was)) scale = was;
  if (off0 > 0 && scale != was) {
    const float f = was / scale;
    uint32_t *p = reinterpret_cast<uint32_t *>(block);
    for (int i = tid; i < off0 * D / 4; i += GROUP) p[i] = rescale4(p[i], f);
  }
  if (tid == 0) *scale_at = scale;
  const float inv = 1.0f / scale;  // exact: scale is a power of two (or what another writer left)
#pragma unroll 4
  for (int i = tid; i < n; i += GROUP) {
    float v[V];
    const int tk = i / kPer, d = (i % kPer) * V;
    turned_piece<T, V>(load_piece<T, V>(x + tk * token + d), x + tk * token, d, a.r, row(tk), v);
    store_e4m3<V>(block + (off0 + tk) * D + d, v, inv);
  }
}

template <typename T, int V, int D, int GROUP>
__global__ void __launch_bounds__(kThreads) k_kv_append(const AppendArgs a) {
  __shared__ int s_warp[kWarps];
  __shared__ float s_max[2][kWarps];
  __shared__ Unit s_unit;
  griddep_wait();
  griddep_launch_dependents();
  Unit u;
  if (a.m.starts == nullptr) {
    // Two units at most of a request whose next_n tokens are no more than a block.
    const int per = (a.m.next_n - 1 + a.block_size - 1) / a.block_size + 1;
    const int b = blockIdx.x / per;
    const int len = __ldg(a.m.seq_lens + b * a.m.sl_stride);
    u = unit_of(b, blockIdx.x - b * per, len - a.m.next_n, len,
                static_cast<int64_t>(b) * a.m.next_n, a.block_size);
  } else {
    u = find_unit(a.m, blockIdx.x, a.block_size, s_warp, &s_unit);
  }
  if (u.count <= 0) return;
  int id = -1;
  if (u.j < a.m.bt_width) id = __ldg(a.m.block_tables + u.b * a.m.bt_stride + u.j);
  if (id < 0 || id >= a.num_blocks || u.tok < 0 || u.tok + u.count > a.m.tokens) {
    if (threadIdx.x == 0) atomicOr(&g_append_status, IDX_DEV_BAD_PAGE);
    return;
  }
  const int warps = GROUP == 32 ? kWarps : 1;
  int set = 0;  // (two sets of maxima: a fast warp may be an item ahead)
  for (int item = blockIdx.y * warps + (GROUP == 32 ? threadIdx.x >> 5 : 0); item < 2 * a.heads;
       item += gridDim.y * warps, set ^= 1)
    append_item<T, V, D, GROUP>(a, u, id, item >> 1, (item & 1) == 0, s_max[set]);
}

template <typename T, int V, int D>
cudaError_t launch_dim(const AppendArgs &a, cudaStream_t stream) {
  const int64_t bs = a.block_size;
  if (a.m.starts == nullptr) {
    const int64_t units = a.m.batch * ((a.m.next_n - 1 + bs - 1) / bs + 1);
    // A draft's few tokens occupy a warp an item; runs of 16 tokens and more the CTA.
    if (a.m.next_n < 16)
      return launch_dependent(k_kv_append<T, V, D, 32>,
                              dim3(static_cast<unsigned>(units), (2 * a.heads + kWarps - 1) / kWarps),
                              dim3(kThreads), 0, stream, a);
    return launch_dependent(k_kv_append<T, V, D, kThreads>,
                            dim3(static_cast<unsigned>(units), 2 * a.heads), dim3(kThreads), 0,
                            stream, a);
  }
  // Every request touches at most (its tokens) / bs + 2 blocks, and no more than its tokens.
  const int64_t most = a.m.tokens / bs + 2 * static_cast<int64_t>(a.m.batch);
  const int64_t units = most < a.m.tokens ? most : a.m.tokens;
  // An item a CTA, until there are some thousands of CTAs; then several, one after the other, which
  // share the search for their block.
  int y = 2 * a.heads;
  while (y % 2 == 0 && units * y > 4096) y /= 2;
  return launch_dependent(k_kv_append<T, V, D, kThreads>, dim3(static_cast<unsigned>(units), y),
                          dim3(kThreads), 0, stream, a);
}

template <typename T, int V>
cudaError_t launch(const AppendArgs &a, cudaStream_t stream) {
  switch (a.dim) {
    case 64: return launch_dim<T, V, 64>(a, stream);
    case 128: return launch_dim<T, V, 128>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, int dtype, bool vectors, cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32:
      return vectors ? launch<float, 4>(a, stream) : launch<float, 1>(a, stream);
    case IDX_DTYPE_F16:
      return vectors ? launch<__half, 8>(a, stream) : launch<__half, 1>(a, stream);
    default:
      return vectors ? launch<__nv_bfloat16, 8>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
  }
}

cudaError_t append_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_append_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_append_status, &zero, sizeof(int32_t));
}

}  // namespace idx
