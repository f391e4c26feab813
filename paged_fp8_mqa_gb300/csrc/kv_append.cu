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

// One item: a block of one head of K or of V.
template <typename T>
struct Item {
  const T *x;  // the first new token's row
  int64_t token;
  uint8_t *block;
  float *scale;
  bool turn;
};

template <typename T>
__device__ __forceinline__ Item<T> item_of(const AppendArgs &a, const Unit &u, int64_t page,
                                           int item, int dim) {
  Item<T> r;
  const int h = item >> 1;
  const bool is_k = (item & 1) == 0;
  r.token = is_k ? a.k_token : a.v_token;
  r.x = static_cast<const T *>(is_k ? a.k : a.v) + u.tok * r.token + h * (is_k ? a.k_head : a.v_head);
  const int64_t at = page * a.heads + h;
  r.block = (is_k ? a.k_pool : a.v_pool) + at * a.block_size * dim;
  r.scale = (is_k ? a.k_scales : a.v_scales) + at;
  r.turn = is_k && a.r.table != nullptr;
  return r;
}

// A token's row of an item in a warp (see kPieces).
template <typename T, int V, int D>
struct Row {
  static constexpr int N = kPieces<V, D>;
  Piece<T, V> own[N];

  __device__ __forceinline__ void load(const Item<T> &it, int tk, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      own[i] = load_piece<T, V>(it.x + tk * it.token + (lane + 32 * i) * V);
  }
  // In float32, turned.
  __device__ __forceinline__ void values(const AppendArgs &a, const Unit &u, const Item<T> &it, int tk,
                                         int lane, float (&v)[N][V]) const {
    const int pos = u.first + tk;
    const float2 *angles = it.turn && pos < a.r.max_positions
                               ? a.r.table + static_cast<int64_t>(pos) * (a.r.rot >> 1)
                               : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int d = (lane + 32 * i) * V;
      turned<T, V>(own[i], it.x + tk * it.token + d, turn_of<V>(a.r, angles, d), v[i]);
    }
  }
};

// The block's scale for new values of magnitude amax at most; where it grows, the tokens before
// off0 are rescaled by the GROUP threads.
template <int D, int GROUP>
__device__ __forceinline__ float settle_scale(uint8_t *block, float was, float amax, int off0,
                                              int tid) {
  float scale = block_scale(amax);
  if (off0 > 0 && !(scale > was)) scale = was;
  if (off0 > 0 && scale != was) {
    const float f = was / scale;
    uint32_t *p = reinterpret_cast<uint32_t *>(block);
    for (int i = tid; i < off0 * D / 4; i += GROUP) p[i] = rescale4(p[i], f);
  }
  return scale;
}

// The page of the request's block, or -1: nothing to do, or flagged.
__device__ __forceinline__ int page_of(const AppendArgs &a, const Unit &u) {
  if (u.count <= 0) return -1;
  int id = -1;
  if (u.j < a.m.bt_width) id = __ldg(a.m.block_tables + u.b * a.m.bt_stride + u.j);
  const bool good = id >= 0 && id < a.num_blocks && u.tok >= 0 && u.tok + u.count <= a.m.tokens;
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    if (!good)
      atomicOr(&g_append_status, IDX_DEV_BAD_PAGE);
    else if (a.r.table != nullptr && u.first + u.count > a.r.max_positions)
      atomicOr(&g_append_status, IDX_DEV_BAD_POSITION);
  }
  return good ? id : -1;
}

// Unit x of equal requests: each touches so many blocks at most.
__device__ __forceinline__ Unit equal_unit(const AppendArgs &a, int x) {
  const int per = (a.m.next_n - 1 + a.block_size - 1) / a.block_size + 1;
  const int b = x / per;
  const int len = __ldg(a.m.seq_lens + b * a.m.sl_stride);
  return unit_of(b, x - b * per, len - a.m.next_n, len, static_cast<int64_t>(b) * a.m.next_n,
                 a.block_size);
}

// A few new tokens a block (kFew at most): a warp an item, whose rows stay in registers between the
// largest magnitude and the writing.
constexpr int kFew = 4;

template <typename T, int V, int D>
__global__ void __launch_bounds__(kThreads) k_append_few(const AppendArgs a) {
  constexpr int N = kPieces<V, D>;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const Unit u = equal_unit(a, blockIdx.x);
  const int id = page_of(a, u);
  if (id < 0 || n >= 2 * a.heads) return;
  const Item<T> it = item_of<T>(a, u, id, n, D);
  const int off0 = u.first - u.j * a.block_size;
  const float was = off0 > 0 ? *it.scale : 0.0f;
  float v[kFew][N][V], amax = 0.0f;
#pragma unroll
  for (int tk = 0; tk < kFew; ++tk) {
    if (tk >= u.count) break;
    Row<T, V, D> row;
    row.load(it, tk, lane);
    row.values(a, u, it, tk, lane, v[tk]);
#pragma unroll
    for (int i = 0; i < N; ++i) amax = largest_finite(v[tk][i], amax);
  }
  amax = warp_max(amax);
  const float scale = settle_scale<D, 32>(it.block, was, amax, off0, lane);
  if (lane == 0) *it.scale = scale;
  const float inv = 1.0f / scale;  // exact: a power of two (or what another writer left)
#pragma unroll
  for (int tk = 0; tk < kFew; ++tk) {
    if (tk >= u.count) break;
#pragma unroll
    for (int i = 0; i < N; ++i)
      store_e4m3<V>(it.block + (off0 + tk) * D + (lane + 32 * i) * V, v[tk][i], inv);
  }
}

// Runs of tokens: a CTA takes one request's block (of 8 * HELD tokens) and, of its 2 * heads items,
// every gridDim.y-th; a warp every eighth token, HELD at most.  All its rows are asked for at once
// (a token past the block's last new one is read as that one: a branch would keep the loads apart),
// and stay in registers between the largest magnitude and the writing.
//
// 217 MB of prompts take 89 us (floor 32): an item is a chain of a search, loads, a barrier and
// stores, of which four CTAs an SM overlap.  With the rows behind branches it was 114 us, with
// 16-byte pieces read twice 98, with one, two or eight items a CTA 112, 93 and 93 (four: 89).
template <typename T, int V, int D, int HELD>
__global__ void __launch_bounds__(kThreads, HELD <= 8 ? 4 : 2) k_append_run(const AppendArgs a) {
  constexpr int N = kPieces<V, D>;
  __shared__ int s_warp[kWarps];
  __shared__ float s_max[2][kWarps];
  __shared__ Unit s_unit;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, items = 2 * a.heads;
  const Unit u = a.m.starts == nullptr ? equal_unit(a, blockIdx.x)
                                       : find_unit(a.m, blockIdx.x, a.block_size, s_warp, &s_unit);
  const int id = page_of(a, u);
  if (id < 0) return;
  const int off0 = u.first - u.j * a.block_size;
  int set = 0;  // (two sets of maxima: a fast warp may be an item ahead)
  for (int n = blockIdx.y; n < items; n += gridDim.y, set ^= 1) {
    const Item<T> it = item_of<T>(a, u, id, n, D);
    const float was = off0 > 0 ? *it.scale : 0.0f;
    Row<T, V, D> row[HELD];
#pragma unroll
    for (int p = 0; p < HELD; ++p) row[p].load(it, min(warp + p * kWarps, u.count - 1), lane);
    float v[HELD][N][V], amax = 0.0f;
#pragma unroll
    for (int p = 0; p < HELD; ++p) {
      row[p].values(a, u, it, min(warp + p * kWarps, u.count - 1), lane, v[p]);
#pragma unroll
      for (int i = 0; i < N; ++i) amax = largest(v[p][i], amax);
    }
    if (is_inf(amax)) {
      amax = 0.0f;
#pragma unroll
      for (int p = 0; p < HELD; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) amax = largest_finite(v[p][i], amax);
    }
    amax = warp_max(amax);
    if (lane == 0) s_max[set][warp] = amax;
    __syncthreads();  // (also: every thread has read the old scale)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, s_max[set][w]);
    const float scale = settle_scale<D, kThreads>(it.block, was, amax, off0, tid);
    if (tid == 0) *it.scale = scale;
    const float inv = 1.0f / scale;  // exact: a power of two (or what another writer left)
#pragma unroll
    for (int p = 0; p < HELD; ++p) {
      const int tk = warp + p * kWarps;
      if (tk < u.count) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          store_e4m3<V>(it.block + (off0 + tk) * D + (lane + 32 * i) * V, v[p][i], inv);
      }
    }
  }
}

template <typename T, int V, int D>
cudaError_t launch_dim(const AppendArgs &a, cudaStream_t stream) {
  const int64_t bs = a.block_size;
  const int items = 2 * a.heads;
  int64_t units = a.m.batch * ((a.m.next_n - 1 + bs - 1) / bs + 1);
  if (a.m.starts == nullptr && a.m.next_n <= kFew)
    return launch_dependent(k_append_few<T, V, D>,
                            dim3(static_cast<unsigned>(units), (items + kWarps - 1) / kWarps),
                            dim3(kThreads), 0, stream, a);
  if (a.m.starts != nullptr) {
    // Every request touches at most (its tokens) / bs + 2 blocks, and no more than its tokens.
    units = a.m.tokens / bs + 2 * static_cast<int64_t>(a.m.batch);
    if (units > a.m.tokens) units = a.m.tokens;
  }
  // An item a CTA, until there are some thousands of CTAs; then several, one after the other, which
  // share the search for their block.
  int y = items;
  while (y % 2 == 0 && units * y > 4096) y /= 2;
  const dim3 grid(static_cast<unsigned>(units), y);
  switch (a.block_size) {
    case 32: return launch_dependent(k_append_run<T, V, D, 4>, grid, dim3(kThreads), 0, stream, a);
    case 64: return launch_dependent(k_append_run<T, V, D, 8>, grid, dim3(kThreads), 0, stream, a);
    default: return launch_dependent(k_append_run<T, V, D, 16>, grid, dim3(kThreads), 0, stream, a);
  }
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

cudaError_t launch_kv_append(const AppendArgs &a, int dtype, bool pairs, cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32:
      return pairs ? launch<float, 2>(a, stream) : launch<float, 1>(a, stream);
    case IDX_DTYPE_F16:
      return pairs ? launch<__half, 2>(a, stream) : launch<__half, 1>(a, stream);
    default:
      return pairs ? launch<__nv_bfloat16, 2>(a, stream) : launch<__nv_bfloat16, 1>(a, stream);
  }
}

cudaError_t append_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_append_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_append_status, &zero, sizeof(int32_t));
}

}  // namespace idx
