// heads.cu -- the heads of queries and keys, normalised and rotated in one pass, and their gradients:
//   r = 1 / sqrt(mean(x^2) + eps),  y = R(x r w),
//   g = R^T dy,  dw = sum over tokens and heads of g x r,  dx = r (g w - x r^2 mean(g w x)),
// with R the rotation of the head's pairs, each by the position on its own axis (time, height, width).
// Without a norm it is the rotation alone.  One rounding, when y or dx is stored.
//
// Memory bounds it: x in and y out (dy, x in and dx out).  What is the same for all heads of a token, the
// angles and the weight, stays in a lane's registers while it walks several heads: a lane holds two pieces
// of eight elements of a head, chosen so that both elements of a pair are its own, and a head's sums
// are a few shuffles.

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace idx {

__device__ int g_heads_status;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = IDX_NORM_MAX_DIM;

__device__ __forceinline__ int axis_of(const Axes &x, int pair) {
  return x.count == 1 ? 0 : (x.axis[pair >> 4] >> (2 * (pair & 15))) & 3;
}

// The angles of one pair of token t, or false: its position is not in the table.
__device__ __forceinline__ bool angle_of(const HeadsArgs &a, int64_t t, int pair, float2 *cs) {
  const int pos = __ldg(a.positions + axis_of(a.axes, pair) * a.axes.stride + t);
  if (static_cast<uint32_t>(pos) >= static_cast<uint32_t>(a.r.max_positions)) return false;
  *cs = __ldg(a.r.table + static_cast<int64_t>(pos) * (a.r.rot >> 1) + pair);
  cs->y *= a.sin_sign;
  return true;
}

// 1 / sqrt(v): the approximation and one step of Newton's method (where v is a positive number).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v > 1e-37f && v < 1e37f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

// A lane's two pieces of a head of D = 16 * (lanes at work) elements, and how they are turned.
struct Pieces {
  int at[2];        // their first elements
  bool on[2];       // rotated
  bool across;      // halves: element j of the first with element j of the second; else within each
  float2 cs[8];     // the angles of the lane's pairs
  uint32_t valid;   // bit j: pair j's position is in the table
};

// Where lane l's pieces lie (which does not depend on the token), and the pairs of their angles 0 and 4.
__device__ __forceinline__ void place_pieces(const Rotation &r, int l, Pieces &p, int (&pair)[2]) {
  const int off = r.offset, rot = r.table != nullptr ? r.rot : 0;
  p.across = !r.interleaved;
  if (r.interleaved) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      p.at[s] = 16 * l + 8 * s;
      p.on[s] = p.at[s] >= off && p.at[s] < off + rot;
      pair[s] = (p.at[s] - off) >> 1;
    }
  } else if (l < rot / 16) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      p.at[s] = off + 8 * l + s * (rot >> 1);
      p.on[s] = true;
      pair[s] = 8 * l + 4 * s;
    }
  } else {  // what is not rotated, piece after piece
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int e = 16 * l - rot + 8 * s;
      p.at[s] = e < off ? e : e + rot;
      p.on[s] = false;
      pair[s] = 0;
    }
  }
}

__device__ __forceinline__ Pieces pieces_of(const HeadsArgs &a, int64_t t, int l) {
  Pieces p;
  const int half = a.r.rot >> 1;
  int pair[2];
  place_pieces(a.r, l, p, pair);
  p.valid = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) p.cs[j] = make_float2(1.0f, 0.0f);
  if (!p.on[0] && !p.on[1]) return p;
  if (a.axes.count == 1) {
    const int pos = __ldg(a.positions + t);
    if (static_cast<uint32_t>(pos) >= static_cast<uint32_t>(a.r.max_positions)) return p;
    const float2 *row = a.r.table + static_cast<int64_t>(pos) * half;
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (p.on[s]) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const float4 two = __ldg(reinterpret_cast<const float4 *>(row + pair[s] + j));
          p.cs[4 * s + j] = make_float2(two.x, two.y * a.sin_sign);
          p.cs[4 * s + j + 1] = make_float2(two.z, two.w * a.sin_sign);
        }
        p.valid |= 0xFu << (4 * s);
      }
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (p.on[s]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (angle_of(a, t, pair[s] + j, &p.cs[4 * s + j])) p.valid |= 1u << (4 * s + j);
      }
  }
  return p;
}

// v, the lane's 16 elements, turned.  A pair that is not turned stays to the bit (a product with a
// sine of 0 would make an infinity's partner NaN).
__device__ __forceinline__ void turn(const Pieces &p, float (&v)[2][8]) {
  if (p.across) {
    if (p.valid == 0xFFu) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[0][j], y = v[1][j];
        v[0][j] = turn_a(x, y, p.cs[j]);
        v[1][j] = turn_b(x, y, p.cs[j]);
      }
    } else if (p.valid != 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[0][j], y = v[1][j];
        const bool go = (p.valid >> j) & 1u;
        v[0][j] = go ? turn_a(x, y, p.cs[j]) : x;
        v[1][j] = go ? turn_b(x, y, p.cs[j]) : y;
      }
    }
  } else if (p.valid != 0) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = v[s][2 * j], y = v[s][2 * j + 1];
        const bool go = (p.valid >> (4 * s + j)) & 1u;
        v[s][2 * j] = go ? turn_a(x, y, p.cs[4 * s + j]) : x;
        v[s][2 * j + 1] = go ? turn_b(x, y, p.cs[4 * s + j]) : y;
      }
  }
}

// The lane's 16 weights in float32 (1 without).
template <typename T>
__device__ __forceinline__ void weights_of(const HeadsArgs &a, int kind, const Pieces &p,
                                           float (&w)[2][8]) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[s][j] = a.weight[kind] == nullptr ? 1.0f
                : a.weight_f32 ? __ldg(static_cast<const float *>(a.weight[kind]) + p.at[s] + j)
                               : to_f32(static_cast<const T *>(a.weight[kind])[p.at[s] + j]);
}

template <int W>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int o = 1; o < W; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// W lanes (a power of two, 16 elements a lane; those past dim idle) walk HEADS heads of one token, of q
// or of k, all of them asked for at once.
template <typename T, int W, int HEADS>
__global__ void __launch_bounds__(kThreads) k_heads(const __grid_constant__ HeadsArgs a,
                                                    int64_t first_token) {
  griddep_wait();
  griddep_launch_dependents();
  const int chunks_q = (a.heads[0] + HEADS - 1) / HEADS;
  const int chunks = chunks_q + (a.heads[1] + HEADS - 1) / HEADS;
  const uint32_t id = blockIdx.x * (kThreads / W) + threadIdx.x / W;
  const uint32_t tok = id / chunks;
  const int64_t t = first_token + tok;
  // (Past the last token or element: the last, and nothing is stored, so that the shuffles find all
  // their lanes.)
  const int lanes = a.dim / 16;
  const bool live = t < a.tokens && static_cast<int>(threadIdx.x % W) < lanes;
  const int64_t tt = min(t, a.tokens - 1);
  const int l = min(static_cast<int>(threadIdx.x % W), lanes - 1);
  int chunk = id - tok * chunks;
  const int kind = chunk >= chunks_q;
  if (kind) chunk -= chunks_q;
  const int h0 = chunk * HEADS, n = min(HEADS, a.heads[kind] - h0);
  const T *x = static_cast<const T *>(a.x[kind]) + tt * a.x_token[kind] + h0 * a.x_head[kind];
  T *out = static_cast<T *>(a.out[kind]) + tt * a.out_token[kind] + h0 * a.out_head[kind];
  const Pieces p = pieces_of(a, tt, l);
  Piece<T, 8> own[HEADS][2];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
#pragma unroll
    for (int s = 0; s < 2; ++s)
      own[h][s] = load_piece<T, 8>(x + min(h, n - 1) * a.x_head[kind] + p.at[s]);
  if (live && h0 == 0 && kind == (a.heads[0] == 0) &&
      p.valid != ((p.on[0] ? 0x0Fu : 0u) | (p.on[1] ? 0xF0u : 0u)))
    atomicOr(&g_heads_status, IDX_DEV_BAD_POSITION);
  float w[2][8];
  if (a.norm) weights_of<T>(a, kind, p, w);
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float v[2][8];
#pragma unroll
    for (int s = 0; s < 2; ++s) piece_f32<T, 8>(own[h][s], v[s]);
    if (a.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[s][j], v[s][j], ss);
      if (static_cast<int>(threadIdx.x % W) >= lanes) ss = 0.0f;
      const float r = inv_sqrt(sum_lanes<W>(ss) / static_cast<float>(a.dim) + a.eps);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[s][j] = v[s][j] * r * w[s][j];
    }
    const bool untouched = !a.norm && p.valid == 0;
    if (!untouched) {
      turn(p, v);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) own[h][s].e[j] = from_f32<T>(v[s][j]);
    }
    if (live && h < n)
#pragma unroll
      for (int s = 0; s < 2; ++s) store_piece<T, 8>(out + h * a.out_head[kind] + p.at[s], own[h][s]);
  }
}

// Any strides, alignments and sizes: a warp a head, in shared memory.
constexpr int kAnyWarps = 4;

template <typename T>
__device__ __forceinline__ float weight_at(const HeadsArgs &a, int kind, int d) {
  if (a.weight[kind] == nullptr) return 1.0f;
  return a.weight_f32 ? static_cast<const float *>(a.weight[kind])[d]
                      : to_f32(static_cast<const T *>(a.weight[kind])[d]);
}

// The elements of pair i.
__device__ __forceinline__ int2 pair_at(const Rotation &r, int i) {
  return r.interleaved ? make_int2(r.offset + 2 * i, r.offset + 2 * i + 1)
                       : make_int2(r.offset + i, r.offset + (r.rot >> 1) + i);
}

template <typename T>
__global__ void __launch_bounds__(32 * kAnyWarps) k_heads_any(const __grid_constant__ HeadsArgs a) {
  __shared__ float s_row[kAnyWarps][kMaxDim];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *row = s_row[warp];
  const int all = a.heads[0] + a.heads[1];
  const int64_t rows = a.tokens * all;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAnyWarps + warp; i < rows;
       i += static_cast<int64_t>(gridDim.x) * kAnyWarps) {
    const int64_t t = i / all;
    int h = static_cast<int>(i - t * all);
    const int kind = h >= a.heads[0];
    if (kind) h -= a.heads[0];
    const T *x = static_cast<const T *>(a.x[kind]) + t * a.x_token[kind] + h * a.x_head[kind];
    T *out = static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h * a.out_head[kind];
    float ss = 0.0f;
    for (int d = lane; d < a.dim; d += 32) {
      const float f = to_f32(x[d]);
      row[d] = f;
      ss = fmaf(f, f, ss);
    }
    if (a.norm) {
      const float r = inv_sqrt(sum_lanes<32>(ss) / static_cast<float>(a.dim) + a.eps);
      for (int d = lane; d < a.dim; d += 32) row[d] = row[d] * r * weight_at<T>(a, kind, d);
    }
    __syncwarp();
    if (a.r.table != nullptr) {
      for (int j = lane; j < a.r.rot / 2; j += 32) {
        float2 cs;
        if (!angle_of(a, t, j, &cs)) {
          atomicOr(&g_heads_status, IDX_DEV_BAD_POSITION);
          continue;
        }
        const int2 at = pair_at(a.r, j);
        const float u = row[at.x], v = row[at.y];
        row[at.x] = turn_a(u, v, cs);
        row[at.y] = turn_b(u, v, cs);
      }
      __syncwarp();
    }
    for (int d = lane; d < a.dim; d += 32) out[d] = from_f32<T>(row[d]);
    __syncwarp();
  }
}

// The gradients: blocks y = 0 take q's heads, y = 1 k's, W lanes a head, two heads of a token at a
// time.  A lane's 16 elements of the weight's gradient stay in its registers over all its heads; a block
// leaves its sums in the workspace and a second launch adds the blocks', in order.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) k_heads_backward(const __grid_constant__ HeadsArgs a) {
  constexpr int GROUPS = kThreads / W;
  extern __shared__ float s_sum[];  // [GROUPS][16 * W]
  griddep_wait();
  griddep_launch_dependents();
  const int kind = blockIdx.y, heads = a.heads[kind], lanes = a.dim / 16;
  const int group = threadIdx.x / W, lw = threadIdx.x % W, l = min(lw, lanes - 1);
  const bool live_lane = lw < lanes;
  constexpr int HEADS = 2;
  const int chunks = (heads + HEADS - 1) / HEADS;
  const int64_t items = a.tokens * chunks;
  float dw[2][8];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[s][j] = 0.0f;
  float w[2][8];
  bool first = true;
  // All groups of a warp make the same number of rounds.
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * GROUPS; i0 < items; i0 += step) {
    const int64_t i = i0 + group;
    const bool live = i < items;
    const int64_t at = min(i, items - 1);
    const int64_t t = at / chunks;
    const int h0 = static_cast<int>(at - t * chunks) * HEADS, n = min(HEADS, heads - h0);
    const T *x = static_cast<const T *>(a.x[kind]) + t * a.x_token[kind] + h0 * a.x_head[kind];
    const T *dy = static_cast<const T *>(a.dy[kind]) + t * a.dy_token[kind] + h0 * a.dy_head[kind];
    T *out = static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h0 * a.out_head[kind];
    const Pieces p = pieces_of(a, t, l);
    Piece<T, 8> px[HEADS][2], pg[HEADS][2];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        px[h][s] = load_piece<T, 8>(x + min(h, n - 1) * a.x_head[kind] + p.at[s]);
        pg[h][s] = load_piece<T, 8>(dy + min(h, n - 1) * a.dy_head[kind] + p.at[s]);
      }
    if (first) {
      weights_of<T>(a, kind, p, w);
      first = false;
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      float v[2][8], g[2][8];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        piece_f32<T, 8>(px[h][s], v[s]);
        piece_f32<T, 8>(pg[h][s], g[s]);
      }
      turn(p, g);
      float ss = 0.0f, dot = 0.0f;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(v[s][j], v[s][j], ss);
          dot = fmaf(g[s][j] * w[s][j], v[s][j], dot);
        }
      if (!live_lane) ss = dot = 0.0f;
      const float dim = static_cast<float>(a.dim);
      const float r = inv_sqrt(sum_lanes<W>(ss) / dim + a.eps);
      const float c = sum_lanes<W>(dot) * r / dim;  // mean(g w x r)
      if (!live || h >= n) continue;
      Piece<T, 8> o[2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float unit = v[s][j] * r;
          dw[s][j] = fmaf(g[s][j], unit, dw[s][j]);
          o[s].e[j] = from_f32<T>(r * fmaf(g[s][j], w[s][j], -unit * c));
        }
      if (live_lane)
#pragma unroll
        for (int s = 0; s < 2; ++s) store_piece<T, 8>(out + h * a.out_head[kind] + p.at[s], o[s]);
    }
  }
  if (a.dweight[kind] == nullptr) return;
  Pieces p;
  int pair[2];
  place_pieces(a.r, l, p, pair);
  if (live_lane)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) s_sum[group * (16 * W) + p.at[s] + j] = dw[s][j];
  __syncthreads();
  for (int d = threadIdx.x; d < a.dim; d += kThreads) {
    float sum = 0.0f;
    for (int g = 0; g < GROUPS; ++g) sum += s_sum[g * (16 * W) + d];
    a.workspace[(static_cast<int64_t>(kind) * gridDim.x + blockIdx.x) * a.dim + d] = sum;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kAnyWarps)
    k_heads_backward_any(const __grid_constant__ HeadsArgs a) {
  extern __shared__ float s_any[];  // [warps][dim] of g, then of the weight's gradient
  griddep_wait();
  griddep_launch_dependents();
  const int kind = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *g = s_any + warp * a.dim, *dw = s_any + (kAnyWarps + warp) * a.dim;
  for (int d = lane; d < a.dim; d += 32) dw[d] = 0.0f;
  const int64_t rows = a.tokens * a.heads[kind];
  const float dim = static_cast<float>(a.dim);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAnyWarps + warp; i < rows;
       i += static_cast<int64_t>(gridDim.x) * kAnyWarps) {
    const int64_t t = i / a.heads[kind];
    const int h = static_cast<int>(i - t * a.heads[kind]);
    const T *x = static_cast<const T *>(a.x[kind]) + t * a.x_token[kind] + h * a.x_head[kind];
    const T *dy = static_cast<const T *>(a.dy[kind]) + t * a.dy_token[kind] + h * a.dy_head[kind];
    T *out = static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h * a.out_head[kind];
    float ss = 0.0f, dot = 0.0f;
    for (int d = lane; d < a.dim; d += 32) g[d] = to_f32(dy[d]);
    __syncwarp();
    if (a.r.table != nullptr) {
      for (int j = lane; j < a.r.rot / 2; j += 32) {
        float2 cs;
        if (!angle_of(a, t, j, &cs)) continue;
        const int2 at = pair_at(a.r, j);
        const float u = g[at.x], v = g[at.y];
        g[at.x] = turn_a(u, v, cs);
        g[at.y] = turn_b(u, v, cs);
      }
      __syncwarp();
    }
    for (int d = lane; d < a.dim; d += 32) {
      const float f = to_f32(x[d]);
      ss = fmaf(f, f, ss);
      dot = fmaf(g[d] * weight_at<T>(a, kind, d), f, dot);
    }
    const float r = inv_sqrt(sum_lanes<32>(ss) / dim + a.eps);
    const float c = sum_lanes<32>(dot) * r / dim;
    for (int d = lane; d < a.dim; d += 32) {
      const float unit = to_f32(x[d]) * r;
      dw[d] = fmaf(g[d], unit, dw[d]);
      out[d] = from_f32<T>(r * fmaf(g[d], weight_at<T>(a, kind, d), -unit * c));
    }
    __syncwarp();
  }
  if (a.dweight[kind] == nullptr) return;
  __syncthreads();
  for (int d = threadIdx.x; d < a.dim; d += 32 * kAnyWarps) {
    float sum = 0.0f;
    for (int w = 0; w < kAnyWarps; ++w) sum += s_any[(kAnyWarps + w) * a.dim + d];
    a.workspace[(static_cast<int64_t>(kind) * gridDim.x + blockIdx.x) * a.dim + d] = sum;
  }
}

// The blocks' sums of a weight's gradient, in order and in 64 bits: a warp an element, block (x, kind).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_weight_gradient(const __grid_constant__ HeadsArgs a,
                                                              int blocks) {
  griddep_wait();
  griddep_launch_dependents();
  const int kind = blockIdx.y, lane = threadIdx.x & 31;
  const int d = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (a.dweight[kind] == nullptr || d >= a.dim) return;
  double sum = 0.0;
  for (int b = lane; b < blocks; b += 32)
    sum += a.workspace[(static_cast<int64_t>(kind) * blocks + b) * a.dim + d];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane != 0) return;
  if (a.weight_f32)
    static_cast<float *>(a.dweight[kind])[d] = static_cast<float>(sum);
  else
    static_cast<T *>(a.dweight[kind])[d] = from_f32<T>(static_cast<float>(sum));
}

template <typename T, int W, int HEADS>
cudaError_t launch_walk(const HeadsArgs &a, cudaStream_t stream) {
  constexpr int GROUPS = kThreads / W;
  const int64_t chunks = (a.heads[0] + HEADS - 1) / HEADS + (a.heads[1] + HEADS - 1) / HEADS;
  // The group's number is 32 bits wide: more tokens than fit it go in several launches.
  const int64_t most = (INT64_C(1) << 30) / chunks;
  for (int64_t t = 0; t < a.tokens; t += most) {
    const int64_t n = a.tokens - t < most ? a.tokens - t : most;
    HeadsArgs part = a;
    part.tokens = t + n;
    const unsigned blocks = static_cast<unsigned>((n * chunks + GROUPS - 1) / GROUPS);
    const cudaError_t e = launch_dependent(k_heads<T, W, HEADS>, dim3(blocks), dim3(kThreads), 0,
                                           stream, part, t);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Four heads a group where that still leaves some thousands of warps, else one.
template <typename T, int W>
cudaError_t launch_pieces(const HeadsArgs &a, cudaStream_t stream) {
  const int64_t warps = a.tokens * (a.heads[0] + a.heads[1]) * W / 32;
  return warps > 16384 ? launch_walk<T, W, 4>(a, stream) : launch_walk<T, W, 1>(a, stream);
}

template <typename T>
cudaError_t launch(const HeadsArgs &a, bool pieces, cudaStream_t stream) {
  if (pieces) {
    const int lanes = a.dim / 16;
    if (lanes <= 4) return launch_pieces<T, 4>(a, stream);
    if (lanes <= 8) return launch_pieces<T, 8>(a, stream);
    return launch_pieces<T, 16>(a, stream);
  }
  const int64_t rows = a.tokens * (a.heads[0] + a.heads[1]);
  const int64_t blocks = (rows + kAnyWarps - 1) / kAnyWarps;
  return launch_dependent(k_heads_any<T>, dim3(static_cast<unsigned>(blocks < 4864 ? blocks : 4864)),
                          dim3(32 * kAnyWarps), 0, stream, a);
}

template <typename T, int W>
cudaError_t launch_backward_pieces(const HeadsArgs &a, int blocks, cudaStream_t stream) {
  return launch_dependent(k_heads_backward<T, W>, dim3(blocks, a.heads[1] > 0 ? 2 : 1),
                          dim3(kThreads), kThreads * 16 * 4, stream, a);
}

template <typename T>
cudaError_t launch_backward(const HeadsArgs &a, bool pieces, int sms, cudaStream_t stream) {
  const int blocks = heads_blocks(sms);
  const int lanes = a.dim / 16;
  cudaError_t e;
  if (!pieces)
    e = launch_dependent(k_heads_backward_any<T>, dim3(blocks, a.heads[1] > 0 ? 2 : 1),
                         dim3(32 * kAnyWarps), 2 * kAnyWarps * a.dim * 4, stream, a);
  else if (lanes <= 4)
    e = launch_backward_pieces<T, 4>(a, blocks, stream);
  else if (lanes <= 8)
    e = launch_backward_pieces<T, 8>(a, blocks, stream);
  else
    e = launch_backward_pieces<T, 16>(a, blocks, stream);
  if (e != cudaSuccess || (a.dweight[0] == nullptr && a.dweight[1] == nullptr)) return e;
  return launch_dependent(k_weight_gradient<T>, dim3((a.dim + 7) / 8, a.heads[1] > 0 ? 2 : 1),
                          dim3(kThreads), 0, stream, a, blocks);
}

}  // namespace

int heads_blocks(int sms) { return 2 * sms; }

cudaError_t launch_heads(const HeadsArgs &a, int dtype, bool pieces, cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32: return launch<float>(a, pieces, stream);
    case IDX_DTYPE_F16: return launch<__half>(a, pieces, stream);
    default: return launch<__nv_bfloat16>(a, pieces, stream);
  }
}

cudaError_t launch_heads_backward(const HeadsArgs &a, int dtype, bool pieces, int sms,
                                  cudaStream_t stream) {
  switch (dtype) {
    case IDX_DTYPE_F32: return launch_backward<float>(a, pieces, sms, stream);
    case IDX_DTYPE_F16: return launch_backward<__half>(a, pieces, sms, stream);
    default: return launch_backward<__nv_bfloat16>(a, pieces, sms, stream);
  }
}

cudaError_t heads_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_heads_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_heads_status, &zero, sizeof(int32_t));
}

}  // namespace idx
