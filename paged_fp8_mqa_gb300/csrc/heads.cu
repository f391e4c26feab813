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
#include "pieces.cuh"
#include "ptx.cuh"

namespace idx {

__device__ int g_heads_status;

namespace {

constexpr int kThreads = 128;
constexpr int kFewWarps = 8192;
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

template <bool ADJ>
__device__ __forceinline__ Pieces pieces_of(const HeadsArgs &a, int64_t t, int l) {
  Pieces p;
  const int half = a.r.rot >> 1;
  int pair[2];
  place_pieces<ADJ>(a.r, a.dim, l, p, pair);
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

// 1 / sqrt(v): the approximation and one step of Newton's method (where v is a positive number).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v > 1e-37f && v < 1e37f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

// A row whose mean square is outside of float32's range, or so small that its squares lose their bits, is
// taken times 2^-96 or 2^96 (its elements are past some 2^59, or, with eps = 0, all below 2^-50).  Rows with
// an infinity or a NaN are taken so too and come out as they would.
__device__ __forceinline__ float rescale(float mean_square) {
  return mean_square >= 7.8886090522101181e-31f && mean_square <= 3.4028234663852886e38f ? 1.0f  // (2^-100)
         : mean_square > 1.0f ? 1.2621774483536189e-29f : 7.922816251426434e28f;
}
// Whether a row's 1 / sqrt(mean square) says that it need not be.
__device__ __forceinline__ bool in_range(float r) { return r > 0.0f && r < 1.1258999068426240e15f; }

// The lane's 16 weights in float32 (1 without), as the elements are unpacked.
template <bool ADJ, typename T>
__device__ __forceinline__ void weights_of(const HeadsArgs &a, int kind, const Pieces &p,
                                           float2 (&w)[2][4]) {
  if (a.weight[kind] == nullptr) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[0][j] = w[1][j] = make_float2(1.0f, 1.0f);
  } else if (a.weight_f32) {
    const float *at = static_cast<const float *>(a.weight[kind]);
    const Piece<float, 8> two[2] = {load_whole(at + p.at[0], a.weight_pieces),
                                    load_whole(at + p.at[1], a.weight_pieces)};
    unpack<ADJ, float>(two, w);
  } else {
    const T *at = static_cast<const T *>(a.weight[kind]);
    const Piece<T, 8> two[2] = {load_whole(at + p.at[0], a.weight_pieces),
                                load_whole(at + p.at[1], a.weight_pieces)};
    unpack<ADJ, T>(two, w);
  }
}

template <int W>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int o = 1; o < W; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The same by the lanes of one group alone.
template <int W>
__device__ __forceinline__ float sum_group(float x) {
  const uint32_t mask = ((1u << W) - 1u) << (threadIdx.x & 31u & ~(W - 1u));
#pragma unroll
  for (int o = 1; o < W; o <<= 1) x += __shfl_xor_sync(mask, x, o);
  return x;
}

// The lane's part of a row's sum of squares, and of sum a b c.
__device__ __forceinline__ float squares(const float2 (&v)[2][4]) {
  float2 sq = __fmul2_rn(v[0][0], v[0][0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) sq = __ffma2_rn(v[j >> 2][j & 3], v[j >> 2][j & 3], sq);
  return sq.x + sq.y;
}
__device__ __forceinline__ float products(const float2 (&a)[2][4], const float2 (&b)[2][4],
                                          const float2 (&c)[2][4]) {
  float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sum = __ffma2_rn(__fmul2_rn(a[j >> 2][j & 3], b[j >> 2][j & 3]), c[j >> 2][j & 3], sum);
  return sum.x + sum.y;
}

// The lane's elements times `by` (see rescale), and (1 / rms of such elements, by).
template <int W>
__device__ __forceinline__ float2 rescaled(float2 (&v)[2][4], bool idle, float inv_dim, float eps) {
  const float by = rescale(fmaf(sum_group<W>(idle ? 0.0f : squares(v)), inv_dim, eps));
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] = __fmul2_rn(v[j >> 2][j & 3], make_float2(by, by));
  return make_float2(inv_sqrt(fmaf(sum_group<W>(idle ? 0.0f : squares(v)), inv_dim, eps * by * by)), by);
}

// The factors with which a row is turned and weighted: y0 = own[0] v0 + cross[0] v1, y1 = own[1] v1 + cross[1] v0.
__device__ __forceinline__ void weigh(uint32_t valid, const float2 (&w)[2][4], float2 (&own)[2][4],
                                      float2 (&cross)[2][4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 c = own[0][j], n = cross[0][j];
    own[0][j] = __fmul2_rn(c, w[0][j]);
    own[1][j] = __fmul2_rn(c, w[1][j]);
    cross[0][j] = __fmul2_rn(n, minus(w[1][j]));
    cross[1][j] = __fmul2_rn(n, w[0][j]);
    // (Where a pair is not turned, an infinite weight times the sine of 0 must not reach its neighbour.)
    if (!((valid >> (2 * j)) & 1u)) cross[0][j].x = cross[1][j].x = 0.0f;
    if (!((valid >> (2 * j + 1)) & 1u)) cross[0][j].y = cross[1][j].y = 0.0f;
  }
}

// W lanes (a power of two, 16 elements a lane; those past dim idle) walk `walk` heads of one token, of q or
// of k, AHEAD heads asked for before they are needed.
template <typename T, int W, bool ADJ, int AHEAD, bool NORM, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS)
    k_heads(const __grid_constant__ HeadsArgs a, int64_t first_token, int walk) {
  griddep_wait();
  griddep_launch_dependents();
  const int chunks_q = (a.heads[0] + walk - 1) / walk;
  const int chunks = chunks_q + (a.heads[1] + walk - 1) / walk;
  const uint32_t id = blockIdx.x * (kThreads / W) + threadIdx.x / W;
  const uint32_t tok = id / chunks;
  const int64_t t = first_token + tok;
  // (Past the last token or element: the last, and nothing is stored, so that the shuffles find all
  // their lanes.)
  const int lanes = a.dim / 16;
  const bool idle = static_cast<int>(threadIdx.x % W) >= lanes;
  const bool live = t < a.tokens && !idle;
  const int64_t tt = min(t, a.tokens - 1);
  const int l = min(static_cast<int>(threadIdx.x % W), lanes - 1);
  int chunk = id - tok * chunks;
  const int kind = chunk >= chunks_q;
  if (kind) chunk -= chunks_q;
  const int h0 = chunk * walk, n = min(walk, a.heads[kind] - h0);
  const int rounds = __reduce_max_sync(0xffffffffu, n);  // (the same for the whole warp)
  const int64_t x_head = a.x_head[kind], out_head = a.out_head[kind];
  const T *x = static_cast<const T *>(a.x[kind]) + tt * a.x_token[kind] + h0 * x_head;
  T *out = static_cast<T *>(a.out[kind]) + tt * a.out_token[kind] + h0 * out_head;
  const Pieces p = pieces_of<ADJ>(a, tt, l);
  Piece<T, 8> own[AHEAD][2];
#pragma unroll
  for (int d = 0; d < AHEAD; ++d)
#pragma unroll
    for (int s = 0; s < 2; ++s)
      own[d][s] = load_piece<T, 8>(x + min(d, n - 1) * x_head + p.at[s]);
  if (live && h0 == 0 && kind == (a.heads[0] == 0) &&
      p.valid != ((p.on[0] ? 0x0Fu : 0u) | (p.on[1] ? 0xF0u : 0u)))
    atomicOr(&g_heads_status, IDX_DEV_BAD_POSITION);
  float2 own_f[NORM ? 2 : 1][4], cross[NORM ? 2 : 1][4];
  angles_of(p, own_f[0], cross[0]);
  const uint32_t valid = p.valid;
  if constexpr (NORM) {
    float2 w[2][4];
    weights_of<ADJ, T>(a, kind, p, w);
    weigh(valid, w, own_f, cross);
  }
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  const int at0 = p.at[0], at1 = p.at[1];
  const T *next = x + AHEAD * x_head;
  for (int r0 = 0; r0 < rounds; r0 += AHEAD) {
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) {
      const int h = r0 + d;
      if (h >= rounds) break;
      const bool store = live && h < n;
      if (NORM || valid != 0) {
        float2 v[2][4];
        unpack<ADJ, T>(own[d], v);
        if constexpr (NORM) {
          const float square = fmaf(sum_lanes<W>(idle ? 0.0f : squares(v)), inv_dim, a.eps);
          float r = inv_sqrt(square);
          // (A vote, so that the branch is the warp's: parted lanes, or these rows once more behind the loop,
          // measured 55 to 62 us for 52 with 8192 tokens of 72 heads of 128.)
          if (__any_sync(0xffffffffu, !in_range(r))) {
            const float by = rescale(square);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] = __fmul2_rn(v[j >> 2][j & 3], make_float2(by, by));
            r = inv_sqrt(fmaf(sum_lanes<W>(idle ? 0.0f : squares(v)), inv_dim, a.eps * by * by));
            const float2 r2 = make_float2(r, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // (What is not turned must not meet its neighbour, which may not be finite, not even times 0.)
              const float2 x = v[0][j], y = v[1][j];
              float2 c0 = __fmul2_rn(y, cross[0][j]), c1 = __fmul2_rn(x, cross[1][j]);
              if (!((valid >> (2 * j)) & 1u)) c0.x = c1.x = 0.0f;
              if (!((valid >> (2 * j + 1)) & 1u)) c0.y = c1.y = 0.0f;
              v[0][j] = __fmul2_rn(__ffma2_rn(x, own_f[0][j], c0), r2);
              v[1][j] = __fmul2_rn(__ffma2_rn(y, own_f[1][j], c1), r2);
            }
          } else {
            const float2 r2 = make_float2(r, r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = v[0][j], y = v[1][j];
              v[0][j] = __fmul2_rn(__ffma2_rn(x, own_f[0][j], __fmul2_rn(y, cross[0][j])), r2);
              v[1][j] = __fmul2_rn(__ffma2_rn(y, own_f[1][j], __fmul2_rn(x, cross[1][j])), r2);
            }
          }
        } else {
          turn(valid, own_f[0], cross[0], v);
        }
        pack<ADJ, T>(v, own[d]);
      }
      if (store) {
        store_piece<T, 8>(out + at0, own[d][0]);
        store_piece<T, 8>(out + at1, own[d][1]);
      }
      out += out_head;
      if (h + AHEAD < n) {  // (past the last: what is there, which is stored nowhere)
        own[d][0] = load_piece<T, 8>(next + at0);
        own[d][1] = load_piece<T, 8>(next + at1);
      }
      next += x_head;
    }
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
      float square = sum_lanes<32>(ss) / static_cast<float>(a.dim) + a.eps;
      const float by = rescale(square);  // (the same for all lanes)
      if (by != 1.0f) {
        ss = 0.0f;
        for (int d = lane; d < a.dim; d += 32) ss = fmaf(row[d] * by, row[d] * by, ss);
        square = sum_lanes<32>(ss) / static_cast<float>(a.dim) + a.eps * by * by;
      }
      const float r = inv_sqrt(square);
      for (int d = lane; d < a.dim; d += 32) row[d] = row[d] * by * r * weight_at<T>(a, kind, d);
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

// How the gradients' blocks are shared: the first `q` of them take q's heads, the others k's, `walk`
// heads of a token at a time.
struct BackwardSplit {
  int32_t q, k, walk;
};

// The rows of the calling group whose squares leave float32's range, once more; their parts of the weight's
// gradient are added to the group's sums.  (A function of its own behind the loop, so that it takes no
// register from it: in the loop 55 to 59 us for 51.)
template <typename T, int W, bool ADJ>
__device__ __noinline__ void gradients_again(const HeadsArgs &a, const BackwardSplit &split, float *s_sum) {
  constexpr int GROUPS = kThreads / W;
  const int kind = static_cast<int>(blockIdx.x) >= split.q, walk = split.walk;
  const int block = blockIdx.x - (kind ? split.q : 0), blocks = kind ? split.k : split.q;
  const int heads = a.heads[kind], lanes = a.dim / 16, chunks = (heads + walk - 1) / walk;
  const int group = threadIdx.x / W, lw = threadIdx.x % W, l = min(lw, lanes - 1);
  const bool idle = lw >= lanes;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  const int64_t items = a.tokens * chunks, step = static_cast<int64_t>(blocks) * GROUPS;
  float2 w[2][4];
  for (int64_t i = static_cast<int64_t>(block) * GROUPS + group; i < items; i += step) {
    const int64_t t = i / chunks;
    const int h0 = static_cast<int>(i - t * chunks) * walk, h1 = min(h0 + walk, heads);
    const Pieces p = pieces_of<ADJ>(a, t, l);
    float2 c[4], m[4];
    angles_of(p, c, m);
    weights_of<ADJ, T>(a, kind, p, w);
    for (int h = h0; h < h1; ++h) {
      const T *x = static_cast<const T *>(a.x[kind]) + t * a.x_token[kind] + h * a.x_head[kind];
      const T *dy = static_cast<const T *>(a.dy[kind]) + t * a.dy_token[kind] + h * a.dy_head[kind];
      T *out = static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h * a.out_head[kind];
      Piece<T, 8> row[2] = {load_piece<T, 8>(x + p.at[0]), load_piece<T, 8>(x + p.at[1])};
      float2 v[2][4], g[2][4];
      unpack<ADJ, T>(row, v);
      if (in_range(inv_sqrt(fmaf(sum_group<W>(idle ? 0.0f : squares(v)), inv_dim, a.eps)))) continue;
      const float2 r_by = rescaled<W>(v, idle, inv_dim, a.eps);
      row[0] = load_piece<T, 8>(dy + p.at[0]);
      row[1] = load_piece<T, 8>(dy + p.at[1]);
      unpack<ADJ, T>(row, g);
      turn(p.valid, c, m, g);
      const float dot = sum_group<W>(idle ? 0.0f : products(g, w, v)), mean = -dot * r_by.x * inv_dim;
      const float2 r2 = make_float2(r_by.x, r_by.x), k2 = make_float2(mean, mean);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 unit = __fmul2_rn(v[s][j], r2), dw = __fmul2_rn(g[s][j], unit);
          v[s][j] = __fmul2_rn(__fmul2_rn(__ffma2_rn(g[s][j], w[s][j], __fmul2_rn(unit, k2)), r2),
                               make_float2(r_by.y, r_by.y));
          if (!idle && a.dweight[kind] != nullptr) {
            s_sum[group * (16 * W) + element_at<ADJ>(p, s, j, 0)] += dw.x;
            s_sum[group * (16 * W) + element_at<ADJ>(p, s, j, 1)] += dw.y;
          }
        }
      pack<ADJ, T>(v, row);
      if (!idle) {
        store_piece<T, 8>(out + p.at[0], row[0]);
        store_piece<T, 8>(out + p.at[1], row[1]);
      }
    }
  }
}

// The gradients, W lanes a head.  8192 tokens of 32 + 8 heads of 128 (252 MB) take 51 us with the second
// launch, 37 at the copy rate: 128 registers leave 16 warps an SM (three blocks of them 3 us more, five 22).
// Walks of two heads 55 us, of eight 52; loads three heads ahead through shared memory 50.5, not worth it.  A
// lane's 16 elements of the weight's gradient stay in its registers over all its heads (a float32 sum of as many
// terms as there are heads for each of 4 * SMs * 128 / W groups: 34 of 8192 x 40); a block leaves its sums in the
// workspace and a second launch adds the blocks', in order and with what the roundings left out.
template <typename T, int W, bool ADJ>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    k_heads_backward(const __grid_constant__ HeadsArgs a, const __grid_constant__ BackwardSplit split) {
  constexpr int GROUPS = kThreads / W;
  extern __shared__ float s_sum[];  // [GROUPS][16 * W]
  griddep_wait();
  griddep_launch_dependents();
  const int kind = static_cast<int>(blockIdx.x) >= split.q;
  const int block = blockIdx.x - (kind ? split.q : 0), blocks = kind ? split.k : split.q;
  const int heads = a.heads[kind], lanes = a.dim / 16, walk = split.walk;
  const int group = threadIdx.x / W, lw = threadIdx.x % W, l = min(lw, lanes - 1);
  const bool live_lane = lw < lanes;
  const int chunks = (heads + walk - 1) / walk;
  const int64_t items = a.tokens * chunks, step = static_cast<int64_t>(blocks) * GROUPS;
  const int64_t x_head = a.x_head[kind], dy_head = a.dy_head[kind], out_head = a.out_head[kind];
  Pieces p;
  int pair[2];
  place_pieces<ADJ>(a.r, a.dim, l, p, pair);
  const int at0 = p.at[0], at1 = p.at[1];
  float2 dw[2][4], w[2][4];
  weights_of<ADJ, T>(a, kind, p, w);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[s][j] = make_float2(0.0f, 0.0f);
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  float least = 1.0f;  // of the rows' r (the same in all lanes of a group)
  // (All groups of a warp make the same number of rounds, so that the shuffles find all their lanes.)
  for (int64_t i0 = static_cast<int64_t>(block) * GROUPS; i0 < items; i0 += step) {
    const int64_t i = i0 + group, at = min(i, items - 1), t = at / chunks;
    const int h0 = static_cast<int>(at - t * chunks) * walk, n = min(walk, heads - h0);
    const int rounds = __reduce_max_sync(0xffffffffu, n);
    const T *x = static_cast<const T *>(a.x[kind]) + t * a.x_token[kind] + h0 * x_head;
    const T *dy = static_cast<const T *>(a.dy[kind]) + t * a.dy_token[kind] + h0 * dy_head;
    T *out = static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h0 * out_head;
    Piece<T, 8> px[2], pg[2];
    px[0] = load_piece<T, 8>(x + at0);
    px[1] = load_piece<T, 8>(x + at1);
    pg[0] = load_piece<T, 8>(dy + at0);
    pg[1] = load_piece<T, 8>(dy + at1);
    float2 c[4], m[4];
    p = pieces_of<ADJ>(a, t, l);
    angles_of(p, c, m);
    for (int h = 0; h < rounds; ++h) {
      float2 v[2][4], g[2][4];
      unpack<ADJ, T>(px, v);
      unpack<ADJ, T>(pg, g);
      x += x_head;
      dy += dy_head;
      if (h + 1 < n) {
        px[0] = load_piece<T, 8>(x + at0);
        px[1] = load_piece<T, 8>(x + at1);
        pg[0] = load_piece<T, 8>(dy + at0);
        pg[1] = load_piece<T, 8>(dy + at1);
      }
      turn(p.valid, c, m, g);
      float2 sq = make_float2(0.0f, 0.0f), sd = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sq = __ffma2_rn(v[s][j], v[s][j], sq);
          sd = __ffma2_rn(__fmul2_rn(g[s][j], w[s][j]), v[s][j], sd);
        }
      const float ss = sum_lanes<W>(live_lane ? sq.x + sq.y : 0.0f);
      const float dot = sum_lanes<W>(live_lane ? sd.x + sd.y : 0.0f);
      const float r_row = inv_sqrt(fmaf(ss, inv_dim, a.eps));
      // (A row out of range counts nothing here: it is taken once more below.)
      const float r = in_range(r_row) ? r_row : 0.0f;
      least = fminf(least, r);
      const float mean = -dot * r * inv_dim;  // -mean(g w x r)
      if (i < items && h < n) {
        const float2 r2 = make_float2(r, r), k2 = make_float2(mean, mean);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 unit = __fmul2_rn(v[s][j], r2);
            dw[s][j] = __ffma2_rn(g[s][j], unit, dw[s][j]);
            v[s][j] = __fmul2_rn(__ffma2_rn(g[s][j], w[s][j], __fmul2_rn(unit, k2)), r2);
          }
        if (live_lane) {
          Piece<T, 8> o[2];
          pack<ADJ, T>(v, o);
          store_piece<T, 8>(out + at0, o[0]);
          store_piece<T, 8>(out + at1, o[1]);
        }
      }
      out += out_head;
    }
  }
  if (live_lane && a.dweight[kind] != nullptr)
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s_sum[group * (16 * W) + element_at<ADJ>(p, s, j, 0)] = dw[s][j].x;
        s_sum[group * (16 * W) + element_at<ADJ>(p, s, j, 1)] = dw[s][j].y;
      }
  if (least == 0.0f) gradients_again<T, W, ADJ>(a, split, s_sum);
  if (a.dweight[kind] == nullptr) return;
  __syncthreads();
  for (int d = threadIdx.x; d < a.dim; d += kThreads) {
    float sum = 0.0f;
    for (int g = 0; g < GROUPS; ++g) sum += s_sum[g * (16 * W) + d];
    a.workspace[static_cast<int64_t>(blockIdx.x) * a.dim + d] = sum;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kAnyWarps)
    k_heads_backward_any(const __grid_constant__ HeadsArgs a, const BackwardSplit split) {
  extern __shared__ float s_any[];  // [warps][dim] of g, then of the weight's gradient
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kind = static_cast<int>(blockIdx.x) >= split.q;
  const int block = blockIdx.x - (kind ? split.q : 0), blocks = kind ? split.k : split.q;
  float *g = s_any + warp * a.dim, *dw = s_any + (kAnyWarps + warp) * a.dim;
  for (int d = lane; d < a.dim; d += 32) dw[d] = 0.0f;
  const int64_t rows = a.tokens * a.heads[kind];
  const float dim = static_cast<float>(a.dim);
  for (int64_t i = static_cast<int64_t>(block) * kAnyWarps + warp; i < rows;
       i += static_cast<int64_t>(blocks) * kAnyWarps) {
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
    float square = sum_lanes<32>(ss) / dim + a.eps;
    const float by = rescale(square);  // (the same for all lanes)
    if (by != 1.0f) {
      ss = dot = 0.0f;
      for (int d = lane; d < a.dim; d += 32) {
        const float f = to_f32(x[d]) * by;
        ss = fmaf(f, f, ss);
        dot = fmaf(g[d] * weight_at<T>(a, kind, d), f, dot);
      }
      square = sum_lanes<32>(ss) / dim + a.eps * by * by;
    }
    const float r = inv_sqrt(square);  // (of the elements times `by`)
    const float c = sum_lanes<32>(dot) * r / dim;
    for (int d = lane; d < a.dim; d += 32) {
      const float unit = to_f32(x[d]) * by * r;
      dw[d] = fmaf(g[d], unit, dw[d]);
      out[d] = from_f32<T>(r * fmaf(g[d], weight_at<T>(a, kind, d), -unit * c) * by);
    }
    __syncwarp();
  }
  if (a.dweight[kind] == nullptr) return;
  __syncthreads();
  for (int d = threadIdx.x; d < a.dim; d += 32 * kAnyWarps) {
    float sum = 0.0f;
    for (int w = 0; w < kAnyWarps; ++w) sum += s_any[(kAnyWarps + w) * a.dim + d];
    a.workspace[static_cast<int64_t>(blockIdx.x) * a.dim + d] = sum;
  }
}

// A sum and what its roundings left out (exact for each addition).
struct Sum2 {
  float sum, rest;
};
__device__ __forceinline__ void add2(Sum2 &s, float x) {
  const float t = __fadd_rn(s.sum, x), y = __fsub_rn(t, s.sum);
  s.rest = __fadd_rn(s.rest, __fadd_rn(__fsub_rn(s.sum, __fsub_rn(t, y)), __fsub_rn(x, y)));
  s.sum = t;
}

// The blocks' sums of a weight's gradient, in order and in two floats: 32 elements a block (x, kind), a warp
// every 32nd row of them.  (In 64 bits, whose units are few, the two launches took 60 us for 53, as they were then.)
template <typename T>
__global__ void __launch_bounds__(1024) k_weight_gradient(const __grid_constant__ HeadsArgs a,
                                                          const BackwardSplit split) {
  __shared__ Sum2 s_part[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int kind = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = blockIdx.x * 32 + lane;
  if (a.dweight[kind] == nullptr) return;
  const int begin = kind ? split.q : 0, end = begin + (kind ? split.k : split.q);
  Sum2 sum{0.0f, 0.0f};
  if (d < a.dim) {
#pragma unroll 4
    for (int b = begin + warp; b < end; b += 32) add2(sum, a.workspace[static_cast<int64_t>(b) * a.dim + d]);
  }
  s_part[warp][lane] = sum;
  __syncthreads();
  sum = s_part[lane][warp];  // element `warp` of the block's, part `lane`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, sum.sum, o);
    const float rest = __shfl_xor_sync(0xffffffffu, sum.rest, o);
    add2(sum, other);
    sum.rest += rest;
  }
  const int e = blockIdx.x * 32 + warp;
  if (lane != 0 || e >= a.dim) return;
  // (Of an infinite sum the rest is NaN.)
  const float all = fabsf(sum.sum) < __int_as_float(0x7F800000) ? sum.sum + sum.rest : sum.sum;
  if (a.weight_f32)
    static_cast<float *>(a.dweight[kind])[e] = all;
  else
    static_cast<T *>(a.dweight[kind])[e] = from_f32<T>(all);
}

template <typename T, int W, bool ADJ, int AHEAD, bool NORM, int BLOCKS = 1>
cudaError_t launch_walk(const HeadsArgs &a, int walk, cudaStream_t stream) {
  constexpr int GROUPS = kThreads / W;
  const int64_t chunks = (a.heads[0] + walk - 1) / walk + (a.heads[1] + walk - 1) / walk;
  // The group's number is 32 bits wide: more tokens than fit it go in several launches.
  const int64_t most = (INT64_C(1) << 30) / chunks;
  for (int64_t t = 0; t < a.tokens; t += most) {
    const int64_t n = a.tokens - t < most ? a.tokens - t : most;
    HeadsArgs part = a;
    part.tokens = t + n;
    const unsigned blocks = static_cast<unsigned>((n * chunks + GROUPS - 1) / GROUPS);
    const cudaError_t e = launch_dependent(k_heads<T, W, ADJ, AHEAD, NORM, BLOCKS>, dim3(blocks), dim3(kThreads), 0,
                                           stream, part, t, walk);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// As many heads a group as leave 8192 warps, 16 at most; a small call takes one head a group.  Norms of 72 heads
// of 128 in bfloat16, us with 1, 2, 4, 8, 16 heads a group: 64 tokens 2.6, 2.7, 3.2, 4.3, 6.8 (1 is taken); 512
// tokens 8.4, 6.9, 6.0, 5.1, 7.6 (1); 1024 14.9, 10.6, 8.7, 9.0, 10.2 (2); 2048 28.3, 19.6, 14.6, 14.5, 14.7 (4);
// 8192 117, 75, 56, 51, 52 (16).  So right at both ends; between 256 and 1024 tokens more heads a group
// would be faster.
template <typename T, int W, bool ADJ>
cudaError_t launch_pieces(const HeadsArgs &a, cudaStream_t stream) {
  int walk = 16;
  while (walk > 1 && a.tokens * ((a.heads[0] + a.heads[1]) / walk) * W / 32 < kFewWarps) walk /= 2;
  // Heads asked for ahead, and blocks of 128 threads that an SM holds (see k_heads).
  constexpr int AHEAD = sizeof(T) == 2 ? 3 : 2, TURN_AHEAD = sizeof(T) == 2 ? 4 : 2;
  constexpr int BLOCKS = sizeof(T) == 2 ? 6 : 4;
  if (a.norm)
    return walk == 1 ? launch_walk<T, W, ADJ, 1, true>(a, 1, stream)
                     : launch_walk<T, W, ADJ, AHEAD, true, BLOCKS>(a, walk, stream);
  return walk == 1 ? launch_walk<T, W, ADJ, 1, false>(a, 1, stream)
                   : launch_walk<T, W, ADJ, TURN_AHEAD, false, BLOCKS>(a, walk, stream);
}

template <typename T>
cudaError_t launch(const HeadsArgs &a, bool pieces, cudaStream_t stream) {
  if (pieces) {
    const int lanes = a.dim / 16;
    if (a.r.interleaved) {
      if (lanes <= 4) return launch_pieces<T, 4, true>(a, stream);
      if (lanes <= 8) return launch_pieces<T, 8, true>(a, stream);
      return launch_pieces<T, 16, true>(a, stream);
    }
    if (lanes <= 4) return launch_pieces<T, 4, false>(a, stream);
    if (lanes <= 8) return launch_pieces<T, 8, false>(a, stream);
    return launch_pieces<T, 16, false>(a, stream);
  }
  const int64_t rows = a.tokens * (a.heads[0] + a.heads[1]);
  const int64_t blocks = (rows + kAnyWarps - 1) / kAnyWarps;
  return launch_dependent(k_heads_any<T>, dim3(static_cast<unsigned>(blocks < 4864 ? blocks : 4864)),
                          dim3(32 * kAnyWarps), 0, stream, a);
}

template <typename T, int W>
cudaError_t launch_backward_pieces(const HeadsArgs &a, const BackwardSplit &s, cudaStream_t stream) {
  return a.r.interleaved ? launch_dependent(k_heads_backward<T, W, true>, dim3(s.q + s.k),
                                            dim3(kThreads), kThreads * 16 * 4, stream, a, s)
                         : launch_dependent(k_heads_backward<T, W, false>, dim3(s.q + s.k),
                                            dim3(kThreads), kThreads * 16 * 4, stream, a, s);
}

template <typename T>
cudaError_t launch_backward(const HeadsArgs &a, bool pieces, int sms, cudaStream_t stream) {
  // Blocks in proportion to the heads of q and of k, no more than there are heads for.
  const int lanes = a.dim / 16, width = lanes <= 4 ? 4 : lanes <= 8 ? 8 : 16;
  const int at_once = pieces ? kThreads / width : kAnyWarps;
  const int64_t all = heads_blocks(sms), heads = a.heads[0] + a.heads[1] + (a.heads[0] + a.heads[1] == 0);
  BackwardSplit s;
  s.walk = 4;
  while (pieces && s.walk > 1 && a.tokens * heads < all * at_once * s.walk) s.walk /= 2;
  if (!pieces) s.walk = 1;
  const auto blocks = [&](int h) {
    const int64_t share = all * h / heads, need = (a.tokens * ((h + s.walk - 1) / s.walk) + at_once - 1) / at_once;
    return static_cast<int>(h == 0 ? 0 : need < share ? need : share > 0 ? share : 1);
  };
  s.k = blocks(a.heads[1]);
  s.q = blocks(a.heads[0]);
  cudaError_t e = cudaSuccess;
  if (s.q + s.k == 0)
    ;  // (no tokens or no heads: the weights' gradients are sums over nothing)
  else if (!pieces)
    e = launch_dependent(k_heads_backward_any<T>, dim3(s.q + s.k), dim3(32 * kAnyWarps),
                         2 * kAnyWarps * a.dim * 4, stream, a, s);
  else if (width == 4)
    e = launch_backward_pieces<T, 4>(a, s, stream);
  else if (width == 8)
    e = launch_backward_pieces<T, 8>(a, s, stream);
  else
    e = launch_backward_pieces<T, 16>(a, s, stream);
  if (e != cudaSuccess || (a.dweight[0] == nullptr && a.dweight[1] == nullptr)) return e;
  return launch_dependent(k_weight_gradient<T>, dim3((a.dim + 31) / 32, a.dweight[1] != nullptr ? 2 : 1),
                          dim3(1024), 0, stream, a, s);
}

}  // namespace

int heads_blocks(int sms) { return 4 * sms; }

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
