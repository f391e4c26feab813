// attention_kernel.cuh -- attention over the 8-bit K/V cache: for row (b, t) and query head h with
// K/V head g = h / (heads / kv_heads),
//   z_p = scale * ks[page(p), g] * (q . k_p),  out = sum_p softmax(z)_p * vs[page(p), g] * v_p
// over the positions p <= seq_lens[b] - next_n + t, or over those of them that the select stored
// in the row's slots.
//
// Both products run on the tensor core in 8 bits, straight from the cache's bytes: the cache is
// never converted.  The other operand keeps its precision by being split into 8-bit parts:
//   * a query row is scaled by a power of two to [2^14, 2^15) and written as three parts, each the
//     e5m2 nearest to what is left: 3 + 4 + 4 bits (a rest has a sign) hold a bfloat16's 8 or a
//     float16's 11 exactly, down to 2^-31 of the row's largest magnitude.  Products of 8-bit values
//     are exact and sums float32, so the scores are those of the unrounded queries.  The parts'
//     products go into the same accumulator.  (e4m3 parts, two would do for bfloat16, end at 2^-18: an
//     outlier that meets no key's element silenced the rest of its row.)
//   * a weight is written as such parts too, three for bfloat16 and four for float16, held 2^3, 2^7
//     and 2^11 up after the first: within 2^-10 of itself (2^-14 with four), or 2^-34 (2^-38) of the
//     row's largest.  The parts stand in columns of their own and are added when O is read.  e5m2 for
//     its reach: a first token of no value that takes most of a row's weight, or a block with a
//     large value scale, leaves an output that is all small weights, and the denominator counts
//     them all.  (Two e4m3 parts ended 2^-18 below the largest: with 131,072 positions behind
//     such a token the output was 0.8 of itself off.  e4m3 and e5m2 reach as far, but hold what is
//     2^-14 below the largest to one part in eight.)
// The weights that meet V carry the block scales: with z' = log2(e) z + log2|vs| they are
// u = 2^(z' - ref), sign(vs) applied, so that O = sum u v needs no scale of its own and may be
// accumulated in tensor memory over tiles of any scales, and the softmax's denominator is
// l = sum u / |vs| in float32; out = O / l.  ref follows the running maximum of z' from below: it
// moves (to the maximum) only when some u would leave e5m2's range, and then O and l are rescaled.
//
// A tile is 128 positions of one K/V head.  S^T[128 positions x rows] = K Q^T puts a position in
// each lane of tensor memory and the rows that share the K/V head (query heads times draft slots)
// in its columns, so that K and V are read once for all of them and the softmax of a position's
// rows is one thread's work; O^T[dim x rows] = V^T P^T takes V as it lies (M-major) and a
// dimension in each lane.
//
// The tiles of all (request, K/V head) groups in one line are cut into equal runs, one for each CTA
// of the grid; a group that a run's end cuts leaves partial sums in the workspace and a second
// launch joins them in order.  Every wait has a limit; nothing waits on another CTA.
#pragma once

#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"
#include "runs.h"

namespace idx {
namespace {

__device__ int g_attention_status;

constexpr int kTile = 128;                     // positions of a tile
constexpr uint64_t kWaitNs = 1000000000ull;    // 1 s: far beyond any legitimate wait
constexpr int kNone = INT_MAX;                 // the position of a token that no row sees
constexpr float kRefNone = -1e30f;             // the reference of a row that has seen nothing
// Weights are 2^(z' - ref), at most 2^11 when ref is set; ref moves when one would pass 2^15.8 = 57,052,
// just inside e5m2's 57,344, that is when a row's maximum has grown 28-fold.  Each part's rounding
// leaves at most 2^-3 of the binade to the second and 2^-4 to those after it, so that no part leaves
// the range either, and the last of three ends at 2^-24, the last of four at 2^-28.
constexpr float kTop = 11.0f, kMost = 15.8f, kUp2 = 8.0f, kUp = 16.0f;
constexpr float kLeastScale = 7.8886090522101180541e-31f;  // 2^-100: a value scale below it is 0

// One kernel's shape: R rows, PARTS parts a weight, head_dim D.
template <int D_, int R_, int PARTS_, bool SELECT_>
struct AttnCfg {
  static constexpr int D = D_, R = R_, PARTS = PARTS_;
  static constexpr bool SELECT = SELECT_;
  static constexpr int QPARTS = 3;                    // parts of a query
  // With R = 8 a query's parts stand side by side, in columns that are added when read (the last
  // eight of 32 mean nothing); else each part is a product of its own into the same columns.  (Three
  // products with R = 8 too: tiny 9.1 us for 8.7, serving 96 for 94.)
  static constexpr bool CAT = R == 8;
  static constexpr int NS = CAT ? 32 : R;             // columns of S
  static constexpr int PASSES = CAT ? 1 : QPARTS;     // products that make S
  static constexpr int NO = (R * PARTS + 15) / 16 * 16;  // columns of O (N in steps of 16)
  static constexpr int WG = R == 64 ? 2 : 1;          // softmax warpgroups, R / WG rows each
  static constexpr int RT = R / WG;
  static constexpr int SOFT_WARPS = 4 * WG;
  // Warps that load: one for whole pages; up to four share the rows of a selection, as many as the
  // softmax's registers leave room for.
  static constexpr int LOADERS = !SELECT || R == 32 ? 1 : R == 8 ? 4 : 2;
  static constexpr int THREADS = 32 * (LOADERS + 1 + SOFT_WARPS);
  static constexpr int COLS = 2 * NS + NO;            // two of S, one of O
  static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  // CTAs on an SM, each with a pipeline of its own, so that one's loads and products run beside the
  // other's softmax.  Three of two stages instead of two of three: decode took 1.4 times as long, as
  // what the next launch needs no longer fits beside them.  64 rows in chunks of 32, two CTAs an SM:
  // one long request 1.07 times as long, a batch of 64 requests with 64 heads on one 1.3 times.
  static constexpr int CTAS = R == 64 ? 1 : 2;
  static constexpr int KV_BYTES = 2 * kTile * D;
  static constexpr int Q_BYTES = NS * (CAT ? 1 : QPARTS) * D;
  static constexpr int P_BYTES = NO * kTile;          // a tile's weights
  // They take the place of the tile's keys, which have been read by then, where they fit it; else
  // two buffers of their own.
  static constexpr bool OVER_K = P_BYTES <= kTile * D;
  static constexpr int AUX = kTile * 16;              // a stage's Token records
  static constexpr int MISC = 48 * R + 3 * D * 4 + 256;
  static constexpr int FIXED = 1024 + Q_BYTES + (OVER_K ? 0 : 2 * P_BYTES) + MISC;
  static constexpr int ROOM = CTAS == 2 ? 115456 : 231424;
  static constexpr int FIT = (ROOM - FIXED) / (KV_BYTES + AUX);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM = FIXED + STAGES * (KV_BYTES + AUX);
  static_assert(STAGES >= 2 && SMEM <= 232448, "fits the 227 KiB per-CTA limit");
  static_assert(Q_BYTES % 1024 == 0 && (!CAT || PARTS == 3), "aligned; eight rows: three parts");
};

// What a tile's position brings to its scores and weights.
struct alignas(16) Token {
  float k;       // softmax_scale * log2(e) * k_scale
  float log_v;   // log2|v_scale|
  float inv_v;   // 1 / |v_scale|, with v_scale's sign
  int32_t pos;   // its position (0 with SELECT), or kNone
};

__device__ __forceinline__ Token token_of(float k, float v_scale, int pos) {
  Token t;
  const float held = fmaxf(fabsf(v_scale), kLeastScale);
  t.k = k;
  // (A NaN makes the weight one in the rows that see the position, and only in those: a weight of 0
  // meets inv_v, which stays a number.)
  t.log_v = v_scale == v_scale ? __log2f(held) : v_scale;
  t.inv_v = copysignf(1.0f / held, v_scale);
  t.pos = pos;
  return t;
}

// Where the runs' parts of a group are, written by the CTA that has the group's first tile.
struct GroupParts {
  int32_t cta;    // that CTA
  int32_t parts;  // CTAs that share the group (1: written whole; 0: no tiles)
};

__device__ __forceinline__ void attn_flag(int bits) { atomicOr(&g_attention_status, bits); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Float16 pairs rounded to e5m2, which is their upper bytes: half a unit added, in sign and
// magnitude (halves go up; what is left over is exact, whichever way).  The value stands in bytes 1
// and 3; the low bytes mean nothing.  (A NaN becomes -0: its row's sum is NaN.)
__device__ __forceinline__ uint32_t round_e5m2(uint32_t h2) { return h2 + 0x00800080u; }
// The four e5m2 bytes of two rounded pairs.
__device__ __forceinline__ uint32_t e5m2_bytes(uint32_t lo, uint32_t hi) {
  return __byte_perm(lo, hi, 0x7531);
}
// up times what rounding left of a pair, exact.
__device__ __forceinline__ uint32_t rest_e5m2(uint32_t h2, uint32_t rounded, float up) {
  const uint32_t d = rounded & 0xFF00FF00u;
  const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&h2),
                                    *reinterpret_cast<const __half2 *>(&d)),
                            __float2half2_rn(up));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Four weights (0 .. 2^kMost) as W e5m2 parts each, a word a part.
template <int W>
__device__ __forceinline__ void weight_parts(float2 p0, float2 p1, uint32_t (&out)[W]) {
  uint32_t h0, h1;
  constexpr int FIRST = W == 4 ? 1 : 0;
  if constexpr (W == 4) {
    // A float16 holds 2^-11 of the whole weight; of what a first part leaves, 2^-15.
    uint32_t lo = round_e5m2(half2_bits(p0.x, p0.y)), hi = round_e5m2(half2_bits(p1.x, p1.y));
    out[0] = e5m2_bytes(lo, hi);
    lo &= 0xFF00FF00u, hi &= 0xFF00FF00u;
    const float2 up = make_float2(kUp2, kUp2), down = make_float2(-kUp2, -kUp2);
    p0 = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&lo)), down, __fmul2_rn(p0, up));
    p1 = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&hi)), down, __fmul2_rn(p1, up));
  }
  h0 = half2_bits(p0.x, p0.y);
  h1 = half2_bits(p1.x, p1.y);
#pragma unroll
  for (int part = FIRST; part < W; ++part) {
    const uint32_t lo = round_e5m2(h0), hi = round_e5m2(h1);
    out[part] = e5m2_bytes(lo, hi);
    if (part + 1 < W) {
      h0 = rest_e5m2(h0, lo, part == 0 ? kUp2 : kUp);
      h1 = rest_e5m2(h1, hi, part == 0 ? kUp2 : kUp);
    }
  }
}

// Each thread of the warp reads NC consecutive columns of its TMEM lane.
template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[NC]) {
  static_assert(NC == 8 || NC == 16 || NC == 32, "columns");
  if constexpr (NC == 32) {
    tmem_ld_32x32b_x32(taddr, r);
  } else if constexpr (NC == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
  }
}

// Each thread of the warp writes NC consecutive columns of its TMEM lane.
template <int NC>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[NC]) {
  static_assert(NC == 8 || NC == 16 || NC == 32, "columns");
#pragma unroll
  for (int i = 0; i < NC; i += 8)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
            taddr + i),
        "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]),
        "r"(r[i + 6]), "r"(r[i + 7])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory descriptor of an M- or N-major operand whose rows (one for each k) are ROW bytes
// with the matching swizzle: groups of eight k lie 8 * ROW bytes apart (stride offset).
template <int ROW>
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  return smem_desc_rows<ROW>(saddr);
}

// An N-major operand without swizzle: 16-byte rows of 16 n, eight k contiguous (128 bytes); the
// next eight k follow at 128 bytes (leading offset), the next 16 n at kTile * 16 (stride offset).
__device__ __forceinline__ uint64_t smem_desc_p(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128u >> 4) << 16;
  d |= static_cast<uint64_t>((kTile * 16u) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  return d;
}

constexpr uint32_t kMajorMN_A = 1u << 15, kMajorMN_B = 1u << 16;
constexpr uint32_t kE5m2_B = 1u << 10;  // (the operands' types are set one by one)

// Byte offset of byte x of row n in K-major rows of D bytes with the matching swizzle.
template <int D>
__device__ __forceinline__ uint32_t swizzled(uint32_t n, uint32_t x) {
  if constexpr (D == 128)
    return n * 128 + (x ^ ((n & 7) << 4));
  else
    return n * 64 + (x ^ (((n >> 1) & 3) << 4));
}

// Keys of the line of groups: a request (all its draft slots see one list of positions), or with
// SELECT a row.  Each has kv_heads * chunks groups.
template <bool SELECT>
__device__ __forceinline__ int key_length(const AttentionArgs &a, int key) {
  if constexpr (SELECT) {
    const int rows = a.batch * a.next_n;
    const int lo = max(0, __ldg(a.ranges + key));
    return max(0, min(__ldg(a.ranges + rows + key), a.slots) - lo);
  } else {
    return max(0, min(__ldg(a.seq_lens + key * a.sl_stride), INT_MAX - kTile));
  }
}

__device__ __forceinline__ int tiles_for(int length) {
  return length / kTile + (length % kTile != 0);
}

// A CTA's run over the line: the segments (group, first tile, tiles) in order.  Every warp walks
// its own copy, all its lanes together: keys without positions are passed over 32 at a time.
template <bool SELECT>
struct Walk {
  int64_t left;  // tiles of the run not yet handed out
  int key, group, tile, length, tiles;
  int seg_tile, seg_tiles;  // the current segment

  __device__ __forceinline__ bool next(const AttentionArgs &a, int groups, int keys) {
    if (left <= 0) return false;
    if (tile >= tiles) {  // the group is finished: the next one of this key, or the next key's
      tile = 0;
      if (++group >= groups) {
        group = 0;
        const int lane = threadIdx.x & 31;
        for (;;) {
          const int n = key + 1 + lane < keys ? key_length<SELECT>(a, key + 1 + lane) : 0;
          const unsigned some = __ballot_sync(0xffffffffu, n > 0);
          if (some != 0) {
            const int at = __ffs(some) - 1;
            key += 1 + at;
            length = __shfl_sync(0xffffffffu, n, at);
            break;
          }
          key += 32;
          if (key >= keys) return false;  // (lengths that changed under the call)
        }
        tiles = tiles_for(length);
      }
    }
    seg_tile = tile;
    seg_tiles = static_cast<int>(min(static_cast<int64_t>(tiles - tile), left));
    tile += seg_tiles;
    left -= seg_tiles;
    return true;
  }
};

// Rows of one segment: query heads of one K/V head, times draft slots unless selected.
struct RowMap {
  int b, g;
  int first, rows;  // rows [first, first + rows) of the group's key
  int t_select;     // the draft slot (SELECT)
};

template <class C>
__device__ __forceinline__ RowMap rows_of(const AttentionArgs &a, int key, int group, int chunks,
                                          int chunk_rows) {
  RowMap m;
  const int per = a.heads / a.kv_heads;
  const int all = C::SELECT ? per : per * a.next_n;
  m.g = group / chunks;
  m.first = (group - m.g * chunks) * chunk_rows;
  m.rows = min(chunk_rows, all - m.first);
  m.b = C::SELECT ? key / a.next_n : key;
  m.t_select = C::SELECT ? key - m.b * a.next_n : 0;
  return m;
}

// Draft slot and query head of row i of the group.
template <class C>
__device__ __forceinline__ int2 slot_head(const AttentionArgs &a, const RowMap &m, int i) {
  const int per = a.heads / a.kv_heads;
  i += m.first;
  if constexpr (C::SELECT) return make_int2(m.t_select, m.g * per + i);
  const int t = i / per;
  return make_int2(t, m.g * per + i - t * per);
}

struct AttnSplit {
  int32_t chunks, chunk_rows;  // of a K/V head's rows
};

// Offsets in the workspace: partial sums of slots 2 * cta (a group continued from the CTA before)
// and 2 * cta + 1 (a group that the CTA begins and does not finish): R rows of D floats, then the
// rows' maxima, then their sums; after all slots the groups' GroupParts.
template <class C>
__device__ __forceinline__ float *partial(const AttentionArgs &a, int slot) {
  return a.workspace + static_cast<int64_t>(slot) * C::R * (C::D + 2);
}

template <class C, typename T>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    k_attention(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const AttentionArgs a, const AttnSplit split, GroupParts *parts) {
  constexpr int D = C::D, R = C::R, RT = C::RT, NS = C::NS, PARTS = C::PARTS, QPARTS = C::QPARTS;
  extern __shared__ uint8_t s_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(s_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *s_kv = base;                              // [stage][K tile, V tile]
  uint8_t *s_q = s_kv + C::STAGES * C::KV_BYTES;     // [QPARTS * R][D], K-major, swizzled
  uint8_t *at = s_q + C::Q_BYTES;
  // A tile's weights, [NO / 16][kTile][16].
  uint8_t *s_p = at;
  if constexpr (!C::OVER_K) at += 2 * C::P_BYTES;
  const auto weights_of = [&](uint32_t tile, int stage) {
    return C::OVER_K ? s_kv + stage * C::KV_BYTES : s_p + (tile & 1) * C::P_BYTES;
  };
  Token *s_tok = reinterpret_cast<Token *>(at);      // [stage][kTile]
  at += C::STAGES * C::AUX;
  float *s_max = reinterpret_cast<float *>(at);      // [R][4 warps]
  at += R * 16;
  float *s_sum = reinterpret_cast<float *>(at);      // [R][4 warps]
  at += R * 16;
  float *s_rs = reinterpret_cast<float *>(at);       // [R]: a query row's power of two, undone
  at += R * 4;
  int *s_ext = reinterpret_cast<int *>(at);          // [R]: positions a row sees
  at += R * 4;
  int *s_row = reinterpret_cast<int *>(at);          // [2][R]: a row's (b, t, h) in line, by segment
  at += 2 * R * 4;
  int *s_nan = reinterpret_cast<int *>(at);          // [3][D]: see below
  at += 3 * D * 4;
  uint64_t *bars = reinterpret_cast<uint64_t *>(at);
  uint64_t *kv_full = bars, *kv_empty = bars + C::STAGES, *s_full = bars + 2 * C::STAGES,
           *p_full = s_full + 2, *pv_done = p_full + 2, *q_full = pv_done + 2, *drain = q_full + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(drain + 1);
  __shared__ int64_t s_scan[C::THREADS / 32];
  __shared__ int64_t s_begin;  // the run's first tile within its key
  __shared__ int s_key;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = a.kv_heads * split.chunks;
  const int keys = C::SELECT ? a.batch * a.next_n : a.batch;

  if (warp == 0 && lane == 0) {
    if constexpr (!C::SELECT) {
      prefetch_tensor_map(&k_map);
      prefetch_tensor_map(&v_map);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      // A loading lane's arrival; with SELECT also one when its copies have landed.
      mbar_init(&kv_full[i], C::SELECT ? 64 * C::LOADERS : 32);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    // (Two, as the softmax may finish a tile before the issuer has seen the one before.)
    mbar_init(&p_full[0], C::SOFT_WARPS);
    mbar_init(&p_full[1], C::SOFT_WARPS);
    mbar_init(&pv_done[0], 1);
    mbar_init(&pv_done[1], 1);
    mbar_init(q_full, C::SOFT_WARPS);
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, C::TMEM);
    tmem_relinquish();
  }
  for (int i = tid; i < 3 * D; i += C::THREADS) s_nan[i] = 0;
  griddep_wait();
  griddep_launch_dependents();

  // ---- the run ---------------------------------------------------------------------------------
  const int per = (keys + C::THREADS - 1) / C::THREADS;
  const int k_lo = min(tid * per, keys), k_hi = min(k_lo + per, keys);
  int64_t mine = 0;
  for (int k = k_lo; k < k_hi; ++k) mine += tiles_for(key_length<C::SELECT>(a, k));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  total *= groups;
  // (No more runs than tiles: a group's parts lie in consecutive CTAs.)
  const int64_t runs = max(static_cast<int64_t>(1), min(total, static_cast<int64_t>(gridDim.x)));
  int64_t f0 = total, f1 = total;
  if (blockIdx.x < runs) {
    f0 = run_begin(total, runs, blockIdx.x);
    f1 = run_begin(total, runs, blockIdx.x + 1);
  }
  if (f0 < f1 && f0 >= before * groups && f0 < (before + mine) * groups) {
    for (int k = k_lo; k < k_hi; ++k) {
      const int n = tiles_for(key_length<C::SELECT>(a, k));
      if (f0 < (before + n) * groups) {
        s_key = k;
        s_begin = f0 - before * groups;
        break;
      }
      before += n;
    }
  }
  __syncthreads();

  const uint32_t tmem = *s_tmem;
  Walk<C::SELECT> w;
  w.left = f1 - f0;
  w.seg_tile = w.seg_tiles = 0;
  if (w.left > 0) {
    w.key = s_key;
    w.length = key_length<C::SELECT>(a, w.key);
    w.tiles = tiles_for(w.length);
    const int64_t at0 = s_begin;
    w.group = at0 < INT_MAX ? static_cast<int>(at0) / w.tiles : static_cast<int>(at0 / w.tiles);
    w.tile = static_cast<int>(at0 - static_cast<int64_t>(w.group) * w.tiles);
  }
  bool ok = true;
  uint32_t issued = 0;  // producer: tiles whose copies were started; MMA: nothing
  int stage = 0;
  uint32_t phase = 0;

  if (warp == 0 || warp >= 2 + C::SOFT_WARPS) {
    // ============================== loaders =====================================================
    const uint64_t policy = l2_policy_evict_first();
    const int shift = a.block_size == 32 ? 5 : a.block_size == 64 ? 6 : 7;
    const float z_unit = a.scale * 1.4426950408889634f;  // scores in units of ln 2
    const auto stage_free = [&]() {
      ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[stage], phase ^ 1, kWaitNs));
      return ok;
    };
    const auto next_stage = [&]() {
      ++issued;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    };
    if constexpr (C::SELECT) {
      // A lane looks after EACH tokens of a tile, 32 apart: position, then page, then the page's
      // scales, each read one tile further ahead than the next (segments and all), so that a tile
      // pays for one memory round trip and not for three.
      constexpr int EACH = 4 / C::LOADERS;
      const int loader = warp == 0 ? 0 : warp - 1 - C::SOFT_WARPS;
      const int token0 = loader * 32 * EACH + lane;
      struct Ahead {
        int pos[EACH];
        const int32_t *table;
        int extent, g;
        bool live;
      };
      const int2 *cand = nullptr;
      Ahead far{};
      int slot = 0, end = 0;  // of the walk: the tile's first slot, and the segment's end
      const auto positions = [&]() {
        if (slot >= end) {
          far.live = w.next(a, groups, keys);
          if (!far.live) return;
          const RowMap m = rows_of<C>(a, w.key, w.group, split.chunks, split.chunk_rows);
          far.table = a.block_tables + m.b * a.bt_stride;
          far.extent = __ldg(a.seq_lens + m.b * a.sl_stride) - a.next_n + m.t_select + 1;
          far.g = m.g;
          cand = a.candidates + w.key * a.cand_stride + max(0, __ldg(a.ranges + w.key));
          slot = w.seg_tile * kTile;
          end = min((w.seg_tile + w.seg_tiles) * kTile, w.length);
        }
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const int s = slot + token0 + 32 * j;
          far.pos[j] = s < end ? __ldg(&cand[s].x) : -1;
        }
        slot += kTile;
      };
      // Each token's row of the pool, or -1.
      const auto pool_rows = [&](int (&row)[EACH]) {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          row[j] = -1;
          if (far.live && far.pos[j] >= 0 && far.pos[j] < far.extent) {
            const int blk = far.pos[j] >> shift;
            const int id = blk < a.bt_width ? __ldg(far.table + blk) : -1;
            if (id >= 0 && id < a.num_blocks)
              row[j] = ((id * a.kv_heads + far.g) << shift) + (far.pos[j] & (a.block_size - 1));
            else
              bad = true;
          }
        }
        if (bad) attn_flag(IDX_DEV_BAD_PAGE);
      };
      const auto scales = [&](const int (&row)[EACH], float (&ks)[EACH], float (&vs)[EACH]) {
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          ks[j] = row[j] >= 0 ? __ldg(a.k_scales + (row[j] >> shift)) : 0.0f;
          vs[j] = row[j] >= 0 ? __ldg(a.v_scales + (row[j] >> shift)) : 0.0f;
        }
      };
      int row0[EACH], row1[EACH];
      float ks0[EACH], vs0[EACH], ks1[EACH], vs1[EACH];
      positions();
      bool live0 = far.live, live1 = false, primed = false;
      pool_rows(row0);
      scales(row0, ks0, vs0);
      if (live0) positions();
      // 16 bytes a lane and copy: a warp's copy is 512 / D rows of K or of V, stored with the swizzle
      // that the products expect.  (As gathers of four rows by the TMA unit, 64 a tile, a tile took
      // 2.1 us to issue, and the serving mix's 343 MB of selected rows 176 us.)
      constexpr int kLanes = D / 16, kRows = 32 / kLanes;
      const int x = (lane % kLanes) * 16, sub = lane / kLanes;
      while (live0) {
        if (primed) scales(row1, ks1, vs1);
        if (!stage_free()) break;
        uint8_t *kt = s_kv + stage * C::KV_BYTES, *vt = kt + kTile * D;
#pragma unroll
        for (int q = 0; q < EACH; ++q)
#pragma unroll
          for (int j = 0; j < 32 / kRows; ++j) {
            const int n = j * kRows + sub;  // lane n's q-th token
            const int row = __shfl_sync(0xffffffffu, row0[q], n);
            if (row < 0) continue;  // (the softmax clears the value row of a token that is not)
            const int64_t src = static_cast<int64_t>(row) * D + x;
            const uint32_t dst = swizzled<D>(token0 - lane + 32 * q + n, x);
            cp_async_16(kt + dst, a.k_pool + src, policy);
            cp_async_16(vt + dst, a.v_pool + src, policy);
          }
        if (!primed) {  // (the first tile's copies go out before anything waits for the second's ids)
          primed = true;
          pool_rows(row1);
          live1 = far.live;
          if (live1) positions();
          scales(row1, ks1, vs1);
        }
#pragma unroll
        for (int j = 0; j < EACH; ++j)
          s_tok[stage * kTile + token0 + 32 * j] =
              token_of(ks0[j] * z_unit, vs0[j], row0[j] >= 0 ? 0 : kNone);
        cp_async_arrive_noinc(&kv_full[stage]);
        mbar_arrive(&kv_full[stage]);
        next_stage();
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          row0[j] = row1[j];
          ks0[j] = ks1[j];
          vs0[j] = vs1[j];
        }
        live0 = live1;
        pool_rows(row1);
        live1 = far.live;
        if (live1) positions();
      }
    } else {
      while (ok && w.next(a, groups, keys)) {
        const RowMap m = rows_of<C>(a, w.key, w.group, split.chunks, split.chunk_rows);
        const int32_t *table = a.block_tables + m.b * a.bt_stride;
        // A lane reads one page's id and scales, 32 pages ahead of the ones in hand: the ids while
        // the first tile of a batch is issued, their scales after it.
        const int n_pages = (w.length + a.block_size - 1) >> shift;
        const int per_tile = kTile >> shift;
        int first = w.seg_tile * per_tile;  // the page of lane 0
        const auto ids = [&](int page) {
          if (page >= n_pages || page >= (w.seg_tile + w.seg_tiles) * per_tile) return -1;
          const int id = page < a.bt_width ? __ldg(table + page) : -1;
          if (id >= 0 && id < a.num_blocks) return id;
          attn_flag(IDX_DEV_BAD_PAGE);
          return -1;
        };
        int id = ids(first + lane), id_next = -1;
        float ks = 0.0f, vs = 0.0f, ks_next = 0.0f, vs_next = 0.0f;
        const auto scales = [&](int block, float &k, float &v) {
          const int page = block * a.kv_heads + m.g;
          k = block >= 0 ? __ldg(a.k_scales + page) : 0.0f;
          v = block >= 0 ? __ldg(a.v_scales + page) : 0.0f;
        };
        scales(id, ks, vs);
        id_next = ids(first + 32 + lane);
        Token mine = token_of(ks * z_unit, vs, 0);
        bool fetch = true;  // the next batch's scales are still to be read
        for (int i = w.seg_tile; i < w.seg_tile + w.seg_tiles; ++i) {
          if (i * per_tile >= first + 32) {
            first += 32;
            id = id_next;
            mine = token_of(ks_next * z_unit, vs_next, 0);
            id_next = ids(first + 32 + lane);
            fetch = true;
          }
          const int p = i * kTile + lane * 4;
          const int from = (p >> shift) - first;  // the lane that holds this lane's page
          const int block = __shfl_sync(0xffffffffu, id, from);
          Token tok;
          tok.k = __shfl_sync(0xffffffffu, mine.k, from);
          tok.log_v = __shfl_sync(0xffffffffu, mine.log_v, from);
          tok.inv_v = __shfl_sync(0xffffffffu, mine.inv_v, from);
          if (!stage_free()) break;
          uint8_t *kt = s_kv + stage * C::KV_BYTES, *vt = kt + kTile * D;
          if (block >= 0 && (p & (a.block_size - 1)) == 0) {
            const int row = (block * a.kv_heads + m.g) << shift;
            mbar_expect_tx(&kv_full[stage], 2 * D * a.block_size);
            tma_load_2d(kt + lane * 4 * D, &k_map, &kv_full[stage], 0, row, policy);
            tma_load_2d(vt + lane * 4 * D, &v_map, &kv_full[stage], 0, row, policy);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            tok.pos = block >= 0 && p + j < w.length ? p + j : kNone;
            s_tok[stage * kTile + lane * 4 + j] = tok;
          }
          mbar_arrive(&kv_full[stage]);
          next_stage();
          if (fetch) {
            scales(id_next, ks_next, vs_next);
            fetch = false;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ============================== MMA issuer ==================================================
    constexpr uint32_t idesc_s = idesc_e4m3_f32(kTile, NS) | kE5m2_B;
    constexpr uint32_t idesc_o = idesc_e4m3_f32(D, C::NO) | kE5m2_B | kMajorMN_A | kMajorMN_B;
    const uint64_t q_desc = smem_desc_rows<D>(smem_addr(s_q));
    const uint32_t o_tmem = tmem + 2 * NS;
    uint32_t tile = 0, seg = 0;
    const auto scores = [&](uint32_t n, int st) {  // S of tile n of the run, from stage st
      const uint64_t k_desc = smem_desc_rows<D>(smem_addr(s_kv + st * C::KV_BYTES));
#pragma unroll
      for (int part = 0; part < C::PASSES; ++part)
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          mma_f8f6f4(tmem + (n & 1) * NS, k_desc + 2 * k, q_desc + part * (R * D >> 4) + 2 * k,
                     idesc_s, part + k > 0);
      mma_commit(&s_full[n & 1]);
    };
    const auto keys_here = [&]() {
      // (The selected rows were written by ordinary asynchronous copies.)
      if constexpr (C::SELECT) fence_proxy_async_shared();
      tc_fence_after_sync();
    };
    // One thread's work: the segment's products; false if a wait gave up.
    const auto segment = [&]() {
      if (!mbar_wait(q_full, seg & 1, kWaitNs)) return false;
      tc_fence_after_sync();
      bool ahead = false;  // S of the tile has been issued already
      for (int i = 0; i < w.seg_tiles; ++i, ++tile) {
        if (!ahead) {
          if (!mbar_wait(&kv_full[stage], phase, kWaitNs)) return false;
          keys_here();
          scores(tile, stage);
        }
        // The next tile's scores, if its keys are here, before this tile's weights are.
        const int next = stage + 1 == C::STAGES ? 0 : stage + 1;
        const uint32_t next_phase = next == 0 ? phase ^ 1 : phase;
        ahead = i + 1 < w.seg_tiles && mbar_try_wait(&kv_full[next], next_phase);
        if (ahead) {
          keys_here();
          scores(tile + 1, next);
        }
        if (!mbar_wait(&p_full[tile & 1], (tile >> 1) & 1, kWaitNs)) return false;
        tc_fence_after_sync();
        const uint64_t v_desc = smem_desc_mn<D>(smem_addr(s_kv + stage * C::KV_BYTES + kTile * D));
        const uint64_t p_desc = smem_desc_p(smem_addr(weights_of(tile, stage)));
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k)
          mma_f8f6f4(o_tmem, v_desc + k * (32 * D >> 4), p_desc + k * (512 >> 4), idesc_o, i + k > 0);
        mma_commit(&pv_done[tile & 1]);
        mma_commit(&kv_empty[stage]);
        stage = next;
        phase = next_phase;
      }
      return true;
    };
    while (ok && w.next(a, groups, keys)) {
      if (lane == 0) ok = segment();
      ok = __shfl_sync(0xffffffffu, ok, 0) != 0;
      ++seg;
    }
    if (lane == 0) mma_commit(drain);
    __syncwarp();
  } else {
    // ============================== softmax =====================================================
    const int wg = (warp - 2) >> 2, quarter = warp & 3;
    const int r0 = wg * RT;                      // the thread's rows
    const int token = quarter * 32 + lane;       // the thread's position in the tile
    // The thread's dimension of the output, or -1 (M = 64: 16 lanes of each quarter).
    const int dim = D == 128 ? token : lane < 16 ? quarter * 16 + lane : -1;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t tile = 0;
    int seg = 0;
    // Once a wait has given up the warp goes on without waiting, so that the barriers below (which
    // have no limit of their own) find every warp of the warpgroup.
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs));
    };
    const auto any_of_group = [&](bool x) {
      uint32_t y;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
          : "=r"(y)
          : "r"(static_cast<uint32_t>(x)), "r"(1 + wg)
          : "memory");
      return y != 0;
    };
    const auto sync_group = [&]() {
      asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + wg) : "memory");
    };
    while (w.next(a, groups, keys)) {
      const RowMap m = rows_of<C>(a, w.key, w.group, split.chunks, split.chunk_rows);
      const int len = C::SELECT ? 0 : w.length;
      ++seg;
      // ---- the rows' queries, in parts -----------------------------------------------------------
      {
        constexpr int LANES = D / 8;  // eight elements a lane
        constexpr int PER = 128 / LANES;                       // rows at a time
        constexpr int ROUNDS = RT > PER ? RT / PER : 1;
        const int x = (tid & (LANES - 1)) * 8;
        const int mine = (tid - 64 - wg * 128) / LANES;
        Piece<T, 8> v[ROUNDS];
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
          const int r = r0 + mine + i * PER;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i].e[j] = from_f32<T>(0.0f);
          if (r < r0 + RT && r < m.rows) {
            const int2 th = slot_head<C>(a, m, r);
            v[i] = load_piece<T, 8>(static_cast<const T *>(a.q) + m.b * a.q_batch +
                                    th.x * a.q_token + th.y * a.q_head + x);
          }
        }
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
          const int r = r0 + mine + i * PER;
          if (r >= r0 + RT) break;  // (whole warps)
          const int2 th = slot_head<C>(a, m, r);
          float f[8], amax = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[j] = to_f32(v[i].e[j]);
            amax = fmaxf(amax, fabsf(f[j]));
          }
#pragma unroll
          for (int o = 1; o < LANES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // 2^e <= amax < 2^(e+1); rows below 2^-100 keep their scores to 2^-131 only.
          const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
          const float up = e > 127 ? __int_as_float(0x7FC00000)  // an infinity: the row is NaN
                                   : __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - 14 + min(e, 127)) << 23);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= up;
#pragma unroll
          for (int part = 0; part < QPARTS; ++part) {
            const uint2 b = make_uint2(e5m2x4(f[0], f[1], f[2], f[3]), e5m2x4(f[4], f[5], f[6], f[7]));
            *reinterpret_cast<uint2 *>(s_q + swizzled<D>(part * R + r, x)) = b;
            if (part + 1 < QPARTS) {
              const float2 b0 = e5m2x2_to_f32(b.x), b1 = e5m2x2_to_f32(b.x >> 16);
              const float2 b2 = e5m2x2_to_f32(b.y), b3 = e5m2x2_to_f32(b.y >> 16);
              f[0] -= b0.x, f[1] -= b0.y, f[2] -= b1.x, f[3] -= b1.y;
              f[4] -= b2.x, f[5] -= b2.y, f[6] -= b3.x, f[7] -= b3.y;
            }
          }
          if (x == 0) {
            s_rs[r] = down;
            s_row[(seg & 1) * R + r] = (m.b * a.next_n + th.x) * a.heads + th.y;
            s_ext[r] = r >= m.rows ? 0 : C::SELECT ? 1 : max(0, len - a.next_n + th.x + 1);
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        wait(q_full, (seg - 1) & 1);
      }
      // Pairs of rows, for the packed float32 operations: the sums and minus the references.
      float2 sum[RT / 2], nref[RT / 2];
      constexpr bool kHoldRs = RT <= 8;  // (more rows would spill: read from shared memory then)
      float2 rs[kHoldRs ? RT / 2 : 1];
      const float2 *rs_at = reinterpret_cast<const float2 *>(s_rs + r0);
#pragma unroll
      for (int r = 0; r < RT / 2; ++r) {
        sum[r] = nref[r] = make_float2(0.0f, 0.0f);
        if constexpr (kHoldRs) rs[r] = rs_at[r];
      }
      uint32_t unset = 0xFFFFFFFFu;  // bit r: row r0 + r has seen nothing yet, and ref[r] means nothing
      // Positions below this are seen by every row of the segment.
      const int all_see = C::SELECT ? kNone : len - a.next_n + 1 + (slot_head<C>(a, m, 0).x);
      for (int i = 0; i < w.seg_tiles; ++i, ++tile) {
        wait(&kv_full[stage], phase);
        wait(&s_full[tile & 1], (tile >> 1) & 1);
        tc_fence_after_sync();
        const Token tok = s_tok[stage * kTile + token];
        float2 y[RT / 2];  // the weights' logarithms
        {
          uint32_t v[RT];
          tmem_ld_cols<RT>(lane_base + (tile & 1) * NS + r0, v);
          if constexpr (C::CAT) {
            uint32_t u[RT], t[RT];
            tmem_ld_cols<RT>(lane_base + (tile & 1) * NS + R, u);
            tmem_ld_cols<RT>(lane_base + (tile & 1) * NS + 2 * R, t);
            tmem_ld_wait();
            reg_fence(v);
            reg_fence(u);
            reg_fence(t);
#pragma unroll
            for (int r = 0; r < RT; ++r)
              v[r] = __float_as_uint(__uint_as_float(v[r]) +
                                     (__uint_as_float(u[r]) + __uint_as_float(t[r])));
          } else {
            tmem_ld_wait();
            reg_fence(v);
          }
          const float2 k2 = make_float2(tok.k, tok.k), lv2 = make_float2(tok.log_v, tok.log_v);
#pragma unroll
          for (int r = 0; r < RT / 2; r += 2) {
            float4 f;
            if constexpr (kHoldRs)
              f = make_float4(rs[r].x, rs[r].y, rs[r + 1].x, rs[r + 1].y);
            else
              f = *reinterpret_cast<const float4 *>(rs_at + r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 s2 = make_float2(__uint_as_float(v[2 * (r + h)]),
                                            __uint_as_float(v[2 * (r + h) + 1]));
              y[r + h] = __ffma2_rn(s2, __fmul2_rn(h ? make_float2(f.z, f.w) : make_float2(f.x, f.y), k2),
                                    __fadd2_rn(lv2, nref[r + h]));
            }
          }
        }
        const bool seen = tok.pos < all_see;
        if (!__all_sync(0xffffffffu, seen)) {
          if (!seen) {
#pragma unroll
            for (int r = 0; r < RT / 2; ++r) {
              if (tok.pos >= s_ext[r0 + 2 * r]) y[r].x = -INFINITY;
              if (tok.pos >= s_ext[r0 + 2 * r + 1]) y[r].y = -INFINITY;
            }
          }
        }
        float most = fmaxf(y[0].x, y[0].y);
#pragma unroll
        for (int r = 1; r < RT / 2; ++r) most = fmaxf(most, fmaxf(y[r].x, y[r].y));
        bool move = most > kMost;
        if (unset != 0) {
#pragma unroll
          for (int r = 0; r < RT / 2; ++r) {
            move |= ((unset >> (2 * r)) & 1u) != 0 && y[r].x != -INFINITY;
            move |= ((unset >> (2 * r + 1)) & 1u) != 0 && y[r].y != -INFINITY;
          }
        }
        if (any_of_group(move)) {
          // Some weight would leave e5m2's range, or a row sees its first position: the references
          // move to the maxima so far.
          float mine = -INFINITY;  // lane r: row r0 + r
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float x = warp_max(r & 1 ? y[r / 2].y : y[r / 2].x);
            if (lane == r) mine = x;
          }
          if (lane < RT) s_max[(r0 + lane) * 4 + quarter] = mine;
          sync_group();
          float up = 0.0f, keep = 1.0f;
          bool set = false;
          if (lane < RT) {
            const float4 t4 = *reinterpret_cast<const float4 *>(s_max + (r0 + lane) * 4);
            const float t = fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
            set = t > -INFINITY;
            if ((unset >> lane) & 1u) {
              up = set ? t - kTop : 0.0f;  // (its sums are 0: nothing to rescale)
            } else {
              up = fmaxf(t - kTop, 0.0f);
              keep = fast_exp2(-up);
            }
          }
          unset &= ~__ballot_sync(0xffffffffu, set);
          sync_group();  // (s_max may be written again)
#pragma unroll
          for (int r = 0; r < RT / 2; ++r) {
            const float2 d = make_float2(-__shfl_sync(0xffffffffu, up, 2 * r),
                                         -__shfl_sync(0xffffffffu, up, 2 * r + 1));
            y[r] = __fadd2_rn(y[r], d);
            nref[r] = __fadd2_rn(nref[r], d);
            sum[r].x *= __shfl_sync(0xffffffffu, keep, 2 * r);
            sum[r].y *= __shfl_sync(0xffffffffu, keep, 2 * r + 1);
          }
          if (i > 0) {
            wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
            tc_fence_after_sync();
#pragma unroll 1
            for (int part = 0; part < PARTS; ++part) {
              const uint32_t o_at = lane_base + 2 * NS + part * R + r0;
              uint32_t v[RT];
              tmem_ld_cols<RT>(o_at, v);
              tmem_ld_wait();
              reg_fence(v);
#pragma unroll
              for (int r = 0; r < RT; ++r)
                v[r] = __float_as_uint(__uint_as_float(v[r]) * __shfl_sync(0xffffffffu, keep, r));
              tmem_st_cols<RT>(o_at, v);
            }
            tmem_st_wait();
          }
        }
        // ---- weights, their parts, the running sums ------------------------------------------------
        // The weights' buffer was last read by the product two tiles ago.  (In the place of the keys
        // they need not wait; but whoever waits for a barrier has to see all its phases.)
        if (tile >= 2) wait(&pv_done[tile & 1], ((tile >> 1) - 1) & 1);
        uint8_t *sp = weights_of(tile, stage) + token * 16;
        const float inv_v = fabsf(tok.inv_v);
        // The weights of a position whose value scale is negative or 0 (as good as): rare, so asked
        // of the whole warp.
        const bool odd = __any_sync(0xffffffffu, tok.inv_v < 0.0f || inv_v >= 1.0f / kLeastScale);
        const uint32_t flip = tok.inv_v < 0.0f ? 0x80808080u : 0u;
        const uint32_t live = inv_v < 1.0f / kLeastScale ? 0xFFFFFFFFu : 0u;
        uint32_t bytes[PARTS][4];
        const float2 inv2 = make_float2(inv_v, inv_v);
#pragma unroll
        for (int r = 0; r < RT; r += 4) {
          float2 p[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[j] = make_float2(fast_exp2(y[r / 2 + j].x), fast_exp2(y[r / 2 + j].y));
            sum[r / 2 + j] = __ffma2_rn(p[j], inv2, sum[r / 2 + j]);
          }
          uint32_t four[PARTS];
          weight_parts<PARTS>(p[0], p[1], four);
#pragma unroll
          for (int part = 0; part < PARTS; ++part) bytes[part][(r / 4) % 4] = four[part];
          if (odd && (r % 16 == 12 || r + 4 == RT)) {
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
              for (int q = 0; q < (RT < 16 ? RT / 4 : 4); ++q)
                bytes[part][q] = (bytes[part][q] & live) ^ flip;
          }
          if constexpr (C::CAT) {  // a group of 16 n: the first two parts of the eight rows; then the third
            if (r == 4) {
              *reinterpret_cast<uint4 *>(sp) =
                  make_uint4(bytes[0][0], bytes[0][1], bytes[1][0], bytes[1][1]);
              *reinterpret_cast<uint2 *>(sp + kTile * 16) = make_uint2(bytes[2][0], bytes[2][1]);
            }
          } else if (r % 16 == 12) {
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              *reinterpret_cast<uint4 *>(sp + (part * R + r0 + r - 12) / 16 * (kTile * 16)) =
                  make_uint4(bytes[part][0], bytes[part][1], bytes[part][2], bytes[part][3]);
          }
        }
        // A value that some row does not see must not meet its weight of 0 as a NaN (a code of the
        // cache, or bytes that were never written): what no row sees becomes 0; in the newest
        // tokens, which only the later draft slots see, a NaN becomes 0 and is noted in s_nan (as
        // this segment's number) for the rows that do see it.
        if (wg == 0 && !seen) {
          uint8_t *v = s_kv + stage * C::KV_BYTES + kTile * D;
          if (tok.pos == kNone) {
            for (int x = 0; x < D; x += 16)
              *reinterpret_cast<uint4 *>(v + token * D + x) = make_uint4(0, 0, 0, 0);
          } else {
            for (int x = 0; x < D; x += 4) {
              const uint32_t at4 = swizzled<D>(token, x);
              const uint32_t four = *reinterpret_cast<const uint32_t *>(v + at4);
              if ((((four & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) == 0) continue;
              for (int e = 0; e < 4; ++e)
                if (((four >> (8 * e)) & 0x7F) == 0x7F) {
                  v[at4 + e] = 0;
                  s_nan[(len - 1 - tok.pos) * D + x + e] = seg;
                }
            }
          }
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[tile & 1]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      // ---- the segment's sums ------------------------------------------------------------------------
      wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
      tc_fence_after_sync();
      float acc[RT];
#pragma unroll
      for (int part = PARTS - 1; part >= 0; --part) {
        uint32_t v[RT];
        tmem_ld_cols<RT>(lane_base + 2 * NS + part * R + r0, v);
        tmem_ld_wait();
        reg_fence(v);
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[r] = part == PARTS - 1
                       ? __uint_as_float(v[r])
                       : fmaf(acc[r], 1.0f / (part == 0 ? kUp2 : kUp), __uint_as_float(v[r]));
      }
      tc_fence_before_sync();
      float m_run = kRefNone;  // lane r: the reference of row r0 + r
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (lane == r && ((unset >> r) & 1u) == 0) m_run = -(r & 1 ? nref[r / 2].y : nref[r / 2].x);
      // ---- the segment's result ----------------------------------------------------------------------
      // (s_rs and s_ext are not read past the barrier below: the next segment's are written then.)
      if (!C::SELECT && a.next_n > 1) {
        for (int u = 0; u < a.next_n - 1; ++u) {
          const bool noted = dim >= 0 && s_nan[u * D + max(dim, 0)] == seg;
          if (!__any_sync(0xffffffffu, noted)) continue;
#pragma unroll
          for (int r = 0; r < RT; ++r)
            if (noted && len - 1 - u < s_ext[r0 + r]) acc[r] = __int_as_float(0x7FC00000);
        }
      }
      // The lanes' sums, a row to a lane: halves of the rows change places at each step.
      {
        float v[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) v[r] = r & 1 ? sum[r / 2].y : sum[r / 2].x;
#pragma unroll
        for (int o = RT / 2; o > 0; o >>= 1)
#pragma unroll
          for (int r = 0; r < o; ++r) {
            const float send = (lane & o) ? v[r] : v[r + o];
            const float hold = (lane & o) ? v[r + o] : v[r];
            v[r] = hold + __shfl_xor_sync(0xffffffffu, send, o);
          }
#pragma unroll
        for (int o = RT; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        if (lane < RT) s_sum[(r0 + lane) * 4 + quarter] = v[0];
      }
      sync_group();
      float l = 0.0f;  // lane r: the sum of row r0 + r
      if (lane < RT) {
        const float4 t4 = *reinterpret_cast<const float4 *>(s_sum + (r0 + lane) * 4);
        l = (t4.x + t4.y) + (t4.z + t4.w);
      }
      const bool from_start = w.seg_tile == 0, to_end = w.seg_tile + w.seg_tiles == w.tiles;
      const int64_t gid = static_cast<int64_t>(w.key) * groups + w.group;
      if (from_start && wg == 0 && quarter == 2 && lane == 0) {
        // The run that holds the group's last tile has its last part.
        int n = 1;
        if (!to_end) {
          const int64_t last = f1 - 1 + (w.tiles - (w.seg_tile + w.seg_tiles));
          n = run_of(total, runs, last) - static_cast<int>(blockIdx.x) + 1;
        }
        parts[gid] = GroupParts{static_cast<int>(blockIdx.x), n};
      }
      if (from_start && to_end) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int *rows = s_row + (seg & 1) * R + r0;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float f = __shfl_sync(0xffffffffu, inv, r);
          if (r0 + r < m.rows && dim >= 0)
            static_cast<T *>(a.out)[static_cast<int64_t>(rows[r]) * D + dim] =
                from_f32<T>(f == 0.0f ? 0.0f : acc[r] * f);
        }
        if (a.lse != nullptr && quarter == 0 && lane < RT && r0 + lane < m.rows)
          a.lse[rows[lane]] = l == 0.0f ? -INFINITY : (m_run + log2f(l)) * 0.6931471805599453f;
      } else {
        float *ws = partial<C>(a, 2 * blockIdx.x + (from_start ? 1 : 0));
#pragma unroll
        for (int r = 0; r < RT; ++r)
          if (r0 + r < m.rows && dim >= 0) ws[(r0 + r) * D + dim] = acc[r];
        if (quarter == 0 && lane < RT) {
          ws[R * D + r0 + lane] = m_run;
          ws[R * D + R + r0 + lane] = l;
        }
      }
    }
  }

  // Keys without positions: their rows are zeros, their groups have no parts.
  for (int k = blockIdx.x; k < keys; k += gridDim.x) {
    if (key_length<C::SELECT>(a, k) > 0) continue;
    for (int g = tid; g < groups; g += C::THREADS)
      parts[static_cast<int64_t>(k) * groups + g] = GroupParts{0, 0};
    const int slots = C::SELECT ? 1 : a.next_n;
    const int64_t row0 = static_cast<int64_t>(k) * slots * a.heads;
    T *out = static_cast<T *>(a.out) + row0 * D;
    for (int i = tid; i < slots * a.heads * D / 8; i += C::THREADS)
      reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr)
      for (int i = tid; i < slots * a.heads; i += C::THREADS) a.lse[row0 + i] = -INFINITY;
  }

  // ---- teardown ----------------------------------------------------------------------------------
  if (__syncthreads_or(!ok)) {
    // A wait gave up: let the copies and products in flight end before the memory is given back.
    if (!ok) attn_flag(IDX_DEV_WAIT_TIMEOUT);
    if (warp == 0 && lane == 0) {
      const uint32_t tail = issued < C::STAGES ? issued : C::STAGES;
      for (uint32_t d = 1; d <= tail; ++d) {
        const uint32_t n = issued - d;
        if (!mbar_wait(&kv_full[n % C::STAGES], (n / C::STAGES) & 1, kWaitNs))
          attn_flag(IDX_DEV_WAIT_TIMEOUT);
      }
    }
  }
  if (warp == 1 && lane == 0 && !mbar_wait(drain, 0, kWaitNs)) attn_flag(IDX_DEV_WAIT_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM);
}

constexpr int kJoinThreads = 256;

// Joins the parts of one group's rows: block (group, y) takes rows y, y + gridDim.y, ...; its
// warps share a row's parts, eight at a time (their maxima, sums and vectors read at once, none
// waiting for another), and the warps' results are joined in order.
template <class C, typename T>
__global__ void __launch_bounds__(kJoinThreads)
    k_attention_join(const AttentionArgs a, const AttnSplit split, const GroupParts *parts) {
  constexpr int D = C::D, R = C::R, W = kJoinThreads / 32, E = D / 32, AT_ONCE = 8;
  __shared__ float s_o[W][D], s_m[W], s_l[W];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t gid = blockIdx.x;
  const GroupParts p = parts[gid];
  if (p.parts <= 1) return;
  const int groups = a.kv_heads * split.chunks;
  const int key = static_cast<int>(gid / groups);
  const RowMap m = rows_of<C>(a, key, static_cast<int>(gid - static_cast<int64_t>(key) * groups),
                              split.chunks, split.chunk_rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = blockIdx.y; r < m.rows; r += gridDim.y) {
    float top = kRefNone, l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    for (int i0 = warp; i0 < p.parts; i0 += W * AT_ONCE) {
      float pm[AT_ONCE], pl[AT_ONCE];
      Piece<float, E> v[AT_ONCE];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const int i = i0 + j * W;
        pm[j] = kRefNone;
        pl[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[j].e[e] = 0.0f;
        if (i < p.parts) {
          const float *ws = partial<C>(a, 2 * (p.cta + i) + (i == 0));
          pm[j] = ws[R * D + r];
          pl[j] = ws[R * D + R + r];
          v[j] = load_piece<float, E>(ws + r * D + lane * E);
        }
      }
      float now = top;
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) now = fmaxf(now, pm[j]);
      const float keep = fast_exp2(top - now);
      top = now;
      l *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const float f = fast_exp2(pm[j] - now);
        l += f * pl[j];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * v[j].e[e];
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    if (lane == 0) {
      s_m[warp] = top;
      s_l[warp] = l;
    }
    __syncthreads();
    if (threadIdx.x < D) {
#pragma unroll
      for (int y = 0; y < W; ++y) top = fmaxf(top, s_m[y]);
      float x = 0.0f, all = 0.0f;
#pragma unroll
      for (int y = 0; y < W; ++y) {
        const float f = fast_exp2(s_m[y] - top);
        x += f * s_o[y][threadIdx.x];
        all += f * s_l[y];
      }
      const int2 th = slot_head<C>(a, m, r);
      const int64_t row = (static_cast<int64_t>(m.b) * a.next_n + th.x) * a.heads + th.y;
      static_cast<T *>(a.out)[row * D + threadIdx.x] = from_f32<T>(all == 0.0f ? 0.0f : x / all);
      if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[row] = all == 0.0f ? -INFINITY : (top + log2f(all)) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

// Rows that share a K/V head, cut into chunks of at most 64, and the kernel's R for a chunk.
struct AttnShape {
  int chunks, chunk_rows, r;
};
inline AttnShape attn_shape(int rows, bool f16) {
  AttnShape s;
  s.chunks = (rows + 63) / 64;
  s.chunk_rows = (rows + s.chunks - 1) / s.chunks;
  s.r = s.chunk_rows <= 8 && !f16 ? 8 : s.chunk_rows <= 16 ? 16 : s.chunk_rows <= 32 ? 32 : 64;
  return s;
}

inline int64_t attn_slots_bytes(int64_t ctas, int r, int dim) {
  return (2 * ctas * r * (dim + 2) * 4 + 255) / 256 * 256;
}

template <class C, typename T>
cudaError_t launch_cfg(const CUtensorMap &k_map, const CUtensorMap &v_map, const AttentionArgs &a,
                       const AttnShape &s, int sms, cudaStream_t stream) {
  static PerDeviceOnce configured;
  cudaError_t e = configured.run([] {
    return cudaFuncSetAttribute(k_attention<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::SMEM);
  });
  if (e != cudaSuccess) return e;
  const int ctas = sms * C::CTAS;
  const AttnSplit split{s.chunks, s.chunk_rows};
  auto *parts = reinterpret_cast<GroupParts *>(reinterpret_cast<uint8_t *>(a.workspace) +
                                               attn_slots_bytes(ctas, C::R, C::D));
  e = launch_dependent(k_attention<C, T>, dim3(ctas), dim3(C::THREADS), C::SMEM, stream, k_map,
                       v_map, a, split, parts);
  if (e != cudaSuccess) return e;
  const int64_t groups = static_cast<int64_t>(C::SELECT ? a.batch * a.next_n : a.batch) *
                         a.kv_heads * s.chunks;
  // A row a block while that is at most eight blocks an SM (groups that were not cut leave at once).
  const int64_t spread = (8 * sms + groups - 1) / groups;
  const int y = static_cast<int>(spread < s.chunk_rows ? spread : s.chunk_rows);
  return launch_dependent(k_attention_join<C, T>, dim3(static_cast<unsigned>(groups), y),
                          dim3(kJoinThreads), 0, stream, a, split, parts);
}

template <int D, bool SELECT>
cudaError_t launch_rows(const CUtensorMap &k_map, const CUtensorMap &v_map, const AttentionArgs &a,
                        int dtype, int sms, cudaStream_t stream) {
  const bool f16 = dtype == IDX_DTYPE_F16;
  const AttnShape s = attn_shape(a.heads / a.kv_heads * (SELECT ? 1 : a.next_n), f16);
  if (f16) {
    switch (s.r) {
      case 16: return launch_cfg<AttnCfg<D, 16, 4, SELECT>, __half>(k_map, v_map, a, s, sms, stream);
      case 32: return launch_cfg<AttnCfg<D, 32, 4, SELECT>, __half>(k_map, v_map, a, s, sms, stream);
      default: return launch_cfg<AttnCfg<D, 64, 4, SELECT>, __half>(k_map, v_map, a, s, sms, stream);
    }
  }
  using B = __nv_bfloat16;
  switch (s.r) {
    case 8: return launch_cfg<AttnCfg<D, 8, 3, SELECT>, B>(k_map, v_map, a, s, sms, stream);
    case 16: return launch_cfg<AttnCfg<D, 16, 3, SELECT>, B>(k_map, v_map, a, s, sms, stream);
    case 32: return launch_cfg<AttnCfg<D, 32, 3, SELECT>, B>(k_map, v_map, a, s, sms, stream);
    default: return launch_cfg<AttnCfg<D, 64, 3, SELECT>, B>(k_map, v_map, a, s, sms, stream);
  }
}

// The CTAs on an SM of the kernel that a shape takes.
template <int D, bool SELECT>
int ctas_for(int r, bool f16) {
  if (f16)
    return r == 16 ? AttnCfg<D, 16, 4, SELECT>::CTAS
                   : r == 32 ? AttnCfg<D, 32, 4, SELECT>::CTAS : AttnCfg<D, 64, 4, SELECT>::CTAS;
  return r == 8 ? AttnCfg<D, 8, 3, SELECT>::CTAS
                : r == 16 ? AttnCfg<D, 16, 3, SELECT>::CTAS
                          : r == 32 ? AttnCfg<D, 32, 3, SELECT>::CTAS
                                    : AttnCfg<D, 64, 3, SELECT>::CTAS;
}

inline cudaError_t read_attention_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_attention_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(int32_t));
}

}  // namespace
}  // namespace idx
