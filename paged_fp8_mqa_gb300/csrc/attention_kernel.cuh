// attention_kernel.cuh -- attention over the 8-bit and the 4-bit K/V cache: for row (b, t) and query head h with
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
//
// The 4-bit cache (FP4) is not converted either.  A key's scales, one for each 32 elements, are what the
// tensor core's block scaling takes: S^T = K Q^T is kind::mxf8f6f4 with K as e2m1 and its scale bytes copied
// from shared to tensor memory, Q's parts as e5m2 with the constant scale 2^-14; so S comes scaled and
// only softmax_scale is left to the rows.  A value row's float32 scale goes into the weight, as a block's
// does above, and O^T = V^T P^T is kind::f8f6f4 with V as e2m1.  Both read e2m1 from the padded layout (16
// elements in the lower eight of 16 bytes), which the TMA unit writes from the packed rows: a tile takes as
// much shared memory, and as many of its cycles, as in 8 bits, for half the bytes of memory.
//   * The TMA unit pads rows of 128 elements.  Rows of 64 come to it two tokens at a time (PAIRS).  Selected
//     rows are fetched packed, 16 bytes a copy, into a ring of their own and spread by the warp that asked
//     for them.
//   * Keys and values have rings of their own: a key's stage is free once its scores are there, a tile's
//     worth of time before its values' is, and stages are what bounds the loads in flight.
//   * Scales come by asynchronous copies, with whole pages four rows' at a time, with selected rows a row's.
//     What a position's scales give its weights (a logarithm, a reciprocal) its softmax thread works out while
//     its scores come.
//   * The MMA warp waits on the next tile's keys and on this tile's weights at once (test_wait and a short
//     try_wait in turn): scores of the next tile go ahead of the product of this one when they can.
// What bounds it, head_dim 128, whole pages (DRAM rates of the copy): with few rows (64 requests of
// 1K..32K, 8 rows: 218 us for 173) the shared memory's port, 312 cycles for a tile's writes, 161 for each read
// by the tensor core, and what separates them, of 870 that a tile takes on an SM; with 32 rows (draft
// verification, 179 us for 87) the same with three reads of K and the weights' parts, and the softmax warps'
// latency.  Float16 queries have four parts a weight and at least 16 rows: the same decode 299 us, draft
// verification 213, head_dim 64 115 for 78.  Selected rows: 64-byte rows and their scales from places of their
// own, of which DRAM moves twice what is used (serving mix, 102 us for 27).  From L2 instead of DRAM decode
// takes 208 us.  Not kept:
// prefetches into L2 by any unit (231 to 273 us), softmax warpgroups in turn on tiles (228 for 219), two or
// more loading warps a ring (220), two tiles' positions a softmax thread as with PAIRS (261: the stages that
// two tiles hold are missed by the loads), with 32 rows two buffers of weights and a stage of values fewer
// (draft verification 197 for 178), 8-byte copies of selected rows (serving 160 us).
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

// One kernel's shape: R rows, PARTS parts a weight, head_dim D; FP4: the cache in four bits.
template <int D_, int R_, int PARTS_, bool SELECT_, bool FP4_>
struct AttnCfg {
  static constexpr int D = D_, R = R_, PARTS = PARTS_;
  static constexpr bool SELECT = SELECT_, FP4 = FP4_;
  // Whole pages of rows of 64 in four bits, by the TMA unit, whose 4-bit boxes are 128 elements wide: two
  // tokens a row.  A tile is then 256 positions, the first tokens of the pairs and the second ones, which have
  // columns of S, weights and sums of their own; a softmax thread takes both positions of a pair, whose
  // chains run side by side.  (Each by itself, tile after tile: 101 us for 78 with 32 requests of 4K..64K, 32
  // heads on 4; rows by ordinary copies 133.  More than 16 rows have no columns for two of O.)
  static constexpr bool PAIRS = FP4 && !SELECT && D == 64;
  static constexpr int SUBS = PAIRS ? 2 : 1, POS = kTile * SUBS;  // positions of a row, and of a tile
  static constexpr int ROW = PAIRS ? 128 : D;         // bytes of a tile's row
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
  // In four bits whole pages have two, one for keys and one for values, where there is room: what holds
  // a loader up is handing its copies to the TMA unit.
  static constexpr int LOADERS = !SELECT ? (FP4 && R <= 16 ? 2 : 1) : R == 32 ? 1 : R == 8 ? 4 : 2;
  static constexpr int THREADS = 32 * (LOADERS + 1 + SOFT_WARPS);
  // Two of S, one of O (PAIRS: O of either token's weights with both tokens' values; half of each is
  // used); with FP4 the keys' scale factors, two tiles of them, and the queries' (1).
  static constexpr int OUT = 2 * SUBS * NS, SFA = OUT + SUBS * NO, SFB = SFA + 8;
  static constexpr int COLS = FP4 ? SFB + 4 : SFA;
  static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  // CTAs on an SM, each with a pipeline of its own, so that one's loads and products run beside the
  // other's softmax.  Three of two stages instead of two of three: decode took 1.4 times as long, as
  // what the next launch needs no longer fits beside them.  64 rows in chunks of 32, two CTAs an SM:
  // one long request 1.07 times as long, a batch of 64 requests with 64 heads on one 1.3 times.
  static constexpr int CTAS = R == 64 ? 1 : 2;        // (ctas_for, for the workspace, says the same)
  static constexpr int T_BYTES = kTile * ROW;         // a tile of K, or of V, as the products read it
  static constexpr int Q_BYTES = NS * (CAT ? 1 : QPARTS) * D;
  static constexpr int P_BYTES = SUBS * NO * kTile;   // a tile's weights
  // They take the place of the tile's keys, which have been read by then, where they fit it; else
  // they have buffers of their own.  (FP4: always, see below.)
  static constexpr bool OVER_K = !FP4 && P_BYTES <= kTile * D;
  // With two buffers a tile's weights need not wait for the product of the tile before, and S of this
  // tile, which was issued after the product of the tile before that, says that theirs is free.
  static constexpr int P_BUFS = OVER_K ? 0 : FP4 && (R == 32 || (R < 32 && SELECT && D == 128)) ? 1 : 2;
  // What a stage of K (FP4: its scale factors, where they are used and, by the TMA unit, as they came)
  // and of V holds besides: Token records, or (FP4, by the TMA unit) value scales, scale factors and
  // which of the tokens are there.
  static constexpr int K_AUX = !FP4 ? 0 : SELECT ? kTile * 4 : kTile * 8;
  static constexpr int V_AUX = FP4 ? kTile * 4 * (SUBS + 1) + (SELECT ? 0 : 16) : kTile * 16;
  static constexpr int MISC = 48 * R + (FP4 ? 0 : 3 * D * 4) + 256;
  static constexpr int FIXED = 1024 + Q_BYTES + P_BUFS * P_BYTES + MISC;
  static constexpr int ROOM = CTAS == 2 ? 115456 : 231424;
  static constexpr int LEFT = ROOM - FIXED;
  // FP4 copies land as they lie in the pool, K and V and what goes with them, and are spread by the
  // warp that asked for them: what is in flight takes half the room that the products need.
  static constexpr int RAW_BYTES = SELECT && FP4 ? kTile * (D + 16) : 0;
  // Stages of K and of V.  In 8 bits they are the same ones.  In four, a tile takes the room of 8 bits
  // for half the bytes, so that stages are what bounds the loads in flight: a key's is given back as soon
  // as its scores are there, long before its values' is.
  static constexpr int VS8 = LEFT / (2 * T_BYTES + V_AUX);
  static constexpr int KS = !FP4 ? (VS8 > 6 ? 6 : VS8) : SELECT && D == 128 && R != 64 ? 1 : R == 64 && !SELECT ? 3 : 2;
  static constexpr int K_ROOM = KS * (T_BYTES + K_AUX);
  static constexpr int VS4 = SELECT ? 2 : (LEFT - K_ROOM) / (T_BYTES + V_AUX);
  static constexpr int VS = !FP4 ? KS : VS4 > 6 ? 6 : VS4;
  static constexpr int V_ROOM = VS * (T_BYTES + V_AUX);
  static constexpr int RAW_FIT = RAW_BYTES == 0 ? 0 : (LEFT - K_ROOM - V_ROOM) / (RAW_BYTES + !RAW_BYTES);
  static constexpr int RAW = RAW_FIT > 6 ? 6 : RAW_FIT;
  static constexpr int SMEM = FIXED + K_ROOM + V_ROOM + RAW * RAW_BYTES;
  static_assert(VS >= 2 && (RAW_BYTES == 0 || RAW >= 1) && SMEM <= 232448, "fits the 227 KiB per-CTA limit");
  static_assert(!PAIRS || (WG == 1 && R * D * 4 <= P_BUFS * P_BYTES), "room for the second tokens' sums");
  static_assert(Q_BYTES % 1024 == 0 && (!CAT || PARTS == 3), "aligned; eight rows: three parts");
};

// What a tile's position brings to its scores and weights.
struct alignas(16) Token {
  float k;       // softmax_scale * log2(e) * k_scale
  float log_v;   // log2|v_scale|
  float inv_v;   // 1 / |v_scale|, with v_scale's sign
  int32_t pos;   // its position (0 with SELECT), or kNone
};
// The same with FP4, as the loaders leave it; the rest is the position's softmax thread's work.
struct alignas(8) Token4 {
  float v_scale;  // NaN where the key's scale is
  int32_t pos;
};

template <bool APPROX = false>
__device__ __forceinline__ Token token_of(float k, float v_scale, int pos) {
  Token t;
  const float held = fmaxf(fabsf(v_scale), kLeastScale);
  t.k = k;
  // (A NaN makes the weight one in the rows that see the position, and only in those: a weight of 0
  // meets inv_v, which stays a number.)
  t.log_v = v_scale == v_scale ? __log2f(held) : v_scale;
  // (APPROX: to one unit or so, as good as the sum that it goes into; past 2^125 it would be 0.)
  t.inv_v = copysignf(APPROX && held < 4.2e37f ? __fdividef(1.0f, held) : 1.0f / held, v_scale);
  t.pos = pos;
  return t;
}

// A byte of 0xFF among a key's factors is NaN, which its rows' weights take from the value scale.
template <int D>
__device__ __forceinline__ float scale_of(uint32_t factors, float v_scale) {
  if constexpr (D != 128) factors |= factors << 16;
  return __vcmpeq4(factors, 0xFFFFFFFFu) != 0 ? __int_as_float(0x7FC00000) : v_scale;
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
constexpr uint32_t kE2m1_A = 5u << 7;

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
template <class C>
__device__ __forceinline__ int key_length(const AttentionArgs &a, int key) {
  if constexpr (C::SELECT) {
    const int rows = a.batch * a.next_n;
    const int lo = max(0, __ldg(a.ranges + key));
    return max(0, min(__ldg(a.ranges + rows + key), a.slots) - lo);
  } else {
    return max(0, min(__ldg(a.seq_lens + key * a.sl_stride), INT_MAX - C::POS));
  }
}

template <class C>
__device__ __forceinline__ int tiles_for(int length) {
  return length / C::POS + (length % C::POS != 0);
}

// A place in a ring of N stages, and the parity of its present use.
template <int N>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// A CTA's run over the line: the segments (group, first tile, tiles) in order.  Every warp walks
// its own copy, all its lanes together: keys without positions are passed over 32 at a time.
template <class C>
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
          const int n = key + 1 + lane < keys ? key_length<C>(a, key + 1 + lane) : 0;
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
        tiles = tiles_for<C>(length);
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
  // K tiles and V tiles, in 8 bits side by side in one stage.
  const auto k_tile = [&](int st) { return base + st * (C::FP4 ? 1 : 2) * C::T_BYTES; };
  const auto v_tile = [&](int st) {
    return C::FP4 ? base + (C::KS + st) * C::T_BYTES : base + (2 * st + 1) * C::T_BYTES;
  };
  uint8_t *s_q = base + (C::KS + C::VS) * C::T_BYTES;  // [QPARTS * R][D], K-major, swizzled
  uint8_t *at = s_q + C::Q_BYTES;
  // A tile's weights, [SUBS][NO / 16][kTile][16].
  uint8_t *s_p = at;
  at += C::P_BUFS * C::P_BYTES;
  const auto weights_of = [&](uint32_t tile, int stage) {
    return C::OVER_K ? k_tile(stage) : s_p + (C::P_BUFS == 2 ? tile & 1 : 0) * C::P_BYTES;
  };
  uint8_t *s_raw_kv = at;                            // [RAW][K, V][kTile][D / 2]
  at += C::RAW * kTile * D;
  uint4 *s_raw_aux = reinterpret_cast<uint4 *>(at);  // [RAW][kTile]: factors, value scale, pos, row
  at += C::RAW * (C::RAW_BYTES - kTile * D);
  Token *s_tok = reinterpret_cast<Token *>(at);      // [stage of V][kTile]
  Token4 *s_tok4 = reinterpret_cast<Token4 *>(at);
  uint32_t *s_aux = reinterpret_cast<uint32_t *>(at);
  at += C::VS * C::V_AUX;
  // [stage of K][32][4]: token t's at [t % 32][t / 32]; by the TMA unit each followed by [kTile].
  uint32_t *s_sf = reinterpret_cast<uint32_t *>(at);
  at += C::KS * C::K_AUX;
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
  if constexpr (!C::FP4) at += 3 * D * 4;
  uint64_t *bars = reinterpret_cast<uint64_t *>(at);
  uint64_t *k_full = bars, *k_empty = k_full + C::KS, *v_full = C::FP4 ? k_empty + C::KS : k_full,
           *v_empty = C::FP4 ? v_full + C::VS : k_empty, *s_full = v_empty + C::VS, *p_full = s_full + 2,
           *pv_done = p_full + 2, *q_full = pv_done + 2, *drain = q_full + 1;
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
    for (int i = 0; i < C::KS; ++i) {
      // A loading lane's arrival, and (SELECT) one when its own copies have landed.  With FP4 one for each
      // loading warp, or the loader's and one for each lane's copies (of scales).
      mbar_init(&k_full[i], !C::FP4 ? (C::SELECT ? 64 : 32) * C::LOADERS : C::SELECT ? C::LOADERS : 33);
      mbar_init(&k_empty[i], 1);
    }
    if constexpr (C::FP4)
      for (int i = 0; i < C::VS; ++i) {
        mbar_init(&v_full[i], C::SELECT ? C::LOADERS : 33);
        mbar_init(&v_empty[i], 1);
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
  if constexpr (!C::FP4)
    for (int i = tid; i < 3 * D; i += C::THREADS) s_nan[i] = 0;
  griddep_wait();
  griddep_launch_dependents();

  // ---- the run ---------------------------------------------------------------------------------
  const int per = (keys + C::THREADS - 1) / C::THREADS;
  const int k_lo = min(tid * per, keys), k_hi = min(k_lo + per, keys);
  int64_t mine = 0;
  for (int k = k_lo; k < k_hi; ++k) mine += tiles_for<C>(key_length<C>(a, k));
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
      const int n = tiles_for<C>(key_length<C>(a, k));
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
  Walk<C> w;
  w.left = f1 - f0;
  w.seg_tile = w.seg_tiles = 0;
  if (w.left > 0) {
    w.key = s_key;
    w.length = key_length<C>(a, w.key);
    w.tiles = tiles_for<C>(w.length);
    const int64_t at0 = s_begin;
    w.group = at0 < INT_MAX ? static_cast<int>(at0) / w.tiles : static_cast<int>(at0 / w.tiles);
    w.tile = static_cast<int>(at0 - static_cast<int64_t>(w.group) * w.tiles);
  }
  bool ok = true;
  uint32_t issued_k = 0, issued_v = 0;  // loaders: tiles whose copies were started
  Ring<C::KS> kr;
  Ring<C::VS> vr;  // (in 8 bits the same as kr, and not used)

  if (warp == 0 || warp >= 2 + C::SOFT_WARPS) {
    // ============================== loaders =====================================================
    const uint64_t policy = l2_policy_evict_first();
    const int shift = a.block_size == 32 ? 5 : a.block_size == 64 ? 6 : 7;
    const float z_unit = a.scale * 1.4426950408889634f;  // scores in units of ln 2
    const auto free_now = [&](uint64_t *empty, uint32_t phase) {
      ok = __all_sync(0xffffffffu, mbar_wait(empty, phase ^ 1, kWaitNs));
      return ok;
    };
    const auto stage_free = [&]() { return free_now(&k_empty[kr.at], kr.phase); };
    const auto next_stage = [&]() {
      ++issued_k;
      kr.advance();
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
          far.g = m.g;
          far.extent = __ldg(a.seq_lens + m.b * a.sl_stride) - a.next_n + m.t_select + 1;
          cand = a.candidates + w.key * a.cand_stride + max(0, __ldg(a.ranges + w.key));
          slot = w.seg_tile * kTile;
          end = min((w.seg_tile + w.seg_tiles) * kTile, w.length);
        }
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const int s = slot + token0 + 32 * j;
          far.pos[j] = s >= end ? -1 : __ldg(&cand[s].x);
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
      if constexpr (C::FP4) {
        // 16 bytes a lane and copy, as they lie in the pool, RAW tiles ahead; each lane spreads what it
        // asked for itself, 16 elements to the lower half of 16 bytes, with the swizzle that the products
        // expect.  (Copies of eight bytes, which need no spreading, go through L1, of which there is
        // hardly any left: the serving mix took 160 us.)
        constexpr int kLanes = D / 32, kRows = 32 / kLanes;
        const int piece = lane % kLanes, sub = lane / kLanes;
        Ring<C::RAW> in, out;
        int row0[EACH], pos0[EACH];
        // Each read of the chain position -> page has a tile's time to come back.
        Ahead mid{};                 // a tile whose pages are being read
        int id_mid[EACH];
        const auto pages = [&]() {   // of far's tile
          mid = far;
#pragma unroll
          for (int j = 0; j < EACH; ++j) {
            const int blk = mid.pos[j] >> shift;
            const bool seen = mid.live && mid.pos[j] >= 0 && mid.pos[j] < mid.extent;
            if (!seen) mid.pos[j] = -1;
            id_mid[j] = seen && blk < a.bt_width ? __ldg(mid.table + blk) : -1;
          }
        };
        const auto rows = [&](int (&row)[EACH], int (&pos)[EACH]) {  // of mid's tile
          bool bad = false;
#pragma unroll
          for (int j = 0; j < EACH; ++j) {
            row[j] = -1;
            pos[j] = kNone;
            if (mid.pos[j] < 0) continue;
            if (id_mid[j] >= 0 && id_mid[j] < a.num_blocks) {
              row[j] = ((id_mid[j] * a.kv_heads + mid.g) << shift) + (mid.pos[j] & (a.block_size - 1));
              pos[j] = 0;
            } else {
              bad = true;
            }
          }
          if (bad) attn_flag(IDX_DEV_BAD_PAGE);
        };
        const auto issue = [&]() {
          uint8_t *raw = s_raw_kv + in.at * (kTile * D) + piece * 16;  // (K rows, then V rows)
#pragma unroll
          for (int q = 0; q < EACH; ++q) {
            const int t0 = token0 - lane + 32 * q;
#pragma unroll
            for (int j = 0; j < 32 / kRows; ++j) {
              const int n = j * kRows + sub;  // lane n's q-th token
              const int row = __shfl_sync(0xffffffffu, row0[q], n);
              if (row < 0) continue;  // (any code is a number, and its weight will be 0)
              const int64_t src = static_cast<int64_t>(row) * (D / 2) + piece * 16;
              cp_async_16(raw + (t0 + n) * (D / 2), a.k_pool + src, policy);
              cp_async_16(raw + (kTile + t0 + n) * (D / 2), a.v_pool + src, policy);
            }
            uint32_t *aux = reinterpret_cast<uint32_t *>(s_raw_aux + in.at * kTile + t0 + lane);
            if (row0[q] >= 0) {
              cp_async_4(aux, static_cast<const uint8_t *>(a.k_scales) +
                                  (D == 128 ? static_cast<int64_t>(row0[q]) : row0[q] >> 1) * 4);
              cp_async_4(aux + 1, a.v_scales + row0[q]);
            }
            *reinterpret_cast<int2 *>(aux + 2) = make_int2(pos0[q], row0[q]);
          }
          in.advance();
        };
        const auto spread = [&](uint8_t *tile, int half) {
          const uint8_t *raw = s_raw_kv + (out.at * 2 + half) * (kTile * D / 2) + piece * 16;
#pragma unroll
          for (int q = 0; q < EACH; ++q)
#pragma unroll
            for (int j = 0; j < 32 / kRows; ++j) {
              const int t = token0 - lane + 32 * q + j * kRows + sub;
              const uint4 u = *reinterpret_cast<const uint4 *>(raw + t * (D / 2));
              *reinterpret_cast<uint2 *>(tile + swizzled<D>(t, piece * 32)) = make_uint2(u.x, u.y);
              *reinterpret_cast<uint2 *>(tile + swizzled<D>(t, piece * 32 + 16)) = make_uint2(u.z, u.w);
            }
        };
        // A tile that has landed, to the stages.
        const auto hand_over = [&]() {
          uint4 aux[EACH];
#pragma unroll
          for (int q = 0; q < EACH; ++q) {
            aux[q] = s_raw_aux[out.at * kTile + token0 + 32 * q];
            if (D != 128) aux[q].x = aux[q].w & 1 ? aux[q].x >> 16 : aux[q].x & 0xFFFFu;
          }
          if (!stage_free()) return false;
          spread(k_tile(kr.at), 0);
#pragma unroll
          for (int q = 0; q < EACH; ++q) {
            const int t = token0 + 32 * q;
            s_sf[(kr.at * 32 + t % 32) * 4 + t / 32] = aux[q].x;
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_full[kr.at]);
          next_stage();
          if (!free_now(&v_empty[vr.at], vr.phase)) return false;
          spread(v_tile(vr.at), 1);
#pragma unroll
          for (int q = 0; q < EACH; ++q)
            s_tok4[vr.at * kTile + token0 + 32 * q] =
                Token4{scale_of<D>(aux[q].x, __uint_as_float(aux[q].y)), static_cast<int>(aux[q].z)};
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[vr.at]);
          ++issued_v;
          vr.advance();
          out.advance();
          return true;
        };
        positions();
        pages();
        if (far.live) positions();
        bool live0 = mid.live;
        rows(row0, pos0);
        pages();
        if (far.live) positions();
        int ahead = 0;  // tiles asked for and not handed over
        bool ending = false;
        while (live0 || ahead > 0) {
          if (live0) {
            issue();
            ++ahead;
            live0 = mid.live;
            rows(row0, pos0);
            pages();
            if (far.live) positions();
          }
          // A group a round, empty ones too, so that RAW - 1 groups follow the oldest of the tiles ahead
          // when it is waited for.
          cp_async_commit();
          if (!live0 && !ending) {
            ending = true;
            for (int i = ahead; i < C::RAW; ++i) cp_async_commit();
          }
          if (ahead == C::RAW || ending) {
            cp_async_wait_group<C::RAW - 1>();
            if (!hand_over()) break;
            --ahead;
          }
        }
        cp_async_wait_all();
      } else {
        const auto scales = [&](const int (&row)[EACH], float (&ks)[EACH], float (&vs)[EACH]) {
#pragma unroll
          for (int j = 0; j < EACH; ++j) {
            ks[j] = row[j] >= 0 ? __ldg(static_cast<const float *>(a.k_scales) + (row[j] >> shift)) : 0.0f;
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
          uint8_t *kt = k_tile(kr.at), *vt = v_tile(kr.at);
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
            s_tok[kr.at * kTile + token0 + 32 * j] =
                token_of(ks0[j] * z_unit, vs0[j], row0[j] >= 0 ? 0 : kNone);
          cp_async_arrive_noinc(&k_full[kr.at]);
          mbar_arrive(&k_full[kr.at]);
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
      }
    } else if constexpr (C::FP4) {
      const bool leader = elect_one(), keys_too = C::LOADERS == 1 || warp == 0,
                 values_too = C::LOADERS == 1 || warp != 0;
      const int sh = C::PAIRS ? shift - 1 : shift;  // rows of a page, of tokens or pairs of them
      while (ok && w.next(a, groups, keys)) {
        const RowMap m = rows_of<C>(a, w.key, w.group, split.chunks, split.chunk_rows);
        const int32_t *table = a.block_tables + m.b * a.bt_stride;
        // A lane reads one page's id, 32 pages ahead of the ones in hand.  All else of a tile is copied
        // without passing through a register, and the copies of pages are one thread's with the warp's
        // operands (as many threads' they come one after the other, each with operands of its own): the
        // loader's instructions are what paces the tiles.
        const int n_pages = (w.length + a.block_size - 1) >> shift;
        const int per_tile = kTile >> sh;
        int first = w.seg_tile * per_tile;  // the page of lane 0
        const auto ids = [&](int page) {
          if (page >= n_pages || page >= (w.seg_tile + w.seg_tiles) * per_tile) return -1;
          const int id = page < a.bt_width ? __ldg(table + page) : -1;
          if (id >= 0 && id < a.num_blocks) return id;
          attn_flag(IDX_DEV_BAD_PAGE);
          return -1;
        };
        int id = ids(first + lane), id_next = ids(first + 32 + lane);
        const int end = w.seg_tile + w.seg_tiles;
        for (int i = w.seg_tile; i < end; ++i) {
          if (i * per_tile >= first + 32) {
            first += 32;
            id = id_next;
            id_next = ids(first + 32 + lane);
          }
          // The pool's first row of the page that holds this lane's four rows, or -1.
          const int block = __shfl_sync(0xffffffffu, id, i * per_tile + ((lane * 4) >> sh) - first);
          const int page4 = block < 0 ? -1 : (block * a.kv_heads + m.g) << sh;
          const unsigned there = __ballot_sync(0xffffffffu, page4 >= 0);  // bit r / 4: row r's page is there
          const int bytes = (C::ROW / 2) * 4 * __popc(there);
          const int row4 = page4 + ((lane * 4) & ((1 << sh) - 1));
          if (keys_too) {
            if (!stage_free()) break;
            // (The barrier counts the bytes read, half of those that the rows take here.)
            if (leader) mbar_arrive_expect_tx(&k_full[kr.at], bytes);
            for (int pg = 0; pg < per_tile; ++pg) {
              const int row = __shfl_sync(0xffffffffu, page4, pg << (sh - 2));
              if (leader && row >= 0)
                tma_load_2d(k_tile(kr.at) + (pg << sh) * C::ROW, &k_map, &k_full[kr.at], 0, row, policy);
            }
            if (page4 >= 0)
              cp_async_16(s_sf + (kr.at * 2 + 1) * kTile + lane * 4,
                          static_cast<const uint32_t *>(a.k_scales) + row4, policy);
            cp_async_arrive_noinc(&k_full[kr.at]);
            next_stage();
          }
          if (values_too) {
            if (!free_now(&v_empty[vr.at], vr.phase)) break;
            uint32_t *aux = s_aux + vr.at * (C::V_AUX / 4);
            if (leader) {
              aux[C::POS + kTile] = there;
              mbar_arrive_expect_tx(&v_full[vr.at], bytes);
            }
            for (int pg = 0; pg < per_tile; ++pg) {
              const int row = __shfl_sync(0xffffffffu, page4, pg << (sh - 2));
              if (leader && row >= 0)
                tma_load_2d(v_tile(vr.at) + (pg << sh) * C::ROW, &v_map, &v_full[vr.at], 0, row, policy);
            }
            if (page4 >= 0) {
#pragma unroll
              for (int j = 0; j < C::SUBS; ++j)
                cp_async_16(aux + lane * 4 * C::SUBS + j * 4, a.v_scales + row4 * C::SUBS + j * 4, policy);
              cp_async_16(aux + C::POS + lane * 4, static_cast<const uint32_t *>(a.k_scales) + row4, policy);
            }
            cp_async_arrive_noinc(&v_full[vr.at]);
            ++issued_v;
            vr.advance();
          }
        }
      }
      cp_async_wait_all();
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
          k = block >= 0 ? __ldg(static_cast<const float *>(a.k_scales) + page) : 0.0f;
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
          uint8_t *kt = k_tile(kr.at), *vt = v_tile(kr.at);
          if (block >= 0 && (p & (a.block_size - 1)) == 0) {
            const int row = (block * a.kv_heads + m.g) << shift;
            mbar_expect_tx(&k_full[kr.at], 2 * D * a.block_size);
            tma_load_2d(kt + lane * 4 * D, &k_map, &k_full[kr.at], 0, row, policy);
            tma_load_2d(vt + lane * 4 * D, &v_map, &k_full[kr.at], 0, row, policy);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            tok.pos = block >= 0 && p + j < w.length ? p + j : kNone;
            s_tok[kr.at * kTile + lane * 4 + j] = tok;
          }
          mbar_arrive(&k_full[kr.at]);
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
    constexpr uint32_t idesc_o =
        idesc_e4m3_f32(C::ROW, C::NO) | kE5m2_B | kMajorMN_A | kMajorMN_B | (C::FP4 ? kE2m1_A : 0u);
    const uint64_t q_desc = smem_desc_rows<D>(smem_addr(s_q));
    const uint32_t o_tmem = tmem + C::OUT;
    uint32_t tile = 0, seg = 0;
    const bool leader = elect_one();
    const auto all_wait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs)) != 0;
    };
    const auto scores = [&](uint32_t n, int st) {  // S of tile n of the run, from stage st
      const uint64_t k_desc = smem_desc_rows<C::ROW>(smem_addr(k_tile(st)));
      const uint32_t factors = tmem + C::SFA + (n & 1) * 4;
      if (!leader) return;
      if constexpr (C::FP4) tmem_copy_factors(factors, smem_desc_factors(smem_addr(s_sf + st * (C::K_AUX / 4))));
#pragma unroll
      for (int sub = 0; sub < C::SUBS; ++sub)
#pragma unroll
        for (int part = 0; part < C::PASSES; ++part)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const uint32_t to = tmem + ((n & 1) * C::SUBS + sub) * NS;
            const uint64_t k_at = k_desc + sub * (D >> 4) + 2 * k, q_at = q_desc + part * (R * D >> 4) + 2 * k;
            if constexpr (C::FP4)
              mma_mxf8f6f4(to, k_at, q_at, idesc_mx(kTile, NS, sub * (D / 32) + k), factors, tmem + C::SFB,
                           part + k > 0);
            else
              mma_f8f6f4(to, k_at, q_at, idesc_s, part + k > 0);
          }
      mma_commit(&s_full[n & 1]);
      if constexpr (C::FP4) mma_commit(&k_empty[st]);
    };
    const auto keys_here = [&](int st) {
      if constexpr (C::FP4 && !C::SELECT) {
        // Their scale factors, which came in the tokens' order, to where the tensor core expects them.
        const uint4 u = *reinterpret_cast<const uint4 *>(s_sf + (st * 2 + 1) * kTile + lane * 4);
        uint32_t *to = s_sf + st * 2 * kTile + (lane % 8) * 16 + lane / 8;
        to[0] = u.x, to[4] = u.y, to[8] = u.z, to[12] = u.w;
      }
      // (What ordinary copies and stores wrote.)
      if constexpr (C::SELECT || C::FP4) fence_proxy_async_shared();
      __syncwarp();
      tc_fence_after_sync();
    };
    // The segment's products; false if a wait gave up.  The whole warp walks through it, so that the
    // descriptors are the warp's and not one thread's; one thread issues.
    const auto segment = [&]() {
      if (!all_wait(q_full, seg & 1)) return false;
      tc_fence_after_sync();
      bool ahead = false;  // S of the tile has been issued already
      for (int i = 0; i < w.seg_tiles; ++i, ++tile) {
        if (!ahead) {
          if (!all_wait(&k_full[kr.at], kr.phase)) return false;
          keys_here(kr.at);
          scores(tile, kr.at);
        }
        // The next tile's scores as soon as its keys are here, this tile's sum as soon as its weights are.
        Ring<C::KS> next = kr;
        next.advance();
        ahead = i + 1 >= w.seg_tiles;
        uint64_t begin = 0;
        for (;;) {
          if (!ahead && __all_sync(0xffffffffu, mbar_test_wait(&k_full[next.at], next.phase))) {
            ahead = true;
            keys_here(next.at);
            scores(tile + 1, next.at);
          }
          if (__all_sync(0xffffffffu, mbar_try_wait_sleep(&p_full[tile & 1], (tile >> 1) & 1, ahead ? 100000u : 100u)))
            break;
          const uint64_t now = global_timer_ns();
          if (begin == 0) begin = now;
          if (__any_sync(0xffffffffu, now - begin > kWaitNs)) return false;
        }
        ahead = ahead && i + 1 < w.seg_tiles;
        if (C::FP4 && !all_wait(&v_full[vr.at], vr.phase)) return false;
        if constexpr (C::FP4) fence_proxy_async_shared();
        tc_fence_after_sync();
        const uint64_t v_desc = smem_desc_mn<C::ROW>(smem_addr(v_tile(C::FP4 ? vr.at : kr.at)));
        const uint64_t p_desc = smem_desc_p(smem_addr(weights_of(tile, kr.at)));
        if (leader) {
#pragma unroll
          for (int sub = 0; sub < C::SUBS; ++sub)
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma_f8f6f4(o_tmem + sub * C::NO, v_desc + k * (32 * C::ROW >> 4),
                         p_desc + sub * (C::NO * kTile >> 4) + k * (512 >> 4), idesc_o, i + k > 0);
          mma_commit(&pv_done[tile & 1]);
          mma_commit(C::FP4 ? &v_empty[vr.at] : &k_empty[kr.at]);
        }
        kr = next;
        vr.advance();
      }
      return true;
    };
    while (ok && w.next(a, groups, keys)) {
      ok = segment();
      ++seg;
    }
    if (leader) mma_commit(drain);
    __syncwarp();
  } else {
    // ============================== softmax =====================================================
    const int wg = (warp - 2) >> 2, quarter = warp & 3;
    const int r0 = wg * RT;                      // the thread's rows
    const int token = quarter * 32 + lane;       // the thread's position in the tile
    // The thread's dimension of the output, or -1 (M = 64: 16 lanes of each quarter; PAIRS: the first tokens'
    // values, to which the second tokens' sums are added).
    const int dim = C::ROW == 128 ? (token < D ? token : -1) : lane < 16 ? quarter * 16 + lane : -1;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float z_unit = a.scale * 1.4426950408889634f;  // (FP4: what the tokens' keys share)
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
    if (C::FP4 && wg == 0) {  // the queries' scale factors: 2^-14, whatever the place
      constexpr uint32_t f = 0x71717171u;
      asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(lane_base +
                                                                                       C::SFB),
                   "r"(f)
                   : "memory");
      tmem_st_wait();
      tc_fence_before_sync();  // (of the first arrival at q_full)
    }
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
          const float down =  // (times softmax_scale log2(e) with FP4: -100 <= e, so that it stays normal)
              __uint_as_float(static_cast<uint32_t>(127 - (C::FP4 ? 0 : 14) + min(e, 127)) << 23);
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
            s_rs[r] = C::FP4 ? down * z_unit : down;
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
        {
          // (Usually both are through: asked for at once, as each answer takes its time.)
          uint64_t *there = C::FP4 ? &v_full[vr.at] : &k_full[kr.at];
          const uint32_t use = C::FP4 ? vr.phase : kr.phase;
          const bool v_there = mbar_test_wait(there, use);
          const bool s_there = mbar_test_wait(&s_full[tile & 1], (tile >> 1) & 1);
          if (!__all_sync(0xffffffffu, v_there && s_there)) {
            wait(there, use);
            wait(&s_full[tile & 1], (tile >> 1) & 1);
          }
        }
        tc_fence_after_sync();
        Token tok[C::SUBS];
        float2 y[C::SUBS][RT / 2];  // the weights' logarithms
        {
          uint32_t v[C::SUBS][RT], u[C::SUBS][C::CAT ? RT : 8], t[C::SUBS][C::CAT ? RT : 8];
#pragma unroll
          for (int sub = 0; sub < C::SUBS; ++sub) {
            const uint32_t s_at = lane_base + ((tile & 1) * C::SUBS + sub) * NS;
            tmem_ld_cols<RT>(s_at + r0, v[sub]);
            if constexpr (C::CAT) {
              tmem_ld_cols<RT>(s_at + R, u[sub]);
              tmem_ld_cols<RT>(s_at + 2 * R, t[sub]);
            }
          }
          // (While they come: what the position brings.)
#pragma unroll
          for (int sub = 0; sub < C::SUBS; ++sub) {
            if constexpr (C::FP4) {
              Token4 t4;
              if constexpr (C::SELECT) {
                t4 = s_tok4[vr.at * kTile + token];
              } else {
                const uint32_t *aux = s_aux + vr.at * (C::V_AUX / 4);
                const int p = (w.seg_tile + i) * C::POS + token * C::SUBS + sub;
                uint32_t factors = aux[C::POS + token];
                if constexpr (C::PAIRS) factors = (factors >> (16 * sub)) & 0xFFFFu;
                t4.v_scale = scale_of<D>(factors, __uint_as_float(aux[token * C::SUBS + sub]));
                t4.pos = ((aux[C::POS + kTile] >> (token / 4)) & 1u) != 0 && p < len ? p : kNone;
              }
              tok[sub] = token_of<true>(1.0f, t4.v_scale, t4.pos);
            } else {
              tok[sub] = s_tok[kr.at * kTile + token];
            }
          }
          tmem_ld_wait();
#pragma unroll
          for (int sub = 0; sub < C::SUBS; ++sub) {
            reg_fence(v[sub]);
            if constexpr (C::CAT) {
              reg_fence(u[sub]);
              reg_fence(t[sub]);
#pragma unroll
              for (int r = 0; r < RT; ++r)
                v[sub][r] = __float_as_uint(__uint_as_float(v[sub][r]) +
                                            (__uint_as_float(u[sub][r]) + __uint_as_float(t[sub][r])));
            }
            const float2 k2 = make_float2(tok[sub].k, tok[sub].k);
            const float2 lv2 = make_float2(tok[sub].log_v, tok[sub].log_v);
#pragma unroll
            for (int r = 0; r < RT / 2; r += 2) {
              float4 f;
              if constexpr (kHoldRs)
                f = make_float4(rs[r].x, rs[r].y, rs[r + 1].x, rs[r + 1].y);
              else
                f = *reinterpret_cast<const float4 *>(rs_at + r);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float2 s2 = make_float2(__uint_as_float(v[sub][2 * (r + h)]),
                                              __uint_as_float(v[sub][2 * (r + h) + 1]));
                const float2 unit = h ? make_float2(f.z, f.w) : make_float2(f.x, f.y);
                // (FP4: the tensor core has applied the key's scale, and unit holds the rest.)
                y[sub][r + h] = __ffma2_rn(s2, C::FP4 ? unit : __fmul2_rn(unit, k2),
                                           __fadd2_rn(lv2, nref[r + h]));
              }
            }
          }
        }
        bool all_seen = true;
#pragma unroll
        for (int sub = 0; sub < C::SUBS; ++sub) all_seen = all_seen && tok[sub].pos < all_see;
        if (!__all_sync(0xffffffffu, all_seen)) {
#pragma unroll
          for (int sub = 0; sub < C::SUBS; ++sub)
            if (!(tok[sub].pos < all_see)) {
#pragma unroll
              for (int r = 0; r < RT / 2; ++r) {
                if (tok[sub].pos >= s_ext[r0 + 2 * r]) y[sub][r].x = -INFINITY;
                if (tok[sub].pos >= s_ext[r0 + 2 * r + 1]) y[sub][r].y = -INFINITY;
              }
            }
        }
        // The larger of a row's logarithms at the thread's positions.
        const auto top = [&](int r) {
          float x = r & 1 ? y[0][r / 2].y : y[0][r / 2].x;
#pragma unroll
          for (int sub = 1; sub < C::SUBS; ++sub) x = fmaxf(x, r & 1 ? y[sub][r / 2].y : y[sub][r / 2].x);
          return x;
        };
        float most = top(0);
#pragma unroll
        for (int r = 1; r < RT; ++r) most = fmaxf(most, top(r));
        bool move = most > kMost;
        if (unset != 0) {
#pragma unroll
          for (int r = 0; r < RT; ++r) move |= ((unset >> r) & 1u) != 0 && top(r) != -INFINITY;
        }
        if (any_of_group(move)) {
          // Some weight would leave e5m2's range, or a row sees its first position: the references
          // move to the maxima so far.
          float mine = -INFINITY;  // lane r: row r0 + r
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float x = warp_max(top(r));
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
#pragma unroll
            for (int sub = 0; sub < C::SUBS; ++sub) y[sub][r] = __fadd2_rn(y[sub][r], d);
            nref[r] = __fadd2_rn(nref[r], d);
            sum[r].x *= __shfl_sync(0xffffffffu, keep, 2 * r);
            sum[r].y *= __shfl_sync(0xffffffffu, keep, 2 * r + 1);
          }
          if (i > 0) {
            wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
            tc_fence_after_sync();
#pragma unroll 1
            for (int part = 0; part < PARTS * C::SUBS; ++part) {
              const uint32_t o_at =
                  lane_base + C::OUT + (part < PARTS ? part * R : C::NO + (part - PARTS) * R) + r0;
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
        if constexpr (C::FP4 && C::P_BUFS == 2) {
        } else if constexpr (C::P_BUFS == 1) {
          if (tile >= 1) wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
        } else {
          if (tile >= 2) wait(&pv_done[tile & 1], ((tile >> 1) - 1) & 1);
        }
#pragma unroll
        for (int sub = 0; sub < C::SUBS; ++sub) {
          uint8_t *sp = weights_of(tile, kr.at) + sub * (C::NO * kTile) + token * 16;
          const float inv_v = fabsf(tok[sub].inv_v);
          // The weights of a position whose value scale is negative or 0 (as good as): rare, so asked
          // of the whole warp.
          const bool odd = __any_sync(0xffffffffu, tok[sub].inv_v < 0.0f || inv_v >= 1.0f / kLeastScale);
          const uint32_t flip = tok[sub].inv_v < 0.0f ? 0x80808080u : 0u;
          const uint32_t live = inv_v < 1.0f / kLeastScale ? 0xFFFFFFFFu : 0u;
          uint32_t bytes[PARTS][4];
          const float2 inv2 = make_float2(inv_v, inv_v);
#pragma unroll
          for (int r = 0; r < RT; r += 4) {
            float2 p[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              p[j] = make_float2(fast_exp2(y[sub][r / 2 + j].x), fast_exp2(y[sub][r / 2 + j].y));
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
        }
        // A value that some row does not see must not meet its weight of 0 as a NaN (a code of the
        // cache, or bytes that were never written): what no row sees becomes 0; in the newest
        // tokens, which only the later draft slots see, a NaN becomes 0 and is noted in s_nan (as
        // this segment's number) for the rows that do see it.
        // (Four bits hold no NaN.)
        if (!C::FP4 && wg == 0 && !all_seen) {
          uint8_t *v = v_tile(kr.at);
          if (tok[0].pos == kNone) {
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
                  s_nan[(len - 1 - tok[0].pos) * D + x + e] = seg;
                }
            }
          }
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[tile & 1]);
        kr.advance();
        vr.advance();
      }
      // ---- the segment's sums ------------------------------------------------------------------------
      wait(&pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1);
      tc_fence_after_sync();
      float acc[RT];
#pragma unroll
      for (int part = PARTS - 1; part >= 0; --part) {
        uint32_t v[RT];
        // (PAIRS: the upper lanes' are the second tokens' dimensions, and the second tiles' weights'.)
        tmem_ld_cols<RT>(lane_base + C::OUT + (C::PAIRS && token >= D ? C::NO : 0) + part * R + r0, v);
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
      if (!C::FP4 && !C::SELECT && a.next_n > 1) {
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
      // (The weights' place is free: their products are done, and the next segment's come after its
      // queries, for which every warp waits.)
      float *half = reinterpret_cast<float *>(s_p);
      if constexpr (C::PAIRS) {
        if (token >= D) {
#pragma unroll
          for (int r = 0; r < RT; ++r) half[r * D + token - D] = acc[r];
        }
      }
      sync_group();
      if constexpr (C::PAIRS) {
        if (token < D) {
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r] += half[r * D + token];
        }
      }
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
    if (key_length<C>(a, k) > 0) continue;
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
    if ((warp == 0 || warp >= 2 + C::SOFT_WARPS) && lane == 0) {
      const auto landed = [&](uint64_t *full, uint32_t issued, uint32_t stages) {
        const uint32_t tail = issued < stages ? issued : stages;
        for (uint32_t d = 1; d <= tail; ++d) {
          const uint32_t n = issued - d;
          if (!mbar_wait(&full[n % stages], (n / stages) & 1, kWaitNs)) attn_flag(IDX_DEV_WAIT_TIMEOUT);
        }
      };
      landed(k_full, issued_k, C::KS);
      if constexpr (C::FP4) landed(v_full, issued_v, C::VS);
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

// Rows that share a K/V head, cut into chunks of at most `most`, and the kernel's R for a chunk.
struct AttnShape {
  int chunks, chunk_rows, r;
};
inline AttnShape attn_shape(int rows, bool f16, int most) {
  AttnShape s;
  s.chunks = (rows + most - 1) / most;
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

// Rows in a chunk: 64, or with PAIRS 16, as many as have columns for two of O (draft verification with 32
// rows of 64 in two chunks 204 us, in one by ordinary copies 249).
constexpr int most_rows(int dim, bool select, bool four) { return four && dim == 64 && !select ? 16 : 64; }

template <int D, bool SELECT, bool FP4>
cudaError_t launch_rows(const CUtensorMap &k_map, const CUtensorMap &v_map, const AttentionArgs &a,
                        int dtype, int sms, cudaStream_t stream) {
  const bool f16 = dtype == IDX_DTYPE_F16;
  constexpr int MOST = most_rows(D, SELECT, FP4);
  const AttnShape s = attn_shape(a.heads / a.kv_heads * (SELECT ? 1 : a.next_n), f16, MOST);
  using B = __nv_bfloat16;
  if constexpr (MOST == 16) {
    return f16 ? launch_cfg<AttnCfg<D, 16, 4, SELECT, FP4>, __half>(k_map, v_map, a, s, sms, stream)
               : s.r == 8 ? launch_cfg<AttnCfg<D, 8, 3, SELECT, FP4>, B>(k_map, v_map, a, s, sms, stream)
                          : launch_cfg<AttnCfg<D, 16, 3, SELECT, FP4>, B>(k_map, v_map, a, s, sms, stream);
  } else {
    if (f16) {
      switch (s.r) {
        case 16: return launch_cfg<AttnCfg<D, 16, 4, SELECT, FP4>, __half>(k_map, v_map, a, s, sms, stream);
        case 32: return launch_cfg<AttnCfg<D, 32, 4, SELECT, FP4>, __half>(k_map, v_map, a, s, sms, stream);
        default: return launch_cfg<AttnCfg<D, 64, 4, SELECT, FP4>, __half>(k_map, v_map, a, s, sms, stream);
      }
    }
    switch (s.r) {
      case 8: return launch_cfg<AttnCfg<D, 8, 3, SELECT, FP4>, B>(k_map, v_map, a, s, sms, stream);
      case 16: return launch_cfg<AttnCfg<D, 16, 3, SELECT, FP4>, B>(k_map, v_map, a, s, sms, stream);
      case 32: return launch_cfg<AttnCfg<D, 32, 3, SELECT, FP4>, B>(k_map, v_map, a, s, sms, stream);
      default: return launch_cfg<AttnCfg<D, 64, 3, SELECT, FP4>, B>(k_map, v_map, a, s, sms, stream);
    }
  }
}

// The CTAs on an SM of the kernel that takes chunks of r rows (see AttnCfg).
inline int ctas_for(int r) { return r == 64 ? 1 : 2; }

inline cudaError_t read_attention_status(int32_t *value, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_attention_status, sizeof(int32_t));
  if (e != cudaSuccess || !clear) return e;
  const int32_t zero = 0;
  return cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(int32_t));
}

}  // namespace
}  // namespace idx
