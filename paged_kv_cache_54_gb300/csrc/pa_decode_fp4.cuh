// Paged decode attention over a four-bit cache (PA_FP4) for sm_103a.
//
// Work decomposition.  The (sequence, KV head) pairs, in sequence order, are
// laid end to end in units of 64 tokens (a pair's tokens, and kPairCost units
// for what a piece costs beside them), and CTA b of n takes the units
// [b U / n, (b + 1) U / n) of the U in all: equal shares whatever the
// lengths, found by each CTA from a scan of the lengths (no plan launch, no
// claims).  A CTA's share is a run of pieces, one per pair it touches.  A
// pair that falls to one CTA whole is written out by it; the pieces of a cut
// pair leave (m, l, O / l) partials, joined by a merge kernel (the
// flash-decoding reduction).  Partials live in the layout every cache type's
// workspace has, [sequence, partition, query head]: piece j of a pair uses
// the place of partition j.  A share is at least two partitions (2P tokens)
// long, so a pair of L tokens has at most L / 2P + 2 pieces, and that many
// places whenever max_parts is two or more; calls of short sequences deal
// pairs out whole.  Sequences that share blocks are each read on their own:
// shared blocks come from L2, but are widened once for each.
//
// A CTA is four warps, and an SM holds four CTAs.  Within a piece warp w takes
// the 32-token steps w, w + 4, ..., each warp with its own online softmax; the
// four states meet in shared memory at the piece's end.  A warp's steps
// stream through a two-slot ring of its own in shared memory: 16-byte
// asynchronous copies bring the next step, which may be the next piece's
// first, while one is worked on, so warps wait for one another only where a
// piece ends.  (Bulk copies of whole tiles would be fewer instructions, but a
// thread starts one per 113 ns and an SM one per 30: with four threads at it,
// and nothing else to do, tiles of 1152 bytes (16 tokens at head_dim 128) come
// at 5.9 TB/s and tiles of 576 at 3.0, the ring's copies at 6.6.)
//
// A step is two slices of 16 tokens; a slice is two small products on
// mma.sync m16n8k16 with fp16 operands and fp32 accumulation, S^T = K Q^T and
// O^T = V^T P^T: tokens, then head dimensions, as M, and the query group
// padded to 8 as N.  Codes widen to fp16 exactly (a code times its group's
// scale is an fp16 value), so the only roundings are those of P to fp16 and
// of the output.
//
// What bounds it: the bytes and the instructions, about equally.  One
// sequence of 1048575 tokens, 64/8 heads (1.21 GB): 207 us, 5.8 TB/s; the
// copies alone take 184 us, the products alone 188 us, at 285 warp
// instructions a slice, 62% of the issue slots.  32/32 heads of 64 sequences
// of 512..4096 tokens (681 MB): 116 us, 5.9 TB/s.  128 sequences of 256..32768
// tokens, 64/8 heads (1.0 GB): 181 us, 5.5 TB/s.  head_dim 64 spreads the
// softmax and the shuffles of a slice over half the bytes: the same two
// batches take 76 us (340 MB, 4.5 TB/s) and 119 us (502 MB, 4.2 TB/s), with
// blocks of 8 81 and 122, of 32 73 and 115.  The rest of a short call:
// 1.2 us until the shares are known, 5 us until the first steps have landed,
// 1 us a piece for its end, 4 us for the merge.  Five CTAs an SM (96
// registers) took 3% longer than four, two CTAs of eight warps 8%, copies two
// steps ahead the same.
//
// Fragment orders (lane = 4 gq + tq), chosen so that every lane reads runs of
// its own:
//   S^T: row gq is token 2 gq, row gq + 8 token 2 gq + 1.  Lane tq's columns
//     are the dimensions [tq D/4, (tq + 1) D/4): k-step kk uses its local
//     dimensions 4kk .. 4kk + 3.
//   O^T: column k = 2tq, 2tq + 1, 2tq + 8, 2tq + 9 is token 4 tq + 0, 1, 2, 3.
//     Lane gq's rows are the dimensions [gq D/8, (gq + 1) D/8): m-tile mi has
//     local dimension mi in row gq and D/16 + mi in row gq + 8.
// The two codes of one A register of V^T come from two tokens: the code words
// of a token pair are interleaved (even dimensions, odd dimensions) so that
// one conversion of a byte gives the pair.
#pragma once

#include <limits.h>

#include "pa_fp4.cuh"
#include "pa_fp4.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kFpThreads = 32 * kWarps;
constexpr int kCtas = 4;        // CTAs an SM
constexpr int kSlice = 16;      // tokens of the products
constexpr int kStep = 32;       // tokens of a warp's step
constexpr int kUnit = 64;       // tokens of a unit of work
// Units that a pair is charged beside its tokens': its q, its first step's
// latency, the join.  128 sequences of 256..32768 tokens, 64/8 heads: 200 us
// at 1, 189 at 3, 181 at 5, 183 at 8; 64 of 512..4096, 32/32 heads: 118, 116,
// 116, 118.
constexpr int kPairCost = 5;
// Pairs of up to 512 tokens are dealt out whole, and there is no merge; with
// no more pairs than CTAs fit the GPU, each has a CTA of its own.  Whole
// against cut, us of one call among others in a graph (64/8 heads; the
// pairs' lengths from an eighth of the bound to the bound):
//   pairs        8          64         256        608        768        2048
//   of 256    4.5/8.0    4.7/10.0   5.9/10.9   8.5/14.1  13.0/16.1  24.8/24.7
//   of 512    6.1/7.3    6.3/10.4   7.8/12.8  11.8/16.6  17.1/19.5  33.5/33.5
//   of 1024   9.2/7.5    9.4/11.6  11.7/15.1  18.2/22.2  24.1/25.4  51.3/53.5
// and with 1024 tokens each 9.2/7.6, 9.6/13.5, 12.3/17.9, 20.4/23.1,
// 36.5/34.6, 72.7/73.1: a bound of 512 never loses, one of 1024 does with few
// pairs and with a little more than a CTA's worth each.  16 pairs of 32/32
// heads and up to 512 tokens: 5.4/6.9.
constexpr int kWholeTokens = 512;
constexpr float kLazy = 8.f;    // rescale when the maximum grows by more (base 2)
constexpr float kFar = 0x1p24f;
constexpr float kWritten = -1.f;  // l of a partial that marks the end of a pair's pieces

struct Fp4Params {
  void *out;
  const uint8_t *q;
  const uint8_t *k_cache;
  const uint8_t *v_cache;
  const int32_t *block_tables;
  const int32_t *seq_lens;
  int num_seqs, num_q_heads, num_kv_heads, num_blocks, max_blocks;
  int len_cap, max_parts, partition_size;
  int cut;  // whether a pair may be cut among CTAs (and the merge follows)
  float qk_scale_log2, v_scale;
  const float *k_head_scale, *v_head_scale;
  float2 *part_ml;
  float *part_o;
  int *err;
};

// Codes and scales of one slice as a lane reads them.
template <int D>
struct KSlice {
  static constexpr int W = D / 32;  // words of a row a lane reads (8 codes each)
  uint32_t c[2][W];   // tokens 2gq, 2gq + 1
  // their scales (two bytes), one for each 16 local dimensions; spread: of the
  // groups of columns 2tq and 2tq + 1
  uint32_t s[2];
};
template <int D>
struct VSlice {
  static constexpr int W = D / 64;
  uint32_t c[4][W];  // tokens 4tq .. 4tq + 3
  uint32_t s;        // their scales in the lane's group
};

template <int D>
struct State {
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;
  uint32_t qb[KSTEPS][2];
  float o[MT][4];
  float m[2], l[2];
  float top[2];            // unscaled scores above these bring the maximum up
  float mult[2], lift[2];  // of the scores, and their reciprocals
  bool far;                // some maximum is past 2^24 (warp-uniform)
};

// Few queries leave columns of the scores' product unused.  When a query's
// groups of 16 dimensions fit them too (G D / 16 <= 8), each gets a column of
// its own, Q laid out block-diagonally: a token's score is then the sum of
// its groups' columns, each times the group's scale in fp32, and no code is
// scaled before the product.  64 sequences of 512..4096 tokens, 32/32 heads:
// 127 us with the codes scaled, 116 us so.
template <int D, int G>
constexpr bool kSpread = G * D / kFp4Group <= 8;

// q rows of the group (G x D at `q`) as B fragments: column gq is query gq
// (spread: group gq % (D / 16) of query gq / (D / 16)), lane tq's local
// dimensions.  bf16 queries are rounded to fp16 after a multiplication by the
// query's own power of two, undone on its scores.
template <int QT, int D, int G>
__device__ __forceinline__ void load_q(State<D> &st, const uint8_t *q, float scale) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  constexpr int QW = D / 8;  // words of the lane
  uint32_t w[QW];
  const int query = kSpread<D, G> ? gq / (D / kFp4Group) : gq;  // of column gq
  const uint4 *row =
      reinterpret_cast<const uint4 *>(q + (static_cast<size_t>(query < G ? query : 0) * D + tq * (D / 4)) * 2);
#pragma unroll
  for (int i = 0; i < QW / 4; ++i) {
    const uint4 x = query < G ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
    w[4 * i] = x.x;
    w[4 * i + 1] = x.y;
    w[4 * i + 2] = x.z;
    w[4 * i + 3] = x.w;
  }
  float f = 1.f;
  if constexpr (QT == kBF16) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < QW; ++i) {
      const float2 x = half2_bits_to_float2<kBF16>(w[i]);
      top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    f = query_factor(top, scale);
#pragma unroll
    for (int i = 0; i < QW; ++i) {
      const float2 x = half2_bits_to_float2<kBF16>(w[i]);
      w[i] = pack2_rn<kF16>(x.x * f, x.y * f);
    }
  }
  // the scores' multiplier is positive: its sign goes to q, and a zero one
  // becomes zero queries
#pragma unroll
  for (int i = 0; i < QW; ++i) w[i] = scale > 0.f ? w[i] : scale < 0.f ? w[i] ^ 0x80008000u : 0u;
  st.far = false;
  const float mult = scale == 0.f ? 1.f : fabsf(scale) / f;  // of column gq
  if constexpr (kSpread<D, G>) {  // a column keeps one group's dimensions
    const int group = gq % (D / kFp4Group);
#pragma unroll
    for (int i = 0; i < QW; ++i)  // word i: local dimensions 2i, 2i + 1
      if (tq * (D / 64) + i / 8 != group) w[i] = 0u;
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    // (the lane's scores are of columns 2tq and 2tq + 1: one query's, when spread)
    st.mult[r] = __shfl_sync(0xffffffffu, mult, (2 * tq + (kSpread<D, G> ? 0 : r)) * 4);
    st.lift[r] = 1.f / st.mult[r];
    st.top[r] = -INFINITY;
  }
#pragma unroll
  for (int kk = 0; kk < State<D>::KSTEPS; ++kk) {
    st.qb[kk][0] = w[2 * kk];
    st.qb[kk][1] = w[2 * kk + 1];
  }
#pragma unroll
  for (int i = 0; i < State<D>::MT; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;
}

__device__ __forceinline__ uint32_t lo2(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t hi2(uint32_t h) { return __byte_perm(h, h, 0x3232); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// c += A * B, fp16 operands
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c = A * B with a zero addend (no registers to clear first)
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// S^T of a slice, unscaled: s[0], s[1] are token 2gq against queries 2tq and
// 2tq + 1, s[2], s[3] token 2gq + 1.
template <int D>
__device__ __forceinline__ void scores(const State<D> &st, const KSlice<D> &c, float (&s)[4]) {
  float acc[2][4];
#pragma unroll
  for (int w = 0; w < KSlice<D>::W; ++w) {
    const uint32_t s2 = e4m3x2_to_half2(c.s[w / 2]);
    const uint32_t s0 = lo2(s2), s1 = hi2(s2);
    uint32_t a[4], b[4];
    e2m1x8_to_half2x4(c.c[0][w], a);
    e2m1x8_to_half2x4(c.c[1][w], b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = hmul2_bits(a[i], s0);
      b[i] = hmul2_bits(b[i], s1);
    }
    if (w == 0) {
      mma_first(acc[0], a[0], b[0], a[1], b[1], st.qb[0][0], st.qb[0][1]);
      mma_first(acc[1], a[2], b[2], a[3], b[3], st.qb[1][0], st.qb[1][1]);
    } else {
      mma(acc[0], a[0], b[0], a[1], b[1], st.qb[2 * w][0], st.qb[2 * w][1]);
      mma(acc[1], a[2], b[2], a[3], b[3], st.qb[2 * w + 1][0], st.qb[2 * w + 1][1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = acc[0][i] + acc[1][i];
}

// The same when spread: s[0] is token 2gq, s[1] token 2gq + 1, against the
// query of columns 2tq and 2tq + 1, in every lane that has the query.
template <int D>
__device__ __forceinline__ void scores_spread(const State<D> &st, const KSlice<D> &c, float (&s)[2]) {
  float acc[2][4];
#pragma unroll
  for (int w = 0; w < KSlice<D>::W; ++w) {
    uint32_t a[4], b[4];
    e2m1x8_to_half2x4(c.c[0][w], a);
    e2m1x8_to_half2x4(c.c[1][w], b);
    if (w == 0) {
      mma_first(acc[0], a[0], b[0], a[1], b[1], st.qb[0][0], st.qb[0][1]);
      mma_first(acc[1], a[2], b[2], a[3], b[3], st.qb[1][0], st.qb[1][1]);
    } else {
      mma(acc[0], a[0], b[0], a[1], b[1], st.qb[2 * w][0], st.qb[2 * w][1]);
      mma(acc[1], a[2], b[2], a[3], b[3], st.qb[2 * w + 1][0], st.qb[2 * w + 1][1]);
    }
  }
  // scales of tokens 2gq, 2gq + 1 in the groups of columns 2tq and 2tq + 1
  const float2 g0 = half2_bits_to_float2<kF16>(e4m3x2_to_half2(c.s[0]));
  const float2 g1 = half2_bits_to_float2<kF16>(e4m3x2_to_half2(c.s[1]));
  s[0] = fmaf(acc[0][1] + acc[1][1], g1.x, (acc[0][0] + acc[1][0]) * g0.x);
  s[1] = fmaf(acc[0][3] + acc[1][3], g1.y, (acc[0][2] + acc[1][2]) * g0.y);
#pragma unroll
  for (int o = 1; o < D / 32; o <<= 1) {  // the lanes of one query
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    s[1] += __shfl_xor_sync(0xffffffffu, s[1], o);
  }
}

// the low nibbles of a's bytes and the high nibbles of b's
__device__ __forceinline__ uint32_t low_nibbles(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(d) : "r"(a), "r"(b), "n"(0x0f0f0f0f));
  return d;
}

// P^T of a slice as B fragments (column gq: query gq; w0: tokens 4tq, 4tq + 1,
// w1: 4tq + 2, 4tq + 3) from its weights, laid out as its scores.
__device__ __forceinline__ void weights(const float (&p)[4], uint32_t &w0, uint32_t &w1) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const uint32_t pa = pack2_rn<kF16>(p[0], p[2]), pb = pack2_rn<kF16>(p[1], p[3]);  // tokens 2gq, 2gq + 1
  const int from0 = (2 * tq) * 4 + (gq >> 1), from1 = from0 + 4;
  const uint32_t a0 = __shfl_sync(0xffffffffu, pa, from0), b0 = __shfl_sync(0xffffffffu, pb, from0);
  const uint32_t a1 = __shfl_sync(0xffffffffu, pa, from1), b1 = __shfl_sync(0xffffffffu, pb, from1);
  w0 = (gq & 1) ? b0 : a0;
  w1 = (gq & 1) ? b1 : a1;
}
// The same when spread (queries past the group's repeat one of them).
template <int D, int G>
__device__ __forceinline__ void weights_spread(const float (&p)[2], uint32_t &w0, uint32_t &w1) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const uint32_t pk = pack2_rn<kF16>(p[0], p[1]);
  const int from = (2 * tq) * 4 + (G == 2 ? 2 * (gq & 1) : 0);  // (query 1's scores are in lanes tq 2 and 3)
  w0 = __shfl_sync(0xffffffffu, pk, from);
  w1 = __shfl_sync(0xffffffffu, pk, from + 4);
}

// O^T += V^T P^T of a slice.
template <int D>
__device__ __forceinline__ void accumulate(State<D> &st, const VSlice<D> &c, uint32_t w0, uint32_t w1) {
  const uint32_t sA = e4m3x2_to_half2(c.s), sB = e4m3x2_to_half2(c.s >> 16);  // tokens (4tq, +1), (+2, +3)
  uint32_t eA[VSlice<D>::W][4], oA[VSlice<D>::W][4], eB[VSlice<D>::W][4], oB[VSlice<D>::W][4];
#pragma unroll
  for (int w = 0; w < VSlice<D>::W; ++w) {
    const uint32_t v0 = c.c[0][w], v1 = c.c[1][w], v2 = c.c[2][w], v3 = c.c[3][w];
    e2m1x8_to_half2x4(low_nibbles(v0, v1 << 4), eA[w]);
    e2m1x8_to_half2x4(low_nibbles(v0 >> 4, v1), oA[w]);
    e2m1x8_to_half2x4(low_nibbles(v2, v3 << 4), eB[w]);
    e2m1x8_to_half2x4(low_nibbles(v2 >> 4, v3), oB[w]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      eA[w][i] = hmul2_bits(eA[w][i], sA);
      oA[w][i] = hmul2_bits(oA[w][i], sA);
      eB[w][i] = hmul2_bits(eB[w][i], sB);
      oB[w][i] = hmul2_bits(oB[w][i], sB);
    }
  }
#pragma unroll
  for (int mi = 0; mi < State<D>::MT; ++mi) {
    // local dimensions mi (row gq) and MT + mi (row gq + 8)
    const int lo = mi, hi = State<D>::MT + mi;
    const uint32_t r0 = (lo & 1) ? oA[lo / 8][lo % 8 / 2] : eA[lo / 8][lo % 8 / 2];
    const uint32_t r1 = (hi & 1) ? oA[hi / 8][hi % 8 / 2] : eA[hi / 8][hi % 8 / 2];
    const uint32_t r2 = (lo & 1) ? oB[lo / 8][lo % 8 / 2] : eB[lo / 8][lo % 8 / 2];
    const uint32_t r3 = (hi & 1) ? oB[hi / 8][hi % 8 / 2] : eB[hi / 8][hi % 8 / 2];
    mma(st.o[mi], r0, r1, r2, r3, w0, w1);
  }
}

// ---- a warp's ring of steps in shared memory
//
// A slot holds two slices, each K's 16 rows of codes, V's, and each one's
// scales as [group][token].  The 16-byte chunks of a 128-byte line of code
// rows are exchanged within the line (slot ^ swizzle(line)) so that the eight
// lanes (K) or sixteen (V) of a shared-memory phase read different banks.
constexpr int kRing = 2;  // slots a warp

template <int D>
struct Ring {
  static constexpr int CODES = kSlice * D / 2;
  static constexpr int SCALES = kSlice * D / kFp4Group;
  static constexpr int V = CODES, KS = 2 * CODES, VS = KS + SCALES, SLICE = VS + SCALES, SLOT = 2 * SLICE;
  static constexpr int CHUNKS = CODES / 16;  // 16-byte chunks of a slice's codes: 64 or 32
  __device__ __forceinline__ static int swizzle(int line) {
    return D == 128 ? (2 * ((line >> 1) & 3)) ^ (4 * (line & 1)) : 2 * (line & 3);
  }
  // place of the 16-byte chunk c of a slice's rows (row-major)
  __device__ __forceinline__ static int place(int c) { return (c >> 3) * 128 + (((c & 7) ^ swizzle(c >> 3)) << 4); }
};

// The lane's codes and scales of a slice.
template <int D, bool SPREAD>
__device__ __forceinline__ KSlice<D> read_k(const uint8_t *slice) {
  using R = Ring<D>;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  KSlice<D> k;
#pragma unroll
  for (int r = 0; r < 2; ++r) {  // rows 2gq, 2gq + 1
    if constexpr (D == 128) {
      const uint4 x = lds128(slice + R::place((2 * gq + r) * 4 + tq));
      k.c[r][0] = x.x;
      k.c[r][1] = x.y;
      k.c[r][2] = x.z;
      k.c[r][3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2 *>(slice + R::place((2 * gq + r) * 2 + (tq >> 1)) + (tq & 1) * 8);
      k.c[r][0] = x.x;
      k.c[r][1] = x.y;
    }
  }
  constexpr bool TWO = SPREAD || D == 128;
  const int group = SPREAD ? 2 * tq % (D / kFp4Group) : tq * (D / 64);
#pragma unroll
  for (int i = 0; i < (TWO ? 2 : 1); ++i)
    k.s[i] = *reinterpret_cast<const uint16_t *>(slice + R::KS + (group + i) * 16 + 2 * gq);
  return k;
}
template <int D>
__device__ __forceinline__ VSlice<D> read_v(const uint8_t *slice) {
  using R = Ring<D>;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  VSlice<D> v;
#pragma unroll
  for (int r = 0; r < 4; ++r) {  // rows 4tq .. 4tq + 3
    if constexpr (D == 128) {
      const uint2 x =
          *reinterpret_cast<const uint2 *>(slice + R::V + R::place((4 * tq + r) * 4 + (gq >> 1)) + (gq & 1) * 8);
      v.c[r][0] = x.x;
      v.c[r][1] = x.y;
    } else {
      v.c[r][0] =
          *reinterpret_cast<const uint32_t *>(slice + R::V + R::place((4 * tq + r) * 2 + (gq >> 2)) + (gq & 3) * 4);
    }
  }
  v.s = *reinterpret_cast<const uint32_t *>(slice + R::VS + (gq * (D / 8) / kFp4Group) * 16 + 4 * tq);
  return v;
}

// The step in a slot, n of its 32 tokens valid (1..32).  Places behind them
// may hold any bits, NaN scales among them: their scores become -inf and
// their V scales 0.
template <int D>
__device__ __forceinline__ void attend(State<D> &st, const uint8_t *slot, int n) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  float a[4], b[4];
  scores<D>(st, read_k<D, false>(slot), a);
  scores<D>(st, read_k<D, false>(slot + Ring<D>::SLICE), b);
  if (n < kStep) {  // warp-uniform
    if (2 * gq >= n) a[0] = a[1] = -INFINITY;
    if (2 * gq + 1 >= n) a[2] = a[3] = -INFINITY;
    if (kSlice + 2 * gq >= n) b[0] = b[1] = -INFINITY;
    if (kSlice + 2 * gq + 1 >= n) b[2] = b[3] = -INFINITY;
  }
  // ---- online softmax of query columns 2tq, 2tq + 1.  The maximum is brought
  // up, and the state rescaled, only when some score passes it by 2^8; each
  // lane compares its own scores, so a step that does not need it shuffles
  // nothing.
  float x0 = fmaxf(max3(a[0], a[2], b[0]), b[2]), x1 = fmaxf(max3(a[1], a[3], b[1]), b[3]);
  if (__any_sync(0xffffffffu, x0 > st.top[0] || x1 > st.top[1])) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
    }
    const bool up0 = x0 > st.top[0], up1 = x1 > st.top[1];
    const float n0 = x0 * st.mult[0], n1 = x1 * st.mult[1];
    const float f0 = up0 ? ex2(st.m[0] - n0) : 1.f, f1 = up1 ? ex2(st.m[1] - n1) : 1.f;
    if (up0) {
      st.m[0] = n0;
      st.top[0] = fmaf(kLazy, st.lift[0], x0);
    }
    if (up1) {
      st.m[1] = n1;
      st.top[1] = fmaf(kLazy, st.lift[1], x1);
    }
#pragma unroll
    for (int i = 0; i < State<D>::MT; ++i) {
      st.o[i][0] *= f0;
      st.o[i][2] *= f0;
      st.o[i][1] *= f1;
      st.o[i][3] *= f1;
    }
    st.l[0] *= f0;
    st.l[1] *= f1;
    st.far = __any_sync(0xffffffffu, !(fmaxf(fabsf(st.m[0]), fabsf(st.m[1])) <= kFar));
  }
  if (!st.far) {
    // (the rounding of m is one factor of all of a query's weights: at most 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = ex2(fmaf(a[i], st.mult[i & 1], -st.m[i & 1]));
      b[i] = ex2(fmaf(b[i], st.mult[i & 1], -st.m[i & 1]));
    }
  } else {  // scores whose product has to be rounded as the maximum's was
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = ex2(__fsub_rn(__fmul_rn(a[i], st.mult[i & 1]), st.m[i & 1]));
      b[i] = ex2(__fsub_rn(__fmul_rn(b[i], st.mult[i & 1]), st.m[i & 1]));
    }
  }
  st.l[0] += (a[0] + a[2]) + (b[0] + b[2]);
  st.l[1] += (a[1] + a[3]) + (b[1] + b[3]);
  VSlice<D> va = read_v<D>(slot), vb = read_v<D>(slot + Ring<D>::SLICE);
  if (n < kStep) {
    const int la = n - 4 * tq, lb = la - kSlice;  // valid ones of the lane's four tokens of a slice
    va.s &= la >= 4 ? 0xffffffffu : la <= 0 ? 0u : (1u << (8 * la)) - 1u;
    vb.s &= lb >= 4 ? 0xffffffffu : lb <= 0 ? 0u : (1u << (8 * lb)) - 1u;
  }
  uint32_t w0, w1;
  weights(a, w0, w1);
  accumulate<D>(st, va, w0, w1);
  weights(b, w0, w1);
  accumulate<D>(st, vb, w0, w1);
}

// The same when spread: a lane has two tokens' scores a slice, of one query,
// and its state in m[0], l[0], top[0].
template <int D, int G>
__device__ __forceinline__ void attend_spread(State<D> &st, const uint8_t *slot, int n) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  float a[2], b[2];
  scores_spread<D>(st, read_k<D, true>(slot), a);
  scores_spread<D>(st, read_k<D, true>(slot + Ring<D>::SLICE), b);
  if (n < kStep) {
    if (2 * gq >= n) a[0] = -INFINITY;
    if (2 * gq + 1 >= n) a[1] = -INFINITY;
    if (kSlice + 2 * gq >= n) b[0] = -INFINITY;
    if (kSlice + 2 * gq + 1 >= n) b[1] = -INFINITY;
  }
  float x = fmaxf(max3(a[0], a[1], b[0]), b[1]);
  if (__any_sync(0xffffffffu, x > st.top[0])) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    const bool up = x > st.top[0];
    const float y = x * st.mult[0], f = up ? ex2(st.m[0] - y) : 1.f;
    if (up) {
      st.m[0] = y;
      st.top[0] = fmaf(kLazy, st.lift[0], x);
    }
    st.l[0] *= f;
    // columns 2tq and 2tq + 1 of O^T: queries 0 and 1 in lanes tq 0
    const float f1 = G == 2 ? __shfl_sync(0xffffffffu, f, gq * 4 + 2) : f;
#pragma unroll
    for (int i = 0; i < State<D>::MT; ++i) {
      st.o[i][0] *= f;
      st.o[i][2] *= f;
      st.o[i][1] *= f1;
      st.o[i][3] *= f1;
    }
    st.far = __any_sync(0xffffffffu, !(fabsf(st.m[0]) <= kFar));
  }
  if (!st.far) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = ex2(fmaf(a[i], st.mult[0], -st.m[0]));
      b[i] = ex2(fmaf(b[i], st.mult[0], -st.m[0]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = ex2(__fsub_rn(__fmul_rn(a[i], st.mult[0]), st.m[0]));
      b[i] = ex2(__fsub_rn(__fmul_rn(b[i], st.mult[0]), st.m[0]));
    }
  }
  st.l[0] += (a[0] + a[1]) + (b[0] + b[1]);
  VSlice<D> va = read_v<D>(slot), vb = read_v<D>(slot + Ring<D>::SLICE);
  if (n < kStep) {
    const int la = n - 4 * tq, lb = la - kSlice;
    va.s &= la >= 4 ? 0xffffffffu : la <= 0 ? 0u : (1u << (8 * la)) - 1u;
    vb.s &= lb >= 4 ? 0xffffffffu : lb <= 0 ? 0u : (1u << (8 * lb)) - 1u;
  }
  uint32_t w0, w1;
  weights_spread<D, G>(a, w0, w1);
  accumulate<D>(st, va, w0, w1);
  weights_spread<D, G>(b, w0, w1);
  accumulate<D>(st, vb, w0, w1);
}

// 16 or 8 bytes from global to shared memory (address in the shared window).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// What a lane needs to start the copies of a step into a slot: its own places
// in the first tile and in the slot, so that a copy costs one multiply-add
// for its source.
template <int D, int BS>
struct Copier {
  using R = Ring<D>;
  static constexpr uint32_t TILE = BS * fp4_row_bytes(D), CODES = BS * fp4_code_bytes(D);
  static constexpr int GROUPS = D / kFp4Group;
  static constexpr int BLOCKS = kStep / BS;  // of a step: 1, 2 or 4
  // Chunks lane and lane + 32 of a slice go to place(lane) and, two pairs of
  // lines on, to place(lane) ^ 64 past 512 bytes.
  static constexpr int ROUNDS = R::CHUNKS / 32;
  const uint8_t *k, *v;  // the lane's chunk of a slice in the first tile
  const uint8_t *scale;  // the lane's scale row there, of K or of V
  uint32_t chunk, row;   // places in a slot of the chunk and of the scale row

  __device__ __forceinline__ explicit Copier(const Fp4Params &p) {
    const int lane = threadIdx.x & 31;
    // (blocks of 8 at D 64: the upper half of the lanes copies a slice's second block)
    const int c = BLOCKS == 4 && ROUNDS == 1 ? lane & 15 : lane;
    k = p.k_cache + c * 16;
    v = p.v_cache + c * 16;
    chunk = R::place(lane);
    scale = (lane / GROUPS & 1 ? p.v_cache : p.k_cache) + CODES + lane % GROUPS * BS;
    row = R::KS + lane % (2 * GROUPS) * 16;
    // the upper lanes' scale rows: the second slice's, or (blocks of 8) a
    // slice's second block's 8 bytes
    if (lane >= 2 * GROUPS) {
      row += BLOCKS == 4 ? 8 : R::SLICE;
      if (BLOCKS == 1) scale += 16;
    }
  }
  __device__ __forceinline__ static const uint8_t *at(const uint8_t *base, uint32_t tile) {
    return base + static_cast<uint64_t>(tile) * TILE;
  }
  // t[i]: the tiles (block * KV heads + head) of the step's blocks
  __device__ __forceinline__ void operator()(uint32_t slot, const uint32_t (&t)[BLOCKS]) const {
    const int lane = threadIdx.x & 31;
    const uint32_t to0 = slot + chunk, to1 = slot + (chunk ^ 64u) + 512;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // the slices
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const uint32_t even = t[2 * half % BLOCKS], odd = t[(2 * half + 1) % BLOCKS];  // (blocks of 8: the slice's two)
        const uint32_t tile = BLOCKS < 4 ? t[half * (BLOCKS - 1)] : (ROUNDS == 2 ? i == 0 : lane < 16) ? even : odd;
        // bytes past the lane's chunk of the tile: the first slice, the first 32 chunks
        const int off = (BLOCKS == 1 ? half * R::CODES : 0) + (BLOCKS == 4 ? 0 : i * 512);
        const uint32_t dst = (i == 0 ? to0 : to1) + half * R::SLICE;
        copy_async<16>(dst, at(k, tile) + off);
        copy_async<16>(dst + R::V, at(v, tile) + off);
      }
    }
    const bool upper = lane >= 2 * GROUPS;
    if constexpr (BLOCKS < 4) {  // rows of 16: (slice, K | V, group)
      if (4 * GROUPS == 32 || lane < 4 * GROUPS)
        copy_async<16>(slot + row, at(scale, upper ? t[BLOCKS - 1] : t[0]));
    } else {  // of 8: (block of the slice, K | V, group)
      if (4 * GROUPS == 32 || lane < 4 * GROUPS) {
        copy_async<8>(slot + row, at(scale, upper ? t[1] : t[0]));
        copy_async<8>(slot + row + R::SLICE, at(scale, upper ? t[BLOCKS - 1] : t[BLOCKS - 2]));
      }
    }
  }
};

// Rows of the warps' states in shared memory, padded so that the rows
// of neighbouring queries start 4 banks apart.
template <int D>
constexpr int kRow = D + 4;

__device__ __forceinline__ int clamp_length(int L, int cap) { return min(max(L, 0), cap); }

// A piece of a pair: tokens [t0, t1) of sequence s for KV head h.
struct Piece {
  int s, h, L, t0, t1;
  bool first, last;  // whether it holds the pair's first, last token
};

template <int QT, int D, int G, int BS>
__global__ void __launch_bounds__(kFpThreads, kCtas) decode_fp4_kernel(const __grid_constant__ Fp4Params p) {
  // the warps' rings, then their states at a piece's end, [warp][query][kRow<D>]
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int RING = kRing * Ring<D>::SLOT;
  float *s_o = reinterpret_cast<float *>(smem + kWarps * RING);
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ long long s_wsum[kWarps];
  __shared__ long long s_base;
  __shared__ int s_first;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int S = p.num_seqs, H = p.num_kv_heads;

  // ---- the share: its first piece is KV head h of sequence s from unit off
  // of the pair, the number-th of the pair's pieces; left: units not yet taken
  // (lengths only: this kernel may start before the one ahead of it ends)
  auto length = [&](int s) { return clamp_length(__ldg(p.seq_lens + s), p.len_cap); };
  auto checked_length = [&](int s, bool reports) {
    const int L = __ldg(p.seq_lens + s);
    if (reports && (L < 0 || L > p.len_cap)) record_error(p.err, kErrSeqLen);
    return clamp_length(L, p.len_cap);
  };
  auto units = [&](int L) { return kPairCost + max(1, (L + kUnit - 1) / kUnit); };  // of a pair
  const bool cut = p.cut != 0;
  const long long b = blockIdx.x;
  int s, h, off = 0, number = 0;
  long long left;
  if (!cut && gridDim.x == static_cast<long long>(S) * H) {  // a CTA for each pair
    s = blockIdx.x / H;
    h = blockIdx.x - s * H;
    left = units(checked_length(s, h == 0 && tid == 0));
    grid_dependency_wait();
    launch_dependents();
  } else {
    // units of all pairs before each thread's run of sequences
    const int per = (S + kFpThreads - 1) / kFpThreads;
    const int a0 = min(S, tid * per), a1 = min(S, a0 + per);
    long long mine = 0;
    for (int i = a0; i < a1; ++i) mine += static_cast<long long>(units(checked_length(i, blockIdx.x == 0))) * H;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_wsum[warp] = upto;
    __syncthreads();
    long long U = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_wsum[w];
      U += s_wsum[w];
    }
    before += upto - mine;  // units before this thread's run
    // (cut pairs' pieces have their places when a share is two partitions long)
    long long n = gridDim.x;
    if (cut) n = min(n, max(1ll, U * kUnit / (2ll * p.partition_size)));
    const long long u0 = b * U / n;
    left = b < n ? (b + 1) * U / n - u0 : 0;
    // the sequence that holds unit u0, and the units before it
    if (left > 0 && before <= u0 && u0 < before + mine) {
      long long base = before;
      int i = a0;
      for (; i < a1 - 1; ++i) {
        const long long x = static_cast<long long>(units(length(i))) * H;
        if (u0 < base + x) break;
        base += x;
      }
      s_first = i;
      s_base = base;
    }
    __syncthreads();
    grid_dependency_wait();
    launch_dependents();  // the merge (or the next call, which waits for this grid before it writes)
    if (left <= 0) return;
    s = s_first;
    const int nu = units(length(s));
    const long long rel = u0 - s_base;
    h = static_cast<int>(rel / nu);
    off = static_cast<int>(rel - static_cast<long long>(h) * nu);
    // (counted from the holder of the pair's first token)
    if (off > kPairCost) number = static_cast<int>(b - ((u0 - off + kPairCost + 1) * n - 1) / U);
    if (!cut && off > 0) {  // whole pairs go to the CTA that holds their first unit
      left -= nu - off;
      off = 0;
      ++h;
    }
  }
  auto advance = [&](Piece &x) {
    if (left <= 0) return false;
    if (h == H) {
      h = off = 0;
      ++s;
    }
    x.s = s;
    x.h = h;
    x.L = length(s);
    const int nu = units(x.L);
    const int end = cut && left < nu - off ? off + static_cast<int>(left) : nu;
    left -= end - off;
    x.first = off <= kPairCost;
    x.last = end == nu;
    x.t0 = max(0, off - kPairCost) * kUnit;
    x.t1 = min(x.L, (end - kPairCost) * kUnit);
    off = end;
    if (x.last) {
      off = 0;
      ++h;
    }
    return end > kPairCost;  // (else the share ends before the pair's first token)
  };

  uint8_t *ring = smem + warp * RING;
  const uint32_t ring_addr = smem_addr(ring);
  const Copier<D, BS> copy(p);
  constexpr int BLOCKS = Copier<D, BS>::BLOCKS, WIN = 32 / BLOCKS;  // steps of a window of blocks
  // The warp's steps i = 0, 1, ... of a piece: from token t0 + 32 (warp + 4 i).
  auto steps_of = [&](const Piece &x) {
    const int t = x.t0 + kStep * warp;
    return t < x.t1 ? (x.t1 - t + kStep * kWarps - 1) / (kStep * kWarps) : 0;
  };
  // The tiles of steps i0 .. i0 + WIN - 1: lane i has that of block i % BLOCKS
  // of step i0 + i / BLOCKS (past the last block, the last one's).
  auto window = [&](const Piece &x, int i0, int steps) {
    uint32_t tile = 0;
    const int i = i0 + lane / BLOCKS;
    if (i < steps) {
      const int t = x.t0 + kStep * (warp + kWarps * i);
      int blk = __ldg(p.block_tables + static_cast<size_t>(x.s) * p.max_blocks +
                      min(t / BS + lane % BLOCKS, (x.L - 1) / BS));
      if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks)) {
        record_error(p.err, kErrBlockIndex);
        blk = 0;
      }
      tile = static_cast<uint32_t>(blk) * H + x.h;
    }
    return tile;
  };
  uint32_t slot = 0;  // the ring slot in use; the next step goes to the other
  auto issue = [&](uint32_t win, int i, uint32_t to) {  // step i of its window
    uint32_t t[BLOCKS];
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) t[j] = __shfl_sync(0xffffffffu, win, i * BLOCKS + j);
    copy(ring_addr + to, t);
  };

  Piece cur, nxt;
  if (!advance(cur)) return;
  int steps = steps_of(cur);
  uint32_t win = window(cur, 0, steps);
  if (steps > 0) issue(win, 0, slot);
  while (true) {  // the pieces of the share
    // ahead of this piece's loop: its next window, the next piece and its first window
    uint32_t win2 = window(cur, WIN, steps);
    const bool more = advance(nxt);
    const int nsteps = more ? steps_of(nxt) : 0;
    const uint32_t nwin = more ? window(nxt, 0, nsteps) : 0;
    State<D> st;
    float qk = p.qk_scale_log2, vsc = p.v_scale;
    if (p.k_head_scale != nullptr) {
      qk *= __ldg(p.k_head_scale + cur.h);
      vsc = __ldg(p.v_head_scale + cur.h);
    }
    load_q<QT, D, G>(st, p.q + (static_cast<size_t>(cur.s) * p.num_q_heads + cur.h * G) * D * 2, qk);
    if (steps == 0 && nsteps > 0) issue(nwin, 0, slot);
    int valid = cur.t1 - cur.t0 - kStep * warp;  // tokens from the step's first to the piece's end
    for (int i = 0, w = 1; i < steps; ++i, ++w, valid -= kStep * kWarps) {  // w: the next step's place in its window
      cp_async_commit();
      cp_async_wait<0>();  // the step has landed for this lane
      __syncwarp();        // and for the others; the one before has been read by all
      const uint32_t other = slot ^ Ring<D>::SLOT;
      if (i + 1 < steps) {
        if (w == WIN) {
          win = win2;
          win2 = window(cur, i + 1 + WIN, steps);
          w = 0;
        }
        issue(win, w, other);
      } else if (nsteps > 0) {
        issue(nwin, 0, other);
      }
      if constexpr (kSpread<D, G>)
        attend_spread<D, G>(st, ring + slot, min(kStep, valid));
      else
        attend<D>(st, ring + slot, min(kStep, valid));
      slot = other;
    }

    if constexpr (kSpread<D, G> && G == 2) {  // query 1's statistics to the lanes of its column of O^T
      st.m[1] = __shfl_sync(0xffffffffu, st.m[0], gq * 4 + 2);
      st.l[1] = __shfl_sync(0xffffffffu, st.l[0], gq * 4 + 2);
    }
    // ---- the warps' states meet (the last piece's have been read by then)
    __syncthreads();
    float l0 = st.l[0], l1 = st.l[1];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = 2 * tq + r;
      if (j < G) {
        float *dst = s_o + (warp * G + j) * kRow<D> + gq * (D / 8);
        if (gq == 0) {
          s_m[warp][j] = st.m[r];
          s_l[warp][j] = r ? l1 : l0;
        }
#pragma unroll
        for (int i = 0; i < State<D>::MT; i += 4) {
          *reinterpret_cast<float4 *>(dst + i) =
              make_float4(st.o[i][r], st.o[i + 1][r], st.o[i + 2][r], st.o[i + 3][r]);
          *reinterpret_cast<float4 *>(dst + D / 16 + i) =
              make_float4(st.o[i][2 + r], st.o[i + 1][2 + r], st.o[i + 2][2 + r], st.o[i + 3][2 + r]);
        }
      }
    }
    __syncthreads();
    {
      constexpr int E = D / 32;  // columns a lane
      const int piece = cur.first ? 0 : number;
      for (int j = warp; j < G; j += kWarps) {  // a warp joins queries warp, warp + 4
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][j]);
        float den = 0.f, x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = s_m[w][j] == -INFINITY ? 0.f : ex2(s_m[w][j] - M);
          den = fmaf(f, s_l[w][j], den);
          const float *src = s_o + (w * G + j) * kRow<D> + lane * E;
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = fmaf(f, src[e], x[e]);
        }
        const float inv = den == 0.f ? 0.f : vsc / den;
        const int hq = cur.h * G + j;
        if (cur.first && cur.last) {
          const size_t at = (static_cast<size_t>(cur.s) * p.num_q_heads + hq) * D + lane * E;
          uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + at);
#pragma unroll
          for (int e = 0; e < E; e += 2) out[e / 2] = pack2_rn<QT>(x[e] * inv, x[e + 1] * inv);
        } else {
          const size_t at = (static_cast<size_t>(cur.s) * p.max_parts + piece) * p.num_q_heads + hq;
#pragma unroll
          for (int e = 0; e < E; e += 2)
            *reinterpret_cast<float2 *>(p.part_o + at * D + lane * E + e) = make_float2(x[e] * inv, x[e + 1] * inv);
          if (lane == 0) p.part_ml[at] = make_float2(M, den);
        }
        // the end of the pair's pieces (none at all when the output is written)
        if (lane == 0 && cur.last && cut) {
          const int e = cur.first ? 0 : piece + 1;
          if (e < p.max_parts)
            p.part_ml[(static_cast<size_t>(cur.s) * p.max_parts + e) * p.num_q_heads + hq] = make_float2(0.f, kWritten);
        }
      }
    }
    if (!more) break;
    cur = nxt;
    steps = nsteps;
    win = nwin;
  }
}

// W warps per (sequence, query head) join its pieces' partials,
// out = sum_j w_j o_j / sum_j w_j with w_j = exp2(m_j - M) l_j, up to the mark
// that ends them.  Warp w takes the pieces w, w + W, ..., eight of them in
// flight; lane l owns D / 32 columns.  One warp (CTAs of four heads) is enough
// for pairs in one or a few pieces, as when there are as many pairs as SMs;
// fewer pairs have more pieces each and get sixteen warps a head: one
// sequence of 131071 tokens with 8 KV heads has 76, and its call took 38.2 us
// with four warps a head, 36.4 with sixteen; 48 sequences of 1000..9000 with
// 8 KV and 16 query heads 51.5 with sixteen, 47.1 with one.
constexpr int kMergeFew = 16;
__host__ __device__ constexpr int merge_warps(int W) { return W == 1 ? 4 : W; }  // of a CTA

template <int QT, int D, int W>
__global__ void __launch_bounds__(32 * merge_warps(W)) merge_fp4_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int E = D / 32, CW = merge_warps(W);
  __shared__ float s_o[W][D];
  __shared__ float s_m[W], s_l[W];
  __shared__ int s_end[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % W;
  const long long head = W == 1 ? blockIdx.x * static_cast<long long>(CW) + warp : blockIdx.x;
  grid_dependency_wait();
  if (W == 1 && head >= static_cast<long long>(p.num_seqs) * p.num_q_heads) return;
  const int s = static_cast<int>(head / p.num_q_heads), hq = static_cast<int>(head % p.num_q_heads);
  const size_t at = static_cast<size_t>(s) * p.max_parts * p.num_q_heads + hq;
  const float2 *ml = p.part_ml + at;
  const float *po = p.part_o + at * D + lane * E;
  const size_t stride = p.num_q_heads;
  float M = -INFINITY, den = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int j0 = 0; j0 < p.max_parts; j0 += 32 * W) {
    // this round: lane l has piece j0 + w0 + W l, and the first mark is the end
    const int j = j0 + w0 + W * lane;
    float2 x = make_float2(-INFINITY, kWritten);
    if (j < p.max_parts) x = ml[j * stride];
    const unsigned marks = __ballot_sync(0xffffffffu, x.y == kWritten);
    int end = marks ? j0 + w0 + W * (__ffs(marks) - 1) : INT_MAX;
    if constexpr (W > 1) {
      if (j0 > 0) __syncthreads();  // (the round before has been read)
      if (lane == 0) s_end[warp] = end;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) end = min(end, s_end[w]);
    }
    if (end == 0) return;  // written by the CTA that held the whole pair
    const int mine = min(32, (min(end, j0 + 32 * W) - j0 - w0 + W - 1) / W);  // (negative: none)
    if (lane >= mine) x = make_float2(-INFINITY, 0.f);
    float top = x.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float N = fmaxf(M, top);
    const float old = M == -INFINITY ? 0.f : ex2(M - N);
    M = N;
    const float w = x.x == -INFINITY ? 0.f : ex2(x.x - N) * x.y;
    float ws = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    den = den * old + ws;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
    const float *src = po + (j0 + w0) * stride * D;
    for (int k0 = 0; k0 < mine; k0 += 8) {
      float2 v[8][E / 2];
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
          v[k][e] = k0 + k < mine ? reinterpret_cast<const float2 *>(src + (k0 + k) * W * stride * D)[e]
                                  : make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          acc[2 * e] = fmaf(wk, v[k][e].x, acc[2 * e]);
          acc[2 * e + 1] = fmaf(wk, v[k][e].y, acc[2 * e + 1]);
        }
      }
    }
    if (end <= j0 + 32 * W) break;
  }
  uint16_t *out = static_cast<uint16_t *>(p.out) + (static_cast<size_t>(s) * p.num_q_heads + hq) * D;
  if constexpr (W == 1) {
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      reinterpret_cast<uint32_t *>(out + lane * E)[e / 2] = pack2_rn<QT>(acc[e] * inv, acc[e + 1] * inv);
  } else {
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = den;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
    __syncthreads();
    const int d = threadIdx.x * 2;
    if (d >= D) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w]);
    float l = 0.f, a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - top);
      l = fmaf(f, s_l[w], l);
      a = fmaf(f, s_o[w][d], a);
      b = fmaf(f, s_o[w][d + 1], b);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint32_t *>(out + d) = pack2_rn<QT>(a * inv, b * inv);
  }
}

template <int QT, int D, int G, int BS>
pa_status launch(const Fp4Params &p, const DeviceInfo &dev, cudaStream_t stream) {
  constexpr int smem = kWarps * (kRing * Ring<D>::SLOT + G * kRow<D> * 4);
  static_assert(kCtas * (smem + 2048) <= kSmemPerSm, "the CTAs of an SM fit its shared memory");
  static bool configured[64];  // per device: dynamic shared memory already allowed
  int id = 0;
  cudaError_t e = cudaGetDevice(&id);
  if (e != cudaSuccess) return cuda_fail(e);
  if (id < 0 || id >= 64 || !configured[id]) {
    e = cudaFuncSetAttribute(decode_fp4_kernel<QT, D, G, BS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e);
    if (id >= 0 && id < 64) configured[id] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // no more CTAs than pairs (when they are dealt out whole) or than the
  // longest lengths give units
  const long long pairs = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
  const long long most = p.cut ? pairs * p.max_parts : pairs;
  const long long slots = static_cast<long long>(dev.sm_count) * kCtas;
  cfg.gridDim = dim3(static_cast<unsigned>(most < slots ? most : slots));
  cfg.blockDim = dim3(kFpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_fp4_kernel<QT, D, G, BS>, p);
  if (e != cudaSuccess) return cuda_fail(e);
  if (p.cut) {
    const long long heads = static_cast<long long>(p.num_seqs) * p.num_q_heads;
    const bool many = pairs >= dev.sm_count;
    const int warps = merge_warps(many ? 1 : kMergeFew);
    cfg.gridDim = dim3(static_cast<unsigned>(many ? (heads + warps - 1) / warps : heads));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, many ? merge_fp4_kernel<QT, D, 1> : merge_fp4_kernel<QT, D, kMergeFew>, p);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return PA_OK;
}

template <int BS, int QT, int D>
pa_status by_group(int group, const Fp4Params &p, const DeviceInfo &dev, cudaStream_t s) {
  switch (group) {
    case 1: return launch<QT, D, 1, BS>(p, dev, s);
    case 2: return launch<QT, D, 2, BS>(p, dev, s);
    case 4: return launch<QT, D, 4, BS>(p, dev, s);
    case 8: return launch<QT, D, 8, BS>(p, dev, s);
  }
  return PA_ERR_UNSUPPORTED;
}

// The instantiations of one block size.
template <int BS>
pa_status dispatch(int q_dtype, int head_dim, int group, const DecodeParams &d, const DeviceInfo &dev,
                   cudaStream_t stream) {
  Fp4Params p{};
  p.out = d.out;
  p.q = d.q;
  p.k_cache = d.k_cache;
  p.v_cache = d.v_cache;
  p.block_tables = d.block_tables;
  p.seq_lens = d.seq_lens;
  p.num_seqs = d.num_seqs;
  p.num_q_heads = d.num_q_heads;
  p.num_kv_heads = d.num_kv_heads;
  p.num_blocks = d.num_blocks;
  p.max_blocks = d.max_blocks;
  p.len_cap = d.len_cap;
  p.max_parts = d.max_parts;
  p.partition_size = d.partition_size;
  p.cut = d.max_parts > 1 && d.len_cap > kWholeTokens;
  p.qk_scale_log2 = d.qk_scale_log2;
  p.v_scale = d.v_scale;
  p.k_head_scale = d.k_head_scale;
  p.v_head_scale = d.v_head_scale;
  p.part_ml = d.part_ml;
  p.part_o = d.part_o;
  p.err = d.err;
  if (q_dtype == kF16)
    return head_dim == 64 ? by_group<BS, kF16, 64>(group, p, dev, stream)
                          : by_group<BS, kF16, 128>(group, p, dev, stream);
  return head_dim == 64 ? by_group<BS, kBF16, 64>(group, p, dev, stream)
                        : by_group<BS, kBF16, 128>(group, p, dev, stream);
}

}  // namespace
}  // namespace pa
