// Paged decode attention over a four-bit cache (PA_FP4) for sm_103a.
//
// Work decomposition.  The (sequence, KV head) pairs, in sequence order, are
// laid end to end in units of 64 tokens, and CTA b of n takes the units
// [b U / n, (b + 1) U / n) of the U in all: equal shares whatever the
// lengths, found by each CTA from a scan of the lengths (no plan launch, no
// claims).  A CTA's share is a run of pieces, one per pair it touches.  A
// pair that falls to one CTA whole is written out by it; the pieces of a cut
// pair leave (m, l, O / l) partials, joined by a merge kernel (the
// flash-decoding reduction).  Partials live in the layout every cache type's
// workspace has, [sequence, partition, query head]: piece j of a pair uses
// the place of partition j.  A share is at least two partitions long, so a
// pair of L tokens has at most ceil(L / 2P) + 1 pieces, which is at most the
// workspace's max_parts when that is two or more; when it is one, pairs are
// dealt out whole.
//
// A CTA is eight warps.  Within a piece warp w takes the 16-token slices w,
// w + 8, ..., each warp with its own online softmax; the eight states meet
// in shared memory at the piece's end.
//
// One slice is two small products on mma.sync m16n8k16 with fp16 operands
// and fp32 accumulation, S^T = K Q^T and O^T = V^T P^T: tokens, then head
// dimensions, as M, and the query group padded to 8 as N.  Codes widen to
// fp16 exactly (a code times its group's scale is an fp16 value), so the only
// roundings are those of P to fp16 and of the output.
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
#include <limits.h>

#include "pa_fp4.cuh"
#include "pa_fp4.h"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kFpThreads = 32 * kWarps;
constexpr int kSlice = 16;      // tokens of a warp's step
constexpr int kUnit = 64;       // tokens of a unit of work
constexpr float kLazy = 8.f;    // rescale when the maximum grows by more (base 2)
constexpr float kWritten = -1.f;  // l of a partial that marks the end of a pair's pieces

struct Fp4Params {
  void *out;
  const uint8_t *q;
  const uint8_t *k_cache;
  const uint8_t *v_cache;
  const int32_t *block_tables;
  const int32_t *seq_lens;
  int num_seqs, num_q_heads, num_kv_heads, num_blocks, max_blocks;
  int bs, bs_shift;
  int len_cap, max_parts, partition_size;
  float qk_scale_log2, v_scale;
  const float *k_head_scale, *v_head_scale;
  float2 *part_ml;
  float *part_o;
  int *err;
};

// Codes and scales of one slice as a lane reads them.
template <int D>
struct Slice {
  static constexpr int KW = D / 32;  // words of a K row a lane reads (8 codes each)
  static constexpr int VW = D / 64;  // words of a V row a lane reads
  uint32_t k[2][KW];   // tokens 2gq, 2gq + 1
  uint32_t v[4][VW];   // tokens 4tq .. 4tq + 3
  uint32_t ks[KW / 2]; // their scales (two bytes), one for each 16 local dimensions
  uint32_t vs;         // scales of tokens 4tq .. 4tq + 3 in the lane's group
};

template <int D>
struct State {
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;
  uint32_t qb[KSTEPS][2];
  float o[MT][4];
  float m[2], l[2];
  float mult;
};

// q rows of the group (G x D at `q`) as B fragments: column gq is query gq,
// lane tq's local dimensions.  bf16 queries are rounded to fp16 after a
// multiplication by the power of two that brings the group's largest entry
// into [2^13, 2^14), undone on the scores, so that nothing overflows and what
// underflows is 2^-38 of the largest.
template <int QT, int D, int G>
__device__ __forceinline__ void load_q(State<D> &st, const uint8_t *q, float scale) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  constexpr int QW = D / 8;  // words of the lane
  uint32_t w[QW];
  const uint4 *row = reinterpret_cast<const uint4 *>(q + (static_cast<size_t>(gq < G ? gq : 0) * D + tq * (D / 4)) * 2);
#pragma unroll
  for (int i = 0; i < QW / 4; ++i) {
    const uint4 x = gq < G ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
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
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > 0.f && top <= 3.4e38f) {
      int e;
      frexpf(top, &e);
      f = ldexpf(1.f, min(14 - e, 100));
    }
#pragma unroll
    for (int i = 0; i < QW; ++i) {
      const float2 x = half2_bits_to_float2<kBF16>(w[i]);
      w[i] = pack2_rn<kF16>(x.x * f, x.y * f);
    }
  }
#pragma unroll
  for (int kk = 0; kk < State<D>::KSTEPS; ++kk) {
    st.qb[kk][0] = w[2 * kk];
    st.qb[kk][1] = w[2 * kk + 1];
  }
  st.mult = scale / f;
#pragma unroll
  for (int i = 0; i < State<D>::MT; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
  st.m[0] = st.m[1] = -INFINITY;
  st.l[0] = st.l[1] = 0.f;
}

__device__ __forceinline__ uint32_t lo2(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t hi2(uint32_t h) { return __byte_perm(h, h, 0x3232); }

// n: valid tokens of the slice (1..16).  Places behind them may hold any
// bits, NaN scales among them: their scores become -inf and their V scales 0.
template <int D>
__device__ __forceinline__ void attend(State<D> &st, const Slice<D> &c, int n) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  // ---- S^T = K Q^T
  float acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a) acc[a][0] = acc[a][1] = acc[a][2] = acc[a][3] = 0.f;
#pragma unroll
  for (int w = 0; w < Slice<D>::KW; ++w) {
    const uint32_t s2 = e4m3x2_to_half2(c.ks[w / 2]);
    const uint32_t s0 = lo2(s2), s1 = hi2(s2);
    uint32_t a[4], b[4];
    e2m1x8_to_half2x4(c.k[0][w], a);
    e2m1x8_to_half2x4(c.k[1][w], b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = hmul2_bits(a[i], s0);
      b[i] = hmul2_bits(b[i], s1);
    }
    mma16816<kF16>(acc[(2 * w) & 3], a[0], b[0], a[1], b[1], st.qb[2 * w][0], st.qb[2 * w][1]);
    mma16816<kF16>(acc[(2 * w + 1) & 3], a[2], b[2], a[3], b[3], st.qb[2 * w + 1][0], st.qb[2 * w + 1][1]);
  }
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = ((acc[0][i] + acc[1][i]) + (acc[2][i] + acc[3][i])) * st.mult;
  uint32_t vs = c.vs;
  if (n < kSlice) {  // warp-uniform
    if (2 * gq >= n) s[0] = s[1] = -INFINITY;
    if (2 * gq + 1 >= n) s[2] = s[3] = -INFINITY;
    const int left = n - 4 * tq;  // of the lane's four tokens
    vs &= left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
  }
  // ---- online softmax of query columns 2tq, 2tq + 1
  float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
  }
  const bool up0 = x0 > st.m[0] + kLazy, up1 = x1 > st.m[1] + kLazy;
  if (__any_sync(0xffffffffu, up0 || up1)) {
    const float f0 = up0 ? exp2f(st.m[0] - x0) : 1.f, f1 = up1 ? exp2f(st.m[1] - x1) : 1.f;
    if (up0) st.m[0] = x0;
    if (up1) st.m[1] = x1;
#pragma unroll
    for (int i = 0; i < State<D>::MT; ++i) {
      st.o[i][0] *= f0;
      st.o[i][2] *= f0;
      st.o[i][1] *= f1;
      st.o[i][3] *= f1;
    }
    st.l[0] *= f0;
    st.l[1] *= f1;
  }
  const float p0 = exp2f(s[0] - st.m[0]), p1 = exp2f(s[1] - st.m[1]);
  const float p2 = exp2f(s[2] - st.m[0]), p3 = exp2f(s[3] - st.m[1]);
  st.l[0] += p0 + p2;
  st.l[1] += p1 + p3;
  const uint32_t pa = pack2_rn<kF16>(p0, p2), pb = pack2_rn<kF16>(p1, p3);  // tokens 2gq, 2gq + 1
  const int from0 = (2 * tq) * 4 + (gq >> 1), from1 = from0 + 4;
  const uint32_t a0 = __shfl_sync(0xffffffffu, pa, from0), b0 = __shfl_sync(0xffffffffu, pb, from0);
  const uint32_t a1 = __shfl_sync(0xffffffffu, pa, from1), b1 = __shfl_sync(0xffffffffu, pb, from1);
  const uint32_t w0 = (gq & 1) ? b0 : a0, w1 = (gq & 1) ? b1 : a1;
  // ---- O^T += V^T P^T
  const uint32_t sA = e4m3x2_to_half2(vs), sB = e4m3x2_to_half2(vs >> 16);  // tokens (4tq, +1), (+2, +3)
  uint32_t eA[Slice<D>::VW][4], oA[Slice<D>::VW][4], eB[Slice<D>::VW][4], oB[Slice<D>::VW][4];
#pragma unroll
  for (int w = 0; w < Slice<D>::VW; ++w) {
    constexpr uint32_t LO = 0x0f0f0f0fu;
    const uint32_t v0 = c.v[0][w], v1 = c.v[1][w], v2 = c.v[2][w], v3 = c.v[3][w];
    e2m1x8_to_half2x4((v0 & LO) | ((v1 << 4) & ~LO), eA[w]);
    e2m1x8_to_half2x4(((v0 >> 4) & LO) | (v1 & ~LO), oA[w]);
    e2m1x8_to_half2x4((v2 & LO) | ((v3 << 4) & ~LO), eB[w]);
    e2m1x8_to_half2x4(((v2 >> 4) & LO) | (v3 & ~LO), oB[w]);
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
    mma16816<kF16>(st.o[mi], r0, r1, r2, r3, w0, w1);
  }
}

// The lane's codes and scales of the slice of 16 tokens from position t of
// the sequence whose block-table row is `row`; blocks at or past nblk are not
// looked up (their tokens are not valid), nor is one outside the pool.
template <int D>
__device__ __forceinline__ void load_slice(Slice<D> &c, const Fp4Params &p, const int32_t *row, int nblk, int h, int t) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const int tile = p.bs * fp4_row_bytes(D), codes = p.bs * fp4_code_bytes(D);
  auto base = [&](int tok) -> size_t {  // of the token's (block, head) tile
    const int j = min(tok >> p.bs_shift, nblk - 1);
    int b = __ldg(row + j);
    if (static_cast<unsigned>(b) >= static_cast<unsigned>(p.num_blocks)) {
      record_error(p.err, kErrBlockIndex);
      b = 0;
    }
    return (static_cast<size_t>(b) * p.num_kv_heads + h) * tile;
  };
  {  // K: tokens 2gq, 2gq + 1 (of one block)
    const int tok = t + 2 * gq, off = tok & (p.bs - 1);
    const uint8_t *at = p.k_cache + base(tok);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t *src = at + (off + r) * fp4_code_bytes(D) + tq * (D / 8);
      if constexpr (D == 128) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
        c.k[r][0] = x.x;
        c.k[r][1] = x.y;
        c.k[r][2] = x.z;
        c.k[r][3] = x.w;
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
        c.k[r][0] = x.x;
        c.k[r][1] = x.y;
      }
    }
#pragma unroll
    for (int i = 0; i < Slice<D>::KW / 2; ++i)
      c.ks[i] = __ldg(reinterpret_cast<const uint16_t *>(at + codes + (tq * (D / 64) + i) * p.bs + off));
  }
  {  // V: tokens 4tq .. 4tq + 3 (of one block)
    const int tok = t + 4 * tq, off = tok & (p.bs - 1);
    const uint8_t *at = p.v_cache + base(tok);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t *src = at + (off + r) * fp4_code_bytes(D) + gq * (D / 16);
      if constexpr (D == 128) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
        c.v[r][0] = x.x;
        c.v[r][1] = x.y;
      } else {
        c.v[r][0] = __ldg(reinterpret_cast<const uint32_t *>(src));
      }
    }
    c.vs = __ldg(reinterpret_cast<const uint32_t *>(at + codes + (gq * (D / 8) / kFp4Group) * p.bs + off));
  }
}

// Rows of the eight warps' states in shared memory, padded so that the rows
// of neighbouring queries start 4 banks apart.
template <int D>
constexpr int kRow = D + 4;

__device__ __forceinline__ int clamp_length(int L, int cap) { return min(max(L, 0), cap); }

template <int QT, int D, int G>
__global__ void __launch_bounds__(kFpThreads) decode_fp4_kernel(const __grid_constant__ Fp4Params p) {
  extern __shared__ __align__(16) float s_o[];  // [warp][query][kRow<D>]
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  __shared__ long long s_wsum[kWarps];
  __shared__ long long s_first_base;
  __shared__ int s_first;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int S = p.num_seqs, H = p.num_kv_heads;

  // ---- the share: units of all pairs before each thread's run of sequences
  // (lengths only: this kernel may start before the one ahead of it ends)
  auto length = [&](int s) { return clamp_length(__ldg(p.seq_lens + s), p.len_cap); };
  auto units = [&](int s) { return max(1, (length(s) + kUnit - 1) / kUnit); };
  const int per = (S + kFpThreads - 1) / kFpThreads;
  const int a0 = min(S, tid * per), a1 = min(S, a0 + per);
  long long mine = 0;
  for (int s = a0; s < a1; ++s) {
    if (blockIdx.x == 0) {
      const int L = __ldg(p.seq_lens + s);
      if (L < 0 || L > p.len_cap) record_error(p.err, kErrSeqLen);
    }
    mine += static_cast<long long>(units(s)) * H;
  }
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
  grid_dependency_wait();
  launch_dependents();  // the merge (or the next call, which waits for this grid)
  const bool cut = p.max_parts > 1;
  long long n = gridDim.x;
  if (cut) n = min(n, max(1ll, U * kUnit / (2ll * p.partition_size)));
  const long long b = blockIdx.x;
  if (b >= n) return;
  long long u0 = b * U / n, u1 = (b + 1) * U / n;
  if (u0 >= u1) return;
  // the sequence that holds unit u0, and the units before it
  if (before <= u0 && u0 < before + mine) {
    long long base = before;
    int s = a0;
    for (; s < a1 - 1; ++s) {
      const long long x = static_cast<long long>(units(s)) * H;
      if (u0 < base + x) break;
      base += x;
    }
    s_first = s;
    s_first_base = base;
  }
  __syncthreads();
  int s = s_first;
  long long base = s_first_base;

  long long u = u0;
  while (u < u1) {
    const int L = length(s);
    const int nu = max(1, (L + kUnit - 1) / kUnit);
    const int h = static_cast<int>((u - base) / nu);
    if (h >= H) {  // past the sequence
      base += static_cast<long long>(nu) * H;
      ++s;
      continue;
    }
    const long long pair = base + static_cast<long long>(h) * nu;  // the pair's first unit
    const int off = static_cast<int>(u - pair);
    if (!cut && off > 0) {  // whole pairs go to the CTA that holds their first unit
      u = pair + nu;
      continue;
    }
    const int end = cut ? static_cast<int>(min(static_cast<long long>(nu), u1 - pair)) : nu;
    u = pair + end;
    const int t0 = off * kUnit, t1 = min(L, end * kUnit);
    const bool first = off == 0, last = end == nu;

    State<D> st;
    float qk = p.qk_scale_log2, vsc = p.v_scale;
    if (p.k_head_scale != nullptr) {
      qk *= __ldg(p.k_head_scale + h);
      vsc = __ldg(p.v_head_scale + h);
    }
    load_q<QT, D, G>(st, p.q + (static_cast<size_t>(s) * p.num_q_heads + h * G) * D * 2, qk);
    const int32_t *row = p.block_tables + static_cast<size_t>(s) * p.max_blocks;
    const int nblk = (L + p.bs - 1) >> p.bs_shift;
    for (int t = t0 + kSlice * warp; t < t1; t += kSlice * kWarps) {
      Slice<D> c;
      load_slice<D>(c, p, row, nblk, h, t);
      attend<D>(st, c, min(kSlice, t1 - t));
    }

    // ---- the eight warps' states meet
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
          *reinterpret_cast<float4 *>(dst + i) = make_float4(st.o[i][r], st.o[i + 1][r], st.o[i + 2][r], st.o[i + 3][r]);
          *reinterpret_cast<float4 *>(dst + D / 16 + i) =
              make_float4(st.o[i][2 + r], st.o[i + 1][2 + r], st.o[i + 2][2 + r], st.o[i + 3][2 + r]);
        }
      }
    }
    __syncthreads();
    // piece number: the CTAs between this one and the holder of the pair's first unit
    const int piece = first ? 0 : static_cast<int>(b - ((pair + 1) * n - 1) / U);
    for (int i = tid * 2; i < G * D; i += 2 * kFpThreads) {
      const int j = i / D, d = i % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][j]);
      float den = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][j] == -INFINITY ? 0.f : exp2f(s_m[w][j] - M);
        const float2 v = *reinterpret_cast<const float2 *>(s_o + (w * G + j) * kRow<D> + d);
        den = fmaf(f, s_l[w][j], den);
        x = fmaf(f, v.x, x);
        y = fmaf(f, v.y, y);
      }
      const float inv = den == 0.f ? 0.f : vsc / den;
      const int hq = h * G + j;
      if (first && last) {
        uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) +
                                                     (static_cast<size_t>(s) * p.num_q_heads + hq) * D + d);
        *out = pack2_rn<QT>(x * inv, y * inv);
      } else {
        const size_t at = (static_cast<size_t>(s) * p.max_parts + piece) * p.num_q_heads + hq;
        *reinterpret_cast<float2 *>(p.part_o + at * D + d) = make_float2(x * inv, y * inv);
        if (d == 0) p.part_ml[at] = make_float2(M, den);
      }
      // the end of the pair's pieces (none at all when the output is written)
      if (d == 0 && last && cut) {
        const int e = first ? 0 : piece + 1;
        if (e < p.max_parts)
          p.part_ml[(static_cast<size_t>(s) * p.max_parts + e) * p.num_q_heads + hq] = make_float2(0.f, kWritten);
      }
    }
    __syncthreads();
  }
}

// One warp per (sequence, query head): joins its pieces' partials,
// out = sum_j w_j o_j / sum_j w_j with w_j = exp2(m_j - M) l_j, up to the mark
// that ends them.
template <int QT, int D>
__global__ void __launch_bounds__(128) merge_fp4_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long gw = blockIdx.x * 4ll + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (gw >= static_cast<long long>(p.num_seqs) * p.num_q_heads) return;
  const int s = static_cast<int>(gw / p.num_q_heads), hq = static_cast<int>(gw % p.num_q_heads);
  const size_t at = static_cast<size_t>(s) * p.max_parts * p.num_q_heads + hq;
  const float2 *ml = p.part_ml + at;
  const float *po = p.part_o + at * D + lane * E;
  const size_t stride = p.num_q_heads;
  float M = -INFINITY, den = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int j0 = 0; j0 < p.max_parts; j0 += 32) {
    float2 x = make_float2(-INFINITY, kWritten);
    if (j0 + lane < p.max_parts) x = ml[(j0 + lane) * stride];
    const unsigned ended = __ballot_sync(0xffffffffu, x.y == kWritten);
    const int cnt = ended ? __ffs(ended) - 1 : 32;
    if (cnt == 0) {
      if (j0 == 0) return;  // written by the CTA that held the whole pair
      break;
    }
    if (lane >= cnt) x = make_float2(-INFINITY, 0.f);
    float top = x.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float N = fmaxf(M, top);
    const float old = M == -INFINITY ? 0.f : exp2f(M - N);
    M = N;
    const float w = x.x == -INFINITY ? 0.f : exp2f(x.x - N) * x.y;
    float ws = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    den = den * old + ws;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
    for (int k = 0; k < cnt; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float *src = po + (j0 + k) * stride * D;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2 *>(src + e);
        acc[e] = fmaf(wk, v.x, acc[e]);
        acc[e + 1] = fmaf(wk, v.y, acc[e + 1]);
      }
    }
    if (cnt < 32) break;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) +
                                               (static_cast<size_t>(s) * p.num_q_heads + hq) * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack2_rn<QT>(acc[e] * inv, acc[e + 1] * inv);
}

template <int QT, int D, int G>
pa_status launch(const Fp4Params &p, const DeviceInfo &dev, cudaStream_t stream) {
  constexpr int smem = kWarps * G * kRow<D> * 4;
  static_assert(smem <= 48 * 1024, "the states fit the shared memory every kernel may use");
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // no more CTAs than pairs (when they are dealt out whole) or than the
  // longest lengths give units
  const long long pairs = static_cast<long long>(p.num_seqs) * p.num_kv_heads;
  const long long most = p.max_parts > 1 ? pairs * p.max_parts : pairs;
  const long long slots = static_cast<long long>(dev.sm_count) * 2;
  cfg.gridDim = dim3(static_cast<unsigned>(most < slots ? most : slots));
  cfg.blockDim = dim3(kFpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_fp4_kernel<QT, D, G>, p);
  if (e != cudaSuccess) return cuda_fail(e);
  if (p.max_parts > 1) {
    const long long warps = static_cast<long long>(p.num_seqs) * p.num_q_heads;
    cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, merge_fp4_kernel<QT, D>, p);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return PA_OK;
}

template <int QT, int D>
pa_status by_group(int group, const Fp4Params &p, const DeviceInfo &dev, cudaStream_t s) {
  switch (group) {
    case 1: return launch<QT, D, 1>(p, dev, s);
    case 2: return launch<QT, D, 2>(p, dev, s);
    case 4: return launch<QT, D, 4>(p, dev, s);
    case 8: return launch<QT, D, 8>(p, dev, s);
  }
  return PA_ERR_UNSUPPORTED;
}

}  // namespace

pa_status dispatch_decode_fp4(int q_dtype, int head_dim, int group, const DecodeParams &d, const DeviceInfo &dev,
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
  p.bs = d.block_size;
  p.bs_shift = d.block_size == 8 ? 3 : d.block_size == 16 ? 4 : 5;
  p.len_cap = d.len_cap;
  p.max_parts = d.max_parts;
  p.partition_size = d.partition_size;
  p.qk_scale_log2 = d.qk_scale_log2;
  p.v_scale = d.v_scale;
  p.k_head_scale = d.k_head_scale;
  p.v_head_scale = d.v_head_scale;
  p.part_ml = d.part_ml;
  p.part_o = d.part_o;
  p.err = d.err;
  if (q_dtype == kF16)
    return head_dim == 64 ? by_group<kF16, 64>(group, p, dev, stream) : by_group<kF16, 128>(group, p, dev, stream);
  return head_dim == 64 ? by_group<kBF16, 64>(group, p, dev, stream) : by_group<kBF16, 128>(group, p, dev, stream);
}

}  // namespace pa
