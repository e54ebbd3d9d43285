// What the kernels of pa_latent_decode share: parameters, shares of the work,
// the softmax warps' barriers.
#pragma once

#include "pa_latent_common.cuh"
#include "pa_latent.h"
#include "pa_shares.cuh"

namespace pa {

constexpr int kMinTiles = 2;     // a share of fewer tiles only adds joining
constexpr float kLazy = 8.f;     // a row's maximum is raised when a score passes it by more (base 2)
// The largest weight of a row is held as 2^kLift or more: fp16's smallest step
// is 2^-24, so that a weight is off by at most 2^-32 of the largest where it
// would be lost below 2^-25, and the total keeps all of it (131071 tokens 17
// nats below one are 0.4 % of it).  2^(kLazy + kLift) is well inside fp16.
// bf16 has a float's range and needs none of it.
template <int DT>
constexpr float kLift = DT == kF16 ? 7.f : 0.f;
constexpr int kSoftmaxThreads = 256;
// Sequences of up to this many tokens are not split while their blocks (pairs
// of blocks) are at most kWholeWaves for each that the GPU holds: their few
// tiles then take less than a second kernel.  Unsplit and split, in us, 16 and
// 128 heads: 4 sequences of 256 tokens 10.4 / 12.1 and 11.0 / 12.8, of 512
// tokens 15.3 / 12.5 and 14.7 / 15.9; 64 of 256 11.4 / 14.0 and 12.0 / 15.5;
// 152 of 256 (two pairs each, with 128 heads) 11.2 / 20.0 and 24.2 / 23.5; 304
// of 256 23.3 / 25.0 and 56.7 / 47.9; 512 of 64 25.5 / 24.3 and 76.5 / 54.0.
constexpr int kWholeTokens = 256, kWholeWaves = 2;

struct LatentParams {
  CUtensorMap tmap_q;  // [S n H, 576] in boxes of {64, N} (64 rows for a pair)
  CUtensorMap tmap_c;  // the cache, boxes of a slot (or of a block of 8); for a pair, of three of its columns
  CUtensorMap tmap_v;  // for a pair: of four columns
  void *out;
  const uint16_t *cache;
  const int32_t *tables, *lens;
  float2 *part_ml;     // [row tiles, workers, 2, N]
  float *part_o;       // [row tiles, workers, 2, N, 512]
  long long *prefix;   // [S + 1] tiles before sequence s
  int num_seqs, new_tokens, heads, rows, row_tiles /* of a pair's 128 rows */, num_blocks, bs_shift, max_blocks, limit;
  bool whole;          // every share is one sequence: nothing to join
  bool out_sectors;    // out is 32-byte aligned
  float scale_log2;
  int *err;
};

// 64 < rows: a row tile of 128 query rows to a pair of blocks (pa_latent_pair.cu).
// Sets p.row_tiles and *workers, the shares of one row tile.
constexpr int kPairRows = 128, kMaxPairs = 76;
pa_status launch_latent_pair(int dtype, LatentParams &p, const void *q, const void *cache, const pa_latent_desc *desc,
                             int *workers, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return y != 0;
}

__host__ __device__ inline long long worker_count(long long tiles, long long most) {
  const long long n = (tiles + kMinTiles - 1) / kMinTiles;
  return n < most ? n : most;
}

// A drafted token that the rows before it do not see has the weight 0 in them,
// and 0 times a number that is not finite would reach them.  So such numbers
// are taken out of the tokens from a sequence's plain_end on before the second
// product; the rows that do see the token are given not-a-number in those
// dimensions at the end.  (That is what the definition gives: its score is
// infinite or not a number, its weight not a number or 0.)
__device__ __forceinline__ int plain_end(const LatentParams &p, int L) { return L - (p.new_tokens - 1); }

template <int DT>
constexpr uint32_t kNotFinite = DT == kF16 ? 0x7c00u : 0x7f80u;  // an exponent of ones

// Eight elements of which those that are not finite become zero; whether there was one.
template <int DT>
__device__ __forceinline__ bool take_out(uint4 &x) {
  constexpr uint32_t E = kNotFinite<DT>;
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool low = (w[i] & E) == E, high = (w[i] >> 16 & E) == E;
    any |= low || high;
    w[i] &= (low ? 0u : 0xffffu) | (high ? 0u : 0xffff0000u);
  }
  x = make_uint4(w[0], w[1], w[2], w[3]);
  return any;
}

// Token i's row of the cache.
__device__ __forceinline__ const uint16_t *token_row(const LatentParams &p, int s, int i) {
  int b = __ldg(p.tables + static_cast<size_t>(s) * p.max_blocks + (i >> p.bs_shift));
  if (b < 0 || b >= p.num_blocks) b = 0;  // (reported by the TMA warp)
  return p.cache + ((static_cast<size_t>(b) << p.bs_shift) + (i & ((1 << p.bs_shift) - 1))) * kLatentRow;
}

// Zeros to `rows` rows of out from row `first` on, by the whole block.
__device__ __forceinline__ void zero_rows(void *out, long long first, int rows) {
  uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + first * kLatentDim);
  for (int i = threadIdx.x; i < rows * (kLatentDim / 8); i += blockDim.x) to[i] = make_uint4(0u, 0u, 0u, 0u);
}

// One piece of a share: tiles [t0, t1), of TILE tokens, of a sequence, in
// order.
template <int TILE>
struct Walk {
  long long u, end, first;
  int s, L, tiles, t0, t1;
  __device__ __forceinline__ bool next(const LatentParams &p) {
    while (u < end) {
      L = checked_len(p.lens, s, p.limit, nullptr);
      tiles = (L + TILE - 1) / TILE;
      if (tiles == 0) {
        ++s;
        continue;
      }
      t0 = static_cast<int>(u - first);
      t1 = end - u < tiles - t0 ? t0 + static_cast<int>(end - u) : tiles;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ void advance() {
    u += t1 - t0;
    if (t1 == tiles) {
      first += tiles;
      ++s;
    }
  }
};
#endif

}  // namespace pa
