// pa_latent_prefill: expanded causal attention of each sequence's new tokens
// over the latent paged cache.
//
// With c the tokens' latent vectors and r their rotary keys, head h has the
// keys (Uk_h c, r) of 128 + 64 elements and the values Uv_h c of 128.  A new
// token costs 640 operations a head and token of the context against 2176 in
// the absorbed form, and the expansion 262144 a head and token of the
// context, so this form is the cheaper one from about 170 new tokens a
// sequence on.
//
// First kernel (expand): tiles of 128 tokens of a sequence times a head's 256
// rows of (Uk_h; Uv_h) on the 5th-generation tensor cores, two tiles to a pair
// of blocks whose tensor cores work as one (tcgen05 cta_group::2):
//   D = C U^T   M = 256 tokens, N = 256, K = 512
// Each block holds its tile's latent rows (128 KB) for all heads of its share
// and half of the weights' rows, in chunks of 64 columns: a block alone would
// read 64 bytes of weights a clock, more than L2 gives it, a pair reads half
// of that.  D has two buffers in tensor memory (all 512 columns), so that the
// products of a head run while the last one's result is rounded and stored.
// Pairs take equal shares of all (two tiles, head) units.  The result [head,
// token, (key 128, value 128)] and the tokens' rotary keys go to the workspace,
// sequences padded to 128 tokens with zeros.  Keys are rounded to the cache's
// type; values always to fp16, whose step is an eighth of bf16's, times a power
// of two for every 32 tokens of a head where fp16 would not hold them well.
//
// Second kernel (attend): a block is one head and 256 new tokens of a
// sequence, as two tiles of 128, the M of the products:
//   S = Q K^T   N = 64 keys of a stage, K = 192  (S in TMEM, two buffers)
//   O += P V    N = 128, K = 64                  (P over S, O in TMEM)
// Warps 0..7 softmax (a warpgroup a tile, a thread a row), 8 and 11 load keys
// and values, 9 and 10 issue the products, one a tile.  Keys and values have
// rings of their own: a stage's keys are free before its softmax, and a load
// into a freed place takes about 1500 clocks (one ring: 684 and 138 us for the
// two cases below).  The running maximum is raised, and O rescaled, only when
// it grew by more than 2^8.  Sums and maxima are fp32; P is rounded to fp16
// (see kLift), K and V were when they were expanded (half a step each).
// Bound by shared memory, not by the tensor cores: a product's operands come
// from it at 128 bytes a clock, 6 KB for the 32 clocks of one of S, and with
// the stages' arrival that makes about 1660 clocks a stage of both tiles, where
// 1620 are measured and the products alone take 1280.  4095 tokens after 4096,
// 64 heads: 81 us for the expansion, 661 for the attention; 32 sequences of
// 16..512 after 1024, 16 heads: 106 and 126 (768 blocks of about 20 us, five
// rounds of the SMs and a few of a sixth).  That is at 2070 MHz: call after call
// the power limit takes the clock to 1.75 and 1.7 GHz, and the two together
// from 732 to 793 and from 222 to 244 us.  Tried: stages of 128 keys with one S
// buffer a tile (733 us for the 684: the softmax is then in the chain), a third
// of q in tensor memory (747), blocks that go on to the next range (697),
// stages fetched into L2 ahead (even), loads before the block's first barrier
// (even).
// With an fp16 cache P's rounding would show beside the output's where a row
// follows few tokens, so rows of up to 512 tokens take P as two fp16 parts (the
// second is zero for the other rows of their tile: a row's rounding goes by its
// own tokens, whatever comes behind it and wherever its prompt is cut).
#include <limits.h>
#include <math.h>

#include "pa_latent.h"
#include "pa_latent_common.cuh"
#include "pa_shares.cuh"

namespace pa {
namespace {

constexpr int kNope = 128, kValue = 128, kUp = kNope + kValue;  // of a head: keys' share of the latent, values
constexpr int kQk = kNope + kRopeDim;

// ------------------------------------------------------------------ expand
constexpr int kExTokens = 128;
constexpr int kExThreads = 6 * 32;
constexpr int kExTmaWarp = 4, kExMmaWarp = 5;
constexpr int kExGroup32 = 32;                          // tokens with one power of two
constexpr int kExColumns = kLatentDim / 64;             // 128-byte columns of the latent part
constexpr int kExGroup = kExColumns * 1024;             // 8 rows
constexpr int kExABytes = kExTokens / 8 * kExGroup;
constexpr int kExBRows = kUp / 2;                       // of the weights, a block
constexpr int kExBBytes = kExBRows * 128;               // a chunk of 64 columns
constexpr int kExRing = 6;
constexpr int kExSmem = 2048 + kExABytes + kExRing * kExBBytes;

struct ExpandParams {
  CUtensorMap tmap_c;   // the cache's latent columns, a block a box
  CUtensorMap tmap_u;   // [H * 256, 512], boxes of {64, 128}
  const uint8_t *cache;
  const int32_t *tables, *lens;
  uint8_t *kv;          // [H, capacity, 256]
  uint8_t *rope;        // [capacity, 64]
  int32_t *powers;      // [H, capacity / 32]: values are these powers of two times what is stored (kNoValues: zeros)
  long long *prefix;    // [S + 1] token tiles before sequence s
  int num_seqs, heads, num_blocks, bs_shift, max_blocks, limit;
  long long capacity;   // tokens
  int *err;
};

struct ExpandHeader {
  uint64_t a_full, a_empty, b_full[kExRing], b_empty[kExRing], d_full[2], d_empty[2], fin;
  uint32_t tmem;
  int abort;
  ShareScan<128> scan;
};
static_assert(sizeof(ExpandHeader) <= 2048, "the header's place");

// The power of two e for which values of largest magnitude `top` are stored
// as x 2^-e: 0 where fp16 holds them well, from 2^-4 to 2^15 (a step of fp16's
// smallest numbers is then 2^-20 of the largest or less); outside, the multiple
// of four that brings the largest to the near end of that range.  A row's
// weights are scaled by the distance of a group's power from the largest of
// those it follows, and lose bits where that is far: groups of nearly the same
// size have to have nearly the same power, on both sides of the range's ends.
// (Values just below 2^-4 taken to 2^14 would cost their weights 18 bits beside
// a group just above: outputs off by 4 to 9 % at 4096 tokens.)  Multiples of
// four because differing powers cost a second rounding of a stage's weights.
// Groups of zeros take no part.
constexpr int kNoValues = -1024;
__device__ __forceinline__ int value_power(float top) {
  if (top == 0.f) return kNoValues;
  if (!(top > 0.f && top < INFINITY) || (top >= 0x1p-4f && top <= 0x1p15f)) return 0;
  const int lg = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -126);
  return (top < 1.f ? lg + 4 : lg - 11) & ~3;  // to [2^-4, 1) or [2^11, 2^15)
}

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExThreads, 1)
    latent_expand_kernel(const __grid_constant__ ExpandParams p) {
  constexpr uint32_t IDESC = umma_idesc_f16(DT == kF16 ? 0 : 1, 2 * kExTokens, kUp, false);
  extern __shared__ __align__(1024) uint8_t smem[];
  ExpandHeader &hdr = *reinterpret_cast<ExpandHeader *>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster_rank();
  launch_dependents();
  auto tiles_of = [&](int s) -> long long { return (checked_len(p.lens, s, p.limit, p.err) + kExTokens - 1) / kExTokens; };
  ShareScan<128> &scan = hdr.scan;
  scan.scan(p.num_seqs, tiles_of);
  if (blockIdx.x == 0 && threadIdx.x < 128) {  // the sequences' first token tiles, for the second kernel
    const int n = scan.run(p.num_seqs), t = threadIdx.x;
    long long at = scan.base[t];
    for (int s = t * n; s < min(p.num_seqs, (t + 1) * n); ++s) {
      p.prefix[s] = at;
      at += tiles_of(s);
    }
    if (t == 0) p.prefix[p.num_seqs] = scan.total();
  }
  // units: (two token tiles, head)
  const long long tiles = scan.total(), total = (tiles + 1) / 2 * p.heads;
  const long long pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const long long u0 = share_begin(pair, total, pairs), u1 = share_begin(pair + 1, total, pairs);
  if (u0 >= u1) return;  // (both blocks)
  long long u = u0, first;
  int s = scan.find(min(u0 / p.heads * 2 + rank, tiles - 1), p.num_seqs, tiles_of, first);
  volatile int *abort = &hdr.abort;
  uint8_t *as = smem + 2048, *bsm = as + kExABytes;
  if (warp == kExTmaWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_c)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_u)) : "memory");
    mbar_init(&hdr.a_full, 2);  // a block each
    mbar_init(&hdr.a_empty, 1);
    for (int i = 0; i < kExRing; ++i) {
      mbar_init(&hdr.b_full[i], 1);
      mbar_init(&hdr.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hdr.d_full[i], 1);
      mbar_init(&hdr.d_empty[i], 8);  // the warps of both blocks
    }
    mbar_init(&hdr.fin, 1);
    hdr.abort = 0;
    fence_mbar_init();
  }
  if (warp == kExMmaWarp) pair_alloc(&hdr.tmem, 512);
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the other block's mbarriers and tensor memory are there
  tc_fence_after_sync();
  const uint32_t tmem = hdr.tmem;

  // A share as runs of heads of two token tiles, of which this block's is
  // `tile` of sequence s (none past the last: there is nothing to load or
  // store for it, the products of whatever is there go unused).
  struct Run {
    int s, tile, h0, h1, L;
    long long row;  // the tile's first row of the workspace
    bool there;
  };
  auto next = [&](Run &r) {
    if (u >= u1) return false;
    const long long two = u / p.heads, t = two * 2 + rank;
    r.h0 = static_cast<int>(u - two * p.heads);
    r.h1 = u1 - u < p.heads - r.h0 ? r.h0 + static_cast<int>(u1 - u) : p.heads;
    u += r.h1 - r.h0;
    r.there = t < tiles;
    r.row = t * kExTokens;
    r.s = r.tile = r.L = 0;
    if (r.there) {
      for (;; ++s) {
        r.L = checked_len(p.lens, s, p.limit, nullptr);
        const long long n = (r.L + kExTokens - 1) / kExTokens;
        if (t < first + n) break;
        first += n;
      }
      r.s = s;
      r.tile = static_cast<int>(t - first);
    }
    return true;
  };
  Run r;
  if (warp < 4) {
    // -------------------------------------------------------------- results
    bool ok = true;
    int i = 0;
    const int row = threadIdx.x;
    const uint32_t d_empty[2] = {in_block(&hdr.d_empty[0], 0), in_block(&hdr.d_empty[1], 0)};
    while (ok && next(r)) {
      const int token = r.tile * kExTokens + row;
      const bool fits = r.there && r.row + kExTokens <= p.capacity;
      if (r.there && !fits && threadIdx.x == 0) record_error(p.err, kErrSeqLen);
      if (fits && r.h0 == 0) {  // the tile's rotary keys
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (token < r.L) {
          int b = __ldg(p.tables + static_cast<size_t>(r.s) * p.max_blocks + (token >> p.bs_shift));
          if (b < 0 || b >= p.num_blocks) b = 0;  // (reported by the TMA warp)
          const uint8_t *from = p.cache +
                                (((static_cast<size_t>(b) << p.bs_shift) + (token & ((1 << p.bs_shift) - 1))) * kLatentRow +
                                 kLatentDim) * 2;
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __ldg(reinterpret_cast<const uint4 *>(from) + j);
        }
        uint4 *to = reinterpret_cast<uint4 *>(p.rope + (r.row + row) * (kRopeDim * 2));
#pragma unroll
        for (int j = 0; j < 8; ++j) to[j] = x[j];
      }
      for (int h = r.h0; h < r.h1; ++h, ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&hdr.d_full[i & 1], (i >> 1) & 1, abort))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + (i & 1) * kUp + (static_cast<uint32_t>(32 * warp) << 16);
        uint8_t *to = p.kv + ((static_cast<size_t>(h) * p.capacity + r.row + row) * kUp) * 2;
        const bool real = token < r.L;
#pragma unroll
        for (int c = 0; c < kNope; c += 32) {
          uint32_t v[32], w[16];
          tc_ld32(d + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = real ? pack2_rn<DT>(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])) : 0u;
          if (fits) {
            store32(to + c * 2, w);
            store32(to + c * 2 + 32, w + 8);
          }
        }
        float top = 0.f;
        uint32_t v[kValue];
#pragma unroll
        for (int c = 0; c < kValue; c += 32) {
          uint32_t part[32];
          tc_ld32(d + kNope + c, part);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v[c + j] = part[j];
            top = fmaxf(top, fabsf(__uint_as_float(part[j])));
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) pair_arrive(d_empty[i & 1]);
        // (magnitudes compare as their bits do)
        const int e = value_power(__uint_as_float(__reduce_max_sync(0xffffffffu, real ? __float_as_uint(top) : 0u)));
        if (fits && lane == 0)
          p.powers[static_cast<size_t>(h) * (p.capacity / kExGroup32) + r.row / kExGroup32 + warp] = e;
        const float f = e == 0 || e == kNoValues ? 1.f : exp2f(static_cast<float>(-e));
#pragma unroll
        for (int c = 0; c < kValue; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = real ? pack2_rn<kF16>(__uint_as_float(v[c + 2 * j]) * f, __uint_as_float(v[c + 2 * j + 1]) * f) : 0u;
          if (fits) {
            store32(to + (kNope + c) * 2, w);
            store32(to + (kNope + c) * 2 + 32, w + 8);
          }
        }
      }
    }
    if (!ok) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
    }
  } else if (warp == kExTmaWarp) {
    // ------------------------------------------------------------------ TMA
    // (bytes count in the first block, where the products are issued)
    bool ok = true;
    int chunk = 0, runs = 0;
    const uint32_t a_full = in_block(&hdr.a_full, 0);
    while (ok && next(r)) {
      const int boxes = kExTokens >> p.bs_shift;
      const int n_box = r.there ? min(boxes, (r.L - r.tile * kExTokens + (1 << p.bs_shift) - 1) >> p.bs_shift) : 0;
      const uint32_t box = (1u << p.bs_shift) / 8 * kExGroup;
      int b = 0;
      if (lane < n_box) {
        b = __ldg(p.tables + static_cast<size_t>(r.s) * p.max_blocks + r.tile * boxes + lane);
        if (b < 0 || b >= p.num_blocks) {
          record_error(p.err, kErrBlockIndex);
          b = 0;
        }
      }
      if (runs > 0) ok = __all_sync(0xffffffffu, mbar_wait(&hdr.a_empty, (runs - 1) & 1, abort));
      if (!ok) break;
      // each block announces its own tile's bytes
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(a_full), "r"(n_box * box)
                     : "memory");
      __syncwarp();
      if (lane < n_box) pair_load_4d(as + lane * box, &p.tmap_c, 0, 0, 0, b << (p.bs_shift - 3), a_full);
      ++runs;
      if (lane == 0) {
        for (int h = r.h0; ok && h < r.h1; ++h)
          for (int c = 0; c < kExColumns; ++c, ++chunk) {
            const int st = chunk % kExRing;
            if (chunk >= kExRing && !mbar_wait(&hdr.b_empty[st], (chunk / kExRing - 1) & 1, abort)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&hdr.b_full[st], 2 * kExBBytes);
            pair_load_2d(bsm + st * kExBBytes, &p.tmap_u, c * 64, h * kUp + rank * kExBRows, in_block(&hdr.b_full[st], 0));
          }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (ok && runs > 0) {  // the last products' arrivals in this block
      chunk = __shfl_sync(0xffffffffu, chunk, 0);
      for (int j = max(0, chunk - kExRing); j < chunk; ++j)
        ok = ok && mbar_wait(&hdr.b_empty[j % kExRing], (j / kExRing) & 1, abort);
      ok = ok && mbar_wait(&hdr.a_empty, (runs - 1) & 1, abort);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0 && !ok) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
      if (rank == 0) {  // copies in flight land first, within the limit
        if (runs > 0) mbar_wait(&hdr.a_full, (runs - 1) & 1, nullptr);
        for (int j = max(0, chunk - kExRing); j < chunk; ++j)
          mbar_wait(&hdr.b_full[j % kExRing], (j / kExRing) & 1, nullptr);
      }
    }
  } else if (rank == 0 && elect_one()) {
    // ------------------------------------------------------------------ MMA
    bool ok = true;
    int i = 0, chunk = 0;
    for (int runs = 0; ok && next(r); ++runs) {
      ok = mbar_wait(&hdr.a_full, runs & 1, abort);
      for (int h = r.h0; ok && h < r.h1; ++h, ++i) {
        if (i >= 2 && !mbar_wait(&hdr.d_empty[i & 1], ((i >> 1) - 1) & 1, abort)) {
          ok = false;
          break;
        }
        const uint32_t d = tmem + (i & 1) * kUp;
        for (int c = 0; c < kExColumns; ++c, ++chunk) {
          const int st = chunk % kExRing;
          if (!mbar_wait(&hdr.b_full[st], (chunk / kExRing) & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t a0 = umma_desc_sw128(smem_addr(as) + c * 1024, 16, kExGroup);
          const uint64_t b0 = umma_desc_sw128(smem_addr(bsm) + st * kExBBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            pair_mma(d, a0 + (kk * 32 >> 4), b0 + (kk * 32 >> 4), IDESC, (c > 0 || kk > 0) ? 1u : 0u);
          pair_commit(&hdr.b_empty[st]);
        }
        if (ok) pair_commit(&hdr.d_full[i & 1]);
      }
      if (ok) pair_commit(&hdr.a_empty);
    }
    if (!ok) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
    }
    pair_commit(&hdr.fin);
  }
  tc_fence_before_sync();
  __syncthreads();
  // every product has completed, and its arrivals in this block with it, whether the block gave up or not
  if (warp == kExMmaWarp) {
    mbar_wait(&hdr.fin, 0, nullptr);
    __syncwarp();
  }
  cluster_sync();  // both blocks are done with the other's shared memory and tensor memory
  if (warp == kExMmaWarp) {
    tc_fence_after_sync();
    pair_dealloc(tmem, 512);
  }
  cluster_sync();
}

// ------------------------------------------------------------------ attend
constexpr int kRows = 128;                      // of a tile (M)
constexpr int kTiles = 2;
constexpr int kKeys = 64;                       // of a stage
constexpr int kHalf = kKeys * 128;              // 64 keys x 128 bytes
constexpr int kKHalves = kQk / 64, kVHalves = kValue / 64;
constexpr int kStageBytes = (kKHalves + kVHalves) * kHalf;
constexpr int kStages = 3;
constexpr int kQHalf = kRows * 128;
constexpr int kQTile = kKHalves * kQHalf;
constexpr int kQOff = 1024, kStageOff = kQOff + kTiles * kQTile;
constexpr int kAttnSmem = kStageOff + kStages * kStageBytes;
constexpr int kAttnThreads = 12 * 32;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kVTmaWarp = 11;
constexpr uint32_t kTileCols = 256;             // TMEM columns of a tile: S 2 x 64, O 128
constexpr float kLazy = 8.f;
// The largest weight of a row is held as 2^kLift or more: fp16's smallest step
// is 2^-24, so that a weight is off by at most 2^-32 of the largest where it
// would be lost below 2^-25, and the total keeps all of it (131071 tokens 17
// nats below one are 0.4 % of it).  2^(kLazy + kLift) is well inside fp16.
constexpr float kLift = 7.f;
constexpr int kFineTokens = 512;

struct AttendParams {
  CUtensorMap tmap_q;     // [T, H, 192], boxes {64, 1, 128}
  CUtensorMap tmap_kv;    // [H * capacity, 256], boxes {64, 64}
  CUtensorMap tmap_rope;  // [capacity, 64], boxes {64, 64}
  void *out;
  const int32_t *cu_q, *lens;
  const long long *prefix;
  const int32_t *powers;
  unsigned num_seqs, heads, ranges, head_group;  // ranges of 256 new tokens; heads that are worked on together
  int num_q_tokens, max_q_len, limit;
  long long capacity;
  float scale_log2;
  int *err;
};

struct AttendHeader {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], s_full[kTiles][2], p_full[kTiles][2], pv_done[kTiles], o_ready[kTiles],
      q_full, fin[kTiles];
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kAttnThreads, 1) latent_attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int AB = DT == kF16 ? 0 : 1;
  constexpr uint32_t IDESC_QK = umma_idesc_f16(AB, kRows, kKeys, false);
  constexpr uint32_t IDESC_PV = umma_idesc_f16(0, kRows, kValue, true);  // P and V are fp16
  extern __shared__ __align__(1024) uint8_t smem[];
  AttendHeader &hdr = *reinterpret_cast<AttendHeader *>(smem);
  // Blocks in this order: groups of heads whose keys and values stay in L2
  // together; in a group the ranges that end last, which follow most tokens,
  // before the others, so that the last blocks to start are short.
  const unsigned group = blockIdx.x / (p.ranges * p.num_seqs * p.head_group);
  const unsigned heads = min(p.head_group, p.heads - group * p.head_group);
  unsigned at = blockIdx.x - group * (p.ranges * p.num_seqs * p.head_group);
  const int h = static_cast<int>(group * p.head_group + at % heads);
  at /= heads;
  const int s = static_cast<int>(at % p.num_seqs), cta = static_cast<int>(p.ranges - 1 - at / p.num_seqs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kTmaWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_kv)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_rope)) : "memory");
  }
  const int q0 = __ldg(p.cu_q + s), n = __ldg(p.cu_q + s + 1) - q0, L = __ldg(p.lens + s);
  const bool valid = n >= 0 && q0 >= 0 && n <= p.num_q_tokens - q0 && n <= p.max_q_len && L >= n && L <= p.limit;
  if (!valid || cta * kTiles * kRows >= n) {
    if (!valid && threadIdx.x == 0) record_error(p.err, kErrSeqLen);
    // a call without any row must not end, and let the next one in the stream begin, before its expansion has
    if (blockIdx.x == 0) grid_dependency_wait();
    return;
  }
  if ((smem_addr(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) record_error(p.err, kErrSmemAlign);
    return;
  }
  const int tok0 = cta * kTiles * kRows;
  const int tiles = tok0 + kRows < n ? 2 : 1;
  const int pos0 = L - n;
  const int kv_end = pos0 + min(n, tok0 + kTiles * kRows);
  const int n_stages = (kv_end + kKeys - 1) / kKeys;
  auto fine_tile = [&](int t) { return DT == kF16 && pos0 + tok0 + t * kRows < kFineTokens; };  // P in two parts
  auto tile_stages = [&](int t) { return (pos0 + min(n, tok0 + (t + 1) * kRows) + kKeys - 1) / kKeys; };
  uint8_t *qs = smem + kQOff, *stages = smem + kStageOff;
  volatile int *abort = &hdr.abort;
  if (warp == kTmaWarp && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&hdr.k_full[i], 1);
      mbar_init(&hdr.k_empty[i], tiles);
      mbar_init(&hdr.v_full[i], 1);
      mbar_init(&hdr.v_empty[i], tiles);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(&hdr.s_full[t][0], 1);
      mbar_init(&hdr.s_full[t][1], 1);
      mbar_init(&hdr.p_full[t][0], kRows);
      mbar_init(&hdr.p_full[t][1], kRows);
      mbar_init(&hdr.pv_done[t], 1);
      mbar_init(&hdr.o_ready[t], 1);
      mbar_init(&hdr.fin[t], 1);
    }
    mbar_init(&hdr.q_full, 1);
    hdr.abort = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(&hdr.q_full, tiles * kQTile);
    for (int t = 0; t < tiles; ++t)
      for (int c = 0; c < kKHalves; ++c)
        tma_load_3d(qs + t * kQTile + c * kQHalf, &p.tmap_q, c * 64, h, q0 + tok0 + t * kRows, &hdr.q_full);
  }
  if (warp == kMmaWarp) tc_alloc(&hdr.tmem, 512);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = hdr.tmem;
  grid_dependency_wait();  // the expansion
  const long long row0 = p.prefix[s] * kExTokens;
  const bool there = row0 + (static_cast<long long>(L) + kExTokens - 1) / kExTokens * kExTokens <= p.capacity;

  if (!there) {
    // more tokens than the caller's bound: nothing was expanded (reported there)
    if (warp == kTmaWarp && lane == 0) mbar_wait(&hdr.q_full, 0, nullptr);
  } else if (warp < 4 * kTiles) {
    if (warp / 4 < tiles) {
      // ------------------------------------------------------------ softmax
      const int t = warp / 4, r = threadIdx.x & 127;
      const int tok = tok0 + t * kRows + r;
      const int pos = pos0 + min(tok, n - 1);
      const uint32_t trow = tmem + t * kTileCols + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
      const float c = p.scale_log2;
      float m = -INFINITY, l = 0.f;  // m: the maximum less kLift
      bool ok = true;
      const int nst = tile_stages(t);
      const bool fine = fine_tile(t);
      // powers of two of the values, 32 keys each; O is in units of 2^unit,
      // the largest power of those the row has followed
      const int2 *powers =
          reinterpret_cast<const int2 *>(p.powers + (static_cast<size_t>(h) * p.capacity + row0) / kExGroup32);
      int2 power = __ldg(powers);
      int unit = pos >= 32 ? max(power.x, power.y) : power.x;
      for (int i = 0; i < nst; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&hdr.s_full[t][i & 1], (i >> 1) & 1, abort))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int k0 = i * kKeys;
        const int2 here = power;
        if (i + 1 < nst) power = __ldg(powers + i + 1);
        float sv[kKeys];
        {
          uint32_t raw[32];
          tc_ld32(trow + (i & 1) * kKeys, raw);
#pragma unroll
          for (int j = 0; j < 32; ++j) sv[j] = __uint_as_float(raw[j]);
          tc_ld32(trow + (i & 1) * kKeys + 32, raw);
#pragma unroll
          for (int j = 0; j < 32; ++j) sv[32 + j] = __uint_as_float(raw[j]);
        }
        // stages wholly at or before every row of the warp need no mask, and
        // with a positive scale the maximum is taken on the raw scores and
        // the scale folded into the exponent's fma
        const bool plain = __all_sync(0xffffffffu, c > 0.f && k0 + kKeys - 1 <= pos);
        float mx, cm;
        if (plain) {
          float a = sv[0], b = sv[32];
#pragma unroll
          for (int j = 1; j < 31; j += 2) {
            a = fmax3(a, sv[j], sv[j + 1]);
            b = fmax3(b, sv[32 + j], sv[33 + j]);
          }
          mx = fmax3(a, b, fmaxf(sv[31], sv[63])) * c;
          cm = c;
        } else {
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < kKeys; j += 2) {
            sv[j] = (k0 + j <= pos) ? sv[j] * c : -INFINITY;
            sv[j + 1] = (k0 + j + 1 <= pos) ? sv[j + 1] * c : -INFINITY;
            mx0 = fmaxf(mx0, sv[j]);
            mx1 = fmaxf(mx1, sv[j + 1]);
          }
          mx = fmaxf(mx0, mx1);
          cm = 1.f;
        }
        const bool grow = mx - m > kLazy + kLift;  // (a difference: exact where the two are close)
        const float next = mx - kLift;
        const int up = max(max(k0 <= pos ? here.x : unit, k0 + 32 <= pos ? here.y : unit) - unit, 0);
        if (__any_sync(0xffffffffu, (grow && i > 0) || up > 0)) {
          // (pv_done is at most one phase behind: S of this stage was issued
          // after the P V before the previous one, and products complete in order)
          if (!__all_sync(0xffffffffu, mbar_wait(&hdr.pv_done[t], (i - 1) & 1, abort))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const float alpha = (grow ? exp2_fast(m - next) : 1.f) * exp2_fast(static_cast<float>(-up));
          unit += up;
#pragma unroll
          for (int d = 0; d < kValue; d += 32) {
            uint32_t ov[32];
            tc_ld32(trow + 2 * kKeys + d, ov);
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
            tc_st32(trow + 2 * kKeys + d, ov);
          }
        }
        if (grow) {
          l *= exp2_fast(m - next);
          m = next;
        }
        const float base = m == -INFINITY ? 0.f : m;
        const uint64_t cm2 = f2(cm, cm), nb2 = f2(-base, -base);
        uint64_t sum0 = f2(0.f, 0.f), sum1 = sum0;
        uint32_t pw[kKeys / 2];
#pragma unroll
        for (int j = 0; j < kKeys; j += 2) {
          float x, y;
          f2_split(ffma2(f2(sv[j], sv[j + 1]), cm2, nb2), x, y);
          const float a = exp2_fast(x), b = exp2_fast(y);
          sv[j] = a;
          sv[j + 1] = b;
          pw[j / 2] = pack2_rn<kF16>(a, b);
          if ((j & 2) == 0)
            sum0 = fadd2(sum0, f2(a, b));
          else
            sum1 = fadd2(sum1, f2(a, b));
        }
        {
          float l0, l1, l2, l3;
          f2_split(sum0, l0, l1);
          f2_split(sum1, l2, l3);
          l += (l0 + l1) + (l2 + l3);
        }
        if ((here.x ^ unit) | (here.y ^ unit)) {  // (rare: values in other powers of two)
          const float f0 = exp2_fast(static_cast<float>(min(here.x - unit, 0)));  // (above: masked keys)
          const float f1 = exp2_fast(static_cast<float>(min(here.y - unit, 0)));
#pragma unroll
          for (int j = 0; j < kKeys; j += 2) {
            sv[j] *= j < 32 ? f0 : f1;
            sv[j + 1] *= j < 32 ? f0 : f1;
            pw[j / 2] = pack2_rn<kF16>(sv[j], sv[j + 1]);
          }
        }
        tc_st32(trow + (i & 1) * kKeys, pw);  // P over the S buffer just read
        if (fine) {  // and what its rounding left, to rows that follow few tokens
#pragma unroll
          for (int j = 0; j < kKeys; j += 2) {
            const float2 a = half2_bits_to_float2<kF16>(pw[j / 2]);
            pw[j / 2] = pos < kFineTokens ? pack2_rn<kF16>(sv[j] - a.x, sv[j + 1] - a.y) : 0u;
          }
          tc_st32(trow + (i & 1) * kKeys + kKeys / 2, pw);
        }
        tc_fence_before_sync();
        mbar_arrive(&hdr.p_full[t][i & 1]);
      }
      if (ok && __all_sync(0xffffffffu, mbar_wait(&hdr.o_ready[t], 0, abort))) {
        tc_fence_after_sync();
        // O / l through this tile's q buffer, whose products have all
        // completed, so that whole rows leave
        // (two factors: 2^unit / l may leave a float's range)
        const float inv = l == 0.f ? 0.f : 1.f / l, power_of_two = exp2f(static_cast<float>(unit));
        constexpr int RB = kValue * 2, CPR = RB / 16;
        uint8_t *stg = qs + t * kQTile;
#pragma unroll
        for (int d = 0; d < kValue; d += 32) {
          uint32_t ov[32];
          tc_ld32(trow + 2 * kKeys + d, ov);
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = l == 0.f ? 0u : pack2_rn<DT>(__uint_as_float(ov[j + 2 * e]) * inv * power_of_two,
                                                  __uint_as_float(ov[j + 2 * e + 1]) * inv * power_of_two);
            *reinterpret_cast<uint4 *>(stg + r * RB + ((((d + j) / 8) ^ (r & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
        // a warp's own 32 rows
        const int first = tok0 + t * kRows + 32 * (warp & 3);
        const int rows = min(32, n - first);
        uint8_t *obase = static_cast<uint8_t *>(p.out) + (static_cast<size_t>(q0 + first) * p.heads + h) * RB;
        const size_t stride = static_cast<size_t>(p.heads) * RB;
        const uint8_t *wst = stg + 32 * (warp & 3) * RB;
#pragma unroll 4
        for (int idx = lane; idx < rows * CPR; idx += 32) {
          const int rr = idx / CPR, ch = idx % CPR;
          *reinterpret_cast<uint4 *>(obase + rr * stride + ch * 16) =
              *reinterpret_cast<const uint4 *>(wst + rr * RB + ((ch ^ (rr & 7)) << 4));
        }
      } else {
        record_error(p.err, kErrTimeout);
        *abort = 1;
      }
    }
  } else if (warp == kTmaWarp || warp == kVTmaWarp) {
    // ---------------------------------------------------------------- TMA
    // keys by one warp, values by the other: a stage's keys are done with
    // before its softmax, its values long after
    if (lane == 0) {
      const bool is_k = warp == kTmaWarp;
      uint64_t *full = is_k ? hdr.k_full : hdr.v_full, *empty = is_k ? hdr.k_empty : hdr.v_empty;
      bool ok = true;
      int issued = 0;
      const int kvrow = static_cast<int>(h * p.capacity + row0), rrow = static_cast<int>(row0);
      for (int i = 0; i < n_stages; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !mbar_wait(&empty[st], (i / kStages - 1) & 1, abort)) {
          ok = false;
          break;
        }
        uint8_t *to = stages + st * kStageBytes;
        if (is_k) {
          mbar_arrive_expect_tx(&full[st], kKHalves * kHalf);
#pragma unroll
          for (int c = 0; c < kNope / 64; ++c)
            tma_load_2d(to + c * kHalf, &p.tmap_kv, c * 64, kvrow + i * kKeys, &full[st]);
          tma_load_2d(to + (kNope / 64) * kHalf, &p.tmap_rope, 0, rrow + i * kKeys, &full[st]);
        } else {
          mbar_arrive_expect_tx(&full[st], kVHalves * kHalf);
#pragma unroll
          for (int c = 0; c < kVHalves; ++c)
            tma_load_2d(to + (kKHalves + c) * kHalf, &p.tmap_kv, kNope + c * 64, kvrow + i * kKeys, &full[st]);
        }
        issued = i + 1;
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        *abort = 1;
        for (int j = max(0, issued - kStages); j < issued; ++j)
          mbar_wait(&full[j % kStages], (j / kStages) & 1, nullptr);
      }
      if (is_k) mbar_wait(&hdr.q_full, 0, nullptr);
    }
  } else {
    // ---------------------------------------------------------------- MMA
    const int t = warp - kMmaWarp;
    if (t < tiles && elect_one()) {
      bool ok = mbar_wait(&hdr.q_full, 0, abort);
      const uint32_t qt = smem_addr(qs) + t * kQTile, sa = smem_addr(stages), tt = tmem + t * kTileCols;
      auto issue_qk = [&](int i) -> bool {
        const int st = i % kStages;
        if (!mbar_wait(&hdr.k_full[st], (i / kStages) & 1, abort)) return false;
        tc_fence_after_sync();
        const uint64_t a0 = umma_desc_sw128(qt, 16, 1024), b0 = umma_desc_sw128(sa + st * kStageBytes, 16, 1024);
        const uint32_t d = tt + (i & 1) * kKeys;
#pragma unroll
        for (int kk = 0; kk < kQk / 16; ++kk) {
          const uint32_t off = (kk % 4) * 32;
          tc_mma_f16(d, a0 + (((kk / 4) * kQHalf + off) >> 4), b0 + (((kk / 4) * kHalf + off) >> 4), IDESC_QK, kk > 0);
        }
        tc_commit(&hdr.s_full[t][i & 1]);
        tc_commit(&hdr.k_empty[st]);
        return true;
      };
      const int nst = tile_stages(t);
      const bool fine = fine_tile(t);
      if (ok) ok = issue_qk(0);
      for (int i = 0; i < nst && ok; ++i) {
        if (i + 1 < nst && !issue_qk(i + 1)) {
          ok = false;
          break;
        }
        if (!mbar_wait(&hdr.v_full[i % kStages], (i / kStages) & 1, abort) ||
            !mbar_wait(&hdr.p_full[t][i & 1], (i >> 1) & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t b0 = umma_desc_sw128(sa + (i % kStages) * kStageBytes + kKHalves * kHalf, kHalf, 1024);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc_mma_f16_ta(tt + 2 * kKeys, tt + (i & 1) * kKeys + kk * 8, b0 + kk * (2 * 1024 >> 4), IDESC_PV,
                        (i > 0 || kk > 0) ? 1u : 0u);
        if (fine)
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc_mma_f16_ta(tt + 2 * kKeys, tt + (i & 1) * kKeys + kKeys / 2 + kk * 8, b0 + kk * (2 * 1024 >> 4), IDESC_PV, 1u);
        tc_commit(&hdr.pv_done[t]);
        if (i + 1 == nst) tc_commit(&hdr.o_ready[t]);
        tc_commit(&hdr.v_empty[i % kStages]);
      }
      // stages behind this tile's rows: released once filled
      for (int i = nst; i < n_stages && ok; ++i) {
        if (!mbar_wait(&hdr.k_full[i % kStages], (i / kStages) & 1, abort) ||
            !mbar_wait(&hdr.v_full[i % kStages], (i / kStages) & 1, abort)) {
          ok = false;
          break;
        }
        tc_commit(&hdr.k_empty[i % kStages]);
        tc_commit(&hdr.v_empty[i % kStages]);
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        *abort = 1;
      }
      tc_commit(&hdr.fin[t]);
      mbar_wait(&hdr.fin[t], 0, nullptr);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tc_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host
struct Sizes {
  size_t prefix, powers, rope, kv, total;
  long long capacity;
};
bool sizes_of(int S, int H, long long tokens, Sizes *z) {
  if (S < 0 || H <= 0 || tokens < 0 || tokens > INT_MAX / 4) return false;
  // sequences padded to a tile of tokens
  const long long tiles = (tokens + static_cast<long long>(S) * (kExTokens - 1)) / kExTokens + 1;
  z->capacity = tiles * kExTokens;
  if (z->capacity * H > INT_MAX) return false;  // 32-bit rows
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  z->prefix = up(8 * (static_cast<size_t>(S) + 1));
  z->powers = up(static_cast<size_t>(z->capacity / kExGroup32) * H * sizeof(int32_t));
  z->rope = up(static_cast<size_t>(z->capacity) * kRopeDim * 2);
  z->kv = up(static_cast<size_t>(z->capacity) * H * kUp * 2);
  z->total = z->prefix + z->powers + z->rope + z->kv;
  return true;
}

bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT>
pa_status launch(const ExpandParams &ep, const AttendParams &ap, cudaStream_t stream) {
  static bool configured[64];  // per device: dynamic shared memory already allowed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(latent_expand_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kExSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(latent_attend_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  DeviceInfo info;
  if (!current_device_info(&info)) return cuda_fail(cudaGetLastError());
  latent_expand_kernel<DT><<<info.sm_count / 2 * 2, kExThreads, kExSmem, stream>>>(ep);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ap.ranges * ap.num_seqs * ap.heads);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = kAttnSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_attend_kernel<DT>, ap);
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_latent_prefill_workspace_size(int32_t num_seqs, int32_t num_heads, int64_t num_kv_tokens) {
  Sizes z;
  return sizes_of(num_seqs, num_heads, num_kv_tokens, &z) ? z.total : 0;
}

extern "C" pa_status pa_latent_prefill(void *out, const void *q, int32_t q_dtype, int32_t num_q_tokens,
                                       const int32_t *cu_q_lens, int32_t num_seqs, int32_t num_heads,
                                       int32_t max_q_len, const void *up, const void *cache,
                                       const pa_latent_desc *desc, const int32_t *block_tables,
                                       int32_t max_blocks_per_seq, const int32_t *seq_lens, int64_t num_kv_tokens,
                                       float scale, void *workspace, size_t workspace_bytes, int *device_error,
                                       pa_stream_t stream) {
  if (!valid_latent_desc(desc) || num_seqs < 0 || num_heads <= 0 || max_q_len < 0 || num_q_tokens < 0 ||
      num_kv_tokens < 0 || max_blocks_per_seq <= 0 || !isfinite(scale))
    return PA_ERR_INVALID;
  if (num_seqs == 0 || max_q_len == 0 || num_q_tokens == 0) return PA_OK;
  if (!out || !q || !cu_q_lens || !up || !cache || !block_tables || !seq_lens || !workspace) return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(up) || !aligned16(cache) ||
      ((reinterpret_cast<uintptr_t>(cu_q_lens) | reinterpret_cast<uintptr_t>(block_tables) |
        reinterpret_cast<uintptr_t>(seq_lens)) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_INVALID;
  if (!supported_latent_desc(desc) || q_dtype != desc->dtype) return PA_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_heads > 65535) return PA_ERR_UNSUPPORTED;
  Sizes z;
  if (!sizes_of(num_seqs, num_heads, num_kv_tokens, &z)) return PA_ERR_UNSUPPORTED;
  if (workspace_bytes < z.total) return PA_ERR_INVALID;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const long long held = static_cast<long long>(max_blocks_per_seq) * desc->block_size;
  ExpandParams ep{};
  ep.cache = static_cast<const uint8_t *>(cache);
  ep.tables = block_tables;
  ep.lens = seq_lens;
  ep.prefix = reinterpret_cast<long long *>(ws);
  ep.powers = reinterpret_cast<int32_t *>(ws + z.prefix);
  ep.rope = ws + z.prefix + z.powers;
  ep.kv = ws + z.prefix + z.powers + z.rope;
  ep.num_seqs = num_seqs;
  ep.heads = num_heads;
  ep.num_blocks = desc->num_blocks;
  ep.bs_shift = log2_block(desc->block_size);
  ep.max_blocks = max_blocks_per_seq;
  ep.limit = static_cast<int>(held < INT_MAX / 4 ? held : INT_MAX / 4);
  ep.capacity = z.capacity;
  ep.err = device_error;
  AttendParams ap{};
  ap.out = out;
  ap.cu_q = cu_q_lens;
  ap.lens = seq_lens;
  ap.prefix = ep.prefix;
  ap.powers = ep.powers;
  ap.num_seqs = num_seqs;
  ap.heads = num_heads;
  const long long ranges = (static_cast<long long>(max_q_len) + kTiles * kRows - 1) / (kTiles * kRows);
  if (ranges * num_seqs * num_heads > INT_MAX / 2) return PA_ERR_UNSUPPORTED;  // the grid
  ap.ranges = static_cast<unsigned>(ranges);
  // keys and values of a group of heads: up to half of L2
  const long long in_l2 = (64ll << 20) / (z.capacity * kUp * 2);
  ap.head_group = static_cast<unsigned>(in_l2 < 1 ? 1 : in_l2 > num_heads ? num_heads : in_l2);
  ap.num_q_tokens = num_q_tokens;
  ap.max_q_len = max_q_len;
  ap.limit = ep.limit;
  ap.capacity = z.capacity;
  ap.scale_log2 = scale * 1.4426950408889634f;
  ap.err = device_error;
  const cuuint64_t H = num_heads, cap = z.capacity;
  const cuuint64_t du[2] = {kLatentDim, H * kUp}, su[1] = {kLatentDim * 2};
  const cuuint32_t bu[2] = {64, kExBRows};
  const cuuint64_t dq[3] = {kQk, H, static_cast<cuuint64_t>(num_q_tokens)}, sq[2] = {kQk * 2, H * kQk * 2};
  const cuuint32_t bq[3] = {64, 1, kRows};
  const cuuint64_t dk[2] = {kUp, H * cap}, sk[1] = {kUp * 2};
  const cuuint64_t dr[2] = {kRopeDim, cap}, sr[1] = {kRopeDim * 2};
  const cuuint32_t bk[2] = {64, kKeys};
  if (!encode_latent_view(&ep.tmap_c, cache, desc, kExColumns, desc->block_size / 8) ||
      !encode(&ep.tmap_u, up, 2, du, su, bu) || !encode(&ap.tmap_q, q, 3, dq, sq, bq) ||
      !encode(&ap.tmap_kv, ep.kv, 2, dk, sk, bk) || !encode(&ap.tmap_rope, ep.rope, 2, dr, sr, bk))
    return cuda_fail(cudaErrorInvalidValue);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return desc->dtype == PA_F16 ? launch<kF16>(ep, ap, st)
                               : launch<kBF16>(ep, ap, st);
}
