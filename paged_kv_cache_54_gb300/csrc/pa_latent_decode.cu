// pa_latent_decode: absorbed attention of one or a few new tokens a sequence
// over the latent paged cache.
//
// All heads share the token's 576-element row: a (token, head) row r of
// queries gives
//   x[r, i] = scale <q_r, row_i>,   out[r] = sum_i softmax_i(x[r, i]) row_i[:512],
// so a sequence's n * H query rows read its cache once.  Per token of the
// cache that is 1152 bytes and 2176 operations a row.
//
// The products run on the 5th-generation tensor cores with the tokens and the
// latent dimensions as rows and the query rows as columns, so that the tile's
// cost follows the number of query rows:
//   S^T = K Q^T    M = 64 tokens, N = 16, 32 or 64 query rows, K = 576
//   O^T += V^T P^T M = 128 dimensions, N query rows, K = 64 tokens
// K and V are one tile of shared memory, rows of nine 128-byte columns in
// groups of 8 rows of 8-row x 128-byte swizzled atoms.  The first product
// reads it token-major, the second dimension-major.  O^T takes 4 N columns of
// tensor memory, S^T 2 N.
//
// A block takes all query rows and an equal share of all sequences'
// 64-token tiles (pa_shares.cuh).  One sequence of 131071 tokens, 32 query
// rows: 151 MB, 22.6 us at the measured copy rate; this kernel takes 35 (the
// loop keeps up with the memory, 5 us pass until the first tiles land, 3 to 5
// from the last one to the stored sums), the join of 152 pieces a row 6 (10
// when it looked the pieces up after its wait, and read their maxima first).
// Warps:
//   0..7  softmax: a thread owns a token and a quarter of the query rows.  The
//         maximum of a query row is kept for all threads in shared memory and
//         raised only when a score passes it by 2^8 (the largest weight is then
//         1 to 2^8, times 2^7 with fp16 operands), so that almost every
//         tile needs one vote of the block instead of a reduction over
//         tokens; the total weights stay per thread until a sequence ends.
//   8     TMA: q, then the tiles, a 16-token slot at a time
//   9, 10 issue the S^T and O^T products
#include <float.h>
#include <limits.h>
#include <math.h>

#include "pa_latent_decode.cuh"

namespace pa {
namespace {

constexpr int kTile = 64;              // tokens of a tile
constexpr int kSlots = 4;              // 16-token slots of a tile, freed one by one
constexpr int kStages = 2;
constexpr int kCols = kLatentRow / 64; // 128-byte columns of a row
constexpr int kAtom = 1024;
constexpr int kGroup = kCols * kAtom;  // 8 rows
constexpr int kTileBytes = kTile / 8 * kGroup;
constexpr int kDims = 128;             // of one O^T product
constexpr int kBlocksO = kLatentDim / kDims;
constexpr int kTmaWarp = 8, kQkWarp = 9;  // and 10: O^T
constexpr int kThreads = 11 * 32;
constexpr int kMaxWorkers = 152;       // shares, at most; sizes the workspace

template <int N>
struct Layout {
  static constexpr int Q_COL = N * 128;  // a 128-byte column of the query rows
  static constexpr int Q_OFF = 2048;
  static constexpr int Q_BYTES = kCols * Q_COL;
  static constexpr int P_OFF = Q_OFF + Q_BYTES;
  static constexpr int P_BYTES = kTile * 128;
  static constexpr int KV_OFF = P_OFF + P_BYTES;
  static constexpr int SMEM = KV_OFF + kStages * kTileBytes;
  static constexpr uint32_t TMEM_S = kBlocksO * N;  // columns: O^T, then two S^T
  static constexpr uint32_t TMEM_COLS = 8 * N;
  static_assert(SMEM <= 232448 && KV_OFF % 1024 == 0, "shared memory");
};

struct Header {
  uint64_t kv_full[kStages], kv_empty[kStages][kSlots];
  uint64_t s_full[2], s_empty[2], p_full, pv_done, q_full, q_empty, fin[2];
  uint32_t tmem;
  int abort;
  alignas(16) float m[64];  // what the query rows' scores are raised by: kLift minus their maxima (base 2)
  float top[4][64];         // maxima of 16 tokens, then their total weights
  int see[64];              // tokens a query row sees
};
static_assert(sizeof(Header) <= 2048, "the header's place");
// Of a row without a maximum yet, the largest float: with it any score passes
// the threshold (but its own negative, which counts as none), and none (-inf)
// stays -inf.
constexpr float kNone = FLT_MAX;

// NCOL consecutive columns of the warp's lanes
#define PA_R8(a, o) a(r[o]), a(r[o + 1]), a(r[o + 2]), a(r[o + 3]), a(r[o + 4]), a(r[o + 5]), a(r[o + 6]), a(r[o + 7])
template <int NCOL>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[NCOL]) {
  uint32_t r[NCOL];
  if constexpr (NCOL == 32) {
    tc_ld32(taddr, r);
  } else if constexpr (NCOL == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : PA_R8("=r", 0), PA_R8("=r", 8)
        : "r"(taddr)
        : "memory");
  } else {
    static_assert(NCOL == 8, "8, 16 or 32 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PA_R8("=r", 0)
        : "r"(taddr)
        : "memory");
  }
#pragma unroll
  for (int j = 0; j < NCOL; ++j) v[j] = __uint_as_float(r[j]);
}
template <int NCOL>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const float (&v)[NCOL]) {
  uint32_t r[NCOL];
#pragma unroll
  for (int j = 0; j < NCOL; ++j) r[j] = __float_as_uint(v[j]);
  if constexpr (NCOL == 32) {
    tc_st32(taddr, r);
  } else if constexpr (NCOL == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        PA_R8("r", 0), PA_R8("r", 8)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        PA_R8("r", 0)
        : "memory");
  }
}
#undef PA_R8

// Half the warp's lanes are rows (M = 64): lanes 0..15 get NCOL columns from
// taddr, lanes 16..31 the NCOL columns behind them, of the same 16 rows.
#define PA_R4(a, o) a(r[o]), a(r[o + 1]), a(r[o + 2]), a(r[o + 3])
template <int NCOL>
__device__ __forceinline__ void tmem_load_rows16(uint32_t taddr, float (&v)[NCOL]) {
  uint32_t r[NCOL];
  if constexpr (NCOL == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16], 16;\n\ttcgen05.wait::ld.sync.aligned;"
        : PA_R4("=r", 0), PA_R4("=r", 4), PA_R4("=r", 8), PA_R4("=r", 12)
        : "r"(taddr)
        : "memory");
  } else if constexpr (NCOL == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 8;\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PA_R4("=r", 0), PA_R4("=r", 4)
        : "r"(taddr)
        : "memory");
  } else {
    static_assert(NCOL == 4, "4, 8 or 16 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%0, %1, %2, %3}, [%4], 4;\n\ttcgen05.wait::ld.sync.aligned;"
        : PA_R4("=r", 0)
        : "r"(taddr)
        : "memory");
  }
#pragma unroll
  for (int j = 0; j < NCOL; ++j) v[j] = __uint_as_float(r[j]);
}
#undef PA_R4

template <int DT, int N>
__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ LatentParams p, int max_workers) {
  using Lay = Layout<N>;
  constexpr int NQ = N / 4;  // query rows of a softmax thread
  constexpr int NC = N / 2;  // of an O^T thread
  constexpr int AB = DT == kF16 ? 0 : 1;
  constexpr uint32_t IDESC_QK = umma_idesc_f16(AB, kTile, N, false);
  constexpr uint32_t IDESC_PV = umma_idesc_f16(AB, kDims, N, true) | (1u << 15);  // (A dimension-major too)
  extern __shared__ __align__(1024) uint8_t smem[];
  // (the scan is over before the weights' buffer is first written)
  ShareScan<128> &scan = *reinterpret_cast<ShareScan<128> *>(smem + Lay::P_OFF);
  static_assert(sizeof(ShareScan<128>) <= Lay::P_BYTES, "the scan's place");
  Header &hdr = *reinterpret_cast<Header *>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = blockIdx.x;
  if (!p.whole) launch_dependents();  // (the merge)
  const int n_rows = p.rows;  // (at most N)
  auto tiles_of = [&](int s) -> long long { return (checked_len(p.lens, s, p.limit, p.err) + kTile - 1) / kTile; };
  Walk<kTile> walk;
  if (p.whole) {
    walk.u = walk.first = 0;
    walk.s = w;
    walk.end = tiles_of(w);
    if (walk.end == 0) {
      zero_rows(p.out, static_cast<long long>(w) * p.rows, n_rows);
      return;
    }
  } else {
    scan.scan(p.num_seqs, tiles_of);
    if (blockIdx.x == 0 && threadIdx.x < 128) {  // the sequences' first tiles, for the merge
      const int n = scan.run(p.num_seqs), t = threadIdx.x;
      long long at = scan.base[t];
      for (int s = t * n; s < min(p.num_seqs, (t + 1) * n); ++s) {
        p.prefix[s] = at;
        at += tiles_of(s);
      }
      if (t == 0) p.prefix[p.num_seqs] = scan.total();
    }
    const long long total = scan.total(), workers = worker_count(total, max_workers);
    if (w >= workers) return;
    walk.u = share_begin(w, total, workers);
    walk.end = share_begin(w + 1, total, workers);
    walk.s = scan.find(walk.u, p.num_seqs, tiles_of, walk.first);
  }
  if ((smem_addr(smem) & 1023u) != 0) {  // the swizzle needs 1024-byte atoms
    if (threadIdx.x == 0) record_error(p.err, kErrSmemAlign);
    return;
  }
  volatile int *abort = &hdr.abort;
  uint8_t *qs = smem + Lay::Q_OFF, *ps = smem + Lay::P_OFF, *kv = smem + Lay::KV_OFF;
  if (warp == kTmaWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_c)) : "memory");
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&hdr.kv_full[i], 1);
      for (int j = 0; j < kSlots; ++j) mbar_init(&hdr.kv_empty[i][j], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hdr.s_full[i], 1);
      mbar_init(&hdr.s_empty[i], kSoftmaxThreads / 32);
      mbar_init(&hdr.fin[i], 1);
    }
    mbar_init(&hdr.p_full, kSoftmaxThreads / 32);
    mbar_init(&hdr.pv_done, 1);
    mbar_init(&hdr.q_full, 1);
    mbar_init(&hdr.q_empty, 1);
    hdr.abort = 0;
    fence_mbar_init();
  }
  if (warp == kQkWarp) tc_alloc(&hdr.tmem, Lay::TMEM_COLS);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = hdr.tmem;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int quarter = warp & 3;
    const int k = 16 * quarter + (lane & 15);               // the thread's token
    const int c0 = (warp >> 2) * NC + (lane >> 4) * NQ;     // and its first query row
    const int o0 = (warp >> 2) * NC;                        // of O^T: its first query row
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + o0;
    const float c = p.scale_log2;
    // a wait that gave up leaves the warp in step with the others, whose
    // barriers count on it: it goes on without waiting, and nothing is stored
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
      tc_fence_after_sync();
    };
    auto top_of = [&](int h) {
      return fmaxf(fmaxf(hdr.top[0][h], hdr.top[1][h]), fmaxf(hdr.top[2][h], hdr.top[3][h]));
    };
    auto sum_of = [&](int h) { return (hdr.top[0][h] + hdr.top[1][h]) + (hdr.top[2][h] + hdr.top[3][h]); };
    // whether a row's maximum is raised, given what its scores were raised by, and the factor of its sums (differences,
    // which are exact where the numbers are close)
    constexpr float OVER = kLazy + kLift<DT>;
    auto raised = [&](float was, float top) { return was == kNone ? top > -INFINITY : top + was > OVER; };
    auto factor = [&](float was, float top) {
      return !raised(was, top) ? 1.f : was == kNone ? 0.f : exp2_fast((kLift<DT> - top) - was);
    };
    const float4 *m4 = reinterpret_cast<const float4 *>(hdr.m + c0);
    int i = 0;  // tiles so far
    for (int seg = 0; walk.next(p); ++seg) {
      float l[NQ];
#pragma unroll
      for (int j = 0; j < NQ; ++j) l[j] = 0.f;
      softmax_sync();  // the last piece's maxima and totals have been read
      if (threadIdx.x < N) {
        const int h = threadIdx.x;
        hdr.m[h] = kNone;
        hdr.see[h] = h < n_rows ? walk.L - (p.new_tokens - 1 - h / p.heads) : 0;
      }
      softmax_sync();
      // tokens that every query row sees
      const int all_see = n_rows < N ? 0 : walk.L - (p.new_tokens - 1);
      const int plain = plain_end(p, walk.L);
      bool bad = false;  // whether this thread has taken numbers out of V
      for (int tile = walk.t0; tile < walk.t1; ++tile, ++i) {
        wait(&hdr.s_full[i & 1], (i >> 1) & 1);
        float x[NQ];
        tmem_load_rows16<NQ>(tlane + Lay::TMEM_S + (i & 1) * N, x);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&hdr.s_empty[i & 1]);
        const int key = tile * kTile + k;
        if ((tile + 1) * kTile > all_see) {
#pragma unroll
          for (int j = 0; j < NQ; ++j) x[j] = key < hdr.see[c0 + j] ? x[j] * c : -INFINITY;
        } else {
#pragma unroll
          for (int j = 0; j < NQ; ++j) x[j] *= c;
        }
        float y[NQ], over = -INFINITY;
#pragma unroll
        for (int j = 0; j < NQ; j += 4) {
          const float4 m = m4[j / 4];
          y[j] = x[j] + m.x;
          y[j + 1] = x[j + 1] + m.y;
          y[j + 2] = x[j + 2] + m.z;
          y[j + 3] = x[j + 3] + m.w;
          over = fmaxf(over, fmaxf(fmaxf(y[j], y[j + 1]), fmaxf(y[j + 2], y[j + 3])));
        }
        if (softmax_any(over > OVER)) {
          // raise the maxima: over each warp's 16 tokens, then all four
#pragma unroll
          for (int j = 0; j < NQ; ++j) {
            float top = x[j];  // (the maximum of numbers: a NaN is passed over)
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if ((lane & 15) == 0) hdr.top[quarter][c0 + j] = top;
          }
          softmax_sync();
#pragma unroll
          for (int j = 0; j < NQ; ++j) l[j] *= factor(hdr.m[c0 + j], top_of(c0 + j));
          if (tile > walk.t0) {  // O^T holds the tiles before
            wait(&hdr.pv_done, (i - 1) & 1);
#pragma unroll 1
            for (int b = 0; b < kBlocksO; ++b) {
              float o[NC];
              tmem_load<NC>(tlane + b * N, o);
#pragma unroll
              for (int j = 0; j < NC; ++j) o[j] *= factor(hdr.m[o0 + j], top_of(o0 + j));
              tmem_store<NC>(tlane + b * N, o);
            }
          }
          softmax_sync();
          if (threadIdx.x < N) {
            const float top = top_of(threadIdx.x);
            if (raised(hdr.m[threadIdx.x], top)) hdr.m[threadIdx.x] = kLift<DT> - top;
          }
          softmax_sync();
#pragma unroll
          for (int j = 0; j < NQ; ++j) y[j] = x[j] + hdr.m[c0 + j];
        }
        // weights, rounded to the operand type (half a step each; see kLift)
        uint32_t pw[NQ / 2];
#pragma unroll
        for (int j = 0; j < NQ; j += 2) {
          const float a = exp2_fast(y[j]), b = exp2_fast(y[j + 1]);
          l[j] += a;
          l[j + 1] += b;
          pw[j / 2] = pack2_rn<DT>(a, b);
        }
        // the P buffer is free once the last tile's O^T products have completed
        if (i > 0) wait(&hdr.pv_done, (i - 1) & 1);
        uint8_t *row = ps + k * 128;
        if constexpr (NQ >= 8) {
#pragma unroll
          for (int u = 0; u < NQ / 8; ++u)
            *reinterpret_cast<uint4 *>(row + (((c0 / 8 + u) ^ (k & 7)) << 4)) =
                make_uint4(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]);
        } else {
          *reinterpret_cast<uint2 *>(row + ((c0 / 8 ^ (k & 7)) << 4) + (c0 & 7) * 2) = make_uint2(pw[0], pw[1]);
        }
        if ((tile + 1) * kTile > plain) {
          // rows behind the sequence's end hold anything: zero them, 0 * NaN would reach O^T; of drafted tokens
          // before it what is not finite is taken out
          uint8_t *vb = kv + (i & 1) * kTileBytes;
          const int z0 = max(plain - tile * kTile, 0), z1 = walk.L - tile * kTile;
          for (int idx = threadIdx.x; idx < (kTile - z0) * (kLatentDim / 8); idx += kSoftmaxThreads) {
            const int z = z0 + idx / (kLatentDim / 8), e = idx % (kLatentDim / 8);
            uint4 *at = reinterpret_cast<uint4 *>(vb + (z >> 3) * kGroup + (e >> 3) * kAtom + (z & 7) * 128 + (e & 7) * 16);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            bool write = true;
            if (z < z1) {
              x = *at;
              write = take_out<DT>(x);
              bad |= write;
            }
            if (write) *at = x;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&hdr.p_full);
      }
      // the piece's sums: total weights over the tokens, then O^T as rows
#pragma unroll
      for (int st = 0; st < 4; ++st) {  // halve the query rows a lane keeps, while there are several
        const int o = 8 >> st, half = NQ >> (st + 1);
        const bool upper = (lane & o) != 0;
        if (half == 0) {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        } else {
#pragma unroll
          for (int j = 0; j < NQ / 2; ++j)
            if (j < half) {
              const float send = upper ? l[j] : l[j + half], keep = upper ? l[j + half] : l[j];
              l[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
      }
      softmax_sync();
      // (lanes 16 / NQ apart hold the same row where there are fewer rows than lanes)
      hdr.top[quarter][c0 + (lane & 15) / (16 / NQ)] = l[0];
      softmax_sync();
      wait(&hdr.pv_done, (i - 1) & 1);
      const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
      const int d0 = 32 * quarter;  // the thread's dimensions: d0 + lane (+ 128 b)
      // drafted tokens of this piece from which numbers were taken: not-a-number to the rows that see them
      const bool patch = p.new_tokens > 1 && walk.t1 * kTile > plain && softmax_any(bad);
      auto load_o = [&](int b, float (&o)[NC]) {
        tmem_load<NC>(tlane + b * N, o);
        if (patch) {
          int from = max(plain, walk.t0 * kTile);  // the first such token, in this dimension
          const int end = min(walk.L, walk.t1 * kTile);
          while (from < end &&
                 (__ldg(token_row(p, walk.s, from) + d0 + lane + b * kDims) & kNotFinite<DT>) != kNotFinite<DT>)
            ++from;
          if (from < end)
#pragma unroll
            for (int j = 0; j < NC; ++j)
              if (hdr.see[o0 + j] > from) o[j] = __int_as_float(0x7fffffff);
          __syncwarp();
        }
      };
      if (!ok) {
      } else if (whole) {
        // rows of out: neighbouring lanes swap, so that each stores two
        // dimensions of every other query row
        const size_t row0 = static_cast<size_t>(walk.s) * p.rows + o0;
        const bool odd = lane & 1;
        uint16_t *o16 = static_cast<uint16_t *>(p.out) + (row0 + odd) * kLatentDim + d0 + (lane & ~1);
#pragma unroll 1
        for (int b = 0; b < kBlocksO; ++b) {
          float o[NC];
          load_o(b, o);
#pragma unroll
          for (int j = 0; j < NC; j += 2) {
            const float s0 = sum_of(o0 + j), s1 = sum_of(o0 + j + 1);
            const float y0 = s0 == 0.f ? 0.f : __fdividef(o[j], s0);  // (a row that sees nothing)
            const float y1 = s1 == 0.f ? 0.f : __fdividef(o[j + 1], s1);
            const float got = __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
            if (o0 + j + odd < n_rows)
              *reinterpret_cast<uint32_t *>(o16 + static_cast<size_t>(j) * kLatentDim + b * kDims) =
                  odd ? pack2_rn<DT>(got, y1) : pack2_rn<DT>(y0, got);
          }
        }
      } else {
        const size_t slot = static_cast<size_t>(w) * 2 + (seg > 0);
        if (threadIdx.x < N) {
          const float m = hdr.m[threadIdx.x];
          p.part_ml[slot * N + threadIdx.x] = make_float2(m == kNone ? -INFINITY : -m, sum_of(threadIdx.x));
        }
        float *po = p.part_o + (slot * N + o0) * kLatentDim + d0 + lane;
#pragma unroll 1
        for (int b = 0; b < kBlocksO; ++b) {
          float o[NC];
          load_o(b, o);
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (o0 + j < n_rows) po[static_cast<size_t>(j) * kLatentDim + b * kDims] = o[j];
        }
      }
      tc_fence_before_sync();
      walk.advance();
    }
    if (!ok) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
    }
  } else if (warp == kTmaWarp) {
    // -------------------------------------------------------------------- TMA
    // a tile is four boxes of 16 tokens (eight of 8 with blocks of 8): lane j
    // copies box j once its slot is free
    const int box_sh = p.bs_shift < 4 ? 3 : 4, boxes = kTile >> box_sh;
    const uint32_t box_bytes = (1u << box_sh) / 8 * kGroup;
    bool ok = true;
    int i = 0, tiles_issued = 0, qs_issued = 0;  // (the last tile perhaps in part)
    for (int seg = 0; ok && walk.next(p); ++seg) {
      const int32_t *table = p.tables + static_cast<size_t>(walk.s) * p.max_blocks;
      auto entry = [&](int tile) {  // this lane's block of a tile
        const int tok = tile * kTile + (lane << box_sh);
        return lane < boxes && tok < walk.L ? __ldg(table + (tok >> p.bs_shift)) : 0;
      };
      // A tile is fetched into L2 two tiles ahead of its copy: the copy then
      // takes about 1500 clocks in place of 2500 to 4000, and two tiles in
      // shared memory keep up.
      auto row_of = [&](int block, int tile) {
        const int tok = tile * kTile + (lane << box_sh);
        return (block << p.bs_shift) + (tok & ((1 << p.bs_shift) - 1));
      };
      auto fetch = [&](int block, int tile) {
        if (tile < walk.t1 && lane < boxes && tile * kTile + (lane << box_sh) < walk.L && block >= 0 &&
            block < p.num_blocks)
          tma_prefetch_4d(&p.tmap_c, 0, 0, 0, row_of(block, tile) >> 3);
      };
      int phys = entry(walk.t0), phys1 = entry(walk.t0 + 1), phys2 = entry(walk.t0 + 2);
      bool free = true;
      if (lane == 0 && seg > 0) free = mbar_wait(&hdr.q_empty, (seg - 1) & 1, abort);
      if (!__shfl_sync(0xffffffffu, free, 0)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&hdr.q_full, Lay::Q_BYTES);
        const int row = walk.s * p.rows;
        for (int e = 0; e < kCols; ++e)
          tma_load_2d(qs + e * Lay::Q_COL, &p.tmap_q, e * 64, row, &hdr.q_full);
      }
      ++qs_issued;
      for (int tile = walk.t0; tile < walk.t1; ++tile, ++i) {
        const int st = i & 1;
        const int n_box = min(boxes, ((walk.L - tile * kTile) + (1 << box_sh) - 1) >> box_sh);
        int mine = phys;
        if (lane < n_box && (mine < 0 || mine >= p.num_blocks)) {
          record_error(p.err, kErrBlockIndex);
          mine = 0;
        }
        const int row = row_of(mine, tile);
        if (lane == 0 && i >= kStages) free = mbar_wait(&hdr.kv_empty[st][0], ((i >> 1) - 1) & 1, abort);
        if (!__shfl_sync(0xffffffffu, free, 0)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&hdr.kv_full[st], n_box * box_bytes);
        tiles_issued = i + 1;
        __syncwarp();
        for (int g = 0; ok && g < kSlots; ++g) {  // slot by slot, each as soon as it is free
          if (g > 0 && i >= kStages)
            ok = __all_sync(0xffffffffu, mbar_wait(&hdr.kv_empty[st][g], ((i >> 1) - 1) & 1, abort));
          if (ok && lane < n_box && (lane << box_sh) >> 4 == g)
            tma_load_4d(kv + st * kTileBytes + lane * box_bytes, &p.tmap_c, 0, 0, 0, row >> 3, &hdr.kv_full[st]);
        }
        if (!ok) break;
        if (tile == walk.t0) fetch(phys1, tile + 1);
        fetch(phys2, tile + 2);
        phys = phys1;
        phys1 = phys2;
        phys2 = entry(tile + 3);
      }
      if (ok) walk.advance();
    }
    if (!ok && lane == 0) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
      // wait, within the limit, for the copies still in flight
      if (qs_issued > 0) mbar_wait(&hdr.q_full, (qs_issued - 1) & 1, nullptr);
      for (int j = max(0, tiles_issued - kStages); j < tiles_issued; ++j)
        mbar_wait(&hdr.kv_full[j & 1], (j >> 1) & 1, nullptr);
    }
  } else if (warp == kQkWarp) {
    // -------------------------------------------------------------------- S^T
    if (elect_one()) {
      bool ok = true;
      int i = 0;
      const uint32_t qa = smem_addr(qs), ka = smem_addr(kv);
      for (int seg = 0; ok && walk.next(p); ++seg) {
        ok = mbar_wait(&hdr.q_full, seg & 1, abort);
        for (int tile = walk.t0; ok && tile < walk.t1; ++tile, ++i) {
          if (i >= 2) ok = mbar_wait(&hdr.s_empty[i & 1], ((i >> 1) - 1) & 1, abort);
          if (ok) ok = mbar_wait(&hdr.kv_full[i & 1], (i >> 1) & 1, abort);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t tile_at = ka + (i & 1) * kTileBytes;
          const uint64_t a0 = umma_desc_sw128(tile_at, 16, kGroup), b0 = umma_desc_sw128(qa, 16, 1024);
          const uint32_t d = tmem + Lay::TMEM_S + (i & 1) * N;
#pragma unroll
          for (int kk = 0; kk < kCols * 4; ++kk) {
            const uint32_t off = (kk % 4) * 32;
            tc_mma_f16(d, a0 + (((kk / 4) * kAtom + off) >> 4), b0 + (((kk / 4) * Lay::Q_COL + off) >> 4), IDESC_QK,
                       kk > 0);
          }
          tc_commit(&hdr.s_full[i & 1]);
        }
        if (ok) tc_commit(&hdr.q_empty);
        if (ok) walk.advance();
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        *abort = 1;
      }
      tc_commit(&hdr.fin[0]);
      mbar_wait(&hdr.fin[0], 0, nullptr);
    }
  } else {
    // -------------------------------------------------------------------- O^T
    if (elect_one()) {
      bool ok = true;
      int i = 0;
      const uint32_t pa_ = smem_addr(ps), ka = smem_addr(kv);
      while (ok && walk.next(p)) {
        for (int tile = walk.t0; tile < walk.t1; ++tile, ++i) {
          if (!mbar_wait(&hdr.p_full, i & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t a0 = umma_desc_sw128(ka + (i & 1) * kTileBytes, kAtom, kGroup);
          const uint64_t b0 = umma_desc_sw128(pa_, kAtom, 1024);
#pragma unroll
          for (int kk = 0; kk < kSlots; ++kk) {  // 16 tokens: two row groups
#pragma unroll
            for (int b = 0; b < kBlocksO; ++b)
              tc_mma_f16(tmem + b * N, a0 + ((kk * 2 * kGroup + b * 2 * kAtom) >> 4), b0 + ((kk * 2 * 1024) >> 4),
                         IDESC_PV, (tile > walk.t0 || kk > 0) ? 1u : 0u);
            tc_commit(&hdr.kv_empty[i & 1][kk]);
          }
          tc_commit(&hdr.pv_done);
        }
        if (ok) walk.advance();
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        *abort = 1;
      }
      tc_commit(&hdr.fin[1]);
      mbar_wait(&hdr.fin[1], 0, nullptr);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after_sync();
    tc_dealloc(tmem, Lay::TMEM_COLS);
  }
}

// Join the pieces of sequences that several blocks shared, and write the rows
// of sequences without tokens.  Bound by the latency of a chain of small
// loads: where rows are few, many warps take one of them (latent_merge_few),
// where they are many a block takes many rows of one sequence
// (latent_merge_many).
constexpr int kMergeWarps = 16;

// Where a row's pieces lie: n of them, or none where it was written whole.
// The tiles ahead of the sequence come from the lengths where those are few:
// before the wait for the decode kernel, under whose end that stays unseen.
constexpr int kOwnSum = 1024;

template <int N>
struct Pieces {
  int n, late;
  size_t base;
  bool empty;
  // (all threads of the warps that call it, with one s a warp)
  __device__ __forceinline__ Pieces(const LatentParams &p, int max_workers, int s) {
    long long u0 = 0, mine = 0, total = 0;
    if (p.num_seqs <= kOwnSum) {
      constexpr int TILE = N == kPairRows ? 128 : kTile;
      for (int i = threadIdx.x & 31; i < p.num_seqs; i += 32) {
        const int tiles = (checked_len(p.lens, i, p.limit, nullptr) + TILE - 1) / TILE;
        total += tiles;
        u0 += i < s ? tiles : 0;
        mine += i == s ? tiles : 0;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, d);
        u0 += __shfl_xor_sync(0xffffffffu, u0, d);
        mine += __shfl_xor_sync(0xffffffffu, mine, d);
      }
    } else {
      grid_dependency_wait();
      u0 = p.prefix[s];
      mine = p.prefix[s + 1] - u0;
      total = p.prefix[p.num_seqs];
    }
    n = late = 0;
    base = 0;
    empty = mine == 0;
    if (empty) return;
    const long long workers = worker_count(total, max_workers);
    const long long w0 = share_owner(u0, total, workers), w1 = share_owner(u0 + mine - 1, total, workers);
    if (w0 == w1) return;
    n = static_cast<int>(w1 - w0) + 1;
    // a block's first piece is in its place 0; the sequence is not the first of its first block if that began earlier
    late = share_begin(w0, total, workers) < u0;
    base = static_cast<size_t>(w0) * 2 * N;
  }
  // piece i of query row r
  __device__ __forceinline__ size_t at(int i, int r, int max_workers) const {
    return static_cast<size_t>(r / N) * max_workers * 2 * N + base + static_cast<size_t>(2 * i + (i == 0 ? late : 0)) * N +
           r % N;
  }
};

// A lane's VEC fours of dimensions of a row's pieces i, i + step, ...: their
// sum o, its total weight l, both times 2^-top (the lane's fours are 128
// dimensions apart, the first is d0 + 4 lane).  U pieces are on their way at
// a time.
template <int VEC, int U>
struct RowSum {
  float4 o[VEC];
  float l, top;
  template <int N>
  __device__ __forceinline__ RowSum(const LatentParams &p, const Pieces<N> &pieces, int max_workers, int r, int d0,
                                    int i, int step)
      : l(0.f), top(-INFINITY) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; i < pieces.n; i += U * step) {
      float2 ml[U];
      float4 x[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[u][e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + u * step < pieces.n) {
          const size_t at = pieces.at(i + u * step, r, max_workers);
          ml[u] = p.part_ml[at];
          const float4 *from = reinterpret_cast<const float4 *>(p.part_o + at * kLatentDim + d0) + (threadIdx.x & 31);
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[u][e] = from[32 * e];
        }
      }
      const float was = top;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
      const float base = top == -INFINITY ? 0.f : top, f = exp2_fast(was - base);
      l *= f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = make_float4(o[e].x * f, o[e].y * f, o[e].z * f, o[e].w * f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float g = exp2_fast(ml[u].x - base);
        l += g * ml[u].y;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          o[e].x += g * x[u][e].x;
          o[e].y += g * x[u][e].y;
          o[e].z += g * x[u][e].z;
          o[e].w += g * x[u][e].w;
        }
      }
    }
  }
};

// A block joins rows [r0, r0 + per) of a sequence, a warp every 16th, a lane
// 16 of the dimensions.
template <int DT, int N>
__global__ void __launch_bounds__(kMergeWarps * 32, 2) latent_merge_many(const LatentParams p, int max_workers, int per) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (p.rows + per - 1) / per, s = blockIdx.x / chunks, r0 = blockIdx.x % chunks * per;
  const Pieces<N> pieces(p, max_workers, s);
  grid_dependency_wait();
  if (pieces.n == 0 && !pieces.empty) return;
  for (int r = r0 + warp; r < min(p.rows, r0 + per); r += kMergeWarps) {
    const RowSum<4, 2> sum(p, pieces, max_workers, r, 0, 0, 1);
    const float l = sum.l, inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *out = static_cast<uint16_t *>(p.out) + (static_cast<size_t>(s) * p.rows + r) * kLatentDim + lane * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<uint2 *>(out + 128 * e) =
          l == 0.f ? make_uint2(0u, 0u)
                   : make_uint2(pack2_rn<DT>(sum.o[e].x * inv, sum.o[e].y * inv),
                                pack2_rn<DT>(sum.o[e].z * inv, sum.o[e].w * inv));
  }
}

// TEAM warps take one of DSPLIT parts of a row's dimensions, each every
// TEAM-th piece.
template <int DT, int N, int TEAM, int DSPLIT>
__global__ void __launch_bounds__(kMergeWarps * 32) latent_merge_few(const LatentParams p, int max_workers) {
  constexpr int DIMS = kLatentDim / DSPLIT, VEC = DIMS / 128;  // of a block, and the lane's fours of them
  __shared__ float part[kMergeWarps][DIMS];
  __shared__ float sums[kMergeWarps], tops[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mate = warp % TEAM;
  const int row = blockIdx.x / DSPLIT * (kMergeWarps / TEAM) + warp / TEAM, d0 = blockIdx.x % DSPLIT * DIMS;
  const bool exists = row < p.num_seqs * p.rows;
  const Pieces<N> pieces(p, max_workers, exists ? row / p.rows : 0);
  grid_dependency_wait();
  const bool joins = exists && (pieces.n > 0 || pieces.empty);
  const RowSum<VEC, VEC == 1 ? 10 : 3> sum(p, pieces, max_workers, row % p.rows, d0, joins ? mate : pieces.n, TEAM);
  float4 *mine = reinterpret_cast<float4 *>(part[warp]) + lane;
#pragma unroll
  for (int e = 0; e < VEC; ++e) mine[32 * e] = sum.o[e];
  if (lane == 0) {
    sums[warp] = sum.l;
    tops[warp] = sum.top;
  }
  __syncthreads();
  // the team's warps each join a share of the dimensions
  if (!joins) return;
  const int first = warp - mate;
  float top = -INFINITY, l = 0.f, f[TEAM];
#pragma unroll
  for (int i = 0; i < TEAM; ++i) top = fmaxf(top, tops[first + i]);
  if (top == -INFINITY) top = 0.f;
#pragma unroll
  for (int i = 0; i < TEAM; ++i) {
    f[i] = exp2_fast(tops[first + i] - top);
    l += f[i] * sums[first + i];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  constexpr int OWN = DIMS / TEAM / 2;  // pairs of dimensions of a warp
  for (int d = lane; d < OWN; d += 32) {
    const int at = (mate * OWN + d) * 2;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) {
      const float2 z = *reinterpret_cast<const float2 *>(&part[first + i][at]);
      x += f[i] * z.x;
      y += f[i] * z.y;
    }
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + static_cast<size_t>(row) * kLatentDim + d0 + at) =
        l == 0.f ? 0u : pack2_rn<DT>(x * inv, y * inv);
  }
}

template <typename... ARGS>
cudaError_t launch_after(void (*kernel)(ARGS...), unsigned blocks, cudaStream_t stream, ARGS... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DT, int N>
pa_status join(const LatentParams &p, int workers, int sms, cudaStream_t stream) {
  // A row to 64 warps, to 4, or a warp's share of 16 rows.  In us, by the rows
  // of all sequences: one sequence of 131071 tokens, 32 rows 38.1 with 64 warps
  // and 46.2 with 4, 64 rows 46.9 / 54.8, 128 rows 53.5 / 50.4; four of 2048,
  // 32 rows 10.7 / 11.0, 64 rows 13.4 / 11.2, 128 rows 19.7 / 12.4.  With 4 and
  // with a share: four sequences of 4000 tokens, 128 heads, 512 rows 19.2 /
  // 26.7, eight (1024 rows) 28.1 / 30.6, ten (1280) 32.2 / 31.0, 20 of 2000
  // (2560) 36.5 / 29.0, 64 of 2000 (8192) 86.6 / 55.6.
  const long long rows = static_cast<long long>(p.num_seqs) * p.rows;
  cudaError_t e;
  if (rows <= sms / 2) {
    e = launch_after(latent_merge_few<DT, N, 16, 4>, static_cast<unsigned>(rows * 4), stream, p, workers);
  } else if (rows <= sms * 7ll) {
    e = launch_after(latent_merge_few<DT, N, 4, 1>, static_cast<unsigned>((rows + 3) / 4), stream, p, workers);
  } else {
    // as many rows a block as leave one wave of blocks, whole warps of them
    const long long want = rows / (sms * 2ll);
    const int per = want >= p.rows ? p.rows : static_cast<int>((want + kMergeWarps - 1) / kMergeWarps * kMergeWarps);
    e = launch_after(latent_merge_many<DT, N>, static_cast<unsigned>(p.num_seqs) * ((p.rows + per - 1) / per), stream, p,
                     workers, per);
  }
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

// The fewest columns that hold the query rows; pairs of blocks beyond 64.  64
// sequences of 4096 tokens (302 MB, 45 us at the measured copy rate), in us: 16
// rows 61 with 16 columns, 62 with 32, 67 with 64; 32 rows 69 with 32, 74 with
// 64; 40 rows 69 with 64, 74 by pairs; 64 rows 73 with 64, 78 by pairs; 65 rows
// 79 and 128 rows 82 by pairs.
int columns_for(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : kPairRows; }

struct Sizes {
  size_t prefix, ml, o, total;
};
bool sizes_of(int S, int n, int H, Sizes *z) {
  if (S < 0 || n <= 0 || H <= 0) return false;
  const long long rows = static_cast<long long>(n) * H;
  if (rows > INT_MAX / 2 || rows * S > INT_MAX / 2) return false;
  const int N = columns_for(rows);
  // two pieces a share; the row tiles divide the blocks among them, or have one share each
  const long long tiles = (rows + N - 1) / N, most = N == kPairRows ? kMaxPairs : kMaxWorkers;
  const size_t slots = static_cast<size_t>(tiles > most ? tiles : most) * 2;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  z->prefix = up(8 * (static_cast<size_t>(S) + 1));
  z->ml = up(slots * N * sizeof(float2));
  z->o = up(slots * N * kLatentDim * sizeof(float));
  z->total = z->prefix + z->ml + z->o;
  return true;
}

template <int DT, int N>
pa_status launch(LatentParams &p, const void *q, cudaStream_t stream) {
  using Lay = Layout<N>;
  static bool configured[64];  // per device: dynamic shared memory already allowed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(latent_decode_kernel<DT, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::SMEM);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  DeviceInfo info;
  if (!current_device_info(&info)) return cuda_fail(cudaGetLastError());
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return cuda_fail(cudaErrorInvalidValue);
  const cuuint64_t dims[2] = {kLatentRow, static_cast<cuuint64_t>(p.num_seqs) * p.rows};
  const cuuint64_t strides[1] = {kLatentRow * 2};
  const cuuint32_t box[2] = {64, N}, estr[2] = {1, 1};
  if (enc(&p.tmap_q, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(q), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cuda_fail(cudaErrorInvalidValue);
  const int sms = info.sm_count < kMaxWorkers ? info.sm_count : kMaxWorkers;
  const int workers = p.whole ? p.num_seqs : sms;
  latent_decode_kernel<DT, N><<<workers, kThreads, Lay::SMEM, stream>>>(p, workers);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  return p.whole ? PA_OK : join<DT, N>(p, workers, info.sm_count, stream);
}

template <int DT>
pa_status by_rows(LatentParams &p, const void *q, const void *cache, const pa_latent_desc *desc, cudaStream_t stream) {
  switch (columns_for(p.rows)) {
    case 16: return launch<DT, 16>(p, q, stream);
    case 32: return launch<DT, 32>(p, q, stream);
  }
  if (p.rows <= 64) return launch<DT, 64>(p, q, stream);
  int workers = 0;
  const pa_status st = launch_latent_pair(DT, p, q, cache, desc, &workers, stream);
  DeviceInfo info;
  return st != PA_OK || p.whole || !current_device_info(&info) ? st : join<DT, kPairRows>(p, workers, info.sm_count, stream);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_latent_decode_workspace_size(int32_t num_seqs, int32_t new_tokens, int32_t num_heads) {
  Sizes z;
  return sizes_of(num_seqs, new_tokens, num_heads, &z) ? z.total : 0;
}

extern "C" pa_status pa_latent_decode(void *out, const void *q, int32_t q_dtype, int32_t num_seqs, int32_t new_tokens,
                                      int32_t num_heads, const void *cache, const pa_latent_desc *desc,
                                      const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
                                      int32_t max_seq_len, float scale, void *workspace, size_t workspace_bytes,
                                      int *device_error, pa_stream_t stream) {
  if (!valid_latent_desc(desc) || num_seqs < 0 || new_tokens <= 0 || num_heads <= 0 || max_seq_len < 0 ||
      max_blocks_per_seq <= 0 || !isfinite(scale))
    return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !cache || !block_tables || !seq_lens || !workspace) return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(cache) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_INVALID;
  if (!supported_latent_desc(desc) || q_dtype != desc->dtype) return PA_ERR_UNSUPPORTED;
  Sizes z;
  if (!sizes_of(num_seqs, new_tokens, num_heads, &z)) return PA_ERR_UNSUPPORTED;
  if (workspace_bytes < z.total) return PA_ERR_INVALID;
  LatentParams p{};
  const int box_groups = desc->block_size == 8 ? 1 : 2;
  if (!encode_latent_view(&p.tmap_c, cache, desc, kCols, box_groups)) return cuda_fail(cudaErrorInvalidValue);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.out = out;
  p.cache = static_cast<const uint16_t *>(cache);
  p.tables = block_tables;
  p.lens = seq_lens;
  p.prefix = reinterpret_cast<long long *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + z.prefix);
  p.part_o = reinterpret_cast<float *>(ws + z.prefix + z.ml);
  p.num_seqs = num_seqs;
  p.new_tokens = new_tokens;
  p.heads = num_heads;
  p.rows = new_tokens * num_heads;
  p.num_blocks = desc->num_blocks;
  p.bs_shift = log2_block(desc->block_size);
  p.max_blocks = max_blocks_per_seq;
  const long long held = static_cast<long long>(max_blocks_per_seq) * desc->block_size;
  long long limit = held < max_seq_len ? held : max_seq_len;
  if (limit > INT_MAX / 4) limit = INT_MAX / 4;
  p.limit = static_cast<int>(limit);
  DeviceInfo info;
  if (!current_device_info(&info)) return cuda_fail(cudaGetLastError());
  const bool pairs = p.rows > 64;  // of blocks
  const long long units = pairs ? (p.rows + kPairRows - 1ll) / kPairRows * num_seqs : num_seqs;
  p.whole = max_seq_len <= kWholeTokens && units <= kWholeWaves * (pairs ? info.sm_count / 2 : info.sm_count);
  p.out_sectors = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = device_error;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return desc->dtype == PA_F16 ? by_rows<kF16>(p, q, cache, desc, st) : by_rows<kBF16>(p, q, cache, desc, st);
}
