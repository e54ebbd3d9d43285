// pa_latent_decode with more than 64 query rows a sequence: row tiles of 128
// query rows to a pair of blocks, whose tensor cores work as one
// (tcgen05 cta_group::2).
//
// The products of a tile of 128 tokens:
//   S = Q K^T   M = 128 query rows (64 a block), N = 128 tokens, K = 576
//   O += P V    M = 128, N = 256 dimensions (twice), K = 128 tokens
// Each block holds its 64 query rows, half of the tile's tokens for the first
// product and half of the dimensions, of all tokens, for the second; the
// tensor cores of both read the operands of either.  K and V are loaded apart,
// V from L2 a second time: each part of shared memory is then held only from
// its load to its own product, not through the softmax between them, and what
// fits (one tile of each) is in flight most of the time.  A tile of 128 tokens
// takes the tensor cores 2200 clocks and, at the memory's rate, a pair's share
// of it 3200; it takes about 4000: the 278 KB of K and V that a pair draws from
// L2 for it, and the chain from S through the weights to O.  (pa_latent_decode.cu
// with two blocks of 64 rows a tile took 3500 clocks for 64 tokens.)  128
// sequences of 512..4096 tokens with 128 heads: 85 us, and 10 more for the join
// of the pieces; 375 MB, 56 us at the measured copy rate.
//
// Tensor memory of a block: row r of its 64 in lanes r and r + 64, the first
// half of a product's columns in the former, the other half in the latter.
// S has two buffers of 64 columns, O 256 columns.
//
// Warps of either block:
//   0..7  softmax: four threads a query row, 32 tokens each.  The maximum is
//         raised, and O rescaled, only when a score passes it by 2^8.
//   8     TMA: q, then K in three parts of three 128-byte columns
//   9, 10 (first block) issue the products of both
//   11    TMA: V in two parts of 64 tokens
#include <limits.h>
#include <math.h>

#include "pa_latent_decode.cuh"

namespace pa {
namespace {

constexpr int kTile = 128;
constexpr int kHalfRows = kPairRows / 2;
constexpr int kCols = kLatentRow / 64;                  // 128-byte columns of a row
constexpr int kQCol = kHalfRows * 128;
constexpr int kQBytes = kCols * kQCol;
constexpr int kKParts = 3, kKCols = kCols / kKParts;    // parts of K, and their columns
constexpr int kKGroup = kKCols * 1024;                  // 8 tokens of a part
constexpr int kKBytes = 8 * kKGroup;                    // 64 tokens
constexpr int kVParts = 2, kVGroup = 4 * 1024;          // of V: 64 tokens, 256 dimensions each
constexpr int kVBytes = 8 * kVGroup;
constexpr int kPBlock = kHalfRows * 128;                // 64 tokens of P
constexpr int kQOff = 2048, kPOff = kQOff + kQBytes, kKOff = kPOff + 2 * kPBlock, kVOff = kKOff + kKParts * kKBytes;
constexpr int kSmem = kVOff + kVParts * kVBytes;
constexpr int kKTmaWarp = 8, kQkWarp = 9, kVTmaWarp = 11;  // (10: O)
constexpr int kThreads = 12 * 32;
constexpr int kArrivals = 2 * kSoftmaxThreads / 32;     // the softmax warps of both blocks
constexpr uint32_t kTmemS = 256, kTmemCols = 512;
static_assert(kSmem <= 232448 && kKOff % 1024 == 0, "shared memory");

struct Header {
  uint64_t q_full, q_empty, k_full[kKParts], k_empty[kKParts], v_full, v_last, v_empty[kVParts], s_full[2], s_empty[2], p_full,
      pv_done, fin[2];
  uint32_t tmem;
  int abort;
  float top[4][kHalfRows];  // maxima of a row's quarters, then their total weights
};
static_assert(sizeof(Header) <= 2048, "the header's place");

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_pair_kernel(const __grid_constant__ LatentParams p, int max_workers) {
  constexpr int AB = DT == kF16 ? 0 : 1;
  constexpr uint32_t IDESC_QK = umma_idesc_f16(AB, kPairRows, kTile, false);
  constexpr uint32_t IDESC_PV = umma_idesc_f16(AB, kPairRows, 256, true);
  extern __shared__ __align__(1024) uint8_t smem[];
  // (the scan is over before the weights' buffer is first written)
  ShareScan<128> &scan = *reinterpret_cast<ShareScan<128> *>(smem + kPOff);
  static_assert(sizeof(ShareScan<128>) <= 2 * kPBlock, "the scan's place");
  Header &hdr = *reinterpret_cast<Header *>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cluster_rank();
  const int pair = blockIdx.x >> 1, rt = pair % p.row_tiles, w = pair / p.row_tiles;
  if (!p.whole) launch_dependents();  // (the merge)
  auto tiles_of = [&](int s) -> long long { return (checked_len(p.lens, s, p.limit, p.err) + kTile - 1) / kTile; };
  Walk<kTile> walk;
  if (p.whole) {
    walk.u = walk.first = 0;
    walk.s = w;
    walk.end = tiles_of(w);
    if (walk.end == 0) {  // (both blocks)
      const int first = rt * kPairRows + kHalfRows * rank;
      zero_rows(p.out, static_cast<long long>(w) * p.rows + first, min(kHalfRows, p.rows - first));
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
    if (w >= workers) return;  // (both blocks)
    walk.u = share_begin(w, total, workers);
    walk.end = share_begin(w + 1, total, workers);
    walk.s = scan.find(walk.u, p.num_seqs, tiles_of, walk.first);
  }
  volatile int *abort = &hdr.abort;
  uint8_t *qs = smem + kQOff, *ps = smem + kPOff, *ks = smem + kKOff, *vs = smem + kVOff;
  if (warp == kKTmaWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_c)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_v)) : "memory");
    mbar_init(&hdr.q_full, 1);
    mbar_init(&hdr.q_empty, 1);
    for (int i = 0; i < kKParts; ++i) {
      mbar_init(&hdr.k_full[i], 1);
      mbar_init(&hdr.k_empty[i], 1);
    }
    mbar_init(&hdr.v_full, 1);
    mbar_init(&hdr.v_last, 1);
    for (int i = 0; i < kVParts; ++i) mbar_init(&hdr.v_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hdr.s_full[i], 1);
      mbar_init(&hdr.s_empty[i], kArrivals);
    }
    mbar_init(&hdr.p_full, kArrivals);
    mbar_init(&hdr.pv_done, 1);
    mbar_init(&hdr.fin[0], 1);
    mbar_init(&hdr.fin[1], 1);
    hdr.abort = 0;
    fence_mbar_init();
  }
  if (warp == kQkWarp) {
    pair_alloc(&hdr.tmem, kTmemCols);
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // the other block's mbarriers and tensor memory are there
  tc_fence_after_sync();
  const uint32_t tmem = hdr.tmem;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int quadrant = warp & 3, part = warp >> 2;
    const int r = 32 * (quadrant & 1) + lane;                   // the thread's query row among the block's 64
    const int half = quadrant >> 1;                             // of a product's columns
    const int q4 = 2 * half + part;                             // the thread's quarter of the row
    const int row = rt * kPairRows + kHalfRows * rank + r;      // among the sequence's query rows
    const uint32_t tlane = tmem + (static_cast<uint32_t>(32 * quadrant) << 16);
    const float c = p.scale_log2;
    const uint32_t s_empty[2] = {in_block(&hdr.s_empty[0], 0), in_block(&hdr.s_empty[1], 0)};
    const uint32_t p_full = in_block(&hdr.p_full, 0);
    // a wait that gave up leaves the warp in step with the others, whose
    // barriers count on it: it goes on without waiting, and nothing is stored
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
      tc_fence_after_sync();
    };
    int i = 0, lasts = 0;  // tiles so far, and those that end past their sequence's plain end
    for (int seg = 0; walk.next(p); ++seg) {
      const int see = row < p.rows ? walk.L - (p.new_tokens - 1 - row / p.heads) : 0;  // tokens the row sees
      const int all_see = (rt + 1) * kPairRows > p.rows ? 0 : walk.L - (p.new_tokens - 1 - rt * kPairRows / p.heads);
      const int plain = plain_end(p, walk.L);
      float m = -INFINITY, l = 0.f;  // m: the maximum less kLift
      constexpr float OVER = kLazy + kLift<DT>;
      for (int tile = walk.t0; tile < walk.t1; ++tile, ++i) {
        wait(&hdr.s_full[i & 1], (i >> 1) & 1);
        uint32_t raw[32];
        tc_ld32(tlane + kTmemS + (i & 1) * 64 + 32 * part, raw);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) pair_arrive(s_empty[i & 1]);
        float x[32], top = -INFINITY;
        const int key = tile * kTile + 32 * q4;
        if ((tile + 1) * kTile > all_see) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = key + j < see ? __uint_as_float(raw[j]) * c : -INFINITY;
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(raw[j]) * c;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 4) top = fmaxf(top, fmaxf(fmaxf(x[j], x[j + 1]), fmaxf(x[j + 2], x[j + 3])));
        if (softmax_any(top - m > OVER)) {  // (a difference: exact where the two are close)
          hdr.top[q4][r] = top;
          softmax_sync();
          top = fmaxf(fmaxf(hdr.top[0][r], hdr.top[1][r]), fmaxf(hdr.top[2][r], hdr.top[3][r]));
          const bool grow = top - m > OVER;
          const float next = top - kLift<DT>, f = grow ? exp2_fast(m - next) : 1.f;
          l *= f;
          if (grow) m = next;
          if (tile > walk.t0) {  // O holds the tiles before
            wait(&hdr.pv_done, (i - 1) & 1);
#pragma unroll 1
            for (int d = 0; d < 128; d += 32) {
              uint32_t o[32];
              tc_ld32(tlane + part * 128 + d, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc_st32(tlane + part * 128 + d, o);
            }
          }
          softmax_sync();  // the maxima have been read
        }
        // weights, rounded to the operand type (half a step each; see kLift)
        const float base = m == -INFINITY ? 0.f : m;
        uint32_t pw[16];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float a = exp2_fast(x[j] - base), b = exp2_fast(x[j + 1] - base);
          sum[j & 2] += a;
          sum[(j & 2) + 1] += b;
          pw[j / 2] = pack2_rn<DT>(a, b);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // the P buffer is free once the last tile's O products have completed
        if (i > 0) wait(&hdr.pv_done, (i - 1) & 1);
        uint8_t *to = ps + half * kPBlock + r * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4 *>(to + (((4 * part + u) ^ (r & 7)) << 4)) =
              make_uint4(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]);
        if ((tile + 1) * kTile > plain) {
          // rows behind the sequence's end hold anything: zero them, 0 * NaN would reach O; of drafted tokens before
          // it what is not finite is taken out
          wait(&hdr.v_last, lasts++ & 1);
          const int z0 = max(plain - tile * kTile, 0), z1 = walk.L - tile * kTile;
          for (int idx = threadIdx.x; idx < (kTile - z0) * 32; idx += kSoftmaxThreads) {
            const int z = z0 + idx / 32, e = idx % 32;  // token, and 16 bytes of its 256 dimensions
            uint4 *at = reinterpret_cast<uint4 *>(vs + (z >> 3) * kVGroup + (e >> 3) * 1024 + (z & 7) * 128 + (e & 7) * 16);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (z < z1) {
              x = *at;
              if (!take_out<DT>(x)) continue;
            }
            *at = x;
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) pair_arrive(p_full);
      }
      softmax_sync();  // (the maxima have been read)
      hdr.top[q4][r] = l;
      softmax_sync();
      l = (hdr.top[0][r] + hdr.top[1][r]) + (hdr.top[2][r] + hdr.top[3][r]);
      // drafted tokens of this piece that are not finite in some dimension (V's other half lies in the other block: their
      // rows are read again, under the last products)
      const int from = max(plain, walk.t0 * kTile), end = min(walk.L, walk.t1 * kTile);
      bool patch = false;
      if (p.new_tokens > 1 && from < end) {
        for (int idx = threadIdx.x; idx < (end - from) * (kLatentDim / 8); idx += kSoftmaxThreads) {
          uint4 x = __ldg(reinterpret_cast<const uint4 *>(token_row(p, walk.s, from + idx / (kLatentDim / 8))) +
                          idx % (kLatentDim / 8));
          patch |= take_out<DT>(x);
        }
        patch = softmax_any(patch);
      }
      wait(&hdr.pv_done, (i - 1) & 1);
      const bool whole = walk.t0 == 0 && walk.t1 == walk.tiles;
      const int d0 = half * 256 + part * 128;  // the thread's dimensions
      const bool mine = ok && row < p.rows;
      auto load_o = [&](int d, uint32_t (&o)[32]) {  // 32 of them
        tc_ld32(tlane + part * 128 + d, o);
        if (patch) {  // not-a-number where a token that the row sees is not finite
          for (int t = from; t < min(end, see); ++t) {
            const uint4 *x4 = reinterpret_cast<const uint4 *>(token_row(p, walk.s, t) + d0 + d);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 x = __ldg(x4 + u);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if ((w[j / 2] >> 16 * (j & 1) & kNotFinite<DT>) == kNotFinite<DT>) o[8 * u + j] = 0x7fffffffu;
            }
          }
          __syncwarp();
        }
      };
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that sees nothing)
        uint8_t *to = static_cast<uint8_t *>(p.out) + ((static_cast<size_t>(walk.s) * p.rows + row) * kLatentDim + d0) * 2;
#pragma unroll 1
        for (int d = 0; d < 128; d += 32) {
          uint32_t o[32], y[16];
          load_o(d, o);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            y[j] = l == 0.f ? 0u
                            : pack2_rn<DT>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
          if (mine && p.out_sectors) {
            store32(to + d * 2, y);
            store32(to + d * 2 + 32, y + 8);
          } else if (mine) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              *reinterpret_cast<uint4 *>(to + d * 2 + j * 4) = make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]);
          }
        }
      } else {
        const size_t slot =
            ((static_cast<size_t>(rt) * max_workers + w) * 2 + (seg > 0)) * kPairRows + kHalfRows * rank + r;
        if (mine && q4 == 0) p.part_ml[slot] = make_float2(m, l);
        uint8_t *to = reinterpret_cast<uint8_t *>(p.part_o + slot * kLatentDim + d0);
#pragma unroll 1
        for (int d = 0; d < 128; d += 32) {
          uint32_t o[32];
          load_o(d, o);
          if (mine)
#pragma unroll
            for (int j = 0; j < 32; j += 8) store32(to + (d + j) * 4, o + j);
        }
      }
      tc_fence_before_sync();
      walk.advance();
    }
    if (!ok) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
    }
  } else if (warp == kKTmaWarp || warp == kVTmaWarp) {
    // -------------------------------------------------------------------- TMA
    // boxes of 16 tokens (of 8 with blocks of 8): K, of the block's 64 tokens
    // of a tile, lane (part, box); V, of all 128, lane (64 tokens, box).  Bytes
    // count in the first block, for the products' issue, but for V tiles that
    // end past their sequence's plain end: those count in each block, whose
    // softmax warps put the rows behind it right before the weights are announced.
    const bool is_k = warp == kKTmaWarp;
    const int box_sh = p.bs_shift < 4 ? 3 : 4, boxes = 64 >> box_sh;  // boxes of 64 tokens
    const int piece = lane / boxes, box = lane % boxes;               // this lane's part, and box in it
    const int parts = is_k ? kKParts : kVParts;
    const bool in = piece < parts;
    const int tok0 = (is_k ? 64 * rank : 64 * piece) + (box << box_sh);  // its first token in a tile
    const uint32_t bytes = (1u << box_sh) / 8 * (is_k ? kKGroup : kVGroup);
    uint8_t *to = is_k ? ks + piece * kKBytes + box * bytes : vs + piece * kVBytes + box * bytes;
    const int column = is_k ? piece * kKCols : 4 * rank;
    uint64_t *empty = is_k ? hdr.k_empty : hdr.v_empty;
    const uint32_t q_full = in_block(&hdr.q_full, 0);
    const uint32_t full = in_block(is_k ? &hdr.k_full[in ? piece : 0] : &hdr.v_full, 0);
    bool ok = true;
    // tiles done, parts of the next one, V tiles announced in v_full and in v_last, sequences whose q is
    int i = 0, issued = 0, fulls = 0, lasts = 0, qs_issued = 0;
    for (int seg = 0; ok && walk.next(p); ++seg) {
      const int32_t *table = p.tables + static_cast<size_t>(walk.s) * p.max_blocks;
      auto entry = [&](int tile) {
        const int tok = tile * kTile + tok0;
        return in && tok < walk.L ? __ldg(table + (tok >> p.bs_shift)) : 0;
      };
      // K is fetched into L2 two tiles ahead of its copy (V then comes from there)
      auto row8_of = [&](int block, int tile) {
        const int tok = tile * kTile + tok0;
        return ((block << p.bs_shift) + (tok & ((1 << p.bs_shift) - 1))) >> 3;
      };
      auto fetch = [&](int block, int tile) {
        if (is_k && in && tile < walk.t1 && tile * kTile + tok0 < walk.L && block >= 0 && block < p.num_blocks)
          tma_prefetch_4d(&p.tmap_c, 0, 0, column, row8_of(block, tile));
      };
      int phys = entry(walk.t0), phys1 = entry(walk.t0 + 1), phys2 = entry(walk.t0 + 2);
      if (is_k) {
        bool free = true;
        if (lane == 0 && seg > 0) free = mbar_wait(&hdr.q_empty, (seg - 1) & 1, abort);
        if (!__shfl_sync(0xffffffffu, free, 0)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&hdr.q_full, 2 * kQBytes);
          const int row = walk.s * p.rows + rt * kPairRows + kHalfRows * rank;
          for (int e = 0; e < kCols; ++e) pair_load_2d(qs + e * kQCol, &p.tmap_q, e * 64, row, q_full);
        }
        ++qs_issued;
      }
      for (int tile = walk.t0; tile < walk.t1; ++tile, ++i) {
        const int tok = tile * kTile + tok0;
        int mine = phys;
        const bool loads = in && tok < walk.L;
        if (loads && (mine < 0 || mine >= p.num_blocks)) {
          record_error(p.err, kErrBlockIndex);
          mine = 0;
        }
        const int left = walk.L - tile * kTile;  // tokens of the tile, and boxes of them
        const int n = (min(left, kTile) + (1 << box_sh) - 1) >> box_sh;
        const bool last = (tile + 1) * kTile > plain_end(p, walk.L);
        const int row8 = row8_of(mine, tile);
        // part by part, each as soon as it is free
        for (int g = 0; ok && g < parts; ++g) {
          if (i > 0) ok = __all_sync(0xffffffffu, mbar_wait(empty + g, (i - 1) & 1, abort));
          if (!ok) break;
          if (g == 0) ++(last ? lasts : fulls);
          issued = g + 1;
          if (lane == 0) {
            if (is_k && rank == 0) mbar_arrive_expect_tx(&hdr.k_full[g], n * bytes);
            if (!is_k && g == 0 && last) mbar_arrive_expect_tx(&hdr.v_last, n * bytes);
            if (!is_k && g == 0 && !last && rank == 0) mbar_arrive_expect_tx(&hdr.v_full, 2 * n * bytes);
          }
          __syncwarp();
          if (loads && piece == g) {
            if (!is_k && last)
              tma_load_4d(to, &p.tmap_v, 0, 0, column, row8, &hdr.v_last);
            else
              pair_load_4d(to, is_k ? &p.tmap_c : &p.tmap_v, 0, 0, column, row8, full);
          }
        }
        if (!ok) break;
        issued = 0;
        if (tile == walk.t0) fetch(phys1, tile + 1);
        fetch(phys2, tile + 2);
        phys = phys1;
        phys1 = phys2;
        phys2 = entry(tile + 3);
      }
      if (ok) walk.advance();
    }
    if (ok && i > 0) {  // the last products' arrivals in this block
      for (int g = 0; g < parts; ++g) ok = ok && mbar_wait(empty + g, (i - 1) & 1, abort);
      if (is_k) ok = ok && mbar_wait(&hdr.q_empty, (qs_issued - 1) & 1, abort);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok && lane == 0) {
      record_error(p.err, kErrTimeout);
      *abort = 1;
      // wait, within the limit, for the copies still in flight (of those that count in the first block it is that block
      // that waits, and the other stays until it has)
      if (is_k && rank == 0) {
        if (qs_issued > 0) mbar_wait(&hdr.q_full, (qs_issued - 1) & 1, nullptr);
        for (int g = 0; g < kKParts; ++g) {
          const int n = i + (g < issued);  // of this part
          if (n > 0) mbar_wait(&hdr.k_full[g], (n - 1) & 1, nullptr);
        }
      } else if (!is_k) {
        if (fulls > 0 && rank == 0) mbar_wait(&hdr.v_full, (fulls - 1) & 1, nullptr);
        if (lasts > 0) mbar_wait(&hdr.v_last, (lasts - 1) & 1, nullptr);
      }
    }
  } else if (warp == kQkWarp) {
    // -------------------------------------------------------------------- S
    if (rank == 0 && elect_one()) {
      bool ok = true;
      int i = 0;
      const uint32_t qa = smem_addr(qs), ka = smem_addr(ks);
      for (int seg = 0; ok && walk.next(p); ++seg) {
        ok = mbar_wait(&hdr.q_full, seg & 1, abort);
        for (int tile = walk.t0; ok && tile < walk.t1; ++tile, ++i) {
          if (i >= 2) ok = mbar_wait(&hdr.s_empty[i & 1], ((i >> 1) - 1) & 1, abort);
          const uint32_t d = tmem + kTmemS + (i & 1) * 64;
          for (int g = 0; ok && g < kKParts; ++g) {
            ok = mbar_wait(&hdr.k_full[g], i & 1, abort);
            if (!ok) break;
            tc_fence_after_sync();
            const uint64_t a0 = umma_desc_sw128(qa + g * kKCols * kQCol, 16, 1024);
            const uint64_t b0 = umma_desc_sw128(ka + g * kKBytes, 16, kKGroup);
#pragma unroll
            for (int kk = 0; kk < kKCols * 4; ++kk) {
              const uint32_t off = (kk % 4) * 32;
              pair_mma(d, a0 + (((kk / 4) * kQCol + off) >> 4), b0 + (((kk / 4) * 1024 + off) >> 4), IDESC_QK,
                       (g > 0 || kk > 0) ? 1u : 0u);
            }
            pair_commit(&hdr.k_empty[g]);
          }
          if (ok) pair_commit(&hdr.s_full[i & 1]);
        }
        if (ok) pair_commit(&hdr.q_empty);
        if (ok) walk.advance();
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        *abort = 1;
      }
      pair_commit(&hdr.fin[0]);
    }
  } else {
    // -------------------------------------------------------------------- O
    if (rank == 0 && elect_one()) {
      bool ok = true;
      int i = 0, fulls = 0;
      const uint32_t pa_ = smem_addr(ps), va = smem_addr(vs);
      while (ok && walk.next(p)) {
        for (int tile = walk.t0; tile < walk.t1; ++tile, ++i) {
          if (!mbar_wait(&hdr.p_full, i & 1, abort)) {
            ok = false;
            break;
          }
          // (of a tile that ends past its sequence's plain end, the weights' arrival says that V is there)
          if ((tile + 1) * kTile <= plain_end(p, walk.L) && !mbar_wait(&hdr.v_full, fulls++ & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
#pragma unroll
          for (int g = 0; g < kVParts; ++g) {  // 64 tokens
            const uint64_t a0 = umma_desc_sw128(pa_ + g * kPBlock, 16, 1024);
            const uint64_t b0 = umma_desc_sw128(va + g * kVBytes, 1024, kVGroup);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int b = 0; b < 2; ++b)  // 128 dimensions of either block
                pair_mma(tmem + b * 128, a0 + (kk * 32 >> 4), b0 + ((kk * 2 * kVGroup + b * 2 * 1024) >> 4), IDESC_PV,
                         (tile > walk.t0 || g > 0 || kk > 0) ? 1u : 0u);
            pair_commit(&hdr.v_empty[g]);
          }
          pair_commit(&hdr.pv_done);
        }
        if (ok) walk.advance();
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        *abort = 1;
      }
      pair_commit(&hdr.fin[1]);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  // every product has completed, and its arrivals in this block with it, whether the block gave up or not
  if (warp == kQkWarp) {
    mbar_wait(&hdr.fin[0], 0, nullptr);
    mbar_wait(&hdr.fin[1], 0, nullptr);
    __syncwarp();
  }
  cluster_sync();  // both blocks are done with the other's shared memory and tensor memory
  if (warp == kQkWarp) {
    tc_fence_after_sync();
    pair_dealloc(tmem, kTmemCols);
  }
  cluster_sync();
}

template <int DT>
pa_status launch(const LatentParams &p, int workers, cudaStream_t stream) {
  static bool configured[64];  // per device: dynamic shared memory already allowed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(latent_pair_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  latent_pair_kernel<DT><<<2 * workers * p.row_tiles, kThreads, kSmem, stream>>>(p, workers);
  e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace

pa_status launch_latent_pair(int dtype, LatentParams &p, const void *q, const void *cache, const pa_latent_desc *desc,
                             int *workers, cudaStream_t stream) {
  DeviceInfo info;
  if (!current_device_info(&info)) return cuda_fail(cudaGetLastError());
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint64_t dims[2] = {kLatentRow, static_cast<cuuint64_t>(p.num_seqs) * p.rows};
  const cuuint64_t strides[1] = {kLatentRow * 2};
  const cuuint32_t box[2] = {64, kHalfRows}, estr[2] = {1, 1};
  const int groups = desc->block_size == 8 ? 1 : 2;
  if (enc == nullptr ||
      enc(&p.tmap_q, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(q), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      !encode_latent_view(&p.tmap_c, cache, desc, kKCols, groups) || !encode_latent_view(&p.tmap_v, cache, desc, 4, groups))
    return cuda_fail(cudaErrorInvalidValue);
  p.row_tiles = (p.rows + kPairRows - 1) / kPairRows;
  const int pairs = info.sm_count / 2 < kMaxPairs ? info.sm_count / 2 : kMaxPairs;
  *workers = p.whole ? p.num_seqs : pairs / p.row_tiles > 0 ? pairs / p.row_tiles : 1;
  if (2ll * *workers * p.row_tiles > INT_MAX) return PA_ERR_UNSUPPORTED;
  return dtype == kF16 ? launch<kF16>(p, *workers, stream) : launch<kBF16>(p, *workers, stream);
}

}  // namespace pa
