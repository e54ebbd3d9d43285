// pa_decode_weights: single-query decode attention that also adds every
// token's attention weight to an accumulator.
//
// For a (sequence, KV head) pair with G query heads and tokens i < L:
//   x[g, i] = scale <q_g, k_i>,  w[g, i] = exp(x[g, i] - m_g) / l_g,
//   out[g]  = sum_i w[g, i] v_i,  weights_out[i] = decay weights_in[i] + sum_g w[g, i].
// A token's weight is known only once m_g and l_g are, after the whole row.
// Reading K a second time would cost half as much again as the attention;
// instead the first kernel leaves the scores (G fp32 a token and head, 32
// bytes against 512 of K and V at G = 8, head_dim 128, 16 bits) and a second
// one turns them into weights.
//
// First kernel: every warp takes an equal share of all (sequence, head,
// 16-token) steps and keeps K and V in registers, loaded straight from
// global memory a step ahead; nothing is staged in shared memory.
//   S = Q K^T   m16n8k16: rows are queries (8 of 16 used), columns tokens;
//   O^T += V^T P^T  rows are dimensions, columns queries.
// A product's order of k does not matter, so a lane takes whole 16-byte
// pieces of a row as its fragments: lane (g, t) of K reads token
// 4 (g / 2) + g % 2 (+ 2) and feeds consecutive words to consecutive
// products, q in the same order.  The score fragment of the lane is then
// exactly its P^T fragment (query g, tokens 4t..4t+3), and V's words of
// two tokens are paired by byte permutes.
// Sums and maxima are fp32, P is rounded to the operand type (half a step of
// it a weight, averaged over tokens; see kLift); the weights that are handed
// out come from the fp32 scores.
//
// Second kernel: joins the shares of a pair (out), and adds the weights.
//
// 64 sequences of 256..32768 tokens, 64/8 heads, head_dim 128, bf16: 1.83 GB,
// 273 us at the measured copy rate; 300 us here (bound by memory, 0.12 GB of
// scores and pieces on top) and 30 for the second kernel, whose launch runs
// under the end of the first.
#include <limits.h>
#include <math.h>

#include "pa_fp4.cuh"
#include "pa_host.h"
#include "pa_latent_common.cuh"
#include "pa_shares.cuh"

namespace pa {
namespace {

constexpr int kStep = 16;             // tokens of a step
constexpr int kWarps = 4;             // of a block
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWorkers = 152 * 16; // warps, at most; sizes the workspace
constexpr int kMinSteps = 4;          // a share smaller than this only adds joining
// Pairs of up to this many tokens are not split: one warp weighs, joins and
// writes them, and there is no second kernel.  Unsplit and split, 32/8 heads of
// 128, in us: 4 sequences of 64 tokens 7.3 / 10.4, of 128 10.8 / 10.0, of 192
// 14.1 / 10.6; 64 of 128 11.8 / 15.8, of 192 17.4 / 16.8; 512 of 128 58 / 67,
// of 256 106 / 107.
constexpr int kWholeTokens = 128;
constexpr float kLazy = 8.f;          // a row's maximum is raised when it grew by more than this (base 2)
// The largest weight of a row is held as 2^kLift or more: fp16's smallest step
// is 2^-24, so that a weight is off by at most 2^-32 of the largest where it
// would be lost below 2^-25, and the total keeps all of it (131071 tokens 17
// nats below one are 0.4 % of it).  2^(kLazy + kLift) is well inside fp16.
// bf16 has a float's range and needs none of it.
template <int MT>
constexpr float kLift = MT == kF16 ? 7.f : 0.f;

struct WeighParams {
  void *out;
  const void *q;
  const uint8_t *k, *v;
  const int32_t *tables, *lens;
  const float *weights_in;
  float *weights_out;
  float *logits;       // [S, Hq, width]
  float2 *part_ml;     // [pairs + workers, G]
  float *part_o;       // [pairs + workers, G, D]
  long long *prefix;   // [S + 1] steps of one head before sequence s
  int num_seqs, q_heads, kv_heads, G, num_blocks, bs_shift, max_blocks, limit, width;
  long long weights_width;
  float scale_log2, v_scale, decay;
  bool whole;          // a warp takes all of a pair: nothing to join
  const float *k_head_scale, *v_head_scale;
  int *err;
};

// K and V are read once: they leave L2 first, so that the scores and sums
// written on the way are still there for the second kernel.
__device__ __forceinline__ uint4 ldg_stream(const void *p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ uint2 ldg_stream2(const void *p, uint64_t policy) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v2.b32 {%0, %1}, [%2], %3;"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ uint32_t lows(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// workers of a call with `steps` steps in all
__device__ __forceinline__ long long worker_count(long long steps, long long most) {
  const long long n = (steps + kMinSteps - 1) / kMinSteps;
  return n < most ? n : most;
}

template <int KVT, int QT, int D>
__global__ void __launch_bounds__(kThreads, 3) weigh_kernel(const WeighParams p, int max_workers) {
  constexpr bool BYTE = is_byte(KVT);
  constexpr int MT = BYTE ? kF16 : KVT;  // the products' type
  constexpr int EB = elt_bytes(KVT);
  constexpr int ROW = D * EB;
  constexpr int KW = ROW / 64;          // 16-byte words of a K row a lane holds
  constexpr int QWORDS = D / 8;         // 32-bit words of q a lane holds
  constexpr int VWORDS = ROW / 32;      // 32-bit words of a V row a lane holds
  constexpr int ACC = D / 16;           // accumulator tiles
  __shared__ ShareScan<kThreads> scan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (!p.whole) launch_dependents();  // (the second kernel)
  auto steps_of = [&](int s) {
    return static_cast<long long>((checked_len(p.lens, s, p.limit, p.err) + kStep - 1) / kStep) * p.kv_heads;
  };
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + warp;
  long long u, end, first;
  int s;
  if (p.whole) {
    if (w >= static_cast<long long>(p.num_seqs) * p.kv_heads) return;
    s = static_cast<int>(w / p.kv_heads);
    const int h = static_cast<int>(w - static_cast<long long>(s) * p.kv_heads);
    const long long steps = steps_of(s) / p.kv_heads;
    first = 0;
    u = h * steps;
    end = u + steps;
    if (steps == 0)  // no token
      for (int i = lane; i < p.G * D / 2; i += 32)
        reinterpret_cast<uint32_t *>(p.out)[(static_cast<size_t>(s) * p.q_heads + h * p.G) * (D / 2) + i] = 0u;
  } else {
    scan.scan(p.num_seqs, steps_of);
    if (blockIdx.x == 0) {  // the sequences' first steps, for the second kernel
      const int n = scan.run(p.num_seqs);
      long long at = scan.base[threadIdx.x];
      for (int i = threadIdx.x * n; i < min(p.num_seqs, (static_cast<int>(threadIdx.x) + 1) * n); ++i) {
        p.prefix[i] = at;
        at += steps_of(i);
      }
      if (threadIdx.x == 0) p.prefix[p.num_seqs] = scan.total();
    }
    const long long total = scan.total();
    const long long workers = worker_count(total, max_workers);
    if (total == 0 || w >= workers) return;
    u = share_begin(w, total, workers);
    end = share_begin(w + 1, total, workers);
    if (u >= end) return;
    s = scan.find(u, p.num_seqs, steps_of, first);
  }

  const uint64_t policy = l2_policy_evict_first(), keep = l2_policy_evict_last();
  const int bs = 1 << p.bs_shift, bmask = bs - 1;
  const int ktok = 4 * (g >> 1) + (g & 1);  // this lane's K tokens in a step: ktok, ktok + 2; V: 4t .. 4t + 3
  while (u < end) {
    const int L = checked_len(p.lens, s, p.limit, nullptr);
    const int steps = (L + kStep - 1) / kStep;
    if (steps == 0) {
      ++s;
      continue;
    }
    const int h = static_cast<int>((u - first) / steps);
    int step = static_cast<int>((u - first) - static_cast<long long>(h) * steps);
    const int begin = step;
    const long long left = end - u;
    const int last = left < steps - step ? step + static_cast<int>(left) : steps;  // this piece: [step, last)
    const long long slot = static_cast<long long>(s) * p.kv_heads + h + w;
    const int32_t *table = p.tables + static_cast<size_t>(s) * p.max_blocks;
    const int last_block = (L - 1) >> p.bs_shift;
    auto block_of = [&](int token) {
      const int b = __ldg(table + min(token >> p.bs_shift, last_block));
      if (b >= 0 && b < p.num_blocks) return b;
      record_error(p.err, kErrBlockIndex);
      return 0;
    };
    auto row_of = [&](int block, int token) {
      return (static_cast<size_t>(block) * p.kv_heads + h) * bs + (token & bmask);
    };

    // the query row g, in the order of the K words
    uint32_t qw[QWORDS];
    float c = p.scale_log2;
    if (p.k_head_scale != nullptr) c *= __ldg(p.k_head_scale + h);
    {
      const uint8_t *row = static_cast<const uint8_t *>(p.q) +
                           (static_cast<size_t>(s) * p.q_heads + h * p.G + min(g, p.G - 1)) * (D * 2);
#pragma unroll
      for (int i = 0; i < QWORDS / 4; ++i) {
        const int at = BYTE ? (i / 2) * 128 + t * 32 + (i & 1) * 16 : i * 64 + t * 16;
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(row + at));
        qw[4 * i] = x.x;
        qw[4 * i + 1] = x.y;
        qw[4 * i + 2] = x.z;
        qw[4 * i + 3] = x.w;
      }
      if constexpr (BYTE && QT == kBF16) {  // as fp16, times the row's own power of two
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < QWORDS; ++i) {
          const float2 x = half2_bits_to_float2<kBF16>(qw[i]);
          top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float f = query_factor(top, c);
#pragma unroll
        for (int i = 0; i < QWORDS; ++i) {
          const float2 x = half2_bits_to_float2<kBF16>(qw[i]);
          qw[i] = pack2_rn<kF16>(x.x * f, x.y * f);
        }
        c /= f;
      }
    }
    float acc[ACC][4];
#pragma unroll
    for (int i = 0; i < ACC; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    float m = -INFINITY, l = 0.f;  // m: the maximum less kLift

    uint4 kr[2][KW];
    uint32_t vr[4][VWORDS];
    auto load_k = [&](int tok0, int block) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t *row = p.k + row_of(block, tok0 + ktok + 2 * j) * ROW + t * 16;
#pragma unroll
        for (int i = 0; i < KW; ++i) kr[j][i] = ldg_stream(row + i * 64, policy);
      }
    };
    auto load_v = [&](int tok0, int block) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t *row = p.v + row_of(block, tok0 + 4 * t + j) * ROW;
        if constexpr (VWORDS >= 4) {
#pragma unroll
          for (int i = 0; i < VWORDS / 4; ++i) {
            const uint4 x = ldg_stream(row + i * 128 + g * 16, policy);
            vr[j][4 * i] = x.x;
            vr[j][4 * i + 1] = x.y;
            vr[j][4 * i + 2] = x.z;
            vr[j][4 * i + 3] = x.w;
          }
        } else {
          const uint2 x = ldg_stream2(row + g * 8, policy);
          vr[j][0] = x.x;
          vr[j][1] = x.y;
        }
      }
    };
    int tok0 = step * kStep;
    load_k(tok0, block_of(tok0 + ktok));
    load_v(tok0, block_of(tok0 + 4 * t));
    float *logits = p.logits + (static_cast<size_t>(s) * p.q_heads + h * p.G + min(g, p.G - 1)) * p.width + 4 * t;
    for (; step < last; ++step) {
      const int next = min(step + 1, last - 1) * kStep;
      const int kb = block_of(next + ktok), vb = block_of(next + 4 * t);
      tok0 = step * kStep;
      float sc[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const uint32_t x[4] = {kr[j][i].x, kr[j][i].y, kr[j][i].z, kr[j][i].w};
          if constexpr (BYTE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t lo, hi;
              byte4_to_half2x2<KVT>(x[e], lo, hi);
              mma16816<MT>(sc[j], qw[8 * i + 2 * e], 0u, qw[8 * i + 2 * e + 1], 0u, lo, hi);
            }
          } else {
            mma16816<MT>(sc[j], qw[4 * i], 0u, qw[4 * i + 1], 0u, x[0], x[1]);
            mma16816<MT>(sc[j], qw[4 * i + 2], 0u, qw[4 * i + 3], 0u, x[2], x[3]);
          }
        }
      }
      load_k(next, kb);
      float x[4] = {sc[0][0] * c, sc[0][1] * c, sc[1][0] * c, sc[1][1] * c};  // tokens 4t .. 4t + 3
      const bool tail = tok0 + kStep > L;
      if (tail) {  // the sequence's last step: tokens behind its end weigh nothing, whatever their rows hold
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tok0 + 4 * t + e >= L) {
            x[e] = -INFINITY;
#pragma unroll
            for (int i = 0; i < VWORDS; ++i) vr[e][i] = 0u;
          }
      }
      if (g < p.G) st_global_f4_hint(logits + tok0, make_float4(x[0], x[1], x[2], x[3]), keep);
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const bool grow = mx - m > kLazy + kLift<MT>;  // (a difference: exact where the two are close)
      if (__any_sync(0xffffffffu, grow)) {
        const float next = mx - kLift<MT>, alpha = grow ? exp2_fast(m - next) : 1.f;
        if (grow) m = next;
        l *= alpha;
        const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t), a1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < ACC; ++i) {
          acc[i][0] *= a0;
          acc[i][1] *= a1;
          acc[i][2] *= a0;
          acc[i][3] *= a1;
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[e] = exp2_fast(x[e] - base);
      l += (pr[0] + pr[1]) + (pr[2] + pr[3]);
      const uint32_t b0 = pack2_rn<MT>(pr[0], pr[1]), b1 = pack2_rn<MT>(pr[2], pr[3]);
#pragma unroll
      for (int i = 0; i < VWORDS; ++i) {
        if constexpr (BYTE) {
          uint32_t a[4][2];
#pragma unroll
          for (int e = 0; e < 4; ++e) byte4_to_half2x2<KVT>(vr[e][i], a[e][0], a[e][1]);
#pragma unroll
          for (int f = 0; f < 2; ++f)
            mma16816<MT>(acc[2 * i + f], lows(a[0][f], a[1][f]), highs(a[0][f], a[1][f]), lows(a[2][f], a[3][f]),
                         highs(a[2][f], a[3][f]), b0, b1);
        } else {
          mma16816<MT>(acc[i], lows(vr[0][i], vr[1][i]), highs(vr[0][i], vr[1][i]), lows(vr[2][i], vr[3][i]),
                       highs(vr[2][i], vr[3][i]), b0, b1);
        }
      }
      load_v(next, vb);
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    constexpr int VD = BYTE ? D / 8 : 8;  // consecutive dimensions of a lane
    if (p.whole) {
      const float vs = p.v_head_scale != nullptr ? __ldg(p.v_head_scale + h) : p.v_scale;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (no score above -inf)
      const float i0 = __shfl_sync(0xffffffffu, inv, 8 * t) * vs, i1 = __shfl_sync(0xffffffffu, inv, 8 * t + 4) * vs;
      uint16_t *out = static_cast<uint16_t *>(p.out) + (static_cast<size_t>(s) * p.q_heads + h * p.G + 2 * t) * D;
#pragma unroll
      for (int i = 0; i < ACC; ++i) {
        const int d = (2 * i / VD) * (8 * VD) + g * VD + 2 * i % VD;
        if (2 * t < p.G)
          *reinterpret_cast<uint32_t *>(out + d) = i0 == 0.f ? 0u : pack2_rn<QT>(acc[i][0] * i0, acc[i][2] * i0);
        if (2 * t + 1 < p.G)
          *reinterpret_cast<uint32_t *>(out + D + d) = i1 == 0.f ? 0u : pack2_rn<QT>(acc[i][1] * i1, acc[i][3] * i1);
      }
      __syncwarp();  // the warp's scores are there
      const float base = m == -INFINITY ? 0.f : m;
      const float *x = p.logits + (static_cast<size_t>(s) * p.q_heads + h * p.G) * p.width;
      const size_t at = (static_cast<size_t>(s) * p.kv_heads + h) * p.weights_width;
      float bm[8], bi[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        bm[q] = __shfl_sync(0xffffffffu, base, 4 * q);
        bi[q] = q < p.G ? __shfl_sync(0xffffffffu, inv, 4 * q) : 0.f;
      }
      for (int i = lane; i < L; i += 32) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < p.G) sum += exp2_fast(__ldcg(x + static_cast<size_t>(q) * p.width + i) - bm[q]) * bi[q];
        p.weights_out[at + i] = (p.weights_in == nullptr ? 0.f : p.decay * p.weights_in[at + i]) + sum;
      }
      return;
    }
    // the piece: unnormalised sums with their maximum and total weight
    if (t == 0 && g < p.G) p.part_ml[slot * p.G + g] = make_float2(m, l);
    float *po = p.part_o + slot * p.G * D;
#pragma unroll
    for (int i = 0; i < ACC; ++i) {
      const int d = (2 * i / VD) * (8 * VD) + g * VD + 2 * i % VD;
      if (2 * t < p.G) *reinterpret_cast<float2 *>(po + (2 * t) * D + d) = make_float2(acc[i][0], acc[i][2]);
      if (2 * t + 1 < p.G) *reinterpret_cast<float2 *>(po + (2 * t + 1) * D + d) = make_float2(acc[i][1], acc[i][3]);
    }
    u += last - begin;
    if (u >= first + static_cast<long long>(steps) * p.kv_heads) {
      first += static_cast<long long>(steps) * p.kv_heads;
      ++s;
    }
  }
}

// Adds the tokens' weights and joins the pairs' pieces: the first
// weight_blocks blocks take `chunk` tokens of a pair each, the others write the
// rows of out, TEAM warps a row (four where rows are few), each every TEAM-th
// piece.
template <int QT, int D, int TEAM>
__global__ void __launch_bounds__(kThreads) weigh_finish_kernel(const WeighParams p, int max_workers, int weight_blocks,
                                                                int chunk) {
  constexpr int PER = D / 32;  // dimensions of a lane
  __shared__ float part[TEAM > 1 ? kWarps : 1][D];
  __shared__ float sums[kWarps];
  grid_dependency_wait();
  const long long total = p.prefix[p.num_seqs];
  const long long workers = worker_count(total, max_workers);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) >= weight_blocks) {
    const long long row = (static_cast<long long>(blockIdx.x) - weight_blocks) * (kWarps / TEAM) + warp / TEAM;
    const bool exists = row < static_cast<long long>(p.num_seqs) * p.q_heads;
    const int s = static_cast<int>(row / p.q_heads), hq = static_cast<int>(row % p.q_heads), h = hq / p.G, gq = hq % p.G;
    const int mate = warp % TEAM;
    float o[PER], l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    if (exists) {
      const long long first = p.prefix[s], all = p.prefix[s + 1] - first;
      if (all > 0) {
        const long long steps = all / p.kv_heads, u0 = first + h * steps;
        const long long pair = static_cast<long long>(s) * p.kv_heads + h;
        const long long s0 = pair + share_owner(u0, total, workers);
        const int n = static_cast<int>(pair + share_owner(u0 + steps - 1, total, workers) - s0) + 1;
        const float2 *ml = p.part_ml + s0 * p.G + gq;
        const float *po = p.part_o + (s0 * p.G + gq) * D + lane * PER;
        float m = -INFINITY;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, ml[static_cast<size_t>(i) * p.G].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (m == -INFINITY) m = 0.f;
#pragma unroll 4
        for (int i = mate; i < n; i += TEAM) {
          const float2 a = ml[static_cast<size_t>(i) * p.G];
          const float *x = po + static_cast<size_t>(i) * p.G * D;
          const float f = exp2_fast(a.x - m);
          l += f * a.y;
          if constexpr (PER == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(x);
            o[0] += f * y.x;
            o[1] += f * y.y;
            o[2] += f * y.z;
            o[3] += f * y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2 *>(x);
            o[0] += f * y.x;
            o[1] += f * y.y;
          }
        }
      }
    }
    if constexpr (TEAM > 1) {
#pragma unroll
      for (int e = 0; e < PER; ++e) part[warp][lane * PER + e] = o[e];
      if (lane == 0) sums[warp] = l;
      __syncthreads();
      if (mate > 0) return;
#pragma unroll
      for (int i = 1; i < TEAM; ++i) {
        l += sums[warp + i];
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] += part[warp + i][lane * PER + e];
      }
    }
    if (!exists) return;
    const float vs = p.v_head_scale != nullptr ? __ldg(p.v_head_scale + h) : p.v_scale;
    const float f = l == 0.f ? 0.f : vs / l;  // (no token, or none with a weight)
    uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + static_cast<size_t>(row) * D) +
                    lane * (PER / 2);
#pragma unroll
    for (int e = 0; e < PER; e += 2) out[e / 2] = l == 0.f ? 0u : pack2_rn<QT>(o[e] * f, o[e + 1] * f);
    return;
  }
  const int chunks = (p.limit + chunk - 1) / chunk;
  const long long pair = blockIdx.x / chunks;
  const int s = static_cast<int>(pair / p.kv_heads), h = static_cast<int>(pair - static_cast<long long>(s) * p.kv_heads);
  const long long first = p.prefix[s], all = p.prefix[s + 1] - first;
  if (all == 0) return;
  const int L = __ldg(p.lens + s);
  const int i0 = static_cast<int>(blockIdx.x - pair * chunks) * chunk, i1 = min(L, i0 + chunk);
  if (i0 >= L) return;
  const long long steps = all / p.kv_heads, u0 = first + h * steps;
  const long long s0 = pair + share_owner(u0, total, workers), s1 = pair + share_owner(u0 + steps - 1, total, workers);
  const float *x = p.logits + (static_cast<size_t>(s) * p.q_heads + h * p.G) * p.width;
  const size_t at = static_cast<size_t>(pair) * p.weights_width;
  const float *win = p.weights_in == nullptr ? nullptr : p.weights_in + at;
  float *wout = p.weights_out + at;
  // four tokens a lane (the scores' rows are aligned; the weights' may not
  // be); the first ones are on their way while the pair's sums are joined
  float4 sc[8];
  float before[4];
  auto load = [&](int j) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < p.G) sc[q] = __ldcs(reinterpret_cast<const float4 *>(x + static_cast<size_t>(q) * p.width + j));
#pragma unroll
    for (int e = 0; e < 4; ++e) before[e] = win == nullptr ? 0.f : win[j + e];
  };
  int i = i0 + 128 * warp;
  if (i + 128 <= i1) load(i + 4 * lane);
  // the pair's maximum and total of query lane / 4, four lanes along the pieces
  const int gq = min(lane >> 2, p.G - 1);
  float m = -INFINITY, l = 0.f;
  for (long long j = s0 + (lane & 3); j <= s1; j += 4) {
    const float2 ml = p.part_ml[j * p.G + gq];
    const float top = fmaxf(m, ml.x);
    if (top > -INFINITY) l = l * exp2_fast(m - top) + ml.y * exp2_fast(ml.x - top);
    m = top;
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, d), ol = __shfl_xor_sync(0xffffffffu, l, d);
    const float top = fmaxf(m, om);
    if (top > -INFINITY) l = l * exp2_fast(m - top) + ol * exp2_fast(om - top);
    m = top;
  }
  if (m == -INFINITY) m = 0.f;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float bm[8], bi[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    bm[q] = __shfl_sync(0xffffffffu, m, 4 * q);
    bi[q] = q < p.G ? __shfl_sync(0xffffffffu, inv, 4 * q) : 0.f;
  }
  for (; i + 128 <= i1; i += kThreads * 4) {
    const int j = i + 4 * lane;
    float sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = p.decay * before[e];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < p.G) {
        sum[0] += exp2_fast(sc[q].x - bm[q]) * bi[q];
        sum[1] += exp2_fast(sc[q].y - bm[q]) * bi[q];
        sum[2] += exp2_fast(sc[q].z - bm[q]) * bi[q];
        sum[3] += exp2_fast(sc[q].w - bm[q]) * bi[q];
      }
    if (i + kThreads * 4 + 128 <= i1) load(j + kThreads * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) wout[j + e] = sum[e];
  }
  for (i += lane; i < i1; i += 32) {  // the chunk's last tokens, where they are this warp's
    float sum = win == nullptr ? 0.f : p.decay * win[i];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < p.G) sum += exp2_fast(__ldcs(x + static_cast<size_t>(q) * p.width + i) - bm[q]) * bi[q];
    wout[i] = sum;
  }
}

struct Sizes {
  size_t prefix, ml, o, logits, total;
  int width;
};
bool sizes_of(int S, int Hq, int H, int D, int max_len, Sizes *z) {
  if (S < 0 || Hq <= 0 || H <= 0 || Hq % H || (D != 64 && D != 128) || max_len < 0 || Hq / H > 8) return false;
  if (max_len > INT_MAX - 8192) return false;
  auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
  z->width = (max_len + kStep - 1) / kStep * kStep;
  const size_t G = Hq / H, slots = static_cast<size_t>(S) * H + kMaxWorkers;
  z->prefix = up(8 * (static_cast<size_t>(S) + 1));
  z->ml = up(slots * G * sizeof(float2));
  z->o = up(slots * G * D * sizeof(float));
  z->logits = up(static_cast<size_t>(S) * Hq * z->width * sizeof(float));
  z->total = z->prefix + z->ml + z->o + z->logits;
  return true;
}

template <int QT, int D, int TEAM>
cudaError_t launch_finish(const WeighParams &p, int workers, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int per = kWarps / TEAM;  // rows of a block
  // 2048 tokens a block, more where the bound on the lengths would make many blocks without any
  const long long pairs = static_cast<long long>(p.num_seqs) * p.kv_heads;
  const long long most = pairs >= 16384 ? 1 : 16384 / pairs;  // of a pair
  long long chunk = (p.limit + most - 1) / most;
  chunk = chunk < 2048 ? 2048 : (chunk + 127) / 128 * 128;
  const long long blocks = pairs * ((p.limit + chunk - 1) / chunk);
  cfg.gridDim = dim3(static_cast<unsigned>((p.num_seqs * p.q_heads + per - 1) / per + blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weigh_finish_kernel<QT, D, TEAM>, p, workers, static_cast<int>(blocks),
                            static_cast<int>(chunk));
}

template <int KVT, int QT, int D>
pa_status launch(const WeighParams &p, cudaStream_t stream) {
  DeviceInfo info;
  if (!current_device_info(&info)) return cuda_fail(cudaGetLastError());
  const int blocks = info.sm_count * 3 * kWarps > kMaxWorkers ? kMaxWorkers / kWarps : info.sm_count * 3;
  const int workers = blocks * kWarps;
  if (p.whole) {
    const long long pairs = static_cast<long long>(p.num_seqs) * p.kv_heads;
    weigh_kernel<KVT, QT, D><<<static_cast<unsigned>((pairs + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p, 0);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
  }
  weigh_kernel<KVT, QT, D><<<blocks, kThreads, 0, stream>>>(p, workers);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  // Four warps a row of out or one: one sequence of 131071 tokens, 64/8 heads,
  // 100.5 / 114.5 us, two of 32768 54.8 / 61.6, four 95.5 / 96.6; 16 of 4096
  // (1024 rows) 53.6 / 53.7, 32 (2048 rows) 99.0 / 95.7.
  const long long rows = static_cast<long long>(p.num_seqs) * p.q_heads;
  e = rows <= info.sm_count * 8ll ? launch_finish<QT, D, 4>(p, workers, stream)
                                  : launch_finish<QT, D, 1>(p, workers, stream);
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

template <int KVT, int QT>
pa_status by_dim(int D, const WeighParams &p, cudaStream_t stream) {
  return D == 64 ? launch<KVT, QT, 64>(p, stream) : launch<KVT, QT, 128>(p, stream);
}
template <int KVT>
pa_status by_query(int q_dtype, int D, const WeighParams &p, cudaStream_t stream) {
  return q_dtype == kF16 ? by_dim<KVT, kF16>(D, p, stream) : by_dim<KVT, kBF16>(D, p, stream);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_weights_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                   int32_t head_dim, int32_t max_seq_len) {
  Sizes z;
  return sizes_of(num_seqs, num_q_heads, num_kv_heads, head_dim, max_seq_len, &z) ? z.total : 0;
}

extern "C" pa_status pa_decode_weights(void *out, float *weights_out, const float *weights_in, float decay,
                                       int64_t weights_width, const void *q, int32_t q_dtype, int32_t num_seqs,
                                       int32_t num_q_heads, const void *k_cache, const void *v_cache,
                                       const pa_cache_desc *cache, const int32_t *block_tables,
                                       int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t max_seq_len,
                                       float scale, void *workspace, size_t workspace_bytes, int *device_error,
                                       pa_stream_t stream) {
  if (!valid_cache_desc(cache) || num_seqs < 0 || num_q_heads <= 0 || max_seq_len < 0 || max_blocks_per_seq <= 0 ||
      weights_width < max_seq_len || !isfinite(scale) || !isfinite(decay))
    return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!out || !weights_out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !workspace)
    return PA_ERR_INVALID;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(weights_out) & 3u) || (reinterpret_cast<uintptr_t>(weights_in) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_INVALID;
  if (num_q_heads % cache->kv_heads) return PA_ERR_INVALID;
  const int G = num_q_heads / cache->kv_heads;
  if ((G != 1 && G != 2 && G != 4 && G != 8) || !supported_cache_shape(cache) || cache->dtype == PA_FP4)
    return PA_ERR_UNSUPPORTED;
  const bool byte_codes = cache->dtype >= PA_FP8_E4M3;
  if (byte_codes ? (q_dtype != PA_F16 && q_dtype != PA_BF16) : q_dtype != cache->dtype) return PA_ERR_UNSUPPORTED;
  Sizes z;
  if (!sizes_of(num_seqs, num_q_heads, cache->kv_heads, cache->head_dim, max_seq_len, &z)) return PA_ERR_UNSUPPORTED;
  if (workspace_bytes < z.total) return PA_ERR_INVALID;
  if (static_cast<long long>(num_seqs) * num_q_heads > INT_MAX / 2) return PA_ERR_UNSUPPORTED;  // the grid

  WeighParams p{};
  p.out = out;
  p.q = q;
  p.k = static_cast<const uint8_t *>(k_cache);
  p.v = static_cast<const uint8_t *>(v_cache);
  p.tables = block_tables;
  p.lens = seq_lens;
  p.weights_in = weights_in;
  p.weights_out = weights_out;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.prefix = reinterpret_cast<long long *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + z.prefix);
  p.part_o = reinterpret_cast<float *>(ws + z.prefix + z.ml);
  p.logits = reinterpret_cast<float *>(ws + z.prefix + z.ml + z.o);
  p.num_seqs = num_seqs;
  p.q_heads = num_q_heads;
  p.kv_heads = cache->kv_heads;
  p.G = G;
  p.num_blocks = cache->num_blocks;
  p.bs_shift = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
  p.max_blocks = max_blocks_per_seq;
  const long long held = static_cast<long long>(max_blocks_per_seq) * cache->block_size;
  p.limit = held < max_seq_len ? static_cast<int>(held) : max_seq_len;
  p.width = z.width;
  p.weights_width = weights_width;
  const bool per_head = byte_codes && cache->k_head_scales != nullptr;
  p.scale_log2 = scale * (byte_codes && !per_head ? cache->k_scale : 1.f) * 1.4426950408889634f;
  p.v_scale = byte_codes && !per_head ? cache->v_scale : 1.f;
  p.k_head_scale = per_head ? cache->k_head_scales : nullptr;
  p.v_head_scale = per_head ? cache->v_head_scales : nullptr;
  p.decay = decay;
  p.whole = max_seq_len <= kWholeTokens;
  p.err = device_error;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int D = cache->head_dim;
  switch (cache->dtype) {
    case PA_F16: return by_dim<kF16, kF16>(D, p, st);
    case PA_BF16: return by_dim<kBF16, kBF16>(D, p, st);
    case PA_FP8_E4M3: return by_query<kE4M3>(q_dtype, D, p, st);
    case PA_FP8_E5M2: return by_query<kE5M2>(q_dtype, D, p, st);
    case PA_INT8: return by_query<kI8>(q_dtype, D, p, st);
  }
  return PA_ERR_UNSUPPORTED;
}
