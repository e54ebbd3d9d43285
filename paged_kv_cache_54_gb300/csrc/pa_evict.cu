// pa_evict_tokens: each head's most heavily weighted tokens, and the most
// recent ones, moved to new blocks in their order.
//
// Select: one block a (sequence, KV head) pair.  The weights become unsigned
// keys that ascend with them; a radix selection in three digits (11, 11 and
// 10 bits) finds the k-th largest key T and how many of the keys equal to it
// are kept.  The weights are read three times: for the first digit's
// histogram; to gather the keys of T's bin, on which the other digits are
// found; and to place the kept tokens in order (keys above T, the first of
// those equal to it, and the recent ones).  Where the bin holds more than fits
// (many equal weights), the other digits read all weights too.  Bound by
// issued instructions and the chain of steps between the passes: 256 pairs of
// 4096..16384 tokens take 29 us (a pass more for each of the other digits: 32).
// Move: rows copied from their old slots to their new ones, every warp with
// four accesses of K and four of V in flight.  The selection leaves slots, not
// tokens: looking the blocks up here, a load more ahead of the rows, takes 15
// us more.  4096 of those tokens a pair, 256-byte rows: 1.08 GB, 162 us at the
// measured copy rate, in 166.
#include <limits.h>

#include "pa_common.cuh"
#include "pa_host.h"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kGathered = 4096;  // keys of a bin that fit
constexpr int kMoveThreads = 256;

struct EvictParams {
  const uint8_t *k, *v;
  uint8_t *k_out, *v_out;  // the same caches
  const int32_t *tables, *lens, *new_tables;
  int32_t *new_lens;
  const float *weights;
  float *new_weights;
  int32_t *list;  // [pairs, budget] the kept tokens' slots, -1 for a bad block
  int num_seqs, kv_heads, num_blocks, bs_shift, max_blocks, max_new_blocks, budget, recent, limit;
  long long width, new_width;
  int *err;
};

// Ascends with the weight; a NaN lies below every number, -0 equals 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);  // (-0 + 0 = 0)
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive sum of x over the block's threads; `tmp` holds kSelWarps ints.
__device__ __forceinline__ int block_exclusive(int x, int *tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = y;
  __syncthreads();
  if (warp == 0) {
    int v = lane < kSelWarps ? tmp[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += z;
    }
    if (lane < kSelWarps) tmp[lane] = v;
  }
  __syncthreads();
  return y - x + (warp > 0 ? tmp[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[kBins];
  __shared__ int tmp[kSelWarps];
  __shared__ int above[kSelWarps], equal[kSelWarps];
  __shared__ uint32_t bin_key[kGathered];
  __shared__ uint8_t bin_warp[kGathered];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_gathered;
  launch_dependents();
  const long long pair = blockIdx.x;
  const int s = static_cast<int>(pair / p.kv_heads), h = static_cast<int>(pair % p.kv_heads);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = __ldg(p.lens + s);
  if (L < 0 || L > p.limit) {
    if (tid == 0) {
      record_error(p.err, kErrSeqLen);
      if (h == 0) p.new_lens[s] = 0;
    }
    return;
  }
  const int B = min(L, p.budget), r = min(p.recent, B), n = L - r, k = B - r;
  if (tid == 0 && h == 0) p.new_lens[s] = B;
  const float *w = p.weights + pair * p.width;
  // a warp has a run of tokens, a lane every 32nd of it; f(first token, keys)
  // for four steps of the warp at a time, in order
  const int run = (L + kSelThreads - 1) / kSelThreads * 32;
  const int i0 = min(warp * run, L), i1 = min(i0 + run, L);
  constexpr int kBatch = 4;
  auto each = [&](auto f) {
    for (int base = i0; base < i1; base += 32 * kBatch) {
      uint32_t x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = base + 32 * j + lane;
        x[j] = i < i1 ? __float_as_uint(__ldg(w + i)) : 0u;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) x[j] = weight_key(__uint_as_float(x[j]));
      f(base, x);
    }
  };
  // the digit, from the top, in which the need-th key lies (all threads; a
  // thread has four bins, the highest first)
  uint32_t prefix = 0;
  int need = k;  // of the keys that share the prefix, how many are kept
  auto pick = [&](int shift) {
    constexpr int kOwn = kBins / kSelThreads;
    const int b0 = kBins - 1 - kOwn * tid;
    int c[kOwn], sum = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) sum += c[j] = hist[b0 - j];
    int before = block_exclusive(sum, tmp);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      if (before < need && need <= before + c[j]) {
        s_prefix = prefix | (static_cast<uint32_t>(b0 - j) << shift);
        s_need = need - before;
      }
      before += c[j];
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
  };
  int gt = 0, eq = 0;  // of the warp's candidates: surely kept, and equal to T
  const int end = min(i1, n);
  if (k > 0 && k < n) {
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    if (tid == 0) s_gathered = 0;
    if (lane == 0) above[warp] = equal[warp] = 0;
    __syncthreads();
    each([&](int base, const uint32_t (&x)[kBatch]) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (base + 32 * j + lane < end) atomicAdd(&hist[x[j] >> 21], 1);
    });
    __syncthreads();
    pick(21);
    // the bin's keys, and how many lie above it
    each([&](int base, const uint32_t (&x)[kBatch]) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const bool in = base + 32 * j + lane < end;
        const uint32_t digit = x[j] >> 21;
        gt += in && digit > (prefix >> 21);
        const bool here = in && digit == (prefix >> 21);
        const unsigned mask = __ballot_sync(0xffffffffu, here);
        if (mask != 0) {
          int at = 0;
          if (lane == 0) at = atomicAdd(&s_gathered, __popc(mask));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1u));
          if (here && at < kGathered) {
            bin_key[at] = x[j];
            bin_warp[at] = static_cast<uint8_t>(warp);
          }
        }
      }
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    __syncthreads();
    const int gathered = s_gathered;
    for (int level = 1; level < 3; ++level) {
      const int shift = level == 1 ? 10 : 0;
      const uint32_t mask = level == 1 ? 0xffe00000u : 0xfffffc00u, digit = level == 1 ? 0x7ffu : 0x3ffu;
      if (gathered <= kGathered) {
        for (int i = tid; i < gathered; i += kSelThreads)
          if ((bin_key[i] & mask) == prefix) atomicAdd(&hist[(bin_key[i] >> shift) & digit], 1);
      } else {
        each([&](int base, const uint32_t (&x)[kBatch]) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (base + 32 * j + lane < end && (x[j] & mask) == prefix) atomicAdd(&hist[(x[j] >> shift) & digit], 1);
        });
      }
      __syncthreads();
      pick(shift);
    }
    if (gathered <= kGathered) {
      for (int i = tid; i < gathered; i += kSelThreads) {
        if (bin_key[i] > prefix) atomicAdd(&above[bin_warp[i]], 1);
        if (bin_key[i] == prefix) atomicAdd(&equal[bin_warp[i]], 1);
      }
    } else {
      int g = 0;
      each([&](int base, const uint32_t (&x)[kBatch]) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const bool in = base + 32 * j + lane < end;
          g += in && x[j] > prefix && (x[j] >> 21) == (prefix >> 21);
          eq += in && x[j] == prefix;
        }
      });
      g = __reduce_add_sync(0xffffffffu, g);
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        above[warp] = g;
        equal[warp] = eq;
      }
    }
    __syncthreads();
    gt += above[warp];
    eq = equal[warp];
  } else {
    // every candidate is kept, or none: no key is T
    prefix = 0xffffffffu;
    need = 0;
    gt = k > 0 ? max(end - i0, 0) : 0;
    eq = 0;
  }
  __syncthreads();
  if (lane == 0) {
    above[warp] = gt + max(i1 - max(i0, n), 0);  // and the recent ones
    equal[warp] = eq;
  }
  __syncthreads();
  const int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? above[lane & (kSelWarps - 1)] : 0);
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? equal[lane & (kSelWarps - 1)] : 0);
  int at = gt0 + min(eq0, need);
  const int from = k >= n ? 0 : n;  // tokens from here on are kept whatever their weight
  int32_t *list = p.list + pair * p.budget;
  float *new_weights = p.new_weights + pair * p.new_width;
  const int32_t *table = p.tables + static_cast<size_t>(s) * p.max_blocks;
  const int bmask = (1 << p.bs_shift) - 1;
  each([&](int base, const uint32_t (&x)[kBatch]) {
    const unsigned below = (1u << lane) - 1u;
    int to[kBatch], block[kBatch];
    float weight[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = base + 32 * j + lane;
      const bool sure = i < i1 && (i >= from || x[j] > prefix);
      const bool tie = i < i1 && !sure && x[j] == prefix;
      const unsigned ties = __ballot_sync(0xffffffffu, tie);
      const bool keep = sure || (tie && eq0 + __popc(ties & below) < need);
      const unsigned kept = __ballot_sync(0xffffffffu, keep);
      to[j] = keep ? at + __popc(kept & below) : -1;
      at += __popc(kept);
      eq0 += __popc(ties);
    }
    // (the kept tokens' blocks and weights are on their way together)
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = base + 32 * j + lane;
      block[j] = to[j] >= 0 ? __ldg(table + (i >> p.bs_shift)) : 0;
      weight[j] = to[j] >= 0 ? __ldg(w + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (to[j] >= 0) {
        const bool ok = block[j] >= 0 && block[j] < p.num_blocks;
        if (!ok) record_error(p.err, kErrBlockIndex);
        list[to[j]] = ok ? (block[j] << p.bs_shift) + ((base + 32 * j + lane) & bmask) : -1;
        new_weights[to[j]] = weight[j];
      }
  });
}

template <int ROW>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, long long items, int per_pair) {
  constexpr int LPR = ROW / 16;  // lanes of a row
  constexpr int RPI = 32 / LPR;  // rows of one access
  constexpr int U = 4;           // accesses of K and of V in flight
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
  const int bmask = (1 << p.bs_shift) - 1;
  const int col = (lane % LPR) * 16;
  for (long long i = blockIdx.x * static_cast<long long>(kMoveThreads / 32) + (threadIdx.x >> 5); i < items; i += warps) {
    const long long pair = i / per_pair;
    const int first = static_cast<int>(i - pair * per_pair) * (U * RPI) + lane / LPR;
    const int s = static_cast<int>(pair / p.kv_heads), h = static_cast<int>(pair - static_cast<long long>(s) * p.kv_heads);
    const int count = p.new_lens[s];
    uint32_t from[U], to[U];  // (rows of the caches, fewer than 2^31)
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = first + u * RPI;
      ok[u] = row < count;
      from[u] = to[u] = 0;
      if (ok[u]) {
        const int slot = p.list[pair * p.budget + row];
        const int block = __ldg(p.new_tables + static_cast<size_t>(s) * p.max_new_blocks + (row >> p.bs_shift));
        ok[u] = slot >= 0;
        if (block < 0 || block >= p.num_blocks) {
          record_error(p.err, kErrBlockIndex);
          ok[u] = false;
        }
        if (ok[u]) {
          from[u] = ((static_cast<uint32_t>(slot >> p.bs_shift) * p.kv_heads + h) << p.bs_shift) + (slot & bmask);
          to[u] = ((static_cast<uint32_t>(block) * p.kv_heads + h) << p.bs_shift) + (row & bmask);
        }
      }
    }
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ok[u]) {
        a[u] = *reinterpret_cast<const uint4 *>(p.k + static_cast<size_t>(from[u]) * ROW + col);
        b[u] = *reinterpret_cast<const uint4 *>(p.v + static_cast<size_t>(from[u]) * ROW + col);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ok[u]) {
        *reinterpret_cast<uint4 *>(p.k_out + static_cast<size_t>(to[u]) * ROW + col) = a[u];
        *reinterpret_cast<uint4 *>(p.v_out + static_cast<size_t>(to[u]) * ROW + col) = b[u];
      }
  }
}

bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < a_bytes : x - y < b_bytes;
}

template <int ROW>
pa_status launch_move(const EvictParams &p, cudaStream_t stream) {
  constexpr int rows = 4 * (32 / (ROW / 16));  // of a warp's step
  const int per_pair = (p.budget + rows - 1) / rows;
  const long long items = static_cast<long long>(p.num_seqs) * p.kv_heads * per_pair;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_for(items * 32, kMoveThreads));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_move_kernel<ROW>, p, items, per_pair);
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_evict_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t budget) {
  if (num_seqs < 0 || num_kv_heads <= 0 || budget < 0) return 0;
  return static_cast<size_t>(num_seqs) * num_kv_heads * budget * sizeof(int32_t) + 256;
}

extern "C" pa_status pa_evict_tokens(void *k_cache, void *v_cache, const pa_cache_desc *cache,
                                     const int32_t *block_tables, int32_t num_seqs, int32_t max_blocks_per_seq,
                                     const int32_t *seq_lens, const float *weights, int64_t weights_width,
                                     const int32_t *new_tables, int32_t max_new_blocks, int32_t *new_lens,
                                     float *new_weights, int64_t new_width, int32_t budget, int32_t recent,
                                     void *workspace, size_t workspace_bytes, int *device_error, pa_stream_t stream) {
  if (!valid_cache_desc(cache) || num_seqs < 0 || max_blocks_per_seq <= 0 || max_new_blocks <= 0 || budget <= 0 ||
      recent < 0 || recent > budget || weights_width < 0 || new_width < budget)
    return PA_ERR_INVALID;
  if (static_cast<long long>(max_new_blocks) * cache->block_size < budget) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !seq_lens || !weights || !new_tables || !new_lens || !new_weights ||
      !workspace)
    return PA_ERR_INVALID;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(new_tables) |
        reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(new_weights)) & 3u))
    return PA_ERR_INVALID;
  if (!supported_cache_shape(cache) || cache->dtype == PA_FP4) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(cache->num_blocks) * cache->block_size * cache->kv_heads > INT_MAX)
    return PA_ERR_UNSUPPORTED;  // 32-bit rows
  if (static_cast<long long>(num_seqs) * cache->kv_heads > INT_MAX) return PA_ERR_UNSUPPORTED;             // the grid
  if (workspace_bytes < pa_evict_workspace_size(num_seqs, cache->kv_heads, budget)) return PA_ERR_INVALID;
  // a block writes its results while others still read the lengths and the weights
  const size_t lens_bytes = static_cast<size_t>(num_seqs) * sizeof(int32_t), row = lens_bytes * cache->kv_heads;
  if (overlap(new_lens, lens_bytes, seq_lens, lens_bytes) ||
      overlap(new_weights, row * new_width, weights, row * weights_width))
    return PA_ERR_INVALID;
  EvictParams p{};
  p.k = p.k_out = static_cast<uint8_t *>(k_cache);
  p.v = p.v_out = static_cast<uint8_t *>(v_cache);
  p.tables = block_tables;
  p.lens = seq_lens;
  p.new_tables = new_tables;
  p.new_lens = new_lens;
  p.weights = weights;
  p.new_weights = new_weights;
  p.list = static_cast<int32_t *>(workspace);
  p.num_seqs = num_seqs;
  p.kv_heads = cache->kv_heads;
  p.num_blocks = cache->num_blocks;
  p.bs_shift = cache->block_size == 8 ? 3 : cache->block_size == 16 ? 4 : 5;
  p.max_blocks = max_blocks_per_seq;
  p.max_new_blocks = max_new_blocks;
  p.budget = budget;
  p.recent = recent;
  long long limit = static_cast<long long>(max_blocks_per_seq) * cache->block_size;
  if (weights_width < limit) limit = weights_width;
  p.limit = limit < INT_MAX / 2 ? static_cast<int>(limit) : INT_MAX / 2;  // (steps past the end must not wrap)
  p.width = weights_width;
  p.new_width = new_width;
  p.err = device_error;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  evict_select_kernel<<<num_seqs * cache->kv_heads, kSelThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  switch (cache->head_dim * (cache->dtype >= PA_FP8_E4M3 ? 1 : 2)) {
    case 64: return launch_move<64>(p, st);
    case 128: return launch_move<128>(p, st);
  }
  return launch_move<256>(p, st);
}
