// Equal shares of ragged work.  The sequences' tokens are laid out in one
// line of units (a few tokens of one sequence, times whatever a token is
// repeated for), and worker w of n takes the units [w U / n, (w + 1) U / n):
// every worker has the same work whatever the lengths, and no host plan is
// needed.  A sequence (or a head of it) that several workers share is joined
// from their parts afterwards.
#pragma once

#include "pa_common.cuh"

namespace pa {

// a / b of numbers that mostly fit 32 bits (a 64-bit division is a chain of
// about 100 instructions, and several lie ahead of a join's first loads).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  const unsigned long long x = static_cast<unsigned long long>(a), y = static_cast<unsigned long long>(b);
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return static_cast<long long>(x / y);
}

// First unit of worker w, and the worker that owns unit u.
__device__ __forceinline__ long long share_begin(long long w, long long units, long long workers) {
  return quotient(w * units, workers);
}
__device__ __forceinline__ long long share_owner(long long u, long long units, long long workers) {
  return quotient((u + 1) * workers - 1, units);
}

// A length as the kernels use it: one outside [0, limit] counts as zero.
__device__ __forceinline__ int checked_len(const int32_t *lens, int s, int limit, int *err) {
  const int L = __ldg(lens + s);
  if (L >= 0 && L <= limit) return L;
  record_error(err, kErrSeqLen);
  return 0;
}

// The units of all sequences, found by the block's first THREADS threads:
// each sums a run of sequences, the runs' sums are scanned in shared memory.
template <int THREADS>
struct ShareScan {
  static_assert((THREADS & (THREADS - 1)) == 0, "a power of two");
  long long base[THREADS + 1];  // units before thread t's run; the total
  static __device__ __forceinline__ int run(int num_seqs) { return (num_seqs + THREADS - 1) / THREADS; }

  // units_of(s): the units of sequence s.  All threads of the block (the
  // others only keep step); ends with a barrier.
  template <typename F>
  __device__ __forceinline__ void scan(int num_seqs, F units_of) {
    const int n = run(num_seqs), t = threadIdx.x;
    if (t < THREADS) {
      long long sum = 0;
      for (int s = t * n; s < min(num_seqs, (t + 1) * n); ++s) sum += units_of(s);
      base[t + 1] = sum;
      if (t == 0) base[0] = 0;
    }
    __syncthreads();
    for (int d = 1; d < THREADS; d <<= 1) {
      const long long x = t < THREADS && t >= d ? base[t + 1 - d] : 0;
      __syncthreads();
      if (t < THREADS) base[t + 1] += x;
      __syncthreads();
    }
  }
  __device__ __forceinline__ long long total() const { return base[THREADS]; }

  // The sequence that holds unit u < total(), and its first unit.
  template <typename F>
  __device__ __forceinline__ int find(long long u, int num_seqs, F units_of, long long &first) const {
    int lo = 0, hi = THREADS - 1;  // the last run whose base is at or before u and that is not empty
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (base[mid + 1] <= u) lo = mid + 1;
      else hi = mid;
    }
    first = base[lo];
    int s = lo * run(num_seqs);
    for (; s < num_seqs - 1; ++s) {
      const long long n = units_of(s);
      if (u < first + n) break;
      first += n;
    }
    return s;
  }
};

}  // namespace pa
