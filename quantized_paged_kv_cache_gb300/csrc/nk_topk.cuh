// nk_topk.cuh -- the `need` largest of n keys, by one block.
//
// Keys are whole 64-bit numbers (ordered images of scores), so the choice is
// exact; of equal keys the lowest index is taken. The block finds the threshold
// (kt, it) with exactly `need` elements above it, where element i is above when
// key(i) > kt or key(i) == kt and i <= it; the caller then takes those in one
// ordered pass.
//
// Each round counts the keys of the range that is still in doubt in 2,048 equal
// bins and keeps the bin that the threshold falls in. Scores of one row lie
// within a few binades, so the first round leaves a handful of keys, which are
// ranked against each other; a range spread over all exponents takes six rounds
// at most, eleven bits each.
#pragma once

#include <stdint.h>

namespace nk {

// Image of a double that is not NaN whose order as a whole number is its order.
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

constexpr int kTopBins = 2048;
constexpr int kTopList = 64;

template <int NTH>
struct TopSmem {
  unsigned hist[kTopBins];
  uint64_t list_key[kTopList];
  int list_idx[kTopList];
  uint64_t lo[NTH / 32], hi[NTH / 32];
  int warp[NTH / 32];
  int bin, above, in_bin, count, it;
  uint64_t kt;
};

// Exclusive sum of v over the block; `total` is the sum. Two barriers.
template <int NTH>
__device__ __forceinline__ int block_exclusive(int v, int* warp_tot, int& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // (an earlier call's readers are done)
  if (lane == 31) warp_tot[wid] = incl;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < NTH / 32; ++w) {
    const int x = warp_tot[w];
    if (w < wid) base += x;
    sum += x;
  }
  total = sum;
  return base + incl - v;
}

// A thread's run of elements in the ordered passes: an odd number of 8-byte
// keys, so that the threads' reads of shared memory hit distinct banks.
template <int NTH>
__device__ __forceinline__ int top_run(int n) {
  return ((n + NTH - 1) / NTH) | 1;
}

// Bin width of a round, as a shift, for keys between lo and hi.
__device__ __forceinline__ int top_shift(uint64_t lo, uint64_t hi) {
  const int bits = 64 - __clzll((long long)(hi - lo));
  return bits > 11 ? bits - 11 : 0;
}

// 1 <= need <= n; [klo, khi] must hold every key. `counted`: sm.hist already holds
// the first round's counts (and sm.count 0). Called by all NTH threads; ends with
// a barrier.
template <int NTH, class Key>
__device__ void block_threshold(const Key& key, int n, int need, uint64_t klo, uint64_t khi, TopSmem<NTH>& sm,
                                uint64_t& kt, int& it, bool counted = false) {
  const int tid = threadIdx.x;
  static_assert(kTopBins % NTH == 0, "whole bins per thread");
  constexpr int BPT = kTopBins / NTH;
  uint64_t lo = klo, hi = khi;
  for (;;) {
    const int shift = top_shift(lo, hi);
    if (!counted) {
#pragma unroll
      for (int i = 0; i < BPT; ++i) sm.hist[tid + i * NTH] = 0;
      if (tid == 0) sm.count = 0;
      __syncthreads();
      for (int i = tid; i < n; i += NTH) {
        const uint64_t k = key(i);
        if (k >= lo && k <= hi) atomicAdd(&sm.hist[(int)((k - lo) >> shift)], 1u);
      }
      __syncthreads();
    }
    counted = false;
    // bins from the top: thread t holds bins kTopBins - 1 - t * BPT downwards
    int c[BPT], sum = 0;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      c[i] = (int)sm.hist[kTopBins - 1 - tid * BPT - i];
      sum += c[i];
    }
    int total;
    int run = block_exclusive<NTH>(sum, sm.warp, total);
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      if (run < need && run + c[i] >= need) {  // (of one thread, once)
        sm.bin = kTopBins - 1 - tid * BPT - i;
        sm.above = run;
        sm.in_bin = c[i];
      }
      run += c[i];
    }
    __syncthreads();
    need -= sm.above;
    const int in_bin = sm.in_bin;
    const uint64_t width = (uint64_t)1 << shift;
    lo += (uint64_t)sm.bin << shift;
    if (hi - lo >= width) hi = lo + width - 1;
    if (need == in_bin) {  // the whole bin
      kt = lo;
      it = 0x7fffffff;
      break;
    }
    if (shift == 0) {  // equal keys: the first `need` of them
      const int per = top_run<NTH>(n), a = tid * per, e = a + per < n ? a + per : n;
      int mine = 0;
      for (int i = a; i < e; ++i) mine += key(i) == lo;
      int before = block_exclusive<NTH>(mine, sm.warp, total);
      if (before < need && before + mine >= need) {
        int i = a;
        for (;; ++i) {
          before += key(i) == lo;
          if (before == need) break;
        }
        sm.it = i;
      }
      __syncthreads();
      kt = lo;
      it = sm.it;
      break;
    }
    if (in_bin <= kTopList) {  // a few: each is ranked against the others
      for (int i = tid; i < n; i += NTH) {
        const uint64_t k = key(i);
        if (k >= lo && k <= hi) {
          const int at = atomicAdd(&sm.count, 1);
          sm.list_key[at] = k;
          sm.list_idx[at] = i;
        }
      }
      __syncthreads();
      if (tid < in_bin) {
        const uint64_t k = sm.list_key[tid];
        const int i = sm.list_idx[tid];
        int rank = 0;
        for (int j = 0; j < in_bin; ++j) {
          const uint64_t kj = sm.list_key[j];
          rank += kj > k || (kj == k && sm.list_idx[j] < i);
        }
        if (rank == need - 1) {
          sm.kt = k;
          sm.it = i;
        }
      }
      __syncthreads();
      kt = sm.kt;
      it = sm.it;
      break;
    }
    __syncthreads();
  }
  __syncthreads();
}

// Smallest and largest of the block's keys: each thread's own into shared memory by
// warps (top_range), and after a barrier those of all (range_of).
template <int NTH>
__device__ __forceinline__ void top_range(uint64_t lo, uint64_t hi, TopSmem<NTH>& sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t l2 = __shfl_xor_sync(0xffffffffu, lo, o), h2 = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = l2 < lo ? l2 : lo;
    hi = h2 > hi ? h2 : hi;
  }
  if ((threadIdx.x & 31) == 0) {
    sm.lo[threadIdx.x >> 5] = lo;
    sm.hi[threadIdx.x >> 5] = hi;
  }
}
template <int NTH>
__device__ __forceinline__ void range_of(uint64_t& lo, uint64_t& hi, const TopSmem<NTH>& sm) {
#pragma unroll
  for (int w = 0; w < NTH / 32; ++w) {
    lo = sm.lo[w] < lo ? sm.lo[w] : lo;
    hi = sm.hi[w] > hi ? sm.hi[w] : hi;
  }
}

// The same of n >= 1 keys. Ends with a barrier.
template <int NTH, class Key>
__device__ void block_range(const Key& key, int n, TopSmem<NTH>& sm, uint64_t& klo, uint64_t& khi) {
  uint64_t lo = ~0ull, hi = 0;
  for (int i = threadIdx.x; i < n; i += NTH) {
    const uint64_t k = key(i);
    lo = k < lo ? k : lo;
    hi = k > hi ? k : hi;
  }
  top_range(lo, hi, sm);
  __syncthreads();
  range_of(lo, hi, sm);
  klo = lo;
  khi = hi;
  __syncthreads();
}

}  // namespace nk
