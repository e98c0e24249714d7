// rank_select.cuh -- the n-th largest of a set of 32-bit keys by digits, most
// significant first (11, 11 and 10 bits): one histogram of the keys that match
// the digits found so far per pass, then the digit whose bin holds the rank.
// Ordering by an unsigned image of a float (order_key_bits) makes ties exact.
#pragma once
#include <cuda_runtime.h>
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace ddt {

constexpr int kBins = 2048;
constexpr int kDigits = 3;
__host__ __device__ constexpr int digit_shift(int pass) { return pass == 0 ? 21 : (pass == 1 ? 10 : 0); }
__host__ __device__ constexpr uint32_t digit_mask(int pass) { return pass == 2 ? 0x3ffu : 0x7ffu; }
// the bits above a pass's digit, which a key must share to be counted in it
__host__ __device__ constexpr uint32_t above_mask(int pass) {
  return pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
}

__device__ __forceinline__ uint32_t order_key(float w) { return order_key_bits(__float_as_uint(w)); }

// Counts `key` in hist if it matches `prefix` above the pass's digit.  Lanes
// that count the same bin are added up first: weights crowd into few bins.
__device__ __forceinline__ void count_key(int* hist, uint32_t key, uint32_t prefix, int pass, bool live) {
  const bool in = live && (key & above_mask(pass)) == prefix;
  const uint32_t bin = in ? (key >> digit_shift(pass)) & digit_mask(pass) : 0xffffffffu;
  const uint32_t same = __match_any_sync(0xffffffffu, bin);
  if (in && (threadIdx.x & 31) == static_cast<unsigned>(__ffs(same) - 1)) atomicAdd(&hist[bin], __popc(same));
}

// The bin of the want-th largest key (want >= 1), bins counted from the top:
// returns the bin and the keys in higher bins.  count(bin) gives a bin's
// total; every thread of the block (kThreads of them, a multiple of 32 that
// divides kBins) calls this.  tmp: kThreads / 32 + 2 ints of shared memory.
template <int kThreads, class CountFn>
__device__ __forceinline__ void find_bin(int want, CountFn count, int* tmp, int* bin, int* above) {
  constexpr int kPer = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int c[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {  // thread t holds bins kBins - 1 - kPer t downwards
    c[i] = count(kBins - 1 - kPer * tid - i);
    sum += c[i];
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) tmp[warp] = incl;
  __syncthreads();
  int before = incl - sum;
  for (int w = 0; w < warp; ++w) before += tmp[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before < want && want <= before + c[i]) {
      tmp[kThreads / 32] = kBins - 1 - kPer * tid - i;
      tmp[kThreads / 32 + 1] = before;
    }
    before += c[i];
  }
  __syncthreads();
  *bin = tmp[kThreads / 32];
  *above = tmp[kThreads / 32 + 1];
  __syncthreads();
}

}  // namespace ddt
