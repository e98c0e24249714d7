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

// Counts `key` in hist if it matches `prefix` above the pass's digit; a whole
// warp calls it.  Equal weights (zeros, ties) would serialise on one bin: a
// warp whose counted lanes all share one bin adds them in one atomic.
__device__ __forceinline__ void count_key(int* hist, uint32_t key, uint32_t prefix, int pass, bool live) {
  const bool in = live && (key & above_mask(pass)) == prefix;
  const uint32_t vote = __ballot_sync(0xffffffffu, in);
  if (vote == 0) return;
  const uint32_t bin = (key >> digit_shift(pass)) & digit_mask(pass);
  const uint32_t lead_bin = __shfl_sync(0xffffffffu, bin, __ffs(vote) - 1);
  if (__all_sync(0xffffffffu, !in || bin == lead_bin)) {
    if ((threadIdx.x & 31) == static_cast<unsigned>(__ffs(vote) - 1)) atomicAdd(&hist[bin], __popc(vote));
  } else if (in) {
    atomicAdd(&hist[bin], 1);
  }
}

struct BinResult {
  int bin;        // the bin of the want-th largest key, bins counted from the top
  int above;      // keys in higher bins
  int own_above;  // of this block's own histogram: keys in higher bins, and in the bin
  int own_in;
};

// find_bin for a histogram spread over several blocks: total(bin) gives a bin's
// sum over all of them, own[] is this block's share.  Every thread of the block
// (kThreads, a multiple of 32 that divides kBins) calls it.  tmp: 2 *
// kThreads / 32 + 4 ints of shared memory.
template <int kThreads, class TotalFn>
__device__ __forceinline__ BinResult find_bin(int want, TotalFn total, const int* own, int* tmp) {
  constexpr int kPer = kBins / kThreads, kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int top = kBins - 1 - kPer * tid;  // thread t holds bins top, top - 1, ...
  int c[kPer], o[kPer], sum = 0, osum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c[i] = total(top - i);
    o[i] = own[top - i];
    sum += c[i];
    osum += o[i];
  }
  int incl = sum, oincl = osum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off), ov = __shfl_up_sync(0xffffffffu, oincl, off);
    if (lane >= off) {
      incl += v;
      oincl += ov;
    }
  }
  if (lane == 31) {
    tmp[warp] = incl;
    tmp[kWarps + warp] = oincl;
  }
  __syncthreads();
  // every warp sums the warps before it
  int w = lane < kWarps && lane < warp ? tmp[lane] : 0, ow = lane < kWarps && lane < warp ? tmp[kWarps + lane] : 0;
  int before = incl - sum + __reduce_add_sync(0xffffffffu, w);
  int obefore = oincl - osum + __reduce_add_sync(0xffffffffu, ow);
  int* res = tmp + 2 * kWarps;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before < want && want <= before + c[i]) {
      res[0] = top - i;
      res[1] = before;
      res[2] = obefore;
      res[3] = o[i];
    }
    before += c[i];
    obefore += o[i];
  }
  __syncthreads();
  BinResult r{res[0], res[1], res[2], res[3]};
  __syncthreads();
  return r;
}

}  // namespace ddt
