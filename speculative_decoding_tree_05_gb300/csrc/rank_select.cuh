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

// Counts `key` in hist if it matches `prefix` above the pass's digit.  (Adding
// the constant 1 to shared memory, the hardware takes a warp's equal bins in one go.)
__device__ __forceinline__ void count_key(int* hist, uint32_t key, uint32_t prefix, int pass) {
  if ((key & above_mask(pass)) == prefix) atomicAdd(&hist[(key >> digit_shift(pass)) & digit_mask(pass)], 1);
}

// The bin of the want-th largest key (want >= 1), bins counted from the top, and
// the keys in higher bins.  Every thread of the block (kThreads, a multiple of
// 32 that divides kBins) calls it.  tmp: kThreads / 32 + 2 ints of shared memory.
template <int kThreads>
__device__ __forceinline__ int2 find_bin(int want, const int* hist, int* tmp) {
  constexpr int kPer = kBins / kThreads, kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int top = kBins - 1 - kPer * tid;  // thread t holds bins top, top - 1, ...
  int c[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c[i] = hist[top - i];
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
  // every warp sums the warps before it
  int before = incl - sum + __reduce_add_sync(0xffffffffu, lane < kWarps && lane < warp ? tmp[lane] : 0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before < want && want <= before + c[i]) {
      tmp[kWarps] = top - i;
      tmp[kWarps + 1] = before;
    }
    before += c[i];
  }
  __syncthreads();
  return make_int2(tmp[kWarps], tmp[kWarps + 1]);
}

// Ordered emission.  A warp owns a run of consecutive positions and classes each
// (2: kept, 1: tied at the last weight kept, 0: not kept).
struct WarpRun {
  int begin, end;  // positions
};
__device__ __forceinline__ WarpRun warp_run(int begin, int end, int warps, int warp) {
  const int per = ((end - begin + warps - 1) / warps + 31) / 32 * 32;
  WarpRun r;
  r.begin = min(end, begin + warp * per);
  r.end = min(end, r.begin + per);
  return r;
}
// Kept and tied positions of a run.
template <class KlassFn>
__device__ __forceinline__ int2 count_run(WarpRun r, KlassFn klass) {
  const int lane = threadIdx.x & 31;
  int g = 0, e = 0;
#pragma unroll 4
  for (int i0 = r.begin; i0 < r.end; i0 += 32) {
    const int c = i0 + lane < r.end ? klass(i0 + lane) : 0;
    g += __popc(__ballot_sync(0xffffffffu, c == 2));
    e += __popc(__ballot_sync(0xffffffffu, c == 1));
  }
  return make_int2(g, e);
}
// emit(position, kept, rank among the kept positions before it) for a run, with
// g kept and e tied positions before the run, of which `ties` in all are kept.
template <class KlassFn, class EmitFn>
__device__ __forceinline__ void emit_run(WarpRun r, int g, int e, int ties, KlassFn klass, EmitFn emit) {
  const int lane = threadIdx.x & 31;
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 4
  for (int i0 = r.begin; i0 < r.end; i0 += 32) {
    const int i = i0 + lane;
    const int c = i < r.end ? klass(i) : 0;
    const uint32_t mg = __ballot_sync(0xffffffffu, c == 2), me = __ballot_sync(0xffffffffu, c == 1);
    const int eb = e + __popc(me & lt);
    if (i < r.end) emit(i, c == 2 || (c == 1 && eb < ties), g + __popc(mg & lt) + min(eb, ties));
    g += __popc(mg);
    e += __popc(me);
  }
}

}  // namespace ddt
