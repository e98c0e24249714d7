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
// the keys in higher bins and in it; total(bin) is a bin's count.  Every thread of the block (kThreads, a multiple of
// 32 that divides kBins) calls it.  tmp: kThreads / 32 + 3 ints of shared memory.
template <int kThreads, class TotalFn>
__device__ __forceinline__ int3 find_bin(int want, TotalFn total, int* tmp) {
  constexpr int kPer = kBins / kThreads, kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int top = kBins - 1 - kPer * tid;  // thread t holds bins top, top - 1, ...
  int c[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c[i] = total(top - i);
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
      tmp[kWarps + 2] = c[i];
    }
    before += c[i];
  }
  __syncthreads();
  return make_int3(tmp[kWarps], tmp[kWarps + 1], tmp[kWarps + 2]);
}

// One digit further: T gets the bin's digit, want becomes the rank within it.
// True when the search is over: after the last digit, or as soon as the whole bin
// is wanted (for most data after two digits: its keys are then those above T - 1
// with no ties to choose among).
__device__ __forceinline__ bool take_digit(int3 r, int pass, uint32_t* T, int* want) {
  *T |= static_cast<uint32_t>(r.x) << digit_shift(pass);
  *want -= r.y;
  if (pass + 1 == kDigits) return true;
  if (r.z != *want) return false;
  *T -= 1;  // no key is 0: the lowest, of -inf, is 0x7fffff
  *want = 0;
  return true;
}

// Ordered emission.  A warp owns a run of consecutive positions; a position is
// kept if its key is above T, or at T among the first `ties` of those.
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
// Positions of a run above T and at T (keys of 0 lie below every T).
template <class KeyFn>
__device__ __forceinline__ int2 count_run(WarpRun r, uint32_t T, KeyFn key_of) {
  const int lane = threadIdx.x & 31;
  int g = 0, e = 0;
#pragma unroll 4
  for (int i = r.begin + lane; i < r.end; i += 32) {
    const uint32_t k = key_of(i);
    g += k > T;
    e += k == T;
  }
  return make_int2(__reduce_add_sync(0xffffffffu, g), __reduce_add_sync(0xffffffffu, e));
}
// Keys in shared memory are counted by ballots that stay: lane j holds those of
// the 32 positions from begin + 32 j on, for a span of up to 1024 positions.
constexpr int kSpan = 1024;
struct SpanMasks {
  uint32_t gt, eq;  // above T, at T
};
template <class KeyFn>
__device__ __forceinline__ SpanMasks span_masks(int begin, int end, uint32_t T, KeyFn key_of) {
  const int lane = threadIdx.x & 31;
  SpanMasks m = {0, 0};
#pragma unroll 4
  for (int j = 0; j < 32; ++j) {
    const int i = begin + 32 * j;
    if (i >= end) break;
    const bool in = i + lane < end;
    const uint32_t k = in ? key_of(i + lane) : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, k > T), eq = __ballot_sync(0xffffffffu, in && k == T);
    if (lane == j) m = {gt, eq};
  }
  return m;
}
// Positions above T (x) and at T (y) in the span before the lane's; the span's in all.
__device__ __forceinline__ int2 span_before(SpanMasks m, int2* all) {
  const int lane = threadIdx.x & 31;
  const int own = __popc(m.gt) | __popc(m.eq) << 16;
  int incl = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  const int sum = __shfl_sync(0xffffffffu, incl, 31);
  *all = make_int2(sum & 0xffff, sum >> 16);
  return make_int2((incl - own) & 0xffff, (incl - own) >> 16);
}
// The lowest n set bits of m.
__device__ __forceinline__ uint32_t lowest_bits(uint32_t m, int n) {
  if (n >= __popc(m)) return m;
  uint32_t left = m;
  for (int i = 0; i < n; ++i) left &= left - 1;
  return m ^ left;
}

// emit(position, value, kept, rank among the kept positions before it) for a run
// with g positions above T and e at T before it; fetch(position) gives the value,
// loaded for kEmitBatch positions at a time.
constexpr int kEmitBatch = 6;
template <class Value, bool kTies, class KeyFn, class FetchFn, class EmitFn>
__device__ __forceinline__ void emit_run_of(WarpRun r, uint32_t T, int g, int e, int ties, KeyFn key_of, FetchFn fetch,
                                         EmitFn emit) {
  const int lane = threadIdx.x & 31;
  const uint32_t lt = (1u << lane) - 1u;
  for (int i0 = r.begin; i0 < r.end; i0 += 32 * kEmitBatch) {
    Value v[kEmitBatch];
    uint32_t k[kEmitBatch];
#pragma unroll
    for (int u = 0; u < kEmitBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      k[u] = 0;
      if (i < r.end) {
        v[u] = fetch(i);
        k[u] = key_of(i);
      }
    }
#pragma unroll
    for (int u = 0; u < kEmitBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      const uint32_t mg = __ballot_sync(0xffffffffu, k[u] > T);
      bool kept = k[u] > T;
      int at = g + __popc(mg & lt);
      g += __popc(mg);
      if (kTies) {
        const uint32_t me = __ballot_sync(0xffffffffu, k[u] == T && i < r.end);
        const int eb = e + __popc(me & lt);
        kept = kept || (k[u] == T && eb < ties);
        at += min(eb, ties);
        e += __popc(me);
      }
      if (i < r.end) emit(i, v[u], kept, at);
    }
  }
}
template <class Value, class KeyFn, class FetchFn, class EmitFn>
__device__ __forceinline__ void emit_run(WarpRun r, uint32_t T, int g, int e, int ties, KeyFn key_of, FetchFn fetch,
                                         EmitFn emit) {
  if (ties > 0)
    emit_run_of<Value, true>(r, T, g, e, ties, key_of, fetch, emit);
  else  // the usual case
    emit_run_of<Value, false>(r, T, g, e, ties, key_of, fetch, emit);
}

}  // namespace ddt
