// kv_evict.cu -- keep each request's heaviest positions and list the freed slots.
//
// Request b keeps n = min(keep_len, L) of its L positions: the first `sink` and
// the last `recent` rank before all others, then the larger weight, then the
// lower position; what is kept stays in order.  One cluster of CTAs per request,
// CTA r holding the r-th share of the positions:
//   1. two or three digit histograms of the unprotected positions' weights give the
//      weight of the last position kept (T) and how many of the positions tied at
//      T are kept.  Each CTA adds the bins that it filled to the totals of their
//      owner (a share of the bins each) through distributed shared memory and
//      reads the totals back from the owners: one cluster barrier a digit (every
//      CTA reading every histogram took 18,000 cycles a digit, this 3,000);
//   2. every warp counts what it keeps of a run of consecutive positions, and
//      prefix sums over the CTA and the cluster say where its entries start;
//   3. the warps write both lists in position order, without further barriers.
// The weights are read once for the ranking and stay in shared memory, as order
// keys, where they fit; the slots are on their way to L2 meanwhile (64 requests:
// 45.8 -> 42.3 us).  The work is a few bytes per position, so the time is
// the latency of these dependent steps, not bandwidth, until the batch fills the
// GPU: small batches take clusters of 16.
#include <cuda_runtime.h>
#include "cache_ops.cuh"
#include "ptx.cuh"
#include "rank_select.cuh"

namespace ddt {
namespace {

constexpr int kEvMaxCluster = 16;
constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBatch = 12;                      // weights in flight per thread
constexpr int kEvMaxCached = 40960;               // order keys a CTA keeps in shared memory
constexpr int kEvMaxOrdered = 256;                // requests whose lengths every CTA ranks
static_assert(kEvMaxOrdered <= kBins, "the lengths lie in the histogram");

struct EvictShared {
  int hist[kBins];            // this CTA's histogram of a digit
  int total[kDigits][kBins];  // the cluster's, in the bins that this CTA owns
  int tmp[kEvWarps + 3];
  int warp_gt[kEvWarps], warp_eq[kEvWarps];
  int own[2];                 // this CTA's positions kept for sure, at T
};

// kCached: the order keys of the CTA's share lie in shared memory.
template <bool kCached>
__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(EvictParams p, bool by_length) {
  extern __shared__ uint32_t keys_sh[];           // [share] if kCached
  __shared__ EvictShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = gridDim.x;  // one cluster spans x
  auto length_of = [&](int i) {
    const int n = __ldg(p.prefix_len + i);
    return n < 0 ? 0 : (n > p.max_prefix_len ? p.max_prefix_len : n);
  };
  int b = blockIdx.y;
  if (by_length) {  // the y-th longest request, the earlier one of equals
    const int batch = gridDim.y;
    for (int i = tid; i < batch; i += kEvThreads) sh.hist[i] = length_of(i);
    __syncthreads();
    for (int i = tid; i < batch; i += kEvThreads) {
      const int mine = sh.hist[i];
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < batch; ++j) before += sh.hist[j] > mine || (sh.hist[j] == mine && j < i);
      if (before == static_cast<int>(blockIdx.y)) sh.tmp[0] = i;
    }
    __syncthreads();
    b = sh.tmp[0];
  }
  const int L = length_of(b);
  if (rank == 0 && blockIdx.y == 0) {
    // The lengths are all that can be wrong, so one CTA looks at every request's
    // and writes the status word as a whole: no clear before the launch.
    bool bad = false;
    for (int i = tid; i < gridDim.y; i += kEvThreads) {
      const int n = __ldg(p.prefix_len + i);
      bad = bad || n < 0 || n > p.max_prefix_len;
    }
    bad = __syncthreads_or(bad) != 0;
    if (tid == 0) *p.status = bad ? kStatusBadPrefix : 0;
  }
  const int keep = min(max(__ldg(p.keep_len + b), 0), L);
  const int lo = min(p.sink, L), hi = max(lo, L - min(p.recent, L));  // [lo, hi): unprotected
  const int prot = lo + (L - hi);
  const int need = keep - prot;                   // unprotected positions to keep (<= 0: none)
  const int64_t row = static_cast<int64_t>(b) * p.stride;
  const float* weight = p.weight + row;
  // this CTA's share of the positions, in order
  const int share = (L + ctas - 1) / ctas;
  const int begin = min(L, rank * share), end = min(L, begin + share);

  // protected positions that stay: all of them, or the lowest `keep`
  const int held = min(prot, keep), held_lo = min(lo, held), held_hi = hi + (held - held_lo);
  // order keys, protected positions above (they stay) or below (they do not) every weight's
  auto key_from = [&](int i, float w) -> uint32_t {
    if (i >= lo && i < hi) return order_key_bits(__float_as_uint(w));
    return i < held_lo || (i >= hi && i < held_hi) ? 0xffffffffu : 0u;
  };
  for (int i = tid; i < kDigits * kBins; i += kEvThreads) (&sh.total[0][0])[i] = 0;
  cluster_arrive();  // this CTA's totals may be added to
  if (kCached) {
    for (int i0 = begin + tid; i0 < end; i0 += kEvBatch * kEvThreads) {
      float w[kEvBatch];
#pragma unroll
      for (int k = 0; k < kEvBatch; ++k)
        if (i0 + k * kEvThreads < end) w[k] = __ldg(weight + i0 + k * kEvThreads);
#pragma unroll
      for (int k = 0; k < kEvBatch; ++k)
        if (i0 + k * kEvThreads < end) keys_sh[i0 + k * kEvThreads - begin] = key_from(i0 + k * kEvThreads, w[k]);
    }
  }
  for (int i = begin + 32 * tid; i < end; i += 32 * kEvThreads) prefetch_l2(p.slot_idx + row + i);  // for step 3
  auto key_of = [&](int i) { return kCached ? keys_sh[i - begin] : key_from(i, __ldg(weight + i)); };
  cluster_wait();

  // T: order key of the last unprotected position kept, `ties` of those at T stay
  uint32_t T = need <= 0 && keep < L ? 0xfffffffeu : 0u;  // only the protected ones, or every position
  int ties = 0;
  const bool select = need > 0 && keep < L;  // the same in every CTA of the cluster
  if (select) {
    const int from = max(begin, lo), to = min(end, hi);
    const int log_own = 31 - __clz(kBins / ctas);  // bins per owner
    int want = need;
    bool found = false;  // the same in every CTA
#pragma unroll
    for (int pass = 0; pass < kDigits; ++pass) {
      if (found) break;
      for (int i = tid; i < kBins; i += kEvThreads) sh.hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int i = from + tid; i < to; i += kEvThreads) count_key(sh.hist, key_of(i), T, pass);
      __syncthreads();
      for (int i = tid; i < kBins; i += kEvThreads) {
        const int n = sh.hist[i];
        if (n != 0) red_shared_cluster_add(mapa_shared(smem_u32(&sh.total[pass][i]), i >> log_own), n);
      }
      cluster_sync();  // every CTA's counts have arrived
      found = take_digit(find_bin<kEvThreads>(want, [&](int x) {
        return ld_shared_cluster_b32(mapa_shared(smem_u32(&sh.total[pass][x]), x >> log_own));
      }, sh.tmp), pass, &T, &want);
    }
    ties = want;
  }

  __syncthreads();
  const WarpRun run = warp_run(begin, end, kEvWarps, warp);
  const int2 mine = count_run(run, T, key_of);
  if (lane == 0) {
    sh.warp_gt[warp] = mine.x;
    sh.warp_eq[warp] = mine.y;
  }
  __syncthreads();
  const int wg = sh.warp_gt[lane], we = sh.warp_eq[lane];
  int g = __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0), e = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0);
  if (warp == 0) {
    const int all_g = __reduce_add_sync(0xffffffffu, wg), all_e = __reduce_add_sync(0xffffffffu, we);
    if (lane == 0) {
      sh.own[0] = all_g;
      sh.own[1] = all_e;
    }
  }
  cluster_sync();
  {
    const int pg = lane < rank ? ld_shared_cluster_b32(mapa_shared(smem_u32(&sh.own[0]), lane)) : 0;
    const int pe = lane < rank ? ld_shared_cluster_b32(mapa_shared(smem_u32(&sh.own[1]), lane)) : 0;
    g += __reduce_add_sync(0xffffffffu, pg);
    e += __reduce_add_sync(0xffffffffu, pe);
  }
  cluster_arrive();  // this thread no longer reads a peer's shared memory
  int32_t *slot_out = p.slot_out + row, *freed = p.freed + row;
  float* weight_out = p.weight_out + row;
  emit_run<int2>(run, T, g, e, ties, key_of,
                 [&](int i) { return make_int2(__ldg(p.slot_idx + row + i), __float_as_int(__ldg(weight + i))); },
                 [&](int i, int2 v, bool kept, int at) {
                   (kept ? slot_out : freed)[kept ? at : i - at] = v.x;  // one store for both: no divergence
                   if (kept) weight_out[at] = __int_as_float(v.y);
                 });
  if (rank == 0 && tid == 0) p.len_out[b] = keep;
  cluster_wait();  // no CTA leaves while a peer may still read its counts
}

}  // namespace

cudaError_t configure_evict() {
  cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvMaxCached * 4);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kv_evict_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kv_evict_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t launch_kv_evict(const EvictParams& p, int batch, int sm_count, cudaStream_t stream) {
  // One CTA (1024 threads, 64 registers) fills an SM.  The largest cluster, up to
  // 16, with which the batch takes at most two rounds of the SMs: more CTAs a
  // request shorten its steps, further rounds repeat their fixed costs (64
  // requests of up to 131072, in the batch's order: 81 us in clusters of 8, 54 us in clusters of 4).
  int ctas = kEvMaxCluster;
  while (ctas > 1 && int64_t(ctas) * batch > 2 * sm_count) ctas /= 2;
  // Where the clusters take more than one round, the long requests go first, so that
  // the last to start are short (the same batch 54 -> 44 us).
  // Beyond 256 requests the rounds are many and even out.
  const bool by_length = int64_t(ctas) * batch > sm_count && batch <= kEvMaxOrdered;
  const int64_t share = (int64_t(p.max_prefix_len) + ctas - 1) / ctas;
  const bool cached = share <= kEvMaxCached;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas, batch);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = cached ? static_cast<size_t>(share) * 4 : 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cached ? kv_evict_kernel<true> : kv_evict_kernel<false>, p, by_length);
}

}  // namespace ddt
