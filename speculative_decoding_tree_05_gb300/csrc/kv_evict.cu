// kv_evict.cu -- keep each request's heaviest positions and list the freed slots.
//
// Request b keeps n = min(keep_len, L) of its L positions: the first `sink` and
// the last `recent` rank before all others, then the larger weight, then the
// lower position; what is kept stays in order.  One cluster of CTAs per request,
// CTA r holding the r-th share of the positions:
//   1. three digit histograms of the unprotected positions' weights, summed over
//      the cluster through distributed shared memory, give the weight of the last
//      position kept (T) and how many of the positions tied at T are kept;
//   2. every CTA counts its positions above and at T; the cluster's prefix sums
//      say where its kept and freed entries start;
//   3. a pass in position order writes both lists (ballots and one scan a tile).
// The weights are read from memory once: their order keys stay in shared memory
// where they fit.  The work is a few bytes per position, so the time is the
// latency of these dependent steps, not bandwidth, until the batch fills the GPU.
#include <cuda_runtime.h>
#include "cache_ops.cuh"
#include "ptx.cuh"
#include "rank_select.cuh"

namespace ddt {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvCluster = 8;
constexpr int kEvItems = 4;                       // positions per thread and tile of the ordered pass
constexpr int kEvTile = kEvThreads * kEvItems;
constexpr int kEvMaxCached = 40960;               // order keys a CTA keeps in shared memory

__global__ void __launch_bounds__(kEvThreads) __cluster_dims__(kEvCluster, 1, 1)
    kv_evict_kernel(EvictParams p, int cached) {
  extern __shared__ uint32_t keys_sh[];           // [cached] order keys of this CTA's share
  __shared__ int hist[kDigits][kBins];
  __shared__ int tmp[kEvThreads / 32 + 2];
  __shared__ int tile_gt[kEvItems * 32], tile_eq[kEvItems * 32];
  __shared__ int own[2];                          // this CTA's positions above T, at T
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int b = blockIdx.y;
  int L = __ldg(p.prefix_len + b);
  if (L < 0 || L > p.max_prefix_len) {
    if (rank == 0 && tid == 0) atomicOr(p.status, kStatusBadPrefix);
    L = L < 0 ? 0 : p.max_prefix_len;
  }
  const int keep = min(max(__ldg(p.keep_len + b), 0), L);
  const int lo = min(p.sink, L), hi = max(lo, L - min(p.recent, L));  // [lo, hi): unprotected
  const int prot = lo + (L - hi);
  const int need = keep - prot;                   // unprotected positions to keep (<= 0: none)
  const int64_t row = static_cast<int64_t>(b) * p.stride;
  const float* weight = p.weight + row;
  // this CTA's share of the positions, in order
  const int share = (L + kEvCluster - 1) / kEvCluster;
  const int begin = min(L, rank * share), end = min(L, begin + share);

  for (int i = tid; i < kDigits * kBins; i += kEvThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto key_of = [&](int i) { return cached > 0 ? keys_sh[i - begin] : order_key(__ldg(weight + i)); };

  uint32_t T = 0;   // order key of the last unprotected position kept
  int ties = 0;     // positions at T that are kept
  const bool select = need > 0 && keep < L;       // the same in every CTA of the cluster
  if (cached > 0 && select) {
    for (int i = begin + tid; i < end; i += kEvThreads) keys_sh[i - begin] = order_key(__ldg(weight + i));
    __syncthreads();
  }
  if (select) {
    int want = need;
    for (int pass = 0; pass < kDigits; ++pass) {
      for (int i0 = begin; i0 < end; i0 += kEvThreads) {
        const int i = i0 + tid;
        const bool live = i < end && i >= lo && i < hi;
        count_key(hist[pass], live ? key_of(i) : 0u, T, pass, live);
      }
      cluster_sync();  // every CTA's histogram of this pass is complete
      int bin, above;
      find_bin<kEvThreads>(want, [&](int x) {
        int n = 0;
        const uint32_t a = smem_u32(&hist[pass][x]);
#pragma unroll
        for (int r = 0; r < kEvCluster; ++r) n += ld_shared_cluster_b32(mapa_shared(a, r));
        return n;
      }, tmp, &bin, &above);
      T |= static_cast<uint32_t>(bin) << digit_shift(pass);
      want -= above;
    }
    ties = want;
  }

  // kept: protected positions (class 2), above T (class 1), at T (class 0)
  auto klass = [&](int i) -> int {                // 2: kept, 1: tied at T, 0: freed
    if (keep == L) return 2;
    if (i < lo || i >= hi) {
      if (need >= 0) return 2;
      const int q = i < lo ? i : lo + (i - hi);   // rank among the protected positions
      return q < keep ? 2 : 0;
    }
    if (!select) return 0;
    const uint32_t k = key_of(i);
    return k > T ? 2 : (k == T ? 1 : 0);
  };

  int gt = 0, eq = 0;
  for (int i = begin + tid; i < end; i += kEvThreads) {
    const int c = klass(i);
    gt += c == 2;
    eq += c == 1;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (tid == 0) own[0] = own[1] = 0;
  __syncthreads();
  if (lane == 0) {
    atomicAdd(&own[0], gt);
    atomicAdd(&own[1], eq);
  }
  cluster_sync();
  int gt_base = 0, eq_base = 0;
  for (int r = 0; r < rank; ++r) {
    gt_base += ld_shared_cluster_b32(mapa_shared(smem_u32(&own[0]), r));
    eq_base += ld_shared_cluster_b32(mapa_shared(smem_u32(&own[1]), r));
  }
  cluster_arrive();  // this thread no longer reads a peer's shared memory

  for (int t0 = begin; t0 < end; t0 += kEvTile) {
    int c[kEvItems];
    uint32_t mgt[kEvItems], meq[kEvItems];
#pragma unroll
    for (int k = 0; k < kEvItems; ++k) {
      const int i = t0 + k * kEvThreads + tid;
      c[k] = i < end ? klass(i) : -1;
      mgt[k] = __ballot_sync(0xffffffffu, c[k] == 2);
      meq[k] = __ballot_sync(0xffffffffu, c[k] == 1);
      if (lane == 0) {
        tile_gt[k * 32 + warp] = __popc(mgt[k]);
        tile_eq[k * 32 + warp] = __popc(meq[k]);
      }
    }
    __syncthreads();
    if (warp < 2) {  // exclusive prefix of the (item, warp) counts, in position order
      int* t = warp == 0 ? tile_gt : tile_eq;
      int run = 0;
#pragma unroll
      for (int k = 0; k < kEvItems; ++k) {
        const int v = t[k * 32 + lane];
        int incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += o;
        }
        t[k * 32 + lane] = run + incl - v;
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) tmp[warp] = run;
    }
    __syncthreads();
    const uint32_t lt = (1u << lane) - 1u;
#pragma unroll
    for (int k = 0; k < kEvItems; ++k) {
      const int i = t0 + k * kEvThreads + tid;
      if (i < end) {
        const int g = gt_base + tile_gt[k * 32 + warp] + __popc(mgt[k] & lt);
        const int e = eq_base + tile_eq[k * 32 + warp] + __popc(meq[k] & lt);
        const int kept_before = g + min(e, ties);
        const int slot = __ldg(p.slot_idx + row + i);
        if (c[k] == 2 || (c[k] == 1 && e < ties)) {
          p.slot_out[row + kept_before] = slot;
          p.weight_out[row + kept_before] = __ldg(weight + i);
        } else {
          p.freed[row + i - kept_before] = slot;
        }
      }
    }
    gt_base += tmp[0];
    eq_base += tmp[1];
    __syncthreads();
  }
  if (rank == 0 && tid == 0) p.len_out[b] = keep;
  cluster_wait();  // no CTA leaves while a peer may still read its counts
}

}  // namespace

cudaError_t configure_evict() {
  return cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvMaxCached * 4);
}

cudaError_t launch_kv_evict(const EvictParams& p, int batch, cudaStream_t stream) {
  const int64_t share = (int64_t(p.max_prefix_len) + kEvCluster - 1) / kEvCluster;
  const int cached = share <= kEvMaxCached ? static_cast<int>(share) : 0;
  kv_evict_kernel<<<dim3(kEvCluster, batch), kEvThreads, cached * 4, stream>>>(p, cached);
  return cudaGetLastError();
}

}  // namespace ddt
