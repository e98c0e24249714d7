// kv_evict.cu -- keep each request's heaviest positions and list the freed slots.
//
// Request b keeps n = min(keep_len, L) of its L positions: the first `sink` and
// the last `recent` rank before all others, then the larger weight, then the
// lower position; what is kept stays in order.  One cluster of CTAs per request,
// CTA r holding the r-th share of the positions:
//   1. three digit histograms of the unprotected positions' weights, summed over
//      the cluster through distributed shared memory (each CTA adds up its share
//      of the bins and hands the totals to all: every CTA reading every
//      histogram took 18,000 cycles a pass), give the weight of the last
//      position kept (T) and how many of the positions tied at T are kept;
//   2. the histograms also say how many of a CTA's own positions lie above and at
//      T; prefix sums over the cluster say where its kept and freed entries start;
//   3. a pass in position order writes both lists (ballots and one scan a tile).
// The weights are read from memory once and stay in shared memory where they
// fit.  The work is a few bytes per position, so the time is the latency of
// these dependent steps, not bandwidth, until the batch fills the GPU: small
// batches take clusters of 16.
#include <cuda_runtime.h>
#include "cache_ops.cuh"
#include "ptx.cuh"
#include "rank_select.cuh"

namespace ddt {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvMaxCluster = 16;
constexpr int kEvItems = 8;                       // positions per thread and tile of the ordered pass
constexpr int kEvTile = kEvThreads * kEvItems;
constexpr int kEvMaxCached = 40960;               // weights a CTA keeps in shared memory

__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(EvictParams p, int cached) {
  extern __shared__ uint32_t bits_sh[];           // [cached] the weights of this CTA's share
  __shared__ int hist[kDigits][kBins];
  __shared__ int tmp[2 * kEvThreads / 32 + 4];
  __shared__ int tile_gt[kEvItems * 32], tile_eq[kEvItems * 32];
  __shared__ int total[kBins];                    // the cluster's histogram of a pass
  __shared__ int own[2];                          // this CTA's positions kept for sure, at T
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = gridDim.x;  // one cluster spans x
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
  const int share = (L + ctas - 1) / ctas;
  const int begin = min(L, rank * share), end = min(L, begin + share);

  for (int i = tid; i < kDigits * kBins; i += kEvThreads) (&hist[0][0])[i] = 0;
  if (cached > 0) {
#pragma unroll 8
    for (int i = begin + tid; i < end; i += kEvThreads) bits_sh[i - begin] = __float_as_uint(__ldg(weight + i));
  }
  __syncthreads();
  auto bits_of = [&](int i) { return cached > 0 ? bits_sh[i - begin] : __float_as_uint(__ldg(weight + i)); };

  uint32_t T = 0;   // order key of the last unprotected position kept
  int ties = 0;     // positions at T that are kept
  int gt = 0, eq = 0;
  const bool select = need > 0 && keep < L;       // the same in every CTA of the cluster
  if (select) {
    int want = need;
    for (int pass = 0; pass < kDigits; ++pass) {
#pragma unroll 4
      for (int i0 = begin; i0 < end; i0 += kEvThreads) {
        const int i = i0 + tid;
        const bool live = i < end && i >= lo && i < hi;
        count_key(hist[pass], live ? order_key_bits(bits_of(i)) : 0u, T, pass, live);
      }
      cluster_sync();  // every CTA's histogram of this pass is complete
      // bins [rank seg, + seg) are added up here: `parts` threads a bin, which
      // share the CTAs to read from and, the sum known, to write to
      const int seg = kBins / ctas, parts = kEvThreads / seg;
      const int bin = rank * seg + tid / parts, part = tid % parts;
      int n = 0;
      for (int c = part; c < ctas; c += parts) n += ld_shared_cluster_b32(mapa_shared(smem_u32(&hist[pass][bin]), c));
      for (int off = 1; off < parts; off <<= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
      for (int c = part; c < ctas; c += parts) st_shared_cluster_b32(mapa_shared(smem_u32(&total[bin]), c), n);
      cluster_sync();  // the totals have arrived
      const BinResult r = find_bin<kEvThreads>(want, [&](int x) { return total[x]; }, hist[pass], tmp);
      T |= static_cast<uint32_t>(r.bin) << digit_shift(pass);
      want -= r.above;
      gt += r.own_above;
      eq = r.own_in;
    }
    ties = want;
  }
  // protected positions that stay: all of them, or the lowest `keep`
  const int held = min(prot, keep), held_lo = min(lo, held), held_hi = hi + (held - held_lo);
  auto within = [&](int x0, int x1) { return max(0, min(end, x1) - max(begin, x0)); };
  gt += within(0, held_lo) + within(hi, held_hi);
  if (keep == L) gt = end - begin;
  // 2: kept, 1: tied at T, 0: freed
  auto klass = [&](int i, uint32_t bits) -> int {
    if (keep == L || i < held_lo || (i >= hi && i < held_hi)) return 2;
    if (!select || i < lo || i >= hi) return 0;
    const uint32_t k = order_key_bits(bits);
    return k > T ? 2 : (k == T ? 1 : 0);
  };

  if (tid == 0) {
    own[0] = gt;
    own[1] = eq;
  }
  cluster_sync();
  int gt_base = 0, eq_base = 0;
  {
    const int g = lane < rank ? ld_shared_cluster_b32(mapa_shared(smem_u32(&own[0]), lane)) : 0;
    const int e = lane < rank ? ld_shared_cluster_b32(mapa_shared(smem_u32(&own[1]), lane)) : 0;
    gt_base = __reduce_add_sync(0xffffffffu, g);
    eq_base = __reduce_add_sync(0xffffffffu, e);
  }
  cluster_arrive();  // this thread no longer reads a peer's shared memory

  for (int t0 = begin; t0 < end; t0 += kEvTile) {
    int c[kEvItems], slot[kEvItems];
    uint32_t w[kEvItems];
#pragma unroll
    for (int k = 0; k < kEvItems; ++k) {
      const int i = t0 + k * kEvThreads + tid;
      slot[k] = i < end ? __ldg(p.slot_idx + row + i) : 0;
      w[k] = i < end ? bits_of(i) : 0;
    }
#pragma unroll
    for (int k = 0; k < kEvItems; ++k) {
      const int i = t0 + k * kEvThreads + tid;
      c[k] = i < end ? klass(i, w[k]) : -1;
      const uint32_t mg = __ballot_sync(0xffffffffu, c[k] == 2), me = __ballot_sync(0xffffffffu, c[k] == 1);
      if (lane == 0) {
        tile_gt[k * 32 + warp] = __popc(mg);
        tile_eq[k * 32 + warp] = __popc(me);
      }
    }
    __syncthreads();
    if (warp < 2) {  // exclusive prefix of the (item, warp) counts, in position order
      int* t = warp == 0 ? tile_gt : tile_eq;
      int v[kEvItems], sum = 0;  // lane l scans entries [8 l, 8 l + 8)
#pragma unroll
      for (int k = 0; k < kEvItems; ++k) {
        v[k] = t[lane * kEvItems + k];
        sum += v[k];
      }
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      int run = incl - sum;
#pragma unroll
      for (int k = 0; k < kEvItems; ++k) {
        t[lane * kEvItems + k] = run;
        run += v[k];
      }
      if (lane == 31) tmp[warp] = run;
    }
    __syncthreads();
    const uint32_t lt = (1u << lane) - 1u;
#pragma unroll
    for (int k = 0; k < kEvItems; ++k) {
      const int i = t0 + k * kEvThreads + tid;
      const uint32_t mg = __ballot_sync(0xffffffffu, c[k] == 2), me = __ballot_sync(0xffffffffu, c[k] == 1);
      if (i < end) {
        const int g = gt_base + tile_gt[k * 32 + warp] + __popc(mg & lt);
        const int e = eq_base + tile_eq[k * 32 + warp] + __popc(me & lt);
        const int kept_before = g + min(e, ties);
        if (c[k] == 2 || (c[k] == 1 && e < ties)) {
          p.slot_out[row + kept_before] = slot[k];
          p.weight_out[row + kept_before] = __uint_as_float(w[k]);
        } else {
          p.freed[row + i - kept_before] = slot[k];
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
  cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvMaxCached * 4);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t launch_kv_evict(const EvictParams& p, int batch, cudaStream_t stream) {
  // 16 CTAs a request while the clusters of the batch fit the GPU side by side
  // (at most 8 of 16 CTAs: clusters stay within a GPC), 8 beyond that
  const int ctas = batch <= 8 ? kEvMaxCluster : 8;
  const int64_t share = (int64_t(p.max_prefix_len) + ctas - 1) / ctas;
  const int cached = share <= kEvMaxCached ? static_cast<int>(share) : 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas, batch);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = cached * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_evict_kernel, p, cached);
}

}  // namespace ddt
