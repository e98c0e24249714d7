// block_select.cu -- the blocks that each tree node reads: 8-bit query rows, and
// the best blocks of a node's scores (the scores themselves: key_scores.cu).
//
//   query row r:  qs = max |q| / 127,  q_int = round(q / qs) in [-127, 127]
//   score(t, j) = scale_j * max over the heads h of (qs_h * (q_int_h . summary_j))
// The integer product is exact in fp32 and both roundings are fixed by this
// order, so the ranking is the definition's on every run and tiling.
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "ptx.cuh"
#include "rank_select.cuh"

namespace ddt {
namespace {

constexpr int kQuWarps = 8;

// One warp per query row: 72 pieces of 16 bytes, lanes 0-7 take a third one.
__global__ void __launch_bounds__(kQuWarps * 32) quant_rows_kernel(QuantParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kQuWarps + (threadIdx.x >> 5);
  if (r >= p.rows) return;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + r * kDqk);
  uint4 v[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] = lane + 32 * i < kChunks ? __ldg(src + lane + 32 * i) : make_uint4(0, 0, 0, 0);
  // |x| of bf16 orders like its bits, infinities and NaN above every number
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  const bool finite = m < 0x7f80u;
  const float scale = finite ? __fdiv_rn(__uint_as_float(m << 16), 127.f) : CUDART_NAN_F;
  uint4* dst = reinterpret_cast<uint4*>(p.q_int + r * kDqk);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a = 0.f, c = 0.f;
      if (finite && scale > 0.f) {
        a = fminf(fmaxf(rintf(__fdiv_rn(__uint_as_float(w[k] << 16), scale)), -127.f), 127.f);
        c = fminf(fmaxf(rintf(__fdiv_rn(__uint_as_float(w[k] & 0xffff0000u), scale)), -127.f), 127.f);
      }
      o[k] = (__float_as_uint(a) >> 16) | (__float_as_uint(c) & 0xffff0000u);
    }
    if (lane + 32 * i < kChunks) dst[lane + 32 * i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (lane == 0) p.q_scale[r] = scale;
}

constexpr int kTkThreads = 256;
constexpr int kTkCached = 16384;  // order keys kept in shared memory

// One CTA per node: the digit select of rank_select.cuh over its scores, then
// the chosen blocks in ascending order.
__global__ void __launch_bounds__(kTkThreads) block_topk_kernel(TopkParams p, int cached) {
  extern __shared__ uint32_t keys_sh[];
  __shared__ int hist[kBins];
  __shared__ int tmp[kTkThreads / 32 + 2];
  __shared__ int cnt_gt[kTkThreads / 32], cnt_eq[kTkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, b = blockIdx.y;
  int L = __ldg(p.prefix_len + b);
  if (L < 0 || L > p.max_prefix_len) {
    if (t == 0 && tid == 0) atomicOr(p.status, kStatusBadPrefix);
    L = L < 0 ? 0 : p.max_prefix_len;
  }
  const int n = (L + p.block - 1) / p.block;
  const float* score = p.score + (static_cast<int64_t>(b) * p.nodes + t) * p.blocks;
  int32_t* out = p.block_idx + (static_cast<int64_t>(b) * p.nodes + t) * p.topk;
  const int keep = min(p.topk, n);
  for (int i = keep + tid; i < p.topk; i += kTkThreads) out[i] = -1;
  if (keep == n) {
    for (int i = tid; i < n; i += kTkThreads) out[i] = i;
    return;
  }
  const int lo = min(p.first, n), hi = max(lo, n - min(p.last, n));  // [lo, hi): chosen by score
  const int need = keep - (lo + (n - hi));
  if (need <= 0) {  // only forced blocks fit: the lowest ones
    for (int i = tid; i < keep; i += kTkThreads) out[i] = i < lo ? i : hi + (i - lo);
    return;
  }
  const bool in_sh = n <= cached;
  if (in_sh)
    for (int i = tid; i < n; i += kTkThreads) keys_sh[i] = order_key(__ldg(score + i));
  auto key_of = [&](int i) { return in_sh ? keys_sh[i] : order_key(__ldg(score + i)); };
  uint32_t T = 0;
  int want = need;
  for (int pass = 0; pass < kDigits; ++pass) {
    for (int i = tid; i < kBins; i += kTkThreads) hist[i] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kTkThreads) {
      const int i = i0 + tid;
      const bool live = i >= lo && i < hi;
      count_key(hist, live ? key_of(i) : 0u, T, pass, live);
    }
    __syncthreads();
    int bin, above;
    find_bin<kTkThreads>(want, [&](int x) { return hist[x]; }, tmp, &bin, &above);
    T |= static_cast<uint32_t>(bin) << digit_shift(pass);
    want -= above;
  }
  const int ties = want;
  int gt_base = 0, eq_base = 0;
  for (int i0 = 0; i0 < n; i0 += kTkThreads) {
    const int i = i0 + tid;
    int c = 0;
    if (i < n) {
      if (i < lo || i >= hi) {
        c = 2;
      } else {
        const uint32_t k = key_of(i);
        c = k > T ? 2 : (k == T ? 1 : 0);
      }
    }
    const uint32_t mg = __ballot_sync(0xffffffffu, c == 2), me = __ballot_sync(0xffffffffu, c == 1);
    if (lane == 0) {
      cnt_gt[warp] = __popc(mg);
      cnt_eq[warp] = __popc(me);
    }
    __syncthreads();
    int g = gt_base, e = eq_base;
#pragma unroll
    for (int w = 0; w < kTkThreads / 32; ++w) {
      if (w < warp) {
        g += cnt_gt[w];
        e += cnt_eq[w];
      }
      gt_base += cnt_gt[w];
      eq_base += cnt_eq[w];
    }
    const uint32_t lt = (1u << lane) - 1u;
    g += __popc(mg & lt);
    e += __popc(me & lt);
    if (c == 2 || (c == 1 && e < ties)) out[g + min(e, ties)] = i;
    __syncthreads();
  }
}

}  // namespace

cudaError_t configure_topk() {
  return cudaFuncSetAttribute(block_topk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTkCached * 4);
}

cudaError_t launch_quant_rows(const QuantParams& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  const int64_t grid = (p.rows + kQuWarps - 1) / kQuWarps;
  quant_rows_kernel<<<static_cast<unsigned>(grid), kQuWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_block_topk(const TopkParams& p, int batch, cudaStream_t stream) {
  if (batch == 0) return cudaSuccess;
  const int cached = p.blocks <= kTkCached ? p.blocks : kTkCached;
  block_topk_kernel<<<dim3(p.nodes, batch), kTkThreads, cached * 4, stream>>>(p, cached);
  return cudaGetLastError();
}

}  // namespace ddt
