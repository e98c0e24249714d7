// block_select.cu -- the blocks that each tree node reads: 8-bit query rows, and
// the best blocks of a node's scores (the scores themselves: key_scores.cu).
//
//   query row r:  qs = max |q| * (1/127),  q_int = round(q / qs) in [-127, 127]
//   score(t, j) = scale_j * max over the heads h of (qs_h * (q_int_h . summary_j))
// The integer product is exact in fp32 and both roundings are fixed by this
// order, so the ranking is the definition's on every run and tiling.
#include <cuda_runtime.h>
#include <type_traits>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "ptx.cuh"
#include "rank_select.cuh"

namespace ddt {
namespace {

constexpr int kQuWarps = 8;

// One warp per query row: 72 pieces of 16 bytes, lanes 0-7 take a third one.
__global__ void __launch_bounds__(kQuWarps * 32) quant_rows_kernel(QuantParams p) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  grid_dep_launch();
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
  const float scale = finite ? __fmul_rn(__uint_as_float(m << 16), 1.f / 127.f) : CUDART_NAN_F;
  // round(x / scale), half to even: x * (1 / scale) is within 1e-4 of the quotient
  // (3 roundings of at most 127), so only a value that close to a half, or one that
  // is not finite, needs the division.  |t| < 2^22, so adding 1.5 * 2^23 rounds it.
  const float inv = finite && scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
  auto quantized = [&](float x) {
    const float t = x * inv;
    float n = __fadd_rn(__fadd_rn(t, 12582912.f), -12582912.f);
    if (!(fabsf(t - n) < 0.4999f)) n = rintf(__fdiv_rn(x, scale));
    return fminf(fmaxf(n, -127.f), 127.f);
  };
  uint4* dst = reinterpret_cast<uint4*>(p.q_int + r * kDqk);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a = 0.f, c = 0.f;
      if (finite && scale > 0.f) {
        a = quantized(__uint_as_float(w[k] << 16));
        c = quantized(__uint_as_float(w[k] & 0xffff0000u));
      }
      o[k] = (__float_as_uint(a) >> 16) | (__float_as_uint(c) & 0xffff0000u);
    }
    if (lane + 32 * i < kChunks) dst[lane + 32 * i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (lane == 0) p.q_scale[r] = scale;
}

constexpr int kTkCached = 16384;  // scores kept in shared memory
// Threads per node: 256 up to 1024 blocks (four scores a thread); beyond, 1024,
// which fill an SM, or 512, three CTAs to an SM, where there are more nodes than SMs.
constexpr int kTkSmall = 256, kTkMany = 512, kTkLarge = 1024, kTkSmallBlocks = 1024;
// a warp's run of scores in shared memory is one span
static_assert(kTkCached <= kTkMany / 32 * kSpan && kTkSmallBlocks <= kTkSmall / 32 * kSpan, "");

// One CTA per node: the digit select of rank_select.cuh over its scores, then
// the chosen blocks in ascending order.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kTkMany ? 3 : 1) block_topk_kernel(TopkParams p, int cached) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t keys_sh[];
  __shared__ int hist[kDigits][kBins];
  __shared__ int tmp[kWarps + 3];
  __shared__ int warp_gt[32], warp_eq[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, b = blockIdx.y;
  int L = __ldg(p.prefix_len + b);
  const bool bad_len = L < 0 || L > p.max_prefix_len;
  L = L < 0 ? 0 : (L > p.max_prefix_len ? p.max_prefix_len : L);
  auto wait_scores = [&] {  // the scores, and the status word cleared
    grid_dep_wait();
    if (bad_len && t == 0 && tid == 0) atomicOr(p.status, kStatusBadPrefix);
  };
  const int n = (L + p.block - 1) / p.block;
  const float* score = p.score + (static_cast<int64_t>(b) * p.nodes + t) * p.blocks;
  int32_t* out = p.block_idx + (static_cast<int64_t>(b) * p.nodes + t) * p.topk;
  const int keep = min(p.topk, n);
  for (int i = keep + tid; i < p.topk; i += kThreads) out[i] = -1;
  if (keep == n) {
    for (int i = tid; i < n; i += kThreads) out[i] = i;
    wait_scores();
    return;
  }
  const int lo = min(p.first, n), hi = max(lo, n - min(p.last, n));  // [lo, hi): chosen by score
  const int need = keep - (lo + (n - hi));
  if (need <= 0) {  // only forced blocks fit: the lowest ones
    for (int i = tid; i < keep; i += kThreads) out[i] = i < lo ? i : hi + (i - lo);
    wait_scores();
    return;
  }
  for (int i = tid; i < kDigits * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  wait_scores();
  const bool in_sh = n <= cached;
  auto key_from = [&](int i, float x) { return i < lo || i >= hi ? 0xffffffffu : order_key_bits(__float_as_uint(x)); };
  if (in_sh) {
    constexpr int kBatch = kThreads == kTkSmall ? kTkSmallBlocks / kTkSmall : 12;  // scores in flight per thread
    for (int i0 = tid; i0 < n; i0 += kBatch * kThreads) {
      float x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) x[u] = __ldcg(score + min(i0 + u * kThreads, n - 1));
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i0 + u * kThreads < n) keys_sh[i0 + u * kThreads] = key_from(i0 + u * kThreads, x[u]);
    }
  }
  if (tid < 32) warp_gt[tid] = warp_eq[tid] = 0;
  __syncthreads();
  auto choose = [&](auto key_of, auto in_shared) {
    uint32_t T = 0;
    int want = need;
    bool found = false;
#pragma unroll
    for (int pass = 0; pass < kDigits; ++pass) {
      if (found) break;
#pragma unroll 4
      for (int i = lo + tid; i < hi; i += kThreads) count_key(hist[pass], key_of(i), T, pass);
      __syncthreads();
      found = take_digit(find_bin<kThreads>(want, [&](int x) { return hist[pass][x]; }, tmp), pass, &T, &want);
    }
    const int ties = want;
    const WarpRun run = warp_run(0, n, kWarps, warp);
    auto before = [&](int2 mine) {  // the run's positions above T and at T -> those of the runs before it
      if (lane == 0) {
        warp_gt[warp] = mine.x;
        warp_eq[warp] = mine.y;
      }
      __syncthreads();
      return make_int2(__reduce_add_sync(0xffffffffu, lane < warp ? warp_gt[lane] : 0),
                       __reduce_add_sync(0xffffffffu, lane < warp ? warp_eq[lane] : 0));
    };
    if constexpr (!decltype(in_shared)::value) {
      const int2 at = before(count_run(run, T, key_of));
      emit_run<int>(run, T, at.x, at.y, ties, key_of, [](int i) { return i; }, [&](int, int v, bool kept, int to) {
        if (kept) out[to] = v;
      });
    } else {
      // few of the blocks are kept: the emission visits set bits alone
      const SpanMasks masks = span_masks(run.begin, run.end, T, key_of);
      int2 all;
      const int2 in_run = span_before(masks, &all), at = before(all);
      const int e = at.y + in_run.y;
      int to = at.x + in_run.x + min(e, ties);
      for (uint32_t m = masks.gt | lowest_bits(masks.eq, ties - e); m != 0; m &= m - 1)
        out[to++] = run.begin + 32 * lane + __ffs(m) - 1;
    }
  };
  if (in_sh)
    choose([&](int i) { return keys_sh[i]; }, std::true_type());
  else
    choose([&](int i) { return key_from(i, __ldcg(score + i)); }, std::false_type());
}

}  // namespace

cudaError_t configure_topk() {
  for (auto kernel : {block_topk_kernel<kTkSmall>, block_topk_kernel<kTkMany>, block_topk_kernel<kTkLarge>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTkCached * 4);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_quant_rows(const QuantParams& p, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  const int64_t grid = (p.rows + kQuWarps - 1) / kQuWarps;
  quant_rows_kernel<<<static_cast<unsigned>(grid), kQuWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_block_topk(const TopkParams& p, int batch, int sm_count, cudaStream_t stream) {
  if (batch == 0) return cudaSuccess;
  const int cached = p.blocks <= kTkCached ? p.blocks : kTkCached;
  // programmatic dependent of the scores: its set-up overlaps their end
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.nodes, batch);
  cfg.dynamicSmemBytes = cached * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.blocks <= kTkSmallBlocks) {
    cfg.blockDim = dim3(kTkSmall);
    return cudaLaunchKernelEx(&cfg, block_topk_kernel<kTkSmall>, p, cached);
  }
  const bool many = int64_t(p.nodes) * batch > sm_count;
  cfg.blockDim = dim3(many ? kTkMany : kTkLarge);
  return cudaLaunchKernelEx(&cfg, many ? block_topk_kernel<kTkMany> : block_topk_kernel<kTkLarge>, p, cached);
}

}  // namespace ddt
