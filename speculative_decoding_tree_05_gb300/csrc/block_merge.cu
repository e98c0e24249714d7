// block_merge.cu -- the merge of block attention's key splits.
//
// out = sum over the splits of w_s o_s / sum of w_s with w_s = exp(lse_s - max),
// the o_s normalised; lse = max + log of the sum of w_s.  One warp per (node,
// head) row, four splits' loads in flight at a time.
// Bound by reading the partials, which the attention kernel has just written to
// L2: bytes per row splits * 2052 + 1028.
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "merge_row.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kBmWarps = 8;
constexpr int kBmBatch = 4;  // splits in flight

__global__ void __launch_bounds__(kBmWarps * 32) block_merge_kernel(const __grid_constant__ BlockMergeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kBmWarps + (threadIdx.x >> 5);
  const int64_t grow = blockIdx.y * p.rows + r, base = static_cast<int64_t>(blockIdx.y) * p.splits * p.rows + r;
  grid_dep_wait();  // the partials
  if (r >= p.rows) return;
  // split s's log-sum-exp in log2 units, in lane s
  const float mine = lane < p.splits ? __ldcg(p.lse_part + base + lane * p.rows) * kMergeLog2e : -CUDART_INF_F;
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);  // dims 4 lane + 128 j + {0..3}
  float mx = mine;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  // a NaN (a non-finite key that the row reads) stays one: its weight is NaN
  const float w_mine = mine == -CUDART_INF_F ? 0.f : fast_exp2(mine - mx);
  float wsum = 0.f;
  for (int s0 = 0; s0 < p.splits; s0 += kBmBatch) {
    float4 x[kBmBatch][4];
#pragma unroll
    for (int u = 0; u < kBmBatch; ++u) {
      const float4* op = reinterpret_cast<const float4*>(p.o_part + (base + (s0 + u) * p.rows) * kDv);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[u][j] = s0 + u < p.splits ? __ldcg(op + lane + 32 * j) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kBmBatch; ++u) {
      const float w = __shfl_sync(0xffffffffu, w_mine, (s0 + u) & 31);  // 0 behind the last split
      if (s0 + u >= p.splits) break;
      wsum += w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j].x = fmaf(w, x[u][j].x, acc[j].x);
        acc[j].y = fmaf(w, x[u][j].y, acc[j].y);
        acc[j].z = fmaf(w, x[u][j].z, acc[j].z);
        acc[j].w = fmaf(w, x[u][j].w, acc[j].w);
      }
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint2* dst = reinterpret_cast<uint2*>(p.out + grow * kDv);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    dst[lane + 32 * j] = make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
  if (lane == 0) p.lse[grow] = wsum == 0.f ? -CUDART_INF_F : (mx + log2f(wsum)) * kMergeLn2;
}

}  // namespace

cudaError_t launch_block_merge(const BlockMergeParams& p, int batch, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((p.rows + kBmWarps - 1) / kBmWarps), batch);
  cfg.blockDim = dim3(kBmWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_merge_kernel, p);
}

}  // namespace ddt
