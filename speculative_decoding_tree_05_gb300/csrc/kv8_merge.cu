// kv8_merge.cu -- the merge of a request's units of attention over the 8-bit cache.
//
// out = sum over the units of w_u o_u / sum of w_u with w_u = exp(lse_u - max), the o_u
// normalised; lse = max + log of the sum of w_u. A row is shared by 1 to 16 warps, each
// with every 16th (or so) unit, four units' loads in flight at a time. Bound by reading
// the partials, which the attention kernel has just written to L2: 2052 bytes a row and unit.
// Rows of one unit are written by that unit. (4 to 11 us; 35 for 8320 rows of 7 units.)
#include <cuda_runtime.h>
#include <math_constants.h>
#include "kv8.cuh"
#include "merge_row.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kWarps = 16;
constexpr int kBatch = 4;  // units in flight

__global__ void __launch_bounds__(kWarps * 32) kv8_merge_kernel(const __grid_constant__ Kv8MergeParams p) {
  __shared__ float4 acc_sh[kWarps][kDv / 4];
  __shared__ float sum_sh[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();  // the partials
  const int per_block = kWarps / p.warps, mine = warp % p.warps;
  const int64_t rows = static_cast<int64_t>(p.nodes) * p.heads, all_rows = rows * p.batch;
  const int64_t grow = static_cast<int64_t>(blockIdx.x) * per_block + warp / p.warps;
  int count = 0, first = 0;
  int64_t r = 0;
  if (grow < all_rows) {
    const int b = static_cast<int>(grow / rows);
    r = grow - b * rows;
    if (r < static_cast<int64_t>(kv8_nodes(p.tree_len, b, p.nodes)) * p.heads) {
      const Kv8Piece* piece = p.pieces + b;
      first = __ldcg(&piece->first);
      count = __ldcg(&piece->count);
    }
  }
  const bool join = count > 1;
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);  // dims 4 lane + 128 j + {0..3}
  float mx = -CUDART_INF_F, wsum = 0.f;
  if (join) {
    const float* lse = p.lse_part + first * rows + r;
    for (int s = lane; s < count; s += 32) mx = fmaxf(mx, __ldcg(lse + s * rows));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    for (int s0 = mine; s0 < count; s0 += kBatch * p.warps) {
      float4 x[kBatch][4];
      float v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = s0 + u * p.warps;
        const bool in = s < count;
        v[u] = in ? __ldcg(lse + s * rows) : -CUDART_INF_F;
        const float4* op = reinterpret_cast<const float4*>(p.o_part + ((first + s) * rows + r) * kDv);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u][j] = in ? __ldcg(op + lane + 32 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        // a NaN (a non-finite key that the row reads) stays one: its weight is NaN
        const float w = v[u] == -CUDART_INF_F ? 0.f : fast_exp2((v[u] - mx) * kMergeLog2e);
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
  }
  if (p.warps > 1) {  // the row's warps add up, in their order
    if (mine > 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc_sh[warp][lane + 32 * j] = acc[j];
      if (lane == 0) sum_sh[warp] = wsum;
    }
    __syncthreads();
    if (mine > 0) return;
    for (int k = 1; k < p.warps; ++k) {
      wsum += sum_sh[warp + k];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 y = acc_sh[warp + k][lane + 32 * j];
        acc[j].x += y.x, acc[j].y += y.y, acc[j].z += y.z, acc[j].w += y.w;
      }
    }
  }
  if (!join) return;
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint2* dst = reinterpret_cast<uint2*>(p.out + grow * kDv);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    dst[lane + 32 * j] = make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
  if (lane == 0) p.lse[grow] = wsum == 0.f ? -CUDART_INF_F : mx + log2f(wsum) * kMergeLn2;
}

}  // namespace

cudaError_t launch_kv8_merge(const Kv8MergeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.nodes * p.heads, per_block = kWarps / p.warps;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + per_block - 1) / per_block));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel, p);
}

}  // namespace ddt
