// block_merge.cu -- the tree part of block attention and the merge of its key splits.
//
// Row (node t, head h): attention over t's ancestors and itself (a few rows, on
// the CUDA cores), then the log-sum-exp merge with the normalised partials of the
// key splits, written as bf16.  The same step follows verify attention
// (tail_merge.cu); this kernel differs in what it is bound by: the splits are
// few, so the time is the latency of parents -> slots -> rows -> partials, and
// registers decide how many rows hide it.  One CTA of 8 warps per (request,
// node, up to 16 heads); a warp takes two partials at a time (64 registers, four
// CTAs an SM), and tree rows are staged 32 at a time instead of all T, which
// caps shared memory at 36 KB.  65 nodes of 128 heads: 9.9 us against 22.5 with
// the other kernel.
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "merge_row.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kBmThreads = 256;
constexpr int kBmWarps = kBmThreads / 32;
constexpr int kBmStage = 32;  // tree rows staged at a time

__global__ void __launch_bounds__(kBmThreads, 4) block_merge_kernel(const __grid_constant__ BlockMergeParams p) {
  __shared__ __align__(16) uint8_t rows_sh[kBmStage * kRowBytes];
  __shared__ int par_sh[kMaxNodes], slot_sh[kMaxNodes], vis_sh[kMaxNodes];
  __shared__ int n_vis_sh;
  const int t = blockIdx.x, b = blockIdx.z, T = p.nodes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(p.heads, h0 + p.heads_per_cta);

  for (int i = tid; i < T; i += kBmThreads) {
    par_sh[i] = __ldg(p.tree_parent + static_cast<int64_t>(b) * T + i);
    slot_sh[i] = __ldg(p.tree_slot_idx + static_cast<int64_t>(b) * T + i);
  }
  __syncthreads();
  int32_t flags = 0;
  if (tid == 0) {
    int32_t st = 0;
    n_vis_sh = ancestor_slots(t, T, p.pool_slots, [&](int u) { return par_sh[u]; }, [&](int u) { return slot_sh[u]; },
                              vis_sh, &st);
    flags = blockIdx.y == 0 ? st : 0;
  }
  __syncthreads();
  const int n_vis = n_vis_sh;
  const int64_t req_rows = static_cast<int64_t>(T) * p.heads;

  for (int hb = h0; hb < h1; hb += kBmWarps) {
    const int h = hb + warp;
    const bool live = h < h1;
    const int64_t r = static_cast<int64_t>(t) * p.heads + h, grow = b * req_rows + r;
    // q: lane holds dims {64 i + 2 lane, + 1}, i = 0..8
    uint32_t qv[9];
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(p.q + grow * kDqk);
#pragma unroll
    for (int i = 0; i < 9; ++i) qv[i] = live ? __ldg(qrow + 32 * i + lane) : 0;
    float m = -CUDART_INF_F, l = 0.f, o[16];  // value dims 4 lane + 128 j + {0..3}
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = 0.f;
    for (int v0 = 0; v0 < n_vis; v0 += kBmStage) {
      const int nv = min(kBmStage, n_vis - v0);
      if (hb > h0 || v0 > 0) __syncthreads();  // the rows before are read
      if (hb == h0 || n_vis > kBmStage) {
        for (int i = tid; i < nv * kChunks; i += kBmThreads) {
          const int v = i / kChunks, c = i - v * kChunks;
          reinterpret_cast<uint4*>(rows_sh + v * kRowBytes)[c] =
              __ldg(reinterpret_cast<const uint4*>(p.kv + static_cast<int64_t>(vis_sh[v0 + v]) * kDqk) + c);
        }
        __syncthreads();
      }
      if (!live) continue;
      for (int v = 0; v < nv; ++v) {
        const uint32_t* kr = reinterpret_cast<const uint32_t*>(rows_sh + v * kRowBytes);
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < 9; ++i) {
          const uint32_t kk = kr[32 * i + lane];
          acc = fmaf(bf16_lo(qv[i]), bf16_lo(kk), acc);
          acc = fmaf(bf16_hi(qv[i]), bf16_hi(kk), acc);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        const float s = acc * p.scale_log2;
        const float mn = fmaxf(m, s);
        const float alpha = m == -CUDART_INF_F ? 0.f : fast_exp2(m - mn);
        const float pv = fast_exp2(s - mn);  // NaN for a non-finite score, as the sums become
        l = l * alpha + pv;
        m = mn;
        const uint2* vrow = reinterpret_cast<const uint2*>(kr);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 w = vrow[lane + 32 * j];
          o[4 * j + 0] = fmaf(o[4 * j + 0], alpha, pv * bf16_lo(w.x));
          o[4 * j + 1] = fmaf(o[4 * j + 1], alpha, pv * bf16_hi(w.x));
          o[4 * j + 2] = fmaf(o[4 * j + 2], alpha, pv * bf16_lo(w.y));
          o[4 * j + 3] = fmaf(o[4 * j + 3], alpha, pv * bf16_hi(w.y));
        }
      }
    }
    // (m, l, o) starts the merge as one more partial, not normalised
    grid_dep_wait();  // the splits' partials, and the status word cleared
    if (flags) atomicOr(p.status, flags);
    if (!live) continue;
    const int64_t base = static_cast<int64_t>(b) * p.splits * p.pstride + r;
    // split s's log-sum-exp in log2 units, in lane s (at most 32 splits)
    const float mine = lane < p.splits ? __ldcg(p.lse_part + base + lane * p.pstride) * kMergeLog2e : -CUDART_INF_F;
    float mx = mine;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    mx = fmaxf(mx, m);
    const float wt = m == -CUDART_INF_F ? (l == 0.f ? 0.f : l) : fast_exp2(m - mx);
    float wsum = l * wt;
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] *= wt;
    const float w_mine = mine == -CUDART_INF_F ? 0.f : fast_exp2(mine - mx);
    for (int s = 0; s < p.splits; s += 2) {
      float4 x[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4* op = reinterpret_cast<const float4*>(p.o_part + (base + (s + u) * p.pstride) * kDv);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u][j] = s + u < p.splits ? __ldcg(op + lane + 32 * j) : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float w = __shfl_sync(0xffffffffu, w_mine, (s + u) & 31);  // 0 behind the last split
        wsum += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[4 * j + 0] = fmaf(w, x[u][j].x, o[4 * j + 0]);
          o[4 * j + 1] = fmaf(w, x[u][j].y, o[4 * j + 1]);
          o[4 * j + 2] = fmaf(w, x[u][j].z, o[4 * j + 2]);
          o[4 * j + 3] = fmaf(w, x[u][j].w, o[4 * j + 3]);
        }
      }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    uint2* dst = reinterpret_cast<uint2*>(p.out + grow * kDv);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dst[lane + 32 * j] = make_uint2(pack_bf16x2(o[4 * j] * inv, o[4 * j + 1] * inv),
                                      pack_bf16x2(o[4 * j + 2] * inv, o[4 * j + 3] * inv));
    if (lane == 0) p.lse[grow] = wsum == 0.f ? -CUDART_INF_F : (mx + log2f(wsum)) * kMergeLn2;
  }
}

}  // namespace

cudaError_t launch_block_merge(const BlockMergeParams& p, int batch, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.nodes, (p.heads + p.heads_per_cta - 1) / p.heads_per_cta, batch);
  cfg.blockDim = dim3(kBmThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_merge_kernel, p);
}

}  // namespace ddt
