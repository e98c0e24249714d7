// block_summary.cu -- 8-bit means of consecutive blocks of a request's prefix rows.
//
// For block j of request b (positions [j n, j n + n), cut at the prefix's end):
//   mean = (sum of its rows) / (rows)     576 dims
//   scale = max |mean| * (1/127),  summary = round(mean / scale), integers in [-127, 127]
// The integers are kept as bf16 (exact), the tensor cores' operand type: the
// dot product of two such rows is an integer below 2^24, so block scores come
// out exact in fp32 on any tiling.  The sums carry their rounding errors along
// (two-sum), so the mean is the exact sum's, rounded once, and no integer depends
// on the order of the rows.
//
// Bound by memory: each row is read once (1152 B).  One CTA of 288 threads per
// block: thread (g, c) adds the 16-byte piece c of rows g, g + 4, ...
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kSumGroups = 4;
constexpr int kSumThreads = kSumGroups * kChunks;  // 288
constexpr int kSumBatch = 8;                       // rows in flight per thread
constexpr int kMaxBlock = 128;
constexpr int kSumCtasPerSm = 3;                   // resident at 72 registers

// (hi, lo) + x without losing the rounding error of hi + x, two dims at a time
// (the additions are half of the kernel's instructions: paired ones halve them)
__device__ __forceinline__ void two_sum(uint64_t& hi, uint64_t& lo, uint64_t x) {
  const uint64_t s = add_x2(hi, x);
  const uint64_t v = sub_x2(s, hi);
  lo = add_x2(lo, add_x2(sub_x2(hi, sub_x2(s, v)), sub_x2(x, v)));
  hi = s;
}

__global__ void __launch_bounds__(kSumThreads, kSumCtasPerSm) block_summary_kernel(SummaryParams p) {
  __shared__ int slot_sh[kMaxBlock];
  __shared__ __align__(16) float part[kSumGroups - 1][2][kDqk];
  __shared__ float amax_sh[3];
  __shared__ int bad_sh[2];
  const int tid = threadIdx.x, g = tid / kChunks, c = tid - g * kChunks;
  const int b = blockIdx.y;
  int L = __ldg(p.prefix_len + b);
  if (L < 0 || L > p.max_prefix_len) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, kStatusBadPrefix);
    L = L < 0 ? 0 : p.max_prefix_len;
  }
  const int from = p.from_len != nullptr ? max(0, __ldg(p.from_len + b)) : 0;
  if (from >= L) return;
  const int n_blocks = (L + p.block - 1) / p.block;
  auto slot_of = [&](int j) {  // of this thread's position in block j
    const int64_t pos = static_cast<int64_t>(j) * p.block + tid;
    return tid < p.block && pos < L ? __ldg(p.slot_idx + static_cast<int64_t>(b) * p.slot_stride + pos) : -1;
  };
  const int j0 = from / p.block + blockIdx.x;
  int slot = slot_of(j0);
  for (int j = j0; j < n_blocks; j += gridDim.x) {
    const int pos0 = j * p.block, n = min(p.block, L - pos0);
    if (tid == 0) bad_sh[0] = bad_sh[1] = 0;
    __syncthreads();
    if (tid < n) {
      if (slot < 0 || slot >= p.pool_slots) {
        atomicOr(p.status, kStatusBadSlot);
        atomicAdd(&bad_sh[0], 1);
        slot = -1;
      }
      slot_sh[tid] = slot;
    }
    __syncthreads();
    slot = slot_of(j + gridDim.x);  // the next block's, while this one's rows travel
    uint64_t hi2[4], lo2[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) hi2[d] = lo2[d] = 0;
    for (int r0 = g; r0 < n; r0 += kSumGroups * kSumBatch) {
      uint4 v[kSumBatch];
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) {
        const int r = r0 + u * kSumGroups;
        const int s = r < n ? slot_sh[r] : -1;
        v[u] = s >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.kv + static_cast<int64_t>(s) * kDqk) + c)
                      : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int d = 0; d < 4; ++d)
          two_sum(hi2[d], lo2[d], f32x2(__uint_as_float(w[d] << 16), __uint_as_float(w[d] & 0xffff0000u)));
      }
    }
    if (g > 0) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        reinterpret_cast<uint64_t*>(part[g - 1][0])[4 * c + d] = hi2[d];
        reinterpret_cast<uint64_t*>(part[g - 1][1])[4 * c + d] = lo2[d];
      }
    }
    __syncthreads();
    // group 0 (72 threads) adds the others' sums and finishes the block
    const int count = n - bad_sh[0];
    const float rows = static_cast<float>(max(count, 1));
    float mean[8], am = 0.f;
    bool finite = true;
    if (g == 0) {
      float hi[8], lo[8];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
#pragma unroll
        for (int o = 0; o < kSumGroups - 1; ++o) {
          two_sum(hi2[d], lo2[d], reinterpret_cast<const uint64_t*>(part[o][0])[4 * c + d]);
          lo2[d] = add_x2(lo2[d], reinterpret_cast<const uint64_t*>(part[o][1])[4 * c + d]);
        }
        f32x2_split(hi2[d], hi[2 * d], hi[2 * d + 1]);
        f32x2_split(lo2[d], lo[2 * d], lo[2 * d + 1]);
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        // (hi + lo) / rows in fp32 pairs: the quotient of hi, and that of what is
        // left of hi and lo (64-bit division is slow here and would cost more than the sums)
        const float q = __fdiv_rn(hi[d], rows);
        const float m = __fadd_rn(q, __fdiv_rn(__fadd_rn(__fmaf_rn(-q, rows, hi[d]), lo[d]), rows));
        mean[d] = count > 0 ? m : 0.f;
        // an infinite row leaves a NaN in the carried error: any non-finite sum counts as such
        finite = finite && fabsf(mean[d]) < CUDART_INF_F;
        am = fmaxf(am, fabsf(mean[d]));
      }
    }
    if (tid < 96) {  // three warps hold the 72 threads
      const bool all = __all_sync(0xffffffffu, finite);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, off));
      if ((tid & 31) == 0) {
        amax_sh[tid >> 5] = am;
        if (!all) bad_sh[1] = 1;
      }
    }
    __syncthreads();
    if (g == 0) {
      am = fmaxf(fmaxf(amax_sh[0], amax_sh[1]), amax_sh[2]);
      const bool good = bad_sh[1] == 0;
      const float scale = good ? __fmul_rn(am, 1.f / 127.f) : CUDART_NAN_F;
      uint32_t w[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t two = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float q = 0.f;
          if (good && scale > 0.f) q = fminf(fmaxf(rintf(__fdiv_rn(mean[2 * d + e], scale)), -127.f), 127.f);
          two |= (__float_as_uint(q) >> 16) << (16 * e);  // an integer of 7 bits and sign: exact in bf16
        }
        w[d] = two;
      }
      const int64_t at = static_cast<int64_t>(b) * p.blocks + j;
      reinterpret_cast<uint4*>(p.summary + at * kDqk)[c] = make_uint4(w[0], w[1], w[2], w[3]);
      if (c == 0) p.scale[at] = scale;
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_block_summary(const SummaryParams& p, int batch, int sm_count, cudaStream_t stream) {
  if (batch == 0 || p.blocks == 0) return cudaSuccess;
  // blocks of a request are dealt to at most enough CTAs to fill the GPU: how
  // many are touched (from_len) is known on the device only
  const int64_t fill = (int64_t(sm_count) * kSumCtasPerSm + batch - 1) / batch;
  const unsigned gx = static_cast<unsigned>(p.blocks < fill ? p.blocks : fill);
  block_summary_kernel<<<dim3(gx, batch), kSumThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
