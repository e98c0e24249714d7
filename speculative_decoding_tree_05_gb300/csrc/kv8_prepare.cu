// kv8_prepare.cu -- what the units of attention over the 8-bit cache share: each group's
// query rows as the tensor core reads them, cut into two 8-bit parts once instead of once
// a unit, and the call's first status word.
//
// Four CTAs per (request, group of up to 64 rows) write the 72 KB that its units put into
// tensor and shared memory as they are, and a factor per row:
//   q = (hi + lo) 2^e in e4m3, 2^e the least power of two with |latent values| <= 448 2^e;
//   rope values q 2^-e in bf16.
// A warp a row; bound by latency (and the conversions, 16 a clock and SM), so a kernel of
// its own, that runs while the attention kernel sets itself up: 3 us of a call.
#include <cuda_runtime.h>
#include <math_constants.h>
#include "kv8_cut.cuh"

namespace ddt {
namespace {

constexpr int kThreads = 512;
constexpr int kParts = kKv8Rows / (kThreads / 32);  // CTAs of a group, a warp a row

__global__ void __launch_bounds__(kThreads) kv8_prepare_kernel(const __grid_constant__ Kv8PrepareParams p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y;
  const int g = p.images ? blockIdx.x / kParts : blockIdx.x, part_of = p.images ? blockIdx.x % kParts : kParts - 1;
  grid_dep_launch();
  const Kv8Group u = kv8_group(p.heads, p.group_nodes, kv8_nodes(p.tree_len, b, p.nodes), g);
  const int64_t row0 = static_cast<int64_t>(b) * p.nodes * p.heads + u.row0;
  uint8_t* image = p.images + (static_cast<int64_t>(b) * p.groups + g) * kKv8Image;
  if (p.images && u.rows > 0) {
    const int r = kThreads / 32 * part_of + warp;
    uint32_t w[9];
    load_query(r < u.rows ? p.q + (row0 + r) * kDqk : nullptr, lane, w);
    const CutQuery c = cut_row(w, lane, p.scale_log2);
#pragma unroll
    for (int part = 0; part < 2; ++part)
      *reinterpret_cast<uint4*>(image + (128 * query_piece(lane) + query_lane(r, part)) * 16) = c.part[part];
    *reinterpret_cast<uint32_t*>(image + kKv8ImageRope + query_rope_at(r, lane)) = c.rope;
    if (lane == 0) reinterpret_cast<float*>(image + kKv8ImageFactor)[r] = r < u.rows ? c.factor : 0.f;
  }
  if (part_of != kParts - 1) return;  // (the last has the fewest rows)
  // rows of nodes that are not active
  const int all = kv8_group(p.heads, p.group_nodes, p.nodes, g).rows, live = max(u.rows, 0);
  if (live < all) {
    uint4* o = reinterpret_cast<uint4*>(p.out + (row0 + live) * kDv);
    for (int i = tid; i < (all - live) * (kDv / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (tid < all - live) p.lse[row0 + live + tid] = -CUDART_INF_F;
  }
  if (g == 0 && b == 0) {  // the first of the call's status bits, as a whole word
    int bits = 0;
    for (int i = tid; i < p.batch; i += kThreads) {
      const int L = __ldg(p.prefix_len + i);
      if (L < 0 || L > p.max_prefix_len) bits |= kStatusBadPrefix;
      const int n = p.tree_len ? __ldg(p.tree_len + i) : 0;
      if (n < 0 || n > p.nodes) bits |= kStatusBadTreeLen;
    }
    const int prefix = __syncthreads_or(bits & kStatusBadPrefix), tree = __syncthreads_or(bits & kStatusBadTreeLen);
    if (tid == 0) *p.status = (prefix ? kStatusBadPrefix : 0) | (tree ? kStatusBadTreeLen : 0);
  }
}

}  // namespace

cudaError_t launch_kv8_prepare(const Kv8PrepareParams& p, cudaStream_t stream) {
  // without images: for the rows of inactive nodes, or for the status word alone
  const dim3 grid = p.images ? dim3(kParts * p.groups, p.batch) : p.tree_len ? dim3(p.groups, p.batch) : dim3(1);
  kv8_prepare_kernel<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
