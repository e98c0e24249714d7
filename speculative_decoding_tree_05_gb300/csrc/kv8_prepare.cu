// kv8_prepare.cu -- what the units of attention over the 8-bit cache share: each group's
// query rows as the tensor core reads them, cut into two 8-bit parts once instead of once
// a unit, and the call's first status word.
//
// Four CTAs per (request, group of up to 64 rows) write the 72 KB that its units put into
// tensor and shared memory as they are, and a factor per row:
//   q = (hi + lo) 2^e in e4m3, 2^e the least power of two with |latent values| <= 448 2^e;
//   rope values q 2^-e in bf16.
// A warp a row; bound by latency (and the conversions, 16 a clock and SM), so a kernel of
// its own, that runs while the attention kernel sets itself up. (3 us of a call. Many groups
// are bound by their bytes: 1540 groups over 46 keys each 184 us in all, 195 with a CTA of 1024
// threads a group, two rows a warp.)
#include <cuda_runtime.h>
#include <math_constants.h>
#include "kv8.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kThreads = 512;
constexpr int kParts = kKv8Rows / (kThreads / 32);  // CTAs of a group, a warp a row

// Two query values, of 8 bits and at most 448, in two e4m3 parts; in f16 they are exact down to 2^-17 and in steps of
// 2^-24 below, which is finer than the second part's.
__device__ __forceinline__ void cut_query(float x, float y, uint32_t& hi, uint32_t& lo) {
  uint32_t h, back;
  uint16_t a, b;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(h));
  hi = a;
  lo = b;
}

__global__ void __launch_bounds__(kThreads) kv8_prepare_kernel(const __grid_constant__ Kv8PrepareParams p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.x / kParts, part_of = blockIdx.x % kParts, b = blockIdx.y;
  grid_dep_launch();
  const Kv8Group u = kv8_group(p.heads, p.group_nodes, kv8_nodes(p.tree_len, b, p.nodes), g);
  const int64_t row0 = static_cast<int64_t>(b) * p.nodes * p.heads + u.row0;
  uint8_t* image = p.images + (static_cast<int64_t>(b) * p.groups + g) * kKv8Image;
  if (u.rows > 0) {
    const int r = kThreads / 32 * part_of + warp;
    uint32_t w[9] = {};
    if (r < u.rows) {
      const uint16_t* src = p.q + (row0 + r) * kDqk;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + lane), y = __ldg(reinterpret_cast<const uint4*>(src + 256) + lane);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
      w[8] = __ldg(reinterpret_cast<const uint32_t*>(src + kDv) + lane);
    }
    // the largest magnitudes, latent and rope, as bf16 bits
    uint32_t top = 0, turned = w[8] & 0x7fff7fffu;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
    turned = __reduce_max_sync(0xffffffffu, max(turned & 0xffffu, turned >> 16));
    // a row that is not finite: zeros, and a factor of NaN for its own scores alone
    const bool fine = max(top, turned) < 0x7f80u;
    // 448 = 1.75 2^8 (7 bits stand behind the exponent); rope values stay below 2^121
    const int e = max(static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0),
                      max(static_cast<int>(turned >> 7) - 127 - 120, kKv8MinExp));
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    // A lane has dims 8 lane + {0..7} and 256 + 8 lane + {0..7}; with its neighbour, even lanes take 16 of the
    // first, odd lanes of the second half.
    uint32_t cut[2][4];  // [part][8 bytes of the first half, 8 of the second]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = fine ? w[4 * h + j] : 0u;
        cut_query(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv, hi[j], lo[j]);
      }
      cut[0][2 * h] = hi[0] | (hi[1] << 16), cut[0][2 * h + 1] = hi[2] | (hi[3] << 16);
      cut[1][2 * h] = lo[0] | (lo[1] << 16), cut[1][2 * h + 1] = lo[2] | (lo[3] << 16);
    }
    const bool odd = lane & 1;
    const uint32_t v = fine ? w[8] : 0u;
    const uint32_t rope = pack_bf16x2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int l = 32 * (r >> 4) + (r & 15) + 16 * part, piece = (lane >> 1) + (odd ? 16 : 0);
      const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? cut[part][0] : cut[part][2], 1);
      const uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? cut[part][1] : cut[part][3], 1);
      *reinterpret_cast<uint4*>(image + (128 * piece + l) * 16) =
          odd ? make_uint4(x, y, cut[part][2], cut[part][3]) : make_uint4(cut[part][0], cut[part][1], x, y);
    }
    *reinterpret_cast<uint32_t*>(image + kKv8ImageRope + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | ((lane & 3) << 2))) = rope;
    if (lane == 0)
      reinterpret_cast<float*>(image + kKv8ImageFactor)[r] =
          r >= u.rows ? 0.f : fine ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * p.scale_log2 : CUDART_NAN_F;
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
  kv8_prepare_kernel<<<dim3(kParts * p.groups, p.batch), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
