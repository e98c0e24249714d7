// kv8_cut.cuh -- a query row as the attention over the 8-bit cache takes it, by one warp.
#pragma once
#include <math_constants.h>
#include "kv8.cuh"
#include "ptx.cuh"

namespace ddt {

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

// A row's values as a lane reads them: dims 8 lane + {0..7}, 256 + 8 lane + {0..7}, two rope values; null: zeros.
__device__ __forceinline__ void load_query(const uint16_t* src, int lane, uint32_t (&w)[9]) {
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  w[8] = 0;
  if (src) {
    x = __ldg(reinterpret_cast<const uint4*>(src) + lane), y = __ldg(reinterpret_cast<const uint4*>(src + 256) + lane);
    w[8] = __ldg(reinterpret_cast<const uint32_t*>(src + kDv) + lane);
  }
  w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
}

// Of the row, the lane's 16-byte piece of either part (the parts' piece query_piece(lane)), its pair of rope values and
// the row's factor of a score, NaN for a row that is not finite (which is zeros otherwise).
struct CutQuery {
  uint4 part[2];
  uint32_t rope;
  float factor;
};
__device__ __forceinline__ int query_piece(int lane) { return (lane >> 1) + (lane & 1 ? 16 : 0); }
// where row r's rope values of the lane stand in its 128-byte row, swizzled
__device__ __forceinline__ int query_rope_at(int r, int lane) {
  return r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | ((lane & 3) << 2));
}
__device__ __forceinline__ CutQuery cut_row(const uint32_t (&w)[9], int lane, float scale_log2) {
  CutQuery o;
  // the largest magnitudes, latent and rope, as bf16 bits
  uint32_t top = 0, turned = w[8] & 0x7fff7fffu;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  turned = __reduce_max_sync(0xffffffffu, max(turned & 0xffffu, turned >> 16));
  // a row that is not finite: zeros, and a factor of NaN for its own scores alone
  const bool fine = max(top, turned) < 0x7f80u;
  // 448 = 1.75 2^8 (7 bits stand behind the exponent); rope values stay below 2^48, as those of a key without latent values
  // (whose scale is 2^-60) are large: products of up to 2^73 of them stay inside fp32
  const int e = max(static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0),
                    max(static_cast<int>(turned >> 7) - 127 - 47, kKv8MinExp));
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  // With its neighbour, even lanes take 16 dims of the first, odd lanes of the second half.
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
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? cut[part][0] : cut[part][2], 1);
    const uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? cut[part][1] : cut[part][3], 1);
    o.part[part] = odd ? make_uint4(x, y, cut[part][2], cut[part][3]) : make_uint4(cut[part][0], cut[part][1], x, y);
  }
  const uint32_t v = fine ? w[8] : 0u;
  o.rope = pack_bf16x2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv);
  o.factor = fine ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * scale_log2 : CUDART_NAN_F;
  return o;
}

// The tensor memory's lane of a row's part.
__device__ __forceinline__ int query_lane(int r, int part) { return 32 * (r >> 4) + (r & 15) + 16 * part; }

}  // namespace ddt
