// kv8_rows.cu -- rows into the 8-bit latent cache and back.
//
// In: a row x = (c, r) of 512 latent and 64 rope values becomes
//   c' = c / sqrt(mean(c^2) + eps) * w    (if it is to be normalised)
//   r' = r turned by its position's angles (if it is to be rotated)
//   s  = the least power of two with max |c'| <= 448 s, 448 being e4m3's largest value
//   slot = e4m3(c' / s), bf16(r' / s), scale s.
// All of it is fp32 up to the one rounding of each value. A power of two makes the
// quotients and the way back exact, and in a floating format a finer scale would win
// nothing but the last subnormal step.
// Out: value * s, rounded to bf16 (exact for such s, short of bf16's subnormals).
//
// One warp a row, 16 latent values a lane; no shared memory. Bound by HBM: 1152 + 644
// bytes a row in, 644 + 1152 out.
#include <cuda_runtime.h>
#include <math_constants.h>
#include "kv8.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kRowWarps = 8;

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// a + b to a; returns what the rounding left
__device__ __forceinline__ float add_exact(float& a, float b) {
  const float s = a + b, part = s - a, rest = (a - (s - part)) + (b - part);
  a = s;
  return rest;
}

// kPairs: the rope values (2 i, 2 i + 1) turn together, else (i, i + 32).
template <bool kPairs>
__global__ void __launch_bounds__(kRowWarps * 32) kv8_write_kernel(const __grid_constant__ Kv8WriteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;
  const uint16_t* row = p.rows + i * p.row_stride;
  const int slot = __ldg(p.slots + i);
  const int at = p.rotation ? __ldg(p.position + i) : 0;
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(row) + lane), b = __ldg(reinterpret_cast<const uint4*>(row + 256) + lane);
  float rx, ry;
  if (kPairs) {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(row + kDv) + lane);
    rx = bf16_lo(v), ry = bf16_hi(v);
  } else {
    rx = bf16_lo(__ldg(row + kDv + lane)), ry = bf16_lo(__ldg(row + kDv + kRopePairs + lane));
  }
  const bool bad_slot = slot != -1 && (slot < 0 || slot >= p.pool_slots);
  const bool bad_position = p.rotation && (at < 0 || at >= p.positions);
  if (slot == -1 || bad_slot || bad_position) {
    const int32_t bits = slot == -1 ? 0 : (bad_slot ? kStatusBadSlot : 0) | (bad_position ? kStatusBadPosition : 0);
    if (bits && lane == 0) atomicOr(p.status, bits);
    return;
  }
  float x[16];  // latent values 8 lane + {0..7} and 256 + 8 lane + {0..7}
  unpack8(a, x);
  unpack8(b, x + 8);
  if (p.norm_weight) {
    float w[16];
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.norm_weight) + lane), w);
    unpack8(__ldg(reinterpret_cast<const uint4*>(p.norm_weight + 256) + lane), w + 8);
    // (rows whose squares would leave fp32 are first made smaller, by a power of two)
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]));
    const float fit = warp_max(top) > pow2(50) ? pow2(-80) : 1.f;
    // Sum and root carry what their roundings leave, so that c' is rounded once: a value next to a border between two
    // 8-bit values goes where the formula puts it. (Squares and products of two bf16 values are exact in fp32.)
    uint64_t hi = f32x2(0.f, 0.f), lo = hi;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[2 * k] *= fit, x[2 * k + 1] *= fit;
      const uint64_t v = f32x2(x[2 * k], x[2 * k + 1]), sq = mul_x2(v, v), sum = add_x2(hi, sq), part = sub_x2(sum, hi);
      lo = add_x2(lo, add_x2(sub_x2(hi, sub_x2(sum, part)), sub_x2(sq, part)));
      hi = sum;
    }
    float h, l, h2, l2;
    f32x2_split(hi, h, h2);
    f32x2_split(lo, l, l2);
    l += l2 + add_exact(h, h2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      h2 = __shfl_xor_sync(0xffffffffu, h, o);
      l += __shfl_xor_sync(0xffffffffu, l, o);
      l += add_exact(h, h2);
    }
    h *= 1.f / kDv, l *= 1.f / kDv;
    l += add_exact(h, p.eps * fit * fit);
    const float y = rsqrtf(h), t = h * y;
    // one step towards the root's last bits: y (1 + r / 2), r = 1 - (h + l) y^2
    const float r = fmaf(-l * y, y, fmaf(-fmaf(h, y, -t), y, fmaf(-t, y, 1.f))), more = 0.5f * y * r;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float c = x[k] * w[k];
      x[k] = fmaf(c, y, c * more);
    }
  }
  if (p.rotation) {
    const float* turn = p.rotation + static_cast<int64_t>(at) * (2 * kRopePairs) + lane;
    const float c = __ldg(turn), s = __ldg(turn + kRopePairs);
    // (each rounded once but for the last sum)
    const float ys = ry * s, xs = rx * s;
    const float tx = fmaf(rx, c, -ys) + fmaf(-ry, s, ys);
    ry = fmaf(ry, c, xs) + fmaf(rx, s, -xs);
    rx = tx;
  }
  float top = 0.f, rope = fmaxf(fabsf(rx), fabsf(ry));
  bool fine = fabsf(rx) <= 3.4028235e38f && fabsf(ry) <= 3.4028235e38f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    top = fmaxf(top, fabsf(x[k]));
    fine = fine && fabsf(x[k]) <= 3.4028235e38f;
  }
  fine = __all_sync(0xffffffffu, fine);
  const uint32_t u = __float_as_uint(warp_max(top)), r = __float_as_uint(warp_max(rope));
  // 448 = 1.75 * 2^8; rope quotients stay below 2^121
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, max(static_cast<int>(r >> 23) - 127 - 120, kKv8MinExp));
  const float inv = pow2(-e);
  uint8_t* dst = p.pool + static_cast<int64_t>(slot) * kKv8Row;
  // a row that is not finite: a scale of NaN, and zeros (which do not spread to others through a product with 0)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* y = x + 8 * h + 4 * k;
      v[k] = fine ? pack_e4m3x2(y[0] * inv, y[1] * inv) | (static_cast<uint32_t>(pack_e4m3x2(y[2] * inv, y[3] * inv)) << 16) : 0u;
    }
    *reinterpret_cast<uint2*>(dst + 256 * h + 8 * lane) = make_uint2(v[0], v[1]);
  }
  const uint32_t rope2 = fine ? pack_bf16x2(rx * inv, ry * inv) : 0u;
  uint16_t* rdst = reinterpret_cast<uint16_t*>(dst + kDv);
  if (kPairs) {
    reinterpret_cast<uint32_t*>(rdst)[lane] = rope2;
  } else {
    rdst[lane] = static_cast<uint16_t>(rope2);
    rdst[kRopePairs + lane] = static_cast<uint16_t>(rope2 >> 16);
  }
  if (lane == 0) p.scale[slot] = fine ? pow2(e) : CUDART_NAN_F;
}

__global__ void __launch_bounds__(kRowWarps * 32) kv8_read_kernel(const __grid_constant__ Kv8ReadParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;
  const int slot = __ldg(p.slots + i);
  const bool in = slot >= 0 && slot < p.pool_slots;
  if (!in && slot != -1 && lane == 0) atomicOr(p.status, kStatusBadSlot);
  uint4 a = make_uint4(0, 0, 0, 0);
  uint32_t r = 0;
  float s = 0.f;
  if (in) {
    const uint8_t* src = p.pool + static_cast<int64_t>(slot) * kKv8Row;
    a = __ldg(reinterpret_cast<const uint4*>(src) + lane);
    r = __ldg(reinterpret_cast<const uint32_t*>(src + kDv) + lane);
    s = __ldg(p.scale + slot);
  }
  const uint32_t in4[4] = {a.x, a.y, a.z, a.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float x, y;
    unpack_e4m3x2(static_cast<uint16_t>(in4[k >> 1] >> (16 * (k & 1))), x, y);
    o[k] = pack_bf16x2(x * s, y * s);
  }
  uint16_t* dst = p.rows + i * p.row_stride;
  uint4* d4 = reinterpret_cast<uint4*>(dst) + 2 * lane;
  d4[0] = make_uint4(o[0], o[1], o[2], o[3]);
  d4[1] = make_uint4(o[4], o[5], o[6], o[7]);
  reinterpret_cast<uint32_t*>(dst + kDv)[lane] = pack_bf16x2(bf16_lo(r) * s, bf16_hi(r) * s);
}

unsigned row_blocks(int64_t n) { return static_cast<unsigned>((n + kRowWarps - 1) / kRowWarps); }

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteParams& p, bool interleaved, cudaStream_t stream) {
  if (interleaved)
    kv8_write_kernel<true><<<row_blocks(p.n), kRowWarps * 32, 0, stream>>>(p);
  else
    kv8_write_kernel<false><<<row_blocks(p.n), kRowWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8ReadParams& p, cudaStream_t stream) {
  kv8_read_kernel<<<row_blocks(p.n), kRowWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
