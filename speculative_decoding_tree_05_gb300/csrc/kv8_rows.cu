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
// bytes a row in, 644 + 1152 out. (60001 rows in and back 51 us, 4.5 TB/s, the way in 33 of
// them: 28 warps an SM, each with its next row on the way, behind the sums that a row waits for;
// 185000 scattered rows back 55 us, 6.0 TB/s.)
#include <cuda_runtime.h>
#include <math_constants.h>
#include <algorithm>
#include "kv8.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kRowWarps = 4;
constexpr int kWriteBlocks = 7;  // blocks of an SM (72 registers)

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 <= e <= 127

// a + b to a; returns what the rounding left
__device__ __forceinline__ float add_exact(float& a, float b) {
  const float s = a + b, part = s - a, rest = (a - (s - part)) + (b - part);
  a = s;
  return rest;
}

// What a lane has of a row: latent values 8 lane + {0..7} and 256 + 8 lane + {0..7}, two rope values.
struct RowLane {
  uint4 a, b;
  uint32_t rope;
  int slot, at;
};

// kPairs: the rope values (2 i, 2 i + 1) turn together, else (i, i + 32).
template <bool kPairs, bool kNorm>
__global__ void __launch_bounds__(kRowWarps * 32, kWriteBlocks) kv8_write_kernel(const __grid_constant__ Kv8WriteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowWarps;
  int64_t i = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;
  auto load = [&](int64_t i) {
    const uint16_t* row = p.rows + i * p.row_stride;
    RowLane v;
    v.slot = __ldg(p.slots + i);
    v.at = p.rotation ? __ldg(p.position + i) : 0;
    v.a = __ldg(reinterpret_cast<const uint4*>(row) + lane);
    v.b = __ldg(reinterpret_cast<const uint4*>(row + 256) + lane);
    if (kPairs)
      v.rope = __ldg(reinterpret_cast<const uint32_t*>(row + kDv) + lane);
    else
      v.rope = __ldg(row + kDv + lane) | (static_cast<uint32_t>(__ldg(row + kDv + kRopePairs + lane)) << 16);
    return v;
  };
  uint32_t w[8];  // the norm's weights of the lane's values, two by two
  if (kNorm) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.norm_weight) + lane), y = __ldg(reinterpret_cast<const uint4*>(p.norm_weight + 256) + lane);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
  // the angles a row's position has, read when the position has come
  auto turn_of = [&](int at, float& c, float& s) {
    if (p.rotation && at >= 0 && at < p.positions) {
      const float* turn = p.rotation + static_cast<int64_t>(at) * (2 * kRopePairs) + lane;
      c = __ldg(turn);
      s = __ldg(turn + kRopePairs);
    }
  };
  RowLane next = load(i);
  float c = 1.f, s = 0.f;
  turn_of(next.at, c, s);
#pragma unroll 1
  for (; i < p.n; i += step) {
    const RowLane v = next;
    if (i + step < p.n) next = load(i + step);
    float rx = bf16_lo(v.rope), ry = bf16_hi(v.rope);
    if (p.rotation) {
      // (each rounded once but for the last sum)
      const float ys = ry * s, xs = rx * s;
      const float tx = fmaf(rx, c, -ys) + fmaf(-ry, s, ys);
      ry = fmaf(ry, c, xs) + fmaf(rx, s, -xs);
      rx = tx;
    }
    const uint32_t in[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
    uint64_t x[8];  // two by two
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = f32x2(bf16_lo(in[k]), bf16_hi(in[k]));
    if (kNorm) {
      // The root of the mean square, to its last bits, so that c' is rounded once and a value next to a border between
      // two 8-bit values goes where the formula puts it: the row is first divided by a power of two, to values below 2
      // (at least 2^-40: eps is all that counts in smaller rows). Their squares, exact in fp32, are added onto 2^12,
      // where every sum is a multiple of 2^-11 and so exact over the whole row; what each leaves is added apart.
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = __vmaxu2(m, in[k] & 0x7fff7fffu);
      m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      const int e = min(max(static_cast<int>(m >> 7) - 127, -40), 126);  // (a row that is not finite: anything)
      const float fit = pow2(-e);
      const uint64_t fit2 = f32x2(fit, fit), origin = f32x2(4096.f, 4096.f);
      uint64_t hi = origin, lo = f32x2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = mul_x2(x[k], fit2);
        const uint64_t sq = mul_x2(x[k], x[k]), sum = add_x2(hi, sq);
        lo = add_x2(lo, sub_x2(sq, sub_x2(sum, hi)));
        hi = sum;
      }
      float h, l, h2, l2;
      f32x2_split(sub_x2(hi, origin), h, h2);
      f32x2_split(lo, l, l2);
      h += h2, l += l2;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        h += __shfl_xor_sync(0xffffffffu, h, o);
        l += __shfl_xor_sync(0xffffffffu, l, o);
      }
      h *= 1.f / kDv, l *= 1.f / kDv;
      l += add_exact(h, p.eps * fit * fit);
      l = add_exact(h, l);
      const float y = rsqrtf(h), t = h * y;
      // one step towards the root's last bits: y (1 + r / 2), r = 1 - (h + l) y^2
      const float r = fmaf(-l * y, y, fmaf(-fmaf(h, y, -t), y, fmaf(-t, y, 1.f))), more = 0.5f * y * r;
      const uint64_t y2 = f32x2(y, y), more2 = f32x2(more, more);
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // (the product of two bf16 values is exact)
        const uint64_t c = mul_x2(x[k], f32x2(bf16_lo(w[k]), bf16_hi(w[k])));
        x[k] = fma_x2(c, y2, mul_x2(c, more2));
      }
    }
    if (i + step < p.n) turn_of(next.at, c, s);
    float top = 0.f, none = fmaf(rx, 0.f, ry * 0.f);  // none: NaN if a value is not finite
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, b;
      f32x2_split(x[k], a, b);
      top = fmax3(top, fabsf(a), fabsf(b));
      none = fmaf(a, 0.f, fmaf(b, 0.f, none));
    }
    const bool fine = __all_sync(0xffffffffu, none == 0.f);
    const uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(top)),
                   r = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(rx), fabsf(ry))));
    // 448 = 1.75 * 2^8; rope quotients stay below 2^121
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, max(static_cast<int>(r >> 23) - 127 - 120, kKv8MinExp));
    const float inv = fine ? pow2(-e) : 0.f;
    const uint64_t inv2 = f32x2(inv, inv);
    const bool bad_slot = v.slot != -1 && (v.slot < 0 || v.slot >= p.pool_slots);
    const bool bad_position = p.rotation && (v.at < 0 || v.at >= p.positions);
    if (v.slot == -1 || bad_slot || bad_position) {
      const int32_t bits = v.slot == -1 ? 0 : (bad_slot ? kStatusBadSlot : 0) | (bad_position ? kStatusBadPosition : 0);
      if (bits && p.status && lane == 0) atomicOr(p.status, bits);
      continue;
    }
    uint8_t* dst = p.pool + static_cast<int64_t>(v.slot) * kKv8Row;
    // a row that is not finite: a scale of NaN, and zeros (which do not spread to others through a product with 0)
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b, c, d;
      f32x2_split(mul_x2(x[2 * k], inv2), a, b);
      f32x2_split(mul_x2(x[2 * k + 1], inv2), c, d);
      out[k] = fine ? pack_e4m3x2(a, b) | (static_cast<uint32_t>(pack_e4m3x2(c, d)) << 16) : 0u;
    }
    *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(out[0], out[1]);
    *reinterpret_cast<uint2*>(dst + 256 + 8 * lane) = make_uint2(out[2], out[3]);
    const uint32_t rope2 = fine ? pack_bf16x2(rx * inv, ry * inv) : 0u;
    uint16_t* rdst = reinterpret_cast<uint16_t*>(dst + kDv);
    if (kPairs) {
      reinterpret_cast<uint32_t*>(rdst)[lane] = rope2;
    } else {
      rdst[lane] = static_cast<uint16_t>(rope2);
      rdst[kRopePairs + lane] = static_cast<uint16_t>(rope2 >> 16);
    }
    if (lane == 0) p.scale[v.slot] = fine ? pow2(e) : CUDART_NAN_F;
  }
}

__global__ void __launch_bounds__(kRowWarps * 32) kv8_read_kernel(const __grid_constant__ Kv8ReadParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (i >= p.n) return;
  const int slot = __ldg(p.slots + i);
  const bool in = slot >= 0 && slot < p.pool_slots;
  if (!in && slot != -1 && p.status && lane == 0) atomicOr(p.status, kStatusBadSlot);
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

cudaError_t launch_kv8_write(const Kv8WriteParams& p, bool interleaved, int sm_count, cudaStream_t stream) {
  // as many blocks as run at once: a warp has its next row on the way while it works at one
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(row_blocks(p.n), int64_t(sm_count) * kWriteBlocks));
  if (p.norm_weight) {
    if (interleaved)
      kv8_write_kernel<true, true><<<blocks, kRowWarps * 32, 0, stream>>>(p);
    else
      kv8_write_kernel<false, true><<<blocks, kRowWarps * 32, 0, stream>>>(p);
  } else if (interleaved) {
    kv8_write_kernel<true, false><<<blocks, kRowWarps * 32, 0, stream>>>(p);
  } else {
    kv8_write_kernel<false, false><<<blocks, kRowWarps * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8ReadParams& p, cudaStream_t stream) {
  kv8_read_kernel<<<row_blocks(p.n), kRowWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
