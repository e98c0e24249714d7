// accept.cu -- the drafted tokens of a tree against the target's probabilities, from given random numbers.
//
// At node v the target's next token has p(x) = softmax(logits[v] / temperature). v's
// children are tried in node order: with w the part of p that is left and S its sum, child
// c with token x is accepted if u_c S q(x) < w(x). Drafted tokens that were picked (the
// drafter's best) have q = 1, and a refused one leaves w without x; tokens that were drawn
// from the drafter's distribution q leave max(w - S q, 0), which after several refusals is
// max(w - T q, 0) of the first w, T the sum of their S. Either way the accepted path and the
// token after it follow p exactly. Where no child is accepted the next token is
// the first x with w(0) + ... + w(x) > u_0 S.
//
// Weights are whole numbers: w(x) = 2^((l(x) - max l) log2 e / temperature) in steps of
// 2^-43, their exponent carried in two floats (2 10^-9 of each weight; in one where the weight is below 2^-24, which is
// off by a step or so). So sums are exact in any order, the same tokens come out on any tiling, and a token on the border
// between two answers is decided as 64-bit arithmetic decides it, but for one draw in 10^5 or so.
//
// One cluster per request walks down the tree and reads only the rows that it visits,
// each CTA its share of the vocabulary, which stays in shared memory (logits; with q the
// weights and q) from the maximum to the draw. Each warp has a range of consecutive tokens
// and its sum, so a draw is a prefix over CTAs and warps and one warp's look at its range.
// Bound by the latency of a visit: a row's load, and the two sums over the cluster (its
// maximum, its weights); a refused token that was drawn is one more. The children's rows are
// on their way to L2 meanwhile. (One chain of 9 over 32768 tokens 14.5 us, 8 trees of 65 over
// 131072 34, 16 drawn ones of 9 over 128001 63; about 9000 cycles a visit.)
#include <cuda_runtime.h>
#include <math_constants.h>
#include <algorithm>
#include "accept.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kAccThreads = 512, kAccWarps = kAccThreads / 32;
constexpr int kOne = 43;         // weight 1 is 2^43; up to 2^18 of them fit in 64 bits
constexpr float kNear = 24.f;    // from 2^-kNear on, plain powers
constexpr int kUnroll = 16;      // loads in flight of a thread

// 2^(62 - i / 16), i = 0 to 15: as many as lie in different banks
constexpr int kPowers = 16;
__constant__ unsigned long long c_pow[kPowers] = {
    0x4000000000000000ull, 0x3d495f454921b30bull, 0x3ab031b9f7490e4cull, 0x383337bb0aa53844ull,
    0x35d13f32b5a75abdull, 0x3389230547e12039ull, 0x3159ca845541b6b7ull, 0x2f4228e7d6030db0ull,
    0x2d413cccfe779921ull, 0x2b560fba90a852b2ull, 0x297fb5aa6c544e3bull, 0x27bd4c982468446bull,
    0x260dfc14636e2a5cull, 0x2470f4dceac470ceull, 0x22e57078faa2f5baull, 0x216ab0d9f3121ec5ull,
};

// Whole numbers by an addition, where a conversion instruction takes four times as long: x + kWhole is rounded to one
// (|x| <= 2^22), and its bits count on from kWhole's.
constexpr float kWhole = 12582912.f;  // 1.5 2^23
__device__ __forceinline__ int whole_bits(float x_plus) { return __float_as_int(x_plus) - __float_as_int(kWhole); }

// 2^-(hi + lo) in steps of 2^-43, rounded down; 0 <= hi <= 24, |lo| small. `pow_sh` is c_pow in shared memory.
__device__ __forceinline__ unsigned long long weight_of(float hi, float lo, const unsigned long long* pow_sh) {
  const float kp = fmaf(hi, kPowers, kWhole);
  const int ki = whole_bits(kp);
  const float r = fmaf(kp - kWhole, -1.f / kPowers, hi) + lo;  // (the first difference is exact)
  // 2^-r - 1, |r| <= 2^-5, to 2^-29: its error is the weight's
  const float z = r * -0.69314718055994531f;
  const float g = fmaf(z * z, fmaf(z, fmaf(z, 1.f / 24, 1.f / 6), 0.5f), z);
  const int gi = __float2int_rn(g * 68719476736.f);  // 2^36
  const long long top = static_cast<long long>(pow_sh[ki & (kPowers - 1)]);
  const long long w = top + ((static_cast<long long>(static_cast<int>(top >> 32)) * gi) >> 4);
  return static_cast<unsigned long long>(w) >> ((62 - kOne) + (ki / kPowers));
}

// A row's weights: 2^((l - max) c) with c = log2 e / temperature in two floats, or all of it on one token.
struct RowWeight {
  float max, c_hi, c_lo;
  int only;  // greedy: the token; else -1
  // of token x, whose distance from the largest logit is y in units of a halving
  __device__ __forceinline__ float distance(float l) const { return max - l < CUDART_INF_F ? (max - l) * c_hi : CUDART_INF_F; }
  __device__ __forceinline__ unsigned long long exactly(float l, float y, const unsigned long long* pow_sh) const {
    const float d = max - l, b = d - max, e = (max - (d - b)) - (l + b);  // max - l = d + e exactly
    return weight_of(y, fmaf(d, c_hi, -y) + fmaf(d, c_lo, e * c_hi), pow_sh);
  }
  // Most tokens are far below the largest: a plain power in steps of 2^-43, of at most 2^-24, is within a step or so.
  static __device__ __forceinline__ unsigned long long plainly(float y) {
    return static_cast<uint32_t>(whole_bits(fast_exp2(fminf(kOne - y, kOne - kNear)) + kWhole));
  }
  __device__ __forceinline__ unsigned long long operator()(float l, int x, const unsigned long long* pow_sh) const {
    if (only >= 0) return x == only ? 1ull << kOne : 0;
    const float y = distance(l);
    return y < kNear ? exactly(l, y, pow_sh) : plainly(y);
  }
};
__device__ __forceinline__ RowWeight row_weight(float temperature) {
  RowWeight r;
  r.max = 0.f;
  r.only = -1;
  // log2 e / temperature in two floats
  constexpr float kHi = 1.44269502e+00f, kLo = 1.92596303e-08f;
  r.c_hi = temperature > 0.f ? fminf(kHi / temperature, 1e30f) : 0.f;
  r.c_lo = r.c_hi > 0.f && r.c_hi < 1e30f ? (fmaf(-r.c_hi, temperature, kHi) + kLo) / temperature : 0.f;
  return r;
}

// floor(S u) for u in [0, 1]
__device__ __forceinline__ unsigned long long share_of(unsigned long long S, float u) {
  if (u >= 1.f) return S;
  const uint32_t v = __float_as_uint(u);
  const int e = static_cast<int>(v >> 23);  // at most 126
  const unsigned long long mant = e > 0 ? (v & 0x7fffffu) | 0x800000u : 0;
  return e < 63 ? 0 : __umul64hi(S, mant << 40) >> (126 - e);
}
// 16 T q for many probabilities q in [0, 1], from the 32 leading bits of T: 2^-32 of it off
struct Shares {
  uint32_t top;
  int shift;  // 16 T is top 2^shift
  __device__ __forceinline__ explicit Shares(unsigned long long T) {
    shift = max(0, 32 - __clzll(T));
    top = static_cast<uint32_t>(T >> shift);
    shift += 4;
  }
  __device__ __forceinline__ unsigned long long operator()(float q) const {
    const uint32_t v = __float_as_uint(q);
    const int by = 158 - shift - static_cast<int>(v >> 23);  // q is (2^23 + its last bits) 2^(exponent - 150)
    const unsigned long long x = static_cast<unsigned long long>(top) * ((v & 0x7fffffu) | 0x800000u) << 8;
    return by > 63 ? 0 : by < 0 ? ~0ull : x >> by;
  }
};
__device__ __forceinline__ unsigned long long less(unsigned long long w, unsigned long long s) { return w > s ? w - s : 0; }

__device__ __forceinline__ float logit(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16); }
__device__ __forceinline__ float logit(const float* p) { return __ldg(p); }
// The same, issued where it stands (an ordinary load moves down to its use, behind the row).
__device__ __forceinline__ float logit_now(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ float logit_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
// NaN counts as -inf, +inf as the largest number
__device__ __forceinline__ float tame(float l) { return l >= -3.4028235e38f ? fminf(l, 3.4028235e38f) : -CUDART_INF_F; }

// u in [0, 1), NaN as 0
__device__ __forceinline__ float tame_uniform(float u) { return u > 0.f ? fminf(u, 0.99999994f) : 0.f; }

// The order of logits as whole numbers, the lower index first among equals; and the logit again.
__device__ __forceinline__ unsigned long long order_of(float l, int x) {
  const uint32_t u = __float_as_uint(l);
  const uint32_t key = l == 0.f ? 0x80000000u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(x));
}
__device__ __forceinline__ float max_of(unsigned long long order) {
  const uint32_t key = static_cast<uint32_t>(order >> 32);
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Over a warp, by 16 or 32 bits at a time.
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32), top = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<unsigned long long>(top) << 32) | lo;
}
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  unsigned long long sum = 0;
#pragma unroll
  for (int i = 0; i < 64; i += 16)
    sum += static_cast<unsigned long long>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> i) & 0xffffu)) << i;
  return sum;
}
template <typename T, bool kDrawn>
__global__ void __launch_bounds__(kAccThreads, 2) accept_kernel(const __grid_constant__ AcceptParams p) {
  extern __shared__ unsigned long long dyn_sh[];  // kDrawn: weights, then q; else logits
  __shared__ unsigned long long pow_sh[kPowers];
  // Every warp's part of a reduction, of the whole cluster; two, used in turn: a warp sends its part of the next one when
  // it has read this one, so a part is written again when all have read it.
  __shared__ unsigned long long part_sh[2][kAcceptCluster * kAccWarps];
  __shared__ uint64_t part_bar[2];  // their bytes have come
  __shared__ unsigned long long child_w[kMaxNodes];  // of the nodes that are children
  __shared__ float u_sh[kMaxNodes], child_q[kMaxNodes];
  __shared__ int par_sh[kMaxNodes], tok_sh[kMaxNodes], path_sh[kMaxNodes], bits_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int size = p.cluster, rank = blockIdx.x % size, b = blockIdx.x / size;
  if (tid == 0) {
    mbar_init(&part_bar[0], 1);
    mbar_init(&part_bar[1], 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (size > 1) cluster_arrive();  // (others write to this CTA's shared memory: it has to be there)
  const int64_t node0 = static_cast<int64_t>(b) * p.nodes;
  const int given = p.tree_len ? __ldg(p.tree_len + b) : p.nodes, nodes = min(max(given, 0), p.nodes);
  // this CTA's share of the vocabulary, this warp's range of it
  const int lo = min(p.vocab, rank * p.share), hi = min(p.vocab, lo + p.share);
  const int wlo = min(hi, lo + warp * p.warp_share), whi = min(hi, wlo + p.warp_share);
  // sends for this CTA's share of a node's rows, in 128-byte lines
  auto prefetch = [&](int node, int first, int step) {  // by threads first, first + 1, .. of step
    constexpr int kLine = 128 / sizeof(T);
    const T* row = static_cast<const T*>(p.logits) + (node0 + node) * p.logit_stride;
    for (int x = lo + first * kLine; x < hi; x += step * kLine) prefetch_l2(row + x);
    if (kDrawn)
      for (int x = lo + first * 32; x < hi; x += step * 32) prefetch_l2(p.draft_prob + (node0 + node) * p.draft_stride + x);
  };
  if (nodes > 0) prefetch(0, tid, kAccThreads);
  int bits = given != nodes && tid == 0 ? kStatusBadTreeLen : 0;
  if (tid < kMaxNodes) par_sh[tid] = -1;
  if (tid < nodes) {
    const int up = __ldg(p.tree_parent + node0 + tid), x = __ldg(p.tokens + node0 + tid);
    const bool linked = tid == 0 ? up == -1 : up >= 0 && up < tid, named = tid == 0 || (x >= 0 && x < p.vocab);
    if (!linked) bits |= kStatusBadParent;
    if (!named) bits |= kStatusBadToken;
    if (tid > 0 && linked && named) par_sh[tid] = up;
    tok_sh[tid] = x;
    u_sh[tid] = tame_uniform(__ldg(p.uniform + node0 + tid));
  }
  if (tid == 0) bits_sh = 0;
  if (tid < kPowers) pow_sh[tid] = c_pow[tid];
  const float temperature = __ldg(p.temperature + b);
  const bool greedy = !(temperature > 0.f);
  RowWeight w_of = row_weight(temperature);
  unsigned long long* weight_sh = dyn_sh - (kDrawn ? lo : 0);                     // [x] of token x
  float* value_sh = reinterpret_cast<float*>(dyn_sh + (kDrawn ? p.share : 0)) - lo;  // kDrawn: q, else logits
  int step = 0;  // of the reductions
  // The cluster's sum of one number a thread (or its largest), to all threads, in two halves with work between them; of
  // a sum also what comes before this warp's part.
  unsigned long long before, my_warp;
  bool lost = false;  // a wait ran out
  auto send = [&](unsigned long long v) {  // of a warp
    ++step;
    unsigned long long* part = part_sh[step & 1] + rank * kAccWarps + warp;
    uint64_t* bar = &part_bar[step & 1];
    my_warp = v;
    if (size == 1) {
      if (lane == 0) *part = v;
    } else {
      if (tid == 0) mbar_arrive_expect_tx(bar, size * kAccWarps * 8);
#ifdef DDT_TEST_HOOKS
      if (rank == 0 && warp == 1 && step == p.test_keep_back) return;
#endif
      // (a plain remote store and a barrier of the cluster: 2500 cycles a reduction in place of 1700)
      if (lane < size) st_async_b64(mapa_shared(smem_u32(part), lane), v, mapa_shared(smem_u32(bar), lane));
    }
  };
  auto arrived = [&] {
    if (size == 1) {
      __syncthreads();
    } else {
      bool in = false;
      for (uint32_t i = 0; !in && i < DDT_WAIT_LIMIT; ++i) in = mbar_try_wait_cluster(&part_bar[step & 1], ((step - 1) >> 1) & 1);
      lost = __syncthreads_or(!in);
    }
  };
  auto get_max = [&] {
    arrived();
    unsigned long long all = 0;
    for (int i = lane; i < size * kAccWarps; i += 32) {
      const unsigned long long x = part_sh[step & 1][i];
      all = x > all ? x : all;
    }
    return warp_max(all);
  };
  auto get_sum = [&] {
    arrived();
    unsigned long long all = 0, lower = 0;
    for (int i = lane; i < size * kAccWarps; i += 32) {
      const unsigned long long x = part_sh[step & 1][i];
      all += x;
      if (i < rank * kAccWarps + warp) lower += x;
    }
    before = warp_sum(lower);
    return warp_sum(all);
  };
  if (size > 1) cluster_wait();
  __syncthreads();

  int v = 0, len = nodes > 0 ? 1 : 0, next = -1;
  if (tid == 0) path_sh[0] = 0;
  while (nodes > 0) {
    const int64_t at = node0 + v;
    const T* row = static_cast<const T*>(p.logits) + at * p.logit_stride;
    const float* q = kDrawn ? p.draft_prob + at * p.draft_stride : nullptr;
    // v's children: bit i of the masks, and a thread for each
    uint32_t kids[kMaxNodes / 32];
#pragma unroll
    for (int i = 0; i < kMaxNodes / 32; ++i) kids[i] = __ballot_sync(0xffffffffu, par_sh[32 * i + lane] == v);
    const bool child = tid < nodes && par_sh[tid] == v;
    float l_child = 0.f, q_child = 1.f;
    if (child) {
      l_child = logit_now(row + tok_sh[tid]);
      if (kDrawn) q_child = logit_now(q + tok_sh[tid]);
    }
    // the row's share, and its largest (greedy: where that is, too, as the order of its bits over the lower index)
    unsigned long long best = 0;
    float top = -CUDART_INF_F;
    for (int x0 = wlo + lane; x0 < whi; x0 += kUnroll * 32) {
      float l[kUnroll], d[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int x = x0 + 32 * k;
        l[k] = x < whi ? logit(row + x) : -CUDART_INF_F;
        if (kDrawn) d[k] = x < whi ? __ldg(q + x) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int x = x0 + 32 * k;
        if (x < whi) {
          l[k] = tame(l[k]);
          if (kDrawn) {
            weight_sh[x] = __float_as_uint(l[k]);
            value_sh[x] = fminf(fmaxf(d[k], 0.f), 1.f);  // (a NaN becomes 0)
          } else {
            value_sh[x] = l[k];
          }
          if (greedy) {
            const unsigned long long key = order_of(l[k], x);
            best = key > best ? key : best;
          }
          top = fmaxf(top, l[k]);
        }
      }
    }
    if (!greedy) best = order_of(top, 0);
    send(warp_max(best));
    {  // the first children's rows, on their way meanwhile: 128 threads for each
      int c = -1, skip = tid >> 7;
#pragma unroll
      for (int i = 0; i < kMaxNodes / 32; ++i) {
        uint32_t m = kids[i];
        for (; c < 0 && m != 0; m &= m - 1)
          if (skip-- == 0) c = 32 * i + __ffs(m) - 1;
      }
      if (c >= 0) prefetch(c, tid & 127, 128);
    }
    best = get_max();
    if (lost) break;
    w_of.max = max_of(best);
    w_of.only = greedy ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
    if (!(w_of.max >= -3.4028235e38f)) {  // no logit is a number
      if (tid == 0) bits |= kStatusBadLogits;
      break;
    }
    unsigned long long sum = 0;
    // four tokens a lane at a time, so that their chains overlap
    for (int x0 = wlo + lane; x0 - lane < whi; x0 += 128) {
      float l[4], y[4];
      unsigned long long w[4];
      bool near = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = x0 + 32 * k;
        l[k] = x >= whi ? -CUDART_INF_F : kDrawn ? __uint_as_float(static_cast<uint32_t>(weight_sh[x])) : value_sh[x];
        y[k] = w_of.distance(l[k]);
        near = near || y[k] < kNear;
      }
      if (greedy) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = x0 + 32 * k < whi && x0 + 32 * k == w_of.only ? 1ull << kOne : 0;
      } else if (__any_sync(0xffffffffu, near)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned long long v = w_of.exactly(l[k], fminf(y[k], kNear), pow_sh);
          w[k] = y[k] < kNear ? v : RowWeight::plainly(y[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = RowWeight::plainly(y[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (kDrawn && x0 + 32 * k < whi) weight_sh[x0 + 32 * k] = w[k];
        sum += w[k];
      }
    }
    send(warp_sum(sum));
    if (child) {
      // (a token that an earlier sibling had has been refused by the time it is tried)
      bool again = false;
      if (!kDrawn)
#pragma unroll
        for (int i = 0; i < kMaxNodes / 32; ++i)
          for (uint32_t m = kids[i]; m != 0; m &= m - 1) {
            const int c = 32 * i + __ffs(m) - 1;
            again = again || (c < tid && tok_sh[c] == tok_sh[tid]);
          }
      child_w[tid] = again ? 0 : w_of(tame(l_child), tok_sh[tid], pow_sh);
      child_q[tid] = fminf(fmaxf(q_child, 0.f), 1.f);
    }
    unsigned long long S = get_sum();  // (and the children's weights)
    if (lost) break;
    unsigned long long refused = 0;  // kDrawn: the S of the refusals, in 16s
    int go = -1;
#pragma unroll 1
    for (int i = 0; i < kMaxNodes / 32 && go < 0 && !lost; ++i) {
#pragma unroll 1
      for (uint32_t m = kids[i]; m != 0; m &= m - 1) {
        const int c = 32 * i + __ffs(m) - 1;
        const unsigned long long w = kDrawn ? less(child_w[c], Shares(refused)(child_q[c])) : child_w[c];
        // u S q < w, each product rounded down to a whole number (one step of 2^-43 of the largest weight)
        if (share_of(kDrawn ? share_of(S, child_q[c]) : S, u_sh[c]) < w) {
          go = c;
          break;
        }
        if (!kDrawn) {
          if (w == 0 || w == S) continue;  // (a refusal that would leave nothing changes nothing)
          S -= w;
          const int x = tok_sh[c];
          if (x < wlo) before -= w;
          if (x >= wlo && x < whi) {
            my_warp -= w;
            value_sh[x] = -CUDART_INF_F;  // (the warp's lanes all write it)
          }
        } else {
          const unsigned long long held_before = before, held = my_warp;
          const Shares taken(refused + (S >> 4));
          unsigned long long left = 0;
#pragma unroll 4
          for (int x = wlo + lane; x < whi; x += 32) left += less(weight_sh[x], taken(value_sh[x]));
          send(warp_sum(left));
          left = get_sum();
          if (lost) break;
          if (left == 0) {
            before = held_before, my_warp = held;
          } else {
            refused += S >> 4;
            S = left;
          }
        }
      }
    }
    if (lost) break;
    if (go >= 0) {
      v = go;
      if (tid == 0) path_sh[len] = v;
      ++len;
      __syncthreads();  // the children's weights are read
      continue;
    }
    // the draw: the first x with the sum up to it above floor(u_0 S)
    const unsigned long long target = share_of(S, u_sh[0]);
    if (target >= before && target - before < my_warp) {  // one warp of the cluster
      __syncwarp();
      // lanes take consecutive tokens, an odd number each (so that they meet in no bank)
      const int each = ((whi - wlo + 31) / 32) | 1, first = min(whi, wlo + lane * each), last = min(whi, first + each);
      const Shares taken(refused);
      auto weight = [&](int x) {
        return kDrawn ? less(weight_sh[x], taken(value_sh[x])) : w_of(value_sh[x], x, pow_sh);
      };
      unsigned long long mine = 0;
#pragma unroll 4
      for (int x = first; x < last; ++x) mine += weight(x);
      auto up_to = [&](unsigned long long v) {  // the sum over this lane and those below
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        return v;
      };
      // the lane whose tokens hold the sum, then the token, 32 at a time
      const unsigned long long above = before + up_to(mine);
      const int owner = __ffs(__ballot_sync(0xffffffffu, above > target)) - 1;
      before = __shfl_sync(0xffffffffu, above - mine, owner);
      const int to = __shfl_sync(0xffffffffu, last, owner);
      for (int x0 = __shfl_sync(0xffffffffu, first, owner); x0 < to; x0 += 32) {
        const unsigned long long sum = before + up_to(x0 + lane < to ? weight(x0 + lane) : 0);
        const uint32_t vote = __ballot_sync(0xffffffffu, sum > target);
        if (vote != 0) {
          if (lane == 0) p.next_token[b] = x0 + __ffs(vote) - 1;
          break;
        }
        before = __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    next = 0;  // (written by the warp that found it)
    break;
  }
  if (lost && tid == 0) bits |= kStatusTimeout;
  __syncthreads();
  if (rank == 0) {
    if (tid < p.nodes) p.path[node0 + tid] = tid < len ? path_sh[tid] : -1;
    if (tid == 0) {
      p.path_len[b] = len;
      if (next < 0) p.next_token[b] = -1;
    }
    bits = static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bits)));
    if (lane == 0 && bits) atomicOr(&bits_sh, bits);
    __syncthreads();
    if (tid == 0) {
      if (p.batch == 1)
        *p.status = bits_sh;  // the word as a whole
      else if (bits_sh)
        atomicOr(p.status, bits_sh);
    }
  }
  if (size > 1) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while others may write to it (one whose wait ran out may be behind)
    if (lost && rank != 0 && tid == 0) atomicOr(p.status, kStatusTimeout);
  }
}

struct AccLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  AccLaunch(int requests, int cluster, size_t bytes) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(requests) * cluster);
    cfg.blockDim = dim3(kAccThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

template <typename T, bool kDrawn>
cudaError_t launch(const AcceptParams& p, size_t bytes, cudaStream_t stream) {
  AccLaunch l(p.batch, p.cluster, bytes);
  l.cfg.stream = stream;
  return cudaLaunchKernelEx(&l.cfg, accept_kernel<T, kDrawn>, p);
}

template <typename T, bool kDrawn>
cudaError_t configure() {
  cudaError_t e = cudaFuncSetAttribute(accept_kernel<T, kDrawn>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAcceptBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(accept_kernel<T, kDrawn>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

}  // namespace

cudaError_t configure_accept(AcceptClusters* clusters) {
  cudaError_t e = configure<uint16_t, false>();
  if (e == cudaSuccess) e = configure<uint16_t, true>();
  if (e == cudaSuccess) e = configure<float, false>();
  if (e == cudaSuccess) e = configure<float, true>();
  for (int i = 0; e == cudaSuccess && i < kAcceptSizes; ++i)
    for (int half = 0; half < 2; ++half) {
      AccLaunch l(1, 1 << i, half ? kAcceptBytes / 2 : kAcceptBytes);
      e = cudaOccupancyMaxActiveClusters(&clusters->count[i][half], accept_kernel<float, true>, &l.cfg);
    }
  return e;
}

cudaError_t launch_accept(const AcceptParams& p, bool bf16, cudaStream_t stream) {
  const size_t bytes = static_cast<size_t>(p.share) * accept_value_bytes(p.draft_prob != nullptr);
  if (p.draft_prob) return bf16 ? launch<uint16_t, true>(p, bytes, stream) : launch<float, true>(p, bytes, stream);
  return bf16 ? launch<uint16_t, false>(p, bytes, stream) : launch<float, false>(p, bytes, stream);
}

}  // namespace ddt
