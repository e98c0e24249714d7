// accept.cu -- the drafted tokens of a tree against the target's probabilities, from given random numbers.
//
// At node v the target's next token has p(x) = softmax(logits[v] / temperature). v's
// children are tried in node order: with w the part of p that is left and S its sum, child
// c with token x is accepted if u_c S q(x) < w(x). Drafted tokens that were picked (the
// drafter's best) have q = 1, and a refused one leaves w without x; tokens that were drawn
// from the drafter's distribution q leave max(w - S q, 0). Either way the accepted path
// and the token after it follow p exactly. Where no child is accepted the next token is
// the first x with w(0) + ... + w(x) > u_0 S.
//
// Weights are whole numbers: w(x) = 2^((l(x) - max l) log2 e / temperature) in steps of
// 2^-43, their exponent carried in two floats (3e-10 of each weight). So sums are exact in any order, the
// same tokens come out on any tiling, and a token on the border between two answers is
// decided as 64-bit arithmetic decides it, but for one draw in 10^5 or so.
//
// Kernel 1, a cluster per node: the row's maximum, the sum of its weights, and for each
// child whether it would be accepted if the walk came to its parent. Every row is read at
// once, though the walk will visit few: which ones is known only step by step, and a step
// (read, reduce, decide) takes longer than all rows together.
// Kernel 2, a cluster per request: the walk over those answers (a node's children come
// behind it, so one pass over the nodes), then the draw from what the last node has left:
// a sum per warp, and the one warp whose range holds the token looks it up.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <algorithm>
#include "accept.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kAccThreads = 512, kAccWarps = kAccThreads / 32;
constexpr int kOne = 43;         // weight 1 is 2^43; up to 2^20 of them fit in 64 bits
constexpr int kUnroll = 8;       // loads in flight of a thread

// 2^(62 - i / 64), i = 0 to 63
__constant__ unsigned long long c_pow[64] = {
    0x4000000000000000ull, 0x3f4f83033d21b05dull, 0x3ea0ecb6dc8a80cfull, 0x3df437dcc2b44eeeull,
    0x3d495f454921b30bull, 0x3ca05dcf167fec4eull, 0x3bf92e66f736bd73ull, 0x3b53cc07b6650ae1ull,
    0x3ab031b9f7490e4cull, 0x3a0e5a940f12f71aull, 0x396e41b9df20d22aull, 0x38cfe25cafa29694ull,
    0x383337bb0aa53844ull, 0x37983d209783a449ull, 0x36feede5f6bc8dd5ull, 0x366745709e2bf5edull,
    0x35d13f32b5a75abdull, 0x353cd6aaf3fb7e88ull, 0x34aa07647c4ab917ull, 0x3418ccf6bbcac965ull,
    0x3389230547e12039ull, 0x32fb053fbc9c9f17ull, 0x326e6f619b8bc9e9ull, 0x31e35d322aee6c57ull,
    0x3159ca845541b6b7ull, 0x30d1b3368925d902ull, 0x304b1332999c2516ull, 0x2fc5e66d9e9cc421ull,
    0x2f4228e7d6030db0ull, 0x2ebfd6ac84cf917full, 0x2e3eebd1d8bee7baull, 0x2dbf6478ca345de4ull,
    0x2d413cccfe779921ull, 0x2cc47104aa444922ull, 0x2c48fd6074ab0964ull, 0x2bcede2b5a4290ddull,
    0x2b560fba90a852b2ull, 0x2ade8e6d6a4fb4ceull, 0x2a6856ad3a9f03beull, 0x29f364ed3a594d5aull,
    0x297fb5aa6c544e3bull, 0x290d456b8279a028ull, 0x289c10c0c3125a06ull, 0x282c1443ee5c53f1ull,
    0x27bd4c982468446bull, 0x274fb669cb3fedd4ull, 0x26e34e6e7553954eull, 0x26781164c82dfe99ull,
    0x260dfc14636e2a5cull, 0x25a50b4dc8061680ull, 0x253d3bea3fbdc258ull, 0x24d68acbc4f9ba4bull,
    0x2470f4dceac470ceull, 0x240c7710c519ac77ull, 0x23a90e62d17354f0ull, 0x2346b7d6df96ea79ull,
    0x22e57078faa2f5baull, 0x2285355d525bbf67ull, 0x222603a024b6a14aull, 0x21c7d865a7a34404ull,
    0x216ab0d9f3121ec5ull, 0x210e8a30eb379012ull, 0x20b361a62b0ae876ull, 0x2059347cef00c1ddull,
};

// 2^-(hi + lo) in steps of 2^-43, rounded down; hi >= 0, |lo| small. `pow_sh` is c_pow in shared memory.
__device__ __forceinline__ unsigned long long weight_of(float hi, float lo, const unsigned long long* pow_sh) {
  if (!(hi < 44.f)) return 0;
  const float k = rintf(hi * 64.f);
  const float r = fmaf(k, -0.015625f, hi) + lo;  // (the first difference is exact)
  const int ki = static_cast<int>(k);
  // 2^-r - 1, |r| <= 2^-7: its error, 2^-31, is the weight's
  const float z = r * -0.69314718055994531f;
  const float g = fmaf(z * z, fmaf(z, fmaf(z, 1.f / 24, 1.f / 6), 0.5f), z);
  const int gi = __float2int_rn(g * 274877906944.f);  // 2^38
  const long long top = static_cast<long long>(pow_sh[ki & 63]);
  const long long w = top + ((static_cast<long long>(static_cast<int>(top >> 32)) * gi) >> 6);
  return static_cast<unsigned long long>(w) >> ((62 - kOne) + (ki >> 6));
}

// A row's weights: 2^((l - max) c) with c = log2 e / temperature in two floats, or all of it on one token.
struct RowWeight {
  float max, c_hi, c_lo;
  int only;  // greedy: the token; else -1
  __device__ __forceinline__ unsigned long long operator()(float l, int x, const unsigned long long* pow_sh) const {
    if (only >= 0) return x == only ? 1ull << kOne : 0;
    // max - l = d + e exactly
    const float d = max - l, b = d - max;
    const float e = (max - (d - b)) - (l + b);
    const float hi = d * c_hi;
    return weight_of(hi, fmaf(d, c_hi, -hi) + fmaf(d, c_lo, e * c_hi), pow_sh);
  }
};
__device__ __forceinline__ RowWeight row_weight(float max, int arg, float temperature) {
  RowWeight r;
  r.max = max;
  r.only = temperature > 0.f ? -1 : arg;
  const double c = temperature > 0.f ? fmin(1.4426950408889634 / static_cast<double>(temperature), 1e30) : 0.0;
  r.c_hi = static_cast<float>(c);
  r.c_lo = static_cast<float>(c - static_cast<double>(r.c_hi));
  return r;
}

// floor(S q) for a probability q (clamped to [0, 1]; NaN: 0)
__device__ __forceinline__ unsigned long long share_of(unsigned long long S, float q) {
  if (!(q > 0.f)) return 0;
  if (q >= 1.f) return S;
  const uint32_t u = __float_as_uint(q);
  const int e = static_cast<int>(u >> 23);  // at most 126
  const unsigned long long mant = e > 0 ? (u & 0x7fffffu) | 0x800000u : 0;
  return 126 - e > 63 ? 0 : __umul64hi(S, mant << 40) >> (126 - e);
}
__device__ __forceinline__ unsigned long long less(unsigned long long w, unsigned long long s) { return w > s ? w - s : 0; }

__device__ __forceinline__ float logit(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16); }
__device__ __forceinline__ float logit(const float* p) { return __ldg(p); }
// NaN counts as -inf, +inf as the largest number
__device__ __forceinline__ float tame(float l) { return l >= -3.4028235e38f ? fminf(l, 3.4028235e38f) : -CUDART_INF_F; }

// u in [0, 1), NaN as 0
__device__ __forceinline__ float tame_uniform(float u) { return u > 0.f ? fminf(u, 0.99999994f) : 0.f; }

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long remote_u64(const unsigned long long* p, uint32_t rank) {
  const uint32_t at = mapa_shared(smem_u32(p), rank);
  const uint32_t lo = static_cast<uint32_t>(ld_shared_cluster_b32(at)), hi = static_cast<uint32_t>(ld_shared_cluster_b32(at + 4));
  return lo | (static_cast<unsigned long long>(hi) << 32);
}

// This CTA's share [lo, hi) of the vocabulary, of `size` CTAs.
__device__ __forceinline__ void range_of(int vocab, int rank, int size, int* lo, int* hi) {
  const int each = ((vocab + size - 1) / size + 31) / 32 * 32;
  *lo = min(vocab, rank * each);
  *hi = min(vocab, *lo + each);
}

// f(index, logit, q) over [lo, hi), by the threads first, first + step, ...
template <typename T, typename F>
__device__ __forceinline__ void each(const T* row, const float* q, int lo, int hi, int first, int step, F f) {
  for (int i0 = lo + first; i0 < hi; i0 += kUnroll * step) {
    float l[kUnroll], d[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * step;
      l[k] = i < hi ? logit(row + i) : -CUDART_INF_F;
      d[k] = q && i < hi ? __ldg(q + i) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (i0 + k * step < hi) f(i0 + k * step, tame(l[k]), d[k]);
  }
}

// The sum over a cluster of one value per thread, to all threads. `slot`: two values of shared memory of its own.
__device__ __forceinline__ unsigned long long cluster_sum(unsigned long long v, unsigned long long* warps, unsigned long long* slot,
                                                          int size) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum(v);
  if (lane == 0) warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = warp_sum(lane < kAccWarps ? warps[lane] : 0);
    if (lane == 0) *slot = v;
  }
  cluster_sync();
  v = warp_sum(lane < size ? remote_u64(slot, lane) : 0);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kAccThreads) accept_rows_kernel(const __grid_constant__ AcceptParams p) {
  __shared__ unsigned long long pow_sh[64];
  __shared__ unsigned long long warps_sh[2][kAccWarps];
  __shared__ unsigned long long slot_sh[kMaxNodes + 2];  // of each pass; read by the cluster
  __shared__ unsigned long long mult_sh[kMaxNodes];      // S of the steps that were taken
  __shared__ int child_sh[kMaxNodes], n_child;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int size = p.row_cluster, rank = blockIdx.x % size;
  const int64_t at = blockIdx.x / size;  // of the node
  const int b = static_cast<int>(at / p.nodes), v = static_cast<int>(at - static_cast<int64_t>(b) * p.nodes);
  grid_dep_launch();
  if (blockIdx.x == 0 && tid == 0) *p.status = 0;  // (the second kernel reports)
  const int nodes = p.tree_len ? min(max(__ldg(p.tree_len + b), 0), p.nodes) : p.nodes;
  if (v >= nodes) return;  // the whole cluster
  const T* row = static_cast<const T*>(p.logits) + at * p.logit_stride;
  const float* q = p.draft_prob ? p.draft_prob + at * p.draft_stride : nullptr;
  int lo, hi;
  range_of(p.vocab, rank, size, &lo, &hi);
  if (tid < 64) pow_sh[tid] = c_pow[tid];
  if (warp == 0) {  // v's children that have a token, in node order
    int n = 0;
    for (int i0 = v + 1; i0 < nodes; i0 += 32) {
      const int i = i0 + lane;
      bool is = false;
      if (i < nodes && __ldg(p.tree_parent + static_cast<int64_t>(b) * p.nodes + i) == v) {
        const int x = __ldg(p.tokens + static_cast<int64_t>(b) * p.nodes + i);
        is = x >= 0 && x < p.vocab;
      }
      const uint32_t vote = __ballot_sync(0xffffffffu, is);
      if (is) child_sh[n + __popc(vote & ((1u << lane) - 1u))] = i;
      n += __popc(vote);
    }
    if (lane == 0) n_child = n;
  }
  // the maximum, and where it is first: as one number (the order of the float's bits, then the lower index)
  unsigned long long best = 0;
  each(row, nullptr, lo, hi, tid, kAccThreads, [&](int i, float l, float) {
    const uint32_t u = __float_as_uint(l);
    const uint32_t key = l == 0.f ? 0x80000000u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    const unsigned long long k = (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
    best = k > best ? k : best;
  });
  auto warp_max = [](unsigned long long k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, k, o);
      k = other > k ? other : k;
    }
    return k;
  };
  best = warp_max(best);
  if (lane == 0) warps_sh[0][warp] = best;
  __syncthreads();
  if (warp == 0) {
    best = warp_max(lane < kAccWarps ? warps_sh[0][lane] : 0);
    if (lane == 0) slot_sh[kMaxNodes + 1] = best;
  }
  cluster_sync();
  best = warp_max(lane < size ? remote_u64(&slot_sh[kMaxNodes + 1], lane) : 0);
  const uint32_t key = static_cast<uint32_t>(best >> 32);
  const float max = __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
  const int arg = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
  const bool dead = !(max >= -3.4028235e38f);  // no logit is a number
  const RowWeight w_of = row_weight(max, arg, __ldg(p.temperature + b));
  unsigned long long S = 0;
  if (!dead) each(row, nullptr, lo, hi, tid, kAccThreads, [&](int i, float l, float) { S += w_of(l, i, pow_sh); });
  S = cluster_sum(S, warps_sh[1], &slot_sh[kMaxNodes], size);
  const int n = n_child;
  const int64_t node0 = static_cast<int64_t>(b) * p.nodes;
  if (tid == 0 && rank == 0) {
    p.row_max[at] = max;
    p.row_arg[at] = arg;
  }
  for (int c = 0; c < n; ++c) {
    const int i = child_sh[c], x = __ldg(p.tokens + node0 + i);
    unsigned long long w = dead ? 0 : w_of(tame(logit(row + x)), x, pow_sh);
    const double u = tame_uniform(__ldg(p.uniform + node0 + i));
    unsigned long long taken, left;  // (taken 0: a refusal that would leave nothing changes nothing)
    bool accepted;
    if (!q) {
      for (int j = 0; j < c; ++j)
        if (__ldg(p.tokens + node0 + child_sh[j]) == x) w = 0;  // refused already
      accepted = u * static_cast<double>(S) < static_cast<double>(w);
      left = S - w;
      taken = w;
    } else {
      const float qx = __ldg(q + x);
      for (int j = 0; j < c; ++j) w = less(w, share_of(mult_sh[j], qx));
      accepted = u * static_cast<double>(S) * static_cast<double>(fminf(fmaxf(qx, 0.f), 1.f)) < static_cast<double>(w);
      left = 0;
      if (!dead) {
        each(row, q, lo, hi, tid, kAccThreads, [&](int k, float l, float d) {
          unsigned long long y = w_of(l, k, pow_sh);
          for (int j = 0; j < c; ++j) y = less(y, share_of(mult_sh[j], d));
          left += less(y, share_of(S, d));
        });
      }
      left = cluster_sum(left, warps_sh[c & 1], &slot_sh[c], size);
      taken = S;
    }
    if (left == 0) left = S, taken = 0;
    __syncthreads();
    if (tid == 0) {
      mult_sh[c] = taken;
      if (rank == 0) {
        p.accepted[node0 + i] = accepted ? 1 : 0;
        p.taken[node0 + i] = taken;
      }
    }
    S = left;
    __syncthreads();
  }
  if (tid == 0 && rank == 0) p.left[at] = S;
  cluster_sync();  // no CTA leaves while its slots are read
}

template <typename T>
__global__ void __launch_bounds__(kAccThreads) accept_walk_kernel(const __grid_constant__ AcceptParams p) {
  __shared__ unsigned long long pow_sh[64];
  __shared__ unsigned long long warps_sh[kAccWarps], total_sh;
  __shared__ unsigned long long taken_sh[kMaxNodes];
  __shared__ int par_sh[kMaxNodes], tok_sh[kMaxNodes], acc_sh[kMaxNodes], path_sh[kMaxNodes], child_sh[kMaxNodes];
  __shared__ int last_sh, len_sh, n_child;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int size = p.walk_cluster, rank = blockIdx.x % size, b = blockIdx.x / size;
  const int64_t node0 = static_cast<int64_t>(b) * p.nodes;
  const int given = p.tree_len ? __ldg(p.tree_len + b) : p.nodes, nodes = min(max(given, 0), p.nodes);
  int bits = given != nodes && tid == 0 ? kStatusBadTreeLen : 0;
  if (tid < nodes) {
    const int up = __ldg(p.tree_parent + node0 + tid), x = __ldg(p.tokens + node0 + tid);
    const bool linked = tid == 0 ? up == -1 : up >= 0 && up < tid, named = tid == 0 || (x >= 0 && x < p.vocab);
    if (!linked) bits |= kStatusBadParent;
    if (!named) bits |= kStatusBadToken;
    par_sh[tid] = tid > 0 && linked && named ? up : -1;
    tok_sh[tid] = x;
  }
  if (tid < 64) pow_sh[tid] = c_pow[tid];
  const float u0 = nodes > 0 ? tame_uniform(__ldg(p.uniform + node0)) : 0.f;
  const float temperature = __ldg(p.temperature + b);
  grid_dep_wait();
  if (tid < nodes && tid > 0) acc_sh[tid] = par_sh[tid] >= 0 ? __ldcg(p.accepted + node0 + tid) : 0;
  __syncthreads();
  if (warp == 0) {
    // the first accepted child of the node, its first accepted child, ...: children come behind their parents
    int v = 0, len = nodes > 0 ? 1 : 0;
    if (lane == 0) path_sh[0] = 0;
    for (int i0 = 0; i0 < nodes; i0 += 32) {
      uint32_t seen = 0;  // nodes of these 32 that the walk is past
      for (;;) {
        const int i = i0 + lane;
        const uint32_t vote = __ballot_sync(0xffffffffu, i > v && i < nodes && par_sh[i] == v && acc_sh[i] != 0) & ~seen;
        if (vote == 0) break;
        const int bit = __ffs(vote) - 1;
        v = i0 + bit;
        seen = bit == 31 ? 0xffffffffu : (2u << bit) - 1u;
        if (lane == 0) path_sh[len] = v;
        ++len;
      }
    }
    int n = 0;
    for (int i0 = 0; i0 < nodes; i0 += 32) {
      const bool is = i0 + lane < nodes && i0 + lane > 0 && par_sh[i0 + lane] == v;
      const uint32_t vote = __ballot_sync(0xffffffffu, is);
      if (is) child_sh[n + __popc(vote & ((1u << lane) - 1u))] = i0 + lane;
      n += __popc(vote);
    }
    if (lane == 0) {
      last_sh = v;
      len_sh = len;
      n_child = n;
    }
  }
  __syncthreads();
  const int v = last_sh, n = n_child, len = len_sh;
  if (rank == 0) {
    if (tid < p.nodes) p.path[node0 + tid] = tid < len ? path_sh[tid] : -1;
    if (tid == 0) p.path_len[b] = len;
  }
  if (tid < n) taken_sh[tid] = __ldcg(p.taken + node0 + child_sh[tid]);
  const int64_t at = node0 + v;
  const float max = nodes > 0 ? __ldcg(p.row_max + at) : -CUDART_INF_F;
  const bool dead = !(max >= -3.4028235e38f);
  if (dead) {
    if (rank == 0 && tid == 0) {
      p.next_token[b] = -1;
      if (nodes > 0) bits |= kStatusBadLogits;
    }
    if (rank == 0 && bits) atomicOr(p.status, bits);
    return;  // the whole cluster
  }
  const unsigned long long left = __ldcg(p.left + at);
  const RowWeight w_of = row_weight(max, __ldcg(p.row_arg + at), temperature);
  const T* row = static_cast<const T*>(p.logits) + at * p.logit_stride;
  const float* q = p.draft_prob ? p.draft_prob + at * p.draft_stride : nullptr;
  __syncthreads();
  auto weight = [&](int i, float l, float d) {
    unsigned long long w = w_of(l, i, pow_sh);
    if (q) {
      for (int j = 0; j < n; ++j) w = less(w, share_of(taken_sh[j], d));
    } else {
      for (int j = 0; j < n; ++j)
        if (taken_sh[j] != 0 && tok_sh[child_sh[j]] == i) w = 0;
    }
    return w;
  };
  // the first x with the sum up to it above floor(u_0 S)
  const unsigned long long target = share_of(left, u0);
  int lo, hi;
  range_of(p.vocab, rank, size, &lo, &hi);
  // a warp's part of the CTA's share, in steps of 32
  const int each_warp = ((hi - lo + kAccWarps - 1) / kAccWarps + 31) / 32 * 32;
  const int wlo = min(hi, lo + warp * each_warp), whi = min(hi, wlo + each_warp);
  unsigned long long sum = 0;
  each(row, q, wlo, whi, lane, 32, [&](int i, float l, float d) { sum += weight(i, l, d); });
  sum = warp_sum(sum);
  if (lane == 0) warps_sh[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    const unsigned long long s = warp_sum(lane < kAccWarps ? warps_sh[lane] : 0);
    if (lane == 0) total_sh = s;
  }
  cluster_sync();
  unsigned long long before = warp_sum(lane < rank ? remote_u64(&total_sh, lane) : 0);
  before += warp_sum(lane < warp ? warps_sh[lane] : 0);
  if (target >= before && target - before < sum) {  // one warp of the cluster
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane;
      unsigned long long w = i < whi ? weight(i, tame(logit(row + i)), q ? __ldg(q + i) : 0.f) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      const uint32_t vote = __ballot_sync(0xffffffffu, before + w > target);
      if (vote != 0) {
        if (lane == 0) p.next_token[b] = i0 + __ffs(vote) - 1;
        break;
      }
      before += __shfl_sync(0xffffffffu, w, 31);
    }
  }
  if (rank == 0 && bits) atomicOr(p.status, bits);
  cluster_sync();  // no CTA leaves while its sum is read
}

template <typename K>
cudaError_t launch(K kernel, const AcceptParams& p, int64_t clusters, int size, bool dependent, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * size));
  cfg.blockDim = dim3(kAccThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_accept(const AcceptParams& p, bool bf16, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.nodes;
  cudaError_t e = launch(bf16 ? accept_rows_kernel<uint16_t> : accept_rows_kernel<float>, p, rows, p.row_cluster, false, stream);
  if (e == cudaSuccess)
    e = launch(bf16 ? accept_walk_kernel<uint16_t> : accept_walk_kernel<float>, p, p.batch, p.walk_cluster, true, stream);
  return e;
}

}  // namespace ddt
