// block_summary.cu -- 8-bit means of consecutive blocks of a request's prefix rows.
//
// For block j of request b (positions [j n, j n + n), cut at the prefix's end):
//   mean = (sum of its rows) / (rows)     576 dims
//   scale = max |mean| * (1/127),  summary = round(mean / scale), integers in [-127, 127]
// The integers are kept as bf16 (exact), the tensor cores' operand type: the
// dot product of two such rows is an integer below 2^24, so block scores come
// out exact in fp32 on any tiling.  The sums carry their rounding errors along
// (two-sum): off by at most 2^-34 of the sum of |x| over the block's (up to 128)
// rows, (127 * 2^-24)^2, before the mean is rounded to fp32.  Only where rows
// cancel to that degree can an integer depend on their order.  They are summed at
// 2^-7 of their size (exact: bf16 values stay above the least fp32 number), so no
// partial sum of finite rows overflows.
//
// Bound by memory: each row is read once (1152 B).  One CTA per SM: four warps
// keep up to four stages of 32 rows on their way into shared memory (one bulk
// copy a row; a copy takes its warp about 85 cycles to issue, so one warp stayed
// at 3.3 TB/s), and three teams of 288 threads add up every third block each,
// thread (g, c) of a team the 16-byte piece c of rows g, g + 4, ....  185000
// scattered rows: 51 us (two teams 53, one 70; loads through registers, which
// leave the memory idle while a block is reduced, 55-61).
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kSumGroups = 4;
constexpr int kSumThreads = kSumGroups * kChunks;  // 288 that add up a block
constexpr int kSumTeams = 3;
constexpr int kSumCopiers = 4;                     // and the warps that copy
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSumRows = 32;                       // rows of a stage
constexpr int kSumStages = 4;
constexpr int kSumStageBytes = kSumRows * kRowBytes;

struct SumShared {
  uint64_t full[kSumStages], empty[kSumStages];
  alignas(4) uint8_t rows[kSumStages][kSumCopiers];           // the stage's rows that exist, 8 a copying warp
  float amax[kSumTeams][kSumWarps];
  int abort;
};
constexpr float kSumDown = 1.f / 128.f;            // of a row's value when it is added
constexpr float kSumBig = 1.7014118e38f / 128.f;   // 2^127 at that size
constexpr int kSumOffPart = kSumStages * kSumStageBytes;  // [4 groups][hi, lo][576]
constexpr int kSumPart = kSumGroups * 2 * kDqk;           // floats of a team
constexpr int kSumOffShared = kSumOffPart + kSumTeams * kSumPart * 4;
constexpr int kSumBlockThreads = kSumTeams * kSumThreads + 32 * kSumCopiers;
constexpr int kSumSmem = kSumOffShared + static_cast<int>(sizeof(SumShared)) + 16;

// (hi, lo) + x without losing the rounding error of hi + x, two dims at a time
// (the additions are half of the kernel's instructions: paired ones halve them)
__device__ __forceinline__ void two_sum(uint64_t& hi, uint64_t& lo, uint64_t x) {
  const uint64_t s = add_x2(hi, x);
  const uint64_t v = sub_x2(s, hi);
  lo = add_x2(lo, add_x2(sub_x2(hi, sub_x2(s, v)), sub_x2(x, v)));
  hi = s;
}

__global__ void __launch_bounds__(kSumBlockThreads, 1) block_summary_kernel(SummaryParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  SumShared& sh = *reinterpret_cast<SumShared*>(smem + kSumOffShared);
  volatile int* abort = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y;
  int L = __ldg(p.prefix_len + b);
  if (L < 0 || L > p.max_prefix_len) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, kStatusBadPrefix);
    L = L < 0 ? 0 : p.max_prefix_len;
  }
  const int from = p.from_len != nullptr ? max(0, __ldg(p.from_len + b)) : 0;
  const int n_blocks = L > 0 ? (L - 1) / p.block + 1 : 0;
  const int j0 = from / p.block + static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
  if (from >= L || j0 >= n_blocks) return;
  if (tid == 0) {
    for (int i = 0; i < kSumStages; ++i) {
      mbar_init(&sh.full[i], kSumCopiers);
      mbar_init(&sh.empty[i], kSumTeams * kSumWarps);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const int chunks = (p.block + kSumRows - 1) / kSumRows;  // stages of a block
  bool ok = true;

  if (warp >= kSumTeams * kSumWarps) {
    // ------------------------------------------------------------------ copies: a warp takes 8 rows of the stage
    const int k = warp - kSumTeams * kSumWarps, row8 = 8 * k + (lane & 7);
    const int32_t* slots = p.slot_idx + static_cast<int64_t>(b) * p.slot_stride;
    // the slots of a stage are read two stages before its copies
    struct At {
      int64_t j;  // block (past the last one once the walk is over)
      int c;      // stage of the block
    };
    auto next_of = [&](At x) -> At { return x.c + 1 < chunks ? At{x.j, x.c + 1} : At{x.j + step, 0}; };
    auto pos_of = [&](At x) -> int64_t {
      const int row = x.c * kSumRows + row8;
      const int64_t pos = x.j * p.block + row;
      return lane < 8 && x.j < n_blocks && row < p.block && pos < L ? pos : -1;
    };
    auto slot_of = [&](At x) -> int {
      const int64_t pos = pos_of(x);
      return pos >= 0 ? __ldg(slots + pos) : -1;
    };
    At at{j0, 0}, at1 = next_of(at), at2 = next_of(at1);
    int s0 = slot_of(at), s1 = slot_of(at1);
    uint32_t n = 0;  // stages filled
    while (at.j < n_blocks) {
      const int s2 = slot_of(at2);
      const uint32_t st = n % kSumStages;
      const bool w = n < kSumStages || mbar_wait_abortable(&sh.empty[st], ((n / kSumStages) - 1) & 1, abort, false, __LINE__);
      if (!__all_sync(0xffffffffu, w)) {
        ok = false;
        break;
      }
      const bool here = pos_of(at) >= 0, good = here && s0 >= 0 && s0 < p.pool_slots;
      if (here && !good) atomicOr(p.status, kStatusBadSlot);
      const uint32_t rows = __ballot_sync(0xffffffffu, good);
      if (lane == 0) {
        sh.rows[st][k] = static_cast<uint8_t>(rows);
        mbar_arrive_expect_tx(&sh.full[st], __popc(rows) * kRowBytes);
      }
      __syncwarp();
      if (good) bulk_load(smem_u32(smem) + st * kSumStageBytes + row8 * kRowBytes, p.kv + static_cast<int64_t>(s0) * kDqk, kRowBytes, &sh.full[st]);
      ++n;
      s0 = s1;
      s1 = s2;
      at = at1;
      at1 = at2;
      at2 = next_of(at2);
    }
    // no copy is in flight when the CTA exits (after a give-up the adders leave stages unread)
    for (uint32_t i = n > kSumStages ? n - kSumStages : 0; i < n; ++i) mbar_wait(&sh.full[i % kSumStages], (i / kSumStages) & 1);
  } else {
    // ------------------------------------------------------------------ sums
    const int team = tid / kSumThreads, tt = tid - team * kSumThreads, tw = warp - team * kSumWarps;
    const int g = tt / kChunks, c = tt - g * kChunks;
    float* part = reinterpret_cast<float*>(smem + kSumOffPart) + team * kSumPart;
    // A team passes the other's stages too: it waits for them to land and hands
    // them back at once.  A barrier's parity tells a phase from the next one only,
    // so no thread may fall a phase behind or get one ahead.
    uint32_t n = 0;  // stages passed
    bool failed = false;
    auto land = [&](uint32_t i) {
      if (!mbar_wait_abortable(&sh.full[i % kSumStages], (i / kSumStages) & 1, abort, false, __LINE__)) failed = true;
      __syncwarp();
    };
    auto hand_back = [&](uint32_t i) {
      __syncwarp();
#ifdef DDT_TEST_HOOKS
      if (warp == 0 && static_cast<int>(i) == p.test_keep_back) return;
#endif
      // (not after a give-up: the stage may not have landed, and the copying warps would fill it a second time)
      if (lane == 0 && !failed) mbar_arrive(&sh.empty[i % kSumStages]);
    };
    int turn = 0;
    for (int64_t j = j0; j < n_blocks; j += step, turn = turn + 1 == kSumTeams ? 0 : turn + 1) {
      if (turn != team) {
        for (int ch = 0; ch < chunks; ++ch, ++n) {
          land(n);
          hand_back(n);
        }
        continue;
      }
      uint64_t hi[4], lo[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) hi[d] = lo[d] = 0;
      int count = 0;
      auto add = [&](const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int d = 0; d < 4; ++d)
          two_sum(hi[d], lo[d],
                  mul_x2(f32x2(__uint_as_float(w[d] << 16), __uint_as_float(w[d] & 0xffff0000u)), f32x2(kSumDown, kSumDown)));
      };
      for (int ch = 0; ch < chunks; ++ch, ++n) {
        const uint32_t st = n % kSumStages;
        land(n);
        const uint32_t rows = *reinterpret_cast<const uint32_t*>(sh.rows[st]);
        count += __popc(rows);
        const uint4* src = reinterpret_cast<const uint4*>(smem + st * kSumStageBytes + g * kRowBytes) + c;
        constexpr int kEach = kSumRows / kSumGroups;
        if (rows == 0xffffffffu) {
          uint4 v[kEach];
#pragma unroll
          for (int u = 0; u < kEach; ++u) v[u] = src[u * kSumGroups * kChunks];
#pragma unroll
          for (int u = 0; u < kEach; ++u) add(v[u]);
        } else {
#pragma unroll 2
          for (int u = 0; u < kEach; ++u)
            if ((rows >> (u * kSumGroups + g)) & 1u) add(src[u * kSumGroups * kChunks]);
        }
        hand_back(n);
      }
      uint64_t* mine = reinterpret_cast<uint64_t*>(part + g * 2 * kDqk) + 4 * c;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        mine[d] = hi[d];
        mine[kDqk / 2 + d] = lo[d];
      }
      if (bar_red_or(1 + team, kSumThreads, failed)) {
        ok = false;
        break;
      }
      // dims 2 tt and 2 tt + 1: the four groups' sums, the mean, the largest of all
      const uint64_t* all = reinterpret_cast<const uint64_t*>(part) + tt;
      uint64_t h2 = all[0], l2 = all[kDqk / 2];
#pragma unroll
      for (int o = 1; o < kSumGroups; ++o) {
        two_sum(h2, l2, all[o * kDqk]);
        l2 = add_x2(l2, all[o * kDqk + kDqk / 2]);
      }
      float hs[2], ls[2], mean[2];
      f32x2_split(h2, hs[0], hs[1]);
      f32x2_split(l2, ls[0], ls[1]);
      float am = 0.f;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        // (hi + lo) / rows in fp32 pairs: the quotient of hi, and that of what is
        // left of hi and lo (64-bit division is slow here and would cost more than the sums)
        // a sum beyond fp32 is divided at 2^-7 of its size, by 2^-7 of the rows
        const float up = fabsf(hs[d]) < kSumBig ? 1.f / kSumDown : 1.f;
        const float n_rows = static_cast<float>(max(count, 1)) * (up * kSumDown);
        hs[d] *= up;
        ls[d] *= up;
        const float q = __fdiv_rn(hs[d], n_rows);
        const float m = __fadd_rn(q, __fdiv_rn(__fadd_rn(__fmaf_rn(-q, n_rows, hs[d]), ls[d]), n_rows));
        mean[d] = count > 0 ? m : 0.f;
        // (an infinite row leaves a NaN in the carried error)
        am = fabsf(mean[d]) < CUDART_INF_F ? fmaxf(am, fabsf(mean[d])) : CUDART_INF_F;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, off));
      if (lane == 0) sh.amax[team][tw] = am;
      bar_sync(1 + team, kSumThreads);  // (and the partial sums are read)
#pragma unroll
      for (int i = 0; i < kSumWarps; ++i) am = fmaxf(am, sh.amax[team][i]);
      const bool good = am < CUDART_INF_F;
      const float scale = good ? __fmul_rn(am, 1.f / 127.f) : CUDART_NAN_F;
      uint32_t two = 0;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        float q = 0.f;
        if (good && scale > 0.f) q = fminf(fmaxf(rintf(__fdiv_rn(mean[d], scale)), -127.f), 127.f);
        two |= (__float_as_uint(q) >> 16) << (16 * d);  // an integer of 7 bits and sign: exact in bf16
      }
      const int64_t out = static_cast<int64_t>(b) * p.blocks + j;
      reinterpret_cast<uint32_t*>(p.summary + out * kDqk)[tt] = two;
      if (tt == 0) p.scale[out] = scale;
    }
  }
  if (!ok) {
    *abort = 1;
    atomicOr(p.status, kStatusTimeout);
  }
}

}  // namespace

cudaError_t configure_summary() {
  return cudaFuncSetAttribute(block_summary_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSumSmem);
}

cudaError_t launch_block_summary(const SummaryParams& p, int batch, int sm_count, cudaStream_t stream) {
  if (batch == 0) return cudaSuccess;
  // blocks of a request are dealt to its share of the SMs: how many are touched
  // (from_len) is known on the device only
  const int share = (sm_count + batch - 1) / batch;
  // (without a block one CTA a request still looks its length over for the status word)
  const unsigned gx = static_cast<unsigned>(p.blocks < share ? (p.blocks > 0 ? p.blocks : 1) : share);
  block_summary_kernel<<<dim3(gx, batch), kSumBlockThreads, kSumSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
