// block_attn.cu -- attention of each tree node over its own list of key blocks.
//
// Node t of request b reads the prefix positions of the blocks it lists, each
// list being its own, so the rows that can share a gathered key are the H heads
// of the nodes that list it.  Nodes are taken in groups of up to 64 (node, head)
// rows; a group walks the union of its nodes' lists, with a 64-bit mask per
// block of the rows that listed it (lists of one tree overlap; where they do
// not, the union costs what separate lists would, since a tcgen05.mma takes as
// long for 16 columns as for 64).
//
// With 64 rows the usual roles waste the tensor core's 128 lanes on O (rows as
// M), so they are swapped: keys and value dims are the M side, rows the N side.
//   S^T[64 keys][rows]  = K . Q^T          36 MMAs M64 x N x K16
//   O^T[512 dims][rows] += V^T . P^T       4 x 4 MMAs M128 x N x K16 (V^T: the same
//                                          latent blocks read MN-major)
// O^T takes 256 TMEM columns, so one CTA holds the whole output and nothing is
// exchanged between SMs; scores and sums stay fp32.  P is rounded to bf16, the
// operand type, against row sums of the unrounded values: an error of half a
// bf16 step per weight, averaged over the keys, below the bf16 rounding of out.
//
// Per CTA (416 threads), one unit = (group, split of its key tiles):
//   warp 0      TMEM; one lane issues S(t) dim group by dim group as stage t
//               lands, and P.V(t) when P(t) is written, whichever is ready
//   warps 1-4   softmax: TMEM rows 16 at a time in the 16x256b shape (row r in
//               lanes 4 r .. 4 r + 3), the running max per row in shared memory,
//               raised (and O^T rescaled) only when a score exceeds it by 2^8
//   warps 5-12  gather 64 keys per stage by 16-byte cp.async, two stages of four
//               dim groups, each refilled as soon as its part of P.V is done
// A unit writes the normalised O and the log-sum-exp of its share; the
// tail/merge kernel adds the tree part and merges the splits.
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kBaThreads = 416;
constexpr int kBaProducers = 256;
constexpr int kBaGroups = 4;                    // dims {512-575, 0-127}, {128-255}, {256-383}, {384-511}
constexpr int kBaKeys = 64;
constexpr int kBaRows = kBlockRows;             // 64
constexpr int kBaStages = 2;
constexpr int kBaChunk = kBaKeys * 128;         // 64 dims of 64 keys: 8 KB
constexpr int kBaStageBytes = 9 * kBaChunk;     // 73728
constexpr int kBaOffQ = kBaStages * kBaStageBytes;
constexpr int kBaOffP = kBaOffQ + 9 * kBaChunk;
constexpr int kBaOffMask = kBaOffP + kBaChunk;                  // [2][64] row masks of the stage's keys
constexpr int kBaOffMax = kBaOffMask + kBaStages * kBaKeys * 8; // [64] running max
constexpr int kBaOffAlpha = kBaOffMax + kBaRows * 4;            // [64] rescale factors, later row sums
constexpr int kBaOffBar = kBaOffAlpha + kBaRows * 4;
constexpr int kBaSmem = kBaOffBar + 256 + 1024;
static_assert(kBaSmem <= 232448, "one CTA's shared memory");
constexpr uint32_t kBaColS = 256;               // O^T [0, 256), S buffers 2 x 64
constexpr float kBaUnset = -1e30f;              // running max of a row that has seen no key
constexpr float kBaThreshold = 8.f;             // log2 units
constexpr float kBaLn2 = 0.69314718055994531f;

struct BaShared {
  uint64_t k_full[kBaStages][kBaGroups];
  uint64_t k_empty[kBaStages][kBaGroups];  // this group's part of the tile's P.V is done (and those before it)
  uint64_t s_full[2], s_free[2];
  uint64_t p_ready;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int fail[2];  // softmax: a wait of tile t ran out, by parity of t
};
static_assert(sizeof(BaShared) <= 256, "barrier block");

// 16 TMEM lanes x 64 columns over a warp: v[4 i + 2 h + e] = (lane L/4 + 8 h, column 8 i + 2 (L % 4) + e).
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

struct Group {
  int b, row0, rows;  // request, first row within the request, rows
};
__device__ __forceinline__ Group group_of(const BlockAttnParams& p, int g) {
  Group u;
  u.b = g / p.groups;
  const int k = g - u.b * p.groups;
  if (p.heads <= kBaRows) {
    u.row0 = k * p.group_nodes * p.heads;
    u.rows = min(p.group_nodes * p.heads, p.nodes * p.heads - u.row0);
  } else {
    const int slices = (p.heads + kBaRows - 1) / kBaRows;
    const int t = k / slices, sl = k - t * slices;
    u.row0 = t * p.heads + sl * kBaRows;
    u.rows = min(kBaRows, p.heads - sl * kBaRows);
  }
  return u;
}

__global__ void __launch_bounds__(kBaThreads, 1) block_attn_kernel(const BlockAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  BaShared& sh = *reinterpret_cast<BaShared*>(smem + kBaOffBar);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sh.abort;
  const int g = blockIdx.x, split = blockIdx.y;
  const Group u = group_of(p, g);
  int L = __ldg(p.prefix_len + u.b);
  L = L < 0 ? 0 : (L > p.max_prefix_len ? p.max_prefix_len : L);
  grid_dep_launch();  // the tail/merge kernel
  grid_dep_wait();    // the lists
  const int count = __ldcg(p.list_len + g);
  const BlockEntry* list = p.list + static_cast<int64_t>(g) * p.list_cap;
  const int64_t keys = static_cast<int64_t>(count) * p.block;
  const int64_t all_tiles = (keys + kBaKeys - 1) / kBaKeys;
  const int t0 = static_cast<int>(all_tiles * split / p.splits);
  const int n = static_cast<int>(all_tiles * (split + 1) / p.splits) - t0;  // tiles of this unit
  const int64_t prow0 = (static_cast<int64_t>(u.b) * p.splits + split) * p.pstride + u.row0;

  if (n == 0) {  // no key: a partial of weight zero
    float4* o = reinterpret_cast<float4*>(p.o_part + prow0 * kDv);
    for (int i = tid; i < u.rows * (kDv / 4); i += kBaThreads) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = tid; i < u.rows; i += kBaThreads) p.lse_part[prow0 + i] = -CUDART_INF_F;
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kBaStages; ++i)
      for (int x = 0; x < kBaGroups; ++x) {
        mbar_init(&sh.k_full[i][x], kBaProducers + (x == 0 ? 8 : 0));  // group 0 carries the key masks
        mbar_init(&sh.k_empty[i][x], 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 128);
    }
    mbar_init(&sh.p_ready, 128);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    sh.fail[0] = sh.fail[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  {  // the group's query rows (consecutive in q), zeros behind them
    const uint16_t* q = p.q + (static_cast<int64_t>(u.b) * p.nodes * p.heads + u.row0) * kDqk;
    for (int i = tid; i < kBaRows * kChunks; i += kBaThreads) {
      const int r = i / kChunks, x = i - r * kChunks;
      cp_async16(base + kBaOffQ + (x >> 3) * kBaChunk + r * 128 + (((x & 7) ^ (r & 7)) << 4),
                 r < u.rows ? q + static_cast<int64_t>(r) * kDqk + x * 8 : q, r < u.rows ? 16u : 0u);
    }
    float* mx = reinterpret_cast<float*>(smem + kBaOffMax);
    for (int i = tid; i < kBaRows; i += kBaThreads) mx[i] = kBaUnset;
    cp_async_commit();
    cp_async_wait<0>();
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  bool ok = true;

  if (warp == 0) {
    if (elect_one()) {
      const int ncol = (u.rows + 15) / 16 * 16;
      const uint32_t idesc_s = idesc_bf16_f32(64, ncol, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(128, ncol, true, true);
      const uint64_t d_k = smem_desc(base, 16, 1024, kSwizzle128B);
      const uint64_t d_q = smem_desc(base + kBaOffQ, 16, 1024, kSwizzle128B);
      const uint64_t d_v = smem_desc(base, kBaChunk, 1024, kSwizzle128B);            // MN-major
      const uint64_t d_p = smem_desc(base + kBaOffP, kBaChunk, 1024, kSwizzle128B);  // MN-major
      int s_tile = 0, s_group = 0, pv = 0;
      // P.V(t) first when it is ready: it frees the stage that the loads wait for
      for (uint32_t spin = 0; pv < n;) {
        if (pv < s_tile && mbar_test_wait(&sh.p_ready, pv & 1)) {
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t v = desc_advance(d_v, (pv & 1) * kBaStageBytes);
          const uint32_t more = pv > 0 ? 1u : 0u;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(tmem + mt * kBaRows, desc_advance(v, mt * 2 * kBaChunk + ks * 2048), desc_advance(d_p, ks * 2048),
                     idesc_o, ks > 0 ? 1u : more);
            mma_commit(&sh.k_empty[pv & 1][mt]);
          }
          ++pv;
          spin = 0;
          continue;
        }
        if (s_tile < n && mbar_test_wait(&sh.k_full[s_tile & 1][s_group], (s_tile >> 1) & 1) &&
            (s_group > 0 || s_tile < 2 || mbar_test_wait(&sh.s_free[s_tile & 1], ((s_tile >> 1) - 1) & 1))) {
          fence_proxy_async_smem();  // the stage was written by cp.async
          tc_fence_after();
          const uint64_t k = desc_advance(d_k, (s_tile & 1) * kBaStageBytes);
          const uint32_t d = tmem + kBaColS + (s_tile & 1) * kBaRows;
          if (s_group == 0) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)  // the rope dims
              mma_ss(d, desc_advance(k, 8 * kBaChunk + ks * 32), desc_advance(d_q, 8 * kBaChunk + ks * 32), idesc_s,
                     ks > 0 ? 1u : 0u);
          }
          const uint64_t kg = desc_advance(k, s_group * 2 * kBaChunk), qg = desc_advance(d_q, s_group * 2 * kBaChunk);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss(d, desc_advance(kg, (ks >> 2) * kBaChunk + (ks & 3) * 32),
                   desc_advance(qg, (ks >> 2) * kBaChunk + (ks & 3) * 32), idesc_s, 1u);
          if (++s_group == kBaGroups) {
            mma_commit(&sh.s_full[s_tile & 1]);
            s_group = 0;
            ++s_tile;
          }
          spin = 0;
          continue;
        }
        if (++spin > 16 * DDT_WAIT_LIMIT || ((spin & 255) == 255 && *abort)) {
          ok = false;
          break;
        }
      }
      mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
  } else if (warp >= 5) {
    // ------------------------------------------------------------------ producers: 8 keys per warp
    const int pw = warp - 5;
    const int32_t* slots = p.slot_idx + static_cast<int64_t>(u.b) * p.slot_stride;
    // key of this lane in tile t: its block entry, then its slot
    auto entry_of = [&](int t, int* pos, uint64_t* mask) {
      *pos = -1;
      *mask = 0;
      const int64_t i = (static_cast<int64_t>(t0 + t)) * kBaKeys + 8 * pw + lane;
      if (t < n && lane < 8 && i < keys) {
        const int e = static_cast<int>(i / p.block);
        const uint4 raw = __ldcg(reinterpret_cast<const uint4*>(list + e));
        BlockEntry be;
        be.mask = raw.x | (static_cast<unsigned long long>(raw.y) << 32);
        be.block = static_cast<int>(raw.z);
        const int64_t x = static_cast<int64_t>(be.block) * p.block + (i - static_cast<int64_t>(e) * p.block);
        if (x < L) {
          *pos = static_cast<int>(x);
          *mask = be.mask;
        }
      }
    };
    auto slot_at = [&](int pos) -> int {
      if (pos < 0) return -1;
      const int s = __ldg(slots + pos);
      if (s >= 0 && s < p.pool_slots) return s;
      atomicOr(p.status, kStatusBadSlot);
      return -1;
    };
    int pos_n;
    uint64_t mask_c, mask_n;
    entry_of(0, &pos_n, &mask_c);
    int slot_c = slot_at(pos_n);
    entry_of(1, &pos_n, &mask_n);
    for (int t = 0; t < n; ++t) {
      const int slot_n = slot_at(pos_n);  // of tile t + 1
      int pos_f;
      uint64_t mask_f;
      entry_of(t + 2, &pos_f, &mask_f);
      const int st = t & 1;
      const uint32_t sbase = base + st * kBaStageBytes;
#pragma unroll
      for (int x = 0; x < kBaGroups; ++x) {
        const bool w = t < kBaStages || mbar_wait_abortable(&sh.k_empty[st][x], ((t >> 1) - 1) & 1, abort, false, __LINE__);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        if (x == 0) {
          if (lane < 8)
            reinterpret_cast<uint64_t*>(smem + kBaOffMask)[st * kBaKeys + 8 * pw + lane] = slot_c >= 0 ? mask_c : 0;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[st][0]);  // releases the masks
        }
        // pieces of 16 bytes per row: the group's two latent chunks, and with group 0 the rope chunk
        const int per = x == 0 ? 24 : 16;
#pragma unroll
        for (int i = 0; i < per / 4; ++i) {
          const int e = i * 32 + lane;
          const int r = e / per, y = e - r * per;
          const int c = y < 16 ? 2 * x + (y >> 3) : 8;  // 64-dim chunk
          const int row = __shfl_sync(0xffffffffu, slot_c, r);
          const int rr = 8 * pw + r;
          cp_async16(sbase + c * kBaChunk + rr * 128 + (((y & 7) ^ (rr & 7)) << 4),
                     p.kv + (row < 0 ? 0 : static_cast<int64_t>(row) * kDqk + c * 64 + (y & 7) * 8), row < 0 ? 0u : 16u);
        }
        cp_async_arrive_noinc(&sh.k_full[st][x]);
      }
      if (!ok) break;
      slot_c = slot_n;
      mask_c = mask_n;
      pos_n = pos_f;
      mask_n = mask_f;
    }
    cp_async_wait<0>();
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    const int quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int r0 = quarter * 16 + (lane >> 2);  // keys r0 and r0 + 8 of the tile
    const int c0 = 2 * (lane & 3);              // rows 8 i + c0 + {0, 1}
    float* mx = reinterpret_cast<float*>(smem + kBaOffMax);
    float* alpha_sh = reinterpret_cast<float*>(smem + kBaOffAlpha);
    float* scratch = reinterpret_cast<float*>(smem + kBaOffP);  // [4 warps][64], while no P is in use
    const uint64_t* masks = reinterpret_cast<const uint64_t*>(smem + kBaOffMask);
    const uint64_t full = u.rows == 64 ? ~0ull : ((1ull << u.rows) - 1);
    float l[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) l[i] = 0.f;
    bool failed = false;  // a wait of this thread ran out: the warps leave together at the next barrier
    auto wait_pv = [&](int t) {  // P.V(t) has read P, and O^T holds every tile up to t
      if (!mbar_wait_abortable(&sh.k_empty[t & 1][kBaGroups - 1], (t >> 1) & 1, abort, false, __LINE__)) failed = true;
      tc_fence_after();
    };
    for (int t = 0; t < n; ++t) {
      const int st = t & 1;
      // (the masks were released with the stage's first group)
      if (!mbar_wait_abortable(&sh.s_full[st], (t >> 1) & 1, abort, false, __LINE__) ||
          !mbar_wait_abortable(&sh.k_full[st][0], (t >> 1) & 1, abort, false, __LINE__))
        failed = true;
      tc_fence_after();
      float s[32];
      tmem_ld_16x64(tmem + lane_off + kBaColS + st * kBaRows, s);
      tc_fence_before();
      mbar_arrive(&sh.s_free[st]);
      const uint64_t m0 = masks[st * kBaKeys + r0], m1 = masks[st * kBaKeys + r0 + 8];
      const bool part = __any_sync(0xffffffffu, m0 != full || m1 != full);
      bool bad0 = false, bad1 = false;  // a row of non-finite scores that some rows do not read
      if (part) {
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a0 += fabsf(s[4 * i]) + fabsf(s[4 * i + 1]);
          a1 += fabsf(s[4 * i + 2]) + fabsf(s[4 * i + 3]);
        }
        a0 += __shfl_xor_sync(0xffffffffu, a0, 1);
        a1 += __shfl_xor_sync(0xffffffffu, a1, 1);
        a0 += __shfl_xor_sync(0xffffffffu, a0, 2);
        a1 += __shfl_xor_sync(0xffffffffu, a1, 2);
        bad0 = !(a0 < CUDART_INF_F) && m0 != full && m0 != 0;
        bad1 = !(a1 < CUDART_INF_F) && m1 != full && m1 != 0;
        const uint32_t w0[2] = {static_cast<uint32_t>(m0) >> c0, static_cast<uint32_t>(m0 >> 32) >> c0};
        const uint32_t w1[2] = {static_cast<uint32_t>(m1) >> c0, static_cast<uint32_t>(m1 >> 32) >> c0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[4 * i + e] = (w0[i >> 2] >> (8 * (i & 3) + e)) & 1u ? s[4 * i + e] * p.scale_log2 : -CUDART_INF_F;
            s[4 * i + 2 + e] = (w1[i >> 2] >> (8 * (i & 3) + e)) & 1u ? s[4 * i + 2 + e] * p.scale_log2 : -CUDART_INF_F;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] *= p.scale_log2;
      }
      // s is now in log2 units; a score 2^8 above its row's running max raises the max first
      float over = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 m = *reinterpret_cast<const float2*>(mx + 8 * i + c0);
        over = fmax3(over, s[4 * i] - m.x, s[4 * i + 1] - m.y);
        over = fmax3(over, s[4 * i + 2] - m.x, s[4 * i + 3] - m.y);
      }
      if (failed) sh.fail[st] = 1;
      const bool raise = bar_red_or(1, 128, failed || over > kBaThreshold);
      if (raise && *const_cast<volatile int*>(&sh.fail[st])) {
        ok = false;
        break;
      }
      if (raise) {
        if (t > 0) wait_pv(t - 1);  // the scratch is the P buffer, and O^T is rescaled
        bar_sync(1, 128);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(s[4 * i + e], s[4 * i + 2 + e]);
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            if (lane < 4) scratch[quarter * kBaRows + 8 * i + c0 + e] = v;
          }
        bar_sync(1, 128);
        const int st_id = quarter * 32 + lane;  // one thread per row decides
        if (st_id < kBaRows) {
          const float m = mx[st_id];
          const float top = fmaxf(fmaxf(scratch[st_id], scratch[kBaRows + st_id]),
                                  fmaxf(scratch[2 * kBaRows + st_id], scratch[3 * kBaRows + st_id]));
          const bool up = top > m + kBaThreshold;
          alpha_sh[st_id] = up ? fast_exp2(m - top) : 1.f;
          mx[st_id] = up ? top : m;
        }
        bar_sync(1, 128);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[2 * i + e] *= alpha_sh[8 * i + c0 + e];
          }
        if (t > 0) {
#pragma unroll 1
          for (int c = 0; c < 4 * kBaRows; c += 32) {
            float o[32];
            tmem_ld32(tmem + lane_off + c, o);
            uint32_t ob[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) ob[k] = __float_as_uint(o[k] * alpha_sh[(c & 32) + k]);
            tmem_st32(tmem + lane_off + c, ob);
          }
        }
        bar_sync(1, 128);  // scratch is read before P is written over it
      }
      // P^T, row (key) r of 64 columns, 128-byte swizzle
      uint8_t* pb = smem + kBaOffP;
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 m = *reinterpret_cast<const float2*>(mx + 8 * i + c0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = fast_exp2(s[4 * i + 2 * h] - m.x), y = fast_exp2(s[4 * i + 2 * h + 1] - m.y);
          l[2 * i] += x;
          l[2 * i + 1] += y;
          pk[2 * i + h] = pack_bf16x2(x, y);
        }
      }
      if (t > 0) wait_pv(t - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = r0 + 8 * h;
          *reinterpret_cast<uint32_t*>(pb + key * 128 + ((i ^ (key & 7)) << 4) + c0 * 2) = pk[2 * i + h];
        }
      if (part && __any_sync(0xffffffffu, bad0 || bad1)) {
        // A non-finite key row that not every row of the group reads: 0 * inf
        // would spoil the others' O, so its values become zero and the weights
        // of the rows that do read it NaN.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t m = h ? m1 : m0;
          const int key = r0 + 8 * h;
          if (h ? bad1 : bad0) {
            uint8_t* row = smem + st * kBaStageBytes + key * 128;
            for (int x = lane & 3; x < 64; x += 4)
              *reinterpret_cast<uint4*>(row + (x >> 3) * kBaChunk + ((x & 7) << 4)) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t lo = (m >> (8 * i + c0)) & 1 ? 0x7fc0u : 0u, hi = (m >> (8 * i + c0 + 1)) & 1 ? 0x7fc0u : 0u;
              *reinterpret_cast<uint32_t*>(pb + key * 128 + ((i ^ (key & 7)) << 4) + c0 * 2) = lo | (hi << 16);
              if (lo) l[2 * i] = CUDART_NAN_F;
              if (hi) l[2 * i + 1] = CUDART_NAN_F;
            }
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&sh.p_ready);
    }
    if (ok) {
      wait_pv(n - 1);  // O^T is complete and the P buffer free
      if (bar_red_or(1, 128, failed)) ok = false;
    }
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = l[2 * i + e];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (lane < 4) scratch[quarter * kBaRows + 8 * i + c0 + e] = v;
        }
      bar_sync(1, 128);
      const int c = quarter * 32 + lane;
      if (c < kBaRows) {
        const float sum = (scratch[c] + scratch[kBaRows + c]) + (scratch[2 * kBaRows + c] + scratch[3 * kBaRows + c]);
        alpha_sh[c] = sum != 0.f ? 1.f / sum : 0.f;
        if (c < u.rows) p.lse_part[prow0 + c] = sum != 0.f ? (mx[c] + log2f(sum)) * kBaLn2 : -CUDART_INF_F;
      }
    }
  }
  // every warp but the first writes O: quarter of the lanes by warp, three warps a quarter
  if (warp > 0) {
    if (!bar_red_or(2, kBaThreads - 32, !ok)) {
      tc_fence_after();
      const float* inv_l = reinterpret_cast<const float*>(smem + kBaOffAlpha);
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      // lane = value dim: each row's store is 128 contiguous bytes per warp
#pragma unroll 1
      for (int k0 = (warp - 1) >> 2; k0 < 8; k0 += 3) {
        const int mt = k0 >> 1, cc = (k0 & 1) * 32;
        if (cc >= u.rows) continue;
        float o[32];
        tmem_ld32(tmem + lane_off + mt * kBaRows + cc, o);
        float* dst = p.o_part + prow0 * kDv + mt * 128 + (warp & 3) * 32 + lane;
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (cc + k < u.rows) dst[static_cast<int64_t>(cc + k) * kDv] = o[k] * inv_l[cc + k];
      }
    }
  }
  if (!ok) {
    *abort = 1;
    atomicOr(p.status, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The union of a group's lists, in block order, with the rows that list each
// block.  One CTA per group: a mask per block in shared memory, 2048 blocks at a time.
constexpr int kUnThreads = 256;
constexpr int kUnBlocks = 2048;

__global__ void __launch_bounds__(kUnThreads) block_union_kernel(const BlockAttnParams p) {
  __shared__ unsigned long long mask_sh[kUnBlocks];
  __shared__ int cnt[kUnThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch();
  const int g = blockIdx.x;
  const Group u = group_of(p, g);
  int L = __ldg(p.prefix_len + u.b);
  if (L < 0 || L > p.max_prefix_len) {
    if (tid == 0) atomicOr(p.status, kStatusBadPrefix);
    L = L < 0 ? 0 : p.max_prefix_len;
  }
  const int n_blocks = (L + p.block - 1) / p.block;
  const int t_first = u.row0 / p.heads, t_last = (u.row0 + u.rows - 1) / p.heads;
  const int32_t* lists = p.block_idx + (static_cast<int64_t>(u.b) * p.nodes + t_first) * p.topk;
  const int entries = (t_last - t_first + 1) * p.topk;  // at most 64 lists of 2^20
  BlockEntry* out = p.list + static_cast<int64_t>(g) * p.list_cap;
  int base = 0;
  for (int c0 = 0; c0 < n_blocks || c0 == 0; c0 += kUnBlocks) {
    for (int i = tid; i < kUnBlocks; i += kUnThreads) mask_sh[i] = 0;
    __syncthreads();
    for (int i = tid; i < entries; i += kUnThreads) {
      const int x = __ldg(lists + i);
      if (x < 0 || x >= n_blocks) {
        if (x != -1 && c0 == 0) atomicOr(p.status, kStatusBadBlock);
        continue;
      }
      if (x < c0 || x - c0 >= kUnBlocks) continue;
      const int t = i / p.topk;  // node of the group: its rows [t H, t H + H)
      const int lo = t * p.heads, hi = min(u.rows, lo + p.heads);
      const unsigned long long below = hi == 64 ? ~0ull : ((1ull << hi) - 1);
      atomicOr(&mask_sh[x - c0], below & ~((1ull << lo) - 1));
    }
    __syncthreads();
    const int here = min(kUnBlocks, n_blocks - c0);
    for (int i0 = 0; i0 < here; i0 += kUnThreads) {
      const unsigned long long m = i0 + tid < here ? mask_sh[i0 + tid] : 0;
      const uint32_t vote = __ballot_sync(0xffffffffu, m != 0);
      if (lane == 0) cnt[warp] = __popc(vote);
      __syncthreads();
      int at = base;
#pragma unroll
      for (int w = 0; w < kUnThreads / 32; ++w) {
        if (w < warp) at += cnt[w];
        base += cnt[w];
      }
      if (m != 0) {
        BlockEntry e;
        e.mask = m;
        e.block = c0 + i0 + tid;
        e.pad = 0;
        out[at + __popc(vote & ((1u << lane) - 1u))] = e;
      }
      __syncthreads();
    }
  }
  if (tid == 0) p.list_len[g] = base;
}

}  // namespace

cudaError_t configure_block_attn() {
  return cudaFuncSetAttribute(block_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBaSmem);
}

cudaError_t launch_block_union(const BlockAttnParams& p, cudaStream_t stream) {
  block_union_kernel<<<p.batch * p.groups, kUnThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_block_attn(const BlockAttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.batch * p.groups, p.splits);
  cfg.blockDim = dim3(kBaThreads);
  cfg.dynamicSmemBytes = kBaSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_attn_kernel, p);
}

}  // namespace ddt
