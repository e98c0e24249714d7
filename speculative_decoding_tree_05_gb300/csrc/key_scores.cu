// key_scores.cu -- a reduction of exp(q.k) or of q.k over query rows, per key.
//
// Two operators need, for every key row k_j of a request, a value summed or
// maximised over that request's query rows q_r:
//   key weights     w_j   = sum_r exp(sm_scale q_r.k_j - lse_r)
//   block selection s_tj  = scale_j * max over the heads r of node t of (qs_r * q_r.m_j)
// The keys are the M side of the product and the query rows the N side, the
// reverse of attention: an accumulator lane then belongs to one key and every
// reduction over the rows stays inside a thread (no shuffle, no atomic, one
// fixed order, so the results are the same bits on every run), and each key row
// is fetched from the pool once, whatever the number of query rows.
//
// A pair of CTAs (640 threads each) shares every MMA: M = 256 keys, 128 in each
// CTA, N = up to 128 query rows, half of them loaded by each, which halves the
// query traffic from L2 (each key tile streams all query rows past it).  A loop
// over tiles of 256 keys:
//   warp 0        TMEM; in CTA 0 lane 0 issues the MMAs of the pair
//   warp 1        lane 0 loads its half of the query rows by TMA: 3 stages of 192 dims
//                 (a wait costs the issuing thread as much as three MMAs: 12 MMAs a stage)
//   warp 2        in CTA 1, lane 0 tells CTA 0 which key groups have landed
//   warps 4-11    two epilogue sets: one key per thread, each set takes half of a
//                 tile's query rows, so that a score buffer is free again well
//                 before the tensor core has filled the other one
//   warps 12-19   gather the key rows by 16-byte cp.async, zero-filled where
//                 there is no key, into three 192-dim groups.  A group is
//                 refilled as soon as the last query tile has used it, so with
//                 one query tile (the memory-bound case) two of the three
//                 groups are always in flight.
// The tensor core truncates each 16-dim step of an accumulation, a bias that
// grows with the running sum: dims 0-287 and 288-575 go to two accumulators,
// added in fp32, which halves it (TMEM: 2 tiles x 2 accumulators x 128 columns).
#include <cuda_runtime.h>
#include <math_constants.h>
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kScThreads = 640;
constexpr int kScKeys = 128;                    // per CTA
constexpr int kScChunk = kScKeys * 128;         // 64 dims of 128 keys: 16 KB
constexpr int kScGroups = 3;
constexpr int kScGroupBytes = 3 * kScChunk;     // 192 dims
constexpr int kScStages = 3;
constexpr int kScQChunk = kScoreTileRows / 2 * 128;              // 8 KB: this CTA's half of the rows, 64 dims
constexpr int kScStageBytes = 3 * kScQChunk;
constexpr int kScOffQ = kScGroups * kScGroupBytes;
constexpr int kScOffAux = kScOffQ + kScStages * kScStageBytes;   // [2 sets][128] row constants
constexpr int kScOffComb = kScOffAux + 2 * kScoreTileRows * 4;   // [2][128] sums handed from set 1 to set 0
constexpr int kScSmem = kScOffComb + 2 * kScKeys * 4 + 1024;
constexpr int kScProducers = 256;
constexpr float kScLog2e = 1.4426950408889634f;

struct ScShared {
  uint64_t k_full[kScGroups], k_empty[kScGroups];
  uint64_t k_peer[kScGroups];   // CTA 0: CTA 1's group has landed
  uint64_t q_full[kScStages];   // CTA 0: both halves of the stage have landed
  uint64_t q_empty[kScStages];
  uint64_t s_full[2];
  uint64_t s_free[2];           // CTA 0: the 16 epilogue warps of the pair have read the scores
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ int clamp_len(const int32_t* prefix_len, int b, int max_len) {
  const int L = __ldg(prefix_len + b);
  return L < 0 ? 0 : (L > max_len ? max_len : L);
}

// 16 consecutive columns of two accumulators of this thread's TMEM lane, added.
__device__ __forceinline__ void tmem_ld16_sum(uint32_t a, uint32_t b, float (&v)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(a), "r"(b)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]) + __uint_as_float(r[16 + i]);
}

// Keys of request b: positions, or blocks of positions.
__device__ __forceinline__ int key_count(const ScoreParams& p, int b) {
  const int L = clamp_len(p.prefix_len, b, p.max_prefix_len);
  return (L + p.block - 1) / p.block;
}

// A unit: 256 consecutive keys of one request against one share of its query tiles.
struct ScUnit {
  int b, kt, t0, t1, n;  // request, key tile, query tiles [t0, t1), keys of the request
};
__device__ __forceinline__ bool unit_at(const ScoreParams& p, int u, ScUnit* x) {
  const int s = u % p.splits, v = u / p.splits;
  x->b = v / p.key_tiles;
  x->kt = v - x->b * p.key_tiles;
  x->t0 = static_cast<int>(static_cast<int64_t>(p.tiles) * s / p.splits);
  x->t1 = static_cast<int>(static_cast<int64_t>(p.tiles) * (s + 1) / p.splits);
  x->n = key_count(p, x->b);
  return x->kt * (2 * kScKeys) < x->n;
}

template <int kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kScThreads, 1)
    score_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort = &sh.abort;
  grid_dep_launch();

  if (tid == 0) {
    for (int i = 0; i < kScGroups; ++i) {
      mbar_init(&sh.k_full[i], kScProducers);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.k_peer[i], 1);
    }
    for (int i = 0; i < kScStages; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 16);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(&sh.tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  const int units = p.units;
  bool ok = true;

  // every role walks the same units: those of its pair that hold keys
  ScUnit u;
  if (warp == 0) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(2 * kScKeys, p.tile_n, false, false);
      const uint64_t d_k = smem_desc(base, 16, 1024, kSwizzle128B);
      const uint64_t d_q = smem_desc(base + kScOffQ, 16, 1024, kSwizzle128B);
      uint32_t n_unit = 0, n_stage = 0, n_tile = 0;
      // A probe of a barrier takes as long as three MMAs, so each is probed a step
      // before it is needed, while MMAs are being issued: the next stage of query
      // rows, and at a tile's last stage the other score buffer.
      bool q_ok = false, s_ok = false;
      for (int i = pair; ok && i < units; i += pairs) {
        if (!unit_at(p, i, &u)) continue;
        for (int qt = u.t0; ok && qt < u.t1; ++qt, ++n_tile) {
          const uint32_t buf = n_tile & 1;
          if (n_tile >= 2 && !s_ok &&
              !mbar_wait_abortable(&sh.s_free[buf], ((n_tile >> 1) - 1) & 1, abort, true, __LINE__)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + buf * 2 * kScoreTileRows;
          for (int g = 0; g < kScGroups; ++g, ++n_stage) {
            if (qt == u.t0) {
              if (!mbar_wait_abortable(&sh.k_full[g], n_unit & 1, abort, false, __LINE__) ||
                  !mbar_wait_abortable(&sh.k_peer[g], n_unit & 1, abort, true, __LINE__)) {
                ok = false;
                break;
              }
              fence_proxy_async_smem();  // the rows were written by cp.async
            }
            const uint32_t st = n_stage % kScStages;
            if (!q_ok && !mbar_wait_abortable(&sh.q_full[st], (n_stage / kScStages) & 1, abort, false, __LINE__)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t next = n_stage + 1;
            q_ok = mbar_test_wait(&sh.q_full[next % kScStages], (next / kScStages) & 1);
            if (g == 2) s_ok = n_tile >= 1 && mbar_test_wait_cluster(&sh.s_free[buf ^ 1], (((n_tile + 1) >> 1) - 1) & 1);
            const uint64_t a = desc_advance(d_k, g * kScGroupBytes), q = desc_advance(d_q, st * kScStageBytes);
#pragma unroll
            for (int k = 0; k < 12; ++k) {
              // the accumulators change at step 18, the middle of the second group
              const uint32_t upper = g == 2 || (g == 1 && k >= 6) ? kScoreTileRows : 0;
              const uint32_t fresh = (g == 0 && k == 0) || (g == 1 && k == 6);
              mma_ss_pair(d + upper, desc_advance(a, (k >> 2) * kScChunk + (k & 3) * 32),
                          desc_advance(q, (k >> 2) * kScQChunk + (k & 3) * 32), idesc, fresh ? 0u : 1u);
            }
            mma_commit_pair(&sh.q_empty[st]);
            if (qt == u.t1 - 1) mma_commit_pair(&sh.k_empty[g]);
          }
          if (ok) mma_commit_pair(&sh.s_full[buf]);
        }
        ++n_unit;
      }
      mma_commit_pair(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      grid_dep_wait();  // the query rows may come from the kernel before (packed, 8-bit)
      uint32_t n_stage = 0;
      const int half = p.tile_n / 2;
      for (int i = pair; ok && i < units; i += pairs) {
        if (!unit_at(p, i, &u)) continue;
        for (int qt = u.t0; ok && qt < u.t1; ++qt) {
          for (int g = 0; g < kScGroups; ++g, ++n_stage) {
            const uint32_t st = n_stage % kScStages;
            if (n_stage >= kScStages &&
                !mbar_wait_abortable(&sh.q_empty[st], ((n_stage / kScStages) - 1) & 1, abort, false, __LINE__)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&sh.q_full[st], 3 * p.tile_n * 128);  // both halves
            // rows past the tensor's end read as zero; a start past it is moved to the last row
            const int row = min(u.b * p.rows + qt * p.tile_rows + rank * half, p.batch * p.rows - 1);
            const uint32_t full = mapa_shared(smem_u32(&sh.q_full[st]), 0);
#pragma unroll
            for (int c = 0; c < 3; ++c)
              tma_load_2d_pair(base + kScOffQ + st * kScStageBytes + c * kScQChunk, &p.tmap_q, (3 * g + c) * 64, row, full);
          }
        }
      }
      // after a give-up, the loads still in flight land before the pair exits
      if (!ok && rank == 0)
        for (uint32_t j = n_stage > kScStages ? n_stage - kScStages : 0; j < n_stage; ++j)
          mbar_wait(&sh.q_full[j % kScStages], (j / kScStages) & 1);
    }
  } else if (warp == 2) {
    if (rank == 1 && lane == 0) {
      uint32_t n_unit = 0;
      for (int i = pair; ok && i < units; i += pairs) {
        if (!unit_at(p, i, &u)) continue;
        for (int g = 0; ok && g < kScGroups; ++g) {
          if (!mbar_wait_abortable(&sh.k_full[g], n_unit & 1, abort, false, __LINE__)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          mbar_arrive_remote(mapa_shared(smem_u32(&sh.k_peer[g]), 0));
        }
        ++n_unit;
      }
    }
  } else if (warp >= 12) {
    const int pw = warp - 12;
    uint32_t n_unit = 0;
    for (int i = pair; ok && i < units; i += pairs) {
      if (!unit_at(p, i, &u)) continue;
      // this warp gathers keys 16 pw .. 16 pw + 15 of the CTA's 128, lane l < 16 holding the row of key l
      const int j = (u.kt * 2 + rank) * kScKeys + 16 * pw + lane;
      int row = -1;  // rows stay below 2^31
      if (lane < 16 && j < u.n) {
        if (p.slot_idx != nullptr) {
          const int slot = __ldg(p.slot_idx + static_cast<int64_t>(u.b) * p.slot_stride + j);
          if (slot >= 0 && slot < p.pool_slots) row = slot;
          if (row < 0) {
            grid_dep_wait();  // (the kernel before may clear the word)
            atomicOr(p.status, kStatusBadSlot);
          }
        } else {
          row = static_cast<int>(u.b * p.key_stride + j);
        }
      }
      for (int g = 0; g < kScGroups; ++g) {
        const bool w = n_unit == 0 || mbar_wait_abortable(&sh.k_empty[g], (n_unit - 1) & 1, abort, false, __LINE__);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        // 24 pieces of 16 bytes per row and group: consecutive lanes take consecutive pieces
#pragma unroll 6
        for (int k = 0; k < 12; ++k) {
          const int e = k * 32 + lane;
          const int r = e / 24, x = e - r * 24;
          const int src_row = __shfl_sync(0xffffffffu, row, r);
          const int rr = 16 * pw + r;
          const uint32_t dst = base + g * kScGroupBytes + (x >> 3) * kScChunk + rr * 128 + (((x & 7) ^ (rr & 7)) << 4);
          const uint16_t* src = p.keys + (src_row < 0 ? 0 : static_cast<int64_t>(src_row) * kDqk + g * 192 + x * 8);
          cp_async16(dst, src, src_row < 0 ? 0u : 16u);
        }
        cp_async_arrive_noinc(&sh.k_full[g]);
      }
      ++n_unit;
    }
    cp_async_wait<0>();
  } else if (warp >= 4) {
    const int set = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // key of the CTA's 128 = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* aux = reinterpret_cast<float*>(smem + kScOffAux) + set * kScoreTileRows;
    float* comb = reinterpret_cast<float*>(smem + kScOffComb);
    const uint32_t free0 = mapa_shared(smem_u32(&sh.s_free[0]), 0), free1 = mapa_shared(smem_u32(&sh.s_free[1]), 0);
    uint32_t n_unit = 0, n_tile = 0;
    grid_dep_wait();  // row_aux, as the query rows
    for (int i = pair; ok && i < units; i += pairs) {
      if (!unit_at(p, i, &u)) continue;
      const int b = u.b, n = u.n;
      const int j = (u.kt * 2 + rank) * kScKeys + r;
      float acc = kMode == kScoreWeight ? 0.f : -CUDART_INF_F;
      const float key_scale = kMode == kScoreBlock && j < n ? __ldg(p.key_scale + b * p.key_stride + j) : 0.f;
      int node = 0, left = p.heads;  // kScoreBlock: the node that the next row belongs to, its rows left
      // the set's columns [cb, ce) of a tile: half of its 16-column steps, or of its
      // nodes; with more heads than tile rows a node spans tiles and set 0 takes them all
      int cb, ce;
      if (kMode == kScoreWeight) {
        const int mid = (p.tile_n / 16 + 1) / 2 * 16;
        cb = set ? mid : 0;
        ce = set ? p.tile_n : mid;
      } else {
        const int mid = p.heads <= kScoreTileRows ? (p.tile_rows / p.heads + 1) / 2 * p.heads : p.tile_rows;
        cb = set ? mid : 0;
        ce = set ? p.tile_rows : mid;
      }
      // row constants of a tile: weights -lse in log2 units, -inf where a row counts for nothing
      auto row_const = [&](int qt) -> float {
        const int row = qt * p.tile_rows + r;
        const bool in = r < p.tile_rows && row < p.rows && qt < u.t1;
        if (kMode == kScoreBlock) return in ? __ldcg(p.row_aux + static_cast<int64_t>(b) * p.rows + row) : CUDART_NAN_F;
        const float l = in ? __ldcg(p.row_aux + static_cast<int64_t>(b) * p.rows + row) : CUDART_INF_F;
        return fabsf(l) == CUDART_INF_F ? -CUDART_INF_F : -l * kScLog2e;
      };
      float a_next = row_const(u.t0);
      for (int qt = u.t0; ok && qt < u.t1; ++qt, ++n_tile) {
        const uint32_t buf = n_tile & 1;
        const int row0 = qt * p.tile_rows;
        const int live = min(p.tile_rows, p.rows - row0);
        bar_sync(1 + set, 128);  // the last tile's are read
        aux[r] = a_next;
        a_next = row_const(qt + 1);
        // the set leaves together if a wait of one of its warps ran out
        const bool got = mbar_wait_abortable(&sh.s_full[buf], (n_tile >> 1) & 1, abort, false, __LINE__);
        if (bar_red_or(1 + set, 128, !got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (kMode == kScoreBlock && p.heads <= kScoreTileRows) node = (row0 + cb) / p.heads;
        const uint32_t col = tmem + lane_off + buf * 2 * kScoreTileRows;
        // steps of 16 columns from a multiple of 16 on: none reaches past the accumulator
        for (int c = cb & ~15; c < ce; c += 16) {
          float s[16];
          tmem_ld16_sum(col + c, col + kScoreTileRows + c, s);
          if (kMode == kScoreWeight) {
            const bool all_live = __all_sync(0xffffffffu, aux[c + (lane & 15)] != -CUDART_INF_F);
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            if (all_live) {
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 a = *reinterpret_cast<const float4*>(aux + c + k);
                t[0] += fast_exp2(fmaf(s[k], p.scale_log2, a.x));
                t[1] += fast_exp2(fmaf(s[k + 1], p.scale_log2, a.y));
                t[2] += fast_exp2(fmaf(s[k + 2], p.scale_log2, a.z));
                t[3] += fast_exp2(fmaf(s[k + 3], p.scale_log2, a.w));
              }
            } else {
              // a row without weight may hold anything, NaN included: it is left out, not multiplied by zero
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float a = aux[c + k];
                t[k & 3] += a == -CUDART_INF_F ? 0.f : fast_exp2(fmaf(s[k], p.scale_log2, a));
              }
            }
            acc += (t[0] + t[1]) + (t[2] + t[3]);
          } else {
            const int k0 = max(0, cb - c), nc = min(min(16, ce - c), live - c);
            // both products are rounded to 32 bits: part of the definition of the score; fmaxf drops a NaN scale
            auto emit = [&] {
              if (j < n)
                p.score[(static_cast<int64_t>(b) * p.nodes + node) * p.key_stride + j] = __fmul_rn(acc, key_scale);
              acc = -CUDART_INF_F;
              left = p.heads;
              ++node;
            };
            if (p.heads % 8 == 0) {  // nodes (and so the live rows) end on multiples of 8
#pragma unroll
              for (int k = 0; k < 16; k += 8) {
                if (k >= k0 && k < nc) {
                  const float4 a = *reinterpret_cast<const float4*>(aux + c + k);
                  const float4 d = *reinterpret_cast<const float4*>(aux + c + k + 4);
                  const float m0 = fmax3(__fmul_rn(s[k], a.x), __fmul_rn(s[k + 1], a.y), __fmul_rn(s[k + 2], a.z));
                  const float m1 = fmax3(__fmul_rn(s[k + 3], a.w), __fmul_rn(s[k + 4], d.x), __fmul_rn(s[k + 5], d.y));
                  const float m2 = fmax3(__fmul_rn(s[k + 6], d.z), __fmul_rn(s[k + 7], d.w), acc);
                  acc = fmax3(m0, m1, m2);
                  if ((left -= 8) == 0) emit();
                }
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                if (k >= k0 && k < nc) {
                  acc = fmaxf(acc, __fmul_rn(s[k], aux[c + k]));
                  if (--left == 0) emit();
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        // relaxed: the scores are in registers, and no store has to be seen (a
        // release at cluster scope took 1900 cycles here, most of a tile)
#ifdef DDT_TEST_HOOKS
        if (warp == 4 && static_cast<int>(n_tile) == p.test_keep_back) continue;
#endif
        if (lane == 0) mbar_arrive_remote_relaxed(buf ? free1 : free0);
      }
      if (bar_red_or(3, 256, !ok)) {
        ok = false;
        break;
      }
      if (kMode == kScoreWeight) {
        // set 1 hands its sum to set 0 (two slots: one barrier a unit is enough)
        float* slot = comb + (n_unit & 1) * kScKeys;
        if (set == 1) slot[r] = acc;
        bar_sync(3, 256);
        if (set == 0 && j < n) {
          const int64_t at = static_cast<int64_t>(b) * p.slot_stride + j;
          const int sl = __ldg(p.slot_idx + at);
          const float sum = sl >= 0 && sl < p.pool_slots ? acc + slot[r] : 0.f;
          if (p.splits > 1)
            p.part[(i % p.splits) * p.part_stride + at] = sum;
          else
            p.weight_out[at] = p.weight_in != nullptr ? fmaf(p.decay, p.weight_in[at], sum) : sum;
        }
      }
      ++n_unit;
    }
  }
  if (!ok) {
    *abort = 1;
    grid_dep_wait();  // (the kernel before may clear the word)
    atomicOr(p.status, kStatusTimeout);
  }
  // the leader's commits arrive here too: the last one before this CTA may leave
  if (warp == 0 && rank == 1 && lane == 0) mbar_wait(&sh.drain, 0);
  tc_fence_before();
  cluster_sync();  // nothing of the pair is in flight towards either CTA
  tc_fence_after();
  if (warp == 0) tmem_dealloc_pair(tmem, 512);
  grid_dep_wait();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.batch; b += kScThreads) {
      const int L = __ldg(p.prefix_len + b);
      if (L < 0 || L > p.max_prefix_len) atomicOr(p.status, kStatusBadPrefix);
    }
  if (blockIdx.x == 0 && p.node_idx != nullptr)
    for (int64_t i = tid; i < static_cast<int64_t>(p.batch) * p.sel; i += kScThreads) {
      const int t = __ldg(p.node_idx + i);
      if (t != -1 && (t < 0 || t >= p.nodes)) atomicOr(p.status, kStatusBadNode);
    }
}

// Sums of the query shares of a key, in order, and the decayed old weight.
__global__ void __launch_bounds__(256) weight_sum_kernel(const __grid_constant__ ScoreParams p) {
  const int b = blockIdx.y;
  const int L = clamp_len(p.prefix_len, b, p.max_prefix_len);
  grid_dep_wait();
  for (int j = blockIdx.x * 256 + threadIdx.x; j < L; j += gridDim.x * 256) {
    const int64_t at = static_cast<int64_t>(b) * p.slot_stride + j;
    float sum = 0.f;
    for (int s = 0; s < p.splits; ++s) sum += __ldcg(p.part + s * p.part_stride + at);
    p.weight_out[at] = p.weight_in != nullptr ? fmaf(p.decay, p.weight_in[at], sum) : sum;
  }
}

// One CTA copies one selected node's rows (H x 72 pieces of 16 bytes) and lse.
__global__ void __launch_bounds__(256) pack_nodes_kernel(PackParams p) {
  const int s = blockIdx.x, b = blockIdx.y;
  // The call's first kernel clears the status word; the score kernel reports a bad entry.
  if (s == 0 && b == 0 && threadIdx.x == 0) *p.status = 0;
  grid_dep_launch();
  const int t = __ldg(p.node_idx + static_cast<int64_t>(b) * p.sel + s);
  const bool in = t >= 0 && t < p.nodes;
  const int64_t to = (static_cast<int64_t>(b) * p.sel + s) * p.heads;
  const int64_t from = (static_cast<int64_t>(b) * p.nodes + (in ? t : 0)) * p.heads;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + from * kDqk);
  uint4* dst = reinterpret_cast<uint4*>(p.q_out + to * kDqk);
  for (int i = threadIdx.x; i < p.heads * kChunks; i += 256) dst[i] = in ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  for (int h = threadIdx.x; h < p.heads; h += 256) p.lse_out[to + h] = in ? __ldg(p.lse + from + h) : CUDART_INF_F;
}

}  // namespace

cudaError_t configure_scores() {
  cudaError_t e = cudaFuncSetAttribute(score_kernel<kScoreWeight>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(score_kernel<kScoreBlock>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScSmem);
}

cudaError_t launch_scores(const ScoreParams& p, ScoreMode mode, int sm_count, bool after_kernel, cudaStream_t stream) {
  // (without a key tile one pair still looks the lengths and nodes over for the status word)
  const int pairs = sm_count >= 4 ? sm_count / 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * (p.units < pairs ? (p.units > 0 ? p.units : 1) : pairs));
  cfg.blockDim = dim3(kScThreads);
  cfg.dynamicSmemBytes = kScSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = after_kernel ? 1 : 0;
  if (mode == kScoreBlock) return cudaLaunchKernelEx(&cfg, score_kernel<kScoreBlock>, p);
  cudaError_t e = cudaLaunchKernelEx(&cfg, score_kernel<kScoreWeight>, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  cfg.gridDim = dim3((p.max_prefix_len + 1023) / 1024, p.batch);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weight_sum_kernel, p);
}

cudaError_t launch_pack_nodes(const PackParams& p, int batch, cudaStream_t stream) {
  pack_nodes_kernel<<<dim3(p.sel, batch), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddt
