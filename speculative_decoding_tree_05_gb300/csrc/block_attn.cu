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
//   O^T[512 dims][rows] += V^T . P^T       2 x 4 x 4 MMAs M128 x N x K16 (V^T: the
//                                          same latent blocks read MN-major)
// O^T takes 256 TMEM columns, so one CTA holds the whole output and nothing is
// exchanged between SMs; scores and sums stay fp32.  P is the sum of two bf16
// parts, what the first leaves of the weight in the second: 16 bits of it count
// and the only rounding to 8 is that of out.  With one part out was off by
// 2.05e-3 of its norm beside the 1.65e-3 of its own rounding; the second costs 13 to
// 18 % (8 requests of 33 nodes x 16 heads: 92.7 -> 105.9 us; both parts as the 128
// columns of one MMA, where TMEM has room for that, 105.8).
//
// Per CTA (576 threads), one unit = (group, split of its key tiles):
//   warp 0       TMEM; one lane issues S(t), dim group by dim group as stage t lands
//   warps 1-8    softmax: 16 keys x 32 rows each, in the 16x256b shape (key r in
//                lanes 4 r .. 4 r + 3), the running max per row in shared memory,
//                raised (and O^T rescaled) only when a score exceeds it by 2^8
//   warp 9       one lane issues P.V(t) when P(t) is written
//   warps 10-17  gather 64 keys per stage, two stages of four dim groups, each
//                refilled as soon as its part of P.V is done: warps 10-13 the latent
//                chunks of the first two groups (4 of 9) and the rope chunk by
//                16-byte cp.async, warps 14-17 the other groups by TMA gather4 (85
//                cycles an instruction and warp), at the same time: an SM gathers
//                about 24 B/clk either way and 34 both ways (L2-resident rows).  The
//                rope chunk comes last: P's second part lies there from the softmax to
//                the end of P.V
// What bounds it: a stage lives from its load through S, the softmax and P.V, and
// only two of them fit beside the query rows, so a tile takes half a stage's life.
// The nodes' ancestors and themselves are keys like the others, behind the blocks'
// keys, each with the rows that see it.  One split writes bf16 and the log-sum-exp
// at once; up to eight of a group of few rows are a cluster, whose CTAs join their
// shares through distributed shared memory; else a unit writes the normalised O and the log-sum-exp of its share, and the
// merge kernel joins them.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <type_traits>
#include "cache_ops.cuh"
#include "ptx.cuh"

namespace ddt {
namespace {

constexpr int kBaThreads = 576;
constexpr int kBaSoftmax = 256;
constexpr int kBaCopiers = 128;                 // threads that gather the copied groups
constexpr int kBaCopied = 2;                    // groups gathered by cp.async
constexpr int kBaGroups = 4;                    // dims {0-127}, {128-255}, {256-383}, {384-575}
constexpr int kBaKeys = 64;
constexpr int kBaRows = kBlockRows;             // 64
constexpr int kBaStages = 2;
constexpr int kBaChunk = kBaKeys * 128;         // 64 dims of 64 keys: 8 KB
constexpr int kBaStageBytes = 9 * kBaChunk;     // 73728
constexpr int kBaOffQ = kBaStages * kBaStageBytes;
constexpr int kBaOffP = kBaOffQ + 9 * kBaChunk;                 // P's first part
constexpr int kBaOffLow = 8 * kBaChunk;                         // its second one: the rope chunk of the tile's stage, read by then
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

// 16 TMEM lanes x 32 columns over a warp: v[4 i + 2 h + e] = (lane L/4 + 8 h, column 8 i + 2 (L % 4) + e).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 8 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
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

// kClustered: the splits of a group are one cluster, which joins them.
template <bool kClustered>
__global__ void __launch_bounds__(kBaThreads, 1) block_attn_kernel(const __grid_constant__ BlockAttnParams p) {
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
  grid_dep_launch();  // the merge kernel
  const int64_t prow0 = (static_cast<int64_t>(u.b) * p.splits + split) * p.pstride + u.row0;

  if (tid == 0) {
    for (int i = 0; i < kBaStages; ++i)
      for (int x = 0; x < kBaGroups; ++x) {
        // every copying thread's cp.async (group 0: and each of its warps' key masks), or two gather warps' arrivals
        // with their bytes (the last group: both)
        mbar_init(&sh.k_full[i][x], (x < kBaCopied || x == kBaGroups - 1 ? kBaCopiers : 0) + (x == 0 ? 4 : 0) +
                                        (x < kBaCopied ? 0 : 2));
        mbar_init(&sh.k_empty[i][x], 1);
      }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], kBaSoftmax / 32);
    }
    mbar_init(&sh.p_ready, kBaSoftmax / 32);
    mbar_init(&sh.drain, 2);
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

  grid_dep_wait();  // the lists: everything before this overlaps their making
  const int count = __ldcg(p.list_len + g);
  const BlockEntry* list = p.list + static_cast<int64_t>(g) * p.list_cap;
  const BlockEntry* tree = p.tree + static_cast<int64_t>(g) * p.nodes;
  const int64_t list_keys = static_cast<int64_t>(count) * p.block, keys = list_keys + __ldcg(p.tree_len + g);
  const int64_t all_tiles = (keys + kBaKeys - 1) / kBaKeys;
  const int t0 = static_cast<int>(all_tiles * split / p.splits);
  const int n = static_cast<int>(all_tiles * (split + 1) / p.splits) - t0;  // tiles of this unit
  if (split == 0 && tid == 0) {
    const int32_t flags = __ldcg(p.list_flags + g);
    if (flags) atomicOr(p.status, flags);
  }
  float* mx = reinterpret_cast<float*>(smem + kBaOffMax);
  if (n == 0 && !kClustered) {  // no key: a partial of weight zero
    uint4* o = p.splits == 1 ? reinterpret_cast<uint4*>(p.out + prow0 * kDv) : reinterpret_cast<uint4*>(p.o_part + prow0 * kDv);
    const int each = p.splits == 1 ? kDv / 8 : kDv / 4;
    for (int i = tid; i < u.rows * each; i += kBaThreads) o[i] = make_uint4(0, 0, 0, 0);
    float* l = p.splits == 1 ? p.lse : p.lse_part;
    for (int i = tid; i < u.rows; i += kBaThreads) l[prow0 + i] = -CUDART_INF_F;
    if (warp == 0) tmem_dealloc(tmem, 512);
    return;
  }

  if (n == 0) {
    for (int i = tid; i < kBaRows; i += kBaThreads) mx[i] = -CUDART_INF_F;
  } else if (warp == 0) {
    if (elect_one()) {
      // scores of all 64 columns (rows of zeros behind the group's): every column read out is defined
      const uint32_t idesc = idesc_bf16_f32(64, kBaRows, false, false);
      const uint64_t d_k = smem_desc(base, 16, 1024, kSwizzle128B);
      const uint64_t d_q = smem_desc(base + kBaOffQ, 16, 1024, kSwizzle128B);
      for (int t = 0; ok && t < n; ++t) {
        const int st = t & 1;
        if (t >= 2 && !mbar_wait_abortable(&sh.s_free[st], ((t >> 1) - 1) & 1, abort, false, __LINE__)) {
          ok = false;
          break;
        }
        const uint64_t k = desc_advance(d_k, st * kBaStageBytes);
        const uint32_t d = tmem + kBaColS + st * kBaRows;
#pragma unroll
        for (int x = 0; x < kBaGroups; ++x) {
          if (!mbar_wait_abortable(&sh.k_full[st][x], (t >> 1) & 1, abort, false, __LINE__)) {
            ok = false;
            break;
          }
          if (x < kBaCopied || x == kBaGroups - 1) fence_proxy_async_smem();  // written by cp.async
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss(d, desc_advance(k, (2 * x + (ks >> 2)) * kBaChunk + (ks & 3) * 32),
                   desc_advance(d_q, (2 * x + (ks >> 2)) * kBaChunk + (ks & 3) * 32), idesc, x + ks > 0 ? 1u : 0u);
          if (x == kBaGroups - 1) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)  // the rope dims
              mma_ss(d, desc_advance(k, 8 * kBaChunk + ks * 32), desc_advance(d_q, 8 * kBaChunk + ks * 32), idesc, 1u);
          }
        }
        if (ok) mma_commit(&sh.s_full[st]);
      }
      mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
  } else if (warp == 9) {
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(128, (u.rows + 15) / 16 * 16, true, true);
      const uint64_t d_v = smem_desc(base, kBaChunk, 1024, kSwizzle128B);            // MN-major
      const uint64_t d_p = smem_desc(base + kBaOffP, kBaChunk, 1024, kSwizzle128B);  // MN-major
      const uint64_t d_low = smem_desc(base + kBaOffLow, kBaChunk, 1024, kSwizzle128B);
      for (int t = 0; t < n; ++t) {
        if (!mbar_wait_abortable(&sh.p_ready, t & 1, abort, false, __LINE__)) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t v = desc_advance(d_v, (t & 1) * kBaStageBytes), low = desc_advance(d_low, (t & 1) * kBaStageBytes);
        const uint32_t more = t > 0 ? 1u : 0u;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t a = desc_advance(v, mt * 2 * kBaChunk + ks * 2048);
            mma_ss(tmem + mt * kBaRows, a, desc_advance(d_p, ks * 2048), idesc, ks > 0 ? 1u : more);
            mma_ss(tmem + mt * kBaRows, a, desc_advance(low, ks * 2048), idesc, 1u);
          }
          mma_commit(&sh.k_empty[t & 1][mt]);
        }
      }
      mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
  } else if (warp >= 10) {
    // ------------------------------------------------------------------ producers
    const int32_t* slots = p.slot_idx + static_cast<int64_t>(u.b) * p.slot_stride;
    // A key's row takes two dependent reads, its block entry and its slot, each a
    // tile ahead of its use: nothing is computed from a value in the tile that
    // reads it (an immediate use stalls the warp for the read: 2000 cycles a tile).
    struct Key {
      uint4 entry;    // of tile t + 1: mask, block or tree slot, which of the two
      int slot;       // of tile t, as read; -1: no key
      uint64_t mask;  // of tile t
    };
    // (a list names each block once, so its keys count in 32 bits; blocks are powers of two)
    const int log_block = 31 - __clz(p.block);
    const uint32_t first = static_cast<uint32_t>(t0) * kBaKeys, n_keys = static_cast<uint32_t>(keys),
                   n_list = static_cast<uint32_t>(list_keys);
    auto read_entry = [&](int t, int k) -> uint4 {  // key k of tile t
      const uint32_t i = first + t * kBaKeys + k;
      if (t >= n || k >= kBaKeys || i >= n_keys) return make_uint4(0, 0, 0xffffffffu, 0);
      return __ldcg(reinterpret_cast<const uint4*>(i < n_list ? list + (i >> log_block) : tree + (i - n_list)));
    };
    auto read_slot = [&](int t, int k, Key& key) {  // of tile t, whose entry has arrived
      const uint32_t i = first + t * kBaKeys + k;
      const int blk = static_cast<int>(key.entry.z);
      const uint32_t pos = (static_cast<uint32_t>(blk) << log_block) + (i & (p.block - 1));
      const bool in = blk >= 0 && (key.entry.w != 0 || pos < static_cast<uint32_t>(L));
      key.mask = in ? key.entry.x | (static_cast<uint64_t>(key.entry.y) << 32) : 0;
      key.slot = in ? (key.entry.w != 0 ? blk : __ldg(slots + pos)) : -1;
    };
    auto row_of = [&](Key& key) -> int {
      if (key.mask != 0 && (key.slot < 0 || key.slot >= p.pool_slots)) {
        atomicOr(p.status, kStatusBadSlot);
        key.mask = 0;
      }
      return key.mask != 0 ? key.slot : -1;
    };
    // 16-byte copies, 32 / kPieces rows at a time: kPieces consecutive pieces (8 a chunk) from chunk c0 on of kRows rows from row0 (a multiple of 8)
    // on; zeros for rows without a slot.  A lane keeps its piece, so that a copy
    // costs a shuffle and two address steps.
    auto copy_rows = [&](uint32_t sbase, int row0, int c0, auto pieces, auto rows, int slot) {
      constexpr int kPieces = decltype(pieces)::value, kStep = 32 / kPieces, kRows = decltype(rows)::value;
      const int y = lane & (kPieces - 1), sub = lane / kPieces;  // piece, row within a step
      const uint32_t dst = sbase + (c0 + (y >> 3)) * kBaChunk + (row0 + sub) * 128;
      const uint16_t* src = p.kv + (c0 * 8 + y) * 8;
#pragma unroll
      for (int i = 0; i < kRows / kStep; ++i) {
        const int row = __shfl_sync(0xffffffffu, slot, i * kStep + sub);
        // the row's place in its swizzle atom: steps of kStep rows leave the low bits to sub
        const uint32_t at = ((y & 7) ^ ((i * kStep + sub) & 7)) << 4;
        cp_async16(dst + i * kStep * 128 + at, row < 0 ? p.kv : src + static_cast<int64_t>(row) * kDqk, row < 0 ? 0u : 16u);
      }
    };
    using P16 = std::integral_constant<int, 16>;
    using P8 = std::integral_constant<int, 8>;
    using R32 = std::integral_constant<int, 32>;
    const bool copier = warp < 14;
    const int row0 = copier ? 16 * (warp - 10) : 32 * (warp & 1);  // the warp's first key: 16 or 32 of them
    const int k = copier && lane >= 16 ? kBaKeys : row0 + lane;    // the lane's key
    const int gx = copier ? 0 : kBaCopied + ((warp - 14) >> 1);    // a gather warp's dim group
    Key key;
    key.entry = read_entry(0, k);
    read_slot(0, k, key);
    key.entry = read_entry(1, k);
    int done = 0;
    auto wait_empty = [&](int t, int x) {
      const bool w = t < kBaStages || mbar_wait_abortable(&sh.k_empty[t & 1][x], ((t >> 1) - 1) & 1, abort, false, __LINE__);
      return __all_sync(0xffffffffu, w) != 0;
    };
    for (int t = 0; ok && t < n; ++t) {
      const int slot = row_of(key);
      const uint64_t mask = key.mask;
      read_slot(t + 1, k, key);
      key.entry = read_entry(t + 2, k);
      const int st = t & 1;
      const uint32_t sbase = base + st * kBaStageBytes;
      if (copier) {
        if (!wait_empty(t, 0)) {
          ok = false;
          break;
        }
        if (lane < 16) reinterpret_cast<uint64_t*>(smem + kBaOffMask)[st * kBaKeys + row0 + lane] = mask;
        copy_rows(sbase, row0, 0, P16(), P16(), slot);
        cp_async_arrive_noinc(&sh.k_full[st][0]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full[st][0]);  // releases the masks
        if (!wait_empty(t, 1)) {
          ok = false;
          break;
        }
        copy_rows(sbase, row0, 2, P16(), P16(), slot);
        cp_async_arrive_noinc(&sh.k_full[st][1]);
        // the rope chunk, with the last group: P's second part lies there until P.V is done
        if (!wait_empty(t, kBaGroups - 1)) {
          ok = false;
          break;
        }
        copy_rows(sbase, row0, 8, P8(), P16(), slot);
        cp_async_arrive_noinc(&sh.k_full[st][kBaGroups - 1]);
      } else {
        if (!wait_empty(t, gx)) {
          ok = false;
          break;
        }
        if (__all_sync(0xffffffffu, slot >= 0)) {
          // lanes 0-15: four of the warp's keys, one of the group's two chunks
          if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[st][gx], 32 * 256);
          __syncwarp();
          const int q = 4 * (lane & 7), c = 2 * gx + ((lane >> 3) & 1);
          const int ra = __shfl_sync(0xffffffffu, slot, q), rb = __shfl_sync(0xffffffffu, slot, q + 1);
          const int rc = __shfl_sync(0xffffffffu, slot, q + 2), rd = __shfl_sync(0xffffffffu, slot, q + 3);
          if (lane < 16)
            tma_gather4(sbase + c * kBaChunk + (row0 + q) * 128, &p.tmap_kv, c * 64, ra, rb, rc, rd, &sh.k_full[st][gx]);
        } else {
          // a key is masked (the list's end, a bad slot): zero-filled copies
          copy_rows(sbase, row0, 2 * gx, P16(), R32(), slot);
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[st][gx]);
        }
      }
      done = t + 1;
    }
    cp_async_wait<0>();
    if (!ok && !copier)  // after a give-up the gathers still in flight land before the CTA exits
      for (int v = max(0, done - 2); v <= done && v < n; ++v) mbar_wait(&sh.k_full[v & 1][gx], (v >> 1) & 1, 1u << 16);
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    const int quarter = warp & 3, half = (warp - 1) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int r0 = quarter * 16 + (lane >> 2);     // keys r0 and r0 + 8 of the tile
    const int c0 = 32 * half + 2 * (lane & 3);     // rows c0 + 8 i + {0, 1}, i < 4
    const int id = half * 128 + quarter * 32 + lane;
    float* alpha_sh = reinterpret_cast<float*>(smem + kBaOffAlpha);
    float* scratch = reinterpret_cast<float*>(smem + kBaOffP);  // [4 quarters][64], while no P is in use
    const uint64_t* masks = reinterpret_cast<const uint64_t*>(smem + kBaOffMask);
    const uint64_t full = u.rows == 64 ? ~0ull : ((1ull << u.rows) - 1);
    float l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = 0.f;
    bool failed = false;  // a wait of this thread ran out: the warps leave together at the next barrier
    auto wait_pv = [&](int t) {  // P.V(t) has read P, and O^T holds every tile up to t
      if (!mbar_wait_abortable(&sh.k_empty[t & 1][kBaGroups - 1], (t >> 1) & 1, abort, false, __LINE__)) failed = true;
      tc_fence_after();
    };
    // column sums or maxima over the 16 keys of the warp, to scratch
    auto to_scratch = [&](const float (&v)[8], auto op) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = v[i];
        x = op(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = op(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = op(x, __shfl_xor_sync(0xffffffffu, x, 16));
        if (lane < 4) scratch[quarter * kBaRows + c0 + 8 * (i >> 1) + (i & 1)] = x;
      }
    };
    float m[8];  // the running max of this thread's rows, as in mx
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = kBaUnset;
    for (int t = 0; t < n; ++t) {
      const int st = t & 1;
      // A look at shared memory takes 100 to 300 cycles beside the gathers, so what
      // can be looked at ahead of the scores is: the last tile's P.V, the key masks
      // (released with the stage's first group).
      bool pv_done = t == 0 || mbar_test_wait(&sh.k_empty[(t - 1) & 1][kBaGroups - 1], ((t - 1) >> 1) & 1);
      if (!mbar_wait_abortable(&sh.k_full[st][0], (t >> 1) & 1, abort, false, __LINE__)) failed = true;
      const uint64_t m0 = masks[st * kBaKeys + r0], m1 = masks[st * kBaKeys + r0 + 8];
      const bool part = __any_sync(0xffffffffu, m0 != full || m1 != full);
      if (!mbar_wait_abortable(&sh.s_full[st], (t >> 1) & 1, abort, false, __LINE__)) failed = true;
      __syncwarp();
      tc_fence_after();
      float s[16];
      tmem_ld_16x32(tmem + lane_off + kBaColS + st * kBaRows + 32 * half, s);
      // A key row that is not finite makes every score of it so, the zero rows' too;
      // a query row that is not spoils its own scores alone.
      bool bad0 = false, bad1 = false;
      if (part) {
        float a0 = CUDART_INF_F, a1 = CUDART_INF_F;  // the least magnitude, a number if there is one
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a0 = fminf(a0, fminf(fabsf(s[4 * i]), fabsf(s[4 * i + 1])));
          a1 = fminf(a1, fminf(fabsf(s[4 * i + 2]), fabsf(s[4 * i + 3])));
        }
        // (of this thread's rows; the others' are asked below)
        bad0 = !(a0 < CUDART_INF_F) && m0 != full && m0 != 0;
        bad1 = !(a1 < CUDART_INF_F) && m1 != full && m1 != 0;
      }
      auto mask = [&] {
        if (!part) return;
        const uint32_t w0 = static_cast<uint32_t>(m0 >> c0), w1 = static_cast<uint32_t>(m1 >> c0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!((w0 >> (8 * i + e)) & 1u)) s[4 * i + e] = -CUDART_INF_F;
            if (!((w1 >> (8 * i + e)) & 1u)) s[4 * i + 2 + e] = -CUDART_INF_F;
          }
      };
      // s becomes the distance to the row's running max, in log2 units; a score 2^8 above it raises it first
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], p.scale_log2, -m[2 * (i >> 2) + (i & 1)]);
      mask();
      float over = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < 8; ++i) over = fmax3(over, s[2 * i], s[2 * i + 1]);
      if (failed) sh.fail[st] = 1;
      const bool raise = bar_red_or(1, kBaSoftmax, failed || over > kBaThreshold || bad0 || bad1);
      if (raise && *const_cast<volatile int*>(&sh.fail[st])) {
        ok = false;
        break;
      }
      if (raise) {
        if (!pv_done) wait_pv(t - 1);  // the scratch is the P buffer, and O^T is rescaled
        pv_done = true;
        uint8_t* bad = smem + kBaOffP + 4 * kBaRows * 4;  // [64 keys][8 threads that hold its scores]
        bad[r0 * 8 + half * 4 + (lane & 3)] = bad0;
        bad[(r0 + 8) * 8 + half * 4 + (lane & 3)] = bad1;
        tmem_ld_16x32(tmem + lane_off + kBaColS + st * kBaRows + 32 * half, s);  // the scores again
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= p.scale_log2;
        mask();
        float top8[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top8[2 * i] = fmaxf(s[4 * i], s[4 * i + 2]);
          top8[2 * i + 1] = fmaxf(s[4 * i + 1], s[4 * i + 3]);
        }
        to_scratch(top8, [](float a, float b) { return fmaxf(a, b); });
        bar_sync(1, kBaSoftmax);
        if (id < kBaRows) {  // one thread per row decides
          const float m = mx[id];
          const float top = fmaxf(fmaxf(scratch[id], scratch[kBaRows + id]),
                                  fmaxf(scratch[2 * kBaRows + id], scratch[3 * kBaRows + id]));
          const bool up = top > m + kBaThreshold;
          alpha_sh[id] = up ? fast_exp2(m - top) : 1.f;
          mx[id] = up ? top : m;
        }
        bad0 = reinterpret_cast<const uint64_t*>(bad)[r0] == 0x0101010101010101ull;
        bad1 = reinterpret_cast<const uint64_t*>(bad)[r0 + 8] == 0x0101010101010101ull;
        bar_sync(1, kBaSoftmax);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = c0 + 8 * (i >> 1) + (i & 1);
          l[i] *= alpha_sh[row];
          m[i] = mx[row];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] -= m[2 * (i >> 2) + (i & 1)];
        if (t > 0) {
#pragma unroll 1
          for (int k0 = 0; k0 < 16; ++k0) {  // this warp's half of the columns, 8 at a time
            const int cc = 32 * half + (k0 & 3) * 8;
            uint32_t o[8];
            tmem_ld8(tmem + lane_off + (k0 >> 2) * kBaRows + cc, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha_sh[cc + k]);
            tmem_st8(tmem + lane_off + (k0 >> 2) * kBaRows + cc, o);
          }
        }
        bar_sync(1, kBaSoftmax);  // scratch is read before P is written over it
      }
      tc_fence_before();
      __syncwarp();
#ifdef DDT_TEST_HOOKS
      if (warp != 1 || t != p.test_keep_back)
#endif
      if (lane == 0) mbar_arrive(&sh.s_free[st]);
      // P^T, row (key) r of 64 columns, 128-byte swizzle
      uint8_t* pb = smem + kBaOffP;
      uint8_t* low = smem + st * kBaStageBytes + kBaOffLow;
      auto p_at = [&](uint8_t* part, int key, int i) {
        return reinterpret_cast<uint32_t*>(part + key * 128 + (((4 * half + i) ^ (key & 7)) << 4) + (lane & 3) * 4);
      };
      uint32_t pk[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = fast_exp2(s[4 * i + 2 * h]), y = fast_exp2(s[4 * i + 2 * h + 1]);
          l[2 * i] += x;
          l[2 * i + 1] += y;
          const uint32_t hi = pack_bf16x2(x, y);
          pk[2 * i + h] = hi;
          // (the differences are exact)
          *p_at(low, r0 + 8 * h, i) = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
        }
      }
      if (!pv_done) wait_pv(t - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) *p_at(pb, r0 + 8 * h, i) = pk[2 * i + h];
      if (part && __any_sync(0xffffffffu, bad0 || bad1)) {
        // A non-finite key row that not every row of the group reads: 0 * inf
        // would spoil the others' O, so its values become zero and the weights
        // of the rows that do read it NaN.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t m = static_cast<uint32_t>((h ? m1 : m0) >> c0);
          const int key = r0 + 8 * h;
          if (h ? bad1 : bad0) {
            uint8_t* row = smem + st * kBaStageBytes + key * 128;
            for (int x = lane & 3; x < 64; x += 4)
              *reinterpret_cast<uint4*>(row + (x >> 3) * kBaChunk + ((x & 7) << 4)) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t lo = (m >> (8 * i)) & 1 ? 0x7fc0u : 0u, hi = (m >> (8 * i + 1)) & 1 ? 0x7fc0u : 0u;
              *p_at(pb, key, i) = lo | (hi << 16);
              if (lo) l[2 * i] = CUDART_NAN_F;
              if (hi) l[2 * i + 1] = CUDART_NAN_F;
            }
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_ready);
    }
    if (ok) {
      wait_pv(n - 1);  // O^T is complete and the P buffer free
      if (bar_red_or(1, kBaSoftmax, failed)) ok = false;
    }
    if (ok) {
      to_scratch(l, [](float a, float b) { return a + b; });
      bar_sync(1, kBaSoftmax);
      if (id < kBaRows) {
        const float sum = (scratch[id] + scratch[kBaRows + id]) + (scratch[2 * kBaRows + id] + scratch[3 * kBaRows + id]);
        alpha_sh[id] = sum != 0.f ? 1.f / sum : 0.f;
        const float log2_sum = sum != 0.f ? mx[id] + log2f(sum) : -CUDART_INF_F;
        float* lse = p.splits == 1 ? p.lse : p.lse_part;
        if (kClustered)
          mx[id] = log2_sum;
        else if (id < u.rows)
          lse[prow0 + id] = log2_sum * kBaLn2;
      }
    }
  }
  // the softmax and gather warps write O: quarter of the lanes by warp, four warps a quarter
  if (n > 0 && warp > 0) {
    if (!bar_red_or(2, kBaThreads - 32, !ok) && warp != 9) {
      tc_fence_after();
      const float* inv_l = reinterpret_cast<const float*>(smem + kBaOffAlpha);
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      // lane = value dim: each row's store is 128 contiguous bytes per warp
#pragma unroll 1
      for (int k0 = warp < 9 ? (warp - 1) >> 2 : (warp - 2) >> 2; k0 < 32; k0 += 4) {
        const int mt = k0 >> 3, cc = (k0 & 7) * 8;
        if (cc >= u.rows) continue;
        uint32_t o[8];
        tmem_ld8(tmem + lane_off + mt * kBaRows + cc, o);
        const int dim = mt * 128 + (warp & 3) * 32;
        if (p.splits == 1) {
          // two rows a store: even lanes hold a pair of dims of the first, odd lanes of the second
          uint16_t* dst = p.out + (prow0 + cc + (lane & 1)) * kDv + dim + (lane & ~1);
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float x = __uint_as_float(o[k]) * inv_l[cc + k], y = __uint_as_float(o[k + 1]) * inv_l[cc + k + 1];
            const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
            if (cc + k + (lane & 1) < u.rows)
              *reinterpret_cast<uint32_t*>(dst + k * kDv) = lane & 1 ? pack_bf16x2(got, y) : pack_bf16x2(x, got);
          }
        } else if (kClustered) {  // the stages are free: rows of 512 fp32
          float* dst = reinterpret_cast<float*>(smem) + cc * kDv + dim + lane;
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k * kDv] = __uint_as_float(o[k]) * inv_l[cc + k];
        } else {
          float* dst = p.o_part + (prow0 + cc) * kDv + dim + lane;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (cc + k < u.rows) dst[k * kDv] = __uint_as_float(o[k]) * inv_l[cc + k];
        }
      }
    }
  }
  if (!ok) {
    *abort = 1;
    atomicOr(p.status, kStatusTimeout);
  }
  if (kClustered) {
    // the group's splits are one cluster: each CTA joins a share of the rows from
    // all of them, out = sum of w_s o_s / sum of w_s with w_s = 2^(log2_sum_s - max)
    __syncwarp();
    cluster_sync();
    const int share = (u.rows + p.splits - 1) / p.splits, first = split * share, rows = min(share, u.rows - first);
    const int64_t grow = static_cast<int64_t>(u.b) * p.pstride + u.row0 + first;
    for (int i = tid; i < rows * (kDv / 4); i += kBaThreads) {
      const int r = i / (kDv / 4), d = (i % (kDv / 4)) * 4;
      const uint32_t from_lse = smem_u32(mx + first + r), from_o = base + ((first + r) * kDv + d) * 4;
      float w[kBlockCluster], top = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < kBlockCluster; ++k) {
        w[k] = k < p.splits ? __int_as_float(ld_shared_cluster_b32(mapa_shared(from_lse, k))) : -CUDART_INF_F;
        top = fmaxf(top, w[k]);
      }
      float4 o[kBlockCluster];
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kBlockCluster; ++k) {
        // a NaN (a non-finite key that the row reads) stays one; a share without keys is not read
        w[k] = w[k] == -CUDART_INF_F ? 0.f : fast_exp2(w[k] - top);
        o[k] = w[k] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : ld_shared_cluster_f4(mapa_shared(from_o, k));
        sum += w[k];
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kBlockCluster; ++k) {
        acc.x = fmaf(w[k], o[k].x, acc.x);
        acc.y = fmaf(w[k], o[k].y, acc.y);
        acc.z = fmaf(w[k], o[k].z, acc.z);
        acc.w = fmaf(w[k], o[k].w, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2*>(p.out + (grow + r) * kDv + d) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (d == 0) p.lse[grow + r] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * kBaLn2;
    }
    cluster_sync();  // no CTA leaves while its rows are read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The union of a group's lists, in block order, with the rows that list each
// block, and the tree rows that its nodes see.  One CTA per group: a mask per
// block in shared memory, 4096 blocks at a time.
constexpr int kUnThreads = 1024;
constexpr int kUnWarps = kUnThreads / 32;
constexpr int kUnBlocks = 4096;

// a |= m in shared memory, by halves (32-bit atomics need no loop)
__device__ __forceinline__ void or_mask(unsigned long long* a, unsigned long long m) {
  unsigned* half = reinterpret_cast<unsigned*>(a);
  const unsigned lo = static_cast<unsigned>(m), hi = static_cast<unsigned>(m >> 32);
  if (lo) atomicOr(half, lo);
  if (hi) atomicOr(half + 1, hi);
}

__global__ void __launch_bounds__(kUnThreads) block_union_kernel(const __grid_constant__ BlockAttnParams p) {
  __shared__ unsigned long long mask_sh[kUnBlocks];
  __shared__ unsigned long long tree_sh[kMaxNodes];
  __shared__ int par_sh[kMaxNodes], slot_sh[kMaxNodes];
  __shared__ int cnt[kUnWarps];
  __shared__ int flags_sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.x;
  // The call's first kernel clears the status word; its own findings go to it
  // through the attention kernel, which runs after the clear.
  if (tid == 0) {
    flags_sh = 0;
    if (g == 0) *p.status = 0;
  }
  const Group u = group_of(p, g);
  const int t_first = u.row0 / p.heads, t_last = (u.row0 + u.rows - 1) / p.heads;
  const int32_t* lists = p.block_idx + (static_cast<int64_t>(u.b) * p.nodes + t_first) * p.topk;
  const int entries = (t_last - t_first + 1) * p.topk;  // at most 64 lists of 2^20
  const int entry0 = tid < entries ? __ldg(lists + tid) : -1;  // on its way while the rest is set up
  if (tid < p.nodes) {
    par_sh[tid] = __ldg(p.tree_parent + static_cast<int64_t>(u.b) * p.nodes + tid);
    slot_sh[tid] = __ldg(p.tree_slot_idx + static_cast<int64_t>(u.b) * p.nodes + tid);
    tree_sh[tid] = 0;
  }
  int L = __ldg(p.prefix_len + u.b);
  const int bad_len = L < 0 || L > p.max_prefix_len ? kStatusBadPrefix : 0;
  L = L < 0 ? 0 : (L > p.max_prefix_len ? p.max_prefix_len : L);
  for (int i = tid; i < kUnBlocks; i += kUnThreads) mask_sh[i] = 0;
  __syncthreads();
  grid_dep_launch();
  const int n_blocks = (L + p.block - 1) / p.block;
  auto rows_of = [&](int t) -> unsigned long long {  // of the group's t-th node: its rows [t H, t H + H)
    const int lo = t * p.heads, hi = min(u.rows, lo + p.heads);
    return (hi == 64 ? ~0ull : ((1ull << hi) - 1)) & ~((1ull << lo) - 1);
  };
  const int walker = kUnThreads - 1 - tid;  // the last warps walk while the first mark the lists
  if (walker <= t_last - t_first) {
    // a node's walk to the root: a link that is no earlier node ends it, a slot outside the pool is left out
    int v = t_first + walker, flags = walker == 0 ? bad_len : 0;
    for (int guard = 0; v >= 0 && guard < p.nodes; ++guard) {
      const int slot = slot_sh[v], up = par_sh[v];
      if (slot >= 0 && slot < p.pool_slots)
        or_mask(&tree_sh[v], rows_of(walker));
      else
        flags |= kStatusBadSlot;
      if (v == 0 ? up != -1 : (up < 0 || up >= v)) {
        flags |= kStatusBadParent;
        break;
      }
      v = up;
    }
    if (flags) atomicOr(&flags_sh, flags);
  }
  BlockEntry* out = p.list + static_cast<int64_t>(g) * p.list_cap;
  int base = 0;
  for (int c0 = 0; c0 < n_blocks || c0 == 0; c0 += kUnBlocks) {
    if (c0 > 0) {
      for (int i = tid; i < kUnBlocks; i += kUnThreads) mask_sh[i] = 0;
      __syncthreads();
    }
    for (int i = tid; i < entries; i += kUnThreads) {
      const int x = i == tid ? entry0 : __ldg(lists + i);
      if (x < 0 || x >= n_blocks) {
        if (x != -1 && c0 == 0) atomicOr(&flags_sh, kStatusBadBlock);
        continue;
      }
      if (x >= c0 && x - c0 < kUnBlocks) or_mask(&mask_sh[x - c0], rows_of(i / p.topk));
    }
    __syncthreads();
    const int here = min(kUnBlocks, n_blocks - c0);
    for (int i0 = 0; i0 < here; i0 += kUnThreads) {
      const unsigned long long m = i0 + tid < here ? mask_sh[i0 + tid] : 0;
      const uint32_t vote = __ballot_sync(0xffffffffu, m != 0);
      if (lane == 0) cnt[warp] = __popc(vote);
      __syncthreads();
      const int c = cnt[lane];
      const int at = base + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
      base += __reduce_add_sync(0xffffffffu, c);
      if (m != 0) {
        BlockEntry e;
        e.mask = m;
        e.index = c0 + i0 + tid;
        e.tree = 0;
        out[at + __popc(vote & ((1u << lane) - 1u))] = e;
      }
      __syncthreads();
    }
  }
  if (warp == 0) {  // the tree rows, in node order
    BlockEntry* tree = p.tree + static_cast<int64_t>(g) * p.nodes;
    int n = 0;
    for (int i0 = 0; i0 < p.nodes; i0 += 32) {
      const unsigned long long m = i0 + lane < p.nodes ? tree_sh[i0 + lane] : 0;
      const uint32_t vote = __ballot_sync(0xffffffffu, m != 0);
      if (m != 0) {
        BlockEntry e;
        e.mask = m;
        e.index = slot_sh[i0 + lane];
        e.tree = 1;
        tree[n + __popc(vote & ((1u << lane) - 1u))] = e;
      }
      n += __popc(vote);
    }
    if (lane == 0) {
      p.list_len[g] = base;
      p.tree_len[g] = n;
      p.list_flags[g] = flags_sh;
    }
  }
}
static_assert(kUnWarps == 32, "the prefix over warps takes one lane each");

// The launch of `groups` groups in `splits` splits, a cluster each if `clustered`.
struct BaLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  BaLaunch(int groups, int splits, bool clustered) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.z = 1;
    attr[1].val.clusterDim.y = splits;
    cfg.gridDim = dim3(groups, splits);
    cfg.blockDim = dim3(kBaThreads);
    cfg.dynamicSmemBytes = kBaSmem;
    cfg.attrs = attr;
    cfg.numAttrs = clustered ? 2 : 1;
  }
};

}  // namespace

cudaError_t configure_block_attn(BlockClusters* clusters) {
  cudaError_t e = cudaFuncSetAttribute(block_attn_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBaSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(block_attn_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBaSmem);
  if (e != cudaSuccess) return e;
  for (int s = 2; s <= kBlockCluster; ++s) {
    int n = 0;
    BaLaunch l(1, s, true);
    if (cudaOccupancyMaxActiveClusters(&n, block_attn_kernel<true>, &l.cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;  // a merge kernel does it
    }
    clusters->count[s] = n;
  }
  return cudaSuccess;
}

// A join through distributed shared memory reads at about 25 B/clk, so it suits few
// rows (16 requests of 16 rows in a graph: 17.9 us, 19.0 with a merge kernel; of 64
// rows 29.1 and 25.2); clusters that wait for others' SMs suit none.
bool block_cluster_fits(int64_t groups, int rows, int splits, const BlockClusters& clusters) {
  return rows <= kBlockRows / 2 && splits > 1 && splits <= kBlockCluster && groups <= clusters.count[splits];
}

cudaError_t launch_block_union(const BlockAttnParams& p, cudaStream_t stream) {
  block_union_kernel<<<p.batch * p.groups, kUnThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_block_attn(const BlockAttnParams& p, cudaStream_t stream) {
  BaLaunch l(p.batch * p.groups, p.splits, p.clustered);
  l.cfg.stream = stream;
  return cudaLaunchKernelEx(&l.cfg, p.clustered ? block_attn_kernel<true> : block_attn_kernel<false>, p);
}

}  // namespace ddt
