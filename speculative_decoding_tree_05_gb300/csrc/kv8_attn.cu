// kv8_attn.cu -- verify attention over the 8-bit latent cache.
//
// A key is 512 latent values k in e4m3 and 64 rope values r in bf16, both to be
// multiplied by the slot's scale s. The scale leaves both products:
//   score(i, j) = s_j (q_i . (k_j, r_j)),   o_i = sum over j of (p_ij s_j) k_j / sum of p_ij
// so the tensor core reads the cache's bytes as they are and nothing is dequantised.
// Per row i a running reference r_i follows the largest t_ij = log2(p_ij s_j); the
// weights that enter the second product are 2^(t_ij - r_i), and the sum of p takes
// them divided by s_j, both in fp32 until they are cut into parts.
//
// Operands of 8 bits (fp32 accumulation):
//   q   = (hi + lo) 2^e, e4m3 both, e of the row: bf16's 8 bits, for values down to
//         2^-11 of the row's largest; below that in steps of 2^-18 of it
//   p s = three e5m2 parts of 3 bits each, which hold f16's 11 bits of a weight (2^-12 of it
//         off) down to 2^-13 of the row's largest and lose at most 2^-24 of that below
//
// With all operands in shared memory its 128 B/clk bounded a tile, as an MMA reads both there.
// So the queries are the one operand that stays in tensor memory, both parts of up to 64
// rows as the 128 lanes of one MMA, which sums them apart; and value dims are the M side
// of the second product, so that each 8-bit value is read once for 64 rows and part:
//   S[hi, lo rows][64 keys]      = Q . K^T    16 MMAs M128 x N64 x K32 (8 bit, Q in tensor memory)
//                                             and 4 M64 x N64 x K16 (rope, added to the first parts')
//   O^T[512 dims][rows] += V^T . P^T          3 x 4 x 2 MMAs M128 x N x K32 (V^T: the same bytes read MN-major)
// 48 + 144 KB of operands a tile, and 52 KB written (with both operands of the scores in
// shared memory it was 96 KB more). O^T takes 256 TMEM columns,
// the scores twice 64, the queries 128; one CTA holds the whole output.
// A tile of 64 rows takes 2130 cycles (65 nodes of 128 heads, 65536 keys: 1070 us, 1.11
// PFLOP/s), of which shared memory works 1900, the schedulers issue in 1500 and the tensor core
// works 1410; the gathers run at 18 B/clk and SM, and the softmax's chain of waits is 2000 long,
// of which two overlap. (With two parts of weights, e4m3 and e5m2, it took 2030.) With one query
// row a key it is the gathers alone (16 requests of up to 32768 keys: 54 us, 4 TB/s in the kernel).
//
// Per CTA (896 threads), one unit = (up to 64 (node, head) rows of a request, a share of its tiles):
//   warp 0       TMEM; one lane issues S(t) when stage t has landed
//   warps 1-16   softmax: two sets of eight, for even and odd tiles; 16 rows x 32 keys a warp, in the
//                16x256b shape, the two parts' scores added
//   warp 17      one lane issues P.V(t) when P(t) is written
//   warps 18-25  gather 64 keys per stage of 40 KB, four stages: warps 18-21 three of the five
//                128-byte pieces of a row by 16-byte cp.async, warps 22-25 the others by TMA
//                gather4, at the same time (an SM gathers more both ways than either way)
//   warps 26-27  the keys' scales and row masks
// A request's keys are its prefix and, behind it, all its tree rows, each with the rows
// that see it. The tiles of the whole batch are cut into equal shares, whatever the
// lengths; a request has its share of them, in equal units. One unit writes bf16 and the
// log-sum-exp at once, else each writes its normalised O and the merge kernel joins them.
// A unit of more than kKv8Segment tiles closes a segment there: O^T, its sums and references join those of the segments
// before, in fp32 in the unit's rows of the partials and in shared memory, and start anew.
// The query rows come cut and laid out from the kernel before (kv8_prepare.cu), or (kCut) a unit
// cuts its own.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <type_traits>
#include "kv8_cut.cuh"

namespace ddt {
namespace {

constexpr int kThreads = 896;
constexpr int kSet = 256, kSoftmax = 2 * kSet;       // threads of one softmax set, of both
constexpr int kIssuePv = 17, kFirstCopier = 18, kFirstGather = 22, kFirstKey = 26;  // warps
constexpr int kCopiers = 128;                       // threads that gather the copied groups
constexpr int kKeys = kKv8Keys;
constexpr int kRows = kKv8Rows;
constexpr int kStages = 4;
constexpr int kChunk = kKv8Chunk;                   // 128 bytes of 64 keys: 8 KB
constexpr int kStageBytes = 5 * kChunk;             // 40960
constexpr int kOffCut = 2 * kStageBytes;            // while a unit cuts its query rows: [128 lanes][512 + 16 bytes]
constexpr int kCutRow = 512 + 16;
static_assert(kOffCut + 128 * kCutRow <= kStages * kStageBytes, "the last two stages");
constexpr int kOffRope = kStages * kStageBytes;     // the queries' rope values, [64 rows][128 bytes]
constexpr int kOffQs = kOffRope + kRows * 128;      // [64] the rows' factors of a score
constexpr int kOffP = kOffQs + 1024;                // [2 buffers][3 parts][64 rows][64 keys]
constexpr int kPart = kKeys * kRows, kParts = 3;    // 4096
constexpr int kOffMask = kOffP + 2 * kParts * kPart;      // [stages][64] row masks of the stage's keys
constexpr int kOffKey = kOffMask + kStages * kKeys * 8;   // [stages][3][64] s, log2 s, 1 / s
constexpr int kOffMax = kOffKey + kStages * kKeys * 12;   // [64] running reference
constexpr int kOffAlpha = kOffMax + kRows * 4;      // [64] rescale factors, later 1 / row sums
constexpr int kOffTree = kOffAlpha + kRows * 4;        // [128] row masks of the tree rows
constexpr int kOffSlot = kOffTree + kMaxNodes * 8;  // [128] their slots
constexpr int kOffPar = kOffSlot + kMaxNodes * 4;   // [128] their parents
constexpr int kOffSeg = kOffPar + kMaxNodes * 4;    // of the segments before: [64] references, [64] factors,
constexpr int kOffSegSum = kOffSeg + 2 * kRows * 4; // [512 softmax threads] sums and references of two rows
constexpr int kOffBar = kOffSegSum + kSoftmax * 16;
static_assert(kOffSegSum % 16 == 0 && kKv8Segment % 2 == 0 && (kKv8Segment & (kKv8Segment - 1)) == 0, "read as float4; closed at an even tile");
constexpr int kSmem = kOffBar + 512 + 1024;
static_assert(kSmem <= 232448, "one CTA's shared memory");
constexpr uint32_t kColS = 256, kColQ = 384;        // O^T [0, 256), S buffers 2 x 64, Q
constexpr float kUnset = -1e30f;                    // running reference of a row that has seen no key
// Weights are 2^(t - r + kLift) and r is raised when one would exceed 2^(kLift + kSlack) = 55109
// (e5m2 ends at 57344). A raise takes 3000 cycles, as O^T is rescaled, and r follows the largest
// t, so a row's largest weight is at least 2^kLift. What falls below the parts' last step is at
// most 2^-17 of a weight, 2^-(17 + kLift) of the largest; but behind one dominant key a tail's
// errors may all have one sign, so they count times the keys of a segment, after which references
// start anew: 2^-9 of the largest. 9 nodes of 16 heads, 185000
// keys: 87 us, with a lift of 6 86, of 8 88; with the weights as e4m3 and e5m2, which end at 448
// and left the keys out that were 2^-19 of the largest, 83.
constexpr float kLift = 7.f, kSlack = 8.75f;
// Scales that are used. The sum of p takes weights divided by s, and a weight of less than 2^-126 is zero: with these, less
// than 2^-33 of a row's sum (2^-126 / 2^-60 beside 2^kLift / 2^40).
constexpr float kLeastScale = 0x1p-60f, kMostScale = 0x1p40f;
constexpr float kLn2 = 0.69314718055994531f;

struct Shared {
  uint64_t k_full[kStages][2], k_empty[kStages][2];  // [0]: chunks 0, 1 and 4, copied; [1]: 2 and 3, gathered
  uint64_t f_full[kStages];            // the keys' factors and masks
  uint64_t s_full[2], s_free[2];
  uint64_t p_ready[2];
  uint64_t decided[2];                 // the references of this set's tile stand
  uint64_t q_full;                     // the queries' rope values and factors
  uint64_t q_ready;                    // the queries in tensor memory
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int fail[2];     // softmax: a wait of a thread of the set ran out
  int raises;      // how often the references have been raised
  int flags;
  // where the unit's results go: bf16 rows of out, or fp32 rows of its partials (in shared memory: registers are
  // what the loops lack)
  void* o_dst;
  float* lse_dst;
  float* o_seg;  // fp32 rows of the segments before
  int last;  // the request's one unit
  int shares;
  uint16_t seen[kStages][2];  // whether every row of the group sees all of a key warp's keys
};
static_assert(sizeof(Shared) <= 512, "barrier block");

// 16 TMEM lanes x 16 columns over a warp, from taddr and 16 lanes on, added:
// v[2 i + h] = lane L/4 + 8 h, columns 8 i + 2 (L % 4) + {0, 1}.
__device__ __forceinline__ void tmem_ld_sum(uint32_t taddr, uint64_t (&v)[4]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = add_x2(f32x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                  f32x2(__uint_as_float(r[8 + 2 * i]), __uint_as_float(r[9 + 2 * i])));
}
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
// Two weights in three e5m2 parts, each the nearest to what those before it leave. A pair goes through f16, whose 11 bits
// lose 2^-12 of a weight; an e5m2 value is f16's upper byte, so the differences are exact, and with 3 bits a part nothing of
// f16's 11 is left after the third (but for what is below e5m2's least step, 2^-16).
__device__ __forceinline__ void cut_weights(float x, float y, uint32_t (&part)[kParts]) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    uint16_t a;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(a) : "r"(h));
    part[k] = a;
    if (k + 1 < kParts) asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(__byte_perm(part[k], 0, 0x1404)));
  }
}
// A shuffle that stays where it stands among the copies.
__device__ __forceinline__ int shfl_here(int v, int from) {
  int r;
  asm volatile("shfl.sync.idx.b32 %0, %1, %2, 0x1f, 0xffffffff;" : "=r"(r) : "r"(v), "r"(from) : "memory");
  return r;
}
__device__ __forceinline__ void st_shared_b16(uint32_t at, uint32_t v) {
  asm volatile("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tst.shared.b16 [%0], l;\n\t}" ::"r"(at), "r"(v) : "memory");
}
// a |= m in shared memory, by halves (32-bit atomics need no loop)
__device__ __forceinline__ void or_mask(uint64_t* a, uint64_t m) {
  unsigned* half = reinterpret_cast<unsigned*>(a);
  const unsigned lo = static_cast<unsigned>(m), hi = static_cast<unsigned>(m >> 32);
  if (lo) atomicOr(half, lo);
  if (hi) atomicOr(half + 1, hi);
}

__device__ __forceinline__ int tiles_of(const Kv8AttnParams& p, int b) {
  const int nodes = kv8_nodes(p.tree_len, b, p.nodes);
  return nodes == 0 ? 0 : (kv8_len(p.prefix_len, b, p.max_prefix_len) + nodes + kKeys - 1) / kKeys;
}

// Shares for requests whose trees' lengths the host does not know, at most p.shares (for which the grid and the partials
// are laid out): those that cost least among 32, one a lane, that would just fill one to eight waves. By one whole warp of
// every CTA, so it estimates in fp32. In tiles of 64 keys: a unit costs kUnitTiles more than its tiles, a partial
// kPartialTiles, and the time lies between whole waves of the longest unit and all units' even division among the SMs.
// (8 requests of 4096 to 131072 keys, trees of 1 to 33 nodes of 16 heads: p.shares made 400 units, 2.6 waves, 507 us,
// these 463 then. Other ragged batches: 220 to 167, 129 to 119, 178 to 178, one 152 to 170.)
constexpr int kMaxPlanned = 32;  // requests
constexpr float kUnitTiles = 10.f, kPartialTiles = 0.06f;
__device__ __forceinline__ int plan_shares(const Kv8AttnParams& p, int lane) {
  const bool mine = lane < p.batch;
  const float n = mine ? tiles_of(p, lane) : 0;
  const float g = mine ? kv8_groups(p.heads, p.group_nodes, kv8_nodes(p.tree_len, lane, p.nodes)) : 0;
  float sum = n, groups = g, work = n * g, most = n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    groups += __shfl_xor_sync(0xffffffffu, groups, o);
    work += __shfl_xor_sync(0xffffffffu, work, o);
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  const float sms = p.sms;
  // a request adds between none and one unit to its part of the shares
  const float ctas = (1 + (lane >> 2)) * sms - (lane & 3) * (1.f / 3) * groups;
  int shares = static_cast<int>(fminf(fmaxf(ctas * sum / fmaxf(work, 1.f), 1.f), static_cast<float>(p.shares)));
  if (lane >= 30) shares = lane == 30 ? p.shares : 1;
  const float share = fmaxf(sum / shares, 1.f), per_tile = 1.f / share;
  float units = 0, partials = 0;
#pragma unroll 4
  for (int b = 0; b < p.batch; ++b) {
    const float c = ceilf(__shfl_sync(0xffffffffu, n, b) * per_tile), u = c * __shfl_sync(0xffffffffu, g, b);
    units += u;
    if (c > 1.f) partials += u;
  }
  const float longest = fminf(share, most) + kUnitTiles;
  float cost = 0.5f * ceilf(units / sms) * longest + 0.5f * fmaxf((work + kUnitTiles * units) / sms, longest) + kPartialTiles * partials;
  int best = lane;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, cost, o);
    const int at = __shfl_xor_sync(0xffffffffu, best, o);
    if (other < cost || (other == cost && at < best)) cost = other, best = at;
  }
  return __shfl_sync(0xffffffffu, shares, best);
}

// Unit u of the batch: which request, which of its units. The requests' tiles make K in
// all, a share is C = ceil(K / shares) of them, and a request of n tiles has ceil(n / C)
// units of equal size. Called by whole warps; b < 0: there is no such unit.
struct Unit {
  int b, k, count, first;
};
__device__ __forceinline__ Unit find_unit(const Kv8AttnParams& p, int shares, int u, int lane) {
  Unit r;
  if (shares == 0) {
    r.b = kv8_nodes(p.tree_len, u, p.nodes) > 0 ? u : -1;
    r.k = 0;
    r.count = 1;
    r.first = u;
    return r;
  }
  long long sum = 0;
  for (int i = lane; i < p.batch; i += 32) sum += tiles_of(p, i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int share = static_cast<int>(min((sum + shares - 1) / shares, 1ll << 30));
  int base = 0;
  r.b = -1;
  for (int i0 = 0; i0 < p.batch; i0 += 32) {
    const int n = i0 + lane < p.batch ? tiles_of(p, i0 + lane) : 0;
    const int c = n == 0 ? 0 : (n + share - 1) / share;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int lo = base + incl - c;
    const uint32_t vote = __ballot_sync(0xffffffffu, u >= lo && u < lo + c);
    if (vote != 0) {
      const int src = __ffs(vote) - 1;
      r.b = i0 + src;
      r.first = __shfl_sync(0xffffffffu, lo, src);
      r.count = __shfl_sync(0xffffffffu, c, src);
      r.k = u - r.first;
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// kCut: the query rows are cut here, beside the first tiles' gathers, not by the kernel before.
// kLong: a unit may have more than one segment. (Without that code 1100 requests of 10 to 200 keys take 185 us, with it 190.)
template <bool kCut, bool kLong>
__global__ void __launch_bounds__(kThreads, 1) kv8_attn_kernel(const __grid_constant__ Kv8AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem + kOffBar);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sh.abort;
  const int g = blockIdx.x, unit = blockIdx.y;
  grid_dep_launch();  // the merge kernel
  int shares = p.shares;
  if (shares > 1 && p.tree_len && p.batch <= kMaxPlanned) {
    if (warp == 0) {
      const int s = plan_shares(p, lane);
      if (lane == 0) sh.shares = s;
    }
    __syncthreads();
    shares = sh.shares;
  }
  const Unit un = find_unit(p, shares, unit, lane);
  const int nodes = un.b < 0 ? 0 : kv8_nodes(p.tree_len, un.b, p.nodes);  // active ones
  const Kv8Group gr = kv8_group(p.heads, p.group_nodes, nodes, g);
  const int row0 = gr.row0, rows = gr.rows;
  if (un.b >= 0 && un.k == 0 && g == 0 && tid == 0) {
    Kv8Piece piece;
    piece.first = un.first;
    piece.count = un.count;
    p.pieces[un.b] = piece;
  }
  if (un.b < 0 || rows <= 0) {
    grid_dep_wait();  // (this grid is not done before the one that it follows)
    return;
  }
  const int L = kv8_len(p.prefix_len, un.b, p.max_prefix_len);
  const int keys = L + nodes;
  const int tiles = (keys + kKeys - 1) / kKeys;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * un.k / un.count);
  const int n = static_cast<int>(static_cast<int64_t>(tiles) * (un.k + 1) / un.count) - t0;  // at least one

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.k_full[i][0], kCopiers);  // every copying thread's cp.async
      mbar_init(&sh.k_full[i][1], 4);         // four gather warps, with their bytes
      mbar_init(&sh.k_empty[i][0], 1);        // P.V of the tile is done (and those before it)
      mbar_init(&sh.k_empty[i][1], 1);        // its first half is, of the gathered chunks
      mbar_init(&sh.f_full[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], kSet / 32);
      mbar_init(&sh.p_ready[i], kSet / 32);
      mbar_init(&sh.decided[i], 1);
    }
    mbar_init(&sh.drain, 2);
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_ready, kSoftmax / 32);
    sh.abort = 0;
    sh.fail[0] = sh.fail[1] = sh.raises = 0;
    sh.flags = 0;
    const int64_t all = static_cast<int64_t>(p.nodes) * p.heads, at = (un.count == 1 ? un.b : unit) * all + row0;
    sh.last = un.count == 1;
    sh.o_dst = un.count == 1 ? static_cast<void*>(p.out + at * kDv) : p.o_part + at * kDv;
    sh.lse_dst = (un.count == 1 ? p.lse : p.lse_part) + at;
    sh.o_seg = p.o_part + (unit * all + row0) * kDv;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  float* mx = reinterpret_cast<float*>(smem + kOffMax);
  if (tid < kRows) mx[tid] = kUnset;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  bool ok = true;

  if (warp == 0) {
    if (elect_one()) {
      if (!kCut) {
        grid_dep_wait();  // the query rows: what comes before overlaps their making
        mbar_arrive_expect_tx(&sh.q_full, kKv8Image - kKv8ImageRope);
        bulk_load(base + kOffRope, p.images + (static_cast<int64_t>(un.b) * p.groups + g) * kKv8Image + kKv8ImageRope,
                  kKv8Image - kKv8ImageRope, &sh.q_full);
        ok = mbar_wait_abortable(&sh.q_full, 0, abort, false, __LINE__);
      }
      ok = ok && mbar_wait_abortable(&sh.q_ready, 0, abort, false, __LINE__);
      tc_fence_after();
      const uint32_t idesc8 = idesc_f8_f32(128, kKeys, kE4m3, kE4m3, false, false), idesc = idesc_bf16_f32(64, kKeys, false, false);  // (M64: the first parts' lanes)
      const uint64_t d_k = smem_desc(base, 16, 1024, kSwizzle128B);
      const uint64_t d_rope = smem_desc(base + kOffRope, 16, 1024, kSwizzle128B);
      int st = 0, ph = 0;
      for (int t = 0; ok && t < n; ++t) {
        if (t >= 2 && !mbar_wait_abortable(&sh.s_free[t & 1], ((t >> 1) - 1) & 1, abort, false, __LINE__)) {
          ok = false;
          break;
        }
        const uint64_t k = desc_advance(d_k, st * kStageBytes);
        const uint32_t d = tmem + kColS + (t & 1) * kKeys;
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // the copied chunks land first
          if (!mbar_wait_abortable(&sh.k_full[st][x], ph, abort, false, __LINE__)) {
            ok = false;
            break;
          }
          if (x == 0) fence_proxy_async_smem();  // written by cp.async
          tc_fence_after();
#pragma unroll
          for (int ks = 8 * x; ks < 8 * x + 8; ++ks)
            mma_f8_ts(d, tmem + kColQ + ks * 8, desc_advance(k, (ks >> 2) * kChunk + (ks & 3) * 32), idesc8, ks > 0 ? 1u : 0u);
        }
        if (!ok) break;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // the rope dims
          mma_ss(d, desc_advance(d_rope, ks * 32), desc_advance(k, 4 * kChunk + ks * 32), idesc, 1u);
        mma_commit(&sh.s_full[t & 1]);
        if (++st == kStages) st = 0, ph ^= 1;
      }
      mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
  } else if (warp == kIssuePv) {
    if (elect_one()) {
      const uint32_t cols = (rows + 15) / 16 * 16;
      const uint32_t idesc = idesc_f8_f32(128, cols, kE4m3, kE5m2, true, false);
      const uint64_t d_v = smem_desc(base, kChunk, 1024, kSwizzle128B);          // MN-major, 128 dims a chunk
      const uint64_t d_p = smem_desc(base + kOffP, 16, 512, kSwizzle64B);        // K-major, 64 keys a row
      int st = 0;
      for (int t = 0; t < n; ++t) {
        if (!mbar_wait_abortable(&sh.p_ready[t & 1], (t >> 1) & 1, abort, false, __LINE__)) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t v = desc_advance(d_v, st * kStageBytes), w = desc_advance(d_p, (t & 1) * kParts * kPart);
        const uint32_t more = (kLong ? t & (kKv8Segment - 1) : t) > 0 ? 1u : 0u;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int mt = (y + 2) & 3;  // the gathered chunks first: they take longest to come
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const uint64_t a = desc_advance(v, mt * kChunk + ks * 4096);
#pragma unroll
            for (int part = 0; part < kParts; ++part)
              mma_f8_ss(tmem + mt * kRows, a, desc_advance(w, part * kPart + ks * 32), idesc, ks + part > 0 ? 1u : more);
          }
          if (y & 1) mma_commit(&sh.k_empty[st][y == 1]);
        }
        if (++st == kStages) st = 0;
      }
      mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
  } else if (warp >= kFirstCopier) {
    // ------------------------------------------------------------------ producers
    const int32_t* slots = p.slot_idx + static_cast<int64_t>(un.b) * p.slot_stride;
    uint64_t* tree_mask = reinterpret_cast<uint64_t*>(smem + kOffTree);
    int* tree_slot = reinterpret_cast<int*>(smem + kOffSlot);
    const uint64_t full = rows == 64 ? ~0ull : ((1ull << rows) - 1);
    if ((t0 + n) * kKeys > L) {
      // the tree rows, and which of the group's rows see each: a node's walk to the root sets its rows' bits in
      // itself and every ancestor; a link that is no earlier node ends it, a slot outside the pool is left out
      int* par = reinterpret_cast<int*>(smem + kOffPar);
      const int i = tid - kFirstCopier * 32;
      if (i < nodes) {
        par[i] = __ldg(p.tree_parent + static_cast<int64_t>(un.b) * p.nodes + i);
        tree_slot[i] = __ldg(p.tree_slot_idx + static_cast<int64_t>(un.b) * p.nodes + i);
        tree_mask[i] = 0;
      }
      bar_sync(4, kThreads - kFirstCopier * 32);
      const int first = row0 / p.heads, last = (row0 + rows - 1) / p.heads;
      if (i <= last - first) {
        const int lo = max(0, (first + i) * p.heads - row0), hi = min(rows, (first + i + 1) * p.heads - row0);
        const uint64_t mine = (hi == 64 ? ~0ull : ((1ull << hi) - 1)) & ~((1ull << lo) - 1);
        int v = first + i, flags = 0;
        for (int guard = 0; v >= 0 && guard < nodes; ++guard) {
          const int slot = tree_slot[v], up = par[v];
          if (slot >= 0 && slot < p.pool_slots)
            or_mask(&tree_mask[v], mine);
          else
            flags |= kStatusBadSlot;
          if (v == 0 ? up != -1 : (up < 0 || up >= v)) {
            flags |= kStatusBadParent;
            break;
          }
          v = up;
        }
        if (flags) atomicOr(&sh.flags, flags);
      }
      bar_sync(4, kThreads - kFirstCopier * 32);
    }
    // Key i of the request: its slot as read. Nothing is computed from a value in the tile that reads it: an
    // immediate use stalls the warp for the read (800 cycles a tile).
    auto read_slot = [&](int t, int k) -> int {
      const int i = (t0 + t) * kKeys + k;
      if (t >= n || k >= kKeys || i >= keys) return -1;
      return i < L ? __ldg(slots + i) : tree_slot[i - L];
    };
    auto in_pool = [&](int slot) { return slot >= 0 && slot < p.pool_slots; };
    // 16-byte copies of kPieces consecutive pieces (8 a chunk) from chunk c0 on of 16 rows from row0 on; zeros for
    // rows without a slot
    auto copy_rows = [&](uint32_t sbase, int r0, int c0, auto pieces, int slot) {
      constexpr int kPieces = decltype(pieces)::value, kStep = 32 / kPieces;
      const int y = lane & (kPieces - 1), sub = lane / kPieces;
      const uint32_t dst = sbase + (c0 + (y >> 3)) * kChunk + (r0 + sub) * 128;
      const uint8_t* src = p.kv + c0 * 128 + y * 16;
      // Two shuffles before each two copies, kept in this order: the softmax warps' accesses then queue behind two copies,
      // not behind all of a tile's (attend over 65536 keys by 65 nodes of 128 heads 1036 -> 1023 us).
#pragma unroll
      for (int i = 0; i < 16 / kStep; i += 2) {
        int row[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) row[j] = shfl_here(slot, (i + j) * kStep + sub);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = ((y & 7) ^ (((i + j) * kStep + sub) & 7)) << 4;
          cp_async16(dst + (i + j) * kStep * 128 + at, row[j] < 0 ? p.kv : src + static_cast<int64_t>(row[j]) * kKv8Row,
                     row[j] < 0 ? 0u : 16u);
        }
      }
    };
    using P16 = std::integral_constant<int, 16>;
    using P8 = std::integral_constant<int, 8>;
    const bool copier = warp < kFirstGather, gather = !copier && warp < kFirstKey;
    // the warp's first key of a tile, 16 of them (a key warp: 32); the lane's key
    const int r0 = copier ? 16 * (warp - kFirstCopier) : gather ? 16 * (warp - kFirstGather) : 32 * (warp - kFirstKey);
    const int k = lane < 16 || warp >= kFirstKey ? r0 + lane : kKeys;
    int slot_now = read_slot(0, k), slot_next = read_slot(1, k);
    float scale_now = 1.f;
    if (warp >= kFirstKey && in_pool(slot_now)) scale_now = __ldg(p.scale + slot_now);
    int st = 0, ph = 0, done = 0;
    for (int t = 0; t < n; ++t) {
      const int i = (t0 + t) * kKeys + k;
      uint64_t mask = 0;  // of the rows that see the key
      if (k < kKeys && i < keys) mask = i < L ? full : tree_mask[i - L];
      const bool bad = mask != 0 && !in_pool(slot_now);
      if (bad) mask = 0;
      const int slot = mask != 0 ? slot_now : -1;
      const float scale = scale_now;
      // A key takes two dependent reads, its slot and its scale, each a tile ahead of its use.
      slot_now = slot_next;
      if (warp >= kFirstKey && in_pool(slot_now)) scale_now = __ldg(p.scale + slot_now);
      slot_next = read_slot(t + 2, k);
      const uint32_t sbase = base + st * kStageBytes;
      const bool empty = t < kStages ? !kCut || t < 2 || mbar_wait_abortable(&sh.q_ready, 0, abort, false, __LINE__)
                                     : mbar_wait_abortable(&sh.k_empty[st][gather], ph ^ 1, abort, false, __LINE__);
      if (!__all_sync(0xffffffffu, empty)) {
        ok = false;
        break;
      }
      if (copier) {
        copy_rows(sbase, r0, 0, P16(), slot);
        copy_rows(sbase, r0, 4, P8(), slot);
        cp_async_arrive_noinc(&sh.k_full[st][0]);
      } else if (gather) {
        if (__all_sync(0xffffffffu, slot >= 0 || lane >= 16)) {
          // lanes 0-7: four of the warp's keys, one of the two chunks
          if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[st][1], 16 * 256);
          __syncwarp();
          const int q = 4 * (lane & 3), c = 2 + (lane >> 2);
          const int ra = __shfl_sync(0xffffffffu, slot, q), rb = __shfl_sync(0xffffffffu, slot, q + 1);
          const int rc = __shfl_sync(0xffffffffu, slot, q + 2), rd = __shfl_sync(0xffffffffu, slot, q + 3);
          if (lane < 8) tma_gather4(sbase + c * kChunk + (r0 + q) * 128, &p.tmap, c * 128, ra, rb, rc, rd, &sh.k_full[st][1]);
        } else {
          // a key is masked (the end of the keys, a bad slot): zero-filled copies
          copy_rows(sbase, r0, 2, P16(), slot);
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[st][1]);
        }
      } else {
        if (bad) atomicOr(&sh.flags, kStatusBadSlot);
        reinterpret_cast<uint64_t*>(smem + kOffMask)[st * kKeys + k] = mask;
        const bool all = __all_sync(0xffffffffu, mask == full);
        if (lane == 0) sh.seen[st][warp - kFirstKey] = all;
        // a scale that is not usable: NaN for the rows that see the key
        const bool fine = scale >= kLeastScale && scale <= kMostScale;
        float* f = reinterpret_cast<float*>(smem + kOffKey) + st * 3 * kKeys + k;
        f[0] = fine ? scale : CUDART_NAN_F;
        f[kKeys] = fine ? log2f(scale) : 0.f;
        f[2 * kKeys] = fine ? 1.f / scale : 1.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.f_full[st]);
      }
      done = t + 1;
      if (++st == kStages) st = 0, ph ^= 1;
    }
    cp_async_wait<0>();
    if (!ok && gather)  // after a give-up the gathers still in flight land before the CTA exits
      for (int v = max(0, done - kStages); v < done; ++v) mbar_wait(&sh.k_full[v % kStages][1], (v / kStages) & 1, 1u << 14);
  } else {
    // ------------------------------------------------------------------ softmax
    // Two sets, for even and odd tiles: a tile's way from its scores to its weights is a chain of waits (3000
    // cycles, most of them for shared memory beside the gathers), of which two overlap.
    const int set = (warp - 1) >> 3, quarter = warp & 3, half = ((warp - 1) >> 2) & 1;  // 16 rows, 32 keys of a tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int r0 = quarter * 16 + (lane >> 2);     // rows r0 and r0 + 8
    const int c0 = 32 * half + 2 * (lane & 3);     // keys c0 + 8 i + {0, 1}, i < 4
    const int id = half * 128 + quarter * 32 + lane;
    const int bar = 1 + 4 * set;                   // the set's barrier
    float* alpha_sh = reinterpret_cast<float*>(smem + kOffAlpha);
    const int part4 = (warp - 1) >> 2;  // the queries, a quarter of the lanes' bytes a warp
    if (kCut) {
      const uint16_t* q = p.q + (static_cast<int64_t>(un.b) * p.nodes * p.heads + row0) * kDqk;
      uint32_t w[4][9];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = warp - 1 + 16 * j;
        load_query(r < rows ? q + static_cast<int64_t>(r) * kDqk : nullptr, lane, w[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = warp - 1 + 16 * j;
        CutQuery c = {};
        if (r < rows) c = cut_row(w[j], lane, p.scale_log2);
#pragma unroll
        for (int part = 0; part < 2; ++part)
          *reinterpret_cast<uint4*>(smem + kOffCut + query_lane(r, part) * kCutRow + query_piece(lane) * 16) = c.part[part];
        *reinterpret_cast<uint32_t*>(smem + kOffRope + query_rope_at(r, lane)) = c.rope;
        if (lane == 0) reinterpret_cast<float*>(smem + kOffQs)[r] = c.factor;
      }
      bar_sync(6, kSoftmax);
      uint32_t r[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 v = *reinterpret_cast<const uint4*>(smem + kOffCut + (quarter * 32 + lane) * kCutRow + (8 * part4 + j) * 16);
        r[4 * j] = v.x, r[4 * j + 1] = v.y, r[4 * j + 2] = v.z, r[4 * j + 3] = v.w;
      }
      tmem_st32(tmem + lane_off + kColQ + 32 * part4, r);
      fence_proxy_async_smem();  // the rope values are read, and the last two stages written, by other means
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_ready);
    } else {
      grid_dep_wait();
      const uint4* src = reinterpret_cast<const uint4*>(p.images + (static_cast<int64_t>(un.b) * p.groups + g) * kKv8Image) +
                         8 * part4 * 128 + quarter * 32 + lane;
      uint32_t r[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 v = __ldcg(src + j * 128);
        r[4 * j] = v.x, r[4 * j + 1] = v.y, r[4 * j + 2] = v.z, r[4 * j + 3] = v.w;
      }
      tmem_st32(tmem + lane_off + kColQ + 32 * part4, r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_ready);
    }
    // a wait of this thread ran out: the warps leave together at the next barrier
    bool failed = !kCut && !mbar_wait_abortable(&sh.q_full, 0, abort, false, __LINE__);
    // of this thread's rows: sums (of even and odd keys), score factors and (lowered by kLift) references
    uint64_t l[2];
    float qs[2], m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = f32x2(0.f, 0.f);
      qs[h] = reinterpret_cast<const float*>(smem + kOffQs)[r0 + 8 * h];
      m[h] = kUnset;
    }
    // Where this thread's weights go in a part of P^T (a row's 64 keys, 64-byte swizzle): two keys of row r0, of row
    // r0 + 8 512 bytes on. (i = 1 is eight bytes on, 2 and 3 the next 16-byte piece.)
    const uint32_t p_at = base + kOffP + set * kParts * kPart + r0 * 64 + ((((c0 >> 4) ^ ((r0 >> 1) & 3)) << 4) | (c0 & 15));
    auto wait_pv = [&](int t) {  // P.V(t) has read P, and O^T holds every tile up to t
      if (!mbar_wait_abortable(&sh.k_empty[t % kStages][0], (t / kStages) & 1, abort, false, __LINE__)) failed = true;
      tc_fence_after();
    };
    // sums or maxima over the warp's 32 keys, to scratch [2 halves of the keys][64 rows]
    float* scratch = reinterpret_cast<float*>(smem + kOffP + set * kParts * kPart);
    auto to_scratch = [&](const float (&v)[2], auto op) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = op(v[h], __shfl_xor_sync(0xffffffffu, v[h], 1));
        x = op(x, __shfl_xor_sync(0xffffffffu, x, 2));
        if ((lane & 3) == 0) scratch[half * kRows + r0 + 8 * h] = x;
      }
    };
    // What the segments before have come to, of this thread's rows: sums, times 2^reference. (Thread's own.)
    float4* seg_sum = reinterpret_cast<float4*>(smem + kOffSegSum) + set * kSet + id;
    float *seg_ref = reinterpret_cast<float*>(smem + kOffSeg), *seg_factor = seg_ref + kRows;
    auto close_sums = [&](bool first) {
      const float4 v = first ? make_float4(0.f, 0.f, kUnset, kUnset) : *seg_sum;
      const float all[2] = {v.x, v.y}, ref[2] = {v.z, v.w};
      float sum[2], top[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x, y;
        f32x2_split(l[h], x, y);
        top[h] = fmaxf(ref[h], m[h]);
        sum[h] = fmaf(all[h], fast_exp2(ref[h] - top[h]), (x + y) * fast_exp2(m[h] - top[h]));
        l[h] = f32x2(0.f, 0.f);
      }
      *seg_sum = make_float4(sum[0], sum[1], top[0], top[1]);
    };
    int raises = 0;  // that m and l know of
    for (int t = set; t < n; t += 2) {
      const int st = t % kStages, ph = (t / kStages) & 1;
      const bool p_free = t < 2 || mbar_test_wait(&sh.k_empty[(t - 2) % kStages][0], ((t - 2) / kStages) & 1);
      if (!mbar_wait_abortable(&sh.f_full[st], ph, abort, false, __LINE__)) failed = true;
      const bool part = *reinterpret_cast<const volatile uint32_t*>(sh.seen[st]) != 0x00010001u;
      const float* factor = reinterpret_cast<const float*>(smem + kOffKey) + st * 3 * kKeys + c0;
      if (!mbar_wait_abortable(&sh.s_full[set], (t >> 1) & 1, abort, false, __LINE__)) failed = true;
      __syncwarp();
      tc_fence_after();
      float s[16];  // [4 i + 2 h + e]: row r0 + 8 h, key c0 + 8 i + e: log2 of its weight times its key's scale
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint64_t v[4];
        tmem_ld_sum(tmem + lane_off + kColS + set * kKeys + 32 * half + 16 * j, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t ks = *reinterpret_cast<const uint64_t*>(factor + 16 * j + 8 * i);
          const uint64_t lg = *reinterpret_cast<const uint64_t*>(factor + kKeys + 16 * j + 8 * i);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            f32x2_split(fma_x2(mul_x2(v[2 * i + h], ks), f32x2(qs[h], qs[h]), lg), s[8 * j + 4 * i + 2 * h],
                        s[8 * j + 4 * i + 2 * h + 1]);
        }
      }
      tc_fence_before();
      __syncwarp();
#ifdef DDT_TEST_HOOKS
      if (warp != 1 + 8 * set || t != p.test_keep_back)
#endif
      if (lane == 0) mbar_arrive(&sh.s_free[set]);
      if (part) {
        const uint64_t* masks = reinterpret_cast<const uint64_t*>(smem + kOffMask) + st * kKeys + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t seen = static_cast<uint32_t>(masks[8 * i + e] >> r0);
            if (!(seen & 1u)) s[4 * i + e] = -CUDART_INF_F;
            if (!(seen & 0x100u)) s[4 * i + 2 + e] = -CUDART_INF_F;
          }
      }
      float top[2];  // of the thread's rows
#pragma unroll
      for (int h = 0; h < 2; ++h)
        top[h] = fmax3(fmax3(s[2 * h], s[2 * h + 1], s[4 + 2 * h]), fmax3(s[5 + 2 * h], s[8 + 2 * h], s[9 + 2 * h]),
                       fmaxf(s[12 + 2 * h], s[13 + 2 * h]));
      // The references, as they are after the tile before, of the other set. They are raised for all rows at once:
      // with 64 rows in step, raising the rows that need it alone would come to a raise in most tiles.
      if (t > 0 && !mbar_wait_abortable(&sh.decided[set ^ 1], ((t - 1) >> 1) & 1, abort, false, __LINE__)) failed = true;
      const int raised = *const_cast<volatile int*>(&sh.raises);
      if (raised != raises) {
        raises = raised;
        const bool next = kLong && t > 1 && (t & (kKv8Segment - 1)) == 1;  // a segment's first of the odd tiles
        if (next) close_sums(t == kKv8Segment + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float now = const_cast<volatile float*>(mx)[r0 + 8 * h], a = next ? 0.f : fast_exp2(m[h] - now);
          l[h] = mul_x2(l[h], f32x2(a, a));
          m[h] = now;
        }
      }
      const bool close = kLong && t > 0 && (t & (kKv8Segment - 1)) == 0;  // the segment before is complete (the even tiles' set)
      if (failed) sh.fail[set] = 1;
      const bool raise = bar_red_or(bar, kSet, failed || close || fmaxf(top[0] - m[0], top[1] - m[1]) > kLift + kSlack);
      if (raise) {
        if (*const_cast<volatile int*>(&sh.fail[set])) {
          ok = false;
          break;
        }
        if (t > 0) wait_pv(t - 1);  // O^T is rescaled (and the scratch, the P buffer, is free)
        to_scratch(top, [](float a, float b) { return fmaxf(a, b); });
        bar_sync(bar, kSet);
        if (id < kRows) {  // one thread per row decides
          const float old = mx[id], now = fmaxf(close ? kUnset : old, fmaxf(scratch[id], scratch[kRows + id]) - kLift);
          if (close) {
            const float ref = t == kKv8Segment ? kUnset : seg_ref[id], all = fmaxf(ref, old);
            seg_factor[id] = fast_exp2(ref - all);
            alpha_sh[id] = fast_exp2(old - all);
            seg_ref[id] = all;
          } else {
            alpha_sh[id] = fast_exp2(old - now);
          }
          mx[id] = now;
        }
        if (id == 0) sh.raises = raises + 1;
        ++raises;
        bar_sync(bar, kSet);
        if (close) close_sums(t == kKv8Segment);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = alpha_sh[r0 + 8 * h];
          l[h] = mul_x2(l[h], f32x2(a, a));
          m[h] = mx[r0 + 8 * h];
        }
        if (close) {
          // O^T joins what the segments before have come to; the next product starts it anew
#pragma unroll 1
          for (int k0 = 0; k0 < 16; ++k0) {
            const int mt = k0 >> 2, cc = 32 * half + (k0 & 3) * 8;
            if (cc >= rows) continue;
            uint32_t o[8];
            tmem_ld8(tmem + lane_off + mt * kRows + cc, o);
            float* dst = sh.o_seg + cc * kDv + mt * 128 + quarter * 32 + lane;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (cc + k < rows) {
                const float x = __uint_as_float(o[k]) * alpha_sh[cc + k];
                dst[k * kDv] = t == kKv8Segment ? x : fmaf(dst[k * kDv], seg_factor[cc + k], x);
              }
          }
          tc_fence_before();
        } else if (t > 0) {
#pragma unroll 1
          for (int k0 = 0; k0 < 16; ++k0) {  // half of the columns (rows), 8 at a time
            const int cc = 32 * half + (k0 & 3) * 8;
            uint32_t o[8];
            tmem_ld8(tmem + lane_off + (k0 >> 2) * kRows + cc, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha_sh[cc + k]);
            tmem_st8(tmem + lane_off + (k0 >> 2) * kRows + cc, o);
          }
          tc_fence_before();
        }
        bar_sync(bar, kSet);  // scratch is read before P is written over it, and O^T is rescaled
      }
      if (id == 0) mbar_arrive(&sh.decided[set]);
      if (!p_free && !raise) wait_pv(t - 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t inv = *reinterpret_cast<const uint64_t*>(factor + 2 * kKeys + 8 * i);
        uint32_t cut[2][kParts];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = fast_exp2(s[4 * i + 2 * h] - m[h]), y = fast_exp2(s[4 * i + 2 * h + 1] - m[h]);
          l[h] = fma_x2(f32x2(x, y), inv, l[h]);
          cut_weights(x, y, cut[h]);
        }
        const uint32_t at = (p_at ^ ((i >> 1) * 16)) + 8 * (i & 1);
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          st_shared_b16(at + k * kPart, cut[0][k]);
          st_shared_b16(at + k * kPart + 512, cut[1][k]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_ready[set]);
    }
    if (ok) wait_pv(n - 1);  // O^T is complete and the P buffers free
    if (bar_red_or(6, kSoftmax, failed || !ok)) ok = false;
    if (ok) {
      float sums[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // the last raise may have been the other set's
        const float now = mx[r0 + 8 * h], all = kLong && n > kKv8Segment ? fmaxf(now, seg_ref[r0 + 8 * h]) : now;
        const float a = fast_exp2(m[h] - all);
        float x;
        f32x2_split(l[h], sums[h], x);
        sums[h] = (sums[h] + x) * a;
        if (kLong && n > kKv8Segment + set) sums[h] = fmaf(h ? seg_sum->y : seg_sum->x, fast_exp2((h ? seg_sum->w : seg_sum->z) - all), sums[h]);
      }
      to_scratch(sums, [](float a, float b) { return a + b; });
      bar_sync(6, kSoftmax);
      if (set == 0 && id < kRows) {
        const float* other = scratch + kParts * kPart / 4;
        const float sum = (scratch[id] + scratch[kRows + id]) + (other[id] + other[kRows + id]);
        const float now = mx[id], inv = sum != 0.f ? 1.f / sum : 0.f;
        float all = now;
        if (kLong && n > kKv8Segment) {
          all = fmaxf(now, seg_ref[id]);
          seg_factor[id] = fast_exp2(seg_ref[id] - all) * inv;
        }
        alpha_sh[id] = fast_exp2(now - all) * inv;
        const float lse = sum != 0.f ? (all + log2f(sum)) * kLn2 : -CUDART_INF_F;
        if (id < rows) sh.lse_dst[id] = lse;
      }
    }
  }
  // The softmax and gather warps write O: quarter of the lanes by warp, six warps a quarter, 8 rows of 32 dims at a
  // time; lane = value dim. (Through shared memory and a bulk copy it took 8500 cycles in place of 4400.)
  if (warp > 0) {
    if (!bar_red_or(2, kThreads - 32, !ok) && warp != kIssuePv && warp < kFirstKey) {
      tc_fence_after();
      const float4* inv_l = reinterpret_cast<const float4*>(smem + kOffAlpha);
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
#pragma unroll 1
      for (int k0 = warp < kIssuePv ? (warp - 1) >> 2 : (warp - 2) >> 2; k0 < 32; k0 += 6) {
        const int mt = k0 & 3, cc = (k0 >> 2) * 8, left = rows - cc;
        if (left <= 0) break;
        uint32_t o[8];
        tmem_ld8(tmem + lane_off + mt * kRows + cc, o);
        const float4 f0 = inv_l[cc / 4], f1 = inv_l[cc / 4 + 1];
        float x[8] = {__uint_as_float(o[0]) * f0.x, __uint_as_float(o[1]) * f0.y, __uint_as_float(o[2]) * f0.z,
                      __uint_as_float(o[3]) * f0.w, __uint_as_float(o[4]) * f1.x, __uint_as_float(o[5]) * f1.y,
                      __uint_as_float(o[6]) * f1.z, __uint_as_float(o[7]) * f1.w};
        const int dim = mt * 128 + (warp & 3) * 32;
        if (kLong && n > kKv8Segment) {  // and the segments before
          const float* seg = sh.o_seg + cc * kDv + dim + lane;
          const float* factor = reinterpret_cast<const float*>(smem + kOffSeg) + kRows + cc;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) x[k] = fmaf(seg[k * kDv], factor[k], x[k]);
        }
        if (sh.last) {
          // two rows a store: even lanes hold a pair of dims of the first, odd lanes of the second
          uint16_t* dst = static_cast<uint16_t*>(sh.o_dst) + (cc + (lane & 1)) * kDv + dim + (lane & ~1);
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? x[k] : x[k + 1], 1);
            if (k + (lane & 1) < left)
              *reinterpret_cast<uint32_t*>(dst + k * kDv) = lane & 1 ? pack_bf16x2(got, x[k + 1]) : pack_bf16x2(x[k], got);
          }
        } else {
          float* dst = static_cast<float*>(sh.o_dst) + cc * kDv + dim + lane;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < left) dst[k * kDv] = x[k];
        }
      }
    }
  }
  if (!ok) {
    *abort = 1;
    atomicOr(&sh.flags, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sh.flags != 0) {
    grid_dep_wait();  // (the status word has been written)
    atomicOr(p.status, sh.flags);
  }
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (kCut) grid_dep_wait();  // (this grid is not done before the one that it follows)
}

}  // namespace

cudaError_t configure_kv8_attn() {
  for (const auto& kernel : {kv8_attn_kernel<false, false>, kv8_attn_kernel<false, true>, kv8_attn_kernel<true, false>, kv8_attn_kernel<true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv8_attn(const Kv8AttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.groups, p.units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool is_long = static_cast<int64_t>(p.max_prefix_len) + p.nodes > kKv8Segment * kKv8Keys;
  const auto kernel = p.images ? is_long ? kv8_attn_kernel<false, true> : kv8_attn_kernel<false, false>
                               : is_long ? kv8_attn_kernel<true, true> : kv8_attn_kernel<true, false>;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace ddt
