// kv8.cuh -- launch parameters of the 8-bit latent cache: rows in, rows out, verify attention over it.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "kernels.cuh"

namespace ddt {

#ifdef DDT_TEST_HOOKS
extern int32_t g_test_keep_back;  // api.cu
#endif

// A slot: 512 latent values in e4m3 and 64 rope values in bf16, both divided by the
// slot's scale, which lies in an array of its own (a row is five 128-byte lines, and
// the scales of a pool stay in L2).
constexpr int kKv8Row = 640;
constexpr int kKv8MinExp = -60;   // of a scale; products and quotients with it stay inside fp32
constexpr int kRopePairs = 32;

constexpr int32_t kStatusBadPosition = 128;

// ---------------------------------------------------------------- rows in and out
struct Kv8WriteParams {
  const uint16_t* rows;        // bf16, row i at rows + i * row_stride: 512 latent, 64 rope
  int64_t row_stride;
  const int32_t* slots;        // [n], -1: not written
  const uint16_t* norm_weight; // bf16 [512] or null
  float eps;
  const float* rotation;       // fp32 [positions, 64]: 32 cosines, 32 sines; or null
  const int32_t* position;     // [n]
  int32_t positions;
  uint8_t* pool;               // [N, 640]
  float* scale;                // [N]
  int64_t n, pool_slots;
  int32_t* status;             // or null
};
cudaError_t launch_kv8_write(const Kv8WriteParams& p, bool interleaved, int sm_count, cudaStream_t stream);

struct Kv8ReadParams {
  const uint8_t* pool;
  const float* scale;
  const int32_t* slots;        // [n], -1: a row of zeros
  uint16_t* rows;              // bf16, row i at rows + i * row_stride
  int64_t row_stride;
  int64_t n, pool_slots;
  int32_t* status;             // or null
};
cudaError_t launch_kv8_read(const Kv8ReadParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- verify attention
constexpr int kKv8Rows = 64;      // (node, head) rows of one group
constexpr int kKv8Keys = 64;      // keys of a tile
// Tiles whose products add up in tensor memory; then they join those before in fp32. The tensor core cuts its sums (one unit
// in the last place of fp32 for 32 keys and part, all towards zero: 1.6e-4 of a sum of one sign after 512 tiles, 2.8e-3 after
// 7000), and what small weights lose counts times the keys.
constexpr int kKv8Segment = 512;
constexpr int kKv8MaxShared = 1024;  // requests of a batch whose tiles are shared out

constexpr int kKv8Chunk = kKv8Keys * 128;         // 128 bytes of 64 keys
// A group's query rows as its units take them. Row r has two lanes of the tensor memory, for its two parts:
// lane 32 (r / 16) + r % 16 and 16 lanes on.
//   512 bytes of each of the 128 lanes: 16-byte piece u of lane l at (128 u + l) 16
//   rope values, a 128-byte row for each of the 64, 128-byte swizzle
//   the rows' factors of a score, fp32
constexpr int kKv8ImageRope = 128 * 512, kKv8ImageFactor = kKv8ImageRope + kKv8Rows * 128, kKv8Image = kKv8ImageFactor + 256;

// Rows of a group, within its request, if `nodes` nodes are active (rows <= 0: none).
struct Kv8Group {
  int row0, rows;
};
__host__ __device__ inline Kv8Group kv8_group(int heads, int group_nodes, int nodes, int g) {
  Kv8Group u;
  if (heads <= kKv8Rows) {
    u.row0 = g * group_nodes * heads;
    const int n = nodes - g * group_nodes;
    u.rows = (n < group_nodes ? n : group_nodes) * heads;
  } else {
    const int slices = (heads + kKv8Rows - 1) / kKv8Rows, t = g / slices, sl = g - t * slices, left = heads - sl * kKv8Rows;
    u.row0 = t * heads + sl * kKv8Rows;
    u.rows = t < nodes ? (left < kKv8Rows ? left : kKv8Rows) : 0;
  }
  return u;
}

// Groups of a request with so many active nodes.
__host__ __device__ inline int kv8_groups(int heads, int group_nodes, int nodes) {
  return heads <= kKv8Rows ? (nodes + group_nodes - 1) / group_nodes : nodes * ((heads + kKv8Rows - 1) / kKv8Rows);
}

struct Kv8PrepareParams {
  const uint16_t* q;             // bf16 [B, T, H, 576]
  const int32_t* prefix_len;
  const int32_t* tree_len;
  uint8_t* images;               // [B, groups, kKv8Image], or null: the units cut their rows themselves
  uint16_t* out;                 // rows of inactive nodes are written
  float* lse;
  int32_t batch, nodes, heads, max_prefix_len, groups, group_nodes;
  float scale_log2;              // sm_scale * log2(e)
  int32_t* status;               // written as a whole; the units add to it
};
cudaError_t launch_kv8_prepare(const Kv8PrepareParams& p, cudaStream_t stream);

struct Kv8Piece {                 // a request's units, for the merge
  int32_t first, count;
};

struct Kv8AttnParams {
  CUtensorMap tmap;              // pool as [N][640] bytes, box 128 bytes x 1 row, 128-byte swizzle
  const uint8_t* images;         // [B, groups, kKv8Image], of the kernel before; or null, then
  const uint16_t* q;             // bf16 [B, T, H, 576], and
  float scale_log2;              // sm_scale * log2(e)
  const uint8_t* kv;             // [N, 640]
  const float* scale;            // [N]
  const int32_t* slot_idx;       // [B, slot_stride]
  const int32_t* prefix_len;     // [B]
  const int32_t* tree_parent;    // [B, T]
  const int32_t* tree_slot_idx;  // [B, T]
  const int32_t* tree_len;       // [B] or null
  int64_t pool_slots;
  int32_t batch, nodes, heads, slot_stride, max_prefix_len;
  int32_t groups;                // per request
  int32_t group_nodes;           // nodes of a group (heads <= 64; else a group is 64 heads of one node)
  int32_t shares;                // the batch's tiles in this many equal shares, or less; 0: one unit a request
  int32_t units;                 // bound on the units of a group: shares + batch - 1, or batch
  int32_t sms;
  float* o_part;                 // fp32 [units, T * H, 512], normalised
  float* lse_part;               // fp32 [units, T * H], natural log
  Kv8Piece* pieces;              // [B]
  uint16_t* out;                 // bf16 [B, T, H, 512]
  float* lse;                    // fp32 [B, T, H]
  int32_t* status;
#ifdef DDT_TEST_HOOKS
  int32_t test_keep_back;        // tile whose score buffer is not handed back (-1: none)
#endif
};
cudaError_t configure_kv8_attn();
cudaError_t launch_kv8_attn(const Kv8AttnParams& p, cudaStream_t stream);

struct Kv8MergeParams {
  const float* o_part;
  const float* lse_part;
  const Kv8Piece* pieces;
  const int32_t* tree_len;
  uint16_t* out;
  float* lse;
  int32_t batch, nodes, heads;
  int32_t warps;                 // warps that share a row: 1, 2, 4, 8 or 16
};
cudaError_t launch_kv8_merge(const Kv8MergeParams& p, cudaStream_t stream);

// Requests, lengths and trees as the kernels clamp them.
__device__ __forceinline__ int kv8_len(const int32_t* prefix_len, int b, int max_prefix_len) {
  const int L = __ldg(prefix_len + b);
  return L < 0 ? 0 : (L > max_prefix_len ? max_prefix_len : L);
}
__device__ __forceinline__ int kv8_nodes(const int32_t* tree_len, int b, int nodes) {
  if (!tree_len) return nodes;
  const int n = __ldg(tree_len + b);
  return n < 0 ? 0 : (n > nodes ? nodes : n);
}

}  // namespace ddt
