// cache_ops.cuh -- launch parameters of the cache-size and block-sparse operators:
// key weights, eviction, block summaries, block selection, block attention.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "kernels.cuh"

namespace ddt {

#ifdef DDT_TEST_HOOKS
extern int32_t g_test_keep_back;  // api.cu
#endif

constexpr int32_t kStatusBadNode = 32;
constexpr int32_t kStatusBadBlock = 64;

// ---------------------------------------------------------------- scores of rows against queries
// Shared by key weights and block selection: 256 key rows stay in the shared
// memory of a CTA pair while the query rows stream past them.
constexpr int kScoreTileKeys = 256;
constexpr int kScoreTileRows = 128;  // query rows of one tile
enum ScoreMode : int { kScoreWeight = 0, kScoreBlock = 1 };

struct ScoreParams {
  CUtensorMap tmap_q;        // queries as [rows][576] bf16, box 64 cols x box_rows, 128-byte swizzle
  const uint16_t* keys;      // bf16 [*, 576]
  const int32_t* slot_idx;   // [B, slot_stride], or null: request b's row j is keys[b * key_stride + j]
  const int32_t* prefix_len; // [B]
  int64_t pool_slots;
  int64_t key_stride;        // rows per request when slot_idx is null; row stride of the outputs
  int32_t max_prefix_len;
  int32_t block;             // kScoreBlock: positions per block (rows = ceil(len / block)); else 1
  int32_t slot_stride;
  int32_t batch;
  int32_t rows;              // query rows per request
  int32_t tile_rows;         // query rows per tile
  int32_t tiles;             // ceil(rows / tile_rows)
  int32_t tile_n;            // MMA N: tile_rows rounded up
  int32_t heads;             // kScoreBlock: consecutive rows that make one node
  int32_t nodes;             // kScoreBlock: T
  int32_t key_tiles;         // key tiles of the longest request
  int32_t splits;            // shares of the query tiles (few key tiles, many rows)
  int32_t units;             // batch * key_tiles * splits
  float* part;               // kScoreWeight with splits > 1: [splits, B, slot_stride] partial sums
  int64_t part_stride;       // batch * slot_stride
  float scale_log2;          // kScoreWeight: sm_scale * log2(e)
  float decay;
  const int32_t* node_idx;   // kScoreWeight with packed rows: [B, sel], looked over for the status word; else null
  int32_t sel;
  const float* row_aux;      // [B, rows]: kScoreWeight natural-log lse, kScoreBlock query scales
  const float* weight_in;    // kScoreWeight: [B, slot_stride] or null
  float* weight_out;         // kScoreWeight: [B, slot_stride]
  const float* key_scale;    // kScoreBlock: [B, key_stride]
  float* score;              // kScoreBlock: [B, T, key_stride]
  int32_t* status;
#ifdef DDT_TEST_HOOKS
  int32_t test_keep_back;    // tile whose score buffer is not handed back (-1: none), so that the next wait for it runs out
#endif
};

cudaError_t configure_scores();
// after_kernel: the query rows and row_aux are written by the kernel launched just
// before, which this one follows as a programmatic dependent
cudaError_t launch_scores(const ScoreParams& p, ScoreMode mode, int sm_count, bool after_kernel, cudaStream_t stream);

// Selected nodes' query rows and lse, packed (node_idx[b][s], -1 = none).
struct PackParams {
  const uint16_t* q;
  const float* lse;
  const int32_t* node_idx;   // [B, sel]
  uint16_t* q_out;           // [B, sel, H, 576]
  float* lse_out;            // [B, sel, H]; +inf for rows of no node
  int32_t nodes, heads, sel;
  int32_t* status;
};
cudaError_t launch_pack_nodes(const PackParams& p, int batch, cudaStream_t stream);

// ---------------------------------------------------------------- eviction
struct EvictParams {
  const float* weight;       // [B, stride]
  const int32_t* slot_idx;   // [B, stride]
  const int32_t* prefix_len; // [B]
  const int32_t* keep_len;   // [B]
  int32_t* slot_out;         // [B, stride]
  float* weight_out;         // [B, stride]
  int32_t* len_out;          // [B]
  int32_t* freed;            // [B, stride]
  int32_t stride, max_prefix_len, sink, recent;
  int32_t* status;
};
cudaError_t configure_evict();
cudaError_t launch_kv_evict(const EvictParams& p, int batch, int sm_count, cudaStream_t stream);

// ---------------------------------------------------------------- block summaries and selection
struct SummaryParams {
  const uint16_t* kv;
  const int32_t* slot_idx;
  const int32_t* prefix_len;
  const int32_t* from_len;   // [B] or null
  uint16_t* summary;         // bf16 [B, blocks, 576]: integers in [-127, 127]
  float* scale;              // [B, blocks]
  int64_t pool_slots;
  int32_t slot_stride, max_prefix_len, block, blocks;
  int32_t* status;
#ifdef DDT_TEST_HOOKS
  int32_t test_keep_back;    // stage that is not handed back (-1: none), so that the next wait for it runs out
#endif
};
cudaError_t configure_summary();
cudaError_t launch_block_summary(const SummaryParams& p, int batch, int sm_count, cudaStream_t stream);

struct QuantParams {
  const uint16_t* q;         // bf16 [rows, 576]
  uint16_t* q_int;           // bf16 [rows, 576]: integers in [-127, 127]
  float* q_scale;            // [rows]
  int64_t rows;
  int32_t* status;           // cleared: this is a selection's first kernel
};
cudaError_t launch_quant_rows(const QuantParams& p, cudaStream_t stream);

struct TopkParams {
  const float* score;        // [B, T, blocks]
  const int32_t* prefix_len;
  int32_t* block_idx;        // [B, T, topk]
  int32_t nodes, blocks, block, topk, first, last, max_prefix_len;
  int32_t* status;
};
cudaError_t configure_topk();
cudaError_t launch_block_topk(const TopkParams& p, int batch, int sm_count, cudaStream_t stream);

// ---------------------------------------------------------------- block attention
constexpr int kBlockRows = 64;  // (node, head) rows of one group

struct alignas(16) BlockEntry {
  unsigned long long mask;  // rows of the group that read it
  int32_t index;            // block of the prefix, or pool slot of a tree row
  int32_t tree;             // 1: a tree row
};

struct BlockAttnParams {
  CUtensorMap tmap_kv;        // kv as [N][576], box 64 cols x 1 row, 128-byte swizzle
  const uint16_t* q;          // bf16 [B, T, H, 576]
  const uint16_t* kv;         // bf16 [N, 576]
  const int32_t* slot_idx;    // [B, slot_stride]
  const int32_t* prefix_len;  // [B]
  const int32_t* block_idx;   // [B, T, topk]
  const int32_t* tree_parent;    // [B, T]
  const int32_t* tree_slot_idx;  // [B, T]
  BlockEntry* list;           // [B * groups, list_cap]: union of the group's lists, in block order
  BlockEntry* tree;           // [B * groups, T]: its nodes' ancestors and themselves, in node order
  int32_t* list_len;          // [B * groups]
  int32_t* tree_len;          // [B * groups]
  int32_t* list_flags;        // [B * groups] status bits found while making the lists
  int64_t pool_slots;
  int64_t list_cap;
  int64_t pstride;            // rows between consecutive splits of one request
  int32_t batch, nodes, heads, slot_stride, max_prefix_len, block, topk;
  int32_t groups;             // per request
  int32_t group_nodes;        // nodes of a group (heads <= 64; else a group is 64 heads of one node)
  int32_t splits;
  bool clustered;             // the splits of a group are one cluster, which joins them
  float scale_log2;
  float* o_part;              // fp32 [B, splits, pstride, 512], normalised (splits > 1, not clustered)
  float* lse_part;            // fp32 [B, splits, pstride], natural log
  uint16_t* out;              // bf16 [B, T, H, 512]
  float* lse;                 // fp32 [B, T, H]
  int32_t* status;
#ifdef DDT_TEST_HOOKS
  int32_t test_keep_back;    // tile whose score buffer is not handed back (-1: none), so that the next wait for it runs out
#endif
};
constexpr int kBlockCluster = 8;
struct BlockClusters {
  int count[kBlockCluster + 1] = {};  // clusters of each size that one device runs at once
};
cudaError_t configure_block_attn(BlockClusters* clusters);  // on the current device
// Whether groups of `rows` rows in `splits` splits are clusters: they all run at once, and the join is short.
bool block_cluster_fits(int64_t groups, int rows, int splits, const BlockClusters& clusters);
cudaError_t launch_block_union(const BlockAttnParams& p, cudaStream_t stream);
cudaError_t launch_block_attn(const BlockAttnParams& p, cudaStream_t stream);

// The merge of block attention's key splits.
struct BlockMergeParams {
  int64_t rows;                  // of a request: T * H, also the rows between its splits
  int32_t splits;                // 2 to 32
  const float* o_part;
  const float* lse_part;
  uint16_t* out;                 // bf16 [B, T, H, 512]
  float* lse;                    // fp32 [B, T, H]
};
cudaError_t launch_block_merge(const BlockMergeParams& p, int batch, cudaStream_t stream);

// Map of a score to an unsigned key with the same order: NaN lowest (equal to
// -inf), -0 equal to +0.
__host__ __device__ inline uint32_t order_key_bits(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) u = 0xff800000u;  // NaN -> -inf
  if (u == 0x80000000u) u = 0u;                          // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace ddt
