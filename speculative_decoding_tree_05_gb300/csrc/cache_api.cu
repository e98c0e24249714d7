// cache_api.cu -- the extern "C" entry points of the cache-size and block-sparse
// operators: argument checks, workspace layout, launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cstdint>
#include "../../include/ddtree.h"
#include "cache_ops.cuh"
#include "host.cuh"

namespace ddt {
namespace {

constexpr int kScoreUnitTiles = 4;  // fixed cost of one score unit, in query tiles
constexpr int kWeightSumTiles = 3;  // the launch that adds the shares' sums, in query tiles
// Fixed costs in block attention, in 64-key tiles (2.1 us): of a unit, and of a merge
// kernel behind it.  (8 requests of 17 nodes x 16 heads in a graph: 3 splits in one
// wave 76 to 81 us, 11 splits in three waves 94 us.)
constexpr int kBlockUnitTiles = 5, kBlockMergeTiles = 2;

int round32(int x) { return (x + 31) / 32 * 32; }

// check_dims, and the positions that these kernels count: with steps of a few
// thousand and block sizes added they stay inside 32 bits.
int check_cache_dims(const ddt_dims* d) {
  const int rc = check_dims(d);
  if (rc != DDT_OK) return rc;
  return d->max_prefix_len > (1 << 30) ? DDT_ERR_DIMS : DDT_OK;
}

bool clear_status(void* workspace, cudaStream_t s) {
  return cudaMemsetAsync(workspace, 0, 4 * sizeof(int32_t), s) == cudaSuccess;
}

// Key tiles, and the shares of the query tiles: with fewer key tiles than CTA
// pairs the pairs left over take shares of the rows.  A unit costs its tiles plus
// about kScoreUnitTiles (the gather of its keys and the pipeline's fill), sharing
// itself split_tiles (the sum of the shares).
struct ScoreGrid {
  int key_tiles, splits, units;
};
bool score_grid(int64_t batch, int64_t keys, int tiles, int sm_count, int split_tiles, ScoreGrid* g) {
  const int64_t key_tiles = (keys + kScoreTileKeys - 1) / kScoreTileKeys;
  const int64_t all = batch * key_tiles, pairs = std::max(1, sm_count / 2);
  if (all > INT32_MAX / 64) return false;
  int64_t best = -1;
  int splits = 1;
  for (int s = 1; s <= std::min(tiles, 64); ++s) {
    const int64_t cost =
        (all * s + pairs - 1) / pairs * ((tiles + s - 1) / s + kScoreUnitTiles) + (s > 1 ? split_tiles : 0);
    if (best < 0 || cost < best) {
      best = cost;
      splits = s;
    }
  }
  *g = {static_cast<int>(key_tiles), splits, static_cast<int>(all * splits)};
  return true;
}

// Query rows per tile of the weights: equal tiles of at most kScoreTileRows.
int weight_tile_rows(int rows) {
  const int tiles = (rows + kScoreTileRows - 1) / kScoreTileRows;
  return round32((rows + tiles - 1) / tiles);
}

struct WeightLayout {
  int tile_rows, tiles;
  ScoreGrid grid;
  size_t q_off, lse_off, part_off, bytes;
};
// sm_count 0: the sizes only (no grid, no bytes)
int weight_layout(const ddt_dims* d, int32_t num_sel, int sm_count, WeightLayout* w) {
  const int rc = check_cache_dims(d);
  if (rc != DDT_OK) return rc;
  if (num_sel < 0 || num_sel > 65535) return DDT_ERR_DIMS;
  const int64_t rows = int64_t(num_sel > 0 ? num_sel : d->num_nodes) * d->num_heads;
  if (rows * d->batch > INT32_MAX) return DDT_ERR_DIMS;
  w->tile_rows = weight_tile_rows(static_cast<int>(rows));
  w->tiles = static_cast<int>((rows + w->tile_rows - 1) / w->tile_rows);
  if (!score_grid(d->batch, d->max_prefix_len, w->tiles, std::max(sm_count, 2), kWeightSumTiles, &w->grid)) return DDT_ERR_DIMS;
  const size_t packed = num_sel > 0 ? size_t(rows) * d->batch : 0;
  w->q_off = kStatusBytes;
  w->lse_off = align_up(w->q_off + packed * kRowBytes, 256);
  w->part_off = align_up(w->lse_off + packed * sizeof(float), 256);
  const size_t parts = w->grid.splits > 1 ? size_t(w->grid.splits) * d->batch * d->slot_stride : 0;
  w->bytes = align_up(w->part_off + parts * sizeof(float), 256);
  return DDT_OK;
}

bool block_ok(int32_t block) { return block == 16 || block == 32 || block == 64 || block == 128; }

struct SelectLayout {
  int64_t blocks;
  size_t q_off, scale_off, score_off, bytes;
};
int select_layout(const ddt_dims* d, int32_t block, SelectLayout* w) {
  const int rc = check_cache_dims(d);
  if (rc != DDT_OK) return rc;
  if (!block_ok(block)) return DDT_ERR_DIMS;
  const size_t nodes = size_t(d->batch) * d->num_nodes, rows = nodes * d->num_heads;
  w->blocks = (int64_t(d->max_prefix_len) + block - 1) / block;
  w->q_off = kStatusBytes;
  w->scale_off = align_up(w->q_off + rows * kRowBytes, 256);
  w->score_off = align_up(w->scale_off + rows * sizeof(float), 256);
  w->bytes = align_up(w->score_off + nodes * w->blocks * sizeof(float), 256);
  return DDT_OK;
}

struct BlocksLayout {
  int groups, group_nodes, splits;
  bool clustered;
  int64_t list_cap;
  size_t len_off, tree_len_off, flags_off, list_off, tree_off, lse_off, o_off, bytes;
};

// Groups of up to 64 (node, head) rows, and the key splits of each.  The splits
// minimise waves * (64-key tiles of a unit + kBlockUnitTiles), and kBlockMergeTiles
// where a merge kernel follows; the tiles are those of lists that do not overlap (how
// far they do is known on the device only).
int blocks_layout(const ddt_dims* d, int32_t block, int32_t topk, int sm_count, const BlockClusters& clusters,
                  BlocksLayout* w) {
  const int rc = check_cache_dims(d);
  if (rc != DDT_OK) return rc;
  if (!block_ok(block) || topk < 1 || topk > (1 << 20)) return DDT_ERR_DIMS;
  const int H = d->num_heads, T = d->num_nodes;
  w->group_nodes = H <= kBlockRows ? std::min(T, kBlockRows / H) : 1;
  w->groups = H <= kBlockRows ? (T + w->group_nodes - 1) / w->group_nodes : T * ((H + kBlockRows - 1) / kBlockRows);
  const int64_t all = int64_t(d->batch) * w->groups;
  if (all > (1 << 30)) return DDT_ERR_DIMS;
  const int64_t blocks = (int64_t(d->max_prefix_len) + block - 1) / block;
  w->list_cap = std::min<int64_t>(int64_t(w->group_nodes) * topk, blocks);
  const int64_t tiles = (w->list_cap * block + std::min(T, 16) + 63) / 64;  // with a path of tree rows
  const int group_rows = std::min(w->group_nodes * H, kBlockRows);
  int64_t best_cost = -1;
  w->splits = 1;
  for (int s = 1; s <= std::min<int64_t>(tiles, 32); ++s) {
    const int64_t cost = (all * s + sm_count - 1) / sm_count * ((tiles + s - 1) / s + kBlockUnitTiles) +
                         (s == 1 || block_cluster_fits(all, group_rows, s, clusters) ? 0 : kBlockMergeTiles);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      w->splits = s;
    }
  }
  w->clustered = block_cluster_fits(all, group_rows, w->splits, clusters);
  const size_t part = w->splits > 1 && !w->clustered ? size_t(d->batch) * w->splits * T * H : 0;
  w->len_off = kStatusBytes;
  w->tree_len_off = align_up(w->len_off + all * sizeof(int32_t), 256);
  w->flags_off = align_up(w->tree_len_off + all * sizeof(int32_t), 256);
  w->list_off = align_up(w->flags_off + all * sizeof(int32_t), 256);
  w->tree_off = align_up(w->list_off + size_t(all) * w->list_cap * sizeof(BlockEntry), 256);
  w->lse_off = align_up(w->tree_off + size_t(all) * T * sizeof(BlockEntry), 256);
  w->o_off = align_up(w->lse_off + part * sizeof(float), 256);
  w->bytes = align_up(w->o_off + part * kDv * sizeof(float), 256);
  return DDT_OK;
}

}  // namespace
}  // namespace ddt

using namespace ddt;

extern "C" size_t ddtree_kv_weight_workspace_bytes(const ddt_dims* dims, int32_t num_sel) {
  int sms = 0;
  WeightLayout w;
  if (current_device(&sms) != DDT_OK || weight_layout(dims, num_sel, sms, &w) != DDT_OK) return 0;
  return w.bytes;
}

extern "C" int ddtree_kv_weight(const void* q, const void* kv_pool, const int32_t* slot_idx, const int32_t* prefix_len,
                                const float* lse, const int32_t* node_idx, int32_t num_sel, float sm_scale,
                                float decay, const float* weight_in, float* weight_out, const ddt_dims* dims,
                                void* workspace, size_t workspace_bytes, ddt_stream_t stream) {
  WeightLayout w;
  int rc = weight_layout(dims, num_sel, 0, &w);  // the sizes, before any device query
  if (rc != DDT_OK) return rc;
  if (dims->batch == 0) return DDT_OK;
  if (!q || !kv_pool || !prefix_len || !lse || !workspace || (num_sel > 0 && !node_idx) ||
      ((!slot_idx || !weight_out) && dims->max_prefix_len > 0) || (!weight_in && decay != 0.f))
    return DDT_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(workspace, 256) || !aligned(slot_idx, 4) ||
      !aligned(prefix_len, 4) || !aligned(lse, 4) || !aligned(node_idx, 4) || !aligned(weight_in, 4) ||
      !aligned(weight_out, 4))
    return DDT_ERR_ALIGN;
  // in place, or apart: an entry is written while others' old weights are still to be read
  const size_t table = size_t(dims->batch) * dims->slot_stride * 4;
  if (decay != 0.f && weight_in != weight_out && overlap(weight_in, table, weight_out, table)) return DDT_ERR_ALIAS;
  int sms = 0;
  if ((rc = current_device(&sms)) != DDT_OK) return rc;
  if ((rc = weight_layout(dims, num_sel, sms, &w)) != DDT_OK) return rc;
  if (workspace_bytes < w.bytes) return DDT_ERR_WORKSPACE;
  const bool packed = num_sel > 0;
  ScoreParams p = {};
#ifdef DDT_TEST_HOOKS
  p.test_keep_back = g_test_keep_back;
#endif
  p.batch = dims->batch;
  p.rows = (packed ? num_sel : dims->num_nodes) * dims->num_heads;
  const int64_t q_rows = int64_t(p.batch) * p.rows;
  p.tile_rows = p.tile_n = w.tile_rows;
  p.tiles = w.tiles;
  p.key_tiles = w.grid.key_tiles;
  p.splits = w.grid.splits;
  p.units = w.grid.units;
  p.keys = static_cast<const uint16_t*>(kv_pool);
  p.slot_idx = slot_idx;
  p.prefix_len = prefix_len;
  p.pool_slots = dims->pool_slots;
  p.max_prefix_len = dims->max_prefix_len;
  p.block = 1;
  p.slot_stride = dims->slot_stride;
  p.heads = dims->num_heads;
  p.nodes = dims->num_nodes;
  p.scale_log2 = static_cast<float>(sm_scale * 1.4426950408889634);
  p.decay = decay;
  p.weight_in = decay != 0.f ? weight_in : nullptr;
  p.weight_out = weight_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int32_t*>(ws);
  p.part = reinterpret_cast<float*>(ws + w.part_off);
  p.part_stride = int64_t(dims->batch) * dims->slot_stride;
  const void* qs = packed ? static_cast<const void*>(ws + w.q_off) : q;
  p.row_aux = packed ? reinterpret_cast<const float*>(ws + w.lse_off) : lse;
  if (!encode_pool_map(&p.tmap_q, qs, q_rows, 64, p.tile_n / 2)) return DDT_ERR_LAUNCH;  // one CTA's half of a tile
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // (with packed rows their kernel clears the status word)
  if (!packed && !clear_status(workspace, s)) return DDT_ERR_LAUNCH;
  if (packed) {
    PackParams k = {};
    k.q = static_cast<const uint16_t*>(q);
    k.lse = lse;
    k.node_idx = node_idx;
    k.q_out = reinterpret_cast<uint16_t*>(ws + w.q_off);
    k.lse_out = reinterpret_cast<float*>(ws + w.lse_off);
    k.nodes = dims->num_nodes;
    k.heads = dims->num_heads;
    k.sel = num_sel;
    k.status = p.status;
    p.node_idx = node_idx;
    p.sel = num_sel;
    if (launch_pack_nodes(k, dims->batch, s) != cudaSuccess) return DDT_ERR_LAUNCH;
  }
  return launch_scores(p, kScoreWeight, sms, packed, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

extern "C" int ddtree_kv_evict(const float* weight, const int32_t* slot_idx, const int32_t* prefix_len,
                               const int32_t* keep_len, int32_t sink, int32_t recent, int32_t* slot_idx_out,
                               float* weight_out, int32_t* prefix_len_out, int32_t* freed_slots, const ddt_dims* dims,
                               void* workspace, ddt_stream_t stream) {
  int rc = check_cache_dims(dims);
  if (rc != DDT_OK) return rc;
  if (sink < 0 || recent < 0) return DDT_ERR_DIMS;
  if (dims->batch == 0) return DDT_OK;
  if (!prefix_len || !keep_len || !prefix_len_out || !workspace ||
      ((!weight || !slot_idx || !slot_idx_out || !weight_out || !freed_slots) && dims->max_prefix_len > 0))
    return DDT_ERR_NULL;
  if (!aligned(workspace, 256) || !aligned(weight, 4) || !aligned(slot_idx, 4) || !aligned(prefix_len, 4) ||
      !aligned(keep_len, 4) || !aligned(slot_idx_out, 4) || !aligned(weight_out, 4) || !aligned(prefix_len_out, 4) ||
      !aligned(freed_slots, 4))
    return DDT_ERR_ALIGN;
  // a request's entries are read while others' are written: no output may cover an input or another output
  const size_t table = size_t(dims->batch) * dims->slot_stride * 4, lens = size_t(dims->batch) * 4;
  const struct { const void* p; size_t n; } in[] = {{weight, table}, {slot_idx, table}, {prefix_len, lens}, {keep_len, lens}},
      out[] = {{slot_idx_out, table}, {weight_out, table}, {freed_slots, table}, {prefix_len_out, lens}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return DDT_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return DDT_ERR_ALIAS;
  }
  int sms = 0;
  if ((rc = current_device(&sms)) != DDT_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  EvictParams p = {};
  p.weight = weight;
  p.slot_idx = slot_idx;
  p.prefix_len = prefix_len;
  p.keep_len = keep_len;
  p.slot_out = slot_idx_out;
  p.weight_out = weight_out;
  p.len_out = prefix_len_out;
  p.freed = freed_slots;
  p.stride = dims->slot_stride;
  p.max_prefix_len = dims->max_prefix_len;
  p.sink = sink;
  p.recent = recent;
  p.status = static_cast<int32_t*>(workspace);
  return launch_kv_evict(p, dims->batch, sms, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

extern "C" int ddtree_block_summary(const void* kv_pool, const int32_t* slot_idx, const int32_t* prefix_len,
                                    const int32_t* from_len, int32_t block, void* summary, float* scale,
                                    const ddt_dims* dims, void* workspace, ddt_stream_t stream) {
  int rc = check_cache_dims(dims);
  if (rc != DDT_OK) return rc;
  if (!block_ok(block)) return DDT_ERR_DIMS;
  if (dims->batch == 0) return DDT_OK;
  if (!kv_pool || !prefix_len || !workspace || ((!slot_idx || !summary || !scale) && dims->max_prefix_len > 0))
    return DDT_ERR_NULL;
  if (!aligned(kv_pool, 16) || !aligned(summary, 16) || !aligned(workspace, 256) || !aligned(slot_idx, 4) ||
      !aligned(prefix_len, 4) || !aligned(from_len, 4) || !aligned(scale, 4))
    return DDT_ERR_ALIGN;
  int sms = 0;
  if ((rc = current_device(&sms)) != DDT_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!clear_status(workspace, s)) return DDT_ERR_LAUNCH;
  SummaryParams p = {};
#ifdef DDT_TEST_HOOKS
  p.test_keep_back = g_test_keep_back;
#endif
  p.kv = static_cast<const uint16_t*>(kv_pool);
  p.slot_idx = slot_idx;
  p.prefix_len = prefix_len;
  p.from_len = from_len;
  p.summary = static_cast<uint16_t*>(summary);
  p.scale = scale;
  p.pool_slots = dims->pool_slots;
  p.slot_stride = dims->slot_stride;
  p.max_prefix_len = dims->max_prefix_len;
  p.block = block;
  p.blocks = static_cast<int32_t>((int64_t(dims->max_prefix_len) + block - 1) / block);
  p.status = static_cast<int32_t*>(workspace);
  return launch_block_summary(p, dims->batch, sms, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

extern "C" size_t ddtree_block_select_workspace_bytes(const ddt_dims* dims, int32_t block) {
  SelectLayout w;
  return select_layout(dims, block, &w) == DDT_OK ? w.bytes : 0;
}

extern "C" int ddtree_block_select(const void* q, const void* summary, const float* scale, const int32_t* prefix_len,
                                   int32_t block, int32_t topk, int32_t first, int32_t last, int32_t* block_idx,
                                   const ddt_dims* dims, void* workspace, size_t workspace_bytes,
                                   ddt_stream_t stream) {
  SelectLayout w;
  int rc = select_layout(dims, block, &w);
  if (rc != DDT_OK) return rc;
  if (topk < 1 || topk > (1 << 20) || first < 0 || last < 0) return DDT_ERR_DIMS;
  if (dims->batch == 0) return DDT_OK;
  if (!q || !prefix_len || !block_idx || !workspace || ((!summary || !scale) && w.blocks > 0)) return DDT_ERR_NULL;
  if (!aligned(q, 16) || !aligned(summary, 16) || !aligned(workspace, 256) || !aligned(scale, 4) ||
      !aligned(prefix_len, 4) || !aligned(block_idx, 4))
    return DDT_ERR_ALIGN;
  if (workspace_bytes < w.bytes) return DDT_ERR_WORKSPACE;
  int sms = 0;
  if ((rc = current_device(&sms)) != DDT_OK) return rc;
  const int H = dims->num_heads;
  ScoreParams p = {};
#ifdef DDT_TEST_HOOKS
  p.test_keep_back = g_test_keep_back;
#endif
  p.batch = dims->batch;
  p.rows = dims->num_nodes * H;
  const int64_t q_rows = int64_t(p.batch) * p.rows;
  if (q_rows > INT32_MAX || w.blocks * p.batch > INT32_MAX) return DDT_ERR_DIMS;
  // a tile holds whole nodes (up to 128 heads), so each epilogue set owns its nodes
  p.tile_rows = H <= kScoreTileRows ? std::min(p.rows, kScoreTileRows / H * H) : kScoreTileRows;
  p.tile_n = round32(p.tile_rows);
  p.tiles = (p.rows + p.tile_rows - 1) / p.tile_rows;
  ScoreGrid grid;
  // (a node of more heads spans tiles: its rows are not shared out)
  if (!score_grid(p.batch, w.blocks, H <= kScoreTileRows ? p.tiles : 1, sms, 0, &grid)) return DDT_ERR_DIMS;
  p.key_tiles = grid.key_tiles;
  p.splits = grid.splits;
  p.units = grid.units;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.keys = static_cast<const uint16_t*>(summary);
  p.prefix_len = prefix_len;
  p.key_stride = w.blocks;
  p.max_prefix_len = dims->max_prefix_len;
  p.block = block;
  p.heads = H;
  p.nodes = dims->num_nodes;
  p.row_aux = reinterpret_cast<const float*>(ws + w.scale_off);
  p.key_scale = scale;
  p.score = reinterpret_cast<float*>(ws + w.score_off);
  p.status = reinterpret_cast<int32_t*>(ws);
  if (!encode_pool_map(&p.tmap_q, ws + w.q_off, q_rows, 64, p.tile_n / 2)) return DDT_ERR_LAUNCH;
  QuantParams k = {};
  k.q = static_cast<const uint16_t*>(q);
  k.q_int = reinterpret_cast<uint16_t*>(ws + w.q_off);
  k.q_scale = reinterpret_cast<float*>(ws + w.scale_off);
  k.rows = q_rows;
  TopkParams t = {};
  t.score = p.score;
  t.prefix_len = prefix_len;
  t.block_idx = block_idx;
  t.nodes = dims->num_nodes;
  t.blocks = static_cast<int32_t>(w.blocks);
  t.block = block;
  t.topk = topk;
  t.first = first;
  t.last = last;
  t.max_prefix_len = dims->max_prefix_len;
  t.status = p.status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  k.status = p.status;  // cleared there
  if (launch_quant_rows(k, s) != cudaSuccess ||
      launch_scores(p, kScoreBlock, sms, true, s) != cudaSuccess || launch_block_topk(t, dims->batch, sms, s) != cudaSuccess)
    return DDT_ERR_LAUNCH;
  return DDT_OK;
}

extern "C" size_t ddtree_verify_blocks_workspace_bytes(const ddt_dims* dims, int32_t block, int32_t topk) {
  int sms = 0;
  BlockClusters clusters;
  BlocksLayout w;
  if (current_device(&sms, &clusters) != DDT_OK || blocks_layout(dims, block, topk, sms, clusters, &w) != DDT_OK) return 0;
  return w.bytes;
}

extern "C" int ddtree_verify_attn_blocks(const void* q, const void* kv_pool, const int32_t* slot_idx,
                                         const int32_t* prefix_len, const int32_t* tree_parent,
                                         const int32_t* tree_slot_idx, const int32_t* block_idx, int32_t block,
                                         int32_t topk, float sm_scale, void* out, float* lse, const ddt_dims* dims,
                                         void* workspace, size_t workspace_bytes, ddt_stream_t stream) {
  BlocksLayout w;
  BlockClusters clusters;
  int rc = blocks_layout(dims, block, topk, 1, clusters, &w);  // the sizes, before any device query
  if (rc != DDT_OK) return rc;
  if (dims->batch == 0) return DDT_OK;
  if (!q || !kv_pool || !prefix_len || !tree_parent || !tree_slot_idx || !block_idx || !out || !lse || !workspace ||
      (!slot_idx && dims->max_prefix_len > 0))
    return DDT_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      !aligned(slot_idx, 4) || !aligned(prefix_len, 4) || !aligned(tree_parent, 4) || !aligned(tree_slot_idx, 4) ||
      !aligned(block_idx, 4) || !aligned(lse, 4))
    return DDT_ERR_ALIGN;
  int sms = 0;
  if ((rc = current_device(&sms, &clusters)) != DDT_OK) return rc;
  if ((rc = blocks_layout(dims, block, topk, sms, clusters, &w)) != DDT_OK) return rc;
  if (workspace_bytes < w.bytes) return DDT_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  BlockAttnParams p = {};
#ifdef DDT_TEST_HOOKS
  p.test_keep_back = g_test_keep_back;
#endif
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint16_t*>(kv_pool);
  p.slot_idx = slot_idx;
  p.prefix_len = prefix_len;
  p.block_idx = block_idx;
  p.list = reinterpret_cast<BlockEntry*>(ws + w.list_off);
  p.tree = reinterpret_cast<BlockEntry*>(ws + w.tree_off);
  p.tree_parent = tree_parent;
  p.tree_slot_idx = tree_slot_idx;
  p.list_len = reinterpret_cast<int32_t*>(ws + w.len_off);
  p.tree_len = reinterpret_cast<int32_t*>(ws + w.tree_len_off);
  p.list_flags = reinterpret_cast<int32_t*>(ws + w.flags_off);
  p.pool_slots = dims->pool_slots;
  p.list_cap = w.list_cap;
  p.batch = dims->batch;
  p.nodes = dims->num_nodes;
  p.heads = dims->num_heads;
  p.pstride = int64_t(p.nodes) * p.heads;
  p.slot_stride = dims->slot_stride;
  p.max_prefix_len = dims->max_prefix_len;
  p.block = block;
  p.topk = topk;
  p.groups = w.groups;
  p.group_nodes = w.group_nodes;
  p.splits = w.splits;
  p.clustered = w.clustered;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.o_part = reinterpret_cast<float*>(ws + w.o_off);
  p.lse_part = reinterpret_cast<float*>(ws + w.lse_off);
  p.status = reinterpret_cast<int32_t*>(ws);
  if (!encode_pool_map(&p.tmap_kv, kv_pool, dims->pool_slots, 64, 1)) return DDT_ERR_LAUNCH;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  BlockMergeParams m = {};
  m.rows = p.pstride;
  m.splits = w.splits;
  m.o_part = p.o_part;
  m.lse_part = p.lse_part;
  m.out = p.out;
  m.lse = lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // (the union kernel clears the status word)
  if (launch_block_union(p, s) != cudaSuccess || launch_block_attn(p, s) != cudaSuccess ||
      (w.splits > 1 && !p.clustered && launch_block_merge(m, p.batch, s) != cudaSuccess))
    return DDT_ERR_LAUNCH;
  return DDT_OK;
}

// Host-side introspection of the schedule (not part of the public header; the CPU
// tests use it, no device is needed).  Block attention's layout on a device with
// sm_count SMs that runs clusters[s] clusters of s CTAs at once (s = 2 to 8): out =
// {groups of a request, key splits, 1 if they are clusters}; *bytes: the workspace.
extern "C" __attribute__((visibility("default"))) int ddtree_internal_blocks_plan(const ddt_dims* dims, int32_t block,
                                                                                  int32_t topk, int sm_count,
                                                                                  const int32_t* clusters, int32_t* out,
                                                                                  int64_t* bytes) {
  BlockClusters c;
  for (int s = 2; s <= kBlockCluster; ++s) c.count[s] = clusters[s];
  BlocksLayout w;
  const int rc = blocks_layout(dims, block, topk, sm_count, c, &w);
  if (rc != DDT_OK) return rc;
  out[0] = w.groups;
  out[1] = w.splits;
  out[2] = w.clustered ? 1 : 0;
  *bytes = static_cast<int64_t>(w.bytes);
  return DDT_OK;
}
