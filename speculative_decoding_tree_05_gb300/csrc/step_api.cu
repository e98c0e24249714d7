// step_api.cu -- the extern "C" entry points of the 8-bit latent cache and of the check
// of drafted tokens: argument checks, workspace layout, launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cstdint>
#include "../../include/ddtree.h"
#include "accept.cuh"
#include "host.cuh"
#include "kv8.cuh"

namespace ddt {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;  // of one call

bool clear_status(void* workspace, cudaStream_t s) {
  return cudaMemsetAsync(workspace, 0, 4 * sizeof(int32_t), s) == cudaSuccess;
}
// A call without rows or requests: its status is that nothing was wrong, not what the call before it left.
int nothing_to_do(void* workspace, size_t bytes, ddt_stream_t stream) {
  if (!workspace) return DDT_OK;
  if (!aligned(workspace, 256)) return DDT_ERR_ALIGN;
  if (bytes < kStatusBytes) return DDT_ERR_WORKSPACE;
  return clear_status(workspace, reinterpret_cast<cudaStream_t>(stream)) ? DDT_OK : DDT_ERR_LAUNCH;
}

struct Kv8Layout {
  int groups, group_nodes, shares, units;
  bool images;  // the query rows are cut by a kernel before
  size_t pieces_off, images_off, lse_off, o_off, bytes;
};

// Costs in tiles of 64 keys: of a unit (its prologue, the pipeline's fill, its output),
// of a merge, and of the partials, this many (unit, group)s a tile.
constexpr int kUnitTiles = 9, kMergeTiles = 3, kPartialsPerTile = 32;

// Groups of up to 64 (node, head) rows, and the shares of the batch's tiles: as many as
// minimise waves * (tiles of a share + kUnitTiles) and the merge. Only numbers of shares
// that just fill a number of waves can be best.
int kv8_layout(const ddt_dims* d, int sm_count, Kv8Layout* w) {
  const int rc = check_dims(d);
  if (rc != DDT_OK) return rc;
  if (d->max_prefix_len > (1 << 30)) return DDT_ERR_DIMS;
  const int H = d->num_heads, T = d->num_nodes;
  w->group_nodes = H <= kKv8Rows ? std::min(T, kKv8Rows / H) : 1;
  w->groups = kv8_groups(H, w->group_nodes, T);
  const int64_t B = d->batch, most = (int64_t(d->max_prefix_len) + T + kKv8Keys - 1) / kKv8Keys;
  int64_t tiles = B * most;
  if (d->prefix_len_sum > 0) tiles = std::min(tiles, (int64_t(d->prefix_len_sum) + B * T) / kKv8Keys + B);
  w->shares = 0;
  int64_t units = B;
  if (B > 0 && B <= kKv8MaxShared) {
    int64_t best = -1;
    auto look = [&](int64_t shares) {
      shares = std::max<int64_t>(1, std::min(shares, tiles));
      const int64_t each = (tiles + shares - 1) / shares;
      // (on average a request adds half a unit to the shares)
      const int64_t n = std::max(B, std::min(shares + B - 1, shares + B / 2)) * w->groups;
      const int64_t waves = (n + sm_count - 1) / sm_count;
      const int64_t cost = waves * (std::min(each, most) + kUnitTiles) + (shares > 1 ? kMergeTiles + n / kPartialsPerTile : 0);
      if (best < 0 || cost < best) {
        best = cost;
        w->shares = static_cast<int>(shares);
      }
    };
    look(1);
    for (int64_t waves = 1; waves <= 12; ++waves) {
      const int64_t n = waves * sm_count / w->groups;
      look(n - (B - 1));
      look(n - B / 2);
    }
    units = w->shares + B - 1;
  }
  // the grid's second dimension, and its CTAs in 31 bits
  if (units > 65535 || units * w->groups > INT32_MAX) return DDT_ERR_DIMS;
  w->units = static_cast<int>(units);
  // partials of split requests, and of units of several segments
  const size_t rows = size_t(T) * H, part = w->shares > 1 || most > kKv8Segment ? size_t(units) * rows : 0;
  w->pieces_off = kStatusBytes;
  w->images_off = align_up(w->pieces_off + size_t(B) * sizeof(Kv8Piece), 256);
  // Query rows are cut once a call where units share them, and where there are fewer groups than SMs, for which four CTAs
  // a group are quicker (9 nodes of 16 heads over 40 keys: 14.5 us, 16.5 by the units). Many units of their own groups cut
  // their rows beside their first gathers (1540 groups of 46 keys: 164 us in place of 194, 900 of 16 to 99 103 for 121).
  w->images = w->shares > 1 || B * w->groups <= sm_count;
  w->lse_off = w->images_off + (w->images ? size_t(B) * w->groups * kKv8Image : 0);
  w->o_off = align_up(w->lse_off + part * sizeof(float), 256);
  w->bytes = w->o_off + part * kDv * sizeof(float);
  return DDT_OK;
}

// Warps that share a row of the merge: the least power of two, up to 16, with which a row's units are read in one go,
// while there are SMs for so many (64 requests of 144 rows, few units each: 16 warps a row 243 us in all, one 117).
int merge_warps(const Kv8Layout& w, const ddt_dims* d, int sm_count) {
  const int64_t rows = int64_t(d->batch) * d->num_nodes * d->num_heads, units = w.units - d->batch + 1;  // of one request, at most
  int n = 1;
  while (n < 16 && n * 4 < units && rows * n * 2 <= int64_t(sm_count) * 64) n *= 2;
  return n;
}

int check_accept(const ddt_dims* d, int32_t vocab) {
  if (!d) return DDT_ERR_NULL;
  if (d->batch < 0 || d->batch > 65535 || d->num_nodes < 1 || d->num_nodes > kMaxNodes || vocab < 1 || vocab > kAcceptVocab)
    return DDT_ERR_DIMS;
  return DDT_OK;
}
// CTAs of a request: enough to hold a row in shared memory, and as many as cost least. A
// visit of a row takes about kVisit cycles and, with draft probabilities, 1.5 for each of a
// CTA's tokens (else one), half as much again where two CTAs meet on an SM. Requests that
// find no room wait for others' ends, and as paths differ in length that comes to 0.7 of
// the whole rounds. Graphs, 9 nodes, CTAs a request 1 / 2 / 4 / 8 / 16 in us (the rule's *):
//   8 requests of 131072 tokens                   72 / 45 / 35* (4, 8, 16)
//   64 requests of 32000         90 / 56 / 47* / 48 / 80; drawn - / 70 / 63 / 65* / 113
//   300 requests of 32000   132 / 107* / 113 / 160 / 320; drawn - / 195 / 175* / 242 / 488
//   32 requests of 131072  - / - / 64 / 57 / 60*;          drawn - / - / - / 131 / 109*
constexpr int64_t kVisit = 7000;
void accept_grid(int batch, int vocab, bool drawn, int sm_count, const AcceptClusters& clusters, AcceptParams* p) {
  int64_t best = -1;
  for (int i = 0; i < kAcceptSizes; ++i) {
    const int n = 1 << i, share = ((vocab + n - 1) / n + 63) / 64 * 64, bytes = share * accept_value_bytes(drawn);
    const int active = bytes <= kAcceptBytes ? clusters.count[i][bytes <= kAcceptBytes / 2] : 0;
    if (active < 1) continue;
    const bool meet = int64_t(std::min(batch, active)) * n > sm_count;
    const int64_t visit = 4 * kVisit + int64_t(share) * (drawn ? 3 : 2) * (meet ? 3 : 2);  // quarter cycles
    const int64_t cost = visit * std::max(10 * int64_t(active), 7 * int64_t(batch)) / active;
    if (best < 0 || cost < best) {
      best = cost;
      p->cluster = n;
      p->share = share;
    }
  }
  p->warp_share = ((p->share + 15) / 16 + 31) / 32 * 32;
}

}  // namespace
}  // namespace ddt

using namespace ddt;

extern "C" int ddtree_kv8_write(const void* rows, int64_t row_stride, const int32_t* slots, int64_t n,
                                const void* norm_weight, float eps, const float* rotation, const int32_t* position,
                                int32_t positions, int32_t interleaved, void* kv8_pool, float* kv8_scale, int64_t pool_slots,
                                void* workspace, ddt_stream_t stream) {
  if (n < 0 || n > kMaxRows || row_stride < kDqk || row_stride % 8 != 0 || pool_slots < 1 || pool_slots > kMaxRows ||
      (norm_weight && !(eps >= 1e-12f && eps <= 1.f)) || (rotation && positions < 1))
    return DDT_ERR_DIMS;
  if (n == 0) return nothing_to_do(workspace, kStatusBytes, stream);
  if (!rows || !slots || !kv8_pool || !kv8_scale || (rotation && !position)) return DDT_ERR_NULL;
  if (!aligned(rows, 16) || !aligned(norm_weight, 16) || !aligned(kv8_pool, 16) || !aligned(workspace, 256) ||
      !aligned(slots, 4) || !aligned(rotation, 4) || !aligned(position, 4) || !aligned(kv8_scale, 4))
    return DDT_ERR_ALIGN;
  const size_t pool = size_t(pool_slots) * kKv8Row, scales = size_t(pool_slots) * 4;
  const size_t in = (size_t(n - 1) * row_stride + kDqk) * 2;
  if (overlap(rows, in, kv8_pool, pool) || overlap(rows, in, kv8_scale, scales) || overlap(kv8_pool, pool, kv8_scale, scales) ||
      overlap(slots, size_t(n) * 4, kv8_pool, pool) || overlap(slots, size_t(n) * 4, kv8_scale, scales))
    return DDT_ERR_ALIAS;
  const struct { const void* p; size_t n; } more[] = {{norm_weight, size_t(kDv) * 2},
                                                      {rotation, size_t(rotation ? positions : 0) * (2 * kRopePairs) * 4},
                                                      {rotation ? position : nullptr, size_t(n) * 4}};
  for (const auto& x : more)
    if (overlap(x.p, x.n, kv8_pool, pool) || overlap(x.p, x.n, kv8_scale, scales)) return DDT_ERR_ALIAS;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != DDT_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (workspace && !clear_status(workspace, s)) return DDT_ERR_LAUNCH;
  Kv8WriteParams p = {};
  p.rows = static_cast<const uint16_t*>(rows);
  p.row_stride = row_stride;
  p.slots = slots;
  p.norm_weight = static_cast<const uint16_t*>(norm_weight);
  p.eps = eps;
  p.rotation = rotation;
  p.position = position;
  p.positions = positions;
  p.pool = static_cast<uint8_t*>(kv8_pool);
  p.scale = kv8_scale;
  p.n = n;
  p.pool_slots = pool_slots;
  p.status = static_cast<int32_t*>(workspace);
  return launch_kv8_write(p, interleaved != 0, sms, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

extern "C" int ddtree_kv8_read(const void* kv8_pool, const float* kv8_scale, const int32_t* slots, int64_t n, void* rows,
                               int64_t row_stride, int64_t pool_slots, void* workspace, ddt_stream_t stream) {
  if (n < 0 || n > kMaxRows || row_stride < kDqk || row_stride % 8 != 0 || pool_slots < 1 || pool_slots > kMaxRows)
    return DDT_ERR_DIMS;
  if (n == 0) return nothing_to_do(workspace, kStatusBytes, stream);
  if (!rows || !slots || !kv8_pool || !kv8_scale) return DDT_ERR_NULL;
  if (!aligned(rows, 16) || !aligned(kv8_pool, 16) || !aligned(workspace, 256) || !aligned(slots, 4) || !aligned(kv8_scale, 4))
    return DDT_ERR_ALIGN;
  const size_t out = (size_t(n - 1) * row_stride + kDqk) * 2;
  if (overlap(rows, out, kv8_pool, size_t(pool_slots) * kKv8Row) || overlap(rows, out, kv8_scale, size_t(pool_slots) * 4) ||
      overlap(rows, out, slots, size_t(n) * 4))
    return DDT_ERR_ALIAS;
  int sms = 0;
  const int rc = current_device(&sms);
  if (rc != DDT_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (workspace && !clear_status(workspace, s)) return DDT_ERR_LAUNCH;
  Kv8ReadParams p = {};
  p.pool = static_cast<const uint8_t*>(kv8_pool);
  p.scale = kv8_scale;
  p.slots = slots;
  p.rows = static_cast<uint16_t*>(rows);
  p.row_stride = row_stride;
  p.n = n;
  p.pool_slots = pool_slots;
  p.status = static_cast<int32_t*>(workspace);
  return launch_kv8_read(p, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

extern "C" size_t ddtree_verify_kv8_workspace_bytes(const ddt_dims* dims) {
  int sms = 0;
  Kv8Layout w;
  if (current_device(&sms) != DDT_OK || kv8_layout(dims, sms, &w) != DDT_OK) return 0;
  return w.bytes;
}

extern "C" int ddtree_verify_attn_kv8(const void* q, const void* kv8_pool, const float* kv8_scale, const int32_t* slot_idx,
                                      const int32_t* prefix_len, const int32_t* tree_parent, const int32_t* tree_slot_idx,
                                      const int32_t* tree_len, float sm_scale, void* out, float* lse, const ddt_dims* dims,
                                      void* workspace, size_t workspace_bytes, ddt_stream_t stream) {
  Kv8Layout w;
  int rc = kv8_layout(dims, 1, &w);  // the sizes, before any device query
  if (rc != DDT_OK) return rc;
  if (dims->batch == 0) return nothing_to_do(workspace, workspace_bytes, stream);
  if (!q || !kv8_pool || !kv8_scale || !prefix_len || !tree_parent || !tree_slot_idx || !out || !lse || !workspace ||
      (!slot_idx && dims->max_prefix_len > 0))
    return DDT_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv8_pool, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(kv8_scale, 4) ||
      !aligned(slot_idx, 4) || !aligned(prefix_len, 4) || !aligned(tree_parent, 4) || !aligned(tree_slot_idx, 4) ||
      !aligned(tree_len, 4) || !aligned(lse, 4))
    return DDT_ERR_ALIGN;
  int sms = 0;
  if ((rc = current_device(&sms)) != DDT_OK) return rc;
  if ((rc = kv8_layout(dims, sms, &w)) != DDT_OK) return rc;
  if (workspace_bytes < w.bytes) return DDT_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Kv8AttnParams p = {};
#ifdef DDT_TEST_HOOKS
  p.test_keep_back = g_test_keep_back;
#endif
  if (!encode_kv8_map(&p.tmap, kv8_pool, dims->pool_slots)) return DDT_ERR_LAUNCH;
  p.images = w.images ? ws + w.images_off : nullptr;
  p.q = static_cast<const uint16_t*>(q);
  p.scale_log2 = static_cast<float>(sm_scale * 1.4426950408889634);
  p.kv = static_cast<const uint8_t*>(kv8_pool);
  p.scale = kv8_scale;
  p.slot_idx = slot_idx;
  p.prefix_len = prefix_len;
  p.tree_parent = tree_parent;
  p.tree_slot_idx = tree_slot_idx;
  p.tree_len = tree_len;
  p.pool_slots = dims->pool_slots;
  p.batch = dims->batch;
  p.nodes = dims->num_nodes;
  p.heads = dims->num_heads;
  p.slot_stride = dims->slot_stride;
  p.max_prefix_len = dims->max_prefix_len;
  p.groups = w.groups;
  p.group_nodes = w.group_nodes;
  p.shares = w.shares;
  p.sms = sms;
  p.units = w.units;
  p.o_part = reinterpret_cast<float*>(ws + w.o_off);
  p.lse_part = reinterpret_cast<float*>(ws + w.lse_off);
  p.pieces = reinterpret_cast<Kv8Piece*>(ws + w.pieces_off);
  p.status = reinterpret_cast<int32_t*>(ws);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  Kv8PrepareParams k = {};
  k.q = p.q;
  k.prefix_len = prefix_len;
  k.tree_len = tree_len;
  k.images = const_cast<uint8_t*>(p.images);
  k.out = p.out;
  k.lse = lse;
  k.batch = p.batch;
  k.nodes = p.nodes;
  k.heads = p.heads;
  k.max_prefix_len = p.max_prefix_len;
  k.groups = w.groups;
  k.group_nodes = w.group_nodes;
  k.scale_log2 = p.scale_log2;
  k.status = p.status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_kv8_prepare(k, s) != cudaSuccess || launch_kv8_attn(p, s) != cudaSuccess) return DDT_ERR_LAUNCH;
  if (w.shares <= 1) return DDT_OK;  // a unit a request
  Kv8MergeParams m = {};
  m.o_part = p.o_part;
  m.lse_part = p.lse_part;
  m.pieces = p.pieces;
  m.tree_len = tree_len;
  m.out = p.out;
  m.lse = lse;
  m.batch = p.batch;
  m.nodes = p.nodes;
  m.heads = p.heads;
  m.warps = merge_warps(w, dims, sms);
  return launch_kv8_merge(m, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

extern "C" size_t ddtree_accept_workspace_bytes(const ddt_dims* dims, int32_t vocab) {
  return check_accept(dims, vocab) == DDT_OK ? kStatusBytes : 0;
}

extern "C" int ddtree_accept(const void* logits, int32_t logits_fp32, int64_t logit_stride, int32_t vocab,
                             const float* draft_prob, int64_t draft_stride, const int32_t* tokens, const int32_t* tree_parent,
                             const int32_t* tree_len, const float* uniform, const float* temperature, int32_t* path,
                             int32_t* path_len, int32_t* next_token, const ddt_dims* dims, void* workspace,
                             size_t workspace_bytes, ddt_stream_t stream) {
  int rc = check_accept(dims, vocab);
  if (rc != DDT_OK) return rc;
  if (logit_stride < vocab || (draft_prob && draft_stride < vocab)) return DDT_ERR_DIMS;
  if (dims->batch == 0) return nothing_to_do(workspace, workspace_bytes, stream);
  if (!logits || !tokens || !tree_parent || !uniform || !temperature || !path || !path_len || !next_token || !workspace)
    return DDT_ERR_NULL;
  if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(draft_prob, 4) || !aligned(tokens, 4) || !aligned(tree_parent, 4) ||
      !aligned(tree_len, 4) || !aligned(uniform, 4) || !aligned(temperature, 4) || !aligned(path, 4) || !aligned(path_len, 4) ||
      !aligned(next_token, 4) || !aligned(workspace, 256))
    return DDT_ERR_ALIGN;
  if (workspace_bytes < kStatusBytes) return DDT_ERR_WORKSPACE;
  const int64_t rows = int64_t(dims->batch) * dims->num_nodes;
  const size_t nodes = size_t(rows) * 4, reqs = size_t(dims->batch) * 4;
  const struct { const void* p; size_t n; } in[] = {
      {logits, (size_t(rows - 1) * logit_stride + vocab) * (logits_fp32 ? 4 : 2)},
      {draft_prob, draft_prob ? (size_t(rows - 1) * draft_stride + vocab) * 4 : 0},
      {tokens, nodes}, {tree_parent, nodes}, {tree_len, reqs}, {uniform, nodes}, {temperature, reqs}},
      out[] = {{path, nodes}, {path_len, reqs}, {next_token, reqs}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : in)
      if (overlap(out[i].p, out[i].n, x.p, x.n)) return DDT_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return DDT_ERR_ALIAS;
  }
  int sms = 0;
  if ((rc = current_device(&sms)) != DDT_OK) return rc;
  AcceptParams p = {};
#ifdef DDT_TEST_HOOKS
  p.test_keep_back = g_test_keep_back;
#endif
  p.logits = logits;
  p.logit_stride = logit_stride;
  p.draft_prob = draft_prob;
  p.draft_stride = draft_stride;
  p.tokens = tokens;
  p.tree_parent = tree_parent;
  p.tree_len = tree_len;
  p.uniform = uniform;
  p.temperature = temperature;
  p.batch = dims->batch;
  p.nodes = dims->num_nodes;
  p.vocab = vocab;
  AcceptClusters clusters;
  current_accept_clusters(&clusters);
  accept_grid(p.batch, vocab, draft_prob != nullptr, sms, clusters, &p);
  if (p.cluster == 0) return DDT_ERR_DEVICE;
  p.path = path;
  p.path_len = path_len;
  p.next_token = next_token;
  p.status = static_cast<int32_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.batch > 1 && !clear_status(workspace, s)) return DDT_ERR_LAUNCH;
  return launch_accept(p, !logits_fp32, s) == cudaSuccess ? DDT_OK : DDT_ERR_LAUNCH;
}

// Host-side introspection of the schedule (not part of the public header; the CPU tests
// use it, no device is needed): out = {groups of a request, shares, units}; *bytes: the workspace.
extern "C" __attribute__((visibility("default"))) int ddtree_internal_kv8_plan(const ddt_dims* dims, int sm_count, int32_t* out,
                                                                              int64_t* bytes) {
  Kv8Layout w;
  const int rc = kv8_layout(dims, sm_count, &w);
  if (rc != DDT_OK) return rc;
  out[0] = w.groups;
  out[1] = w.shares;
  out[2] = w.units;
  *bytes = static_cast<int64_t>(w.bytes);
  return DDT_OK;
}
