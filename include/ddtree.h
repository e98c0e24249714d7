/*
 * ddtree.h -- C ABI of the DDTree verify-attention library for one GB300 (sm_103a).
 *
 * Operation ("The Architecture Detective: Uncovering FlashMLA's Potential for
 * Blackwell DDTree Verification", sections "The Message in Full" and "The
 * Discovery: FlashMLA's Hidden Capabilities"; "The Art of Systematic
 * Investigation", section "Input Knowledge Required to Understand This
 * Message"): in speculative decoding with a draft tree, every tree node of a
 * request is verified in one pass.  Each node's query attends to
 *   (a) the request's whole shared prefix, read through a page_size=1 token-slot
 *       table from a KV pool whose slots may be scattered, with no causal limit
 *       among the queries, and
 *   (b) among the tree nodes, only its ancestors and itself.
 * The attention is MLA in absorbed form: one KV head whose rows are 576 bf16
 * values (512 latent + 64 rope dims, 1152 bytes per slot); scores are
 * sm_scale * q.k over all 576 dims, values are the first 512 dims of the same row.
 *
 * Conventions for every entry point:
 *   - All buffers are caller-owned device memory unless stated otherwise.  The
 *     library allocates nothing, keeps no state between calls and never
 *     synchronises the stream (except ddtree_read_device_status, which says so).
 *   - All work is enqueued on `stream`; a call returns without waiting for it.
 *   - Host-side checks return a negative DDT_ERR_* code before anything is
 *     enqueued.  Problems that only the device can see (a slot index outside the
 *     pool, a parent entry that is not a valid earlier node, a prefix length out
 *     of range) never fault: the offending key or link is left out of the
 *     attention and a bit is OR-ed into a status word in the workspace, which
 *     ddtree_read_device_status returns.  The status word is cleared at the start
 *     of every call that takes the workspace.
 *   - Device pointers must be 16-byte aligned; bf16 is IEEE bfloat16.
 */
#ifndef DDTREE_H_
#define DDTREE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DDT_API __attribute__((visibility("default")))
#else
#define DDT_API
#endif

/* Same type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* ddt_stream_t;

/* Host-side return codes. */
#define DDT_OK 0
#define DDT_ERR_NULL (-1)      /* a required pointer is NULL */
#define DDT_ERR_DIMS (-2)      /* unsupported sizes (see ddt_dims) */
#define DDT_ERR_WORKSPACE (-3) /* workspace smaller than ddtree_verify_workspace_bytes() */
#define DDT_ERR_ALIGN (-4)     /* a device pointer is not 16-byte aligned */
#define DDT_ERR_LAUNCH (-5)    /* a kernel launch or CUDA runtime call failed */
#define DDT_ERR_DEVICE (-6)    /* the current device is not an sm_103 GPU */
#define DDT_ERR_ALIAS (-7)     /* ddtree_kv_compact_check: destinations overlap or cover a live row;
                                  ddtree_kv_evict: an output overlaps an input or another output;
                                  ddtree_kv_weight: weight_out overlaps weight_in in part */

/* Device status bits (ddtree_read_device_status). */
#define DDT_STATUS_BAD_SLOT 1      /* a slot index outside [0, pool_slots): key left out */
#define DDT_STATUS_BAD_PARENT 2    /* tree_parent[b][0] != -1 or tree_parent[b][i] not in [0, i): link ignored */
#define DDT_STATUS_BAD_PREFIX 4    /* prefix_len[b] outside [0, max_prefix_len]: clamped */
#define DDT_STATUS_TIMEOUT 8       /* a bounded on-chip wait gave up; outputs are not valid */
#define DDT_STATUS_BAD_TREE_LEN 16 /* tree_len[b] outside [0, num_nodes]: clamped */
#define DDT_STATUS_BAD_NODE 32     /* a node_idx entry outside [0, num_nodes) other than -1: left out */
#define DDT_STATUS_BAD_BLOCK 64    /* a block_idx entry that is no block of the prefix, other than -1: left out */

/*
 * Sizes of one call.  Fixed by the library: D_qk = 576, D_v = 512.
 *   batch          B in [0, 65535] requests
 *   num_nodes      T in [1, 128] tree nodes per request (node 0 is the root)
 *   num_heads      H in [1, 1024] query heads (all share the single latent KV head)
 *   pool_slots     N >= 1 rows in the KV pool
 *   slot_stride    row stride (in entries) of slot_idx, >= max_prefix_len
 *   max_prefix_len upper bound on every prefix_len[b]; it sizes the workspace
 *                  and the launch.
 *   prefix_len_sum optional host-side hint: the sum of prefix_len over the
 *                  batch, or 0 if unknown.  It only steers the choice of the
 *                  key-split length (with 0 the planner assumes every request
 *                  is max_prefix_len long, which over-counts the work units of
 *                  a batch of mixed lengths and picks longer splits than
 *                  needed); results are correct for any value.  The workspace
 *                  size depends on it, so query ddtree_verify_workspace_bytes
 *                  with the same dims that the calls use.
 * The key-range split of each request depends only on these sizes, the
 * device's SM count and prefix_len[b], never on slot addresses, so results are
 * bitwise reproducible and identical for any slot layout of the same logical
 * data.
 */
typedef struct {
  int32_t batch;
  int32_t num_nodes;
  int32_t num_heads;
  int32_t slot_stride;
  int64_t pool_slots;
  int32_t max_prefix_len;
  int32_t prefix_len_sum;
} ddt_dims;

/* Bytes of workspace ddtree_verify_attn needs for these sizes on the current
 * device (0 if the sizes are unsupported).  Needs a current CUDA device. */
DDT_API size_t ddtree_verify_workspace_bytes(const ddt_dims* dims);

/*
 * Verify attention for every (request b, node t, head h).
 *
 *   q             bf16 [B, T, H, 576], contiguous (row id (b*T + t)*H + h)
 *   kv_pool       bf16 [N, 576], one latent row per slot
 *   slot_idx      int32 [B, slot_stride]: request b's prefix position j lives in
 *                 slot slot_idx[b*slot_stride + j], for j < prefix_len[b]
 *   prefix_len    int32 [B], each in [0, max_prefix_len]
 *   tree_parent   int32 [B, T]: parent[b][0] = -1, parent[b][i] in [0, i)
 *                 (nodes in topological order)
 *   tree_slot_idx int32 [B, T]: slot holding node i's own latent row
 *   sm_scale      scale applied to q.k before the softmax
 *   out           fp32 [B, T, H, 512] (written)
 *   lse           fp32 [B, T, H] (written): natural log of the softmax normaliser
 *   workspace     device scratch of >= ddtree_verify_workspace_bytes(dims) bytes,
 *                 256-byte aligned; holds the per-split partial results and the
 *                 status word.  Calls sharing a workspace must not overlap.
 *
 * The prefix part is split-KV over each request's key range, all T*H rows of a
 * request contracted together on the tensor cores; the tree part applies the
 * ancestor rule; a log-sum-exp merge combines them.  The call enqueues a
 * workspace clear, the prefix pass and the tail/merge kernel (exactly
 * ddtree_verify_prefix_phase then ddtree_verify_merge_phase; the second kernel
 * starts as a programmatic dependent of the first).  The key ranges come from
 * the sizes and the SM count: key splits of every request (all of one length,
 * or, for one request whose row tiles leave CTA pairs free, a long first split
 * with short ones behind it for the free pairs), or, for a
 * batch of 2 to 64 requests whose row tiles fit at least twice on the GPU's
 * CTA pairs, key-range groups (the requests' keys laid end to end and cut into
 * equal shares, each computed by one group of pairs).  Capturable in a CUDA
 * graph.  B = 0 enqueues nothing and returns DDT_OK.
 */
DDT_API int ddtree_verify_attn(const void* q, const void* kv_pool, const int32_t* slot_idx,
                       const int32_t* prefix_len, const int32_t* tree_parent,
                       const int32_t* tree_slot_idx, float sm_scale, float* out, float* lse,
                       const ddt_dims* dims, void* workspace, size_t workspace_bytes,
                       ddt_stream_t stream);

/*
 * The same computation as ddtree_verify_attn, always as one launch ("The Art of
 * Systematic Investigation", section "Input Knowledge Required to Understand
 * This Message", item 5, and "The Anatomy of a Kernel Investigation", section
 * "Conclusion": the verify kernel is captured in a CUDA graph; here it is a
 * single node besides the workspace clear).  A persistent grid of CTA pairs
 * works through the (request, key split, 128-row tile) units; the pair that
 * finishes the last split of a (request, row tile) merges its rows (tree tail
 * and log-sum-exp merge), counted with an atomic in the workspace: nothing ever
 * waits on another pair.  Same arguments and checks as ddtree_verify_attn, and
 * the same bits wherever ddtree_verify_attn uses key splits (this
 * launch always does; with key-range groups the partial sums are cut at other
 * keys and the results agree within rounding).  It is slower than
 * ddtree_verify_attn's two launches (the
 * merges run on the pairs that finish row tiles, not on every SM), so it is for
 * callers that want the single launch.
 */
DDT_API int ddtree_verify_attn_fused(const void* q, const void* kv_pool, const int32_t* slot_idx,
                                     const int32_t* prefix_len, const int32_t* tree_parent,
                                     const int32_t* tree_slot_idx, float sm_scale, float* out, float* lse,
                                     const ddt_dims* dims, void* workspace, size_t workspace_bytes,
                                     ddt_stream_t stream);

/*
 * Ragged trees: the same call for a batch whose requests have different node
 * counts (the pages' trees range from 9 to 65 nodes per request; "The Art of
 * Systematic Investigation", section "Input Knowledge Required to Understand
 * This Message", item 1).  Request b has tree_len[b] active nodes, 0..T-1 of
 * its [T]-strided arrays; T = dims->num_nodes is the largest count and keeps
 * every array's shape and stride.
 *   tree_len   int32 [B] device, each in [0, T] (values outside are clamped and
 *              set DDT_STATUS_BAD_TREE_LEN)
 * Rows of active nodes get exactly what ddtree_verify_attn would give that
 * request alone with T = tree_len[b]; rows of inactive nodes (t >= tree_len[b])
 * get out = 0 and lse = -inf, and their parent, slot and q entries are never
 * read.  Tiles of inactive rows skip the prefix pass.  tree_len must not be
 * NULL when B > 0 (DDT_ERR_NULL).
 */
DDT_API int ddtree_verify_attn_ragged(const void* q, const void* kv_pool, const int32_t* slot_idx,
                                      const int32_t* prefix_len, const int32_t* tree_parent,
                                      const int32_t* tree_slot_idx, const int32_t* tree_len, float sm_scale,
                                      float* out, float* lse, const ddt_dims* dims, void* workspace,
                                      size_t workspace_bytes, ddt_stream_t stream);

/*
 * The two phases of ddtree_verify_attn, for callers that schedule them
 * separately (for example to overlap the second with other work, or to time
 * each).  ddtree_verify_attn is exactly: clear the status word, then
 * ddtree_verify_prefix_phase, then ddtree_verify_merge_phase, on one stream.
 *   prefix phase: split-KV attention of every row over its prefix keys; writes
 *                 one normalised partial (o, lse) per key split into the
 *                 workspace.  Clears the status word first.
 *   merge phase:  tree tail (ancestors and self) and the log-sum-exp merge of
 *                 the tail with the prefix partials; writes out and lse.
 * Both take the same arguments and checks as ddtree_verify_attn; the merge
 * phase must follow the prefix phase of the same call on the same workspace.
 */
DDT_API int ddtree_verify_prefix_phase(const void* q, const void* kv_pool, const int32_t* slot_idx,
                               const int32_t* prefix_len, const int32_t* tree_parent,
                               const int32_t* tree_slot_idx, float sm_scale, float* out, float* lse,
                               const ddt_dims* dims, void* workspace, size_t workspace_bytes,
                               ddt_stream_t stream);
DDT_API int ddtree_verify_merge_phase(const void* q, const void* kv_pool, const int32_t* slot_idx,
                              const int32_t* prefix_len, const int32_t* tree_parent,
                              const int32_t* tree_slot_idx, float sm_scale, float* out, float* lse,
                              const ddt_dims* dims, void* workspace, size_t workspace_bytes,
                              ddt_stream_t stream);

/*
 * Sparse-index variant ("The Architecture Detective: Uncovering FlashMLA's
 * Potential for Blackwell DDTree Verification", sections "The Message in Full"
 * and "The Discovery: FlashMLA's Hidden Capabilities": the sparse attention
 * call takes a fixed-length list of key indices per query, -1 marking an
 * invalid entry; the pages set it aside for this workload because every list
 * would have to name the whole prefix).  Each tree node lists its own keys:
 *   indices   int32 [B, T, topk] device, topk = dims->max_prefix_len; node (b, t)
 *             attends, for all its H heads, to the rows kv_pool[indices[b][t][i]]
 *             with indices[b][t][i] != -1.  A slot listed twice counts twice.
 *             Other values outside [0, pool_slots) are left out and set
 *             DDT_STATUS_BAD_SLOT.  A node with no key gets out = 0, lse = -inf.
 *   q, out, lse as in ddtree_verify_attn ([B, T, H, ...]); dims->batch = B,
 *   num_nodes = T, num_heads = H, pool_slots = N, max_prefix_len = topk
 *   (slot_stride and prefix_len_sum are ignored); B * T <= 65535.
 *   workspace >= ddtree_verify_sparse_workspace_bytes(dims).
 * There is no tree part: the lists are the whole visible set.  The work is
 * the prefix pass over each node's list (the node's H heads are the rows of
 * the contraction) and the log-sum-exp merge of its key splits.
 */
DDT_API size_t ddtree_verify_sparse_workspace_bytes(const ddt_dims* dims);
DDT_API int ddtree_verify_attn_sparse(const void* q, const void* kv_pool, const int32_t* indices, float sm_scale,
                                      float* out, float* lse, const ddt_dims* dims, void* workspace,
                                      size_t workspace_bytes, ddt_stream_t stream);

/*
 * KV compaction (defragmentation) of each request's prefix rows
 * ("The Anatomy of a Kernel Investigation", section "The Reasoning Process: A
 * Deep Dive", phase 3; "The Architecture Detective", section "Defragmentation:
 * Separating Signal from Noise"):
 *   kv_dst[dst_start[b] + j] = kv_src[slot_idx[b][j]]       (bit-exact row copy)
 *   slot_idx_out[b][j]       = dst_start[b] + j
 * for j < prefix_len[b].  Entries of slot_idx_out beyond prefix_len[b] are not
 * written.  kv_src and kv_dst both have dims->pool_slots rows and may be the
 * same pool only if no destination row [dst_start[b], dst_start[b]+prefix_len[b])
 * is a source row of any request (the caller's contract; ddtree_kv_compact
 * does not check it -- ddtree_kv_compact_check below does, on the host).
 *   dst_start   int64 [B] device
 *   workspace   >= 256 bytes, 256-byte aligned (status word; bad source or
 *               destination slots set DDT_STATUS_BAD_SLOT and skip the row)
 */
DDT_API int ddtree_kv_compact(const void* kv_src, void* kv_dst, const int32_t* slot_idx,
                      const int32_t* prefix_len, const int64_t* dst_start, int32_t* slot_idx_out,
                      const ddt_dims* dims, void* workspace, ddt_stream_t stream);

/*
 * Debug validator of ddtree_kv_compact's aliasing contract, run on HOST copies
 * of the tables before a compaction ("The Architecture Detective", section
 * "Defragmentation: Separating Signal from Noise": compacting live KV in place
 * is only safe if no copy overwrites a row that is still read).  Pure host code:
 * it needs no GPU and enqueues nothing.
 *   slot_idx       int32 [B, slot_stride] host, as passed to ddtree_kv_compact
 *   prefix_len     int32 [B] host, each in [0, max_prefix_len] (else DDT_ERR_DIMS)
 *   dst_start      int64 [B] host
 *   tree_slot_idx  int32 [B, num_nodes] host, or NULL: the requests' tree rows,
 *                  which an in-place compaction must not overwrite either
 *   same_pool      nonzero when kv_dst is kv_src (in-place compaction)
 *   bad_slot       optional out: the first offending slot, or -1
 * Returns DDT_OK when every destination range [dst_start[b], +prefix_len[b])
 * lies inside the pool and the ranges are pairwise disjoint, and, for
 * same_pool, no destination row is a source slot of any request (a row that
 * is already at its destination, slot_idx[b][j] == dst_start[b] + j, is
 * allowed) or a tree slot; DDT_ERR_ALIAS otherwise.
 */
DDT_API int ddtree_kv_compact_check(const int32_t* slot_idx, const int32_t* prefix_len, const int64_t* dst_start,
                                    const int32_t* tree_slot_idx, const ddt_dims* dims, int32_t same_pool,
                                    int64_t* bad_slot);

/*
 * Verify attention without any allocation, for callers that cannot allocate
 * device memory when they run it (for example code running inside a memory
 * pool or allocator callback, or a plugin that may only use the buffers its
 * host framework hands it).  The pages have no counterpart of this entry point.
 *
 * Same arguments and results as ddtree_verify_attn, minus the workspace: the
 * scratch lives in a fixed 32 MiB device array inside the library, which every
 * GPU that loads the library holds until the process exits.  Sizes whose
 * scratch (ddtree_verify_workspace_bytes) exceeds 32 MiB return
 * DDT_ERR_WORKSPACE before anything is enqueued.  The first call on each device
 * looks up the array's device address (once, with that device current).  That
 * lookup can be the moment CUDA loads the library's device code onto the device
 * and reserves the array (modules load lazily by default), so it may allocate:
 * make the first call on each device at start-up, outside any allocator
 * callback and before any stream capture; later calls allocate nothing.  Size,
 * device and pointer checks return the same codes as ddtree_verify_attn.
 * Every call shares the one array:
 * calls whose work overlaps on the GPU (on different streams, or from several
 * threads) race and must be serialised by the caller.  The device status word
 * of these calls is not readable by the caller.
 */
DDT_API int ddtree_verify_attn_static_scratch(const void* q, const void* kv_pool, const int32_t* slot_idx,
                                              const int32_t* prefix_len, const int32_t* tree_parent,
                                              const int32_t* tree_slot_idx, float sm_scale, float* out,
                                              float* lse, const ddt_dims* dims, ddt_stream_t stream);

/*
 * Keeping a long request's cache small: accumulated attention weights of the
 * prefix keys, and eviction of the positions that weigh least.  (These entry
 * points and the block ones below take max_prefix_len up to 2^30.  Calls, and
 * replays of captured ones, that share a workspace must not overlap.)
 *
 * ddtree_kv_weight adds up what a verify call's softmax gave each prefix key:
 *   weight_out[b][j] = decay * weight_in[b][j]
 *                    + sum over the chosen nodes t and all heads h of
 *                      exp(sm_scale * q[b][t][h].k_j - lse[b][t][h]),  j < prefix_len[b]
 *   q, kv_pool, slot_idx, prefix_len as in ddtree_verify_attn
 *   lse        fp32 [B, T, H]: the verify call's; rows with lse = -inf (inactive
 *              nodes, rows without a key) and +inf add nothing, and their q is
 *              not used
 *   node_idx   int32 [B, num_sel] device, the nodes that count (the accepted
 *              path, say): -1 = none, a node listed twice counts twice, values
 *              outside [0, T) are left out and set DDT_STATUS_BAD_NODE.  NULL
 *              with num_sel = 0: every node.  num_sel <= 65535.
 *   weight_in  fp32 [B, slot_stride], not read when decay is 0 (it may then be
 *              NULL); may be weight_out, but not overlap it otherwise (DDT_ERR_ALIAS)
 *   weight_out fp32 [B, slot_stride]; entries from prefix_len[b] on are not written
 * A key whose slot is outside the pool gains nothing and sets
 * DDT_STATUS_BAD_SLOT.  Sums are in fp32 in a fixed order: the same bits on
 * every run.  workspace >= ddtree_kv_weight_workspace_bytes(dims, num_sel),
 * which needs a current CUDA device.  prefix_len_sum is not used.  The query
 * rows of the batch fit in 31 bits, B * ceil(max_prefix_len / 256) in 25 (else
 * DDT_ERR_DIMS).
 */
DDT_API size_t ddtree_kv_weight_workspace_bytes(const ddt_dims* dims, int32_t num_sel);
DDT_API int ddtree_kv_weight(const void* q, const void* kv_pool, const int32_t* slot_idx, const int32_t* prefix_len,
                             const float* lse, const int32_t* node_idx, int32_t num_sel, float sm_scale, float decay,
                             const float* weight_in, float* weight_out, const ddt_dims* dims, void* workspace,
                             size_t workspace_bytes, ddt_stream_t stream);

/*
 * Eviction: request b keeps n = clamp(keep_len[b], 0, L) of its L = prefix_len[b]
 * positions.  The first `sink` and the last `recent` positions rank before all
 * others, then the larger weight, then the lower position (NaN ranks with -inf;
 * if the budget does not hold all the protected ones, the lowest of them stay).
 *   weight, slot_idx        [B, slot_stride], as in ddtree_kv_weight
 *   keep_len                int32 [B] device
 *   slot_idx_out            int32 [B, slot_stride]: the kept positions' slots, in order
 *   weight_out              fp32 [B, slot_stride]: their weights
 *   prefix_len_out          int32 [B]: n
 *   freed_slots             int32 [B, slot_stride]: the other L - n slots, in order
 * Entries past those counts are not written; slot values are copied, not
 * checked.  The cached rows stay where they are: the new table is a valid
 * prefix for every other call, and ddtree_kv_compact can move it.  Outputs must
 * not overlap inputs or one another (DDT_ERR_ALIAS).  dims gives batch,
 * slot_stride and max_prefix_len.  workspace >= 256 bytes, 256-byte aligned.
 */
DDT_API int ddtree_kv_evict(const float* weight, const int32_t* slot_idx, const int32_t* prefix_len,
                            const int32_t* keep_len, int32_t sink, int32_t recent, int32_t* slot_idx_out,
                            float* weight_out, int32_t* prefix_len_out, int32_t* freed_slots, const ddt_dims* dims,
                            void* workspace, ddt_stream_t stream);

/*
 * Reading a long cache sparsely: 8-bit means of blocks of the prefix, the best
 * blocks of each tree node by a cheap score, and attention over them.  A block
 * is `block` (16, 32, 64 or 128) consecutive positions, the last one cut at the
 * prefix's end; N = ceil(max_prefix_len / block) is the block stride.
 *
 * ddtree_block_summary:
 *   mean of the block's rows (their sum is off by at most 2^-34 of the sum of |x|,
 *   then the mean is rounded once to fp32; where rows cancel to that degree, the
 *   result can depend on their order),
 *   scale = max |mean| * c, c the fp32 nearest to 1/127, summary = round to nearest
 *   even of mean / scale, at most 127 in size
 *   from_len  int32 [B] device or NULL: only blocks that hold a position at or
 *             after from_len[b] are computed (after a decode step: the old length)
 *   summary   bf16 [B, N, 576]: integers in [-127, 127]
 *   scale     fp32 [B, N]
 * Rows whose slot is outside the pool are left out (DDT_STATUS_BAD_SLOT); a
 * block with no row has scale 0, one with a row that is not finite has scale NaN
 * and zeros.  Other blocks' entries are not written.  workspace >= 256 bytes.
 */
DDT_API int ddtree_block_summary(const void* kv_pool, const int32_t* slot_idx, const int32_t* prefix_len,
                                 const int32_t* from_len, int32_t block, void* summary, float* scale,
                                 const ddt_dims* dims, void* workspace, ddt_stream_t stream);

/*
 * ddtree_block_select: for every node t, the topk best of request b's blocks:
 *   qs_h = max |q[b][t][h]| * c, c the fp32 nearest to 1/127,
 *   q_int = round to nearest even of q / qs, at most 127 in size
 *   score(t, j) = scale[b][j] * max over h of (qs_h * (q_int_h . summary[b][j]))
 * with both products rounded to fp32 (the integer dot product is exact).  The
 * first `first` and the last `last` blocks rank before all others, then the
 * larger score, then the lower block (NaN ranks with -inf; a head whose q is not
 * finite is left out).
 *   block_idx  int32 [B, T, topk]: the chosen blocks in ascending order, then -1
 * topk <= 2^20.  dims gives batch, num_nodes, num_heads, slot_stride and
 * max_prefix_len; B * T * H and B * N fit in 31 bits, B * ceil(N / 256) in 25.
 * workspace >= ddtree_block_select_workspace_bytes(dims, block).
 */
DDT_API size_t ddtree_block_select_workspace_bytes(const ddt_dims* dims, int32_t block);
DDT_API int ddtree_block_select(const void* q, const void* summary, const float* scale, const int32_t* prefix_len,
                                int32_t block, int32_t topk, int32_t first, int32_t last, int32_t* block_idx,
                                const ddt_dims* dims, void* workspace, size_t workspace_bytes, ddt_stream_t stream);

/*
 * ddtree_verify_attn_blocks: verify attention over each node's own blocks.  Node
 * (b, t) attends, for all its H heads, to the prefix positions of the blocks in
 * block_idx[b][t] (cut at prefix_len[b]), to its ancestors and to itself.
 *   block_idx  int32 [B, T, topk] device, in any order; -1 = none, a block listed
 *              twice counts once, other values that are no block of the prefix
 *              are left out and set DDT_STATUS_BAD_BLOCK.  topk <= 2^20.
 *   out        bf16 [B, T, H, 512] (the operand type of the product that follows)
 *   lse        fp32 [B, T, H]
 * The other arguments are ddtree_verify_attn's, and with every block listed it
 * attends to the same keys (there out is fp32).  Nodes are processed in groups of
 * up to 64 (node, head) rows over the union of their lists; scores and sums are
 * fp32, softmax weights keep 16 bits, and out is rounded to bf16 once.  A
 * non-finite key row reaches only the nodes that list its block.  Results are the
 * same bits on every run.
 * workspace >= ddtree_verify_blocks_workspace_bytes(dims, block, topk), which
 * needs a current CUDA device.
 */
DDT_API size_t ddtree_verify_blocks_workspace_bytes(const ddt_dims* dims, int32_t block, int32_t topk);
DDT_API int ddtree_verify_attn_blocks(const void* q, const void* kv_pool, const int32_t* slot_idx,
                                      const int32_t* prefix_len, const int32_t* tree_parent,
                                      const int32_t* tree_slot_idx, const int32_t* block_idx, int32_t block,
                                      int32_t topk, float sm_scale, void* out, float* lse, const ddt_dims* dims,
                                      void* workspace, size_t workspace_bytes, ddt_stream_t stream);

/* Waits for `stream`, then copies the status word of the last call that used
 * `workspace` to *host_status.  Returns DDT_OK or DDT_ERR_*.  The kernels write
 * the word asynchronously on the stream the verify call was enqueued on, so
 * the read waits for that stream alone (not the whole device): work on other
 * streams keeps running. */
DDT_API int ddtree_read_device_status(const void* workspace, int32_t* host_status, ddt_stream_t stream);

/* Static text for a DDT_ERR_* return code. */
DDT_API const char* ddtree_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* DDTREE_H_ */
