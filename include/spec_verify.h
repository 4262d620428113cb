/*
 * spec_verify.h -- C ABI of the draft-tree verification step (tree attention, ratio-test
 * verification with residual resampling, KV compaction) for one GB300 (sm_103a) GPU.
 *
 * Sources (page title, section):
 *   [TREE]  "投机推理算法的常见优化手段" (cnblogs zrq96), 草稿树的验证——树形掩码: flattened tree, the
 *           ancestor mask (a token sees itself and its ancestors), the forward call
 *           logits = llm.forward(draft_tree, tree_mask, position_ids, kvcache) and tree
 *           verification level by level.
 *   [RATIO] "推测解码 2026" (guijiagi.com), 数学基础：拒绝采样: accept with min(1, p/q), resample from
 *           relu(p - q) normalised, discard later candidates; 工程实践中的考量 / KV Cache管理:
 *           roll back the K/V of rejected candidates.
 *   [CSDN]  "【模型后训练与深度推理】9 推理加速：推测解码与级联推理", section 7.1 (alpha = min(1, p/q),
 *           residual norm(max(0, p - q)), output distributed as p), section 5 (interface: prompt,
 *           draft length, probability tensors, a boolean accept mask, accepted tokens).
 *   [SURV]  "万字综述 10+ 种 LLM 投机采样推理加速方案" (m.haoling.cc), 5.2 (tree-based parallel
 *           decoding through an attention mask), 4.3 (argmax sampling, temp = 0), 12.4.3
 *           (PagedAttention / FlashDecoding as the framework features to fit).
 *
 * Conventions shared by every entry point:
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise; the caller allocates
 *     and owns all buffers, including workspaces.  The library never allocates, frees or
 *     synchronises; each call enqueues kernels on `stream` and returns.
 *   - The return code covers argument validation and launch errors only.  Errors in DEVICE DATA
 *     (a bad parent index, a token id >= V, a block id out of range, ...) are OR-ed as SPEC_REQ_*
 *     bits into the caller's per-request int32 `req_status[B]`; such a request produces
 *     out_len = 0 / n_acc = -1 and is rolled back by spec_kv_compact.  No kernel traps.
 *   - Nodes of all requests are packed: request r owns global nodes
 *     node_offset[r] .. node_offset[r+1]-1 (CSR, node_offset has B+1 entries); node 0 of a request
 *     is its root (the last committed token, whose K/V is not cached yet); `parent` holds LOCAL
 *     indices with parent[root] = -1 and 0 <= parent[i] < i (BFS / topological order).
 *   - T_r = node_offset[r+1] - node_offset[r] includes the root; T_max (host) bounds every T_r and
 *     may not exceed SPEC_MAX_TREE (256).
 *   - Row-major buffers whose rows are read with 16-byte vector loads (logits, probabilities,
 *     Q, K/V, O) must start on 16-byte boundaries and have 16-byte-multiple row strides.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (pass 0 for the legacy default stream). */
typedef struct CUstream_st* spec_stream_t;

typedef enum {
  SPEC_OK = 0,
  SPEC_ERR_INVALID_ARG = 1,    /* null / misaligned pointer, bad size or stride, tau < 0, ... */
  SPEC_ERR_UNSUPPORTED = 2,    /* a valid but unimplemented shape (e.g. bf16 head_dim != 128) */
  SPEC_ERR_CUDA = 3,           /* a CUDA launch / driver error (see spec_last_cuda_error) */
  SPEC_ERR_TIMEOUT = 4,        /* reserved for host-side waits; device waits report via bits */
  SPEC_ERR_BAD_INPUT_DATA = 5  /* reserved: data errors are reported per request, see below */
} spec_status_t;

/* SPEC_E4M3 (8-bit floats: 4 exponent bits, 3 mantissa bits, largest 448, no infinities) names
 * the element type of an 8-bit cache in spec_kv_fork; the 8-bit cache's own entry points imply it. */
typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1, SPEC_E4M3 = 2 } spec_dtype_t;
typedef enum { SPEC_DRAFT_LOGITS = 0, SPEC_DRAFT_PROBS = 1 } spec_draft_kind_t;
typedef enum {
  SPEC_SIBLING_RESIDUAL = 0,   /* default: child k is tested against the k-fold residual */
  SPEC_SIBLING_INDEPENDENT = 1, /* every sibling tested against p; resample from max(0, p - q) */
  SPEC_SIBLING_MULTI_DRAFT = 2  /* siblings from different draft models, each with its own q:
                                   draft_row[c] names the row CHILD c was drawn from */
} spec_sibling_rule_t;

/* Per-request data-error bits OR-ed into req_status[r]. */
#define SPEC_REQ_BAD_PARENT    1   /* parent[0] != -1 or parent[i] not in [0, i) */
#define SPEC_REQ_BAD_SIZE      2   /* T_r < 1, T_r > T_max, or node_offset not monotone / > N */
#define SPEC_REQ_BAD_TOKEN     4   /* a draft token id outside [0, V) */
#define SPEC_REQ_BAD_DRAFT_ROW 8   /* tau > 0 and a draft row read is outside [0, R): a node
                                      with children's, or under the multi-draft rule a drafted
                                      node's own */
#define SPEC_REQ_BAD_DEPTH     16  /* a root-to-node path longer than max_path */
#define SPEC_REQ_BAD_BLOCK     32  /* a needed block_table entry outside [0, num_blocks) */
#define SPEC_REQ_TIMEOUT       64  /* a bounded device-side wait gave up (the result is invalid) */

#define SPEC_MAX_TREE 256

/* ------------------------------------------------------------------------------------------
 * spec_tree_build  [TREE]
 * For each request: depth[i] = number of proper ancestors of node i (root 0);
 * pos_id[i] = prefix_len[r] + depth[i] (position ids adapted to the tree);
 * anc_mask row i (ceil(T_max/32) uint32 words, bit j of word j/32 = LOCAL node j) has bit j set
 * iff j == i or j is an ancestor of i -- one row of the page's mask table;
 * is_internal[i] = 1 iff node i has at least one child.
 *   parent [N] int32, node_offset [B+1] int32, prefix_len [B] int32: inputs (device).
 *   depth, pos_id [N] int32; anc_mask [N][ceil(T_max/32)] uint32; is_internal [N] uint8: outputs.
 *   req_status [B] int32: output; this call (re)initialises it (0 or a SPEC_REQ_* bit) and the
 *   later calls of the round OR their bits into it.
 * Requests with a data error get their outputs set to -1 / 0 and a SPEC_REQ_BAD_* bit.
 * Errors: SPEC_ERR_INVALID_ARG for null or inconsistent arguments (B < 1, N < 0, T_max outside
 * [1, 256]); SPEC_ERR_CUDA on a launch failure.
 * ------------------------------------------------------------------------------------------ */
spec_status_t spec_tree_build(const int32_t* parent, const int32_t* node_offset,
                              const int32_t* prefix_len, int32_t B, int32_t N, int32_t T_max,
                              int32_t* depth, int32_t* pos_id, uint32_t* anc_mask,
                              uint8_t* is_internal, int32_t* req_status, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_tree_rope_kv_write  [TREE]
 * The step before tree attention: rotary position embedding (RoFormer, Su et al. 2021, section
 * 3.2 -- the pages say only that position ids must follow the tree) of every tree node's q and
 * new k at its position id, and the node's K/V stored where spec_tree_attention reads it.
 * For node n = node_offset[r] + i at position m = pos_id[n] (prefix_len[r] + depth, from
 * spec_tree_build), pair j < rotary_dim/2 of each head row turns by m * base^(-2j/rotary_dim):
 *   (a, b) -> (a cos - b sin, a sin + b cos),
 * pair j being components (2j, 2j+1) when `interleaved` != 0 and (j, j + rotary_dim/2)
 * otherwise (the half-split layout of LLaMA-family checkpoints); components past rotary_dim are
 * copied unchanged.  Rotated q goes to q_out; rotated k and unchanged v go to logical slot
 * prefix_len[r] + i of the paged cache (row slot % block_size of block
 * block_table[r][slot / block_size]).  Arithmetic: angle formed and reduced modulo 2 pi in fp64,
 * rotation in fp32, one rounding to `dtype`.
 * Layouts (element type `dtype`, contiguous, 16-byte aligned): q_in, q_out [N][H_q][head_dim]
 * (q_out == q_in rotates in place; partial overlap is not allowed); k_new, v_new
 * [N][H_kv][head_dim]; k_cache, v_cache [num_blocks][H_kv][block_size][head_dim] (one layer);
 * block_table [B][max_blocks_per_req], prefix_len [B], node_offset [B+1], pos_id [N] int32.
 * Data errors: nodes of a request with req_status[r] != 0 (e.g. from spec_tree_build) are not
 * touched; a request any of whose tree slots maps outside [0, num_blocks) gets
 * SPEC_REQ_BAD_BLOCK and none of its nodes is written.
 * Errors: SPEC_ERR_INVALID_ARG (null / misaligned pointers, bad sizes, rotary_dim odd or outside
 * [2, head_dim], base not positive and finite); SPEC_ERR_UNSUPPORTED when a rotated pair would
 * straddle 16-byte vectors (half-split: rotary_dim/2 must be a multiple of 8 bf16 / 4 fp32
 * elements; interleaved: rotary_dim a multiple of 8 / 4) or rotary_dim > 256; SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;
  int32_t B, N, H_q, H_kv, head_dim, rotary_dim;
  int32_t interleaved;         /* 0: pairs (j, j + rotary_dim/2); 1: pairs (2j, 2j+1) */
  int32_t block_size, num_blocks, max_blocks_per_req;
  double base;                 /* e.g. 10000 (LLaMA-2), 500000 (LLaMA-3), 1e6 (Qwen2) */
  const void* q_in;
  void* q_out;
  const void* k_new;
  const void* v_new;
  void* k_cache;
  void* v_cache;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* node_offset;
  const int32_t* pos_id;
  int32_t* req_status;
} spec_rope_params;

spec_status_t spec_tree_rope_kv_write(const spec_rope_params* p, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_tree_build_rope_kv_write  [TREE]
 * spec_tree_build and spec_tree_rope_kv_write in one launch: the tree outputs of
 * spec_tree_build (same arguments, same results), then -- for every request the tree build
 * accepts -- the rotary embedding and K/V slot write of spec_tree_rope_kv_write at
 * pos = prefix_len + depth, described by `rope` (host pointer; its B and N must equal this
 * call's, and its node_offset, prefix_len, pos_id and req_status must be NULL or this call's
 * buffers).  req_status[r] ends as spec_tree_build's bits, or SPEC_REQ_BAD_BLOCK for a valid
 * tree with a slot outside the pool (nothing of that request is then written to q_out or the
 * cache); the results equal the two calls made in sequence.
 * Errors: those of the two calls.
 * ------------------------------------------------------------------------------------------ */
spec_status_t spec_tree_build_rope_kv_write(const int32_t* parent, const int32_t* node_offset,
                                            const int32_t* prefix_len, int32_t B, int32_t N,
                                            int32_t T_max, int32_t* depth, int32_t* pos_id,
                                            uint32_t* anc_mask, uint8_t* is_internal,
                                            int32_t* req_status, const spec_rope_params* rope,
                                            spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_tree_attention  [TREE], [SURV 5.2, 12.4.3]
 * O[n][h] = sum_j softmax_j(scale * q[n][h] . k_j) v_j over the logical KV slots
 *   j in {0 .. P_r-1} U {P_r + a : a == i or a is an ancestor of i}
 * for node n = node_offset[r] + i.  The caller has written node a's K/V into logical slot
 * P_r + a before the call.  Logical slot s of request r is row s % block_size of physical block
 * block_table[r][s / block_size].  Query head h reads KV head h / (H_q / H_kv).
 * Layouts (element type `dtype`, contiguous, 16-byte aligned):
 *   q [N][H_q][head_dim]; k_cache, v_cache [num_blocks][H_kv][block_size][head_dim] (one layer);
 *   o [N][H_q][head_dim]; lse [N][H_q] fp32 (natural log of the softmax denominator of the
 *   scaled scores) or NULL; block_table [B][max_blocks_per_req] int32; prefix_len [B];
 *   node_offset [B+1]; anc_mask from spec_tree_build; req_status [B] in/out.
 * Paths: dtype BF16 runs on the tcgen05 tensor cores (TMA-staged paged tiles, scores and output
 * accumulated in TMEM) and requires head_dim == 128, block_size == 16 and
 * H_q / H_kv in {1, 2, 4, 8, 16}; dtype F32 runs a CUDA-core kernel (head_dim <= 128,
 * multiple of 4).  Long KV ranges are split across CTAs and merged by log-sum-exp in
 * `workspace` (spec_attention_workspace_size bytes, 256-byte aligned, caller-owned, contents
 * need not be initialised).  scale <= 0 selects 1/sqrt(head_dim).
 * Errors: SPEC_ERR_INVALID_ARG (null / misaligned pointers, inconsistent sizes, too-small
 * workspace), SPEC_ERR_UNSUPPORTED (a shape outside the paths above), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;
  int32_t B, N, T_max;
  int32_t H_q, H_kv, head_dim;
  int32_t block_size;          /* tokens per KV block */
  int32_t num_blocks;          /* physical blocks in the pool (bounds check) */
  int32_t max_blocks_per_req;  /* row stride of block_table */
  float scale;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* node_offset;
  const uint32_t* anc_mask;
  void* o;
  float* lse;
  int32_t* req_status;
} spec_attn_params;

size_t spec_attention_workspace_size(const spec_attn_params* p);
spec_status_t spec_tree_attention(const spec_attn_params* p, void* workspace, size_t ws_bytes,
                                  spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_verify  [RATIO], [CSDN 7.1, 7.2, 5], [TREE], [SURV 4.3]
 * p_i = softmax(target[i] / tau), q_i = softmax(draft[draft_row[i]] / tau) (draft logits) or the
 * given row (draft probabilities).  Walk from the root; at node i test its children c in
 * increasing index with u_acc = uniforms[c][0]:
 *   SIBLING_RESIDUAL: after k rejected siblings the target is R_k = max(0, p_i - C_k q_i),
 *     C_0 = 0, N_k = sum R_k, C_{k+1} = C_k + N_k; accept iff u_acc < R_k(tok)/(N_k q_i(tok))
 *     (k = 0: p/q, the pages' rule);
 *   SIBLING_INDEPENDENT: accept iff u_acc < p_i(tok)/q_i(tok) for every sibling;
 *   SIBLING_MULTI_DRAFT ([SURV 5.1] a group of small models predicting together; [TREE]
 *     merge-based trees from k small models): child c carries its own q_c = softmax(
 *     draft[draft_row[c]] / tau) -- draft_row is indexed by the CHILD, and every non-root node
 *     needs one (tau > 0).  The running target starts as R_0 = p_i, N_0 = 1; child j is
 *     accepted iff u_acc < R_{j-1}(tok)/(N_{j-1} q_c(tok)), and a rejection gives
 *     R_j = max(0, R_{j-1} - N_{j-1} q_c), N_j = sum R_j (the pages' norm(max(0, r - q))
 *     applied sibling after sibling); all rejected: the final token is drawn from R_k.  Needs
 *     two fp32 rows of ceil(V/64)*64 floats per request in the workspace (included in
 *     spec_verify_workspace_size); spec_verify_noalloc refuses it (SPEC_ERR_UNSUPPORTED);
 *   tau == 0: accept iff tok == argmax p_i (lowest id on ties).
 * On acceptance descend to c.  The walk stops at a leaf (the final token is a bonus draw from
 * p_leaf with u_samp = uniforms[leaf][1]) or when every child is rejected (the final token is
 * drawn from the normalised residual with u_samp of that node; from p if the residual mass is
 * 0); tau == 0 takes argmax p instead.  Draws use the inverse CDF over ascending token id: the
 * smallest x with sum_{y<=x} w(y) > u * sum_y w(y).  Randomness is never generated inside.
 * Outputs per request r (row stride max_path): path[r][0..n_acc] = accepted local node ids
 * (root first), out_tokens[r][0..n_acc] = accepted draft tokens then the final token,
 * out_len[r] = n_acc + 1, rejections[r] = rejected children on the walk; unused entries -1.
 * Layouts: target [N][target_ld] (logits_dtype), draft [R][draft_ld] (logits_dtype for
 * logits, fp32 for probabilities), rows 16-byte aligned; draft_row, tokens, parent, depth [N]
 * int32 (depth from spec_tree_build); is_internal [N] uint8; uniforms [N][2] fp32.
 * workspace: spec_verify_workspace_size bytes (256-byte aligned, caller-owned).
 * Errors: SPEC_ERR_INVALID_ARG (null / misaligned pointers, V < 1, ld < V, tau < 0 or not
 * finite, max_path < 1, small workspace), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t logits_dtype;
  spec_draft_kind_t draft_kind;
  spec_sibling_rule_t sibling_rule;
  int32_t B, N, R, V;
  int64_t target_ld, draft_ld;   /* row strides in elements */
  int32_t T_max, max_path;
  float tau;
  const void* target;
  const void* draft;
  const int32_t* draft_row;
  const int32_t* tokens;
  const int32_t* parent;
  const int32_t* node_offset;
  const int32_t* depth;
  const uint8_t* is_internal;
  const float* uniforms;
  int32_t* req_status;
  int32_t* out_tokens;
  int32_t* out_len;
  int32_t* path;
  int32_t* n_acc;
  int32_t* rejections;           /* may be NULL */
  int32_t verify_path;           /* SPEC_VERIFY_PATH_AUTO (0, the default), _SPLIT or _WALK */
} spec_verify_params;

/* verify_path -- no counterpart on the pages: which of the library's forms of the same
 * computation this call launches.
 *   SPEC_VERIFY_PATH_AUTO (0, what a zero-initialised struct asks for): calls with the residual
 *     or independent sibling rule (or tau == 0), T_max <= 32 and
 *     T_max * S_t + (T_max - 1) * S_d <= 200 KiB run as one cluster launch (up to 8 CTAs per
 *     request, each holding its share of the request's rows in shared memory), with
 *     S_t / S_d = ceil(ceil(V / 8) / 8) * 8 * the target / draft element size (S_d = 0 at
 *     tau == 0); the others with those rules and V >= 65536 run the walk form, every other call
 *     the two-launch form;
 *   SPEC_VERIFY_PATH_SPLIT: always the two-launch form (a row statistics kernel for every
 *     internal node's rows, then a walk kernel with a cluster of CTAs per request);
 *   SPEC_VERIFY_PATH_WALK: the walk kernel alone, which forms the statistics (max and sum, or
 *     argmax at tau == 0) of the nodes it visits, one pass over their two rows each, instead of
 *     reading every internal node's rows first (the multi-draft rule always runs the two-launch
 *     form).
 * All forms give the same outputs except where fp32 rounding of the vocabulary sums decides:
 * a ratio test or a draw whose uniform lies within about 1e-6 of its boundary.  The choice is
 * per call: the library keeps no process-wide setting.  Any other value: SPEC_ERR_INVALID_ARG. */
#define SPEC_VERIFY_PATH_AUTO  0
#define SPEC_VERIFY_PATH_SPLIT 1
#define SPEC_VERIFY_PATH_WALK  2

size_t spec_verify_workspace_size(const spec_verify_params* p);
spec_status_t spec_verify(const spec_verify_params* p, void* workspace, size_t ws_bytes,
                          spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_verify_noalloc -- no counterpart on the pages; an addition for callers that may not
 * allocate device memory (an engine that reserves its whole memory budget up front and forbids
 * allocation while serving, or a plugin that is handed only tensors and a stream).
 * Same inputs, outputs and results as spec_verify, but the workspace is a fixed array in device
 * memory that belongs to this library (every GPU that loads the library keeps it until the
 * process exits), so the caller passes none and nothing is allocated.
 * Limits: N <= 32768 tree nodes and R <= 32768 draft rows per call; larger batches return
 * SPEC_ERR_UNSUPPORTED (use spec_verify with a caller-owned workspace instead).
 * The first call on each device looks up the array's device address with that device current;
 * make that first call before any stream capture.  Later calls look it up again unless their
 * stream is being captured, so a device reset between calls is safe.  All calls share the one
 * array: calls whose kernels overlap on the GPU (other streams, other host threads on the same
 * device) race.  The multi-draft sibling rule with tau > 0 is refused (SPEC_ERR_UNSUPPORTED).
 * Errors: as spec_verify, plus SPEC_ERR_UNSUPPORTED for sizes beyond the limits above and
 * SPEC_ERR_CUDA if the address lookup fails.
 * ------------------------------------------------------------------------------------------ */
spec_status_t spec_verify_noalloc(const spec_verify_params* p, spec_stream_t stream);


/* ------------------------------------------------------------------------------------------
 * spec_kv_compact  [RATIO: KV Cache管理], [CSDN 4]
 * Commits the accepted path and rolls back the rest, in place, for every layer and KV head,
 * K and V: new[P_r + d] = old[P_r + path[r][d]] for d = 0 .. n_acc[r] (gather semantics: every
 * source is read as it was before the call), i.e. the cache sequential decoding of the accepted
 * path would hold.  new_kv_len[r] = P_r + n_acc[r] + 1 (the final token has no K/V yet);
 * blocks_in_use[r] = ceil(new_kv_len / block_size); slot_map[r][d] = (src, dst) logical slots,
 * (-1, -1) past n_acc.  A request with req_status != 0 or n_acc < 0 is rolled back entirely
 * (new_kv_len = P_r, nothing copied).  Slots past new_kv_len are released, not cleared.
 * Layouts: k_cache, v_cache point at layer 0 of [num_layers] x [num_blocks][H_kv][block_size]
 * [head_dim] with `layer_stride` elements between layers; head_dim * element size must be a
 * multiple of 16 bytes.  path [B][max_path], n_acc [B] as written by spec_verify;
 * slot_map [B][max_path][2], new_kv_len [B], blocks_in_use [B] int32 outputs.
 * Errors: SPEC_ERR_INVALID_ARG, SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;
  int32_t B, H_kv, head_dim, block_size, num_blocks, max_blocks_per_req, num_layers, max_path;
  int64_t layer_stride;
  void* k_cache;
  void* v_cache;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* path;
  const int32_t* n_acc;
  int32_t* req_status;
  int32_t* new_kv_len;
  int32_t* slot_map;
  int32_t* blocks_in_use;
} spec_compact_params;

spec_status_t spec_kv_compact(const spec_compact_params* p, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_verify_compact -- spec_verify followed by spec_kv_compact, in one call: same inputs,
 * outputs and results as the two calls in that order.  When the verification takes its
 * one-launch form (see verify_path above) the compaction runs inside that launch (one
 * kernel for both); otherwise spec_kv_compact is launched after it.  The compaction reads the
 * verification's own results, so c->path, c->n_acc, c->req_status must be v->path, v->n_acc,
 * v->req_status, with c->B == v->B and c->max_path == v->max_path.
 * Errors: as spec_verify and spec_kv_compact, plus SPEC_ERR_INVALID_ARG when c is NULL or does
 * not match v as above.
 * ------------------------------------------------------------------------------------------ */
spec_status_t spec_verify_compact(const spec_verify_params* v, const spec_compact_params* c,
                                  void* workspace, size_t ws_bytes, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Building the draft tree on the device  [TREE 草稿树的生成, 动态草稿长度]
 * EAGLE-2 expands, level by level, only the K most probable leaves of the newest level (a
 * leaf's score is the sum of the draft log-probabilities along its path, log q =
 * log_softmax(draft_row / tau)[token]); each expansion adds the K most probable tokens of the
 * expanded node's draft row.  ECHO then keeps a batch-wide budget of K_max tokens: every root
 * and the K_max - B best non-root candidates of the batch.  The draft model's forward, which
 * turns the chosen candidates into draft rows, is the caller's.
 * Candidate pool (caller-owned device arrays, request r's candidates at [r * cap, r * cap +
 * count[r])): parent (candidate index, -1 for the root), token, depth, score (fp32), row (the
 * draft row its expansion produced, -1 if never), count.  cap <= 256.
 * Ordering everywhere: by score (or log-probability) descending, ties to the lower candidate
 * index / token id, then (ECHO) the lower request.  Selections compare the fp32 scores exactly.
 * A drafting round: spec_draft_init; for level = 1 .. depth: spec_draft_expand_select, the
 * caller's draft forward for the listed candidates, spec_draft_topk_append; then
 * spec_echo_select_pack, whose outputs feed spec_tree_build / spec_verify (draft_row indexes
 * the rows the caller produced, numbered row_base + r * K + j by the append calls).
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int32_t B, cap;
  int32_t* parent;   /* [B][cap] */
  int32_t* token;    /* [B][cap] */
  int32_t* depth;    /* [B][cap] */
  float* score;      /* [B][cap] */
  int32_t* row;      /* [B][cap] */
  int32_t* count;    /* [B] */
} spec_draft_pool;

/* Pool entry 0 of request r = the root (root_tokens[r]), count = 1. */
spec_status_t spec_draft_init(const spec_draft_pool* pool, const int32_t* root_tokens,
                              spec_stream_t stream);

/* The candidates to expand at `level` (1: the root; else the K best of depth level - 1), in
 * increasing candidate index: expand[r][j], j < K, -1 past the chosen ones.  Grows count[r] by
 * K per chosen candidate; if the pool cannot hold that many, fewer are chosen and req_status[r]
 * (may be NULL) gets SPEC_REQ_BAD_SIZE.  1 <= K <= 16. */
spec_status_t spec_draft_expand_select(const spec_draft_pool* pool, int32_t level, int32_t K,
                                       int32_t* expand, int32_t* req_status,
                                       spec_stream_t stream);

/* For every expand[r][j] >= 0: the K most probable tokens of draft row r * K + j of `rows`
 * ([B * K][ld], dtype F32 / BF16 logits, 16-byte aligned rows, V <= ld), log q =
 * x / tau - logsumexp(row / tau) (one streaming read of the row), appended as the candidate's
 * children in that order with score = its score + log q, depth = level; the candidate's row
 * becomes row_base + r * K + j.  Call after spec_draft_expand_select of the same level.
 * req_status (may be NULL) gets SPEC_REQ_TIMEOUT if the launch's bounded wait ran out (only
 * under the testing hook below); that expansion's children then carry token -1 and score -inf. */
spec_status_t spec_draft_topk_append(const spec_draft_pool* pool, int32_t level, int32_t K,
                                     const int32_t* expand, spec_dtype_t dtype, const void* rows,
                                     int64_t ld, int32_t V, float tau, int32_t row_base,
                                     int32_t* req_status, spec_stream_t stream);

/* Testing only: with chunk >= 0, the following spec_draft_topk_append launches on the current
 * device wait (bounded, about a second) for a device flag that nothing sets, so they run out
 * their wait and report SPEC_REQ_TIMEOUT for those requests, as a lost read would, with
 * children of token -1 and score -inf; -1 restores normal operation.  Synchronous (a
 * host-to-device symbol copy). */
spec_status_t spec_debug_draft_copy_stall(int32_t chunk);

/* ECHO selection and packing: node_offset [B+1]; parent (local, -1 for roots), tokens, depth,
 * draft_row (the node's row if one of its children was kept, else -1) and source (candidate
 * index, may be NULL), each with room for min(K_max, B * cap) entries; N = node_offset[B].
 * Kept candidates stay in candidate order (parents first), so the output is a valid tree in
 * the layout spec_tree_build reads.  workspace: spec_echo_workspace_size(B, cap) bytes,
 * 256-byte aligned. */
size_t spec_echo_workspace_size(int32_t B, int32_t cap);
spec_status_t spec_echo_select_pack(const spec_draft_pool* pool, int32_t K_max,
                                    int32_t* node_offset, int32_t* parent, int32_t* tokens,
                                    int32_t* depth, int32_t* draft_row, int32_t* source,
                                    void* workspace, size_t ws_bytes, spec_stream_t stream);

/* ==========================================================================================
 * The K/V cache in 8 bits -- no counterpart on the pages beyond [SURV 12.4.3] (paged caches).
 * A cache of e4m3 codes [num_blocks][H_kv][block_size][head_dim] (one byte each, 16-byte aligned)
 * with one fp32 scale for each (block, KV head) in [num_blocks][H_kv], K and V apart:
 *   value = code * scale.
 * Scales are finite and >= 0.  spec_kv8_append writes powers of two in [2^-100, 2^119], 2^-100 for
 * rows of zeros; another writer may use any scale there or 0 (the attention reads a V scale below
 * 2^-100 as 2^-100).
 * A block that receives rows belongs to one request (pages shared by a fork are only read).
 * head_dim is a multiple of 16, at most 256.  Round by round: spec_tree_build, rotary embedding,
 * spec_kv8_append of the tree's rows at slots prefix_len .., spec_tree_attention_kv8,
 * spec_verify, spec_kv8_compact.
 * ========================================================================================== */

/* ------------------------------------------------------------------------------------------
 * spec_kv8_append
 * Quantises new K/V rows into the pages: row row_offset[r] + i of k_new / v_new goes to logical
 * slot start[r] + i of request r, i < row_offset[r+1] - row_offset[r] (any length: one token, a
 * tree, a prompt).  For each block, head and cache written, with a = the largest finite |x| of
 * its new rows and `need` = the smallest power of two s with a <= 448 s, clamped to
 * [2^-100, 2^119]:
 *   a block that already holds rows before start[r]: s = max(old scale, need); if s > old, its
 *     earlier rows become e4m3(code * (old / s)) (exact for powers of two except for codes that
 *     leave e4m3's normal range);
 *   any other block: s = need;
 *   new rows: e4m3(x / s), to nearest even; |x / s| > 448 and infinities saturate, NaN stays NaN.
 * Rows of the block after the appended ones keep their codes (their values, if any, are stale).
 *   k_new, v_new: [N][H_kv][head_dim] of `dtype`, token n at n * k_ld (v_ld) elements (>= H_kv *
 *   head_dim, 16-byte multiples), so that slices of a fused projection need no copy; rows from
 *   row_offset[B] on are ignored.  start [B], row_offset [B+1], block_table
 *   [B][max_blocks_per_req], req_status [B] int32.
 * Data errors: a request with other req_status bits than SPEC_REQ_BAD_BLOCK is not touched.  A
 * request, with rows or without, gets SPEC_REQ_BAD_SIZE and nothing is written for it if its start
 * is negative, its slots pass 2^31 - 1, or its row_offset pair is negative, goes backwards, passes N
 * or begins below an offset of an earlier request (so with row_offset 0, 5, 3, 8 the second and the
 * third are refused).  N = 0 launches nothing and reports nothing.
 * Rows whose page is beyond the table row or outside [0, num_blocks) are not written and give
 * SPEC_REQ_BAD_BLOCK.
 * Errors: SPEC_ERR_INVALID_ARG (null / misaligned pointers, bad sizes or strides),
 * SPEC_ERR_UNSUPPORTED (head_dim not a multiple of 16 or above 256, block_size above 1024, more
 * than 2^31 - 1 rows of pages), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;          /* of k_new and v_new */
  int32_t B, N, H_kv, head_dim, block_size, num_blocks, max_blocks_per_req;
  int64_t k_ld, v_ld;          /* elements between tokens */
  const void* k_new;
  const void* v_new;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  const int32_t* start;
  const int32_t* row_offset;
  int32_t* req_status;
} spec_kv8_append_params;

spec_status_t spec_kv8_append(const spec_kv8_append_params* p, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_tree_attention_kv8
 * spec_tree_attention over an 8-bit cache: the same visibility (the prefix, ancestors and the
 * node itself; a tree of one node is plain decoding), K = k code * k_scale, V likewise.  A row
 * that sees no key (an empty mask row and no prefix) gets O = 0 and LSE = -infinity.  q and o
 * have `dtype`, q holds no infinities; scores, softmax statistics and the output are accumulated in
 * fp32.  A NaN (in q, in a code) makes the rows that see it NaN and no others: O and LSE for one in q
 * or K; O alone for one in V, its column at least.
 * On the tensor cores a bf16 q enters the e4m3 products as two pieces, exact to 2^-18 of its row's
 * largest element.  A weight (times its slot's V scale) is kept to 2^-9 of itself or 2^-30 of the
 * row's largest, whichever is more (2^-11 of itself in units of more than 16 query rows).  In these
 * longer units a key whose page's V scale is 2^-s of the largest of its request and head is left out
 * of the softmax's sum where its weight is below 2^(s - 126) of the row's largest: of pages of zeros
 * beside V scales up to 2^2, below 2^-24.
 * Every H_q / H_kv ratio, block_size and head_dim (multiple of 16, <= 256) is accepted; BF16
 * with head_dim 128, block_size 16, 32, 64 or 128 and H_q / H_kv <= 128 runs on the tcgen05
 * tensor cores, everything else on a CUDA-core kernel.
 * Requests with req_status bits other than BAD_BLOCK and TIMEOUT, or with T_r > T_max, have no
 * rows written; a request whose live slots lie beyond its table row (or 2^31 - 1025) gets
 * SPEC_REQ_BAD_BLOCK and no rows written; one with a bad block id gets SPEC_REQ_BAD_BLOCK and unspecified rows.
 * workspace: spec_attention_kv8_workspace_size bytes, 256-byte aligned, contents arbitrary; calls
 * that may overlap on the GPU (other streams, captured graphs) need one each.
 * Errors: as spec_tree_attention.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;          /* of q and o */
  int32_t B, N, T_max;
  int32_t H_q, H_kv, head_dim;
  int32_t block_size, num_blocks, max_blocks_per_req;
  float scale;                 /* <= 0 selects 1/sqrt(head_dim) */
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* node_offset;
  const uint32_t* anc_mask;
  void* o;
  float* lse;                  /* may be NULL */
  int32_t* req_status;
} spec_attn_kv8_params;

size_t spec_attention_kv8_workspace_size(const spec_attn_kv8_params* p);
spec_status_t spec_tree_attention_kv8(const spec_attn_kv8_params* p, void* workspace,
                                      size_t ws_bytes, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_kv8_compact
 * spec_kv_compact in an 8-bit cache: new[P_r + d] = old[P_r + path[r][d]] for every layer, KV
 * head, K and V.  A block that receives rows takes as scale s the largest among the scales of
 * the blocks its rows come from and, if it holds rows below P_r, its own; each of its rows
 * becomes e4m3(code * (its old scale / s)) (bits copied where the scales are equal).  Blocks none
 * of whose rows move keep their codes and scale.
 * new_kv_len, slot_map, blocks_in_use and the data errors are spec_kv_compact's.
 * Layouts: k_cache, v_cache layer 0 with layer_stride bytes between layers; k_scale, v_scale
 * [num_blocks][H_kv] with scale_layer_stride floats between layers.
 * Errors: SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED (as spec_kv8_append), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int32_t B, H_kv, head_dim, block_size, num_blocks, max_blocks_per_req, num_layers, max_path;
  int64_t layer_stride, scale_layer_stride;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* path;
  const int32_t* n_acc;
  int32_t* req_status;
  int32_t* new_kv_len;
  int32_t* slot_map;
  int32_t* blocks_in_use;
} spec_kv8_compact_params;

spec_status_t spec_kv8_compact(const spec_kv8_compact_params* p, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_kv_fork
 * Child sequences of cached ones (several samples of one prompt, branches of a search).  Fork f
 * makes request dst[f] continue request src[f] of length L = kv_len[src[f]]: the first
 * L / block_size entries of its block_table row become the parent's (shared, read-only from then
 * on); if L % block_size > 0 the next entry becomes new_block[f], a page of the caller's, and the
 * parent's rows of that page are copied into it for every layer, head, K and V (and the page's
 * scales in an 8-bit cache); kv_len[dst[f]] = L.  Other entries of the child's row stay.
 * `dtype` SPEC_F32, SPEC_BF16 or SPEC_E4M3; k_scale and v_scale are required for SPEC_E4M3 and
 * ignored otherwise.  block_table [B][max_blocks_per_req], kv_len [B]: in / out.
 * fork_status [F]: 0, or the fork was left undone: SPEC_REQ_BAD_PARENT (src or dst outside
 * [0, B), dst of another fork too, dst a src of this call, or new_block[f] named by another fork
 * that copies a partial page),
 * SPEC_REQ_BAD_SIZE (L < 0 or pages beyond the table row), SPEC_REQ_BAD_BLOCK (new_block[f] or a
 * page of the parent outside [0, num_blocks), or new_block[f] one of the parent's pages).  That no
 * other request uses new_block[f] is the caller's to see to: a page of another row of the table is
 * overwritten.
 * Layouts: layer_stride elements between layers of the caches, scale_layer_stride floats.
 * Errors: SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED (more than 65535 layers), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;
  int32_t B, F, H_kv, head_dim, block_size, num_blocks, max_blocks_per_req, num_layers;
  int64_t layer_stride, scale_layer_stride;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  int32_t* block_table;
  int32_t* kv_len;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* new_block;
  int32_t* fork_status;
} spec_fork_params;

spec_status_t spec_kv_fork(const spec_fork_params* p, spec_stream_t stream);

/* ==========================================================================================
 * Attention over a part of the cache, or over a part that requests have in common -- no counterpart
 * on the pages beyond [SURV 12.4.3] (paged caches that sequences share).  Both calls take
 * spec_tree_attention's parameters as `attn` (the same layouts, masks, scale and data errors) with these
 * differences:
 *   - every H_q / H_kv ratio, block_size and head_dim (multiple of 8 bf16 / 4 fp32 elements, <= 256)
 *     is accepted; BF16 with head_dim 128, block_size 16, 32, 64 or 128 and H_q / H_kv <= 128 runs on
 *     the tcgen05 tensor cores, everything else on a CUDA-core kernel;
 *   - a row that sees no key gets O = 0 and LSE = -infinity;
 *   - a NaN or an infinity in q, K or V reaches the rows that see it and no others (of V: the output's
 *     column at least, or the whole row and its LSE, under weights that underflow as well; a score of
 *     -infinity weighs nothing, and a row that sees no other score is NaN or as one that sees no key).
 *     Slots that no row of a request sees are not looked at;
 *   - scores are fp32: finite ones of any size are told apart to a step of theirs, scale x q.k x log2(e) beyond
 *     its range makes the row unspecified;
 *   - the ancestor mask's bits count only for nodes of the request's own tree;
 *   - a request with T_r outside [1, T_max], a negative prefix or node offsets outside [0, N] gets
 *     SPEC_REQ_BAD_SIZE; one whose slots lie beyond its table row (or 2^31 - 1025) SPEC_REQ_BAD_BLOCK; no
 *     rows are written for either, nor for a request whose req_status holds other bits than BAD_BLOCK
 *     and TIMEOUT.  One with a bad id among the pages of its tree and of the prefix that its rows see gets
 *     SPEC_REQ_BAD_BLOCK and unspecified rows.
 * workspace: the call's workspace_size bytes, 256-byte aligned, contents arbitrary; calls that may
 * overlap on the GPU (other streams, captured graphs) need one each.
 * Errors: SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED (head_dim above 256, 2^31 rows of pages or of
 * queries, more than 65535 x 32 query rows a request and KV head), SPEC_ERR_CUDA.
 * ========================================================================================== */

/* ------------------------------------------------------------------------------------------
 * spec_tree_attention_window
 * A sliding window with sinks: node i at position m = P_r + depth sees the slot of a token at position p
 * (prefix slot p, or an ancestor or itself in the tree) iff p < sinks or m - p < window; window >= 1
 * counts the node itself.  depth is the number of the node's mask bits less one, its ancestors' depths
 * count up in increasing index (what spec_tree_build writes).  Pages all of whose slots are out of sight
 * of every node (from max(sinks, 0) up to P_r - window) are not read, and their table entries may hold
 * anything.
 * Errors: SPEC_ERR_INVALID_ARG also for window < 1 or sinks < 0.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_attn_params attn;
  int32_t window, sinks;
} spec_attn_window_params;

size_t spec_attention_window_workspace_size(const spec_attn_window_params* p);
spec_status_t spec_tree_attention_window(const spec_attn_window_params* p, void* workspace,
                                         size_t ws_bytes, spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_tree_attention_shared
 * spec_tree_attention for requests that have a prefix in common (samples or beams of one prompt, as
 * spec_kv_fork and spec_beam_reorder leave them; requests under one system prompt): group g is the
 * consecutive requests group_offset[g] .. group_offset[g+1]-1 (num_groups + 1 entries from 0 to B), whose
 * first shared_len[g] slots hold the same keys and values.  Those slots are read by the table row of the
 * group's first request, once for all of the group's rows; each request's slots from shared_len on by its
 * own.  shared_len is any length from 0 to the members' prefix lengths; a group may have one member.
 * The result is spec_tree_attention's.
 * Data errors: a request that group_offset puts in no group, whose group's shared_len is negative or
 * beyond its prefix, or whose group's node offsets lie outside [0, N] gets SPEC_REQ_BAD_SIZE and no rows; so does
 * every request of a call whose group_offset goes backwards anywhere (equal entries are a group without requests).
 * Bad ids among the shared pages flag every member with SPEC_REQ_BAD_BLOCK.
 * The workspace grows with N x H_q x head_dim (two fp32 rows of partial results each).
 * Errors: SPEC_ERR_INVALID_ARG also for num_groups outside [1, B] or null group arrays.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_attn_params attn;
  int32_t num_groups;
  const int32_t* group_offset;   /* [num_groups + 1] */
  const int32_t* shared_len;     /* [num_groups] */
} spec_attn_shared_params;

size_t spec_attention_shared_workspace_size(const spec_attn_shared_params* p);
spec_status_t spec_tree_attention_shared(const spec_attn_shared_params* p, void* workspace,
                                         size_t ws_bytes, spec_stream_t stream);

/* ==========================================================================================
 * Beam search -- no counterpart on the pages.  Request b has W beams; beam j's row is row b * W + j of
 * the logits, of the block table and of every call that takes requests.  A step: the model's forward
 * (spec_tree_attention_shared with a group for each request), spec_beam_select on its logits,
 * spec_beam_reorder on the cache.
 * ========================================================================================== */

/* ------------------------------------------------------------------------------------------
 * spec_beam_select
 * The best W continuations of each request.  Beam j with score s (the sum of its tokens' log
 * probabilities) and length n offers, if it is not finished, every token x < V with
 *   score s + log_softmax(row / tau)[x], length n + 1,
 * and if it is finished only itself: token eos, score s, length n.  Continuations are ranked by
 *   score / ((5 + length) / 6)^alpha,
 * largest first, ties to the lower beam, then to the lower token; equal logits of a beam are a tie.  Out
 * comes, best first: parent (beam), token, score, length, finished (1: was finished, or token == eos).
 * A beam with score -infinity (a slot that is not in use yet) or NaN offers nothing, nor do logits of
 * -infinity and NaN; a NaN or +infinity among a row's logits takes the whole row out.  If fewer than W are
 * offered the rest is parent j, token 0, score -infinity, length n of beam j, finished 0 at place j.
 * Sums of exponentials are in fp32 per thread and pairs of fp32 numbers beyond, scores and ranks in fp64,
 * rounded once (a score beyond fp32 becomes -infinity).
 * Layouts: logits [B * W][ld] F32 / BF16, rows 16-byte aligned (ld a multiple of 16 bytes); scores [B][W]
 * fp32, lengths (>= 0), finished [B][W] int32; outputs [B][W].  out_score, out_length and out_finished
 * may be the inputs' own buffers.  eos outside [0, V): no token finishes a beam (a finished one then
 * carries token 0).
 * workspace: spec_beam_select_workspace_size bytes, 256-byte aligned.
 * Errors: SPEC_ERR_INVALID_ARG (null / misaligned pointers, V < 1, ld < V, tau <= 0 or so large or small
 * that log2(e) / tau is no normal fp32 number, alpha < 0, not finite, small workspace),
 * SPEC_ERR_UNSUPPORTED (W > 16, B * W > 65535), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
#define SPEC_MAX_BEAMS 16
typedef struct {
  spec_dtype_t dtype;          /* of logits */
  int32_t B, W, V, eos;
  int64_t ld;                  /* elements between rows */
  double tau, alpha;
  const void* logits;
  const float* scores;
  const int32_t* lengths;
  const int32_t* finished;
  int32_t* parent;
  int32_t* token;
  float* out_score;
  int32_t* out_length;
  int32_t* out_finished;
} spec_beam_select_params;

size_t spec_beam_select_workspace_size(const spec_beam_select_params* p);
spec_status_t spec_beam_select(const spec_beam_select_params* p, void* workspace, size_t ws_bytes,
                               spec_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * spec_beam_reorder
 * Makes beam j of request b continue its beam parent[b][j], in place: the W rows b * W + j of block_table
 * cover kv_len[b] = L tokens each, and entry L / block_size of a row, its writing page (the page of the
 * next token), is the beam's own, also when L is a multiple of block_size.  For each request
 *   - entries 0 .. L / block_size - 1 of row j become the parent's (full pages, shared, read-only);
 *   - a parent's first child takes its writing page over; the parent's other children get, in increasing
 *     order, the writing pages of the beams without children in increasing order, and the parent's
 *     L % block_size rows of that page are copied into them for every layer, head, K and V (and the
 *     page's scales in an 8-bit cache);
 *   - later entries of the row stay.
 * So the W writing pages of a request stay its own, and no page has to be found or given back: with W
 * pages set aside for each entry past the prompt, a search never runs out.  Parents that are 0 for every
 * beam spread one prompt over W beams.
 * beam_status [B]: 0, or the request was left as it was: SPEC_REQ_BAD_PARENT (a parent outside [0, W)),
 * SPEC_REQ_BAD_SIZE (L < 0 or L / block_size beyond the table row), SPEC_REQ_BAD_BLOCK (a writing page
 * outside [0, num_blocks), or one that two beams of the request name).  Writing pages that two requests
 * name are the caller's to avoid.
 * `dtype`, layouts and strides as in spec_kv_fork; W <= 16.
 * workspace: spec_beam_reorder_workspace_size bytes, 256-byte aligned.
 * Errors: SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED (W > 16, more than 65535 layers), SPEC_ERR_CUDA.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  spec_dtype_t dtype;
  int32_t B, W, H_kv, head_dim, block_size, num_blocks, max_blocks_per_req, num_layers;
  int64_t layer_stride, scale_layer_stride;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  int32_t* block_table;          /* [B * W][max_blocks_per_req], in / out */
  const int32_t* kv_len;         /* [B] */
  const int32_t* parent;         /* [B][W] */
  int32_t* beam_status;          /* [B] */
} spec_beam_reorder_params;

size_t spec_beam_reorder_workspace_size(const spec_beam_reorder_params* p);
spec_status_t spec_beam_reorder(const spec_beam_reorder_params* p, void* workspace, size_t ws_bytes,
                                spec_stream_t stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char* spec_status_string(spec_status_t status);

/* The cudaError_t (as int) behind the most recent SPEC_ERR_CUDA on this thread, 0 if none. */
int spec_last_cuda_error(void);

/* No counterpart on the pages: how many kernels this library has enqueued in this process, all
 * threads and devices together (a launch made while a stream is captured counts once, when it
 * is captured; replays of the graph are not launches of the library).  Diagnostics only. */
uint64_t spec_kernel_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
