/*
 * spec_tree.h -- C ABI of a GB300 (sm_103a) library for one tree-verification
 * step of Medusa/Hydra speculative decoding: draft heads fill a candidate tree,
 * the tree tokens attend over a KV-cache prefix plus their own ancestors, and
 * acceptance picks the longest accepted path (greedy, or the min(1, p/q) rule
 * with residual resampling).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - The caller owns every buffer, device scratch ("workspace") included; its
 *    size comes from the matching *_workspace_size call.  Apart from
 *    spec_tree_build (which copies a small host table to the device and waits
 *    for it) no call allocates, frees or synchronises; all work is queued on
 *    the given stream in order.  0 selects the legacy default stream.  A
 *    sequence of calls on one stream can therefore be captured into a CUDA
 *    graph (make one call first, outside the capture, so that one-time setup
 *    such as kernel attributes happens there) and replayed: the replay
 *    repeats the same work on the same buffers without the per-call host
 *    work.  spec_read_device_status synchronises and is not capturable.
 *    Some kernels launch as programmatic dependents of the kernel before
 *    them on the stream; they wait for it before reading anything it could
 *    have written.
 *  - "device" pointers must point to memory of the current CUDA device and be
 *    16-byte aligned (SPEC_EALIGN otherwise); "host" pointers are read during
 *    the call only.
 *  - Every call checks its arguments on the host before it queues anything.
 *    On failure it returns a non-zero spec_status, queues nothing, writes no
 *    output, and spec_last_error() describes the problem (per host thread).
 *    CUDA launch errors are reported as SPEC_ECUDA.
 *  - Kernels never trap and never wait without bound.  A failure detected on
 *    the device (a bounded wait that ran out, a token or page index out of
 *    range) is recorded in the first 16 bytes of the call's workspace;
 *    spec_read_device_status() returns it.  Each call clears those bytes
 *    before its kernels can record anything (any prior content, including
 *    garbage in a fresh workspace, is discarded), so a workspace may be reused
 *    by any later call on the same stream.
 *  - Tokens are int32, logits and outputs float32 unless a call says otherwise;
 *    inputs of the float tensors of a call share one spec_dtype (float32 or
 *    bfloat16 bit patterns).
 *  - Tensor shapes are given outermost first and are densely packed (row-major)
 *    where a call takes no strides.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream (cudaStream_t); declared opaquely so this header needs no CUDA headers. */
typedef struct CUstream_st* spec_stream_t;

typedef enum {
    SPEC_OK = 0,
    SPEC_EINVAL = 1,       /* bad argument: null pointer, size out of range, shape mismatch */
    SPEC_ETREE = 2,        /* malformed tree: parent[0] != -1, parent[i] not in [0, i), duplicate sibling rank */
    SPEC_EALIGN = 3,       /* a device pointer is not 16-byte aligned */
    SPEC_EWORKSPACE = 4,   /* workspace missing or smaller than *_workspace_size */
    SPEC_EUNSUPPORTED = 5, /* a valid combination this build does not implement */
    SPEC_ECUDA = 6,        /* a CUDA runtime call or launch failed */
    SPEC_ETIMEOUT = 7      /* device status only: a bounded wait inside a kernel ran out */
} spec_status;

typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1 } spec_dtype;

#define SPEC_MAX_T 1024      /* tree nodes, root included */
#define SPEC_MAX_DEPTH 16    /* deepest node; also the most draft heads */
#define SPEC_MAX_TOPK 16     /* largest top-k per head */
#define SPEC_MAX_BEAMS 64    /* beams of a sequence */

/*
 * Candidate tree, encoded once per topology by spec_tree_build.
 *
 * Hydra Guide: Sequentially-Dependent Speculative AI, sections "Candidate Tree
 * Construction" (the root is the base token x_t; a depth-k node holds a token
 * proposed by head k; rank = which of the parent head's top-k candidates it
 * is) and "Tree Attention Matrix with Topology-Aware Causal Masking" (the tree
 * is flattened into one sequence; node u may attend to node v iff v is an
 * ancestor of u or v = u).
 *
 * Host fields are filled by spec_tree_build; the pointers point into the
 * caller's device buffer and stay valid as long as that buffer does.
 */
typedef struct {
    int32_t T;                                   /* nodes, root (node 0) included */
    int32_t max_depth;                           /* largest depth (root: 0) */
    int32_t words;                               /* ceil(T / 64): 64-bit words per ancestor mask */
    int32_t n_internal;                          /* nodes that have at least one child */
    int32_t n_at_depth[SPEC_MAX_DEPTH + 1];      /* host: nodes of each depth */
    int32_t n_internal_at_depth[SPEC_MAX_DEPTH + 1]; /* host: nodes of each depth that have children */
    int32_t max_rank_at_depth[SPEC_MAX_DEPTH + 1];   /* host: largest rank among nodes of each depth (depth >= 1) */
    const int32_t* parent;        /* device [T]; parent[0] = -1, parent[i] < i */
    const int32_t* depth;         /* device [T] */
    const int32_t* rank;          /* device [T]; 0 for the root */
    const uint64_t* anc;          /* device [T][words]; bit j of row i set iff j is i or an ancestor of i */
    const int32_t* internal;      /* device [n_internal]: nodes with children, by depth then index */
    const int32_t* internal_off;  /* device [SPEC_MAX_DEPTH + 2]: depth d's nodes start at internal[internal_off[d]] */
    const int32_t* row_of;        /* device [T]: position of a node within its depth's internal list, -1 for leaves */
    const int32_t* child_off;     /* device [T + 1]: children of u are child_idx[child_off[u] .. child_off[u+1]) */
    const int32_t* child_idx;     /* device [max(T - 1, 1)], ascending per parent */
} spec_tree;

/* Bytes of device memory spec_tree_build needs for a tree of T nodes (0 if T is out of range). */
size_t spec_tree_device_bytes(int32_t T);

/*
 * Validate a parent-index tree and encode it for the other calls.
 *   parent  host [T]: parent[0] = -1, 0 <= parent[i] < i.
 *   rank    host [T] or NULL: rank[i] >= 0 is node i's slot among its parent
 *           head's top-k (0 = most probable); distinct among siblings.  NULL
 *           numbers each node's children 0, 1, ... in index order.
 *   T       1 .. SPEC_MAX_T; the tree's depth must be <= SPEC_MAX_DEPTH.
 *   d_buf   device buffer of at least spec_tree_device_bytes(T) bytes.
 *   out     host struct filled on success.
 * Copies the encoded tables to d_buf on stream s and waits for that copy.
 */
spec_status spec_tree_build(const int32_t* parent, const int32_t* rank, int32_t T,
                            void* d_buf, size_t d_bytes, spec_tree* out, spec_stream_t s);

/* Workspace bytes hydra_draft needs for these shapes (0 on invalid arguments). */
size_t hydra_draft_workspace_size(const spec_tree* tree, int32_t B, int32_t d, int32_t V, int32_t K,
                                  const int32_t* cond, const int32_t* topk, spec_dtype dt);

/*
 * Draft heads: fill every candidate node of every sequence with a token.
 *
 * Medusa Heads (ultralytics glossary), section "So sagen die Köpfe voraus": a
 * head is one feed-forward layer with SiLU and a residual, then a projection
 * onto the vocabulary.  Hydra Guide, sections "1. Embedding Conditioning
 * Mechanics" and "Candidate Tree Construction": a sequentially dependent head
 * also reads the base-embedding row of its parent node's token, and each
 * node's children are the top-k of the head run on that node.  Per head k
 * (filling depth k + 1) and parent node u of sequence b:
 *     u_in = h_b                     if cond[k] == 0   (W1[k] is [d, d])
 *     u_in = [h_b || emb[tok(u)]]    if cond[k] == 1   (W1[k] is [d, 2d])
 *     u_in = [h_b || emb[tok(a_1)] || ... || emb[tok(a_k)]]   if cond[k] == 2
 *            (a_1 .. a_k = u's path below the root, depth 1 first; W1[k] is
 *            [d, (k+1) d]; Hydra Guide, "2. Generalizing to Arbitrary Tree Depths")
 *     z    = h_b + SiLU(W1[k] u_in + b1[k])   (rounded to bf16 when dt is bf16)
 *     l    = W2[k] z                 ([V] logits, never written to memory)
 * A child of rank r gets the (r+1)-th largest logit (ties: lower token id).
 *
 *   h          device [B, d]                 hidden state of each sequence
 *   emb        device [V, d]                 base token-embedding table
 *   K          number of heads, >= tree->max_depth, <= SPEC_MAX_DEPTH
 *   W1, b1, W2 host arrays [K] of device pointers: W1[k] [d, d_in_k] (out x in),
 *              b1[k] [d] (a NULL entry or a NULL array means no bias), W2[k] [V, d]
 *   cond, topk host [K]: cond[k] in {0, 1, 2}; topk[k] in 1 .. SPEC_MAX_TOPK and
 *              > the largest rank among depth-(k+1) nodes
 *   root_tok   device [B]                     token of node 0 (the base token x_t)
 *   node_tok   device [B, T] out: node 0 = root_tok, others = drafted tokens
 *   node_logit device [B, T] out: the node's logit in its parent's row (root: 0)
 *   node_logprob device [B, T] out or NULL: cumulative log-probability along
 *              the node's path, log-softmax of each row (root: 0)
 * Shapes: 1 <= B, d % 8 == 0, 1 <= d <= 16384, topk[k] <= V <= 2^24.
 */
spec_status hydra_draft(const void* h, const void* emb, int32_t K,
                        const void* const* W1, const void* const* b1, const void* const* W2,
                        const int32_t* cond, const int32_t* topk, const int32_t* root_tok,
                        const spec_tree* tree, int32_t B, int32_t d, int32_t V, spec_dtype dt,
                        int32_t* node_tok, float* node_logit, float* node_logprob,
                        void* ws, size_t ws_bytes, spec_stream_t s);

/* Bytes of one folded embedding table (V * d fp32), 0 on invalid shapes. */
size_t hydra_fold_table_bytes(int32_t d, int32_t V);

/*
 * Fold the embedding half of a cond-1 head's first layer into a per-token
 * table, once per set of weights (not per step).  Hydra Guide, "1. Embedding
 * Conditioning Mechanics": the head reads u_in = [h_b || emb[tok]], so
 *     W1 u_in = W1[:, 0:d] h_b + tab[tok],   tab[v, m] = sum_j W1[m, d + j] emb[v, j]
 * and the second term depends on the token alone.
 *
 *   W1   device [d, 2d] in dt (the head's first layer, out x in)
 *   emb  device [V, d] in dt
 *   tab  device fp32 [V, d] out (hydra_fold_table_bytes bytes, caller-owned)
 * fp32 accumulation in a fixed order per element: bf16 inputs on the tensor
 * cores (256 vocabulary rows per launch), fp32 inputs on the CUDA cores.  All
 * pointers 16-byte aligned (SPEC_EALIGN); SPEC_EINVAL on NULL or out-of-range
 * shapes.  Launched on s, asynchronous.  The call has no workspace, so no
 * device status: its kernels' bounded waits cannot run out unless the GPU
 * stops making progress, and then the table is left undefined.
 */
spec_status hydra_fold_embedding(const void* W1, const void* emb, int32_t d, int32_t V, spec_dtype dt,
                                 float* tab, spec_stream_t s);

/*
 * hydra_draft with folded first layers: tab is a host array [K] (or NULL) of
 * device tables from hydra_fold_embedding(W1[k], emb, ...).  On the bf16
 * tensor-core path a cond-1 head with a table streams only W1[k][:, 0:d] per
 * step: a[b] = W1[k][:, 0:d] h_b, and the kernel that picks a node's token
 * writes that node's head input z = h_b + SiLU(a[b] + tab[k][tok] + b1[k])
 * itself.  NULL entries, other heads and the fp32 path use the whole W1[k].
 * The results equal hydra_draft's up to fp32 rounding order.  Workspace:
 * hydra_draft_workspace_size.  Tables must be 16-byte aligned (SPEC_EALIGN);
 * everything else as hydra_draft.
 */
spec_status hydra_draft_folded(const void* h, const void* emb, int32_t K,
                               const void* const* W1, const void* const* b1, const void* const* W2,
                               const float* const* tab, const int32_t* cond, const int32_t* topk,
                               const int32_t* root_tok, const spec_tree* tree, int32_t B, int32_t d,
                               int32_t V, spec_dtype dt, int32_t* node_tok, float* node_logit,
                               float* node_logprob, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * One draft head for hydra_draft_heads.  form 0 is hydra_draft's head; form 1
 * is the head form that the Hydra Guide prints as code (fusion MLP
 * Linear -> SiLU -> Linear -> LayerNorm, then a bias-free vocabulary
 * projection; its first head Linear -> SiLU -> LayerNorm, i.e. no W1b):
 *   form 0: z = h_b + SiLU(W1 u_in + b1)                         (hidden == d)
 *   form 1: y = W1b SiLU(W1 u_in + b1) + b1b, or y = SiLU(W1 u_in + b1) when
 *           W1b is NULL (then hidden == d);
 *           z = (y - mean(y)) / sqrt(var(y) + ln_eps) * gamma + beta
 *           (mean and biased variance over the d entries of y)
 * then l = W2 z as in hydra_draft.  u_in follows cond exactly as in
 * hydra_draft; with dt bf16, SiLU(W1 u_in + b1) is rounded to bf16 when it
 * feeds W1b, and z is rounded to bf16.
 */
typedef struct {
    int32_t cond;         /* 0, 1 or 2 (hydra_draft) */
    int32_t topk;         /* 1 .. SPEC_MAX_TOPK (hydra_draft) */
    int32_t form;         /* 0 or 1 */
    int32_t hidden;       /* rows of W1: d for form 0 and for form 1 without W1b */
    const void* W1;       /* device [hidden, d_in] */
    const void* b1;       /* device [hidden] or NULL */
    const void* W1b;      /* form 1: device [d, hidden] or NULL */
    const void* b1b;      /* form 1: device [d] or NULL */
    const void* gamma;    /* form 1: device [d] or NULL (ones) */
    const void* beta;     /* form 1: device [d] or NULL (zeros) */
    const void* W2;       /* device [V, d] (heads may share one) */
} spec_head;

/* Workspace bytes hydra_draft_heads needs (0 on invalid arguments). */
size_t hydra_draft_heads_workspace_size(const spec_tree* tree, int32_t B, int32_t d, int32_t V, int32_t K,
                                        const spec_head* heads, spec_dtype dt);

/*
 * hydra_draft with a per-head description (heads: host array [K]); ln_eps > 0
 * is the LayerNorm epsilon of form-1 heads.  Everything else as hydra_draft.
 */
spec_status hydra_draft_heads(const void* h, const void* emb, int32_t K, const spec_head* heads,
                              const int32_t* root_tok, const spec_tree* tree, int32_t B, int32_t d, int32_t V,
                              float ln_eps, spec_dtype dt, int32_t* node_tok, float* node_logit,
                              float* node_logprob, void* ws, size_t ws_bytes, spec_stream_t s);

/* Workspace bytes tree_attention needs for these shapes on the current device (0 on invalid arguments). */
size_t tree_attention_workspace_size(const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                     int32_t Lmax, int32_t D, spec_dtype dt);

/*
 * Tree attention of one layer.
 *
 * Hydra Guide, section "Tree Attention Matrix with Topology-Aware Causal
 * Masking": every tree token sees the whole cached prefix and, among the tree
 * tokens, only itself and its ancestors (M_tree = 0 there, -inf elsewhere), so
 * its output equals autoregressive attention over [prompt, ancestors, itself].
 * For query head h (KV head h / (Hq / Hkv)), sequence b and node i:
 *     keys  = k_cache[b, :prefix_len[b]] followed by k_tree[b, a] for a in anc*(i)
 *     out   = softmax(scale * q . keys) . values,  lse = log(sum exp(scale * q . keys))
 *
 *   q                 device [B, Hq, T, D]
 *   k_cache, v_cache  device [B, Hkv, Lmax, D]; rows >= prefix_len[b] do not affect the
 *                     result (the tensor-core path reads, then discards, those inside
 *                     the last 128-key tile of a sequence: they must be readable memory)
 *   prefix_len        device [B], each in 0 .. Lmax (values outside are clamped to it)
 *   k_tree, v_tree    device [B, Hkv, T, D]: keys/values of the tree tokens
 *   scale             > 0, or 0 for the usual 1/sqrt(D)
 *   out               device [B, Hq, T, D] float32
 *   lse               device [B, Hq, T] float32, or NULL
 * Shapes: Hq % Hkv == 0, D in {64, 128}, 1 <= Lmax <= 2^22.
 */
spec_status tree_attention(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* prefix_len, const void* k_tree, const void* v_tree,
                           const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t Lmax,
                           int32_t D, float scale, spec_dtype dt, float* out, float* lse,
                           void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * tree_attention without a caller-provided workspace.  The pages have no
 * counterpart to this call: it exists for callers that cannot allocate device
 * memory, such as a plugin running inside a host engine that has already
 * handed out the device memory and forbids further cudaMalloc calls, or a
 * caller whose own interface has no way to pass a workspace pointer through.
 *
 * Arguments, results and errors are those of tree_attention without ws and
 * ws_bytes.  The scratch is a 32 MiB array inside this library's device image
 * (every GPU that loads the library holds it until the process exits); shapes
 * whose tree_attention_workspace_size exceeds 32 MiB are rejected with
 * SPEC_EWORKSPACE before anything is queued.  The call allocates nothing.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  All calls share the one array and it keeps the
 * last call's contents (each call clears what must start at zero): calls
 * whose work overlaps on the GPU -- on different streams, or from different
 * host threads -- race on it and must not be issued.  A failure the kernels
 * detect (a bounded wait that ran out) goes to the status word at the start
 * of the built-in array; tree_attention_noalloc_status reads it.
 */
spec_status tree_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* prefix_len, const void* k_tree, const void* v_tree,
                                   const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t Lmax,
                                   int32_t D, float scale, spec_dtype dt, float* out, float* lse, spec_stream_t s);

/*
 * Device status of the calls that use the built-in scratch (tree_attention_noalloc):
 * the counterpart of spec_read_device_status for a caller workspace.  Waits on
 * stream s for the calls queued before it, copies the status word of the
 * built-in array to *status (host) and returns SPEC_OK, or an error status
 * when the copy fails.  Like tree_attention_noalloc, it looks up the array's
 * address with the current device and allocates nothing.
 */
spec_status tree_attention_noalloc_status(int32_t* status, spec_stream_t s);

/* Workspace bytes tree_attention_paged needs (0 on invalid arguments). */
size_t tree_attention_paged_workspace_size(const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                           int32_t max_blocks, int32_t block_size, int32_t D, spec_dtype dt);

/*
 * Tree attention over a paged KV cache -- Hydra Guide, "Hydra Production
 * Engineering Checklist", item 3 (KV-Cache Tree Branch Management: the tree
 * attention KV cache lives in pre-allocated static blocks).  The same result
 * as tree_attention with k_cache[b, :, j] = k_pool[block_table[b, j / block_size],
 * :, j % block_size] (likewise V).
 *
 *   k_pool, v_pool  device [num_blocks, Hkv, block_size, D]
 *   block_table     device [B, max_blocks] int32: pool block of positions
 *                   j*block_size .. (j+1)*block_size - 1 of sequence b; only the
 *                   first ceil(prefix_len[b] / block_size) entries are read
 *   prefix_len      device [B], each in 0 .. max_blocks * block_size (clamped)
 *   block_size      a positive multiple of 64; max_blocks * block_size <= 2^22
 *   the rest as tree_attention.
 * A table entry outside 0 .. num_blocks-1 is reported as SPEC_EINVAL in the
 * status word and its keys read as zeros (no memory outside the pool is read).
 */
spec_status tree_attention_paged(const void* q, const void* k_pool, const void* v_pool, int32_t num_blocks,
                                 const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                                 const int32_t* prefix_len, const void* k_tree, const void* v_tree,
                                 const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                 float scale, spec_dtype dt, float* out, float* lse, void* ws,
                                 size_t ws_bytes, spec_stream_t s);

/* Workspace bytes tree_accept (mode 0 or 1) or tree_accept_typical (mode 2) needs (0 on invalid arguments). */
size_t tree_accept_workspace_size(int32_t mode, const spec_tree* tree, int32_t B, int32_t V);

/*
 * Acceptance: longest accepted path and the extra token.
 *
 * mode 0, greedy -- Hydra Guide, section "Parallel Verification and Greedy
 *   Acceptance Algorithm": a(u) = argmax logits_p[b, u] (ties: lower id); a
 *   node is accepted when its parent is and its token equals a(parent); the
 *   deepest accepted node u* (lowest index on equal depth) ends the path and
 *   a(u*) is the extra token.  temperature, seed, offset and logits_q unused.
 * mode 1, rejection -- Speculative Decoding (thegustafson.com), sections "The
 *   acceptance criterion", "The correctness guarantee" and "A worked example":
 *   p_u = softmax(logits_p[b, u] / temperature), q_u likewise from logits_q;
 *   the edge into node c with token x is accepted iff u_c < p_par(x) / q_par(x);
 *   u* as above; the extra token is drawn from norm(max(p_u* - q_u*, 0)) when u*
 *   has children (from p_u* if that residual is zero), else from p_u*, by
 *   inverse CDF in ascending token order with uniform u'.  u_c is word 0 and u'
 *   word 1 of Philox4x32-10 (Salmon et al., SC'11) with key (seed low, seed
 *   high) and counter (node, b, offset low, offset high) -- u' from node 0 --
 *   each word w mapped to (w >> 8) * 2^-24.
 *
 *   logits_p     device [B, T, V] float32 target logits (row u predicts the token after u)
 *   logits_q     device [B, T, V] float32 draft logits (rejection; rows of leaves not read) or NULL
 *   node_tok     device [B, T]
 *   accept_len   device [B] out: m, the depth of u*
 *   accept_path  device [B, max_depth + 1] out: node ids root first, -1 padded
 *   next_token   device [B] out: the extra token
 *   margin       device [B] out or NULL: distance of the closest decision to its
 *                threshold (greedy: smallest top-1 minus top-2 logit gap over accepted
 *                nodes; rejection: smallest |u_c - ratio| over decided edges with
 *                ratio < 1, or the sampling draw's distance to a CDF breakpoint over the total)
 * Shapes: 2 <= V <= 2^24; temperature > 0 for mode 1.
 */
spec_status tree_accept(int32_t mode, const float* logits_p, const float* logits_q, const int32_t* node_tok,
                        const spec_tree* tree, int32_t B, int32_t V, float temperature,
                        uint64_t seed, uint64_t offset, int32_t* accept_len, int32_t* accept_path,
                        int32_t* next_token, float* margin, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * Typical acceptance -- Medusa Heads (ultralytics glossary), section "Tree
 * Attention und Akzeptanz": for sampling, a candidate is kept when its
 * probability under the base model exceeds a threshold tied to the entropy of
 * that distribution (more tokens accepted, the distribution no longer exact;
 * Speculative Decoding, section "Beyond draft models: Medusa").  The pages give
 * neither the formula nor the constants; this call takes
 *     p_u = softmax(logits_p[b, u] / temperature),  H_u = -sum_x p_u(x) ln p_u(x),
 *     the edge into node c with token x is accepted iff p_par(x) > min(epsilon, alpha * exp(-H_par)),
 * u* = the deepest accepted node (lowest index on equal depth), and the extra
 * token drawn from p_u* by inverse CDF in ascending token order with the
 * uniform u' of tree_accept (word 1 of Philox4x32-10, counter (0, b, offset)).
 *
 *   margin  device [B] out or NULL: the smallest |p_par(x) / threshold - 1| over
 *           edges with an accepted parent, or the draw's distance to a CDF
 *           breakpoint over the total, whichever is smaller
 *   the rest as tree_accept; epsilon, alpha >= 0 and finite, temperature > 0;
 *   the workspace is tree_accept_workspace_size(2, ...).
 */
spec_status tree_accept_typical(const float* logits_p, const int32_t* node_tok, const spec_tree* tree,
                                int32_t B, int32_t V, float temperature, float epsilon, float alpha,
                                uint64_t seed, uint64_t offset, int32_t* accept_len, int32_t* accept_path,
                                int32_t* next_token, float* margin, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * The uniforms tree_accept draws, for inspection: u_accept [B, T] (entry
 * [b, c] = word 0 of counter (c, b, offset)), u_sample [B] (word 1 of counter
 * (0, b, offset)).  Device pointers.  Salmon et al., SC'11, Philox4x32-10.
 */
spec_status spec_philox_uniform(uint64_t seed, uint64_t offset, int32_t B, int32_t T,
                                float* u_accept, float* u_sample, spec_stream_t s);

/* Workspace bytes tree_kv_commit needs (its status word only). */
size_t tree_kv_commit_workspace_size(void);

/*
 * KV commit of the accepted path -- Speculative Decoding (thegustafson.com),
 * section "The acceptance criterion" (the suffix past the rejection point is
 * discarded from the caches; the next round starts from the last accepted
 * token), and Hydra Guide, section "3. Tree KV-Cache Page Sizing" (discarded
 * candidates are rolled back without deallocation).
 *
 * For every sequence b with m = accept_len[b] and L = prefix_len[b]: the K and
 * V rows of the m + 1 nodes accept_path[b, 0..m] (root first) of every KV head
 * are copied from the tree buffers to cache rows L .. L + m, and prefix_len[b]
 * becomes L + m + 1.  No other cache row changes: the rejected nodes are never
 * copied.  The extra token tree_accept emits is not committed (it is the root
 * of the next round's tree).
 *
 *   k_tree, v_tree    device [B, Hkv, T, D] (dt): the tree nodes' keys/values
 *   k_cache, v_cache  device [B, Hkv, Lmax, D] (dt), updated in place
 *   prefix_len        device [B], updated in place
 *   accept_len        device [B]; accept_path device [B, max_depth + 1]: the
 *                     outputs of tree_accept for the same tree
 *   ws                >= tree_kv_commit_workspace_size() bytes, 16-byte aligned
 * Tree, cache and tree buffers 16-byte aligned; D * element size a multiple of
 * 16 bytes.  Host-checked arguments fail with a status before anything is
 * queued.  A sequence whose path is not root-first along tree edges, whose m is
 * outside 0..max_depth, or whose commit would pass Lmax is left unchanged and
 * SPEC_EINVAL goes to the status word (spec_read_device_status).  Caller owns
 * every buffer; the call queues work on s and does not synchronise.
 */
spec_status tree_kv_commit(const void* k_tree, const void* v_tree, void* k_cache, void* v_cache,
                           int32_t* prefix_len, const int32_t* accept_len, const int32_t* accept_path,
                           const spec_tree* tree, int32_t B, int32_t Hkv, int32_t Lmax, int32_t D,
                           spec_dtype dt, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * KV commit into a paged cache -- the same commit as tree_kv_commit (same
 * sections) with the cache in pre-allocated static blocks (Hydra Guide, "Hydra
 * Production Engineering Checklist", item 3), the layout tree_attention_paged
 * reads: cache position L + i of sequence b is row (L + i) % block_size of pool
 * block block_table[b, (L + i) / block_size] of every KV head.
 *
 *   k_pool, v_pool  device [num_blocks, Hkv, block_size, D] (dt), updated in place
 *   block_table     device [B, max_blocks] int32; only the entries of the blocks
 *                   the commit writes are read
 *   block_size      positive; max_blocks * block_size <= 2^22
 *   the rest as tree_kv_commit (ws >= tree_kv_commit_workspace_size() bytes).
 * Besides tree_kv_commit's checks, a sequence whose commit would pass
 * max_blocks * block_size positions or write a block outside 0 .. num_blocks-1
 * is left unchanged and SPEC_EINVAL goes to the status word.
 */
spec_status tree_kv_commit_paged(const void* k_tree, const void* v_tree, void* k_pool, void* v_pool,
                                 int32_t num_blocks, const int32_t* block_table, int32_t max_blocks,
                                 int32_t block_size, int32_t* prefix_len, const int32_t* accept_len,
                                 const int32_t* accept_path, const spec_tree* tree, int32_t B, int32_t Hkv,
                                 int32_t D, spec_dtype dt, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * What happens to a score between the product and the softmax (NULL: nothing).
 * With P the query's position and p the key's, positions counted over the shared
 * prefix, the cached prefix and a node's depth:
 *     x = scale q.k
 *     x = softcap * tanh(x / softcap)       if softcap > 0
 *     x = x - slopes[h] * (P - p)           if slopes, h the query head
 *     the key is seen only if P - p < window, if window > 0 (the query itself always is)
 * With bf16 inputs a capped score, and with it lse, is off by some 2^-22 of the cap.
 */
typedef struct {
    float softcap;          /* 0: none; else 1e-6 to 4096 */
    int32_t window;         /* 0: none */
    const float* slopes;    /* device [Hq], finite, or NULL */
} spec_score;

/* Workspace bytes tree_attention_shared and its paged form (Lshared = shared_blocks * block_size,
 * Lmax = max_blocks * block_size) need on the current device (0 on invalid arguments). */
size_t tree_attention_shared_workspace_size(const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                            int32_t Lshared, int32_t Lmax, int32_t D, spec_dtype dt);

/*
 * Tree attention of a batch whose sequences share a long prefix (a system prompt, a
 * document, the samples of one prompt): sequence b's keys are the shared ones, then its
 * own cached ones, then its tree's.  The result is tree_attention's over their
 * concatenation; the shared keys are read once for as many sequences as fill a
 * block of query rows, not once per sequence.
 *     keys  = k_shared[:shared_len], k_cache[b, :prefix_len[b]], k_tree[b, a] for a in anc*(i)
 *     out   = softmax(x) . values,  lse = log(sum exp(x)),  x the scores (spec_score)
 *
 *   q                 device [B, Hq, T, D]
 *   k_shared, v_shared  device [Hkv, Lshared, D]
 *   shared_len        device [1], in 0 .. Lshared (clamped)
 *   k_cache, v_cache  device [B, Hkv, Lmax, D]: the sequences' own keys behind the shared ones;
 *                     rows >= prefix_len[b] do not affect the result but must be readable
 *   prefix_len        device [B], each in 0 .. Lmax (clamped), without the shared keys
 *   k_tree, v_tree    device [B, Hkv, T, D]
 *   score             host, or NULL
 *   out               device [B, Hq, T, D] in dt, the inputs' type (tree_attention's is float32);
 *                     it must not overlap an input
 *   lse               device [B, Hq, T] float32, or NULL
 *   scale             > 0, or 0 for the usual 1/sqrt(D)
 * Shapes: Hq % Hkv == 0, D in {64, 128}, 1 <= Lshared, Lmax <= 2^22; T = 1 is the form for
 * single tokens.  With bf16 inputs the softmax's weights are rounded to bf16 before they
 * weigh the values; their sum, and everything else, is in 32 bits.  Values of keys that a
 * node does not see (of other branches, or in front of its window) weigh zero and must be
 * finite to do so.
 */
spec_status tree_attention_shared(const void* q, const void* k_shared, const void* v_shared,
                                  const int32_t* shared_len, int32_t Lshared, const void* k_cache,
                                  const void* v_cache, const int32_t* prefix_len, const void* k_tree,
                                  const void* v_tree, const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                  int32_t Lmax, int32_t D, float scale, const spec_score* score, spec_dtype dt,
                                  void* out, float* lse, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * tree_attention_shared over a paged cache: shared and own keys in the blocks of one pool.
 *   k_pool, v_pool  device [num_blocks, Hkv, block_size, D]
 *   shared_table    device [shared_blocks] int32: the shared prefix's blocks in order; the first
 *                   ceil(shared_len / block_size) entries are read
 *   block_table     device [B, max_blocks] int32: each sequence's own blocks, the first
 *                   ceil(prefix_len[b] / block_size) entries are read
 *   block_size      a positive multiple of 16; max_blocks and shared_blocks times it <= 2^22
 *   the rest as tree_attention_shared.
 * A table entry outside 0 .. num_blocks-1 is reported as SPEC_EINVAL in the status word and
 * no memory outside the pool is read; what the sequences that use the block get is undefined.
 */
spec_status tree_attention_shared_paged(const void* q, const void* k_pool, const void* v_pool, int32_t num_blocks,
                                        const int32_t* shared_table, int32_t shared_blocks,
                                        const int32_t* shared_len, const int32_t* block_table, int32_t max_blocks,
                                        int32_t block_size, const int32_t* prefix_len, const void* k_tree,
                                        const void* v_tree, const spec_tree* tree, int32_t B, int32_t Hq,
                                        int32_t Hkv, int32_t D, float scale, const spec_score* score,
                                        spec_dtype dt, void* out, float* lse, void* ws, size_t ws_bytes,
                                        spec_stream_t s);

/* Workspace bytes tree_attention_scored and its paged form (Lmax = max_blocks * block_size) need
 * on the current device (0 on invalid arguments). */
size_t tree_attention_scored_workspace_size(const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv,
                                            int32_t Lmax, int32_t D, spec_dtype dt);

/*
 * Tree attention with transformed scores: tree_attention_shared without a shared prefix, for
 * models that cap their scores, bias them by distance or look back over a window.  Keys in
 * front of every node's window are not read.
 */
spec_status tree_attention_scored(const void* q, const void* k_cache, const void* v_cache, const int32_t* prefix_len,
                                  const void* k_tree, const void* v_tree, const spec_tree* tree, int32_t B,
                                  int32_t Hq, int32_t Hkv, int32_t Lmax, int32_t D, float scale,
                                  const spec_score* score, spec_dtype dt, void* out, float* lse, void* ws,
                                  size_t ws_bytes, spec_stream_t s);

/* tree_attention_scored over a paged cache (tree_attention_shared_paged's, without the shared blocks). */
spec_status tree_attention_scored_paged(const void* q, const void* k_pool, const void* v_pool, int32_t num_blocks,
                                        const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                                        const int32_t* prefix_len, const void* k_tree, const void* v_tree,
                                        const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                        float scale, const spec_score* score, spec_dtype dt, void* out, float* lse,
                                        void* ws, size_t ws_bytes, spec_stream_t s);

/* Workspace bytes kv_append and kv_append_paged need (their status word only). */
size_t kv_append_workspace_size(void);

/*
 * Append new tokens of a ragged batch to the KV cache, keys rotated to their
 * positions on the way, and rotate their queries in the same launch.  The tokens
 * of sequence b are rows seq_start[b] .. seq_start[b + 1] - 1 of the projections;
 * token number i of them goes to cache position prefix_len[b] + i and is rotated
 * as position
 *     pos = pos_base + prefix_len[b] + i,  angles  phi_j = pos * freq[j]:
 *     x' = x cos(phi_j) - y sin(phi_j),    y' = x sin(phi_j) + y cos(phi_j)
 * for the pairs (x, y) = elements (j, j + rot/2) of a head, or (2j, 2j + 1) when
 * interleaved; elements rot .. D - 1 pass unchanged.  Values are copied.  Angles
 * are taken in 64 bits, the rotation in 32, rounded once to dt.
 * prefix_len is read, not advanced: the layers of a model append at the same place.
 *
 *   q, k, v       device, rows of Hq, Hkv and Hkv heads x D (dense), q_stride, k_stride and
 *                 v_stride elements between tokens: slices of one packed projection, say.  q may
 *                 be NULL (then q_out too).  16-byte aligned, strides multiples of 16 bytes
 *   N             rows of the projections, 0 .. 2^28
 *   seq_start     device [B + 1], not decreasing, within 0 .. N; rows before the first and behind
 *                 the last sequence are neither read into the cache nor written to q_out
 *   prefix_len    device [B]
 *   pos_base      device [1] added to every position (the length of a shared prefix), or NULL
 *   freq          device float64 [rot / 2], radians per position; NULL with rot = 0
 *   rot           even, 0 .. D: leading elements of a head that are rotated
 *   k_cache, v_cache  device [B, Hkv, Lmax, D] (dt), updated in place
 *   q_out         device [N, Hq, D] (dt); it must not overlap q, k or v
 *   ws            >= kv_append_workspace_size() bytes, 16-byte aligned
 * Shapes: D a multiple of 16 bytes, D <= 1024, 1 <= B <= 65535, Lmax <= 2^22.
 * A sequence with a negative prefix_len, whose tokens would pass Lmax or whose
 * offsets decrease or leave 0 .. N is reported as SPEC_EINVAL in the status word;
 * its cache rows are left unchanged, and its q_out too.  Where decreasing offsets
 * give a row to two other sequences, one of them gets it, at its own place; the
 * other's tokens are then written in part.
 */
spec_status kv_append(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, int32_t N, const int32_t* seq_start, int32_t B, int32_t Hq, int32_t Hkv,
                      int32_t D, const int32_t* prefix_len, const int32_t* pos_base, const double* freq,
                      int32_t rot, int32_t interleaved, void* k_cache, void* v_cache, int32_t Lmax,
                      spec_dtype dt, void* q_out, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * kv_append into a paged cache, the layout tree_attention_paged reads: position
 * p of sequence b is row p % block_size of pool block block_table[b, p / block_size].
 *
 *   k_pool, v_pool  device [num_blocks, Hkv, block_size, D] (dt), updated in place
 *   block_table     device [B, max_blocks] int32; only the entries of blocks the append writes
 *                   are read.  A block that is written belongs to one sequence
 *   block_size      positive; max_blocks * block_size <= 2^22
 *   the rest as kv_append, with max_blocks * block_size for Lmax.
 * Tokens whose block lies outside 0 .. num_blocks-1 are not written (their q_out
 * neither) and SPEC_EINVAL goes to the status word.
 */
spec_status kv_append_paged(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int32_t N, const int32_t* seq_start, int32_t B, int32_t Hq,
                            int32_t Hkv, int32_t D, const int32_t* prefix_len, const int32_t* pos_base,
                            const double* freq, int32_t rot, int32_t interleaved, void* k_pool, void* v_pool,
                            int32_t num_blocks, const int32_t* block_table, int32_t max_blocks,
                            int32_t block_size, spec_dtype dt, void* q_out, void* ws, size_t ws_bytes,
                            spec_stream_t s);

/*
 * The tree nodes' projections, rotated and laid out for tree attention: node i of
 * sequence b is row b * T + i of q, k and v and is rotated (kv_append) as position
 *     pos_base + prefix_len[b] + depth[i],
 * the position it would have on its path.  A one-node tree is the form for
 * single tokens.  The rotated keys are the ones tree_kv_commit copies.
 *
 *   q, k, v             device, B * T rows, strides as in kv_append
 *   q_out               device [B, Hq, T, D] (dt) out
 *   k_tree, v_tree      device [B, Hkv, T, D] (dt) out; no output may overlap q, k or v
 *   the rest as kv_append.  The call has no workspace and no device status.
 */
spec_status tree_rope(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const spec_tree* tree, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                      const int32_t* prefix_len, const int32_t* pos_base, const double* freq, int32_t rot,
                      int32_t interleaved, spec_dtype dt, void* q_out, void* k_tree, void* v_tree,
                      spec_stream_t s);

/* Workspace bytes beam_select needs on the current device (0 on invalid arguments).  Never fewer for a larger B, W, V
 * or K: a workspace made for the largest call serves every smaller one. */
size_t beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t K);

/*
 * Selection of a beam search, for drafts that extend their best continuations step by step:
 * of every sequence's W beams the K best (beam, token) pairs.  For a live beam w and a token t
 *     score  = scores[w] + x[w, t] - log sum_u exp x[w, u],   length = length[w] + 1
 * An ended beam (ended[w] != 0) offers itself: token eos, score and length as they are, whatever
 * its logits.  A beam whose score is not finite offers nothing (a first step has one
 * live beam and the others at -inf).  Pairs are ranked by score / max(length, 1)^alpha, in 64
 * bits, equal ones by the lower beam, then the lower token.
 *
 *   logits      device [B, W] rows of V logits (dt), row_stride >= V elements between rows; rows
 *               may start anywhere, the first 16-byte aligned.  NaN counts as -inf, and
 *               -inf is never chosen.  A beam with a logit of +inf offers nothing, and
 *               SPEC_EINVAL goes to the status word
 *   scores      device [B, W] float32: log-probabilities so far
 *   ended, length  device [B, W] or NULL (none ended; lengths 0)
 *   eos         token that ends a beam, or -1 (then ended must be NULL)
 *   alpha       0 (rank by the score) .. 16
 *   token, parent, score  device [B, K] out, best first: the token, the beam it continues and the
 *               new score.  Where fewer pairs exist: -1, -1, -inf
 *   ended_out, length_out  device [B, K] out or NULL: whether it has ended (its parent had, or its
 *               token is eos; 1 where there is no pair), its length (0)
 * Shapes: W, K <= SPEC_MAX_BEAMS, 2 <= V <= 2^24.  With K == W, score may be scores, ended_out
 * ended and length_out length; outputs must not overlap an input otherwise.
 */
spec_status beam_select(const void* logits, int64_t row_stride, const float* scores, const int32_t* ended,
                        const int32_t* length, int32_t B, int32_t W, int32_t V, int32_t K, int32_t eos, float alpha,
                        spec_dtype dt, int32_t* token, int32_t* parent, float* score, int32_t* ended_out,
                        int32_t* length_out, void* ws, size_t ws_bytes, spec_stream_t s);

/* Workspace bytes beam_reorder, kv_reorder and kv_reorder_paged need (their status word only). */
size_t beam_reorder_workspace_size(void);

/*
 * Reorder a state of the beams in place: row w of sequence b becomes what row parent[b, w] was.
 * Rows whose parent is their own beam or -1 stay.
 *   state    device [B, W] rows of row_bytes bytes (a multiple of 4): hidden states, token histories
 *   parent   device [B, W], each in -1 .. W - 1.  Others are reported as SPEC_EINVAL in the status
 *            word and their beams stay
 */
spec_status beam_reorder(void* state, int64_t row_bytes, const int32_t* parent, int32_t B, int32_t W, void* ws,
                         size_t ws_bytes, spec_stream_t s);

/*
 * beam_reorder of the beams' caches: positions start[b] .. end[b] - 1 of every KV head.  What lies in
 * front (a prompt that all beams of the sequence have alike) and behind stays.
 *   k_cache, v_cache  device [B * W, Hkv, Lmax, D] (dt), beam w of sequence b at b * W + w
 *   start, end        device [B], 0 <= start <= end <= Lmax; others are reported as SPEC_EINVAL in
 *                     the status word and the sequence stays
 * Shapes: D a multiple of 16 bytes, D <= 1024.
 */
spec_status kv_reorder(void* k_cache, void* v_cache, const int32_t* parent, const int32_t* start, const int32_t* end,
                       int32_t B, int32_t W, int32_t Hkv, int32_t Lmax, int32_t D, spec_dtype dt, void* ws,
                       size_t ws_bytes, spec_stream_t s);

/*
 * kv_reorder in a paged cache (tree_kv_commit_paged's layout).
 *   block_table  device [B * W, max_blocks]: the entries of positions start[b] .. end[b] - 1 are
 *                read; blocks in that range belong to one beam each.  Positions in a block
 *                outside the pool, of either side, stay, and SPEC_EINVAL goes to the status word
 */
spec_status kv_reorder_paged(void* k_pool, void* v_pool, int32_t num_blocks, const int32_t* block_table,
                             int32_t max_blocks, int32_t block_size, const int32_t* parent, const int32_t* start,
                             const int32_t* end, int32_t B, int32_t W, int32_t Hkv, int32_t D, spec_dtype dt, void* ws,
                             size_t ws_bytes, spec_stream_t s);

/* Workspace bytes kv_weigh and its paged form (Lmax = max_blocks * block_size; path_len 0 without a
 * path) need on the current device (0 on invalid arguments).  Never fewer for a larger B, Lmax, path_len or, without a
 * path, T. */
size_t kv_weigh_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t path_len, int32_t Lmax,
                               int32_t D, spec_dtype dt);

/*
 * Add up the attention weight that cached keys receive, the measure kv_evict goes by.  To be
 * called once the rows' own keys are in the cache (tree_kv_commit, kv_append), with the
 * queries and the lse of the attention they went through:
 *     acc[b, h, j] = decay * acc[b, h, j] + sum over rows r of h's query heads that see key j of
 *                    exp(scale * q_r . k_j - lse_r)
 * The rows that count are the last `count` tokens of the sequence: nodes accept_path[b, 0 ..
 * accept_len[b]] of a tree (tree_accept's outputs), or rows 0 .. n_rows[b] - 1 of q; row i
 * sees keys 0 .. prefix_len[b] - count + i.  The rows' own keys start at 0 instead of decay * acc.
 *
 *   q            device [B, Hq, T, D] (dt), finite in the rows that add something
 *   lse          device [B, Hq, T] float32; a row whose lse is not finite (it saw nothing) adds nothing
 *   k_cache      device [B, Hkv, Lmax, D] (dt), finite below prefix_len[b].  Rows behind that do not affect
 *                the result but must be readable
 *   prefix_len   device [B]: keys in the cache, those of the rows included
 *   seen         device [B] or NULL (prefix_len): tokens of the sequence so far, evicted ones included
 *   n_rows       device [B], 0 .. T, or NULL (T, or those of the path)
 *   accept_len, accept_path  device [B], [B, path_len] or NULL; path_len (max_depth + 1) <= 17
 *   decay        0 .. 1; 0 forgets what acc holds, whatever it is
 *   acc          device [B, Hkv, Lmax] float32, updated below prefix_len[b]
 *   pos          device [B, Hkv, Lmax] int32 or NULL: the rows' own keys get their positions,
 *                seen[b] - prefix_len[b] + j
 *   scale        > 0, or 0 for the usual 1/sqrt(D)
 * Shapes: Hq % Hkv == 0, D in {64, 128}.  Sums are in 32 bits, in a fixed order.  In bf16 calls scale and lse are
 * each rounded once on the way to base 2, so that a weight is off by some 2^-24 (|scale q . k| + |lse|) of itself.  A sequence
 * with more rows than keys, a length outside 0 .. Lmax, rows outside 0 .. T or a path outside the
 * tree is left unchanged and SPEC_EINVAL goes to the status word.
 */
spec_status kv_weigh(const void* q, const float* lse, const void* k_cache, const int32_t* prefix_len,
                     const int32_t* seen, const int32_t* n_rows, const int32_t* accept_len,
                     const int32_t* accept_path, int32_t path_len, int32_t B, int32_t Hq, int32_t Hkv, int32_t T,
                     int32_t Lmax, int32_t D, float scale, float decay, spec_dtype dt, float* acc, int32_t* pos,
                     void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * kv_weigh over a paged cache: pool [num_blocks, Hkv, block_size, D], block_size a multiple of 16,
 * acc and pos [B, Hkv, max_blocks * block_size] by position in the cache.  Keys in a block outside the
 * pool keep their acc, and SPEC_EINVAL goes to the status word.
 */
spec_status kv_weigh_paged(const void* q, const float* lse, const void* k_pool, int32_t num_blocks,
                           const int32_t* block_table, int32_t max_blocks, int32_t block_size,
                           const int32_t* prefix_len, const int32_t* seen, const int32_t* n_rows,
                           const int32_t* accept_len, const int32_t* accept_path, int32_t path_len, int32_t B,
                           int32_t Hq, int32_t Hkv, int32_t T, int32_t D, float scale, float decay, spec_dtype dt,
                           float* acc, int32_t* pos, void* ws, size_t ws_bytes, spec_stream_t s);

/* Workspace bytes kv_evict and its paged form (Lmax = max_blocks * block_size) need (0 on invalid arguments).  Of one
 * budget never fewer for a larger B, Hkv or Lmax; another budget has its own size. */
size_t kv_evict_workspace_size(int32_t B, int32_t Hkv, int32_t Lmax, int32_t budget);

/*
 * Evict keys from the cache: every KV head of a sequence with more than `budget` keys keeps
 * `budget` of them, each head its own.  First come the protected ones, with pos < sink or
 * pos >= seen[b] - recent, then those of the largest acc (NaN last), equal ones by the lower place.
 * Kept keys at places below the budget stay there; the i-th free place below the budget, in
 * ascending order, takes the i-th kept key from behind it, with its value, acc and pos.  So the cache's
 * order is lost, and pos tells where a key belongs: attention over rotated keys (tree_attention,
 * tree_attention_shared without a window or bias) does not depend on it.  New tokens are
 * rotated by `seen` (tree_rope's prefix_len) and go to place len_out[b].
 *
 *   k_cache, v_cache  device [B, Hkv, Lmax, D] (dt)
 *   prefix_len   device [B], 0 .. Lmax
 *   seen         device [B] or NULL (prefix_len): tokens of the sequence so far
 *   acc, pos     device [B, Hkv, Lmax] float32, int32 (kv_weigh).  Positions below prefix_len are taken as they stand: one
 *                that was never set counts as the number it holds, so -1 lies below every sink > 0 and is protected
 *   budget       1 .. 2^22; sink, recent >= 0, together at most the budget
 *   k_out, v_out, acc_out, pos_out  NULL: in place, places from budget on are left as they are.
 *                Else another cache [B, Hkv, Lout, D] and its weights and positions [B, Hkv, Lout], Lout >=
 *                min(budget, Lmax): its first min(prefix_len, budget) places get what the cache would have
 *                there, and the cache stays.  The two must not overlap
 *   len_out      device [B] out: min(prefix_len, budget).  It must not overlap prefix_len or seen
 * Shapes: D a multiple of 16 bytes, D <= 1024, B * Hkv <= 65535.  A sequence with a length
 * outside its room is left unchanged (len_out: its prefix_len) and SPEC_EINVAL goes to the status word.
 */
spec_status kv_evict(void* k_cache, void* v_cache, const int32_t* prefix_len, const int32_t* seen, float* acc,
                     int32_t* pos, int32_t B, int32_t Hkv, int32_t Lmax, int32_t D, int32_t budget, int32_t sink,
                     int32_t recent, void* k_out, void* v_out, float* acc_out, int32_t* pos_out, int32_t Lout,
                     int32_t* len_out, spec_dtype dt, void* ws, size_t ws_bytes, spec_stream_t s);

/*
 * kv_evict in a paged cache (tree_kv_commit_paged's layout); acc and pos [B, Hkv, max_blocks *
 * block_size] by place.  In place, a block in use belongs to one sequence (several sequences that share one would
 * each fill its holes with their own rows: such go to an out_table), and blocks behind the budget's last are free afterwards.
 *   out_table    device [B, out_blocks] or NULL: blocks of the same pool to go to, none of which a
 *                sequence reads; acc_out, pos_out [B, Hkv, out_blocks * block_size] with it
 * A sequence with a table entry in use outside 0 .. num_blocks-1 is left unchanged and
 * SPEC_EINVAL goes to the status word.
 */
spec_status kv_evict_paged(void* k_pool, void* v_pool, int32_t num_blocks, const int32_t* block_table,
                           int32_t max_blocks, int32_t block_size, const int32_t* prefix_len, const int32_t* seen,
                           float* acc, int32_t* pos, int32_t B, int32_t Hkv, int32_t D, int32_t budget, int32_t sink,
                           int32_t recent, const int32_t* out_table, int32_t out_blocks, float* acc_out,
                           int32_t* pos_out, int32_t* len_out, spec_dtype dt, void* ws, size_t ws_bytes,
                           spec_stream_t s);

/* Message of the last failed call on this host thread ("" if none). */
const char* spec_last_error(void);

/* Copy the device status word kept at the start of a workspace to *status and wait for it (SPEC_OK = no failure). */
spec_status spec_read_device_status(const void* ws, int32_t* status, spec_stream_t s);

/*
 * Self-test of the device failure path: queues one kernel that waits on a
 * shared-memory barrier nothing completes, with the bounded wait the
 * tensor-core kernels use; after limit_ns (capped at 1 s) it gives up and
 * records SPEC_ETIMEOUT in the first word of ws (read it back with
 * spec_read_device_status).  ws: device, >= 16 bytes, 16-byte aligned.
 */
spec_status spec_selftest_timeout(void* ws, uint64_t limit_ns, spec_stream_t s);

/*
 * Kernel tracing.  While enabled, every kernel this library launches is
 * bracketed by a pair of CUDA events on its launch stream (at most `capacity`
 * launches are recorded).  spec_trace_end waits for them, totals the time per
 * kernel name into out[0 .. max_entries) and returns the number of entries,
 * or -1 on error.  spec_launch_count counts every kernel launch of this
 * library in this process.  Tracing is process-wide and not thread-safe.
 */
typedef struct {
    char name[48];
    int32_t launches;
    double total_ms;
} spec_trace_entry;

spec_status spec_trace_begin(int32_t capacity);
int32_t spec_trace_end(spec_trace_entry* out, int32_t max_entries);
int64_t spec_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_TREE_H */
