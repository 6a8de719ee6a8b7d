/*
 * kvp.h -- C ABI of the paged, prefix-shared KV pool, its prefix cache and its
 * attention kernels (GB300 / sm_103a).
 *
 * Conventions for every entry point:
 *   - returns KVP_OK (0) or a negative KVP_ERR_* code; out-parameters are
 *     written only on success and state is left unchanged on failure, except
 *     where a function says otherwise (kvp_radix_evict reports how far it
 *     got; seq_accept_draft's bookkeeping stands when its launch fails);
 *   - "device" pointers are CUDA global memory on the current device, owned by
 *     the caller; "host" pointers are ordinary host memory owned by the caller;
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream);
 *     device work is enqueued on it and the call returns without synchronising,
 *     except where a function says it synchronises;
 *   - bf16 tensors are IEEE bfloat16 bit patterns, 16-byte aligned;
 *   - a pool handle is not thread-safe: serialise calls on one pool.
 *
 * Layouts (row-major, innermost last):
 *   K pool, V pool   [L][NB][Hkv][bs][d]  bf16   (one (block, kv head) tile is
 *                                                  a contiguous bs*d run)
 *   block tables     [S][MB] int32 (host), entries past a sequence's blocks ignored
 *   decode q, out    [L][S][Hq][d] bf16;   lse [L][S][Hq] fp32, natural log
 *   verify q, out    [L][B*n][Hq][d] bf16; lse [L][B*n][Hq] fp32
 *   appended k, v    [L][ntok][Hkv][d] bf16
 * Query head h reads kv head h / (Hq / Hkv).
 */
#ifndef KVP_H
#define KVP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    KVP_OK = 0,
    KVP_ERR_INVALID = -1, /* bad argument, unknown sequence, capacity exceeded */
    KVP_ERR_OOM = -2,     /* no free block or sequence slot                   */
    KVP_ERR_STATE = -3,   /* operation not possible in the object's state     */
    KVP_ERR_CUDA = -4,    /* a CUDA runtime call failed                        */
    KVP_ERR_DEVICE = -5,  /* a kernel's own bounds check tripped (see below)  */
    KVP_ERR_WORKSPACE = -6 /* kvp_decode_step: workspace too small (see there) */
};

/* Device error word bits (kvp_device_error). */
enum {
    KVP_DEVERR_BLOCK_ID = 1,     /* a planned block id outside [0, NB): those tokens read as 0 */
    KVP_DEVERR_TREE_PARENT = 2,  /* a parent pointer not in [-1, i): treated as a root       */
    KVP_DEVERR_WAIT_TIMEOUT = 4  /* a tcgen05 pipeline wait ran out: that CTA stopped early  */
};

/* ------------------------------------------------------------------ pool */

/*
 * A block-paged KV pool: NB blocks of bs token slots per layer, shared by many
 * sequences through per-sequence block tables with per-block refcounts.
 * Paper: "Dendrite: O(1) fork latency agent-native inference engine", section
 * details (16-token paged blocks; tree-shaped KV cache with reference
 * counting); "Trellis: RadixAttention", section "RadixAttention in Trellis"
 * (a session holds an ordered list of block ids into one shared pool).
 */
typedef struct kvp_pool kvp_pool;

typedef struct {
    int32_t num_layers;         /* L   */
    int32_t num_blocks;         /* NB  */
    int32_t block_size;         /* bs, tokens per block (16 and 32 are the pages' sizes) */
    int32_t num_kv_heads;       /* Hkv */
    int32_t head_dim;           /* d, a multiple of 8 */
    int32_t max_seqs;           /* sequence ids are 0 .. max_seqs-1, lowest free id first */
    int32_t max_blocks_per_seq; /* MB, block table capacity */
    uint64_t alloc_seed;        /* free-list order: splitmix64-driven Fisher-Yates
                                   shuffle of [0, NB); 0 = identity order */
} kvp_pool_desc;

/* Create a pool over caller-owned device storage k_storage / v_storage, each
 * [L][NB][Hkv][bs][d] bf16.  Both may be NULL for a bookkeeping-only pool, in
 * which case seq_append / seq_append_batch return KVP_ERR_STATE (use
 * seq_reserve).  The pool never allocates or frees KV storage. */
int kv_pool_create(const kvp_pool_desc *desc, void *k_storage, void *v_storage, kvp_pool **out);

/*
 * A pool of 4-bit pages ("Dendrite", section on FlashInfer kernels and
 * TurboQuant integration: 4-bit KV compression that cuts KV memory 3.88x and
 * is computed on directly; the quantiser is not given there).  Each (token,
 * kv head) row of d values is kept as d signed 4-bit codes in [-7, 7] and one
 * power-of-two scale 2^e, e an int8 in [-127, 127]:
 *   e = the smallest integer with max|x| <= 7 * 2^e (-127 for a zero row),
 *   code = x / 2^e rounded half to even, value = code * 2^e,
 * 4 + 8/d bits per value (16 / 4.125 = 3.88x less than bf16 at d = 64).
 * Storage, all device memory owned by the caller, 16-byte aligned:
 *   k_codes, v_codes  [L][NB][Hkv][bs][d/2] bytes: element 2i of a row in
 *                     the low nibble of byte i, 2i+1 in the high nibble
 *                     (two's complement);
 *   k_exps, v_exps    [L][NB][Hkv][bs] int8.
 * Needs d = 64 or 128 and bs a multiple of 16, else KVP_ERR_INVALID.
 * seq_append / seq_append_batch take bf16 K/V as for any pool and quantise
 * them on the device (copy-on-write copies codes and exponents);
 * seq_accept_draft moves codes and exponents.  Attention over such a pool:
 * paged_decode_attention_kv4 with desc->kv_format = KVP_KV_4BIT.
 */
int kv_pool_create_kv4(const kvp_pool_desc *desc, void *k_codes, void *k_exps, void *v_codes,
                       void *v_exps, kvp_pool **out);
int kv_pool_destroy(kvp_pool *pool);

/* New empty sequence ("allocate_sequence" in Dendrite's API example). */
int seq_alloc(kvp_pool *pool, int32_t *seq_out);

/* Copy-on-write fork ("fork_sequence(parent)?" in Dendrite's API example):
 * the child gets a copy of the parent's block table and every block's
 * refcount goes up by one.  No KV bytes move and no device work is issued;
 * cost is O(number of blocks) host integer work, independent of KV size. */
int seq_fork(kvp_pool *pool, int32_t parent, int32_t *child_out);

/* Release a sequence: every block's refcount drops by one and blocks that
 * reach zero go back to the free list, last table entry first ("SGLang
 * RadixAttention", reference-counting section: referenced blocks are never
 * reclaimed). */
int seq_free(kvp_pool *pool, int32_t seq);

/* Speculative accept after tree verify ("CAST", section on speculative
 * decoding: the target model accepts one path of the draft tree).  The
 * sequence holds ctx_len context tokens followed by n_draft draft tokens,
 * draft node i at position ctx_len + i with parent[i] in [-1, i) (-1: a
 * root), n_draft <= 64.  The path from a root down to node `accepted` (-1:
 * none) is kept: its tokens move, in order, to positions ctx_len,
 * ctx_len + 1, ... (K and V, every layer and kv head); the length becomes
 * ctx_len + path length and the blocks past the new end are released, last
 * first.  A block that receives a moved token and is shared with another
 * sequence is copied first (copy-on-write).  Device work is one
 * kv_move_kernel launch on `stream` (none when nothing moves; a pool without
 * K/V storage updates its bookkeeping only).  path_out (n_draft entries,
 * may be NULL) receives the kept node ids, root first, *n_path_out their
 * count.  KVP_ERR_INVALID (bad sequence, lengths or parents) or
 * KVP_ERR_OOM (no block to copy into) change nothing; KVP_ERR_CUDA: the
 * bookkeeping is done but the launch failed. */
int seq_accept_draft(kvp_pool *pool, int32_t seq, int32_t ctx_len, const int32_t *parent, int32_t n_draft,
                     int32_t accepted, int32_t *path_out, int32_t *n_path_out, void *stream);

/* A new sequence that starts from blocks someone already holds (a prefix
 * found in the prefix cache below): its table is blocks[0..n_blocks), one
 * more reference on each, and its length n_blocks * block_size ("Trellis",
 * section "RadixAttention in Trellis": a session acquires the existing
 * prefix blocks, raising their refcount, instead of allocating and
 * recomputing them).  Every block must be in use (refcount > 0), else
 * KVP_ERR_INVALID and nothing changes; KVP_ERR_OOM when no sequence slot is
 * free. */
int seq_alloc_prefix(kvp_pool *pool, const int32_t *blocks, int32_t n_blocks, int32_t *seq_out);

/* Append ntok tokens' K and V (device, [L][ntok][Hkv][d] bf16 each) to a
 * sequence.  Copy-on-write ("Dendrite", section details: data is shared until
 * modified and copied only on write): if the last block is partially filled
 * and other live sequences also hold it, the sequence first gets a fresh
 * block with the used slots copied on the device; a full last block just
 * gets a new block; a block held only by this sequence is written in place.
 * Enqueues at most one kernel.  k and v must stay valid until it has run. */
int seq_append(kvp_pool *pool, int32_t seq, const void *k, const void *v, int32_t ntok,
               void *stream);

/* Append to several distinct sequences in one launch: ntoks[i] tokens to
 * seqs[i] (host arrays), processed in order with the semantics of seq_append;
 * k, v: device [L][sum ntoks][Hkv][d], sequence-major.  All or nothing: if the
 * pool cannot hold every append, nothing changes and KVP_ERR_OOM returns.
 * (Appends beyond a launch's parameters take several; so does a batch in which
 * one sequence copies a shared page and another, cut back in that page by
 * seq_accept_draft, goes on in it: the copies are made first.) */
int seq_append_batch(kvp_pool *pool, int32_t nseq, const int32_t *seqs, const int32_t *ntoks,
                     const void *k, const void *v, void *stream);

/* Bookkeeping half of seq_append with no device work: reserves slots for ntok
 * tokens and reports where they go.  slots_out (host, ntok entries, may be
 * NULL) receives block*bs + slot per token; cow_out (host, 3 entries, may be
 * NULL) receives {source block, copy block, used slots} or {-1, -1, 0} when no
 * copy-on-write happened.  The caller is then responsible for the data. */
int seq_reserve(kvp_pool *pool, int32_t seq, int32_t ntok, int32_t *slots_out, int32_t *cow_out);

/* Host queries. */
int seq_block_table(const kvp_pool *pool, int32_t seq, int32_t *host_out, int32_t cap,
                    int32_t *nblocks_out);
int seq_len(const kvp_pool *pool, int32_t seq, int32_t *len_out);
int block_refcount(const kvp_pool *pool, int32_t block, int32_t *rc_out);
int kvp_free_block_count(const kvp_pool *pool, int32_t *n_out);
int kvp_cow_count(const kvp_pool *pool, int64_t *n_out);
int kvp_pool_shape(const kvp_pool *pool, int32_t *layers_out, int32_t *kv_heads_out);
int kvp_pool_head_dim(const kvp_pool *pool, int32_t *head_dim_out);

/* Block tables and lengths of n sequences into host arrays h_tables
 * [n][width] (padded with -1) and h_lens [n]. */
int kvp_gather_tables(const kvp_pool *pool, const int32_t *seqs, int32_t n, int32_t width,
                      int32_t *h_tables, int32_t *h_lens);

/* Same, written to device arrays d_tables [n][width] and d_lens [n] (either
 * may be NULL) with an asynchronous host-to-device copy on `stream`. */
int kvp_export_tables(kvp_pool *pool, const int32_t *seqs, int32_t n, int32_t width,
                      int32_t *d_tables, int32_t *d_lens, void *stream);

/* ---------------------------------------------------------- prefix cache */

/*
 * A radix-tree prefix cache over a pool's blocks ("SGLang RadixAttention",
 * sections on the node and edge structure, on the three operations match /
 * split / insert, and on reference counting with LRU eviction; "Trellis",
 * section "RadixAttention in Trellis").  The root is the empty sequence; the
 * edge into a node holds a run of token ids and the ids of the blocks that
 * store them.  Everything is in whole blocks of block_size tokens: a run is
 * a whole number of blocks, a match is rounded down to whole agreeing
 * blocks, and edges split on block boundaries.  The cache holds one pool
 * reference on every block in the tree, so a block goes back to the pool
 * only when neither the cache nor a sequence holds it.  "Last used" is a
 * logical clock advanced by every match and insert and stamped on every node
 * of the path it used.  Not thread-safe; destroy the cache before its pool.
 */
typedef struct kvp_radix kvp_radix;

/* KVP_ERR_INVALID on a null pool; KVP_ERR_OOM if memory runs out. */
int kvp_radix_create(kvp_pool *pool, kvp_radix **out);

/* Drops the cache's references (each node's blocks last to first, children
 * before parents) and frees the cache. */
int kvp_radix_destroy(kvp_radix *cache);

/* Longest cached prefix of tokens[0..n_tokens) in whole blocks: its block
 * ids go to blocks_out (cap >= n_tokens / block_size) and their count to
 * *n_blocks_out.  Every node whose blocks were returned (including one whose
 * edge agreed only in part) is locked, i.e. not evictable, until
 * kvp_radix_unlock(cache, *lock_out); *lock_out = -1 when nothing matched. */
int kvp_radix_match(kvp_radix *cache, const int32_t *tokens, int32_t n_tokens, int32_t *blocks_out,
                    int32_t cap, int32_t *n_blocks_out, int32_t *lock_out);

/* Releases a lock from kvp_radix_match (-1: nothing to release).
 * KVP_ERR_STATE, with nothing changed, if that path is not locked. */
int kvp_radix_unlock(kvp_radix *cache, int32_t lock);

/* Caches a sequence's whole blocks: tokens[0..n_tokens) are stored in
 * blocks[0..n_blocks) (block j holds tokens [j*bs, (j+1)*bs)); only the
 * first min(n_tokens / bs, n_blocks) blocks count.  The tree is walked as in
 * match, splitting an edge that agrees for only part of its run (the upper
 * part inherits the lower part's locks); what is not cached yet becomes a
 * new leaf on which the cache takes one reference per block.  Blocks already
 * cached for an equal prefix are kept.  Every new block must be in use, else
 * KVP_ERR_INVALID and nothing changes. */
int kvp_radix_insert(kvp_radix *cache, const int32_t *tokens, int32_t n_tokens, const int32_t *blocks,
                     int32_t n_blocks);

/* Until the pool has need_free free blocks: the unlocked leaf used longest
 * ago gives its blocks back (last to first) and leaves the tree; a parent
 * left childless and unlocked is then a leaf like any other.  *freed_out =
 * blocks that went back to the pool.  KVP_OK when met, KVP_ERR_OOM when
 * nothing more is evictable. */
int kvp_radix_evict(kvp_radix *cache, int32_t need_free, int32_t *freed_out);

/* Canonical dump for tests and tools: depth first from the root, children
 * in increasing order of their first block's tokens; per node the int32
 * words depth, locks, stamp, n_tokens, tokens..., n_blocks, blocks...
 * *n_out = words needed; KVP_ERR_INVALID (nothing written) when cap is too
 * small. */
int kvp_radix_dump(const kvp_radix *cache, int32_t *out, int64_t cap, int64_t *n_out);

/* ------------------------------------------------------------- attention */

typedef struct {
    int32_t num_layers;    /* L: q/out/lse and both pools carry a leading layer axis */
    int32_t num_q_heads;   /* Hq */
    int32_t num_kv_heads;  /* Hkv; Hq % Hkv == 0 and Hq / Hkv <= 64 */
    int32_t head_dim;      /* d: 64 or 128 */
    int32_t block_size;    /* bs: a power of two >= 16 */
    int32_t num_blocks;    /* NB */
    float scale;           /* softmax scale; <= 0 selects 1/sqrt(d) */
    int32_t use_sharing;   /* 1: blocks that several sequences share are read once per
                              tile of up to 64 query rows (cascade); 0: every sequence
                              reads its own blocks (the unshared baseline) */
    int32_t kv_format;     /* KVP_KV_BF16 (0) or KVP_KV_4BIT (1): the pool's page format */
} kvp_attn_desc;

enum { KVP_KV_BF16 = 0, KVP_KV_4BIT = 1 };

/* Device workspace bytes that paged_decode_attention (or, with
 * desc->kv_format = KVP_KV_4BIT, paged_decode_attention_kv4) needs for this
 * batch (same host tables and lengths as the call).  Returns 0 on invalid
 * input. */
size_t kvp_decode_workspace_size(const kvp_attn_desc *desc, const int32_t *block_tables,
                                 const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks);

/*
 * Decode attention over the paged pool: for each layer, sequence s and query
 * head h, out = softmax(q k^T * scale) v over the first seq_lens[s] tokens of
 * sequence s, and lse = the natural-log log-sum-exp of the scaled scores.
 * (Decode is one new token attending to the cached keys and values: "SGLang
 * RadixAttention", section on the KV-cache lifecycle; the pool is the paged
 * cache of "Dendrite", section details.)  The call attends to exactly
 * seq_len tokens; append the new token's K/V first to include it.
 *
 * block_tables [num_seqs][max_blocks] and seq_lens [num_seqs] are HOST arrays
 * (kvp_gather_tables gives them for pool sequences).  The call plans on the
 * host: sequences whose tables hold the same physical blocks at the same
 * positions are grouped so that a shared block is read from HBM once per
 * group of up to 64 query rows instead of once per sequence; long key ranges
 * are split across CTAs and merged by log-sum-exp.  The plan, which carries
 * the physical block ids, is copied into the workspace with an asynchronous
 * copy from host memory on `stream`; no device block table is read, and the
 * host arrays may be reused as soon as the call returns.
 *
 * q: device [L][num_seqs][Hq][d] bf16; k_pool / v_pool: the pool's device
 * storage; out: device [L][num_seqs][Hq][d] bf16; lse: device
 * [L][num_seqs][Hq] fp32 or NULL.  workspace: device, 256-byte aligned,
 * ws_bytes >= kvp_decode_workspace_size(); one call at a time per workspace.
 * Errors: KVP_ERR_INVALID for an empty sequence, a table entry outside
 * [0, NB), a too-small or misaligned workspace, misaligned tensors or
 * unsupported shapes; KVP_ERR_CUDA if a launch fails.
 */
int paged_decode_attention(const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs,
                           int32_t max_blocks, const kvp_attn_desc *desc, void *out, float *lse,
                           void *workspace, size_t ws_bytes, void *stream);

/*
 * Decode attention over a pool of 4-bit pages (kv_pool_create_kv4): the same
 * call and results as paged_decode_attention, with the keys and values being
 * the pages' values code * 2^e.  k_codes / k_exps / v_codes / v_exps are the
 * pool's storage; desc->kv_format must be KVP_KV_4BIT (paged_decode_attention
 * rejects such a descriptor).  HBM traffic per token is (d/2 + 1) bytes per
 * kv head for K and for V instead of 2d.
 */
int paged_decode_attention_kv4(const void *q, const void *k_codes, const void *k_exps,
                               const void *v_codes, const void *v_exps, const int32_t *block_tables,
                               const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks,
                               const kvp_attn_desc *desc, void *out, float *lse, void *workspace,
                               size_t ws_bytes, void *stream);

size_t kvp_verify_workspace_size(const kvp_attn_desc *desc, const int32_t *block_tables,
                                 const int32_t *ctx_lens, int32_t batch, int32_t n_draft,
                                 int32_t max_blocks);

/*
 * Speculative tree-verify attention ("Inference-Cost-Aware Dynamic Tree
 * Construction for Efficient Inference in Large Language Models" (CAST),
 * technical summary sections 1-2: the target model checks a dynamic draft
 * tree of candidate tokens, EAGLE-2/3 style, in one forward pass).
 * Sequence b has ctx_lens[b] context tokens followed, in its pages, by
 * n_draft <= 64 draft tokens.  Draft node i (query row b*n_draft + i) attends
 * to every context token and to the draft tokens of its ancestors and itself,
 * anc*(i) = {i, parent(i), parent(parent(i)), ...}.
 * tree_parent: DEVICE [batch][n_draft] int32, parent < i or -1 for a root
 * (a forest is allowed).  block_tables / ctx_lens: HOST [batch][max_blocks] /
 * [batch].  Other arguments as for paged_decode_attention with
 * num_seqs = batch * n_draft query rows.  A bad parent pointer sets
 * KVP_DEVERR_TREE_PARENT in the workspace error word and that node is
 * treated as a root.  Pages must be bf16 (desc->kv_format = KVP_KV_BF16).
 */
int tree_verify_attention(const void *q, const int32_t *tree_parent, int32_t n_draft,
                          const void *k_pool, const void *v_pool, const int32_t *block_tables,
                          const int32_t *ctx_lens, int32_t batch, int32_t max_blocks,
                          const kvp_attn_desc *desc, void *out, float *lse, void *workspace,
                          size_t ws_bytes, void *stream);

/*
 * Decode attention for callers that cannot allocate device memory -- e.g. a
 * serving process whose memory manager has already given (nearly) all device
 * memory to its own pools, or a plug-in that cannot reach its host program's
 * allocator and must not bypass it.  Same arguments and results as
 * paged_decode_attention, without workspace: the scratch space is a
 * KVP_STATIC_WORKSPACE_BYTES array inside the library, present on every GPU
 * that loads it until the process exits.  The pages have no counterpart; this
 * is an interface for such callers.
 *   - Returns KVP_ERR_INVALID, before enqueuing anything, when the batch's plan
 *     needs more than KVP_STATIC_WORKSPACE_BYTES (see
 *     kvp_decode_workspace_size).
 *   - All calls on a device share the array: calls that overlap on the GPU
 *     race; serialise them.  Each call rewrites the words that must start at
 *     zero (error word, work counters) before its kernels run.
 *   - The first call on each device looks up the array's device address; make
 *     it before any stream capture.  No call allocates device memory.
 * kvp_device_error cannot read this call's error word (there is no caller
 * workspace); bounds violations still skip the access.
 */
#define KVP_STATIC_WORKSPACE_BYTES (32u << 20)
int paged_decode_attention_noalloc(const void *q, const void *k_pool, const void *v_pool,
                                   const int32_t *block_tables, const int32_t *seq_lens,
                                   int32_t num_seqs, int32_t max_blocks, const kvp_attn_desc *desc,
                                   void *out, float *lse, void *stream);

/*
 * Decode attention over pool sequences: paged_decode_attention with the block
 * tables and lengths read from the pool itself, so the caller keeps no host
 * tables.  Row s of q / out / lse is sequence seq_ids[s] (host array) at its
 * current length.  desc must describe the pool (layers, kv heads, head dim,
 * block size, block count and page format); 4-bit pools read their codes and
 * exponents.  kvp_pool_decode_workspace_size returns the workspace bytes for
 * the sequences as they are now (0 on invalid input).
 */
size_t kvp_pool_decode_workspace_size(const kvp_pool *pool, const int32_t *seq_ids, int32_t num_seqs,
                                      const kvp_attn_desc *desc);
int paged_decode_attention_pool(const kvp_pool *pool, const int32_t *seq_ids, int32_t num_seqs,
                                const void *q, void *out, float *lse, const kvp_attn_desc *desc,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * One decode step, host buffers in and out ("Dendrite", API example: every
 * branch appends its new token and attends over its own blocks, the shared
 * prefix included).  In stream order on `stream`:
 *   1. host-to-device copies h_k_new -> d_k_new, h_v_new -> d_v_new and
 *      h_q -> d_q (each skipped when its host pointer is NULL: the data is
 *      already on the device);
 *   2. seq_append_batch of ntok tokens to every sequence (skipped for ntok 0):
 *      its bookkeeping and the plan of step 3 are done on the host first, and
 *      its write kernel is enqueued right before the attention kernels, which
 *      are launched programmatically behind it (they start while it
 *      finishes and wait for it before reading K/V);
 *   3. paged_decode_attention_pool over the sequences at their new lengths,
 *      d_q -> d_out, d_lse;
 *   4. device-to-host copies d_out -> h_out and d_lse -> h_lse (each skipped
 *      when its host pointer is NULL).
 * The call returns once all of it is enqueued; host outputs are valid after
 * the stream synchronises, and host inputs must stay untouched until then.
 * Page-locked host buffers make the copies asynchronous; pageable ones work,
 * but the driver then stages each copy before returning.  With
 * KVP_STEP_HOST_MAPPED in io->flags the host buffers must be page-locked and
 * addressable by the device (cudaHostAlloc, or registered with
 * cudaHostRegisterMapped; under unified addressing any page-locked memory)
 * and 16-byte aligned: the inputs then cross in one copy kernel into the d_*
 * buffers, and the attention kernels write out and lse straight into h_out /
 * h_lse (d_out and d_lse are then neither read nor written and may be NULL),
 * instead of one copy-engine transfer per buffer.
 *
 * Shapes: k_new, v_new [L][num_seqs * ntok][Hkv][d] bf16, sequence-major;
 * q, out [L][num_seqs][Hq][d] bf16; lse [L][num_seqs][Hq] fp32 (d_lse may be
 * NULL, then h_lse must be NULL too).  seq_ids: host, distinct live
 * sequences.  *ws_needed (may be NULL) receives the workspace bytes the
 * attention needed.
 * Errors: KVP_ERR_INVALID (bad arguments, descriptor not matching the pool,
 * unknown flags, misaligned mapped buffers) and KVP_ERR_OOM (the appends do
 * not fit) before anything is enqueued; KVP_ERR_WORKSPACE when ws_bytes <
 * *ws_needed: the copies and the append of steps 1-2 are enqueued and the
 * pool holds the new tokens, nothing else ran; grow the workspace and finish
 * the step with paged_decode_attention_pool.
 */
typedef struct {
    const void *h_k_new, *h_v_new, *h_q; /* host inputs, or NULL */
    void *h_out;                         /* host outputs, or NULL */
    float *h_lse;
    void *d_k_new, *d_v_new, *d_q;       /* device inputs / staging */
    void *d_out;                         /* device outputs */
    float *d_lse;
    uint32_t flags;                      /* KVP_STEP_* */
} kvp_step_io;

enum { KVP_STEP_HOST_MAPPED = 1 };

int kvp_decode_step(kvp_pool *pool, const int32_t *seq_ids, int32_t num_seqs, int32_t ntok,
                    const kvp_step_io *io, const kvp_attn_desc *desc, void *workspace,
                    size_t ws_bytes, size_t *ws_needed, void *stream);

/*
 * kvp_decode_step in two halves, so that the host work of step i + 1 can run
 * while the device runs step i (each sequence appending ntok tokens per step
 * is known before the step's K/V and q are):
 *
 *   kvp_decode_step_plan: the checks of kvp_decode_step that involve the pool,
 *     then the append's bookkeeping (the sequences grow by ntok tokens at once:
 *     slots and copy-on-write copies are assigned) and the attention plan over
 *     the grown sequences, packed into `plan`.  No device work.  *ws_needed
 *     (may be NULL) receives the workspace bytes the run will need.
 *   kvp_decode_step_run: steps 1-4 of kvp_decode_step for that plan, with the
 *     plan's upload into `workspace` right before the append's write.
 *
 * Both kvp_decode_step and kvp_decode_step_run, when the step's inputs are
 * already on the device or in mapped host memory (KVP_STEP_HOST_MAPPED), the
 * pool holds bf16 pages, the append has at most 64 tokens and 16
 * copy-on-write blocks, its copies need not come first (see seq_append_batch)
 * and the plan has at most 24 KB, make steps 1-2 and the
 * plan upload one kernel: the new K/V go straight into their pool slots (from
 * host memory when mapped; d_k_new / d_v_new are then left unwritten), q to
 * d_q, and the plan, carried in the kernel's parameters, into the workspace;
 * attention and merge follow.
 *
 * A plan object (kvp_step_plan_create; kvp_step_plan_destroy frees it) holds
 * one planned step at a time and is reused from step to step.  Planning a
 * plan that is still waiting for its run is KVP_ERR_INVALID, since its
 * tokens are already in the sequences.  Between plan and run no call may
 * change the planned sequences or free blocks; appends and attention on other
 * sequences may run (but no append to a sequence that was cut back in a page
 * which it shared with a planned one: the run still copies that page).
 * `workspace` belongs to the run until the stream passes its kernels, as for
 * every attention call.  The run takes its device
 * buffers from io as kvp_decode_step does (num_seqs and ntok are the plan's).
 * Errors: the plan call as kvp_decode_step's (KVP_ERR_INVALID, KVP_ERR_OOM;
 * nothing changed); the run returns KVP_ERR_INVALID for a plan that is not
 * waiting for its run or bad buffers (the plan then stays ready), and
 * KVP_ERR_WORKSPACE when ws_bytes is short: the inputs' copies and the
 * append's write are enqueued, nothing else; the plan is used up.
 */
typedef struct kvp_step_plan kvp_step_plan;

kvp_step_plan *kvp_step_plan_create(void);
void kvp_step_plan_destroy(kvp_step_plan *plan);
int kvp_decode_step_plan(kvp_pool *pool, const int32_t *seq_ids, int32_t num_seqs, int32_t ntok,
                         const kvp_attn_desc *desc, kvp_step_plan *plan, size_t *ws_needed);
int kvp_decode_step_run(kvp_step_plan *plan, const kvp_step_io *io, void *workspace, size_t ws_bytes,
                        void *stream);

/* ------------------------------------------- bounded caches and drafts */

/*
 * Attention over a sliding window and the first few tokens (attention sinks)
 * of each paged sequence, for decode steps and prompt chunks: sequence s has
 * q_lens[s] query tokens (host; NULL: one each; 0 allowed), the last of its
 * seq_lens[s] cached tokens (append first, then attend).  The query at
 * position p sees the keys j <= p with j > p - window or j < sinks;
 *   out = softmax(q k^T * scale) v over them, lse the natural log-sum-exp.
 * window >= 1 (one at least as long as the sequence gives causal attention),
 * sinks >= 0, lengths below 2^31 - 128.  q, out: [L][T][Hq][d] bf16 and lse:
 * [L][T][Hq] fp32 (or NULL), sequence after sequence, T = sum of q_lens.
 * block_tables, seq_lens, desc, workspace and errors as for
 * paged_decode_attention, ws_bytes >= kvp_window_workspace_size() for the
 * same arguments; pages must be bf16.
 * Weights are rounded to bf16 before they meet V, as in the other attention
 * calls; their sum and the log-sum-exp are not.  The workspace grows with the
 * keys in view; where queries see more than 8192 of them it holds d + 1 floats
 * per 8192 keys, query token, head and layer, and KVP_ERR_INVALID says that
 * 2^31 such rows or more would be needed for one layer and kv head.
 * With desc->use_sharing, batches of one query token per sequence read a
 * block that several of them share and see once.  Tokens that no query of the
 * call sees do not matter; those that one sees must hold finite K and V (for
 * the others they enter the products with weight 0).  A sequence may have no
 * cached token (q_lens[s] = 0 then).  KVP_ERR_STATE while `stream` is being
 * captured: the plan is uploaded from host memory.
 */
size_t kvp_window_workspace_size(const kvp_attn_desc *desc, const int32_t *block_tables,
                                 const int32_t *seq_lens, const int32_t *q_lens, int32_t num_seqs,
                                 int32_t max_blocks, int32_t window, int32_t sinks);
int paged_window_attention(const void *q, const int32_t *q_lens, const void *k_pool,
                           const void *v_pool, const int32_t *block_tables,
                           const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks,
                           int32_t window, int32_t sinks, const kvp_attn_desc *desc, void *out,
                           float *lse, void *workspace, size_t ws_bytes, void *stream);

/*
 * Accumulated attention weight of every cached token, from the log-sum-exp
 * that an attention call left: for each layer, sequence s, kv head h and
 * cached token t < seq_lens[s],
 *   mass_out[l][s][h][t] = decay * mass_in[l][s][h][t]
 *       + sum over the sequence's query tokens i at positions >= t, and over
 *         the query heads of kv head h, of exp(scale * q_i . k_t - lse_i).
 * Sequence s has q_lens[s] query tokens (host; NULL: one each; 0 allowed),
 * the last of its seq_lens[s] cached tokens, as in a decode step (1) or after
 * a prompt chunk; q [L][T][Hq][d] bf16 and lse [L][T][Hq] fp32 (natural log,
 * of attention over every cached token up to the query's own) hold them
 * sequence after sequence, T = sum of q_lens.  A row whose lse is -inf adds
 * nothing.  mass_in and mass_out are device fp32, [L][num_seqs][Hkv]
 * [mass_stride], mass_stride >= the longest sequence; they are one buffer or
 * do not overlap.
 * mass_in holds the first prev_lens[s] tokens (host; NULL: seq_lens - q_lens,
 * the tokens before this step's); later ones count as 0, and with mass_in
 * NULL all do.  Entries of mass_out from seq_lens[s] on are left as they are.
 * K is read once, V not at all.  Pages must be bf16; block_tables, seq_lens,
 * desc (use_sharing is not used) and workspace as for
 * paged_decode_attention, ws_bytes >= kvp_mass_workspace_size().  Cached keys
 * must be finite.  KVP_ERR_INVALID also for layers * kv heads above 65535;
 * KVP_ERR_STATE while `stream` is being captured.
 */
size_t kvp_mass_workspace_size(const kvp_attn_desc *desc, const int32_t *block_tables,
                               const int32_t *seq_lens, const int32_t *q_lens, int32_t num_seqs,
                               int32_t max_blocks);
int kvp_attention_mass(const void *q, const int32_t *q_lens, const float *lse, const void *k_pool,
                       const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs,
                       int32_t max_blocks, const kvp_attn_desc *desc, float decay,
                       const float *mass_in, const int32_t *prev_lens, float *mass_out,
                       int64_t mass_stride, void *workspace, size_t ws_bytes, void *stream);

/*
 * Evicts all but `budget` tokens of each of n distinct sequences, chosen per
 * layer and kv head by accumulated attention weight: the first n_sink and the
 * last n_recent tokens stay, and of the others the heaviest, among equal
 * weights the lowest position (a NaN weighs less than anything).  mass is
 * device fp32 [L][n][Hkv][mass_stride].  The kept tokens' K and V move, in
 * order, to the sequence's first slots (which token a slot holds then differs
 * by layer and head, while the table and the length, `budget`, are the
 * sequence's), and the blocks past them are released.  kept (device int32
 * [L][n][Hkv][budget]) receives the positions that the kept tokens had,
 * mass_out (device, laid out like mass; NULL: not wanted; mass itself or
 * apart from it) their weights in the first `budget` entries (0 for -0, and any
 * NaN for a NaN).  A sequence of at most `budget` tokens stays as it is: kept =
 * 0, 1, ... then -1, its weights copied.  A slot of an evicted sequence is no
 * token position any more: attention over all of it is what it was, but its
 * blocks do not belong in a prefix cache, and a sliding window over it counts
 * slots.
 * Pages that another sequence or the prefix cache also holds are not written:
 * the sequence gets fresh blocks for them, except for pages that hold sink
 * tokens alone, which stay shared.  Sharing is judged at the start of the
 * call, so sequences of one call that share a page with each other both get
 * fresh blocks.
 * seqs is a host array; ws_bytes >= seq_evict_workspace_size(), workspace
 * 256-byte aligned, kept until the stream has passed the call.  All or
 * nothing: KVP_ERR_OOM (no free blocks), KVP_ERR_INVALID and KVP_ERR_STATE (a
 * pool without K/V storage or of 4-bit pages, or a stream being captured)
 * change nothing; after KVP_ERR_CUDA from a launch the bookkeeping stands.
 * (For this and the two calls above, the legacy default stream counts as
 * captured while a stream that synchronises with it is.)
 */
size_t seq_evict_workspace_size(const kvp_pool *pool, const int32_t *seqs, int32_t n, int32_t budget);
int seq_evict(kvp_pool *pool, const int32_t *seqs, int32_t n, const float *mass, int64_t mass_stride,
              int32_t budget, int32_t n_sink, int32_t n_recent, int32_t *kept, float *mass_out,
              void *workspace, size_t ws_bytes, void *stream);

/*
 * Which drafted tokens the target accepts, and the token after them: the step
 * between tree_verify_attention and seq_accept_draft ("CAST", section on
 * speculative decoding: the target model accepts one path of the draft tree).
 * Sequence b has n_draft <= 64 draft nodes with tree_parent [B][n_draft] as
 * for tree_verify_attention (a chain: -1, 0, 1, ...) and draft_tokens
 * [B][n_draft].  Row 0 of target is the target's next-token distribution
 * after the context, row 1 + i that after draft node i; row r of draft is the
 * distribution from which the children of that point were drawn, one after
 * the other in node order (rows of nodes without children are not read).
 * From the root on, the children of the current node are tried in node
 * order: child i with token x is accepted when
 *     u_accept[b][i] * q(x) * Z < p(x) - c * q(x),
 * with c = 0, Z = 1 at the first child and, after each rejection, c += Z,
 * then Z = sum over the vocabulary of max(p - c q, 0); an accepted child
 * becomes the current node.  When none is (left), next_token is the first
 * token at which the running sum of max(p - c q, 0) exceeds u_next[b] times
 * its whole (p itself if nothing is left).  The tokens are then distributed
 * as the target's own samples.  draft NULL stands for drafts that were chosen
 * outright (greedy, or the best few): a child is accepted when
 * u_accept * Z < p(x), and a rejection sets p(x) to 0 and takes it off Z.
 * accepted [B]: the last accepted node or -1 (seq_accept_draft's argument);
 * n_accepted [B]: how many; next_token [B] (-1 if a row of p is all zero).
 *
 * target / draft: device fp32 probabilities (each row sums to about 1; NaN
 * and negative entries count as 0, entries above 1 as 1), element (b, r, x) at b * batch_stride +
 * r * row_stride + x, strides >= 0 (0: one distribution for all).
 * tree_parent, draft_tokens, u_* in [0, 1), and the outputs: device, int32
 * and fp32.  A parent outside [-1, i) makes a root; a node whose token is
 * outside [0, vocab) is left out.  Sums over the vocabulary are exact to
 * 2^-60 an entry (a residual of smaller entries alone is nothing left), so the
 * result does not depend on the row's split over the GPU.  One kernel, no
 * workspace; may be captured into a graph.
 */
int kvp_draft_verify(const float *target, int64_t target_batch_stride, int64_t target_row_stride,
                     const float *draft, int64_t draft_batch_stride, int64_t draft_row_stride,
                     const int32_t *tree_parent, const int32_t *draft_tokens, const float *u_accept,
                     const float *u_next, int32_t batch, int32_t n_draft, int32_t vocab,
                     int32_t *accepted, int32_t *n_accepted, int32_t *next_token, void *stream);

/* --------------------------------- rotated appends, beams, sparse attention */

/*
 * The rotation of keys and queries by position: of each head's d values the
 * first rot_dim (even, 2 .. min(d, 256)) are rot_dim / 2 pairs, pair i being
 * dims (i, i + rot_dim / 2) or, with `interleaved`, (2 i, 2 i + 1).  At
 * position p it becomes
 *   (x cos a - y sin a, y cos a + x sin a) * scale,   a = p * freq_i,
 * freq_i = freqs[i] (host, radians per position, rot_dim / 2 of them; read
 * during the call) or, with freqs NULL, base ^ (-2 i / rot_dim).  The other
 * dims stay as they are.  scale 0 counts as 1.  Angles are reduced in 64-bit
 * fixed point: freq_i / 2 pi modulo 1, a double's quotient, times the whole
 * number p wraps exactly.  So an angle is off by 2^-33 of a turn and by p times
 * the quotient's rounding (2^-56 of a turn for a frequency of 1: 2^-33 at
 * position 2^23, 2^-25 at 2^31), and by what freq_i itself was rounded.
 */
typedef struct {
    int32_t rot_dim;
    int32_t interleaved;
    const double *freqs;
    double base;
    float scale;
} kvp_rope_desc;

/*
 * seq_append_batch with the rotation on the way: the keys go into their pages
 * rotated (in 32 bits, rounded to bf16 once; 4-bit pages quantise those bf16
 * keys as seq_append would), the values as they are, and q (device bf16
 * [L][sum ntoks][num_q_heads][d], or NULL) is rotated into q_out (q itself or
 * apart from it).  positions: device int32 [sum ntoks], any values (evicted
 * caches, whose slots are no positions; draft trees, whose nodes share
 * depths), or NULL: the slots that the tokens take in their sequences.
 * Semantics, copy-on-write and errors of seq_append_batch, all or nothing;
 * KVP_ERR_INVALID also for a rotation outside the above, KVP_ERR_STATE also
 * while `stream` is being captured (a replay would write the same slots again).
 * One kernel for appends of up to 512 sequences, 512 copied blocks and 4096
 * pages (two where the copies come first, see seq_append_batch); no workspace.
 * A batch whose ntoks are all 0 does nothing.  After KVP_ERR_CUDA from a launch
 * the bookkeeping stands.
 */
int seq_append_rope(kvp_pool *pool, int32_t nseq, const int32_t *seqs, const int32_t *ntoks, const void *k,
                    const void *v, const kvp_rope_desc *rope, const int32_t *positions, const void *q, void *q_out,
                    int32_t num_q_heads, void *stream);

/* Beam search's reordering of sequences: sequence dst[i] becomes a
 * copy-on-write fork of what sequence src[i] was before the call (host arrays
 * of n live sequences; each dst at most once, a src as often as wanted, dst
 * and src may name the same sequences; dst[i] == src[i] leaves it as it is).
 * Host bookkeeping only, no K/V moves.  What the dst sequences held before is
 * released, the last of them first, each table from its last entry.
 * KVP_ERR_INVALID changes nothing. */
int seq_reorder(kvp_pool *pool, const int32_t *dst, const int32_t *src, int32_t n);

/*
 * Attention over pages that a cheap score selects for each query.  The four
 * calls below take the batch on the DEVICE: block_tables int32 [num_seqs]
 * [max_blocks] and seq_lens int32 [num_seqs] as kvp_export_tables leaves
 * them, so that they need no plan and no workspace, synchronise nothing and
 * may be captured into a graph, which then follows tables and lengths as they
 * change.  Query rows: q_start NULL means one query token a sequence, num_q =
 * num_seqs; else q_start (device int32 [num_seqs + 1], ascending from 0) gives
 * sequence s the rows q_start[s] .. q_start[s + 1] - 1, which are its last
 * cached tokens (append first); rows from q_start[num_seqs] up to num_q (a
 * padded batch) are left as they are.  A query at position p sees the tokens
 * up to p, in the pages 0 .. p / bs of its sequence; page j is table entry j.
 * A length above max_blocks * bs counts as that.  desc as for
 * paged_decode_attention (bf16 pages; use_sharing is not used), layers * kv
 * heads at most 65535.  These calls, kvp_beam_select and kvp_state_reorder
 * return KVP_ERR_STATE on the legacy default stream while a stream that
 * synchronises with it is being captured.
 *
 * kvp_page_bounds: for every layer, kv head and page that holds one of the
 * last n_new tokens of a sequence (n_new >= its length: every page), the
 * smallest and the largest key value per dim over the page's tokens, into
 * bounds, device bf16 [L][NB][Hkv][2][d] (smallest, then largest), indexed by
 * block like the pool: pages that sequences share have their bounds once.
 * Call it after every append (n_new = tokens appended) and after
 * seq_accept_draft, seq_evict.  NaN keys give NaN bounds.  A page listed
 * with different lengths (a shared page that one sequence was cut back in)
 * must be refreshed by the longer one's call last.  Table entries outside
 * [0, NB) are passed over.  At most 65535 sequences a call.
 */
int kvp_page_bounds(const void *k_pool, const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs,
                    int32_t max_blocks, int32_t n_new, const kvp_attn_desc *desc, void *bounds, void *stream);

/*
 * kvp_page_scores: for each layer l, query row t, kv head h and page j that
 * the query sees,
 *   scores[l][t][h][j] = scale * sum over the query heads of h and the dims i
 *                        of max(q_i * smallest_i, q_i * largest_i),
 * which no sum of the group's scaled scores over a key of the page exceeds.
 * q: bf16 [L][num_q][Hq][d]; scores: fp32 [L][num_q][Hkv][score_stride],
 * score_stride >= max_blocks; entries of other pages are left as they are.
 * The query values are summed in 32 bits and enter the products whole.
 * Pages whose table entry is outside [0, NB) score -inf; queries or bounds
 * that are not finite give scores that are not.
 */
int kvp_page_scores(const void *q, const int32_t *q_start, int32_t num_q, const void *bounds,
                    const int32_t *block_tables, const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks,
                    const kvp_attn_desc *desc, float *scores, int64_t score_stride, void *stream);

/*
 * kvp_page_select: for each layer, query row and kv head, `budget` pages out
 * of those that the query sees: the first n_sink, the last n_recent and, of
 * the others, those with the highest scores, among equal ones the lowest page
 * (a NaN is higher than anything, so that it shows).  selected: int32
 * [L][num_q][Hkv][budget], the pages in ascending order, then -1 where the
 * query sees fewer.  n_sink + n_recent <= budget.  scores may come from
 * anywhere; those of pages that the query does not see are not read.
 */
int kvp_page_select(const float *scores, int64_t score_stride, const int32_t *q_start, int32_t num_q,
                    const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks, const kvp_attn_desc *desc,
                    int32_t budget, int32_t n_sink, int32_t n_recent, int32_t *selected, void *stream);

/*
 * paged_sparse_attention: out = softmax(q k^T * scale) v over the tokens up
 * to the query's own in the pages selected[l][t][h][0 .. budget), lse the
 * natural log-sum-exp.  Entries that are negative, or name a page that the
 * query does not see or whose table entry is outside [0, NB), are passed
 * over; their order does not matter, and a page named twice counts twice.  A
 * row without keys gives out 0 and lse -inf.  q, out (apart from q): bf16
 * [L][num_q][Hq][d]; lse: fp32 [L][num_q][Hq] or NULL.  Keys and values that a
 * row sees should be finite: a NaN among them shows in its results, an infinite
 * value as an infinity or a NaN.  Other slots do not matter, whatever they hold
 * (but neighbouring rows of a chunk are done together, and one by one, several
 * times slower, where one of them names a page twice or a page that one of them
 * names holds a value that is not finite, or one of their scores is beyond 2^28).
 * Chunks share their pages' reads in tables of at most 4096 pages; wider ones are
 * done row by row, some four times slower, however short their sequences.  Softmax
 * statistics and sums are fp32; a weight meets V as two bf16 numbers, which keep 16
 * bits of it.  Repeated calls give equal bits.  A kernel's wait that runs out,
 * which no input causes, leaves NaN in its rows.
 */
int paged_sparse_attention(const void *q, const int32_t *q_start, int32_t num_q, const void *k_pool,
                           const void *v_pool, const int32_t *block_tables, const int32_t *seq_lens,
                           int32_t num_seqs, int32_t max_blocks, const int32_t *selected, int32_t budget,
                           const kvp_attn_desc *desc, void *out, float *lse, void *stream);

/*
 * Beam search's selection: for each of `groups` requests the n_out best
 * continuations out of beams x vocab, best first.  Row r = group * beams +
 * beam of logits (device, type KVP_F32 / KVP_BF16 / KVP_F16, element x of row
 * r at r * row_stride + x) and scores[r] (fp32, the log-probability so far)
 * give
 *   score(r, x) = scores[r] + logits[r][x] - log(sum over y of exp(logits[r][y]));
 * equal scores go by the lower row, then the higher logit, then the lower x.
 * finished (bytes [groups][beams], or NULL): a row with a nonzero byte goes
 * on with pad_token alone at its score as it is; its logits are not read.  A
 * row whose scores[r] is not finite, or whose logits hold a NaN, +inf or
 * nothing above -inf, gives no continuation, nor does a logit of -inf (a
 * masked token).  out_scores fp32, out_rows (r) and out_tokens (x) int32, all
 * [groups][n_out]; where there are fewer than n_out continuations: -inf, -1
 * and -1.  out_scores may be scores itself where n_out == beams; otherwise the
 * results do not overlap scores or finished.  1 <= beams <= 128, 1 <= n_out <=
 * 128.  Exponentials and sums of 32 of them are fp32, sums of those pairs of fp32
 * numbers (48 bits): a row's log-sum-exp is within 2^-21.  Scores are compared as
 * such pairs and rounded to fp32 at the end; they hold 48 bits of the row's largest
 * logit, too (x in magnitude: 2^-47 x), so that a row masked whole by its type's
 * lowest value, instead of -inf, scores about 0: give such a row a score of -inf.
 * A score below fp32's range counts as none.
 * workspace: 16-byte aligned, ws_bytes >= kvp_beam_workspace_size() (0 on
 * invalid input), its content does not matter; one call at a time.  May be
 * captured into a graph.
 */
enum { KVP_F32 = 0, KVP_BF16 = 1, KVP_F16 = 2 };
size_t kvp_beam_workspace_size(int32_t groups, int32_t beams, int32_t vocab, int32_t n_out);
int kvp_beam_select(const void *logits, int32_t logits_type, int64_t row_stride, const float *scores,
                    const uint8_t *finished, int32_t pad_token, int32_t groups, int32_t beams, int32_t vocab,
                    int32_t n_out, float *out_scores, int32_t *out_rows, int32_t *out_tokens, void *workspace,
                    size_t ws_bytes, void *stream);

/*
 * The beams' states after kvp_beam_select: dst[o][i] = src[o][index[i]] for o
 * < outer, i < n_dst, rows of row_bytes bytes, src [outer][n_src] and dst
 * [outer][n_dst] rows (token histories, kvp_attention_mass weights, recurrent
 * states; sequences of the pool go through seq_reorder).  index: device int32
 * [n_dst]; a row whose index is outside [0, n_src) is left as it is.  src and
 * dst do not overlap.
 */
int kvp_state_reorder(const void *src, void *dst, const int32_t *index, int64_t outer, int32_t n_src, int32_t n_dst,
                      int64_t row_bytes, void *stream);

/* Reads (and clears) the device error word that the last attention call on
 * this workspace left; synchronises `stream`.  *err_out = 0 when clean. */
int kvp_device_error(void *workspace, void *stream, int32_t *err_out);

/* Host-side view of the decode plan (no device work; for tests and tools):
 * work items, row tiles, 64-token KV tiles and partial rows per (layer, kv
 * head), and the bytes of distinct (block, valid tokens) one call reads over
 * all layers (K and V rows in the pool's format: d bf16 values, or d/2 code
 * bytes and one exponent byte), planned for a GPU with sm_count SMs.  Any out-pointer may be
 * NULL.  The plan's internal invariants (tile ranges inside the tile list
 * and within the kernels' descriptor stage, rows within each kernel's unit,
 * member intervals inside their items) are checked: KVP_ERR_STATE if one
 * fails, which would be a planner defect. */
int kvp_decode_plan_stats(const kvp_attn_desc *desc, const int32_t *block_tables,
                          const int32_t *seq_lens, int32_t num_seqs, int32_t max_blocks,
                          int32_t sm_count, int32_t *n_items, int32_t *n_row_tiles,
                          int32_t *n_kv_tiles, int32_t *n_partial_rows, int64_t *unique_kv_bytes);

/* Measurement hooks.  kvp_set_kernel_events: cudaEvent_t handles (as void*)
 * that every later attention call on this thread records on its stream
 * immediately before and after its main attention kernel (the work-item
 * kernel), so a caller can time that kernel alone; NULL, NULL turns it off.
 * kvp_kernel_launches: total kernels this library has launched in the
 * process (all threads). */
int kvp_set_kernel_events(void *before, void *after);
int kvp_kernel_launches(int64_t *n_out);

const char *kvp_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* KVP_H */
