/*
 * pa.h -- C ABI of the GB300 (sm_103a) paged decode-attention library.
 *
 * The operations follow four pages on PagedAttention:
 *  [P1] "PagedAttention", ayinedjimi-consultants.fr glossary, "Definition";
 *  [P2] "PagedAttention — Gestion memoire pour LLM a long contexte",
 *       analyticslegends.ai, "Pourquoi c'est important", "Points cles",
 *       "Termes employes sur cette page";
 *  [P3] "PagedAttention", robocikowo.com, "Jak dziala", "Komponenty",
 *       "Pulapki implementacyjne", "Zlozonosc obliczeniowa";
 *  [P4] "PagedAttention et RadixAttention : parlons de KV Cache", aitalk.it,
 *       "PagedAttention : la memoire comme un systeme d'exploitation".
 *
 * Conventions for every call:
 *  - Pointers named *_cache, q, out, k, v, block_tables, context_lens,
 *    slot_mapping, src_dst_pairs, workspace and dev_status are DEVICE pointers
 *    owned by the caller.  The library never allocates device memory.
 *  - `stream` is a cudaStream_t passed as void*; NULL means the legacy default
 *    stream.  Device calls only enqueue work and return before it runs.  They
 *    launch on the calling thread's current CUDA device: every device pointer
 *    (and the stream) must belong to it.
 *  - Every call returns PA_OK (0) or a negative PA_ERR_* code; nothing is
 *    thrown across the ABI.  pa_last_error_string() describes the last failure
 *    of the calling thread.
 *  - Argument errors are reported before anything is enqueued.  Errors that
 *    depend on device data (a block id outside the pool, a context length
 *    beyond the table, a slot outside the pool, a bad copy pair) cannot be
 *    seen on the host: kernels skip the offending access, OR a PA_STATUS_* bit
 *    into *dev_status (when not NULL) and carry on, so no input can make a
 *    kernel read or write outside the buffers described here.
 *
 * Layouts (row-major, element type = `dtype` unless stated):
 *   k_cache, v_cache  [num_blocks][num_kv_heads][block_size][head_dim]
 *   q, out            [num_seqs][num_q_heads][head_dim]
 *   block_tables      [num_seqs][max_blocks_per_seq] int32 (physical ids)
 *   context_lens      [num_seqs] int32
 *   k, v (new tokens) [num_tokens][num_kv_heads][head_dim]
 *   slot_mapping      [num_tokens] int64, slot = block * block_size + offset
 *   src_dst_pairs     [num_pairs][2] int64 (src block, dst block)
 * (the 4-bit caches of the *_q4 calls have a layout of their own, below)
 * Query head h attends with KV head h / (num_q_heads / num_kv_heads).
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- return codes ---------------------------------------------------- */
#define PA_OK 0
#define PA_ERR_INVALID_ARG -1 /* null pointer, bad size, inconsistent shape */
#define PA_ERR_UNSUPPORTED -2 /* valid request the library has no kernel for */
#define PA_ERR_CUDA -3        /* a CUDA runtime/driver call failed */
#define PA_ERR_BAD_INDEX -4   /* host-visible id out of range */
#define PA_ERR_NO_BLOCKS -5   /* block manager: free pool exhausted */
#define PA_ERR_REFCOUNT -6    /* block manager: unknown sequence or id misuse */
#define PA_ERR_WORKSPACE -7   /* workspace missing or too small */

/* ---- element types ---------------------------------------------------- */
#define PA_F32 0  /* IEEE fp32 */
#define PA_BF16 1 /* bfloat16 (fp32 accumulation inside the kernels) */

/* ---- device status bits (OR-ed into *dev_status by the kernels) -------- */
#define PA_STATUS_BAD_BLOCK_ID 1    /* block table entry outside [0, num_blocks) */
#define PA_STATUS_BAD_CONTEXT_LEN 2 /* context_lens[i] < 0 or beyond the table or max_context_len */
#define PA_STATUS_BAD_SLOT 4        /* slot_mapping entry >= num_blocks * block_size, or (fused
                                       write) not the slot of the sequence's last position */
#define PA_STATUS_BAD_PAIR 8        /* copy pair out of range, or its dst is another pair's src/dst */
#define PA_STATUS_WAIT_TIMEOUT 16   /* a bounded wait for staged data gave up */
#define PA_STATUS_SHORT_LIST 32     /* pa_build_tables: fewer block ids or token rows than the lengths need */
#define PA_STATUS_BAD_TREE 64       /* query_start not increasing or outside the rows, a parent that is not an earlier
                                       node, or a tree of more nodes than its mask or PA_TREE_MAX_NODES holds */

/* ---- decode attention --------------------------------------------------
 * [P3] "Jak dziala" / "Komponenty": the attention kernel reads the K/V cache
 * of each sequence through its block table of fixed-size physical blocks;
 * [P4] step two: the table makes the scattered blocks look like one
 * continuous sequence, and paging leaves attention's result unchanged.
 *
 * For every sequence i and query head h, with n = context_lens[i] and KV head
 * kv = h / (num_q_heads / num_kv_heads):
 *   out[i][h] = sum_t softmax_t(scale * q[i][h] . K_i[t]) V_i[t],  t < n,
 *   K_i[t] = k_cache[block_tables[i][t / block_size]][kv][t % block_size].
 * n == 0 gives a zero row.  Cache slots at or past n in the last block are
 * never used, whatever they hold (NaN included).
 *
 * Long contexts are cut into partitions of `partition_size` tokens that are
 * processed independently and merged by a second pass (split-K), which needs
 * `workspace`.  With a workspace, the bf16 pass also hands out its work items
 * through a counter held there, so CTAs that finish early take more.
 * Arithmetic: fp32 accumulation; for PA_BF16 the products q.K and p.V run on
 * bf16 tensor-core MMAs, p entering as the sum of two bf16 parts (about 16
 * significant bits); for PA_F32 on fp32 FMAs.  Results are deterministic for
 * a given input and partition size (which CTA runs an item does not change
 * its arithmetic).
 */
typedef struct pa_decode_args {
    int num_seqs;           /* S >= 0 */
    int max_blocks_per_seq; /* row stride (in entries) of block_tables, >= 1 */
    int num_blocks;         /* physical blocks in each cache tensor, >= 1 */
    int dtype;              /* PA_F32 or PA_BF16: q, k_cache, v_cache and out */
    int partition_size;     /* tokens per split-K partition, multiple of 16 in
                               [16, 4096]; 0 picks 512 */
    int max_context_len;    /* host upper bound of context_lens[i]; longer
                               entries are clamped and flagged */
    void *workspace;        /* device scratch, 256-byte aligned is best: the
                               partition pass's work counter in its first 8
                               bytes, then the split-K partials; may be NULL
                               when max_context_len <= partition_size.  No
                               part needs to start at zero (see
                               skip_counter_reset).  One workspace serves one
                               call at a time: two calls that may run at the
                               same time on the GPU (different streams with no
                               ordering between them) must not share it, since
                               they would race on its work counter and
                               partials.  Calls ordered on one stream may
                               share it. */
    size_t workspace_bytes; /* >= pa_decode_workspace_size(...) */
    int32_t *dev_status;    /* optional device word for PA_STATUS_* bits */
    void *stream;           /* cudaStream_t */
    int phase;              /* PA_PHASE_ALL (0): both passes.  PA_PHASE_PARTITIONS
                               (1): only the per-partition pass (final rows of
                               single-partition sequences, partials of the
                               others).  PA_PHASE_REDUCE (2): only the merge of
                               the partials; it must follow phase 1 on the same
                               stream with identical arguments.  Splitting lets a
                               caller time or overlap the two passes. */
    /* Optional fused cache write (all three NULL to disable).  Sequence i's new
     * token is its last one, position context_lens[i] - 1: the call writes
     * k_new[i] / v_new[i] ([num_seqs][num_kv_heads][head_dim], dtype) into
     * k_cache / v_cache at slot_mapping[i] and attends with those values, the
     * same result as pa_reshape_and_cache followed by pa_decode, in one launch
     * fewer.  slot_mapping[i] < 0 skips sequence i's write.  A slot that is not
     * the slot of position context_lens[i] - 1 is not written and sets
     * PA_STATUS_BAD_SLOT.  When enabled, k_cache and v_cache are written.
     * (Pages: [P3] "Jak dziala", [P4] step three.) */
    const void *k_new;
    const void *v_new;
    const int64_t *slot_mapping;
    int simt;               /* PA_BF16 only: nonzero computes q.K and p.V with
                               plain fp32 FMAs (p kept in fp32, 8 query heads
                               per work item) instead of tensor-core MMAs;
                               0, the default, uses the MMAs.  Same results
                               within the tolerance; for comparison and for
                               callers who want fp32 products throughout. */
    int skip_counter_reset; /* The bf16 pass hands out work items through a
                               counter at the start of the workspace.  Each
                               call leaves that counter zero when it completes,
                               and by default also zeroes it first with a
                               cudaMemsetAsync on `stream` (8 bytes).  Nonzero
                               skips that memset (one operation, a few
                               microseconds, fewer per call): valid once the
                               counter is zero, i.e. after any completed call
                               on this workspace, or when the caller zeroed its
                               first 8 bytes. */
    int max_query_len;      /* pa_decode_tree and pa_decode_cross (others do not
                               look at it): host upper bound of a sequence's
                               queries, 0 for unknown.  It decides which kernels
                               run, never what they compute: with it, a batch of
                               short and long ones runs as both need. */
} pa_decode_args;

#define PA_PHASE_ALL 0
#define PA_PHASE_PARTITIONS 1
#define PA_PHASE_REDUCE 2

/* Supported: head_dim in {64, 128}; block_size in {16, 32}; num_q_heads a
 * multiple of num_kv_heads.  Returns PA_ERR_UNSUPPORTED otherwise. */
int pa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
              const int32_t *block_tables, const int32_t *context_lens,
              int num_q_heads, int num_kv_heads, int head_dim, int block_size,
              float scale, const pa_decode_args *args);

/* Bytes of workspace pa_decode needs for these sizes (0 when no sequence can
 * span more than one partition).  partition_size 0 means the default.  A
 * helper of this library's split-K design: the pages describe no kernel-level
 * split of long contexts, so this call has no counterpart there. */
size_t pa_decode_workspace_size(int num_seqs, int num_q_heads, int head_dim,
                                int max_context_len, int partition_size);

/* ---- decode attention with a sliding window ------------------------------
 * pa_decode over a part of each sequence: with n = context_lens[i], only
 * positions t >= n - window (the last `window` tokens, the newest included)
 * and t < num_sinks (the first tokens, which stay visible) take part; the rest
 * have weight zero, whatever their cache slots hold (NaN included).  window >=
 * 1 (PA_ERR_INVALID_ARG otherwise; a window of n or more attends to
 * everything), num_sinks >= 0.  No counterpart in the pages.
 *
 * Only blocks that hold a visible position are looked up and read, so the
 * blocks between the sinks and the window may have been given back: their
 * table entries may hold anything.  (To the caller's own pool and tables: a
 * pa_bm sequence keeps its blocks until it is freed, and pa_build_tables takes
 * a sequence's whole list and flags ids that are not blocks.)  The fused cache write works as in
 * pa_decode.  args->simt must be 0 for PA_BF16 (PA_ERR_UNSUPPORTED).
 * args->partition_size 0 picks by the batch's sizes (equal partitions of what
 * the window shows).  Everything else, types, layouts, checks, determinism, as
 * pa_decode; the workspace is sized by what is visible. */
int pa_decode_window(void *out, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_tables, const int32_t *context_lens,
                     int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                     float scale, int window, int num_sinks, const pa_decode_args *args);

/* Bytes of workspace pa_decode_window needs (0 when no sequence can show it
 * more than one partition, and for a window or sink count it refuses). */
size_t pa_decode_window_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                       int max_context_len, int partition_size, int window, int num_sinks,
                                       int dtype);

/* ---- decode attention without a caller workspace ----------------------
 * The paper has no counterpart to this call; it is a convenience of this
 * library.
 *
 * For callers that cannot allocate device memory -- a plugin or framework
 * that owns every allocation and passes the library only its inputs and
 * outputs, or a hot path where a cudaMalloc, which may synchronise the
 * device, is not allowed.  Same computation, arguments and results as
 * pa_decode; args->workspace and args->workspace_bytes are ignored.  The
 * split-K scratch is a fixed array of PA_NOALLOC_WORKSPACE_BYTES (64 MiB)
 * inside the library, which every GPU that loads the library keeps until the
 * process exits.  The call allocates and frees nothing.
 *  - Sizes whose pa_decode_workspace_size() exceeds PA_NOALLOC_WORKSPACE_BYTES
 *    are rejected with PA_ERR_WORKSPACE before anything is enqueued.
 *  - The first call on a device that needs the scratch looks up its device
 *    address (cudaGetSymbolAddress) with that device current; make that first
 *    call before any stream capture on the device.  The address is kept for
 *    the life of the process: after cudaDeviceReset (or anything else that
 *    destroys the device's primary context) it is stale, and this call must
 *    not be used on that device again.
 *  - Arguments are checked as pa_decode checks them, before the scratch is
 *    sized; a bad partition_size, block_size or head_dim gives the same code
 *    as there.
 *  - Every call on a device shares the one array, which keeps the last call's
 *    contents; no part of it needs to start at zero (each call writes every
 *    partial it reads, and the work counter is reset before each pass unless
 *    skip_counter_reset is set; the array starts at zero and each completed
 *    call leaves the counter zero, so setting it is valid here).
 *  - Calls that overlap on the GPU -- on different streams without ordering
 *    between them -- race on the array. */
#define PA_NOALLOC_WORKSPACE_BYTES (64u * 1024u * 1024u)

int pa_decode_noalloc(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, const int32_t *context_lens,
                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                      float scale, const pa_decode_args *args);

/* ---- cache write ------------------------------------------------------
 * [P3] "Jak dziala" and [P4] step three: blocks are filled as the sequence
 * grows.  For each token t with slot s = slot_mapping[t] >= 0:
 *   k_cache[s / block_size][h][s % block_size][:] = k[t][h][:]  (all h), same
 *   for v.  Negative slots are padding and are skipped.  Bit-exact copy.
 * Slots must be distinct; two tokens naming one slot race. */
int pa_reshape_and_cache(const void *k, const void *v, void *k_cache, void *v_cache,
                         const int64_t *slot_mapping, int num_tokens, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, int dtype,
                         int32_t *dev_status, void *stream);

/* ---- block copy (copy-on-write) ----------------------------------------
 * [P3] "Komponenty": shared prefix blocks carry reference counts and are
 * duplicated only when one sharer modifies them; [P4] step four.
 * For each pair p: block dst_p of both caches (every KV head and slot)
 * becomes a bit-exact copy of block src_p.  A dst that appears twice, or that
 * is also another pair's src, is rejected on the device: that pair is not
 * copied and PA_STATUS_BAD_PAIR is set.  src == dst is a no-op. */
int pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *src_dst_pairs, int num_pairs,
                   int num_kv_heads, int head_dim, int block_size, int num_blocks, int dtype,
                   int32_t *dev_status, void *stream);

/* ---- block swap between two pools (device cache <-> host memory) --------
 * [P2] "Points cles" / "Termes employes sur cette page" (page eviction): when
 * GPU memory runs out, cold pages are written to CPU RAM and read back when
 * needed.  For each pair p, block dst_p of (dst_k, dst_v) becomes a bit-exact
 * copy of block src_p of (src_k, src_v): every KV head and slot.  The two
 * pools share the block geometry (num_kv_heads, block_size, head_dim, dtype)
 * and must be different allocations; each may be device memory or pinned host
 * memory the device can address (cudaHostAlloc / cudaHostRegister; checked
 * with cudaPointerGetAttributes, anything else is PA_ERR_INVALID_ARG).
 * src_dst_pairs must be device-accessible as well.  A pair out of range, or a
 * dst named twice, is skipped and sets PA_STATUS_BAD_PAIR. */
int pa_swap_blocks(const void *src_k, const void *src_v, void *dst_k, void *dst_v,
                   const int64_t *src_dst_pairs, int num_pairs, int src_num_blocks, int dst_num_blocks,
                   int num_kv_heads, int head_dim, int block_size, int dtype, int32_t *dev_status,
                   void *stream);

/* ---- host block manager -----------------------------------------------
 * [P3] "Komponenty": a block manager hands out and takes back physical
 * blocks from a free pool and keeps per-block reference counts for shared
 * prefixes; [P2] "Pourquoi c'est important": blocks are allocated on demand
 * and released one by one when a request ends; [P1] "Definition": freed
 * blocks are reused at once, and parallel samples share the prompt's blocks
 * until they diverge.
 *
 * Host memory only; not thread-safe (one manager per thread, or external
 * locking).  Allocation order: block 0 first, then 1, 2, ...; a freed block
 * is the next handed out (a LIFO pool); a sequence releases its blocks from
 * the last logical block to the first.  Failed calls leave the state as it
 * was.  Sequence ids are any non-negative int. */
typedef struct pa_bm pa_bm;

pa_bm *pa_bm_create(int num_blocks, int block_size); /* NULL on bad sizes */
void pa_bm_destroy(pa_bm *bm);

/* New sequence holding num_tokens tokens in ceil(num_tokens / block_size)
 * fresh blocks.  PA_ERR_NO_BLOCKS if the pool is short. */
int pa_bm_add_seq(pa_bm *bm, int seq_id, int num_tokens);

/* child shares every block of parent (refcount + 1 each). */
int pa_bm_fork(pa_bm *bm, int parent_id, int child_id);

/* Reserve the slot for the sequence's next token.  If the last block is full
 * a fresh block is appended.  If it is partial and shared (refcount > 1) it
 * is replaced by a fresh block, its refcount drops by one, and
 * (*cow_src, *cow_dst) name the copy the caller must run before writing
 * (pa_copy_blocks); otherwise both are -1.  *slot = block * block_size +
 * offset. */
int pa_bm_append_slot(pa_bm *bm, int seq_id, int64_t *slot, int32_t *cow_src, int32_t *cow_dst);

/* Drop the sequence; each of its blocks loses one reference and returns to
 * the pool at zero. */
int pa_bm_free_seq(pa_bm *bm, int seq_id);

/* Keep the sequence's first num_tokens tokens (at most what it holds): blocks past
 * them lose one reference, the last first, as in pa_bm_free_seq.  For drafted tokens
 * that were not accepted.  A keyed block that is then only partly the sequence's keeps
 * its key until pa_bm_append_slot writes into it (or, shared, copies it first). */
int pa_bm_trim_seq(pa_bm *bm, int seq_id, int num_tokens);

/* Copy the sequence's physical block ids into out[0..cap).  Returns the
 * number of blocks (>= 0), or PA_ERR_INVALID_ARG if cap is too small. */
int pa_bm_block_table(const pa_bm *bm, int seq_id, int32_t *out, int cap);

/* Tokens the sequence holds, or a negative error code. */
int pa_bm_num_tokens(const pa_bm *bm, int seq_id);
int pa_bm_num_free(const pa_bm *bm);   /* free plus cached (both can be handed out) */
int pa_bm_refcount(const pa_bm *bm, int block); /* negative if out of range */

/* ---- automatic prefix caching (chained block hash, tenant salt) --------
 * [P4] "Deux couches, pas deux rivaux": every full block is keyed by a hash of
 * its parent block's key, its own tokens and optional extra data, so equal
 * token prefixes give equal key chains and find blocks already computed;
 * [P4] "Au-dela": a per-tenant salt mixed into the key keeps tenants apart.
 *
 * key_0 = H(0, salt, tokens[0..bs)), key_i = H(key_{i-1}, salt, tokens of block i),
 * H = 64-bit FNV-1a over the little-endian bytes of (parent key u64, salt u64,
 * each token as int32).  A key hit also compares the stored tokens, so hash
 * collisions cannot alias blocks.  Only full blocks are keyed.  A keyed block
 * whose refcount drops to zero stays cached (its K/V intact) and can be reused
 * by a later request until the pool runs short: allocation takes a free block
 * first, then evicts the least recently released cached block. */

/* New sequence of n tokens: leading full blocks whose keys are cached are
 * shared (refcount + 1); the rest are fresh, and the fresh full blocks are
 * keyed.  *num_cached_tokens = tokens whose K/V are already present (the
 * caller must compute and write the others before any other request can use
 * the newly keyed blocks).  PA_ERR_NO_BLOCKS leaves the state unchanged. */
int pa_bm_add_seq_cached(pa_bm *bm, int seq_id, const int32_t *tokens, int n, uint64_t salt,
                         int *num_cached_tokens);

/* Key the sequence's full blocks that are not keyed yet (for example after
 * decoding filled a block); tokens[0..n) are the sequence's tokens, n equal
 * to its length.  A block whose key already names another cached block stays
 * private.  Returns the number of blocks newly keyed, or an error code. */
int pa_bm_register_blocks(pa_bm *bm, int seq_id, const int32_t *tokens, int n, uint64_t salt);

/* Blocks held only by the cache (refcount 0, reusable on a hit). */
int pa_bm_num_cached(const pa_bm *bm);

/* Move a sequence from one manager to another (a device pool and a host pool
 * of the same block size): every block gets a fresh block in `to`, the pairs
 * (from block, to block) are written to pairs[2 * k], pairs[2 * k + 1] for the
 * caller's pa_swap_blocks, and the blocks in `from` are released.  All of the
 * sequence's blocks must be unshared (refcount 1): PA_ERR_REFCOUNT otherwise.
 * PA_ERR_NO_BLOCKS if `to` is short; *num_pairs = blocks moved; cap is the
 * room of pairs in pairs.  On failure nothing changes. */
int pa_bm_move_seq(pa_bm *from, pa_bm *to, int seq_id, int64_t *pairs, int cap, int *num_pairs);

/* Batched decode-step helper: append one slot to each of n sequences in order.
 * slots[k] receives the slot of seq_ids[k]; copy pairs are appended to
 * cow_pairs (int64 [n][2], host) and their count stored in *num_pairs.
 * Stops at the first failure and returns its code; *num_done tells how many
 * sequences were served (their effects stay). */
int pa_bm_append_slots(pa_bm *bm, const int32_t *seq_ids, int n, int64_t *slots,
                       int64_t *cow_pairs, int *num_pairs, int *num_done);

/* Padded block tables and lengths for a batch, ready for pa_decode:
 * tables [n][max_blocks_per_seq] (unused entries = -1), context_lens [n]. */
int pa_bm_build_tables(const pa_bm *bm, const int32_t *seq_ids, int n, int32_t *tables,
                       int max_blocks_per_seq, int32_t *context_lens);

/* Block ids of a batch without padding: sequence by sequence, each one's ids in
 * logical order, into out[0..cap), and (when not NULL) every sequence's tokens
 * into context_lens [n].  Returns the number of ids (PA_ERR_INVALID_ARG if cap
 * is too small).  The block_ids and context_lens of pa_build_tables, which
 * lays the padded tables out on the device: this list is the smaller upload. */
int pa_bm_flat_blocks(const pa_bm *bm, const int32_t *seq_ids, int n, int32_t *out, int cap,
                      int32_t *context_lens);

/* ---- batch tables on the device ------------------------------------------
 * The device counterpart of pa_bm_build_tables, with the step's slot map: from
 * each sequence's length and one flat list of block ids it lays out what the
 * cache write and the decode calls read.  No counterpart in the pages, which
 * say nothing of how tables reach the device.
 *
 * With n_i = context_lens[i] tokens in the cache after this step, the last
 * c_i = new_lens[i] of them new, b_i = ceil(n_i / block_size),
 * first_i = b_0 + ... + b_(i-1) and start_i = c_0 + ... + c_(i-1):
 *   block_tables[i][j] = block_ids[first_i + j] for j < b_i, else -1
 *                                             ([num_seqs][max_blocks_per_seq])
 *   query_start[i] = start_i, query_start[num_seqs] = start_num_seqs = total
 *   row start_i + r (r < c_i) is position p = n_i - c_i + r of sequence i:
 *     positions[row] = p
 *     slot_mapping[row] = block * block_size + p % block_size, with
 *                         block = block_ids[first_i + p / block_size]
 *   rows total .. max_tokens-1: slot_mapping = -1 (padding, which the cache
 *   writes skip), positions = 0.
 * positions and query_start may be NULL; slot_mapping may be NULL when
 * max_tokens is 0, and block_ids when num_ids is 0.  The outputs must not
 * overlap the inputs.  One launch; the sums are taken by every CTA for itself,
 * so there is no workspace and calls on different streams do not meet.
 *
 * Device data is checked as everywhere: a length outside [0,
 * max_blocks_per_seq * block_size] or a new length outside [0, n_i] is clamped
 * and sets PA_STATUS_BAD_CONTEXT_LEN; a block id outside [0, num_blocks) gives
 * table entry -1 and slots -1 and sets PA_STATUS_BAD_BLOCK_ID; ids past
 * num_ids likewise, and rows past max_tokens are dropped, with
 * PA_STATUS_SHORT_LIST. */
int pa_build_tables(int32_t *block_tables, int64_t *slot_mapping, int32_t *positions, int32_t *query_start,
                    const int32_t *block_ids, const int32_t *context_lens, const int32_t *new_lens,
                    int num_seqs, int max_blocks_per_seq, int max_tokens, int num_ids, int block_size,
                    int num_blocks, int32_t *dev_status, void *stream);

/* ---- 4-bit cache -----------------------------------------------------------
 * K and V held in 4 bits a value, with a step and a minimum for every group of
 * group_size (32 or 64) values of a head row.  Each cache is a byte array
 *   [num_blocks][num_kv_heads][page_bytes],
 *   page_bytes = block_size * (head_dim / 2 + 4 * head_dim / group_size),
 * 16-byte aligned.  A page holds its block_size rows' codes (head_dim / 2
 * bytes each), then their parameters: [block_size][head_dim / group_size]
 * pairs (step s, minimum m) of bf16.  Code c of a group stands for s * c + m.
 * Within a row's codes, values go in units of four (16 bits, the first value
 * in the lowest bits); with W = head_dim / 64, unit 16 w + 8 h + g (w < W,
 * h < 2, g < 8) is half h of 32-bit word g * W + w.  (The order gives each lane
 * of the decode kernel its share of a row in one load.)
 *
 * Quantisation of a group, every operation rounded to fp32 unless stated, so
 * that every writer gives the same bits:
 *   m = min(x) rounded down to bf16, +0 where that is zero;  far = max(x) - m;
 *   s = 0 if far = 0, else max(far / 15 rounded up to bf16, 2^-126);
 *   c = round_half_even((x - m) * (1 / s)), 0 where s = 0.
 * Then |s c + m - x| <= s / 2 (up to fp32 rounding).  A group that holds a NaN,
 * an infinity or a magnitude of 2^126 or more stands for NaN throughout (m =
 * NaN, s = 0), as an unquantised cache would let it show.
 *
 * Whole blocks are bytes to pa_copy_blocks and pa_swap_blocks: pass dtype
 * PA_BF16 and head_dim = page_bytes / block_size / 2 with the block size. */

/* Bytes of one page; 0 if the sizes are not supported (head_dim 64 or 128,
 * block_size 16 or 32, group_size 32 or 64). */
size_t pa_q4_page_bytes(int head_dim, int block_size, int group_size);

/* Quantise and write new rows: for each token t with slot s = slot_mapping[t]
 * >= 0, head rows k[t][h] and v[t][h] ([num_tokens][num_kv_heads][head_dim],
 * dtype) go to row s % block_size of pages (s / block_size, h).  Padding (slot
 * < 0), bad slots and repeated slots as in pa_reshape_and_cache. */
int pa_reshape_and_cache_q4(const void *k, const void *v, void *k_cache, void *v_cache,
                            const int64_t *slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
                            int block_size, int group_size, int num_blocks, int dtype, int32_t *dev_status,
                            void *stream);

/* Read rows back as values s * c + m, rounded once to dtype: k[t][h], v[t][h]
 * from the slots of slot_mapping (any order, repeats allowed).  Rows with a
 * negative slot, or (flagged) one past the pool, are left as they were. */
int pa_gather_q4(void *k, void *v, const void *k_cache, const void *v_cache, const int64_t *slot_mapping,
                 int num_tokens, int num_kv_heads, int head_dim, int block_size, int group_size,
                 int num_blocks, int dtype, int32_t *dev_status, void *stream);

/* Decode attention over the 4-bit cache: pa_decode (window == 0) or
 * pa_decode_window (window >= 1) with K_i[t], V_i[t] the values s * c + m that
 * the cache holds.  args->dtype is the type of q and out.  A block id out of
 * range reads as zeros (flagged).
 * Arithmetic: scores, exponentials, maxima and sums are fp32, a row's sums in
 * two levels, 4096 tokens at a time.  The products with the codes run on tensor
 * cores, whose operands are rounded first:
 *  - PA_BF16: q enters exactly, no finer than 2^-35 of its row's largest magnitude;
 *    sums of q over a group, which meet K's minima, as two bf16 parts (16 bits); a
 *    weight times its value's step as one fp16 number (2^-11 relative); a sum of 16
 *    tokens' codes or of a group's is cut off at about 17 bits of its largest term.
 *  - PA_F32: q enters as two fp16 parts (2^-22 relative, no finer than 2^-40 of its
 *    row's largest magnitude), a weight times its step as two as well.
 * A weight times its step is held relative to M, the largest such product so far
 * among its group of values and the query heads of one KV head that are worked
 * on together (4, 8 or 16): no finer than 2^-32 M (PA_BF16) or 2^-43 M (PA_F32), for
 * each token.  Finite results need |scale * q| below 2^115.
 * args->partition_size is 0 (the library picks) or a multiple of 32 in
 * [32, 1024]: contexts of up to so many tokens are never split, longer ones are
 * cut wherever that makes the GPU's warps' shares equal, no finer than that.
 * Results are deterministic for given inputs, sizes and GPU.  No counter is
 * used, so skip_counter_reset says nothing, and a workspace may be shared with
 * pa_decode under the same rule of one call at a time; args->simt must be 0 and
 * k_new, v_new and slot_mapping NULL (PA_ERR_UNSUPPORTED):
 * pa_reshape_and_cache_q4 writes the step's tokens. */
int pa_decode_q4(void *out, const void *q, const void *k_cache, const void *v_cache,
                 const int32_t *block_tables, const int32_t *context_lens, int num_q_heads, int num_kv_heads,
                 int head_dim, int block_size, int group_size, float scale, int window, int num_sinks,
                 const pa_decode_args *args);

/* Bytes of workspace pa_decode_q4 needs (0 when no sequence can span more than
 * one partition). */
size_t pa_decode_q4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                   int max_context_len, int partition_size, int window, int num_sinks);

/* ---- several queries per sequence ------------------------------------------
 * The queries of all sequences lie end to end: q and out are
 * [num_tokens][num_q_heads][head_dim] and sequence i owns rows query_start[i] ..
 * query_start[i + 1] - 1 (int32 [num_seqs + 1], as pa_build_tables makes it), c_i
 * of them, none included.  Rows that belong to no sequence (padding behind the
 * last one) are not read and left as they were.  No counterpart in the pages.
 *
 * pa_decode_tree: verification of drafted tokens.  The queries are the last c_i of
 * the n_i = context_lens[i] tokens, whose K/V the cache already holds: query r is
 * position n_i - c_i + r.  It sees every position below n_i - c_i, and position
 * n_i - c_i + j if bit j of its row of tree_mask is set (uint64
 * [num_tokens][mask_words], bit j % 64 of word j / 64; positions past the words
 * are not seen).  A row may see anything, itself left out; pa_build_tree makes the
 * rows of a tree.  With tree_mask NULL (mask_words 0) the drafted tokens are a
 * chain: query r sees position n_i - c_i + j for j <= r, as a prompt's chunk does.
 *
 * pa_decode_cross: the queries (any number, of a decoder step or prompt, or the
 * beams of one request) see all n_i = context_lens[i] tokens of a cache that holds
 * another sequence: an encoder's states.
 *
 * out = softmax over the seen t of scale * (q . K[t]), times V[t]; a row that sees
 * nothing (n_i = 0, an empty mask) is zero.  What a row does not see has weight
 * zero, whatever its cache slots hold (NaN included).  A value that it sees and that is
 * not finite makes its column of the row what the formula gives: an infinity that
 * infinity, infinities of both signs or a NaN a NaN (and an infinity whose weight is below
 * 2^-100 of the row's largest may come out as a NaN).
 * Arithmetic: scores, maxima, sums and results are fp32.  PA_BF16: q, K and V enter
 * exactly, weights as two bf16 parts (16 bits), whatever the batch.  PA_F32: q, K, V and
 * weights as two tf32 parts each, three of their four products, off by 2^-21 of a
 * product at most and to either side: results as far off as with fp32 operations.  Sums
 * over the tokens are divided at their end, so that values near fp32's largest may
 * overflow in them.
 *
 * args as for pa_decode: num_seqs, max_blocks_per_seq, num_blocks, dtype,
 * max_context_len (longer entries are clamped and flagged), max_query_len (worth giving
 * wherever sequences differ in their queries or q has padding: without it the kernels are
 * picked by num_tokens / num_seqs, and always by max_context_len, so a close bound is the
 * better one), dev_status, stream, and
 * a workspace of pa_decode_tree_workspace_size bytes (both calls), which needs no
 * zeros and may be shared with pa_decode under the same rule of one call at a time
 * (its first 256 bytes are left as they are).  phase, simt, partition_size and the
 * fused write's pointers must be 0 (PA_ERR_UNSUPPORTED).  A sequence whose
 * rows of query_start run backwards or leave [0, num_tokens] has no queries
 * (flagged PA_STATUS_BAD_TREE); one with c_i > n_i in pa_decode_tree gets zero rows
 * (PA_STATUS_BAD_CONTEXT_LEN); a block id out of range reads as zeros (flagged).
 * Rows of two sequences must not overlap.
 * Results are deterministic for given inputs, sizes and GPU. */
#define PA_TREE_MAX_NODES 1024 /* nodes of one tree; mask_words is at most 16 */

int pa_decode_tree(void *out, const void *q, const void *k_cache, const void *v_cache,
                   const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                   const uint64_t *tree_mask, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                   float scale, int num_tokens, int mask_words, const pa_decode_args *args);

int pa_decode_cross(void *out, const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                    int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale, int num_tokens,
                    const pa_decode_args *args);

/* Bytes of workspace that both calls need for up to num_tokens rows; it does not
 * grow with the contexts. */
size_t pa_decode_tree_workspace_size(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim);

/* ---- trees of drafted tokens ------------------------------------------------
 * Sequence i's tree has nodes 0 .. c_i - 1, its rows of the batch as above.
 * parents [num_tokens] holds each node's parent within its tree: an earlier node,
 * or -1 for none.
 *
 * pa_build_tree: tree_mask row of node r = bit r and its parent's row; positions
 * [num_tokens] (may be NULL) = n_i - c_i + depth, depth counted from 0.  Trees of
 * more than 64 * mask_words nodes are flagged (PA_STATUS_BAD_TREE): the nodes past
 * that see nothing.  A parent that is not an earlier node counts as none (flagged).
 * Rows of no sequence are left as they were.  2^30 or more words of masks:
 * PA_ERR_UNSUPPORTED. */
int pa_build_tree(uint64_t *tree_mask, int32_t *positions, const int32_t *parents, const int32_t *query_start,
                  const int32_t *context_lens, int num_seqs, int num_tokens, int mask_words, int32_t *dev_status,
                  void *stream);

/* pa_accept_tree: the path that the target model agrees with.  Node 0 holds the
 * sequence's newest token, the others are drafted; draft_tokens [num_tokens] are the
 * nodes' tokens and target_tokens [num_tokens] the target model's choice behind
 * each.  a_0 = 0, and a_(j+1) is the lowest child of a_j whose token is
 * target_tokens[a_j], as long as there is one and j + 1 < max_accepted.  With the
 * path's L nodes (0 for a sequence that drafted nothing):
 *   accepted_lens[i] = L;   accepted_nodes[i][j] = a_j, -1 from L on;
 *   next_tokens[i] = target_tokens[a_(L-1)], -1 if L = 0;
 *   new_lens[i] = n_i - c_i + L, the sequence's length once its path has moved;
 *   slot_pairs[i][j] = (slot of position n_i - c_i + a_j, slot of n_i - c_i + j)
 *   where a_j != j and j < L, else (-1, -1): the pairs of pa_move_rows
 * ([num_seqs][max_accepted], int32; slot_pairs int64 [num_seqs][max_accepted][2]).
 * parents NULL is a chain.  max_accepted is 1 to PA_TREE_MAX_NODES; nodes past
 * PA_TREE_MAX_NODES are not accepted (flagged).  c_i > n_i, or n_i beyond the
 * table: flagged, L = 0 and new_lens[i] = n_i. */
int pa_accept_tree(int32_t *accepted_lens, int32_t *accepted_nodes, int32_t *next_tokens, int32_t *new_lens,
                   int64_t *slot_pairs, const int32_t *draft_tokens, const int32_t *target_tokens,
                   const int32_t *parents, const int32_t *query_start, const int32_t *context_lens,
                   const int32_t *block_tables, int num_seqs, int num_tokens, int max_accepted,
                   int max_blocks_per_seq, int block_size, int num_blocks, int32_t *dev_status, void *stream);

/* pa_move_rows: K/V rows from slot to slot of one cache, every KV head.
 * slot_pairs [num_groups][pairs_per_group][2] are (source, destination); pairs with
 * a negative slot are skipped, and ones past the pool too (PA_STATUS_BAD_SLOT).
 * Within a group every source is read before any destination is written, so a row
 * may be both.  Destinations must be distinct, and no slot of one group may be a
 * destination of another.  A group's rows of one head must fit in 48 KB (96 rows of
 * 128 fp32 values, 192 of 128 bf16; PA_ERR_UNSUPPORTED): a smaller bound than
 * pa_accept_tree's on max_accepted.  Longer paths go in several calls, pairs j from
 * the first on: since a_j >= j, no call's sources are destinations of one before. */
int pa_move_rows(void *k_cache, void *v_cache, const int64_t *slot_pairs, int num_groups, int pairs_per_group,
                 int num_kv_heads, int head_dim, int block_size, int num_blocks, int dtype, int32_t *dev_status,
                 void *stream);

/* ---- self-test of the bounded wait ----------------------------------------
 * Every wait of the decode kernels on a barrier for staged data (pa_decode and
 * pa_decode_window; pa_decode_q4's copies need none) gives up after about two
 * seconds, sets PA_STATUS_WAIT_TIMEOUT and lets the kernel finish, so a copy
 * that never lands cannot hang the GPU.  This call runs that same wait in a
 * one-thread kernel on a barrier that nothing completes, with a limit of
 * limit_us microseconds (1..1000000), and ORs PA_STATUS_WAIT_TIMEOUT into
 * *dev_status when it gives up (it always does).  For tests of that path. */
int pa_selftest_wait_timeout(int32_t *dev_status, int limit_us, void *stream);

/* ---- misc --------------------------------------------------------------- */
const char *pa_last_error_string(void); /* thread-local, never NULL */
int pa_version(void);                   /* (major << 16) | minor */

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
