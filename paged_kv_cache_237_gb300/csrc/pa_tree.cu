// Trees of drafted tokens for sm_103a: ancestor bits and positions from
// parents, the path the target model agrees with, and the move of that path's
// cache rows to where the sequence goes on (include/pa.h states the formulas).
//
// All three are bound by latency (launch and two or three dependent loads) at
// a decode step's sizes; the move is a byte mover like the cache write.  Measured:
// masks and positions of 8 trees of 5..32 nodes 7.2 us, of 500 trees of up to 250
// nodes 8.2 us (the host's part of a call is 7); accepted paths and moves of 4
// sequences with the write of their rows before it, three launches: 13.5 us on the
// GPU, 24 as calls; of 250 sequences 28.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kMaxNodes = PA_TREE_MAX_NODES;

// Rows start .. start + c - 1 of the batch's drafted tokens are sequence i's
// last c of n; c > n, a length below zero or rows outside [0, num_tokens) are
// bad (the sequence then counts as one that drafted nothing).
struct Drafted {
    int n, c, start;
};

__device__ __forceinline__ Drafted drafted(const int32_t *query_start, const int32_t *context_lens, int i,
                                           int num_tokens, int &flags) {
    const int a = query_start[i], b = query_start[i + 1], n = context_lens[i];
    Drafted d{n < 0 ? 0 : n, b - a, a};
    if (n < 0) flags |= PA_STATUS_BAD_CONTEXT_LEN;
    if (a < 0 || b < a || b > num_tokens) {
        flags |= PA_STATUS_BAD_TREE;
        d.c = d.start = 0;
    } else if (d.c > d.n) {
        flags |= PA_STATUS_BAD_CONTEXT_LEN;
        d.c = 0;
    }
    return d;
}

// Parents of a sequence's nodes in shared memory: -1 for none, and (flagged)
// for one that is not an earlier node.
__device__ __forceinline__ void load_parents(int16_t *s_parent, const int32_t *parents, const Drafted &d, int nodes,
                                             int &flags) {
    for (int r = threadIdx.x; r < nodes; r += blockDim.x) {
        int p = parents ? parents[d.start + r] : r - 1;
        if (p < -1 || p >= r) {
            flags |= PA_STATUS_BAD_TREE;
            p = -1;
        }
        s_parent[r] = static_cast<int16_t>(p);
    }
}

// One CTA per sequence, one thread per (node, word of its row): it walks up
// from the node, collects the ancestors that lie in its word and stops below
// it (a parent comes before its child).  The walk of word 0 goes to the root
// and so knows the depth.
__global__ void __launch_bounds__(kTreeThreads)
    build_tree_kernel(unsigned long long *mask, int32_t *positions, const int32_t *parents, const int32_t *query_start,
                      const int32_t *context_lens, int num_tokens, int words, int32_t *status) {
    __shared__ int16_t s_parent[kMaxNodes];
    int flags = 0;
    const Drafted d = drafted(query_start, context_lens, blockIdx.x, num_tokens, flags);
    const int nodes = min(d.c, min(kMaxNodes, words * 64));
    if (nodes < d.c) flags |= PA_STATUS_BAD_TREE;
    load_parents(s_parent, parents, d, nodes, flags);
    __syncthreads();
    for (int i = threadIdx.x; i < d.c * words; i += kTreeThreads) {
        const int r = i / words, w = i % words;
        unsigned long long bits = 0;
        int depth = -1;
        if (r < nodes)
            for (int at = r; at >= 64 * w; at = s_parent[at]) {
                if (at < 64 * w + 64) bits |= 1ull << (at & 63);
                ++depth;
            }
        mask[static_cast<long long>(d.start + r) * words + w] = bits;
        if (w == 0 && positions) positions[d.start + r] = d.n - d.c + max(depth, 0);
    }
    if (flags) flag_status(status, flags);
}

// One CTA per sequence.  Every node whose token is the target's choice at its
// parent offers itself as that parent's next, the lowest one wins; then one
// thread follows the path.
__global__ void __launch_bounds__(128)
    accept_tree_kernel(int32_t *accepted_lens, int32_t *accepted_nodes, int32_t *next_tokens, int32_t *new_lens,
                       int64_t *slot_pairs, const int32_t *draft, const int32_t *target, const int32_t *parents,
                       const int32_t *query_start, const int32_t *context_lens, const int32_t *tables, int num_tokens,
                       int most, int width, int block_size, int num_blocks, int32_t *status) {
    __shared__ int s_next[kMaxNodes];
    __shared__ int s_path[kMaxNodes];
    __shared__ int s_len;
    int flags = 0;
    const int i = blockIdx.x, tid = threadIdx.x;
    Drafted d = drafted(query_start, context_lens, i, num_tokens, flags);
    if (d.n > static_cast<long long>(width) * block_size) {
        flags |= PA_STATUS_BAD_CONTEXT_LEN;
        d.c = 0;
    }
    const int nodes = min(d.c, kMaxNodes);
    if (nodes < d.c) flags |= PA_STATUS_BAD_TREE;
    for (int r = tid; r < nodes; r += blockDim.x) s_next[r] = INT_MAX;
    __syncthreads();
    for (int r = tid; r < nodes; r += blockDim.x) {
        const int p = parents ? parents[d.start + r] : r - 1;
        if (p < -1 || p >= r)
            flags |= PA_STATUS_BAD_TREE;
        else if (p >= 0 && draft[d.start + r] == target[d.start + p])
            atomicMin(&s_next[p], r);
    }
    __syncthreads();
    if (tid == 0) {
        int len = 0;
        for (int at = nodes > 0 ? 0 : INT_MAX; len < most && at != INT_MAX; at = s_next[at]) s_path[len++] = at;
        s_len = len;
        accepted_lens[i] = len;
        next_tokens[i] = len > 0 ? target[d.start + s_path[len - 1]] : -1;
        new_lens[i] = d.n - d.c + len;
    }
    __syncthreads();
    const int len = s_len;
    auto slot = [&](int pos) -> int64_t {
        const int b = tables[static_cast<long long>(i) * width + pos / block_size];
        if (b < 0 || b >= num_blocks) {
            flags |= PA_STATUS_BAD_BLOCK_ID;
            return -1;
        }
        return static_cast<int64_t>(b) * block_size + pos % block_size;
    };
    for (int j = tid; j < most; j += blockDim.x) {
        const int node = j < len ? s_path[j] : -1;
        int64_t src = -1, dst = -1;
        if (node > j) {
            src = slot(d.n - d.c + node);
            dst = slot(d.n - d.c + j);
            if (src < 0 || dst < 0) src = dst = -1;
        }
        const long long at = static_cast<long long>(i) * most + j;
        accepted_nodes[at] = node;
        slot_pairs[2 * at] = src;
        slot_pairs[2 * at + 1] = dst;
    }
    if (flags) flag_status(status, flags);
}

// grid (groups, KV heads, 2): one CTA moves a group's rows of one head of K or
// V.  All of them are in shared memory before the first is written, so a row
// may be the source of one pair and the destination of another.
__global__ void __launch_bounds__(128)
    move_rows_kernel(uint4 *k_cache, uint4 *v_cache, const int64_t *pairs, int per_group, int row_vecs, int block_size,
                     long long num_slots, int32_t *status) {
    extern __shared__ uint4 s_rows[];
    const int kvh = blockIdx.y, heads = gridDim.y;
    uint4 *cache = blockIdx.z == 0 ? k_cache : v_cache;
    pairs += static_cast<long long>(blockIdx.x) * per_group * 2;
    const int total = per_group * row_vecs;
    auto row_of = [&](int64_t slot) {
        return ((slot / block_size) * heads + kvh) * block_size + slot % block_size;
    };
    bool bad = false;
    auto moves = [&](int64_t src, int64_t dst) {
        if (src < 0 || dst < 0 || src == dst) return false;
        if (src < num_slots && dst < num_slots) return true;
        bad = true;
        return false;
    };
    for (int v = threadIdx.x; v < total; v += blockDim.x) {
        const int j = v / row_vecs, c = v % row_vecs;
        const int64_t src = pairs[2 * j];
        if (moves(src, pairs[2 * j + 1])) cp_async_16(smem_addr(s_rows + v), cache + row_of(src) * row_vecs + c);
    }
    cp_async_wait_all();
    __syncthreads();
    for (int v = threadIdx.x; v < total; v += blockDim.x) {
        const int j = v / row_vecs, c = v % row_vecs;
        const int64_t dst = pairs[2 * j + 1];
        if (moves(pairs[2 * j], dst)) cache[row_of(dst) * row_vecs + c] = s_rows[v];
    }
    if (bad) flag_status(status, PA_STATUS_BAD_SLOT);
}

bool misaligned(std::initializer_list<const void *> ptrs, uintptr_t to) {
    uintptr_t all = 0;
    for (const void *p : ptrs) all |= reinterpret_cast<uintptr_t>(p);
    return (all & (to - 1)) != 0;
}

int launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace
}  // namespace pa

extern "C" int pa_build_tree(uint64_t *tree_mask, int32_t *positions, const int32_t *parents,
                             const int32_t *query_start, const int32_t *context_lens, int num_seqs, int num_tokens,
                             int mask_words, int32_t *dev_status, void *stream) {
    PaTraceRange trace("pa_build_tree");
    if (num_seqs < 0 || num_tokens < 0 || mask_words < 1 || mask_words > PA_TREE_MAX_NODES / 64)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_build_tree: bad sizes");
    if (static_cast<long long>(num_tokens) * mask_words >= INT_MAX / 2)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_build_tree: 2^30 or more words of masks");
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!tree_mask || !parents || !query_start || !context_lens)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_build_tree: null pointer");
    if (pa::misaligned({positions, parents, query_start, context_lens}, 4) || pa::misaligned({tree_mask}, 8))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_build_tree: misaligned pointer");
    pa::build_tree_kernel<<<num_seqs, pa::kTreeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<unsigned long long *>(tree_mask), positions, parents, query_start, context_lens, num_tokens,
        mask_words, dev_status);
    return pa::launched();
}

extern "C" int pa_accept_tree(int32_t *accepted_lens, int32_t *accepted_nodes, int32_t *next_tokens,
                              int32_t *new_lens, int64_t *slot_pairs, const int32_t *draft_tokens,
                              const int32_t *target_tokens, const int32_t *parents, const int32_t *query_start,
                              const int32_t *context_lens, const int32_t *block_tables, int num_seqs, int num_tokens,
                              int max_accepted, int max_blocks_per_seq, int block_size, int num_blocks,
                              int32_t *dev_status, void *stream) {
    PaTraceRange trace("pa_accept_tree");
    if (num_seqs < 0 || num_tokens < 0 || max_accepted < 1 || max_accepted > PA_TREE_MAX_NODES ||
        max_blocks_per_seq < 1 || block_size < 1 || num_blocks < 1)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_accept_tree: bad sizes");
    if (num_seqs == 0) return PA_OK;
    if (!accepted_lens || !accepted_nodes || !next_tokens || !new_lens || !slot_pairs || !query_start ||
        !context_lens || !block_tables || (num_tokens > 0 && (!draft_tokens || !target_tokens)))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_accept_tree: null pointer");
    if (pa::misaligned({accepted_lens, accepted_nodes, next_tokens, new_lens, draft_tokens, target_tokens, parents,
                        query_start, context_lens, block_tables},
                       4) ||
        pa::misaligned({slot_pairs}, 8))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_accept_tree: misaligned pointer");
    pa::accept_tree_kernel<<<num_seqs, 128, 0, static_cast<cudaStream_t>(stream)>>>(
        accepted_lens, accepted_nodes, next_tokens, new_lens, slot_pairs, draft_tokens, target_tokens, parents,
        query_start, context_lens, block_tables, num_tokens, max_accepted, max_blocks_per_seq, block_size, num_blocks,
        dev_status);
    return pa::launched();
}

extern "C" int pa_move_rows(void *k_cache, void *v_cache, const int64_t *slot_pairs, int num_groups,
                            int pairs_per_group, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                            int dtype, int32_t *dev_status, void *stream) {
    PaTraceRange trace("pa_move_rows");
    const int eb = dtype == PA_F32 ? 4 : (dtype == PA_BF16 ? 2 : 0);
    if (eb == 0) return pa_fail(PA_ERR_INVALID_ARG, "pa_move_rows: bad dtype");
    if (num_groups < 0 || pairs_per_group < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_move_rows: bad sizes");
    if (num_groups == 0 || pairs_per_group == 0) return PA_OK;
    if (!k_cache || !v_cache || !slot_pairs) return pa_fail(PA_ERR_INVALID_ARG, "pa_move_rows: null pointer");
    const long long row_bytes = static_cast<long long>(head_dim) * eb;
    if (row_bytes % 16 != 0)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_move_rows: head_dim * element size must be a multiple of 16 bytes");
    if (num_kv_heads > 65535 || pairs_per_group * row_bytes > 48 * 1024)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_move_rows: at most 65535 heads and 48 KB of one head's rows per group");
    if (pa::misaligned({k_cache, v_cache}, 16) || pa::misaligned({slot_pairs}, 8))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_move_rows: misaligned pointer");
    pa::move_rows_kernel<<<dim3(num_groups, num_kv_heads, 2), 128, static_cast<size_t>(pairs_per_group * row_bytes),
                           static_cast<cudaStream_t>(stream)>>>(
        static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), slot_pairs, pairs_per_group,
        static_cast<int>(row_bytes / 16), block_size, static_cast<long long>(num_blocks) * block_size, dev_status);
    return pa::launched();
}
