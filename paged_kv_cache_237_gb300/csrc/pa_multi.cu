// pa_decode_tree and pa_decode_cross: checks, workspace and dispatch.
#include <climits>

#include "pa_multi.cuh"

namespace {

using namespace pa::host;

// Up to how many rows per sequence and KV head the pass for few rows is the faster one,
// in blocks of 16, by what the host knows.  bf16: the few-rows pass reads K and V once per
// block, the tcgen05 pass once per 256 rows; by blocks and the longest context.  Measured,
// few rows against tcgen05 (us): 32 sequences of 2000..4000 tokens, 8 KV heads of 128:
// 16 rows 87 / 100, 24 rows 140 / 100; 64 sequences of 350..700 tokens: 16 rows
// 43 / 68, 32 rows 68 / 68, 48 rows 85 / 71 (heads of 64: 51 / 59, 64 rows 63 / 59);
// 8 sequences of 450..900: 64 rows 32 / 35, 96 rows 36 / 36.
// fp32: items of 16 against 32 rows, 32 sequences of 2000..4000 tokens, 8 KV heads of 128:
// 16 rows 189 / 286, 24 rows 337 / 286 (sums left in the tensor core).
constexpr int kFewBlocks = 6;
int few_blocks(const pa::MultiParams &p, int head_dim, bool f32) {
    if (f32) return 1;
    int blocks = 1;
    while (blocks < kFewBlocks && 1.0 * (blocks + 1) * p.num_seqs * p.num_kv_heads * p.ctx_cap * (head_dim / 64) <= 1.2e6)
        ++blocks;
    return blocks;
}

// The passes of a batch.  One, by the average rows, where no sequence can have many more
// or the caller gave no bound on that (max_query_len 0).  Where one may have more than
// kFewBlocks blocks and twice the average, the sequences of few rows run in one pass and
// the others in another, if both are work enough (blocks of 16 rows x tokens x heads) to pay
// for two more launches; else in one, by which of them are more.  Measured, all in the
// few-rows pass / all in the tcgen05 pass / in both (us), a chunk beside requests of one
// token with contexts of 200 to 1500: 127 and a chunk of 1500 over 8000, 32 heads of 128:
// 1230 / 1011 / 530, fp32 5390 / 5280 / 4690; 127 and 600 over 1500, 32 / 8 heads: 231 /
// 239 / 162, fp32 607 / 671 / 562; 16 heads of 64: 124 / 212 / 137; 7 and 600, 32 / 8
// heads: 202 / 73 / 89; 127 and 1200, 4 / 1 heads: 222 / 69 / 83.
int launch_passes(pa::MultiParams p, int head_dim, int max_query_len, bool f32, int dev, cudaStream_t st) {
    const auto pass = [&](bool few) {
        if (f32) return pa::launch_multi_f32(p, head_dim, few, dev, st);
        return few ? pa::launch_multi_few(p, head_dim, dev, st) : pa::launch_multi_mma(p, head_dim, dev, st);
    };
    p.queries_above = 0;
    p.queries_most = INT_MAX;
    // rows behind the last sequence are none of the batch's
    long long queries = p.num_tokens, most_queries = max_query_len < p.num_tokens ? max_query_len : p.num_tokens;
    if (max_query_len > 0 && queries > most_queries * p.num_seqs) queries = most_queries * p.num_seqs;
    const long long rows = (queries * p.group + p.num_seqs - 1) / p.num_seqs, longest = most_queries * p.group;
    const int most = 16 * few_blocks(p, head_dim, f32);
    if (longest <= 16 * kFewBlocks || longest <= 2 * rows) return pass(rows <= most);
    const double block = 1.0 * p.num_kv_heads * p.ctx_cap * (head_dim / 64);
    if (longest / 16 * block < 1.5e6 || p.num_seqs * block < 0.9e6) return pass(rows <= most && longest <= 16ll * p.num_seqs);
    if (most >= p.group) {
        p.queries_most = most / p.group;
        const int rc = pass(true);
        if (rc != PA_OK) return rc;
        p.queries_above = p.queries_most;
        p.queries_most = INT_MAX;
    }
    return pass(false);
}

struct MultiLayout {
    size_t ml, acc, bytes;   // where the rows' maxima and sums start, where their values do, and the workspace's size
    int rows;                // rows of a place for a partial (the pass for few rows: its own)
};

// num_tokens rows of `group` heads: an item has no more rows than that.
MultiLayout multi_layout(int num_tokens, int group, int head_dim, bool f32) {
    const long long need = static_cast<long long>(num_tokens) * group;
    const auto least = [&](int most) { return static_cast<int>(need < most ? need : most); };
    MultiLayout l;
    // tcgen05: its streams keep sums there before, a half each
    l.rows = f32 ? least(pa::kMultiF32Rows) : 2 * least(pa::kMultiMmaRows / 2);
    size_t slots = 2ull * (f32 ? pa::kMultiFewCtas : pa::kMultiMmaCtas) * l.rows;
    if (!f32) {   // the pass for few rows has more CTAs with fewer rows each; both fit
        const size_t few = 2ull * pa::kMultiFewCtas * least(16);
        slots = slots > few ? slots : few;
    }
    l.ml = kWorkspaceHeader;   // pa_decode's counter stays as it is: the workspace may serve both
    l.acc = l.ml + align256(slots * 2 * sizeof(float));
    l.bytes = l.acc + align256(slots * head_dim * sizeof(float));
    return l;
}

int decode_multi(void *out, const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                 const int32_t *context_lens, const int32_t *query_start, const uint64_t *mask, int see,
                 int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale, int num_tokens,
                 int mask_words, const pa_decode_args *a) {
    if (!a) return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: args is NULL");
    if (a->num_seqs < 0 || num_tokens < 0) return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: negative sizes");
    if (a->dtype != PA_F32 && a->dtype != PA_BF16)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: bad dtype");
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: num_q_heads must be a positive multiple of num_kv_heads");
    if (head_dim != 64 && head_dim != 128)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_tree/cross: head_dim must be 64 or 128");
    if (block_size != 16 && block_size != 32)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_tree/cross: block_size must be 16 or 32");
    if (a->phase != PA_PHASE_ALL || a->simt || a->k_new || a->v_new || a->slot_mapping || a->partition_size)
        return pa_fail(PA_ERR_UNSUPPORTED,
                       "pa_decode_tree/cross: phase, simt, k_new, v_new, slot_mapping and partition_size must be 0");
    if (a->num_blocks <= 0 || a->max_blocks_per_seq <= 0 || a->max_context_len < 0 || a->max_query_len < 0)
        return pa_fail(PA_ERR_INVALID_ARG,
                       "pa_decode_tree/cross: bad num_blocks, max_blocks_per_seq, max_context_len or max_query_len");
    if (a->num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: null tensor pointer");
    if (mask ? mask_words < 1 || mask_words > PA_TREE_MAX_NODES / 64 : mask_words != 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree: mask_words must be 1 to 16, and 0 without a mask");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: out, q and caches must be 16-byte aligned");
    const uintptr_t words = reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
                            reinterpret_cast<uintptr_t>(query_start) | reinterpret_cast<uintptr_t>(a->dev_status);
    if ((words & 3u) || (reinterpret_cast<uintptr_t>(mask) & 7u))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_tree/cross: misaligned pointer");
    const long long total_rows = static_cast<long long>(a->num_blocks) * num_kv_heads * block_size;
    if (total_rows >= INT_MAX || static_cast<long long>(num_tokens) * num_q_heads >= INT_MAX / 2)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_tree/cross: 2^31 or more cache rows, or 2^30 or more query rows");
    const MultiLayout lay = multi_layout(num_tokens, num_q_heads / num_kv_heads, head_dim, a->dtype == PA_F32);
    if (!a->workspace || a->workspace_bytes < lay.bytes || !aligned16(a->workspace))
        return pa_fail(PA_ERR_WORKSPACE,
                       "pa_decode_tree/cross: workspace missing, unaligned or smaller than pa_decode_tree_workspace_size()");
    pa::MultiParams p{};
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.mask = reinterpret_cast<const unsigned long long *>(mask);
    p.part_ml = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + lay.ml);
    p.part_acc = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + lay.acc);
    p.status = a->dev_status;
    p.num_seqs = a->num_seqs;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = a->num_blocks;
    p.width = a->max_blocks_per_seq;
    const long long table_cap = static_cast<long long>(a->max_blocks_per_seq) * block_size;
    const long long cap = a->max_context_len < table_cap ? a->max_context_len : table_cap;
    p.ctx_cap = static_cast<int>(cap < INT_MAX - 1024 ? cap : INT_MAX - 1024);   // positions of a whole tile fit an int
    p.words = mask_words;
    p.see = see;
    p.slot_rows = lay.rows;
    p.total_rows = static_cast<int>(total_rows);
    p.scale_log2 = scale * 1.4426950408889634f;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: no CUDA device");
    if (sm_count(dev) <= 0) return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cannot query the SM count");
    const cudaStream_t st = static_cast<cudaStream_t>(a->stream);
    return launch_passes(p, head_dim, a->max_query_len, a->dtype == PA_F32, dev, st);
}

}  // namespace

extern "C" size_t pa_decode_tree_workspace_size(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim) {
    if (num_tokens <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || head_dim <= 0)
        return 0;
    const int group = num_q_heads / num_kv_heads;
    const size_t bf16 = multi_layout(num_tokens, group, head_dim, false).bytes;
    const size_t f32 = multi_layout(num_tokens, group, head_dim, true).bytes;
    return bf16 > f32 ? bf16 : f32;
}

extern "C" int pa_decode_tree(void *out, const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                              const uint64_t *tree_mask, int num_q_heads, int num_kv_heads, int head_dim,
                              int block_size, float scale, int num_tokens, int mask_words,
                              const pa_decode_args *args) {
    PaTraceRange trace("pa_decode_tree");
    return decode_multi(out, q, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask,
                        tree_mask ? pa::kSeeMask : pa::kSeeChain, num_q_heads, num_kv_heads, head_dim, block_size,
                        scale, num_tokens, mask_words, args);
}

extern "C" int pa_decode_cross(void *out, const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *block_tables, const int32_t *context_lens, const int32_t *query_start,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale,
                               int num_tokens, const pa_decode_args *args) {
    PaTraceRange trace("pa_decode_cross");
    return decode_multi(out, q, k_cache, v_cache, block_tables, context_lens, query_start, nullptr, pa::kSeeAll,
                        num_q_heads, num_kv_heads, head_dim, block_size, scale, num_tokens, 0, args);
}
