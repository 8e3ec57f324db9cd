// Decode attention over the 4-bit paged cache (include/pa.h states the
// format), partition pass for sm_103a.
//
// For a query row q and a token t with codes c, steps s_g and minima m_g:
//   q . K_t = sum_g s_g (sum_{d in g} q_d c_d) + m_g (sum_{d in g} q_d)
//   o_d     = sum_t p_t (s_g c_td + m_g)
// Work items, hand-out, the merge of the warps' states and the split-K merge
// are those of the other passes (pa_decode_common.cuh).
//
// This pass: one warp per token (two at head_dim 64), each lane owning one unit
// of four values, on plain fp32 FMAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_decode_common.cuh"
#include "pa_q4.cuh"

namespace pa {
namespace {

constexpr int kQ4Tile = 8;   // query heads per work item (at most)

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int HD, int G>
__global__ void __launch_bounds__(kWarps * 32)
    decode_q4_fma_kernel(const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache,
                         const DecodeParams p) {
    using F = Q4Format<HD, G>;
    constexpr int LPT = HD / 4;       // lanes per token
    constexpr int TPW = 32 / LPT;     // tokens a warp takes at a time
    constexpr int LD = HD + kEpiPad;
    constexpr int WARP_BYTES = (16 * LD + 32) * 4;
    __shared__ __align__(16) uint8_t smem[kWarps * WARP_BYTES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int u = lane % LPT, sub = lane / LPT;
    const int code_at = ((u % 8) * F::W + u / 16) * 4 + u / 8 % 2 * 2, group = 4 * u / G;
    SeqCursor cur{0, 0};
    griddep_wait();

    __shared__ long long s_next[2];
    const bool dynamic = p.work_ctr != nullptr;
    long long ahead = 0;
    if (dynamic && threadIdx.x == 0) ahead = gridDim.x + next_handout(p.work_ctr);
    int nb = 0;
    for (long long item = blockIdx.x;;) {
        Item it;
        if (!next_item<true>(it, cur, item, p, kQ4Tile, lane)) break;
        float q[kQ4Tile][4], o[kQ4Tile][4], m[kQ4Tile], l[kQ4Tile];
        const T *qb = static_cast<const T *>(p.q) + ((long long)it.seq * p.num_q_heads + it.qh0) * HD + 4 * u;
#pragma unroll
        for (int h = 0; h < kQ4Tile; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[h][j] = h < it.rows ? widen(qb[h * HD + j]) * p.scale_log2 : 0.f;
                o[h][j] = 0.f;
            }
            m[h] = -INFINITY;
            l[h] = 0.f;
        }
        for (int c = warp; c < it.nchunks; c += kWarps) {
            const int tok0 = it.tok_begin + c * kChunk;
            const int pos0 = token_pos<true>(p, it, tok0);
            const uint32_t mask = window_mask(p, it.n, pos0, it.tok_end - tok0);
            if (!mask) continue;
            const int phys = p.block_tables[(long long)it.seq * p.max_blocks_per_seq + pos0 / p.block_size];
            const bool good = phys >= 0 && phys < p.num_blocks;
            if (!good && lane == 0) flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
            const long long page = ((long long)(good ? phys : 0) * p.num_kv_heads + it.kvh) *
                                   ((long long)p.block_size * F::ROW_BYTES);
            for (int r0 = 0; r0 < kChunk; r0 += TPW) {
                const int r = r0 + sub;
                const bool seen = (mask >> r) & 1u;
                if (!__any_sync(kFull, seen)) continue;
                const int row = pos0 % p.block_size + r;
                uint32_t kc = 0, vc = 0, kp = 0, vp = 0;   // a block id out of range reads as zeros
                if (good && seen) {
                    const uint8_t *kb = k_cache + page, *vb = v_cache + page;
                    const int par = p.block_size * F::CODE_BYTES + row * F::PARAM_BYTES + 4 * group;
                    kc = *reinterpret_cast<const uint16_t *>(kb + row * F::CODE_BYTES + code_at);
                    vc = *reinterpret_cast<const uint16_t *>(vb + row * F::CODE_BYTES + code_at);
                    kp = *reinterpret_cast<const uint32_t *>(kb + par);
                    vp = *reinterpret_cast<const uint32_t *>(vb + par);
                }
                float kv[4], vv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    kv[j] = fmaf(static_cast<float>((kc >> (4 * j)) & 15u), q4_step(kp), q4_min(kp));
                    vv[j] = fmaf(static_cast<float>((vc >> (4 * j)) & 15u), q4_step(vp), q4_min(vp));
                }
#pragma unroll
                for (int h = 0; h < kQ4Tile; ++h) {
                    float x = fmaf(q[h][0], kv[0], fmaf(q[h][1], kv[1], fmaf(q[h][2], kv[2], q[h][3] * kv[3])));
#pragma unroll
                    for (int s = 1; s < LPT; s <<= 1) x += __shfl_xor_sync(kFull, x, s);
                    if (!seen) continue;   // the same for all lanes of a token
                    const float mn = fmaxf(m[h], x), ref = mn == -INFINITY ? 0.f : mn;
                    const float alpha = exp2f(m[h] - ref), pr = exp2f(x - ref);
                    m[h] = mn;
                    l[h] = l[h] * alpha + pr;
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[h][j] = fmaf(pr, vv[j], o[h][j] * alpha);
                }
            }
        }
        // The warp's tokens of head_dim 64 are two states: make them one.
#pragma unroll
        for (int s = LPT; s < 32; s <<= 1)
#pragma unroll
            for (int h = 0; h < kQ4Tile; ++h) {
                const float mo = __shfl_xor_sync(kFull, m[h], s);
                const float mn = fmaxf(m[h], mo), ref = mn == -INFINITY ? 0.f : mn;
                const float mine = exp2f(m[h] - ref), theirs = exp2f(mo - ref);
                l[h] = l[h] * mine + __shfl_xor_sync(kFull, l[h], s) * theirs;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[h][j] = o[h][j] * mine + __shfl_xor_sync(kFull, o[h][j], s) * theirs;
                m[h] = mn;
            }
        float *eo = reinterpret_cast<float *>(smem + warp * WARP_BYTES);
        if (sub == 0) {
#pragma unroll
            for (int h = 0; h < kQ4Tile; ++h)
                *reinterpret_cast<float4 *>(eo + h * LD + 4 * u) = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
        }
        if (lane == 0) {
#pragma unroll
            for (int h = 0; h < kQ4Tile; ++h) {
                eo[16 * LD + h] = m[h];
                eo[16 * LD + 16 + h] = l[h];
            }
        }
        if (threadIdx.x == 0) s_next[nb] = dynamic ? ahead : item + gridDim.x;
        __syncthreads();
        merge_and_store<T, HD>(smem, WARP_BYTES, p, it.seq, it.part, it.qh0, it.rows, it.single);
        __syncthreads();
        item = s_next[nb];
        nb ^= 1;
        if (dynamic && threadIdx.x == 0) ahead = gridDim.x + next_handout(p.work_ctr);
    }
    griddep_launch_dependents();
    if (dynamic && threadIdx.x == 0) finish_handouts(p.work_ctr);
}

using namespace host;

template <typename T, int HD, int G>
int launch_fma(const DecodeParams &p, const void *k_cache, const void *v_cache, long long items, int dev,
               cudaStream_t st) {
    static KernelSlot slot;
    auto kernel = decode_q4_fma_kernel<T, HD, G>;
    const int occ = ensure_kernel(kernel, slot, 0, dev);
    if (occ == 0) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: cannot configure the kernel");
    const long long cap = static_cast<long long>(sm_count(dev)) * occ;
    const cudaError_t e = launch_dependent(kernel, static_cast<int>(items < cap ? items : cap), kWarps * 32, 0, st,
                                           static_cast<const uint8_t *>(k_cache),
                                           static_cast<const uint8_t *>(v_cache), p);
    return e == cudaSuccess ? PA_OK : pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
}

template <typename T>
int launch_any(const DecodeParams &p, const void *k, const void *v, int head_dim, int group_size, long long items,
               int dev, cudaStream_t st) {
    if (head_dim == 128)
        return group_size == 64 ? launch_fma<T, 128, 64>(p, k, v, items, dev, st)
                                : launch_fma<T, 128, 32>(p, k, v, items, dev, st);
    return group_size == 64 ? launch_fma<T, 64, 64>(p, k, v, items, dev, st)
                            : launch_fma<T, 64, 32>(p, k, v, items, dev, st);
}

int q4_partition(int partition_size) { return partition_size == 0 ? 512 : partition_size; }

size_t workspace_bytes(int num_seqs, int num_q_heads, int head_dim, int walk_cap, int P, size_t *acc_at) {
    const long long max_parts = (static_cast<long long>(walk_cap) + P - 1) / P;
    if (max_parts <= 1) return 0;
    const size_t rows = static_cast<size_t>(num_seqs) * max_parts * num_q_heads;
    *acc_at = kWorkspaceHeader + align256(rows * 2 * sizeof(float));
    return *acc_at + align256(rows * head_dim * sizeof(float));
}

// A window's edges are rounded to whole blocks (so that a page is walked or
// left out as one); for sizing a workspace, to the largest.
constexpr int kQ4MaxBlock = 32;

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_q4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                              int max_context_len, int partition_size, int window, int num_sinks) {
    const int P = pa::q4_partition(partition_size);
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_context_len <= 0 || P <= 0 ||
        window < 0 || num_sinks < 0)
        return 0;
    size_t acc_at;
    return pa::workspace_bytes(num_seqs, num_q_heads, head_dim,
                               pa::host::seen_cap(max_context_len, window, num_sinks, pa::kQ4MaxBlock), P, &acc_at);
}

extern "C" int pa_decode_q4(void *out, const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *block_tables, const int32_t *context_lens, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int group_size, float scale, int window,
                            int num_sinks, const pa_decode_args *a) {
    PaTraceRange trace("pa_decode_q4");
    using namespace pa::host;
    if (!a) return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: args is NULL");
    if (a->num_seqs < 0) return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: num_seqs < 0");
    if (a->num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: null tensor pointer");
    if (a->dtype != PA_F32 && a->dtype != PA_BF16) return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: bad dtype");
    if (a->phase < PA_PHASE_ALL || a->phase > PA_PHASE_REDUCE)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: bad phase");
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: num_q_heads must be a positive multiple of num_kv_heads");
    if (!pa::q4_sizes_ok(head_dim, block_size, group_size))
        return pa_fail(PA_ERR_UNSUPPORTED,
                       "pa_decode_q4: head_dim must be 64 or 128, block_size 16 or 32, group_size 32 or 64");
    if (a->k_new || a->v_new || a->slot_mapping)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_q4: no fused cache write; call pa_reshape_and_cache_q4 first");
    if (a->simt) return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_q4: simt is not available");
    if (a->num_blocks <= 0 || a->max_blocks_per_seq <= 0 || a->max_context_len < 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: bad num_blocks, max_blocks_per_seq or max_context_len");
    if (window < 0 || num_sinks < 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: window and num_sinks must not be negative");
    const int P = pa::q4_partition(a->partition_size);
    if (P < 32 || P > 4096 || P % 32 != 0)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: partition_size must be a multiple of 32 in [32, 4096]");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: out, q and caches must be 16-byte aligned");

    const long long table_cap = static_cast<long long>(a->max_blocks_per_seq) * block_size;
    const int ctx_cap = static_cast<int>(a->max_context_len < table_cap ? a->max_context_len : table_cap);
    // No window is one that no sequence outgrows; sinks past the end change nothing.
    if (window == 0 || window > ctx_cap) window = ctx_cap > 0 ? ctx_cap : 1;
    if (num_sinks > ctx_cap) num_sinks = ctx_cap;
    const int walk_cap = seen_cap(ctx_cap, window, num_sinks, block_size);
    const int max_parts = walk_cap <= P ? 1 : static_cast<int>((static_cast<long long>(walk_cap) + P - 1) / P);
    pa::DecodeParams p{};
    if (max_parts > 1) {
        size_t acc_at;
        const size_t need = pa::workspace_bytes(a->num_seqs, num_q_heads, head_dim, walk_cap, P, &acc_at);
        if (!a->workspace || a->workspace_bytes < need || !aligned16(a->workspace))
            return pa_fail(PA_ERR_WORKSPACE, "pa_decode_q4: workspace missing, unaligned or smaller than "
                                             "pa_decode_q4_workspace_size()");
        char *ws = static_cast<char *>(a->workspace);
        p.work_ctr = reinterpret_cast<unsigned long long *>(ws);
        p.part_ml = reinterpret_cast<float *>(ws + kWorkspaceHeader);
        p.part_acc = reinterpret_cast<float *>(ws + acc_at);
    }
    p.out = out;
    p.q = q;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.status = a->dev_status;
    p.num_seqs = a->num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = a->num_blocks;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.partition_size = P;
    p.max_parts = max_parts;
    p.ctx_cap = ctx_cap;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.window = window;
    p.num_sinks = num_sinks;
    p.view_gran = block_size;
    p.sink_end = round_up_int(num_sinks, block_size);
    p.tile_rows = p.group < pa::kQ4Tile ? p.group : pa::kQ4Tile;
    p.head_tiles = (p.group + pa::kQ4Tile - 1) / pa::kQ4Tile;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: no CUDA device");
    if (sm_count(dev) <= 0) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: cannot query the SM count");
    cudaStream_t st = static_cast<cudaStream_t>(a->stream);
    const long long items = static_cast<long long>(a->num_seqs) * max_parts * num_kv_heads * p.head_tiles;
    const long long partial_bytes =
        static_cast<long long>(a->num_seqs) * max_parts * num_q_heads * (head_dim + 2) * 4;
    p.reduce_newest_first = max_parts > 1 && partial_bytes > l2_bytes(dev) ? 1 : 0;
    if (items >= (1ll << 31)) p.work_ctr = nullptr;   // hand-out indices are 32 bits wide
    int rc = PA_OK;
    if (a->phase != PA_PHASE_REDUCE) {
        if (p.work_ctr && !a->skip_counter_reset &&
            cudaMemsetAsync(p.work_ctr, 0, sizeof(unsigned long long), st) != cudaSuccess)
            return pa_fail(PA_ERR_CUDA, "pa_decode_q4: cannot reset the work counter");
        rc = a->dtype == PA_F32
                 ? pa::launch_any<float>(p, k_cache, v_cache, head_dim, group_size, items, dev, st)
                 : pa::launch_any<__nv_bfloat16>(p, k_cache, v_cache, head_dim, group_size, items, dev, st);
    }
    if (rc != PA_OK) return rc;
    if (max_parts > 1 && a->phase != PA_PHASE_PARTITIONS) {
        const cudaError_t le = pa::launch_merge(p, a->dtype == PA_F32, head_dim, st);
        if (le != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(le));
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return PA_OK;
}
