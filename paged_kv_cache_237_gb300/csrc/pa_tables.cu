// Batch tables on the device for sm_103a: padded block tables, the step's slot
// map, positions and query starts from lengths and a flat block list
// (include/pa.h states the formulas).
//
// Every sequence's rows start where the sequences before it end, so the work
// is a prefix sum over the batch and then a copy.  Batches are small (tens to
// a few thousand lengths, a few KB that stay in L2), so each CTA sums the
// lengths before its own sequences itself: one launch, no workspace, and no
// CTA waits for another.  Bound by latency (launch, the sum's loads, one id's
// load): 64 sequences' next tokens 2.75 us, 513 sequences of up to 16384 tokens
// with 121,500 new ones 5.9 us, where the bytes would take 0.7.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kTableThreads = 256;

struct TableParams {
    int32_t *tables;
    int64_t *slots;
    int32_t *positions, *query_start;
    const int32_t *ids, *lens, *news;
    int num_seqs, width, max_tokens, num_ids, block_size, num_blocks, seqs_per_cta;
    int32_t *status;
};

struct SeqSize {
    int n, c, blocks;
    bool bad;
};

__device__ __forceinline__ SeqSize seq_size(const TableParams &p, int i, long long cap) {
    const int n0 = p.lens[i], c0 = p.news[i];
    SeqSize s;
    s.n = n0 < 0 ? 0 : static_cast<int>(n0 > cap ? cap : n0);
    s.c = c0 < 0 ? 0 : (c0 > s.n ? s.n : c0);
    s.blocks = static_cast<int>((static_cast<long long>(s.n) + p.block_size - 1) / p.block_size);
    s.bad = s.n != n0 || s.c != c0;
    return s;
}

// grid (sequence ranges, splits): the CTAs of one range share its table
// columns and token rows, and all CTAs share the padding rows.
__global__ void __launch_bounds__(kTableThreads) build_tables_kernel(const TableParams p) {
    const long long cap = static_cast<long long>(p.width) * p.block_size;
    const int s0 = blockIdx.x * p.seqs_per_cta;
    const int s1 = min(p.num_seqs, s0 + p.seqs_per_cta);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    long long sum[3] = {0, 0, 0};   // blocks and new tokens before s0, all new tokens
    for (int i = tid; i < p.num_seqs; i += kTableThreads) {
        const SeqSize s = seq_size(p, i, cap);
        if (i < s0) {
            sum[0] += s.blocks;
            sum[1] += s.c;
        }
        sum[2] += s.c;
    }
    __shared__ long long s_sum[3][kTableThreads / 32];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(kFull, sum[j], o);
        if (lane == 0) s_sum[j][warp] = sum[j];
    }
    __syncthreads();
    long long first = 0, start = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 32; ++w) {
        first += s_sum[0][w];
        start += s_sum[1][w];
        total += s_sum[2][w];
    }

    int flags = 0;
    auto block_id = [&](long long at) {
        if (at >= p.num_ids) {
            flags |= PA_STATUS_SHORT_LIST;
            return -1;
        }
        const int id = p.ids[at];
        if (id < 0 || id >= p.num_blocks) {
            flags |= PA_STATUS_BAD_BLOCK_ID;
            return -1;
        }
        return id;
    };
    const int step = kTableThreads * gridDim.y, at0 = blockIdx.y * kTableThreads + tid;
    for (int i = s0; i < s1; ++i) {
        const SeqSize s = seq_size(p, i, cap);
        if (s.bad) flags |= PA_STATUS_BAD_CONTEXT_LEN;
        int32_t *row = p.tables + static_cast<long long>(i) * p.width;
        for (long long j = at0; j < p.width; j += step) row[j] = j < s.blocks ? block_id(first + j) : -1;
        for (long long r = at0; r < s.c; r += step) {
            const long long t = start + r;
            if (t >= p.max_tokens) {
                flags |= PA_STATUS_SHORT_LIST;
                break;
            }
            const int pos = s.n - s.c + static_cast<int>(r);
            const int b = block_id(first + pos / p.block_size);
            p.slots[t] = b < 0 ? -1 : static_cast<int64_t>(b) * p.block_size + pos % p.block_size;
            if (p.positions) p.positions[t] = pos;
        }
        if (at0 == 0 && p.query_start) p.query_start[i] = static_cast<int32_t>(min(start, (long long)INT_MAX));
        first += s.blocks;
        start += s.c;
    }
    if (p.query_start && at0 == 0 && blockIdx.x == 0)
        p.query_start[p.num_seqs] = static_cast<int32_t>(min(total, (long long)INT_MAX));
    const long long all = static_cast<long long>(gridDim.x) * step;
    for (long long t = total + static_cast<long long>(blockIdx.x) * step + at0; t < p.max_tokens; t += all) {
        p.slots[t] = -1;
        if (p.positions) p.positions[t] = 0;
    }
    if (flags) flag_status(p.status, flags);
}

}  // namespace
}  // namespace pa

extern "C" int pa_build_tables(int32_t *block_tables, int64_t *slot_mapping, int32_t *positions,
                               int32_t *query_start, const int32_t *block_ids, const int32_t *context_lens,
                               const int32_t *new_lens, int num_seqs, int max_blocks_per_seq, int max_tokens,
                               int num_ids, int block_size, int num_blocks, int32_t *dev_status, void *stream) {
    PaTraceRange trace("pa_build_tables");
    if (num_seqs < 0 || max_blocks_per_seq < 1 || max_tokens < 0 || num_ids < 0 || block_size < 1 || num_blocks < 1)
        return pa_fail(PA_ERR_INVALID_ARG, "pa_build_tables: bad sizes");
    if ((num_seqs > 0 && (!block_tables || !context_lens || !new_lens)) || (max_tokens > 0 && !slot_mapping) ||
        (num_ids > 0 && !block_ids))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_build_tables: null pointer");
    const uintptr_t words = reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(positions) |
                            reinterpret_cast<uintptr_t>(query_start) | reinterpret_cast<uintptr_t>(block_ids) |
                            reinterpret_cast<uintptr_t>(context_lens) | reinterpret_cast<uintptr_t>(new_lens);
    if ((words & 3u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_build_tables: misaligned pointer");
    pa::TableParams p{block_tables, slot_mapping, positions, query_start, block_ids, context_lens, new_lens,
                      num_seqs, max_blocks_per_seq, max_tokens, num_ids, block_size, num_blocks, 1, dev_status};
    // At most 1024 ranges of sequences, and as many splits of a range as keep
    // about 1024 CTAs busy with a CTA's width of table columns or token rows.
    constexpr int kCtas = 1024;
    p.seqs_per_cta = num_seqs <= kCtas ? 1 : (num_seqs + kCtas - 1) / kCtas;
    const int gx = num_seqs == 0 ? 1 : (num_seqs + p.seqs_per_cta - 1) / p.seqs_per_cta;
    const long long per_row = max_blocks_per_seq > max_tokens ? max_blocks_per_seq : max_tokens;
    long long gy = (per_row + pa::kTableThreads - 1) / pa::kTableThreads;
    if (gy > kCtas / gx) gy = kCtas / gx;
    if (gy < 1) gy = 1;
    pa::build_tables_kernel<<<dim3(gx, static_cast<unsigned>(gy)), pa::kTableThreads, 0,
                              static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return PA_OK;
}
