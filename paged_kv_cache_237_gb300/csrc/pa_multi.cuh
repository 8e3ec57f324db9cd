// Shared by the passes of pa_decode_tree and pa_decode_cross (attention of any
// number of queries per sequence over a paged cache): what a sequence's queries
// see, and how the work is cut.
//
// Work.  A sequence's c queries times the `group` query heads of one KV head
// are rows R = token * group + head of that head's problem; an item is up to
// ROWS of them, and costs one unit per KT tokens of the cache that any of its
// rows sees, plus START units for its beginning and end.  All items of the
// batch lie end to end on one axis of units (sequence, KV head, row block), and
// each CTA takes an equal stretch of it, whatever the lengths.  A CTA whose
// stretch holds an item whole writes its rows; where a stretch ends inside an
// item, both sides store partials (maximum, sum, unnormalised rows) and a second
// launch joins them in the axis' order.  A CTA has at most two partials, so the
// workspace does not grow with the batch.  No counters, no atomics: results do
// not change from run to run.
#pragma once

#include "pa_decode_common.cuh"

namespace pa {

enum { kSeeAll = 0, kSeeChain = 1, kSeeMask = 2 };

struct MultiParams {
    void *out;
    const void *q, *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens, *query_start;
    const unsigned long long *mask;   // kSeeMask: [num_tokens][words]
    float *part_ml;                   // [2 * CTAs][slot_rows][2] (maximum in log2 units, sum)
    float *part_acc;                  // [2 * CTAs][slot_rows][HD]
    int32_t *status;
    int num_seqs, num_tokens, num_q_heads, num_kv_heads, group;
    int block_size, num_blocks, width, ctx_cap, words, see, slot_rows, total_rows;
    float scale_log2;
};

// Sequence i: n tokens in the cache, c queries from row `start` on.  With a
// chain or a mask the queries are the cache's last c tokens.
struct MultiSeq {
    int n, c, start;
};

__device__ __forceinline__ MultiSeq multi_seq(const MultiParams &p, int i, int &flags) {
    const int a = p.query_start[i], b = p.query_start[i + 1], n = p.context_lens[i];
    MultiSeq s{n < 0 ? 0 : min(n, p.ctx_cap), b - a, a};
    if (s.n != n) flags |= PA_STATUS_BAD_CONTEXT_LEN;
    if (a < 0 || b < a || b > p.num_tokens) {
        flags |= PA_STATUS_BAD_TREE;
        s.c = s.start = 0;
    }
    if (p.see != kSeeAll && s.c > s.n) {   // queries whose rows the cache does not hold see nothing
        flags |= PA_STATUS_BAD_CONTEXT_LEN;
        s.n = 0;
    }
    return s;
}

// A place on the axis: unit `at` of row block m of KV head kvh of sequence seq.
struct MultiSpot {
    int seq, kvh, m, at;
    MultiSeq s;
};

// What a CTA does next: tiles [tile0, tile1) of an item that has `tiles`.
struct MultiItem {
    int seq, kvh, m, tile0, tile1, tiles;
    MultiSeq s;
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (tile0 == 0 ? 1 : 0); }
};

// The axis for items of ROWS rows and units of KT tokens.
template <int ROWS_, int KT, int START>
struct MultiAxis {
    static constexpr int ROWS = ROWS_, kStart = START;

    static __device__ __forceinline__ int row_blocks(const MultiParams &p, const MultiSeq &s) {
        return (s.c * p.group + ROWS - 1) / ROWS;
    }

    // Tokens that any row of row block m sees.
    static __device__ __forceinline__ int seen(const MultiParams &p, const MultiSeq &s, int m) {
        if (p.see != kSeeChain || s.n == 0) return s.n;
        const int last = min(s.c - 1, ((m + 1) * ROWS - 1) / p.group);
        return s.n - s.c + last + 1;
    }

    // An item of a row that sees nothing still has a tile: it writes the zeros.
    static __device__ __forceinline__ int tiles(const MultiParams &p, const MultiSeq &s, int m) {
        const int t = static_cast<int>((seen(p, s, m) + static_cast<unsigned>(KT - 1)) / KT);
        return t > 0 ? t : 1;
    }

    static __device__ __forceinline__ int units(const MultiParams &p, const MultiSeq &s, int m) {
        return tiles(p, s, m) + START;
    }

    // Units of one KV head of a sequence.
    static __device__ __forceinline__ long long head_units(const MultiParams &p, const MultiSeq &s) {
        const int blocks = row_blocks(p, s);
        if (p.see != kSeeChain || s.n == 0) return static_cast<long long>(blocks) * units(p, s, 0);
        long long u = 0;
        for (int m = 0; m < blocks; ++m) u += units(p, s, m);
        return u;
    }

    // The next item of a walk from `spot` over `left` units; false at its end.
    static __device__ __forceinline__ bool next(const MultiParams &p, MultiSpot &spot, long long &left, MultiItem &it) {
        while (left > 0) {
            const int count = tiles(p, spot.s, spot.m), all = count + START;
            const int end = static_cast<int>(spot.at + left < all ? spot.at + left : all);
            it = MultiItem{spot.seq, spot.kvh, spot.m, max(0, spot.at - START), max(0, end - START), count, spot.s};
            left -= end - spot.at;
            spot.at = 0;
            if (++spot.m >= row_blocks(p, spot.s)) {
                spot.m = 0;
                if (++spot.kvh >= p.num_kv_heads) {
                    spot.kvh = 0;
                    int none = 0;
                    do {
                        if (++spot.seq >= p.num_seqs) {
                            left = 0;
                            break;
                        }
                        spot.s = multi_seq(p, spot.seq, none);
                    } while (spot.s.c == 0);
                }
            }
            if (it.tile1 > it.tile0) return true;
        }
        return false;
    }
};

// Units of the whole batch and, for up to two unit indexes, where they lie.
// Called by all THREADS threads of a CTA; the result is the same in all.
template <typename Axis, int THREADS>
struct MultiLocator {
    long long total;
    long long mine, before;   // units of this thread's sequences and of all before them
    int first, last;          // this thread's sequences

    __device__ MultiLocator(const MultiParams &p, int &flags) {
        __shared__ long long s_warp[THREADS / 32];
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int per = (p.num_seqs + THREADS - 1) / THREADS;
        first = min(p.num_seqs, tid * per);
        last = min(p.num_seqs, first + per);
        mine = 0;
        for (int i = first; i < last; ++i) mine += Axis::head_units(p, multi_seq(p, i, flags)) * p.num_kv_heads;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        total = 0;
        before = incl - mine;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += s_warp[w];
            total += s_warp[w];
        }
    }

    // The thread whose sequences hold `unit` (below total) writes its place.
    __device__ __forceinline__ void find(const MultiParams &p, long long unit, MultiSpot *spot) const {
        if (unit < before || unit >= before + mine) return;
        long long rest = unit - before;
        int none = 0;
        for (int i = first; i < last; ++i) {
            const MultiSeq s = multi_seq(p, i, none);
            const long long head = Axis::head_units(p, s);
            if (rest >= head * p.num_kv_heads) {
                rest -= head * p.num_kv_heads;
                continue;
            }
            const int kvh = static_cast<int>(rest / head);
            rest -= kvh * head;
            int m = 0;
            while (rest >= Axis::units(p, s, m)) rest -= Axis::units(p, s, m++);
            *spot = MultiSpot{i, kvh, m, static_cast<int>(rest), s};
            return;
        }
    }
};

// CTAs that share the axis (each has a unit at least), and where CTA b starts.
__device__ __forceinline__ long long multi_ctas(long long total, int grid) { return total < grid ? total : grid; }
__device__ __forceinline__ long long multi_start(long long total, long long ctas, long long b) {
    return b * (total / ctas) + min(b, total % ctas);
}

// Whether a row's query (token `tok` of its sequence) sees cache position u < n.
__device__ __forceinline__ bool multi_sees(const MultiParams &p, const MultiSeq &s, int tok, int u) {
    if (p.see == kSeeAll) return true;
    const int j = u - (s.n - s.c);
    if (p.see == kSeeChain) return j <= tok;
    if (j < 0) return true;
    return (j >> 6) < p.words && ((p.mask[static_cast<long long>(s.start + tok) * p.words + (j >> 6)] >> (j & 63)) & 1ull);
}

// Element offset of row R of KV head kvh's problem in q and out.
__device__ __forceinline__ long long multi_row(const MultiParams &p, const MultiSeq &s, int kvh, int R, int hd) {
    const int tok = R / p.group;
    return ((static_cast<long long>(s.start) + tok) * p.num_q_heads + kvh * p.group + (R - tok * p.group)) * hd;
}

// ------------------------------------------------------------------ join ---
// grid (CTAs of the pass - 1, row chunks): the CTAs of column x look at the
// boundary between stretches x and x + 1; the first boundary inside an item
// owns its join.  out = sum 2^(m_k - M) acc_k / sum 2^(m_k - M) l_k over its
// partials k in the axis' order, a warp per row.
template <typename OutT, int HD, typename Axis>
__global__ void __launch_bounds__(256) multi_join_kernel(const MultiParams p, int pass_grid) {
    constexpr int ROWS = Axis::ROWS, START = Axis::kStart;
    griddep_wait();
    int flags = 0;
    const MultiLocator<Axis, 256> loc(p, flags);
    const long long ctas = multi_ctas(loc.total, pass_grid);
    const long long b = blockIdx.x + 1;
    if (b >= ctas) return;
    __shared__ MultiSpot s_spot;
    const long long unit = multi_start(loc.total, ctas, b);
    loc.find(p, unit, &s_spot);
    __syncthreads();
    const MultiSpot spot = s_spot;
    if (spot.at <= START) return;                              // the item begins with CTA b
    const long long begin = unit - spot.at;
    if (multi_start(loc.total, ctas, b - 1) > begin + START) return;   // an earlier boundary cuts it too
    const long long end = begin + Axis::units(p, spot.s, spot.m);
    int parts = 1;
    while (b + parts - 1 < ctas && multi_start(loc.total, ctas, b + parts - 1) < end) ++parts;
    const int rows = min(ROWS, spot.s.c * p.group - spot.m * ROWS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int V = HD / 32;
    for (int r = blockIdx.y * 8 + warp; r < rows; r += gridDim.y * 8) {
        auto at = [&](int k) {
            const long long slot = k == 0 ? 2 * (b - 1) + 1 : 2 * (b + k - 1);
            return slot * p.slot_rows + r;
        };
        float M = -INFINITY;
        for (int k = lane; k < parts; k += 32) M = fmaxf(M, p.part_ml[2 * at(k)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f, acc[V] = {};
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
            const long long i = at(k);
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * i);
            const float *a = p.part_acc + i * HD + lane * V;
            const float f = exp2f(ml.x - ref);
            L += f * ml.y;
            // a partial that saw nothing has no rows to add (its weight is zero)
            if (ml.x == -INFINITY && ml.y == 0.f) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += f * a[v];
        }
        // l is zero only for a row that sees nothing; a sum that is not a number stays one
        const float inv = L == 0.f ? 0.f : 1.f / L;
        OutT *o = static_cast<OutT *>(p.out) + multi_row(p, spot.s, spot.kvh, spot.m * ROWS + r, HD) + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = static_cast<OutT>(acc[v] * inv);
    }
}

// The join, as a programmatic dependent of the pass: its CTAs may start while the
// pass's last CTAs finish, and wait for the pass before they read.
template <typename OutT, int HD, typename Axis>
int launch_join(const MultiParams &p, int pass_grid, cudaStream_t st) {
    if (pass_grid < 2) return PA_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pass_grid - 1, (min(Axis::ROWS, p.slot_rows) + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, multi_join_kernel<OutT, HD, Axis>, p, pass_grid);
    return e == cudaSuccess ? PA_OK : pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
}

// CTAs of a pass at most (a workspace has two partials for each), and the rows
// of its items.
constexpr int kMultiSimtCtas = 608, kMultiSimtRows = 32;
constexpr int kMultiMmaCtas = 152, kMultiMmaRows = 256;

int launch_multi_simt(const MultiParams &p, int head_dim, int dev, cudaStream_t st);   // fp32
int launch_multi_mma(const MultiParams &p, int head_dim, int dev, cudaStream_t st);    // bf16

}  // namespace pa
