// Shared by the passes of pa_decode_tree and pa_decode_cross (attention of any
// number of queries per sequence over a paged cache): what a sequence's queries
// see, and how the work is cut.
//
// Work.  A sequence's c queries times the `group` query heads of one KV head
// are rows R = token * group + head of that head's problem; an item is up to
// ROWS of them, and costs a unit for each KT tokens of the cache that any of its
// rows sees (two, if it has more than HALF rows), and START units for its
// beginning and end.  All items of the
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
    int queries_above, queries_most;  // the pass' sequences: those of more queries than the one and not more than the other
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
    if (s.c <= p.queries_above || s.c > p.queries_most) s.c = 0;   // another pass takes them
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
template <int ROWS_, int HALF, int KT, int START>
struct MultiAxis {
    static constexpr int ROWS = ROWS_;

    static __device__ __forceinline__ int row_blocks(const MultiParams &p, const MultiSeq &s) {
        return (s.c * p.group + ROWS - 1) / ROWS;
    }

    // Tokens that any row of row block m sees.
    static __device__ __forceinline__ int seen(const MultiParams &p, const MultiSeq &s, int m) {
        if (p.see != kSeeChain || s.n == 0) return s.n;
        const int last = min(s.c - 1, ((m + 1) * ROWS - 1) / p.group);
        return s.n - s.c + last + 1;
    }

    // Tokens that every row of row block m sees (not above s.n; below zero where no row sees anything).
    static __device__ __forceinline__ int clear(const MultiParams &p, const MultiSeq &s, int m) {
        if (p.see == kSeeAll) return s.n;
        if (p.see == kSeeMask || s.n == 0) return s.n - s.c;
        return s.n - s.c + m * ROWS / p.group + 1;   // of a chain, up to its first row's
    }

    // An item of a row that sees nothing still has a tile: it writes the zeros.
    static __device__ __forceinline__ int tiles(const MultiParams &p, const MultiSeq &s, int m) {
        const int t = static_cast<int>((seen(p, s, m) + static_cast<unsigned>(KT - 1)) / KT);
        return t > 0 ? t : 1;
    }

    // Units of one tile.
    static __device__ __forceinline__ int cost(const MultiParams &p, const MultiSeq &s, int m) {
        return HALF < ROWS && s.c * p.group - m * ROWS > HALF ? 2 : 1;
    }

    static __device__ __forceinline__ int units(const MultiParams &p, const MultiSeq &s, int m) {
        return tiles(p, s, m) * cost(p, s, m) + START;
    }

    // Tiles that lie before unit `at` of an item: where a stretch that begins or ends there cuts it.
    static __device__ __forceinline__ int tiles_before(const MultiParams &p, const MultiSeq &s, int m, int at) {
        return at <= START ? 0 : (at - START) >> (cost(p, s, m) - 1);
    }

    // Units of one KV head of a sequence.
    static __device__ __forceinline__ long long head_units(const MultiParams &p, const MultiSeq &s) {
        const int blocks = row_blocks(p, s);
        if (blocks == 0) return 0;
        if (p.see != kSeeChain || s.n == 0)
            return static_cast<long long>(blocks - 1) * units(p, s, 0) + units(p, s, blocks - 1);
        long long u = 0;
        for (int m = 0; m < blocks; ++m) u += units(p, s, m);
        return u;
    }

    // The next item of a walk from `spot` over `left` units; false at its end.
    static __device__ __forceinline__ bool next(const MultiParams &p, MultiSpot &spot, long long &left, MultiItem &it) {
        while (left > 0) {
            const int all = units(p, spot.s, spot.m);
            const int end = static_cast<int>(spot.at + left < all ? spot.at + left : all);
            it = MultiItem{spot.seq, spot.kvh, spot.m, tiles_before(p, spot.s, spot.m, spot.at),
                           tiles_before(p, spot.s, spot.m, end), tiles(p, spot.s, spot.m), spot.s};
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
            const int kvh = rest >> 32 || head >> 32 ? static_cast<int>(rest / head)
                                                     : static_cast<int>(static_cast<unsigned>(rest) / static_cast<unsigned>(head));
            rest -= kvh * head;
            int m = 0;
            while (rest >= Axis::units(p, s, m)) rest -= Axis::units(p, s, m++);
            *spot = MultiSpot{i, kvh, m, static_cast<int>(rest), s};
            return;
        }
    }
};

// The axis in equal stretches: the CTAs that have one (a unit at least), and where
// CTA b's starts.  One division, in 32 bits where the axis is not absurdly long.
struct MultiSplit {
    long long each;
    int ctas, extra;   // the first `extra` stretches have a unit more

    __device__ __forceinline__ MultiSplit(long long total, int grid) {
        ctas = total < grid ? static_cast<int>(total) : grid;
        const unsigned d = ctas > 0 ? ctas : 1;
        if (total >> 32) {
            each = total / d;
        } else {
            each = static_cast<unsigned>(total) / d;
        }
        extra = static_cast<int>(total - each * d);
    }
    __device__ __forceinline__ long long start(int b) const { return b * each + min(b, extra); }
};

// Whether a row's query (token `tok` of its sequence) sees cache position u < n.
__device__ __forceinline__ bool multi_sees(const MultiParams &p, const MultiSeq &s, int tok, int u) {
    if (p.see == kSeeAll) return true;
    const int j = u - (s.n - s.c);
    if (p.see == kSeeChain) return j <= tok;
    if (j < 0) return true;
    return (j >> 6) < p.words && ((p.mask[static_cast<long long>(s.start + tok) * p.words + (j >> 6)] >> (j & 63)) & 1ull);
}

// Which of the 32 positions from u on a row sees, as bits.
__device__ __forceinline__ uint32_t multi_seen_bits(const MultiParams &p, const MultiSeq &s, int tok, int u) {
    const auto below = [](int count) { return count <= 0 ? 0u : (count >= 32 ? ~0u : (1u << count) - 1u); };
    const int base = s.n - s.c;
    if (p.see == kSeeAll) return below(s.n - u);
    if (p.see == kSeeChain) return below(min(s.n, base + tok + 1) - u);
    uint32_t bits = below(base - u);
    const int j = u - base;   // first position's node, negative before the tree
    if (j > -32 && u < s.n) {
        const unsigned long long *row = p.mask + static_cast<long long>(s.start + tok) * p.words;
        const int w = j >> 6;
        const unsigned long long a = w >= 0 && w < p.words ? row[w] : 0ull;
        const unsigned long long b = w + 1 >= 0 && w + 1 < p.words ? row[w + 1] : 0ull;
        const int sh = j & 63;
        bits |= static_cast<uint32_t>(sh ? (a >> sh) | (b << (64 - sh)) : a);
    }
    return bits & below(s.n - u);
}

// Sets the bf16 values of 16 bytes in shared memory that are not finite to zero; whether there were any.
__device__ __forceinline__ bool clear_not_finite(uint4 &at) {
    uint4 x = at;
    uint32_t *w = &x.x;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if ((w[e] & 0x7f80u) == 0x7f80u) bad = true, w[e] &= 0xffff0000u;
        if ((w[e] & 0x7f800000u) == 0x7f800000u) bad = true, w[e] &= 0xffffu;
    }
    if (bad) at = x;
    return bad;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
// Two weights w = hi + lo in bf16 parts (off by 2^-16 of themselves at most).  hi is cut off and lo is what is left and 2^-23 of w, so
// that neither is below zero nor, with w above zero (and not within 2^10 of the smallest fp32), zero: an infinite value stays an infinity in
// both products.  Rounded parts would be off by 2^-17 and make it a NaN.
__device__ __forceinline__ void weight_parts(float2 w, uint32_t &hi, uint32_t &lo) {
    constexpr float over = 1.f + 0x1p-23f;
    hi = __byte_perm(__float_as_uint(w.x), __float_as_uint(w.y), 0x7632);
    const float2 rest = fma2(w, make_float2(over, over),
                             make_float2(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xffff0000u)));
    lo = bf16_pair(rest.x, rest.y);
}

// For tiles that several row blocks read, one after the other.
__device__ __forceinline__ uint64_t l2_normal_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// Element offset of row R of KV head kvh's problem in q and out.
__device__ __forceinline__ long long multi_row(const MultiParams &p, const MultiSeq &s, int kvh, int R, int hd) {
    const int tok = R / p.group;
    return ((static_cast<long long>(s.start) + tok) * p.num_q_heads + kvh * p.group + (R - tok * p.group)) * hd;
}

// CTAs of a pass at most (a workspace has two partials for each), and the rows
// of its items.
constexpr int kMultiFewCtas = 608, kMultiF32Rows = 32;
constexpr int kMultiMmaCtas = 152, kMultiMmaRows = 256;

// ------------------------------------------------------------------ join ---
// grid (CTAs of the pass - 1, row chunks): the CTAs of column x look at the
// boundary between stretches x and x + 1; the first boundary inside an item
// owns its join.  out = sum 2^(m_k - M) acc_k / sum 2^(m_k - M) l_k over its
// partials k in the axis' order, a warp per row.
template <typename OutT, int HD, typename Axis>
__global__ void __launch_bounds__(256) multi_join_kernel(const MultiParams p, int pass_grid) {
    constexpr int ROWS = Axis::ROWS;
    griddep_wait();
    int flags = 0;
    const MultiLocator<Axis, 256> loc(p, flags);
    const MultiSplit split(loc.total, pass_grid);
    const int b = blockIdx.x + 1;
    if (b >= split.ctas) return;
    __shared__ MultiSpot s_spot;
    const long long unit = split.start(b);
    loc.find(p, unit, &s_spot);
    __syncthreads();
    const MultiSpot spot = s_spot;
    const auto cut = [&](long long at) { return Axis::tiles_before(p, spot.s, spot.m, static_cast<int>(at)); };
    if (cut(spot.at) == 0) return;                             // the item begins with CTA b
    const long long begin = unit - spot.at, end = begin + Axis::units(p, spot.s, spot.m);
    if (b > 1 && split.start(b - 1) > begin && cut(split.start(b - 1) - begin) > 0)
        return;                                                // an earlier boundary cuts it too
    // CTA b - 1 has the item's first partial; of those after it, each that holds a tile of the item has one.  Warp 0
    // lists their places in order.
    __shared__ int s_part[kMultiFewCtas];
    __shared__ int s_parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        if (lane == 0) s_part[0] = 2 * (b - 1) + 1;
        int parts = 1;
        for (int first = b;; first += 32) {
            const int cta = first + lane;
            const long long from = split.start(cta), to = split.start(cta + 1);
            const bool inside = cta < split.ctas && from < end;
            const bool has = inside && cut(from - begin) < cut((to < end ? to : end) - begin);
            const unsigned have = __ballot_sync(kFull, has);
            if (has) s_part[parts + __popc(have & ((1u << lane) - 1u))] = 2 * cta;
            parts += __popc(have);
            if (__ballot_sync(kFull, !inside)) break;
        }
        if (lane == 0) s_parts = parts;
    }
    __syncthreads();
    const int parts = s_parts, rows = min(ROWS, spot.s.c * p.group - spot.m * ROWS);
    constexpr int V = HD / 32;
    for (int r = blockIdx.y * 8 + warp; r < rows; r += gridDim.y * 8) {
        // Eight partials at a time, all of their loads in flight at once.
        constexpr int kBatch = 8;
        float M = -INFINITY, L = 0.f, acc[V] = {};
        for (int k0 = 0; k0 < parts; k0 += kBatch) {
            float2 ml[kBatch];
            float a[kBatch][V];
            float top = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) a[k][v] = 0.f;
                if (k0 + k < parts) {
                    const long long i = static_cast<long long>(s_part[k0 + k]) * p.slot_rows + r;
                    ml[k] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * i);
                    if constexpr (V == 4)
                        *reinterpret_cast<float4 *>(a[k]) = *reinterpret_cast<const float4 *>(p.part_acc + i * HD + lane * V);
                    else
                        *reinterpret_cast<float2 *>(a[k]) = *reinterpret_cast<const float2 *>(p.part_acc + i * HD + lane * V);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
            // (a partial that saw nothing is all zeros: its reference is -inf, its sums were never added to)
            const float ref = top == -INFINITY ? 0.f : top, keep = exp2f(M - ref);
            M = top;
            L *= keep;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= keep;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float f = exp2f(ml[k].x - ref);
                L += f * ml[k].y;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] += f * a[k][v];
            }
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
    cfg.gridDim = dim3(pass_grid - 1, min((min(Axis::ROWS, p.slot_rows) + 7) / 8, 16));
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

int launch_multi_f32(const MultiParams &p, int head_dim, bool few, int dev, cudaStream_t st);   // fp32, items of 16 or 32 rows
int launch_multi_mma(const MultiParams &p, int head_dim, int dev, cudaStream_t st);    // bf16
int launch_multi_few(const MultiParams &p, int head_dim, int dev, cudaStream_t st);    // bf16, few rows per sequence

}  // namespace pa
