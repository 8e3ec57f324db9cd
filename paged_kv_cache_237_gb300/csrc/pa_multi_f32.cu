// pa_decode_tree and pa_decode_cross over fp32 caches, on tensor cores.
//
// The products run on mma.m16n8k8 with tf32 operands, each fp32 operand as the
// sum of two of them (x = hi + lo, hi rounded to its 11 bits and lo cut to its own, so
// that one bit of x is lost at most): a b ~ hi hi + hi lo + lo hi, off by 2^-21 of |a b| at
// most, and to either side, so that sums average it out.  Sums are fp32 and rounded: the
// tensor core cuts its sums off, so each product hi hi of 8 columns or tokens starts from
// zero there and is added to its sum by ordinary additions (those with a lo, 2^-11 of it,
// stay in the tensor core over a tile).  Against 64 bits, in the 2-norm: 1.1 * 10^-7 off
// on small trees and on decoders' prompts (plain fp32 operations 1.5 and 3.9); with hi cut
// and sums in the tensor core 5.1 and 5.2, for 308 us against 337 and 257 against 282; with the
// fourth product too 1.1, for 396 and 345.  fp32 FMAs take 521 and 375.
//
// An item is R = 16 MT rows (query tokens x the heads of one KV head) against a
// stretch of the sequence's cache in tiles of 64 tokens, a CTA of 4 warps:
//   scores   each warp 16 of the tile's tokens, all rows (K is split once);
//   weights  row maxima meet in shared memory, P goes there in the order in which
//            the products' operand is read;
//   products each warp a quarter of head_dim, all rows and tokens (V is split once).
// K and V come by cp.async: the next tile's K while this one's products run, its V
// while the next scores do; two to four CTAs per SM fill each other's gaps.
//   MT = 1: few rows per sequence, bound by the copies and their latency.  24
//   multi-head sequences of up to 4000 tokens with 1 to 12 rows: 327 to 339 us,
//   4.4 to 4.6 TB/s (0.65 to 0.67 of the copy rate).
//   MT = 2: many rows, bound by the tensor pipe (8 cycles an instruction, three for
//   each 16 x 8 x 8 products: 98 TFLOP/s, and rows that fill up to 16) and by what lies
//   between its phases; 41 % of its cycles busy.  16 sequences of 100 to 1200 tokens, 24
//   heads of 64, 1 to 300 queries: 274 to 282 us.  Four row tiles would need an SM for one CTA.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_multi.cuh"

namespace pa {
namespace {

constexpr int kTile = 64, kThreads = kWarps * 32;

__device__ __forceinline__ float4 load4(const float *x) { return *reinterpret_cast<const float4 *>(x); }

// x = hi + lo in tf32's 11 bits each: hi to the nearest (half = kNearest) or cut off (half = 0), and what lo cannot hold is
// dropped.  An infinity leaves a NaN in lo, and so does a rounding past the largest fp32.
constexpr uint32_t kNearest = 0x1000u;
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo, uint32_t half = kNearest) {
    hi = (__float_as_uint(x) + half) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

// D = A (16 x 8, row) * B (8 x 8, col) + D.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d += x, two at once.
__device__ __forceinline__ void add2(float *d, const float *x) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(d[0]), "+f"(d[1])
        : "f"(x[0]), "f"(x[1]));
}

// The same with the sum rounded: the product starts from zero.
__device__ __forceinline__ void mma_tf32_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    mma_tf32(x, a, b0, b1);
    add2(d, x);
    add2(d + 2, x + 2);
}

// Place of element (row, col) of a matrix of 16-row tiles in the A operand's order: a lane's four values of a tile's 8
// columns are together.
__device__ __forceinline__ int a_place(int row, int col, int steps) {
    return (((row >> 4) * steps + (col >> 3)) * 32 + (row & 7) * 4 + (col & 3)) * 4 + ((col >> 2) & 1) * 2 + ((row >> 3) & 1);
}

// Place of 16 bytes c of token j in K's and V's tiles: so that an operand's 32 values lie in 32 banks (K's of 8 tokens and
// 4 columns, V's of 4 tokens and 8 columns).
template <int HD>
__device__ __forceinline__ int k_place(int j, int c) { return j * HD + (c ^ (j & 7)) * 4; }
template <int HD>
__device__ __forceinline__ int v_place(int j, int c) { return j * HD + (c ^ (2 * (j & 3))) * 4; }

template <int HD, int MT>
struct Shape {
    static constexpr int R = 16 * MT;
    // Four of the k steps of few rows' Q stay in registers, which leaves room for a third CTA on the SM (24 multi-head
    // sequences of up to 4000 tokens, with sums left in the tensor core: 308 us, two CTAs 339; all of Q there spills, 478).
    static constexpr int QB = HD == 128 && MT == 1 ? 1 : 0;
    static constexpr int Q = 0, K = Q + R * (HD - 32 * QB), V = K + kTile * HD, P = V + kTile * HD, TOP = P + R * kTile;
    static constexpr int BYTES = (TOP + kWarps * R) * 4;
    static constexpr int CTAS = HD == 64 ? 4 : (MT == 1 ? 3 : 2);   // per SM
    using Axis = MultiAxis<R, R, kTile, 1>;
};

template <int HD, int MT>
__global__ void __launch_bounds__(kThreads, Shape<HD, MT>::CTAS) multi_f32_kernel(const MultiParams p) {
    using S = Shape<HD, MT>;
    using Axis = typename S::Axis;
    constexpr int R = S::R, KS = HD / 8 - 4 * S::QB, NV = HD / 32;   // k steps of the scores; n tiles of a warp's columns
    extern __shared__ __align__(16) float smem[];
    __shared__ MultiSpot s_spot;
    __shared__ int s_page[2][kTile / 16];
    __shared__ int s_odd[2];   // first tile of an item with values that are not finite, and the one behind the last
    griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    float *const s_top = smem + S::TOP;
    int flags = 0;
    const MultiLocator<Axis, kThreads> loc(p, flags);
    if (flags && blockIdx.x == 0) flag_status(p.status, flags);
    const MultiSplit cut(loc.total, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= cut.ctas) return;
    const long long unit = cut.start(blockIdx.x);
    long long left = cut.start(blockIdx.x + 1) - unit;
    loc.find(p, unit, &s_spot);
    __syncthreads();
    MultiSpot spot = s_spot;
    const int page_shift = p.block_size == 32 ? 5 : 4, pages = kTile >> page_shift;

    MultiItem it;
    while (Axis::next(p, spot, left, it)) {
        const int R0 = it.m * R, rows = min(R, it.s.c * p.group - R0);
        const int seen = Axis::seen(p, it.s, it.m);
        const int clear = Axis::clear(p, it.s, it.m);   // every row sees every position before
        const int32_t *table = p.block_tables + static_cast<long long>(it.seq) * p.width;
        // First row of page j of tile t in the cache view; -1 for none (zeros).
        const auto page_row = [&](int t, int j) {
            const long long u = static_cast<long long>(t) * kTile + j * p.block_size;
            if (t >= it.tile1 || u >= seen) return -1;
            const int b = table[t * pages + j];
            if (b < 0 || b >= p.num_blocks) {
                flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                return -1;
            }
            return static_cast<int>((static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size);
        };
        const auto copy = [&](int t, const void *cache, float *dst, bool is_k) {
            // a column of pieces per thread, every kThreads / (HD / 4)-th token
            const int c = tid % (HD / 4) * 4;
            const float *src = static_cast<const float *>(cache) + c;
#pragma unroll 8
            for (int j = tid / (HD / 4); j < kTile; j += kThreads / (HD / 4)) {
                const int row = s_page[t & 1][j >> page_shift];
                float *at = dst + (is_k ? k_place<HD>(j, c / 4) : v_place<HD>(j, c / 4));
                if (row >= 0 && t * kTile + j < seen)
                    cp_async_16(smem_addr(at), src + (static_cast<long long>(row) + (j & (p.block_size - 1))) * HD);
                else
                    store4(at, make_float4(0.f, 0.f, 0.f, 0.f));
            }
            cp_async_commit();
        };
        __syncthreads();   // the item before is done with the shared memory
        if (tid == 0) s_odd[0] = it.tile1, s_odd[1] = 0;
        if (tid < 2 * pages) s_page[(it.tile0 + tid / pages) & 1][tid % pages] = page_row(it.tile0 + tid / pages, tid % pages);
        __syncthreads();
        copy(it.tile0, p.k_cache, smem + S::K, true);
        copy(it.tile0, p.v_cache, smem + S::V, false);
        float qr[S::QB ? 4 : 1][4];   // rows g, g + 8 at columns t4, t4 + 4 of the first k steps
        if constexpr (S::QB > 0) {
            const float *lo = static_cast<const float *>(p.q) + multi_row(p, it.s, it.kvh, R0 + min(g, rows - 1), HD) + t4;
            const float *hi = static_cast<const float *>(p.q) + multi_row(p, it.s, it.kvh, R0 + min(g + 8, rows - 1), HD) + t4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qr[i][0] = g < rows ? lo[8 * i] * p.scale_log2 : 0.f;
                qr[i][1] = g + 8 < rows ? hi[8 * i] * p.scale_log2 : 0.f;
                qr[i][2] = g < rows ? lo[8 * i + 4] * p.scale_log2 : 0.f;
                qr[i][3] = g + 8 < rows ? hi[8 * i + 4] * p.scale_log2 : 0.f;
            }
        }
        for (int i = tid; i < R * KS * 2; i += kThreads) {
            const int r = i / (KS * 2), c = i % (KS * 2) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) x = load4(static_cast<const float *>(p.q) + multi_row(p, it.s, it.kvh, R0 + r, HD) + 32 * S::QB + c);
            float *at = smem + S::Q + a_place(r, c, KS);   // columns c .. c + 3 are four lanes apart
            at[0] = x.x * p.scale_log2;
            at[4] = x.y * p.scale_log2;
            at[8] = x.z * p.scale_log2;
            at[12] = x.w * p.scale_log2;
        }

        // This lane's rows: 16 mt + g + 8 h.
        float m[MT][2], l[MT][2];
        float o[MT][NV][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
        }
        for (int t = it.tile0; t < it.tile1; ++t) {
            const int u0 = t * kTile, mine = u0 + 16 * warp;   // first of this warp's tokens
            int next_page = -1;
            if (tid < pages) next_page = page_row(t + 2, tid);
            cp_async_wait_group<1>();   // K is there, V may be on its way
            __syncthreads();
            // The large products and the small ones in sums of their own: an instruction waits some 20 cycles for the
            // one before it in its sum.
            float sc[MT][2][4], low[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[mt][n][e] = low[mt][n][e] = 0.f;
            // Four k steps, which share their places in K's rows; Q's from registers or shared memory.
            const auto steps = [&](int block, const float4 (&q)[MT][4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t bh[2][2], bl[2][2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float *at = smem + S::K + 32 * block + t4;   // of the row's 16 bytes 8 block + 2 i, + 1
                        const int row = 16 * warp + 8 * n + g;
                        split_tf32(at[k_place<HD>(row, 2 * i)], bh[n][0], bl[n][0]);
                        split_tf32(at[k_place<HD>(row, 2 * i + 1)], bh[n][1], bl[n][1]);
                    }
                    uint32_t ah[MT][4], al[MT][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        split_tf32(q[mt][i].x, ah[mt][0], al[mt][0]);
                        split_tf32(q[mt][i].y, ah[mt][1], al[mt][1]);
                        split_tf32(q[mt][i].z, ah[mt][2], al[mt][2]);
                        split_tf32(q[mt][i].w, ah[mt][3], al[mt][3]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_tf32(low[mt][n], al[mt], bh[n][0], bh[n][1]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_tf32(low[mt][n], ah[mt], bl[n][0], bl[n][1]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_tf32_add(sc[mt][n], ah[mt], bh[n][0], bh[n][1]);
                }
            };
            float4 q[MT][4];
            if constexpr (S::QB > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[0][i] = make_float4(qr[i][0], qr[i][1], qr[i][2], qr[i][3]);
                steps(0, q);
            }
#pragma unroll 1
            for (int block = 0; block < KS / 4; ++block) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[mt][i] = load4(smem + S::Q + ((mt * KS + 4 * block + i) * 32 + lane) * 4);
                steps(block + S::QB, q);
            }
            const bool masked = u0 + kTile > clear;
            bool odd = false;   // a score that is not a number
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[mt][n][e] += low[mt][n][e];
                        odd |= sc[mt][n][e] != sc[mt][n][e];
                    }
            if (__any_sync(kFull, odd)) {
                // an infinity's other part, maybe: the plain products say what they come to
                float plain = 0.f;
#pragma unroll 1
                for (int i = 0; i < MT * 8; ++i) {
                    const int row = 16 * (i >> 3) + g + 8 * ((i >> 1) & 1), tok = 16 * warp + 8 * ((i >> 2) & 1) + 2 * t4 + (i & 1);
                    plain = 0.f;
                    const float *q = static_cast<const float *>(p.q) + multi_row(p, it.s, it.kvh, R0 + min(row, rows - 1), HD);
#pragma unroll 1
                    for (int d = 0; d < HD; ++d)
                        plain = fmaf(row < rows ? q[d] * p.scale_log2 : 0.f, smem[S::K + k_place<HD>(tok, d / 4) + d % 4], plain);
#pragma unroll
                    for (int j = 0; j < MT * 8; ++j)
                        if (j == i) sc[j >> 3][(j >> 2) & 1][j & 3] = plain;
                }
            }
            if (masked) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tq = min(R0 + 16 * mt + g + 8 * h, it.s.c * p.group - 1) / p.group;
                        const uint32_t bits = multi_seen_bits(p, it.s, tq, mine) >> (2 * t4);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!((bits >> (8 * n + e)) & 1u)) sc[mt][n][2 * h + e] = -INFINITY;
                    }
            }
            // The warp's maximum of each row.
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = fmaxf(fmaxf(sc[mt][0][2 * h], sc[mt][0][2 * h + 1]), fmaxf(sc[mt][1][2 * h], sc[mt][1][2 * h + 1]));
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                    if (t4 == 0) s_top[warp * R + 16 * mt + g + 8 * h] = top;
                }
            cp_async_wait_group<0>();   // V too
            __syncthreads();            // maxima are there, K is free
            if (t + 1 < it.tile1) copy(t + 1, p.k_cache, smem + S::K, true);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 16 * mt + g + 8 * h;
                    float now = m[mt][h];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) now = fmaxf(now, s_top[w * R + row]);
                    const float ref = now == -INFINITY ? 0.f : now, keep = exp2f(m[mt][h] - ref);
                    m[mt][h] = now;
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float w = exp2f(sc[mt][n][2 * h + e] - ref);
                            sum += w;
                            smem[S::P + a_place(row, 16 * warp + 8 * n + 2 * t4 + e, kTile / 8)] = w;
                        }
                    l[mt][h] = l[mt][h] * keep + sum;   // of this lane's tokens
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        o[mt][n][2 * h] *= keep;
                        o[mt][n][2 * h + 1] *= keep;
                    }
                }
            __syncthreads();            // P is there
            float acc[MT][NV][4], cross[MT][NV][4];
            // A value that is not finite spoils every row here, seen or not (and an infinity becomes a NaN): then the
            // tile's products are taken once more without such values, and the item's end adds them where they are seen.  (The
            // second time V's parts are cut: a value that rounds past the largest fp32 is finite.)
            uint32_t half = kNearest;
#pragma unroll 1
            for (bool again = false;; again = true, half = 0u) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NV; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][n][e] = cross[mt][n][e] = 0.f;
#pragma unroll 2
                for (int kk = 0; kk < kTile / 8; ++kk) {
                    uint32_t ah[MT][4], al[MT][4], bh[NV][2], bl[NV][2];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float4 w = load4(smem + S::P + ((mt * (kTile / 8) + kk) * 32 + lane) * 4);
                        split_tf32(w.x, ah[mt][0], al[mt][0]);
                        split_tf32(w.y, ah[mt][1], al[mt][1]);
                        split_tf32(w.z, ah[mt][2], al[mt][2]);
                        split_tf32(w.w, ah[mt][3], al[mt][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        const float *at = smem + S::V + v_place<HD>(8 * kk + t4, warp * (HD / 16) + 2 * n + (g >> 2)) + (g & 3);
                        split_tf32(at[0], bh[n][0], bl[n][0], half);
                        split_tf32(at[4 * HD], bh[n][1], bl[n][1], half);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < NV; ++n) mma_tf32(cross[mt][n], al[mt], bh[n][0], bh[n][1]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < NV; ++n) mma_tf32_add(acc[mt][n], ah[mt], bh[n][0], bh[n][1]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < NV; ++n) mma_tf32(cross[mt][n], ah[mt], bl[n][0], bl[n][1]);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NV; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][n][e] += cross[mt][n][e];
                float size = 0.f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NV; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) size += fabsf(acc[mt][n][e]);
                if (!__syncthreads_or(!isfinite(size)) || again) break;
#pragma unroll 1
                for (int i = tid; i < kTile * HD; i += kThreads) {
                    float *at = smem + S::V + i;
                    if (!isfinite(*at)) *at = 0.f;
                }
                if (tid == 0) {
                    s_odd[0] = min(s_odd[0], t);
                    s_odd[1] = t + 1;
                }
                __syncthreads();
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][n][e] += acc[mt][n][e];
            if (tid < pages) s_page[t & 1][tid] = next_page;
            if (t + 1 < it.tile1) copy(t + 1, p.v_cache, smem + S::V, false);
        }
        // Sums over the tokens of all warps.
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = l[mt][h];
                x += __shfl_xor_sync(kFull, x, 1);
                x += __shfl_xor_sync(kFull, x, 2);
                if (t4 == 0) s_top[warp * R + 16 * mt + g + 8 * h] = x;
            }
        __syncthreads();
        const bool whole = it.whole(), any_odd = s_odd[1] > 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 16 * mt + g + 8 * h;
                if (r >= rows) continue;
                const float all = (s_top[r] + s_top[R + r]) + (s_top[2 * R + r] + s_top[3 * R + r]);
                const float inv = !whole ? 1.f : (all == 0.f ? 0.f : 1.f / all);
                const long long at = static_cast<long long>(it.slot(blockIdx.x)) * p.slot_rows + r;
                float *dst = (whole ? static_cast<float *>(p.out) + multi_row(p, it.s, it.kvh, R0 + r, HD) : p.part_acc + at * HD) +
                             warp * (HD / 4) + 2 * t4;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    float2 x = make_float2(o[mt][n][2 * h] * inv, o[mt][n][2 * h + 1] * inv);
                    if (any_odd) {
                        const int tq = (R0 + r) / p.group;
                        for (int u = s_odd[0] * kTile; u < min(seen, s_odd[1] * kTile); ++u) {
                            const int b = table[u / p.block_size];
                            if (b < 0 || b >= p.num_blocks || !multi_sees(p, it.s, tq, u)) continue;
                            const float *v = static_cast<const float *>(p.v_cache) +
                                             ((static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size + u % p.block_size) * HD +
                                             warp * (HD / 4) + 2 * t4 + 8 * n;
                            if (!isfinite(v[0])) x.x += v[0];
                            if (!isfinite(v[1])) x.y += v[1];
                        }
                    }
                    *reinterpret_cast<float2 *>(dst + 8 * n) = x;
                }
                if (!whole && warp == 0 && t4 == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(m[mt][h], all);
            }
    }
}

template <int HD, int MT>
int multi_f32(const MultiParams &params, int dev, cudaStream_t st) {
    using S = Shape<HD, MT>;
    static host::KernelSlot slot;
    auto kernel = multi_f32_kernel<HD, MT>;
    const int occ = host::ensure_kernel(kernel, slot, S::BYTES, dev, kThreads);
    if (occ == 0) return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cannot configure the fp32 kernel");
    MultiParams p = params;
    p.slot_rows = min(p.slot_rows, S::R);
    const int grid = min(host::sm_count(dev) * min(occ, S::CTAS), kMultiFewCtas);
    const cudaError_t e = host::launch_dependent(kernel, grid, kThreads, S::BYTES, st, p);
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return launch_join<float, HD, typename S::Axis>(p, grid, st);
}

}  // namespace

int launch_multi_f32(const MultiParams &p, int head_dim, bool few, int dev, cudaStream_t st) {
    if (head_dim == 128) return few ? multi_f32<128, 1>(p, dev, st) : multi_f32<128, 2>(p, dev, st);
    return few ? multi_f32<64, 1>(p, dev, st) : multi_f32<64, 2>(p, dev, st);
}

}  // namespace pa
