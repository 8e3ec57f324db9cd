// pa_decode_tree and pa_decode_cross over fp32 caches, on fp32 FMAs.
//
// An item is R rows (query tokens x the heads of one KV head) against a stretch
// of the sequence's cache in tiles of 64 tokens.  A thread holds four rows: of a
// tile's scores those of 64 / L tokens, of the sums O head_dim / L columns, where
// L lanes share the rows' group.
//   R = 16, L = 32 (128 threads): few rows per sequence.  Bound by the copies and,
//     near it, by shared memory: a row's group reads all of K and V.
//   R = 64, L = 16 (256 threads): many rows.  Bound by the FMAs: 16 scores take
//     8 loads of 16 bytes for 64 FMAs.
// K of the next tile is copied (cp.async) while this one's softmax and products
// run, V while the next scores do; two CTAs per SM fill each other's gaps.
// FMAs are packed in pairs: two steps of head_dim for the scores, two columns for
// the products.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pa_multi.cuh"

namespace pa {
namespace {

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float4 load4(const float *x) { return *reinterpret_cast<const float4 *>(x); }

template <int HD, int R>
struct Shape {
    static constexpr int T = R == 16 ? 32 : 64;                // tokens per tile
    static constexpr int L = R == 16 ? 32 : 16, THREADS = R / 4 * L;
    static constexpr int TOK = T / L, COLS = HD / L;       // a thread's tokens and columns
    static constexpr int LDK = HD + 4, LDP = R + 4;            // padded rows of Q and K, and of P (by token)
    // P lies over K where two CTAs would not fit an SM otherwise; the next K then waits for the products.
    static constexpr bool OVER = HD == 128 && R == 64;
    static constexpr int Q = 0, K = Q + R * LDK, V = K + T * LDK, P = OVER ? K : V + T * HD;
    static constexpr int FLOATS = OVER ? V + T * HD : P + T * LDP;
    static constexpr int BYTES = FLOATS * 4;
    static constexpr int CTAS = R == 64 ? 2 : 4;               // per SM
    using Axis = MultiAxis<R, R, T, 2>;
};

template <int HD, int R>
__global__ void __launch_bounds__(Shape<HD, R>::THREADS, Shape<HD, R>::CTAS) multi_simt_kernel(const MultiParams p) {
    using S = Shape<HD, R>;
    using Axis = typename S::Axis;
    constexpr int kTile = S::T, L = S::L, THREADS = S::THREADS, TOK = S::TOK, COLS = S::COLS, VEC = COLS < 4 ? COLS : 4;
    extern __shared__ __align__(16) float smem[];
    __shared__ MultiSpot s_spot;
    __shared__ int s_page[2][kTile / 16];
    __shared__ int s_dirty;
    griddep_wait();
    const int tid = threadIdx.x, ty = tid / L, tx = tid % L;   // rows 4 ty .. 4 ty + 3; tokens tx + L j
    int flags = 0;
    const MultiLocator<Axis, THREADS> loc(p, flags);
    if (flags && blockIdx.x == 0) flag_status(p.status, flags);
    const MultiSplit split(loc.total, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= split.ctas) return;
    const long long unit = split.start(blockIdx.x);
    long long left = split.start(blockIdx.x + 1) - unit;
    loc.find(p, unit, &s_spot);
    if (tid == 0) s_dirty = 0;
    __syncthreads();
    MultiSpot spot = s_spot;
    const int pages = kTile / p.block_size;

    MultiItem it;
    while (Axis::next(p, spot, left, it)) {
        const int R0 = it.m * R, rows = min(R, it.s.c * p.group - R0);
        const int seen = Axis::seen(p, it.s, it.m), base = it.s.n - it.s.c;
        const int clear = p.see == kSeeAll ? it.s.n : base;   // every row sees every position before
        const int32_t *table = p.block_tables + static_cast<long long>(it.seq) * p.width;
        // First row of a page in the cache view; -1 for none (zeros).
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
        const auto copy = [&](int t, const void *cache, float *dst, int ld) {
            const float *src = static_cast<const float *>(cache);
#pragma unroll 4
            for (int i = tid; i < kTile * (HD / 4); i += THREADS) {
                const int j = i / (HD / 4), c = i % (HD / 4) * 4, at = j / p.block_size;
                const int row = s_page[t & 1][at];
                if (row >= 0 && t * kTile + j < seen)
                    cp_async_16(smem_addr(dst + j * ld + c), src + (static_cast<long long>(row) + j - at * p.block_size) * HD + c);
                else
                    store4(dst + j * ld + c, make_float4(0.f, 0.f, 0.f, 0.f));
            }
            cp_async_commit();
        };
        __syncthreads();   // the item before is done with the shared memory
        if (tid < 2 * pages) s_page[(it.tile0 + tid / pages) & 1][tid % pages] = page_row(it.tile0 + tid / pages, tid % pages);
        for (int i = tid; i < R * (HD / 4); i += THREADS) {
            const int r = i / (HD / 4), c = i % (HD / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) x = load4(static_cast<const float *>(p.q) + multi_row(p, it.s, it.kvh, R0 + r, HD) + c);
            store4(smem + S::Q + r * S::LDK + c, make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2,
                                                             x.w * p.scale_log2));
        }
        __syncthreads();
        copy(it.tile0, p.k_cache, smem + S::K, S::LDK);
        copy(it.tile0, p.v_cache, smem + S::V, HD);

        int tok[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) tok[a] = min(R0 + 4 * ty + a, it.s.c * p.group - 1) / p.group;
        float m[4], l[4];
        float2 o[4][(COLS + 1) / 2];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            m[a] = -INFINITY;
            l[a] = 0.f;
#pragma unroll
            for (int c = 0; c < COLS / 2; ++c) o[a][c] = make_float2(0.f, 0.f);
        }
        for (int t = it.tile0; t < it.tile1; ++t) {
            const int u0 = t * kTile;
            int next_page = -1;
            if (tid < pages) next_page = page_row(t + 2, tid);
            cp_async_wait_group<1>();   // K is there, V may be on its way
            __syncthreads();
            float2 acc[4][TOK];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < TOK; ++j) acc[a][j] = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int d = 0; d < HD; d += 4) {
                float4 k[TOK];
#pragma unroll
                for (int j = 0; j < TOK; ++j) k[j] = load4(smem + S::K + (tx + L * j) * S::LDK + d);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const float4 q = load4(smem + S::Q + (4 * ty + a) * S::LDK + d);
#pragma unroll
                    for (int j = 0; j < TOK; ++j) {
                        acc[a][j] = fma2(make_float2(q.x, q.y), make_float2(k[j].x, k[j].y), acc[a][j]);
                        acc[a][j] = fma2(make_float2(q.z, q.w), make_float2(k[j].z, k[j].w), acc[a][j]);
                    }
                }
            }
            const bool masked = u0 + kTile > clear;
            cp_async_wait_group<0>();   // V too
            if (masked) {
                // values of drafted tokens that are not finite must not meet the zero weights of rows that do not see them
                for (int i = tid; i < kTile * (HD / 4); i += THREADS) {
                    const float4 v = load4(smem + S::V + i * 4);
                    if (!(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) s_dirty = 1;
                }
            }
            if (S::OVER || masked) __syncthreads();   // all are done with K; all have looked at V
            const bool dirty = masked && s_dirty;
            float w[4][TOK];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                bool see[TOK];
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < TOK; ++j) {
                    const int u = u0 + tx + L * j;
                    float x = acc[a][j].x + acc[a][j].y;
                    see[j] = !masked || (u < it.s.n && multi_sees(p, it.s, tok[a], u));
                    if (!see[j]) x = -INFINITY;
                    top = fmaxf(top, x);
                    w[a][j] = x;
                }
#pragma unroll
                for (int i = 1; i < L; i <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
                const float now = fmaxf(m[a], top), ref = now == -INFINITY ? 0.f : now;
                const float keep = exp2f(m[a] - ref);
                m[a] = now;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < TOK; ++j) {
                    const float e = exp2f(w[a][j] - ref);
                    sum += e;
                    w[a][j] = see[j] || !dirty ? e : -1.f;   // -1: not seen
                }
                l[a] = l[a] * keep + sum;   // of this thread's tokens
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) {
                    o[a][c].x *= keep;
                    o[a][c].y *= keep;
                }
            }
#pragma unroll
            for (int j = 0; j < TOK; ++j)
                store4(smem + S::P + (tx + L * j) * S::LDP + 4 * ty, make_float4(w[0][j], w[1][j], w[2][j], w[3][j]));
            __syncthreads();   // P is there, K is free
            if (!S::OVER && t + 1 < it.tile1) copy(t + 1, p.k_cache, smem + S::K, S::LDK);
            const auto products = [&](auto slow) {
#pragma unroll 4
                for (int j = 0; j < kTile; ++j) {
                    const float4 pw = load4(smem + S::P + j * S::LDP + 4 * ty);
                    const float wa[4] = {pw.x, pw.y, pw.z, pw.w};
#pragma unroll
                    for (int c = 0; c < COLS / VEC; ++c) {
                        float v[VEC];
                        const float *at = smem + S::V + j * HD + tx * VEC + L * VEC * c;
                        if constexpr (VEC == 4)
                            *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(at);
                        else
                            *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(at);
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            if (decltype(slow)::value && wa[a] < 0.f) continue;
#pragma unroll
                            for (int e = 0; e < VEC / 2; ++e)
                                o[a][c * (VEC / 2) + e] = fma2(make_float2(wa[a], wa[a]), make_float2(v[2 * e], v[2 * e + 1]),
                                                               o[a][c * (VEC / 2) + e]);
                        }
                    }
                }
            };
            if (dirty)
                products(std::true_type{});
            else
                products(std::false_type{});
            __syncthreads();   // V (and P) are free
            if (tid < pages) s_page[t & 1][tid] = next_page;
            if (masked && tid == 0) s_dirty = 0;
            if (t + 1 < it.tile1) {
                if (S::OVER) copy(t + 1, p.k_cache, smem + S::K, S::LDK);
                copy(t + 1, p.v_cache, smem + S::V, HD);
            }
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float all = l[a];
#pragma unroll
            for (int i = 1; i < L; i <<= 1) all += __shfl_xor_sync(kFull, all, i);
            const int r = 4 * ty + a;
            if (r >= rows) continue;
            const bool whole = it.whole();
            const float inv = !whole ? 1.f : (all == 0.f ? 0.f : 1.f / all);
            const long long at = static_cast<long long>(it.slot(blockIdx.x)) * p.slot_rows + r;
            float *dst = whole ? static_cast<float *>(p.out) + multi_row(p, it.s, it.kvh, R0 + r, HD) : p.part_acc + at * HD;
#pragma unroll
            for (int c = 0; c < COLS / VEC; ++c) {
                const float2 *x = &o[a][c * (VEC / 2)];
                if constexpr (VEC == 4)
                    store4(dst + tx * VEC + L * VEC * c, make_float4(x[0].x * inv, x[0].y * inv, x[1].x * inv, x[1].y * inv));
                else
                    *reinterpret_cast<float2 *>(dst + tx * VEC + L * VEC * c) = make_float2(x[0].x * inv, x[0].y * inv);
            }
            if (!whole && tx == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(m[a], all);
        }
    }
}

template <int HD, int R>
int multi_simt(const MultiParams &p, int dev, cudaStream_t st) {
    using S = Shape<HD, R>;
    static host::KernelSlot slot;
    auto kernel = multi_simt_kernel<HD, R>;
    const int occ = host::ensure_kernel(kernel, slot, S::BYTES, dev, S::THREADS);
    if (occ == 0) return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cannot configure the fp32 kernel");
    const int grid = min(host::sm_count(dev) * min(occ, 4), kMultiSimtCtas);
    const cudaError_t e = host::launch_dependent(kernel, grid, S::THREADS, S::BYTES, st, p);
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return launch_join<float, HD, typename S::Axis>(p, grid, st);
}

}  // namespace

int launch_multi_simt(const MultiParams &p, int head_dim, int dev, cudaStream_t st) {
    // By the batch's average rows per sequence and KV head (all that the host knows): items of 16 rows up to 24.
    const bool few = static_cast<long long>(p.num_tokens) * p.group <= 24ll * p.num_seqs;
    if (head_dim == 128) return few ? multi_simt<128, 16>(p, dev, st) : multi_simt<128, 64>(p, dev, st);
    return few ? multi_simt<64, 16>(p, dev, st) : multi_simt<64, 64>(p, dev, st);
}

}  // namespace pa
