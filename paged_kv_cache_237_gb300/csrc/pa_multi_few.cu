// pa_decode_tree and pa_decode_cross over bf16 caches, few rows per sequence: a
// decoder step's queries, beams, short drafts.
//
// An item is up to 16 rows (query tokens x the heads of one KV head) against a
// stretch of the sequence's cache.  The 16 rows of the tcgen05 pass's 128 would
// leave its tensor memory, its 384 threads and its long pipeline to eight times
// nothing, so these run as pa_decode's pass does: each of a CTA's 4 warps takes
// every fourth 16-token chunk through a ring of its own (TMA, a barrier per
// stage), rows are the M of mma.m16n8k16, p enters as two bf16 parts, and the
// warps' states are merged at the item's end.  Bound by HBM, and by latency where
// little is read: 16 requests of 1500 states and 4 queries, 16 heads of 64 (98 MB):
// 34 us with the join in a cold cache, 18.5 of it this pass, 5.3 TB/s (the tcgen05
// pass 46); 32 sequences of 2000..4000 tokens, 16 rows each of 8 KV heads of 128
// (0.4 GB): 87 us, 4.6 TB/s (100); one request of 777 tokens with 5 drafted: 20 us, of which 13 when
// other work runs before it.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_multi.cuh"

namespace pa {
namespace {

constexpr int kRows = 16, kThreads = kWarps * 32;
using Axis = MultiAxis<kRows, kRows, kWarps * kChunk, 2>;

template <int HD>
struct Ring {
    static constexpr int STAGES = HD == 128 ? 2 : 3, CTAS = HD == 128 ? 3 : 4;   // as pa_decode's pass
    static constexpr int HALVES = HD / 64, HALF_BYTES = kChunk * 128, PAGE = HALVES * HALF_BYTES, STAGE = 2 * PAGE;
    static constexpr int WARP = STAGES * STAGE, BYTES = kWarps * WARP + kWarps * STAGES * 8 + 1024;
    static constexpr int LD = HD + kEpiPad;
    static_assert(WARP >= (kRows * LD + 2 * kRows) * 4, "a warp's results must fit in its stages");
};

template <int HD>
__global__ void __launch_bounds__(kThreads, Ring<HD>::CTAS)
    multi_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const MultiParams p) {
    using M = Ring<HD>;
    constexpr int KT = HD / 16, NT = HD / 8, LD = M::LD;
    extern __shared__ uint8_t smem_raw[];
    __shared__ MultiSpot s_spot;
    __shared__ int s_dirty[kWarps];
    uint8_t *smem = align_1024(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t *wbuf = smem + warp * M::WARP;
    const uint32_t wbuf_s = smem_addr(wbuf), bar_s = smem_addr(smem + kWarps * M::WARP) + warp * M::STAGES * 8;
    if (lane == 0) {
        for (int s = 0; s < M::STAGES; ++s) mbar_init(bar_s + 8 * s, 1);
        fence_mbar_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    griddep_wait();
    int flags = 0;
    const MultiLocator<Axis, kThreads> loc(p, flags);
    if (flags && blockIdx.x == 0) flag_status(p.status, flags);
    const MultiSplit split(loc.total, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= split.ctas) return;
    const long long unit = split.start(blockIdx.x);
    long long left = split.start(blockIdx.x + 1) - unit;
    loc.find(p, unit, &s_spot);
    __syncthreads();
    MultiSpot spot = s_spot;
    const uint64_t once = l2_evict_first_policy(), again = l2_normal_policy();
    uint32_t n_issued = 0, n_done = 0;
    bool failed = false;

    MultiItem it;
    while (Axis::next(p, spot, left, it)) {
        const int R0 = it.m * kRows, rows = min(kRows, it.s.c * p.group - R0);
        const int seen = Axis::seen(p, it.s, it.m);
        const int clear = Axis::clear(p, it.s, it.m);   // every row sees every position before
        const int first = it.tile0 * kWarps, last = min(it.tile1 * kWarps, (seen + kChunk - 1) / kChunk);
        const int my_n = last > first + warp ? (last - first - warp + kWarps - 1) / kWarps : 0;
        const uint64_t policy = Axis::row_blocks(p, it.s) > 1 ? again : once;
        const int32_t *table = p.block_tables + static_cast<long long>(it.seq) * p.width;
        // Row of this warp's k-th chunk in the cache view; past the view for none (reads as zeros).
        const auto chunk_at = [&](int k) {
            if (k >= my_n) return p.total_rows;
            const int u = (first + warp + kWarps * k) * kChunk, b = table[u / p.block_size];
            if (b < 0 || b >= p.num_blocks) {
                flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                return p.total_rows;
            }
            return static_cast<int>((static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size + u % p.block_size);
        };
        int window = 0, now = chunk_at(lane), ahead = chunk_at(32 + lane);   // of 32 chunks, a lane each
        const auto issue = [&](int k) {
            const int here = __shfl_sync(kFull, now, k & 31), next = __shfl_sync(kFull, ahead, k & 31);
            if (failed) return;
            if (lane == 0) {
                const int row = k - window < 32 ? here : next;
                const uint32_t dst = wbuf_s + (n_issued % M::STAGES) * M::STAGE, bar = bar_s + 8 * (n_issued % M::STAGES);
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar, M::STAGE);
#pragma unroll
                for (int h = 0; h < M::HALVES; ++h) {
                    tma_load_2d_hint(dst + h * M::HALF_BYTES, &tmK, h * 64, row, bar, policy);
                    tma_load_2d_hint(dst + M::PAGE + h * M::HALF_BYTES, &tmV, h * 64, row, bar, policy);
                }
            }
            ++n_issued;
        };

        // Q fragments; rows behind the last are zero.
        const int r_lo = min(R0 + g, it.s.c * p.group - 1), r_hi = min(R0 + g + 8, it.s.c * p.group - 1);
        const int tok_lo = r_lo / p.group, tok_hi = r_hi / p.group;
        uint32_t qa[KT][4];
        {
            const __nv_bfloat16 *lo = static_cast<const __nv_bfloat16 *>(p.q) + multi_row(p, it.s, it.kvh, r_lo, HD);
            const __nv_bfloat16 *hi = static_cast<const __nv_bfloat16 *>(p.q) + multi_row(p, it.s, it.kvh, r_hi, HD);
            const bool lo_ok = g < rows, hi_ok = g + 8 < rows;
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                const int c = 16 * kk + 2 * t;
                qa[kk][0] = lo_ok ? *reinterpret_cast<const uint32_t *>(lo + c) : 0u;
                qa[kk][1] = hi_ok ? *reinterpret_cast<const uint32_t *>(hi + c) : 0u;
                qa[kk][2] = lo_ok ? *reinterpret_cast<const uint32_t *>(lo + c + 8) : 0u;
                qa[kk][3] = hi_ok ? *reinterpret_cast<const uint32_t *>(hi + c + 8) : 0u;
            }
        }
        for (int k = 0; k < min(my_n, M::STAGES); ++k) issue(k);

        float o[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
        bool dirty = false;
        for (int k = 0; k < my_n; ++k) {
            if (k - window >= 32) {
                window += 32;
                now = ahead;
                ahead = chunk_at(window + 32 + lane);
            }
            const int s = n_done % M::STAGES;
            const bool ok = !failed && mbar_wait_bounded(bar_s + 8 * s, (n_done / M::STAGES) & 1u);
            if (__any_sync(kFull, !ok)) {
                if (!failed && lane == 0) flag_status(p.status, PA_STATUS_WAIT_TIMEOUT);
                failed = true;
                break;
            }
            ++n_done;
            const uint32_t Ks = wbuf_s + s * M::STAGE, Vs = Ks + M::PAGE;
            const int u0 = (first + warp + kWarps * k) * kChunk;
            uint32_t see_lo = 0xffffu, see_hi = 0xffffu;
            if (u0 + kChunk > clear) {
                see_lo = multi_seen_bits(p, it.s, tok_lo, u0) & 0xffffu;
                see_hi = multi_seen_bits(p, it.s, tok_hi, u0) & 0xffffu;
                // Values that some row does not see: those behind the last seen token become zero, and so do values of
                // drafted tokens that are not finite (added again where they are seen).
                uint8_t *vt = wbuf + s * M::STAGE + M::PAGE;
                for (int i = lane; i < kChunk * M::HALVES * 8; i += 32) {
                    const int j = i / 8 % kChunk;   // token; the order of pieces does not matter
                    uint4 *at = reinterpret_cast<uint4 *>(vt + i * 16);
                    if (u0 + j >= seen) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else if (u0 + j >= clear) {
                        dirty |= clear_not_finite(*at);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            }

            // S = Q K^T over the 16 tokens (two n-tiles of 8 tokens).
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const int mi = lane >> 3;
            {
                const int r = (lane & 7) + ((mi >> 1) << 3);
#pragma unroll
                for (int kk = 0; kk < KT; ++kk) {
                    const int ch = 2 * kk + (mi & 1);
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4(Ks + (ch >> 3) * M::HALF_BYTES + r * 128 + (((ch & 7) ^ (r & 7)) << 4), b0, b1, b2, b3);
                    mma_bf16_16816(sc[0], qa[kk], b0, b1);
                    mma_bf16_16816(sc[1], qa[kk], b2, b3);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = 8 * nt + 2 * t + (j & 1);
                    sc[nt][j] = ((j < 2 ? see_lo : see_hi) >> tok) & 1u ? sc[nt][j] * p.scale_log2 : -INFINITY;
                }
            // Online softmax, base 2: row g in sc[.][0..1], row g + 8 in sc[.][2..3].
            float mx_lo = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
            float mx_hi = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
#pragma unroll
            for (int i = 1; i < 4; i <<= 1) {
                mx_lo = fmaxf(mx_lo, __shfl_xor_sync(kFull, mx_lo, i));
                mx_hi = fmaxf(mx_hi, __shfl_xor_sync(kFull, mx_hi, i));
            }
            const float mn_lo = fmaxf(m_lo, mx_lo), mn_hi = fmaxf(m_hi, mx_hi);
            const float ref_lo = mn_lo == -INFINITY ? 0.f : mn_lo, ref_hi = mn_hi == -INFINITY ? 0.f : mn_hi;
            const float alpha_lo = exp2f(m_lo - ref_lo), alpha_hi = exp2f(m_hi - ref_hi);
            m_lo = mn_lo;
            m_hi = mn_hi;
            float pr[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                pr[nt][0] = exp2f(sc[nt][0] - ref_lo);
                pr[nt][1] = exp2f(sc[nt][1] - ref_lo);
                pr[nt][2] = exp2f(sc[nt][2] - ref_hi);
                pr[nt][3] = exp2f(sc[nt][3] - ref_hi);
            }
            l_lo = l_lo * alpha_lo + ((pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]));
            l_hi = l_hi * alpha_hi + ((pr[0][2] + pr[0][3]) + (pr[1][2] + pr[1][3]));
            // p = hi + lo, both bf16, in the A fragment's order: (row g, 2t..), (g + 8, 2t..), (g, 8 + 2t..), (g + 8, 8 + 2t..)
            uint32_t pa[4], pb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float *x = &pr[e >> 1][2 * (e & 1)];
                weight_parts(make_float2(x[0], x[1]), pa[e], pb[e]);
            }
            if (__any_sync(kFull, alpha_lo != 1.f || alpha_hi != 1.f)) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][0] *= alpha_lo;
                    o[j][1] *= alpha_lo;
                    o[j][2] *= alpha_hi;
                    o[j][3] *= alpha_hi;
                }
            }
            // O += P V (k = 16 tokens, n = head_dim in tiles of 8).
            {
                const int r = (lane & 7) + ((mi & 1) << 3);
#pragma unroll
                for (int jj = 0; jj < KT; ++jj) {
                    const int ch = 2 * jj + (mi >> 1);
                    uint32_t b0, b1, b2, b3;
                    ldmatrix_x4_trans(Vs + (ch >> 3) * M::HALF_BYTES + r * 128 + (((ch & 7) ^ (r & 7)) << 4), b0, b1, b2, b3);
                    mma_bf16_16816(o[2 * jj], pa, b0, b1);
                    mma_bf16_16816(o[2 * jj + 1], pa, b2, b3);
                    mma_bf16_16816(o[2 * jj], pb, b0, b1);
                    mma_bf16_16816(o[2 * jj + 1], pb, b2, b3);
                }
            }
            __syncwarp();
            if (k + M::STAGES < my_n) issue(k + M::STAGES);
        }

        // This warp's state goes into its (now idle) stages, then all merge.
#pragma unroll
        for (int i = 1; i < 4; i <<= 1) {
            l_lo += __shfl_xor_sync(kFull, l_lo, i);
            l_hi += __shfl_xor_sync(kFull, l_hi, i);
        }
        {
            float *eo = reinterpret_cast<float *>(wbuf);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                *reinterpret_cast<float2 *>(eo + g * LD + 8 * j + 2 * t) = make_float2(o[j][0], o[j][1]);
                *reinterpret_cast<float2 *>(eo + (g + 8) * LD + 8 * j + 2 * t) = make_float2(o[j][2], o[j][3]);
            }
            if (t == 0) {
                eo[kRows * LD + g] = m_lo;
                eo[kRows * LD + g + 8] = m_hi;
                eo[kRows * LD + kRows + g] = l_lo;
                eo[kRows * LD + kRows + g + 8] = l_hi;
            }
            const bool any = __any_sync(kFull, dirty);
            if (lane == 0) s_dirty[warp] = any;
        }
        __syncthreads();
        const bool any_dirty = s_dirty[0] || s_dirty[1] || s_dirty[2] || s_dirty[3], whole = it.whole();
        for (int task = threadIdx.x; task < rows * (HD / 4); task += kThreads) {
            const int r = task / (HD / 4), d = task % (HD / 4) * 4;
            float top = -INFINITY, all = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top = fmaxf(top, reinterpret_cast<const float *>(smem + w * M::WARP)[kRows * LD + r]);
            const float ref = top == -INFINITY ? 0.f : top;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *eo = reinterpret_cast<const float *>(smem + w * M::WARP);
                const float f = exp2f(eo[kRows * LD + r] - ref);
                const float4 v = *reinterpret_cast<const float4 *>(eo + r * LD + d);
                all += f * eo[kRows * LD + kRows + r];
                acc.x += f * v.x;
                acc.y += f * v.y;
                acc.z += f * v.z;
                acc.w += f * v.w;
            }
            if (any_dirty) {
                const int tok = (R0 + r) / p.group;
                for (int u = max(max(clear, 0), first * kChunk); u < min(seen, last * kChunk); ++u) {
                    if (!multi_sees(p, it.s, tok, u)) continue;
                    const int b = table[u / p.block_size];
                    if (b < 0 || b >= p.num_blocks) continue;
                    const __nv_bfloat16 *vr =
                        static_cast<const __nv_bfloat16 *>(p.v_cache) +
                        ((static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size + u % p.block_size) * HD + d;
                    const float x[4] = {__bfloat162float(vr[0]), __bfloat162float(vr[1]), __bfloat162float(vr[2]),
                                        __bfloat162float(vr[3])};
                    if (!isfinite(x[0])) acc.x += x[0];
                    if (!isfinite(x[1])) acc.y += x[1];
                    if (!isfinite(x[2])) acc.z += x[2];
                    if (!isfinite(x[3])) acc.w += x[3];
                }
            }
            if (whole) {
                const float inv = all == 0.f ? 0.f : 1.f / all;
                store4(static_cast<__nv_bfloat16 *>(p.out) + multi_row(p, it.s, it.kvh, R0 + r, HD) + d,
                       make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
            } else {
                const long long at = static_cast<long long>(it.slot(blockIdx.x)) * p.slot_rows + r;
                store4(p.part_acc + at * HD + d, acc);
                if (d == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(top, all);
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
    }
    griddep_launch_dependents();
    // A wait gave up: let copies still in flight land before the CTA exits.
    if (failed && lane == 0)
        for (uint32_t i = n_done; i < n_issued; ++i) mbar_wait_bounded(bar_s + 8 * (i % M::STAGES), (i / M::STAGES) & 1u);
}

template <int HD>
int multi_few(const MultiParams &p, int dev, cudaStream_t st) {
    static host::KernelSlot slot;
    auto kernel = multi_few_kernel<HD>;
    const int occ = host::ensure_kernel(kernel, slot, Ring<HD>::BYTES, dev);
    if (occ == 0) return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cannot configure the bf16 kernel");
    CUtensorMap mk, mv;
    if (!host::make_map(&mk, p.k_cache, p.total_rows, HD) || !host::make_map(&mv, p.v_cache, p.total_rows, HD))
        return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cuTensorMapEncodeTiled failed");
    const int grid = min(host::sm_count(dev) * min(occ, Ring<HD>::CTAS), kMultiFewCtas);
    const cudaError_t e = host::launch_dependent(kernel, grid, kThreads, Ring<HD>::BYTES, st, mk, mv, p);
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return launch_join<__nv_bfloat16, HD, Axis>(p, grid, st);
}

}  // namespace

int launch_multi_few(const MultiParams &params, int head_dim, int dev, cudaStream_t st) {
    MultiParams p = params;
    p.slot_rows = static_cast<int>(min(static_cast<long long>(p.num_tokens) * p.group, static_cast<long long>(kRows)));
    return head_dim == 128 ? multi_few<128>(p, dev, st) : multi_few<64>(p, dev, st);
}

}  // namespace pa
