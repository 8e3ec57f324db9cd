// Decode attention over the 4-bit paged cache (include/pa.h states the
// format), partition pass for sm_103a.
//
// For a query row q and a token t with codes c, steps s_g and minima m_g:
//   q . K_t = sum_g s_g (sum_{d in g} q_d c_d) + m_g (sum_{d in g} q_d)
//   o_d     = sum_t p_t (s_g c_td + m_g)
// Work items, hand-out, the merge of the warps' states and the split-K merge
// are those of the other passes (pa_decode_common.cuh).
//
// The products run on fp16 tensor-core MMAs with tokens as rows of both: S = K
// Q^T has K's codes as its A operand, O^T = V^T W has V's.  With tokens as
// rows, up to eight query heads are one tile of columns.  For bf16 q and out, a
// code masked out of its word is already the fp16 subnormal code * 2^-24 (the
// next nibble up: code * 2^-20), so unpacking eight codes is one shift and four
// ands, and the powers of two are undone where they cost nothing, in q and in
// the output.  The tensor core aligns a subnormal's products by its nominal
// exponent, which leaves sums about 17 bits: plenty for a bf16 result (8), not
// for fp32.  fp32 q and out take codes as the normal value 16 + code (the 16
// goes into the minimum: s c + m = s (16 + c) + (m - 16 s)), and two fp16 parts
// of q and of the weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>

#include "pa_decode_common.cuh"
#include "pa_q4.cuh"

namespace pa {
namespace {

// Four consecutive values of a q row.
__device__ __forceinline__ float4 load_unit(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load_unit(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
    __half2 h;
    memcpy(&h, &u, 4);
    return __half22float2(h);
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The two nibble pairs (a nibble of each half-word) at a time that make the
// codes of two units fp16 operands: values 0, 1, 2, 3 of both units.  NORMAL:
// 16 + code.  Otherwise code * 2^-24, and code * 2^-20 for values 1 and 3.
template <bool NORMAL>
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t (&r)[4]) {
    if constexpr (NORMAL) {
        r[0] = ((x << 6) & 0x03c003c0u) | 0x4c004c00u;
        r[1] = ((x << 2) & 0x03c003c0u) | 0x4c004c00u;
        r[2] = ((x >> 2) & 0x03c003c0u) | 0x4c004c00u;
        r[3] = ((x >> 6) & 0x03c003c0u) | 0x4c004c00u;
    } else {
        r[0] = x & 0x000f000fu;
        r[1] = x & 0x00f000f0u;
        x >>= 8;
        r[2] = x & 0x000f000fu;
        r[3] = x & 0x00f000f0u;
    }
}

// The smallest power of two above x >= 0, within [2^-100, 2^120].
__device__ __forceinline__ float pow2_above(float x) {
    const float c = fminf(fmaxf(x, 0x1p-101f), 0x1p119f);
    return __uint_as_float((__float_as_uint(c) + 0x800000u) & 0x7f800000u);
}

// Launch shape per head_dim: stages per warp and the CTAs per SM the kernel is
// built for.
template <int HD, int NT>
struct Q4Shape {
    static constexpr int NSTAGE = HD == 128 ? 2 : 3;
    static constexpr int CPS = NT == 2 ? 2 : 3;
};

constexpr int kUnit = 32;   // tokens per stage: one block of 32 or two of 16

// T: type of q and out.  fp32 splits q and the weights into two fp16 parts.
// NT: tiles of 8 query heads per work item.
template <typename T, int HD, int G, int NT>
__global__ void __launch_bounds__(kWarps * 32, Q4Shape<HD, NT>::CPS)
    decode_q4_kernel(const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache, const DecodeParams p) {
    using F = Q4Format<HD, G>;
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int PARTS = SPLIT ? 2 : 1;
    constexpr int NSTAGE = Q4Shape<HD, NT>::NSTAGE;
    constexpr int W = F::W, NG = F::GROUPS;
    constexpr int HALF_BYTES = kUnit * F::ROW_BYTES;   // a stage's K, then its V
    constexpr int STAGE_BYTES = 2 * HALF_BYTES;
    constexpr int WARP_BYTES = NSTAGE * STAGE_BYTES;
    constexpr int ROWS = 8 * NT;
    constexpr int LD = HD + kEpiPad;
    constexpr int OW = HD / 32;    // code words a lane feeds to one token row's products
    constexpr int MT = HD / 16;    // m-tiles of the output
    static_assert(WARP_BYTES >= (ROWS * LD + 2 * ROWS) * 4, "epilogue tile must fit in a warp's stages");

    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t *wbuf = smem + warp * WARP_BYTES;
    const uint32_t wbuf_s = smem_addr(wbuf);
    const uint32_t bar_s = smem_addr(smem + kWarps * WARP_BYTES) + warp * NSTAGE * 8;
    if (lane == 0) {
        for (int s = 0; s < NSTAGE; ++s) mbar_init(bar_s + 8 * s, 1);
        fence_mbar_init();
    }
    __syncwarp();

    // Where the 16-token halves of a stage begin: two pages, or one of 32 rows.
    const int bs = p.block_size;
    const int page_bytes = bs * F::ROW_BYTES;
    const int code_half = bs == 16 ? page_bytes : 16 * F::CODE_BYTES;
    const int par_0 = bs * F::CODE_BYTES, par_half = bs == 16 ? page_bytes : 16 * F::PARAM_BYTES;
    // Token of matrix row g (row g + 8 is 8 further): neighbours swapped in
    // every other pair, so that a lane octet's reads of V hit both halves of
    // the banks.
    const int row_g = g ^ ((g >> 1) & 1);
    const int tok_a = (2 * t) ^ (t & 1), tok_b = (2 * t + 1) ^ (t & 1);   // matrix rows 2 t and 2 t + 1

    uint32_t n_issued = 0, n_done = 0;
    bool failed = false;
    SeqCursor cur{0, 0};
    const uint64_t kv_policy = l2_evict_first_policy();
    griddep_wait();   // everything above touched only this CTA's registers and shared memory

    __shared__ long long s_next[2];
    const bool dynamic = p.work_ctr != nullptr;
    long long ahead = 0;
    if (dynamic && threadIdx.x == 0) ahead = gridDim.x + next_handout(p.work_ctr);
    int nb = 0;
    for (long long item = blockIdx.x;;) {
        Item it;
        if (!next_item<true>(it, cur, item, p, ROWS, lane)) break;
        const int units = (it.tok_end - it.tok_begin + kUnit - 1) / kUnit;
        const int my_n = units > warp ? (units - warp + kWarps - 1) / kWarps : 0;   // at most 32

        // Pages of this warp's units: lane k holds unit k's first and (block
        // size 16) second, as block * heads + head; -1 is a block id out of
        // range, -2 a page past the item's tokens.
        long long page_a = -2, page_b = -2;
        auto page_of = [&](int v) -> long long {
            if (v >= it.tok_end) return -2;
            const int phys = p.block_tables[(long long)it.seq * p.max_blocks_per_seq + token_pos<true>(p, it, v) / bs];
            if (phys < 0 || phys >= p.num_blocks) {
                flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                return -1;
            }
            return (long long)phys * p.num_kv_heads + it.kvh;
        };
        if (lane < my_n) {
            const int v = it.tok_begin + (warp + kWarps * lane) * kUnit;
            page_a = page_of(v);
            if (bs == 16) page_b = page_of(v + 16);
        }
        auto issue = [&](int k) {
            const long long a = __shfl_sync(kFull, page_a, k), b = __shfl_sync(kFull, page_b, k);
            if (failed) return;
            if (lane == 0) {
                const int s = n_issued % NSTAGE;
                const uint32_t dst = wbuf_s + s * STAGE_BYTES, bar = bar_s + 8 * s;
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar, ((a >= 0) + (b >= 0)) * 2 * page_bytes);
                if (a >= 0) {
                    bulk_load_hint(dst, k_cache + a * page_bytes, page_bytes, bar, kv_policy);
                    bulk_load_hint(dst + HALF_BYTES, v_cache + a * page_bytes, page_bytes, bar, kv_policy);
                }
                if (b >= 0) {
                    bulk_load_hint(dst + page_bytes, k_cache + b * page_bytes, page_bytes, bar, kv_policy);
                    bulk_load_hint(dst + HALF_BYTES + page_bytes, v_cache + b * page_bytes, page_bytes, bar, kv_policy);
                }
            }
            ++n_issued;
        };
        const int pro = my_n < NSTAGE ? my_n : NSTAGE;
        for (int k = 0; k < pro; ++k) issue(k);

        // q as B operands: lane (g, t) holds head g of each tile, the units of
        // its code words, divided by a power of two that brings the row's
        // largest magnitude into [2^14, 2^15) (exact for bf16: 8 bits of an
        // fp16's 11), and by 16 where a code comes out 16 times too large.
        uint32_t qf[PARTS][NT][OW][4];
        float qs[NT][2];            // per column (head): undoes the scaling, times scale * log2(e)
        float qsum[NT][2][NG];      // sum of q over a group, times scale * log2(e)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = 8 * nt + g;
            const bool live = head < it.rows;
            const T *qb = static_cast<const T *>(p.q) +
                          ((long long)it.seq * p.num_q_heads + it.qh0 + (live ? head : 0)) * HD;
            float4 lo[OW], hi[OW];
            float top = 0.f, sum[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < OW; ++j) {
                const int u = G == 64 ? 16 * (j / 2) + 2 * t + (j & 1) : 8 * j + 2 * t;
                lo[j] = hi[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live) {
                    lo[j] = load_unit(qb + 4 * u);
                    hi[j] = load_unit(qb + 4 * (G == 64 ? u + 8 : u + 1));
                }
                top = fmaxf(top, fmaxf(fmaxf(fmaxf(fabsf(lo[j].x), fabsf(lo[j].y)), fmaxf(fabsf(lo[j].z), fabsf(lo[j].w))),
                                       fmaxf(fmaxf(fabsf(hi[j].x), fabsf(hi[j].y)), fmaxf(fabsf(hi[j].z), fabsf(hi[j].w)))));
                sum[G == 64 ? j / 2 : j] += ((lo[j].x + lo[j].y) + (lo[j].z + lo[j].w)) +
                                            ((hi[j].x + hi[j].y) + (hi[j].z + hi[j].w));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
#pragma unroll
                for (int i = 0; i < NG; ++i) sum[i] += __shfl_xor_sync(kFull, sum[i], o);
            }
            const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -126);
            const float f = pow2i(-e), f16th = SPLIT ? f : f * 0.0625f;
#pragma unroll
            for (int j = 0; j < OW; ++j) {
                const float x[4][2] = {{lo[j].x * f, hi[j].x * f}, {lo[j].y * f16th, hi[j].y * f16th},
                                       {lo[j].z * f, hi[j].z * f}, {lo[j].w * f16th, hi[j].w * f16th}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qf[0][nt][j][i] = pack_f16(x[i][0], x[i][1]);
                    if constexpr (SPLIT) {
                        const float2 h = unpack_f16(qf[0][nt][j][i]);
                        qf[PARTS - 1][nt][j][i] = pack_f16(x[i][0] - h.x, x[i][1] - h.y);
                    }
                }
            }
            // To the columns of the accumulators: heads 2 t and 2 t + 1.
            const float back = p.scale_log2 * (SPLIT ? 1.f : 0x1p24f) * pow2i(e);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                qs[nt][c] = __shfl_sync(kFull, back, 4 * (2 * t + c));
#pragma unroll
                for (int i = 0; i < NG; ++i) qsum[nt][c][i] = __shfl_sync(kFull, sum[i] * p.scale_log2, 4 * (2 * t + c));
            }
        }

        float o[MT][NT][4];          // [row g or g + 8][column]: sums of w * code, see below
        float om[NT][2][NG];         // this lane's tokens' sum of p * m
        float ref[NT][2], l[NT][2];
        float S[NG], inv[NG];        // w = p * s * inv, inv = 2^7 / S
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            S[i] = 0x1p-100f;
            inv[i] = 0x1p107f;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                ref[nt][c] = -0x1p126f;
                l[nt][c] = 0.f;
#pragma unroll
                for (int i = 0; i < NG; ++i) om[nt][c][i] = 0.f;
            }
        }

        for (int k = 0; k < my_n; ++k) {
            const int s = n_done % NSTAGE;
            bool ok = !failed && mbar_wait_bounded(bar_s + 8 * s, (n_done / NSTAGE) & 1u);
            if (__any_sync(kFull, !ok)) {
                if (!failed && lane == 0) flag_status(p.status, PA_STATUS_WAIT_TIMEOUT);
                failed = true;
                break;
            }
            ++n_done;
            uint8_t *stage = wbuf + s * STAGE_BYTES;
            const int v0 = it.tok_begin + (warp + kWarps * k) * kUnit;
            {
                // A block id out of range reads as zeros.
                const bool bad_a = __shfl_sync(kFull, page_a, k) == -1, bad_b = __shfl_sync(kFull, page_b, k) == -1;
                if (bad_a || bad_b) {
                    for (int i = lane * 4; i < page_bytes; i += 128)
                        for (int h = 0; h < 2; ++h) {
                            if (bad_a) *reinterpret_cast<uint32_t *>(stage + h * HALF_BYTES + i) = 0u;
                            if (bad_b) *reinterpret_cast<uint32_t *>(stage + h * HALF_BYTES + page_bytes + i) = 0u;
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int v = v0 + 16 * half;
                if (v >= it.tok_end) break;
                const uint32_t mask = window_mask(p, it.n, token_pos<true>(p, it, v), it.tok_end - v);
                if (!mask) continue;
                const uint8_t *Kc = stage + half * code_half, *Kp = stage + par_0 + half * par_half;
                const uint8_t *Vc = Kc + HALF_BYTES, *Vp = Kp + HALF_BYTES;
                const bool seen0 = (mask >> row_g) & 1u, seen1 = (mask >> (row_g + 8)) & 1u;

                // ---- S = K Q^T: rows are tokens, columns heads; one accumulator per group.
                float acc[NT][NG][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < NG; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
                {
                    uint32_t w0[OW], w1[OW];   // the lane's words of rows g and g + 8
                    const uint8_t *r0 = Kc + row_g * F::CODE_BYTES + t * 4 * OW, *r1 = r0 + 8 * F::CODE_BYTES;
                    if constexpr (OW == 4) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(r0), y = *reinterpret_cast<const uint4 *>(r1);
                        w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
                        w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(r0), y = *reinterpret_cast<const uint2 *>(r1);
                        w0[0] = x.x, w0[1] = x.y;
                        w1[0] = y.x, w1[1] = y.y;
                    }
#pragma unroll
                    for (int j = 0; j < OW; ++j) {
                        uint32_t x, y;
                        if constexpr (G == 64) {
                            const int i = W * (j & 1) + j / 2;   // word (2 t + (j & 1), j / 2)
                            x = w0[i];
                            y = w1[i];
                        } else {
                            // halves of words (2 t, j / 2) and (2 t + 1, j / 2): one group each
                            x = __byte_perm(w0[j / 2], w0[W + j / 2], j & 1 ? 0x7632 : 0x5410);
                            y = __byte_perm(w1[j / 2], w1[W + j / 2], j & 1 ? 0x7632 : 0x5410);
                        }
                        uint32_t xr[4], yr[4];
                        codes_f16<SPLIT>(x, xr);
                        codes_f16<SPLIT>(y, yr);
                        const uint32_t a0[4] = {xr[0], yr[0], xr[1], yr[1]}, a1[4] = {xr[2], yr[2], xr[3], yr[3]};
                        const int i = G == 64 ? j / 2 : j;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int q = 0; q < PARTS; ++q) {
                                mma_f16_16816(acc[nt][i], a0, qf[q][nt][j][0], qf[q][nt][j][1]);
                                mma_f16_16816(acc[nt][i], a1, qf[q][nt][j][2], qf[q][nt][j][3]);
                            }
                    }
                }

                float sc[NT][4];
                {
                    uint32_t kp[2][NG];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t *pp = reinterpret_cast<const uint32_t *>(Kp + (row_g + 8 * r) * F::PARAM_BYTES);
#pragma unroll
                        for (int i = 0; i < NG; ++i) kp[r][i] = pp[i];
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int r = c >> 1, col = c & 1;
                            float x = 0.f, y = 0.f;
#pragma unroll
                            for (int i = 0; i < NG; ++i) {
                                x = fmaf(q4_step(kp[r][i]), acc[nt][i][c], x);
                                y = fmaf(SPLIT ? fmaf(-16.f, q4_step(kp[r][i]), q4_min(kp[r][i])) : q4_min(kp[r][i]),
                                         qsum[nt][col][i], y);
                            }
                            sc[nt][c] = (r ? seen1 : seen0) ? fmaf(x, qs[nt][col], y) : -INFINITY;
                        }
                }

                // ---- weights.  w = p s / S in fp16 carries the value's step, so
                // that the codes enter the second product as they are.
                float sv[2][NG], mv[2][NG];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t *pp = reinterpret_cast<const uint32_t *>(Vp + (row_g + 8 * r) * F::PARAM_BYTES);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        const uint32_t pair = (r ? seen1 : seen0) ? pp[i] : 0u;
                        sv[r][i] = q4_step(pair);
                        mv[r][i] = SPLIT ? fmaf(-16.f, sv[r][i], q4_min(pair)) : q4_min(pair);
                    }
                }
                float pr[NT][4], w[NT][NG][4], most = 0.f;
                bool far = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float x = sc[nt][c] - ref[nt][c & 1];
                        far |= x > 8.f;
                        pr[nt][c] = exp2f(x);
#pragma unroll
                        for (int i = 0; i < NG; ++i) {
                            w[nt][i][c] = pr[nt][c] * (sv[c >> 1][i] * inv[i]);
                            most = fmaxf(most, w[nt][i][c]);
                        }
                    }
                if (__any_sync(kFull, far || most > 32768.f)) {
                    // A score 8 above its reference, or a weight past fp16's
                    // range: raise the references to the running maxima and
                    // choose S anew.  Rare after a sequence's first tokens.
                    float alpha[NT][2], keep = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float mx = fmaxf(sc[nt][c], sc[nt][c + 2]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                            const float now = fmaxf(ref[nt][c], mx);
                            alpha[nt][c] = exp2f(ref[nt][c] - now);
                            ref[nt][c] = now;
                            l[nt][c] *= alpha[nt][c];
                            keep = fmaxf(keep, alpha[nt][c]);
#pragma unroll
                            for (int i = 0; i < NG; ++i) om[nt][c][i] *= alpha[nt][c];
                        }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) pr[nt][c] = exp2f(sc[nt][c] - ref[nt][c & 1]);
                    float ratio[NG];
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        float mx = 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) mx = fmaxf(mx, pr[nt][c] * sv[c >> 1][i]);
                        mx = fmaxf(mx, keep * S[i]);
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                        const float now = pow2_above(mx);
                        ratio[i] = S[i] / now;
                        S[i] = now;
                        inv[i] = 0x1p7f / now;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) w[nt][i][c] = pr[nt][c] * (sv[c >> 1][i] * inv[i]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float r = ratio[G == 64 ? mt / 4 : mt / 2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[mt][nt][c] *= alpha[nt][c & 1] * r;
                    }
                }
                uint32_t pb[PARTS][NT][NG][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        l[nt][c] += pr[nt][c] + pr[nt][c + 2];
#pragma unroll
                        for (int i = 0; i < NG; ++i)
                            om[nt][c][i] = fmaf(pr[nt][c], mv[0][i], fmaf(pr[nt][c + 2], mv[1][i], om[nt][c][i]));
                    }
#pragma unroll
                    for (int i = 0; i < NG; ++i)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float x = w[nt][i][2 * r], y = w[nt][i][2 * r + 1];
                            const uint32_t h = pack_f16(x, y);
                            pb[0][nt][i][r] = movmatrix_trans(h);
                            if constexpr (SPLIT) {
                                const float2 b = unpack_f16(h);
                                pb[PARTS - 1][nt][i][r] = movmatrix_trans(pack_f16(x - b.x, y - b.y));
                            }
                        }
                }

                // ---- O += V^T W: rows are values, k is the tokens.
                {
                    const uint8_t *va = Vc + g * 4 * W;
                    uint32_t x[4][W];   // tokens of matrix rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = (i & 1 ? tok_b : tok_a) + (i & 2 ? 8 : 0);
                        const uint8_t *at = va + tok * F::CODE_BYTES;
                        if constexpr (W == 2) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(at);
                            x[i][0] = v.x, x[i][1] = v.y;
                        } else {
                            x[i][0] = *reinterpret_cast<const uint32_t *>(at);
                        }
                    }
#pragma unroll
                    for (int wd = 0; wd < W; ++wd)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t sel = hf ? 0x7632 : 0x5410;
                            uint32_t y[4], z[4];
                            codes_f16<SPLIT>(__byte_perm(x[0][wd], x[1][wd], sel), y);
                            codes_f16<SPLIT>(__byte_perm(x[2][wd], x[3][wd], sel), z);
                            const int i = G == 64 ? wd : 2 * wd + hf;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t a[4] = {y[2 * e], y[2 * e + 1], z[2 * e], z[2 * e + 1]};
                                const int mt = 4 * wd + 2 * hf + e;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int q = 0; q < PARTS; ++q)
                                        mma_f16_16816(o[mt][nt], a, pb[q][nt][i][0], pb[q][nt][i][1]);
                            }
                        }
                }
            }
            __syncwarp();
            if (k + NSTAGE < my_n) issue(k + NSTAGE);
        }

        // Epilogue: undo the scalings, add the minima's part, publish this
        // warp's state in its (now idle) stages.
        __syncwarp();
        {
            float *eo = reinterpret_cast<float *>(wbuf);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l[nt][c] += __shfl_xor_sync(kFull, l[nt][c], d);
#pragma unroll
                        for (int i = 0; i < NG; ++i) om[nt][c][i] += __shfl_xor_sync(kFull, om[nt][c][i], d);
                    }
                    const int head = 8 * nt + 2 * t + c;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const int u = 16 * (mt / 4) + 8 * (mt / 2 % 2) + g;
                        const int i = G == 64 ? mt / 4 : mt / 2;
                        const float even = fmaf(o[mt][nt][c] * (SPLIT ? 0x1p-7f : 0x1p17f), S[i], om[nt][c][i]);
                        const float odd = fmaf(o[mt][nt][c + 2] * (SPLIT ? 0x1p-7f : 0x1p13f), S[i], om[nt][c][i]);
                        *reinterpret_cast<float2 *>(eo + head * LD + 4 * u + 2 * (mt & 1)) = make_float2(even, odd);
                    }
                    if (g == 0) {
                        eo[ROWS * LD + head] = ref[nt][c];
                        eo[ROWS * LD + ROWS + head] = l[nt][c];
                    }
                }
        }
        if (threadIdx.x == 0) s_next[nb] = dynamic ? ahead : item + gridDim.x;
        __syncthreads();
        merge_and_store<T, HD, kWarps, ROWS>(smem, WARP_BYTES, p, it.seq, it.part, it.qh0, it.rows, it.single);
        fence_proxy_async_smem();
        __syncthreads();
        item = s_next[nb];
        nb ^= 1;
        if (dynamic && threadIdx.x == 0) ahead = gridDim.x + next_handout(p.work_ctr);
    }
    griddep_launch_dependents();
    if (dynamic && threadIdx.x == 0) finish_handouts(p.work_ctr);

    // A wait gave up: let copies still in flight land before the CTA exits.
    if (failed && lane == 0) {
        for (uint32_t gi = n_done; gi < n_issued; ++gi)
            mbar_wait_bounded(bar_s + 8 * (gi % NSTAGE), (gi / NSTAGE) & 1u);
    }
}

using namespace host;

template <typename T, int HD, int G, int NT>
int launch_one(const DecodeParams &p, const void *k_cache, const void *v_cache, long long items, int dev,
               cudaStream_t st) {
    constexpr int NS = Q4Shape<HD, NT>::NSTAGE;
    constexpr int SMEM = kWarps * NS * (2 * kUnit * Q4Format<HD, G>::ROW_BYTES + 8);
    static KernelSlot slot;
    auto kernel = decode_q4_kernel<T, HD, G, NT>;
    const int occ = ensure_kernel(kernel, slot, SMEM, dev);
    if (occ == 0) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: cannot configure the kernel");
    const long long cap = static_cast<long long>(sm_count(dev)) * occ;
    const cudaError_t e = launch_dependent(kernel, static_cast<int>(items < cap ? items : cap), kWarps * 32, SMEM, st,
                                           static_cast<const uint8_t *>(k_cache),
                                           static_cast<const uint8_t *>(v_cache), p);
    return e == cudaSuccess ? PA_OK : pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
}

template <typename T, int HD, int G>
int launch_tile(const DecodeParams &p, const void *k, const void *v, long long items, int dev, cudaStream_t st) {
    return p.group > 8 ? launch_one<T, HD, G, 2>(p, k, v, items, dev, st)
                       : launch_one<T, HD, G, 1>(p, k, v, items, dev, st);
}

template <typename T>
int launch_any(const DecodeParams &p, const void *k, const void *v, int head_dim, int group_size, long long items,
               int dev, cudaStream_t st) {
    if (head_dim == 128)
        return group_size == 64 ? launch_tile<T, 128, 64>(p, k, v, items, dev, st)
                                : launch_tile<T, 128, 32>(p, k, v, items, dev, st);
    return group_size == 64 ? launch_tile<T, 64, 64>(p, k, v, items, dev, st)
                            : launch_tile<T, 64, 32>(p, k, v, items, dev, st);
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
    const int tile = p.group > 8 ? 16 : 8;   // query heads per work item, as launch_tile picks them
    p.tile_rows = p.group < tile ? p.group : tile;
    p.head_tiles = (p.group + tile - 1) / tile;

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
