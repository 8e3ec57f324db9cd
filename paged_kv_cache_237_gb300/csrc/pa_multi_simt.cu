// pa_decode_tree and pa_decode_cross on plain fp32 FMAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_multi.cuh"

namespace pa {
namespace {

constexpr int kRows = 32, kTile = 16, kThreads = 128, kTok = kTile / 8;
using Axis = MultiAxis<kRows, kRows, kTile, 2>;

__device__ __forceinline__ float4 load4(const float *x) { return *reinterpret_cast<const float4 *>(x); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *x) {
    const uint2 u = *reinterpret_cast<const uint2 *>(x);
    __nv_bfloat162 a, b;
    memcpy(&a, &u.x, 4);
    memcpy(&b, &u.y, 4);
    const float2 lo = __bfloat1622float2(a), hi = __bfloat1622float2(b);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}

__device__ __forceinline__ bool finite4(float4 v) {
    return isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) multi_simt_kernel(const MultiParams p) {
    constexpr int LD = HD + 4, C = HD / 32;   // C: groups of four columns a thread holds
    __shared__ float s_q[kRows][LD], s_k[kTile][LD], s_v[kTile][HD], s_p[kRows][kTile + 1];
    __shared__ MultiSpot s_spot;
    __shared__ int s_dirty;
    griddep_wait();
    const int tid = threadIdx.x, ty = tid >> 3, tx = tid & 7;   // rows 2 ty, 2 ty + 1; tokens tx + 8 j
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

    MultiItem it;
    while (Axis::next(p, spot, left, it)) {
        const int R0 = it.m * kRows, rows = min(kRows, it.s.c * p.group - R0);
        __syncthreads();
        for (int i = tid; i < kRows * (HD / 4); i += kThreads) {
            const int r = i / (HD / 4), c = i % (HD / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) x = load4(static_cast<const T *>(p.q) + multi_row(p, it.s, it.kvh, R0 + r, HD) + c);
            store4(&s_q[r][c], make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2,
                                           x.w * p.scale_log2));
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float4 o[2][C];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int c = 0; c < C; ++c) o[a][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int seen = Axis::seen(p, it.s, it.m);
        for (int t = it.tile0; t < it.tile1; ++t) {
            const int u0 = t * kTile;
            __syncthreads();
            if (tid == 0) s_dirty = 0;
            __syncthreads();
            for (int i = tid; i < kTile * (HD / 4); i += kThreads) {
                const int j = i / (HD / 4), c = i % (HD / 4) * 4, u = u0 + j;
                float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
                if (u < seen) {
                    const int b = p.block_tables[static_cast<long long>(it.seq) * p.width + u / p.block_size];
                    if (b < 0 || b >= p.num_blocks) {
                        flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                    } else {
                        const long long row =
                            (static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size + u % p.block_size;
                        k = load4(static_cast<const T *>(p.k_cache) + row * HD + c);
                        v = load4(static_cast<const T *>(p.v_cache) + row * HD + c);
                        if (!finite4(v)) s_dirty = 1;
                    }
                }
                store4(&s_k[j][c], k);
                store4(&s_v[j][c], v);
            }
            __syncthreads();
            float sc[2][kTok] = {};
            for (int d = 0; d < HD; d += 4) {
                const float4 q0 = load4(&s_q[2 * ty][d]), q1 = load4(&s_q[2 * ty + 1][d]);
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    const float4 k = load4(&s_k[tx + 8 * j][d]);
                    sc[0][j] += q0.x * k.x + q0.y * k.y + q0.z * k.z + q0.w * k.w;
                    sc[1][j] += q1.x * k.x + q1.y * k.y + q1.z * k.z + q1.w * k.w;
                }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int R = R0 + 2 * ty + a, tok = R / p.group;
                bool see[kTok];
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    const int u = u0 + tx + 8 * j;
                    see[j] = 2 * ty + a < rows && u < it.s.n && multi_sees(p, it.s, tok, u);
                    if (!see[j]) sc[a][j] = -INFINITY;
                    top = fmaxf(top, sc[a][j]);
                }
#pragma unroll
                for (int w = 1; w < 8; w <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, w));
                const float now = fmaxf(m[a], top), ref = now == -INFINITY ? 0.f : now;
                const float keep = exp2f(m[a] - ref);
                m[a] = now;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    const float e = exp2f(sc[a][j] - ref);
                    sum += e;
                    // -1 marks what the row does not see, for values that are not finite
                    s_p[2 * ty + a][tx + 8 * j] = see[j] || !s_dirty ? e : -1.f;
                }
#pragma unroll
                for (int w = 1; w < 8; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
                l[a] = l[a] * keep + sum;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    o[a][c].x *= keep;
                    o[a][c].y *= keep;
                    o[a][c].z *= keep;
                    o[a][c].w *= keep;
                }
            }
            __syncwarp();
            for (int j = 0; j < kTile; ++j) {
                float w[2];
#pragma unroll
                for (int a = 0; a < 2; ++a) w[a] = s_p[2 * ty + a][j];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    if (w[a] < 0.f) continue;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float4 v = load4(&s_v[j][tx * 4 + 32 * c]);
                        o[a][c].x += w[a] * v.x;
                        o[a][c].y += w[a] * v.y;
                        o[a][c].z += w[a] * v.z;
                        o[a][c].w += w[a] * v.w;
                    }
                }
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int r = 2 * ty + a;
            if (r >= rows) continue;
            if (it.whole()) {
                const float inv = l[a] == 0.f ? 0.f : 1.f / l[a];
                T *out = static_cast<T *>(p.out) + multi_row(p, it.s, it.kvh, R0 + r, HD);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    store4(out + tx * 4 + 32 * c, make_float4(o[a][c].x * inv, o[a][c].y * inv, o[a][c].z * inv,
                                                              o[a][c].w * inv));
            } else {
                const long long at = static_cast<long long>(it.slot(blockIdx.x)) * p.slot_rows + r;
#pragma unroll
                for (int c = 0; c < C; ++c) store4(p.part_acc + at * HD + tx * 4 + 32 * c, o[a][c]);
                if (tx == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(m[a], l[a]);
            }
        }
    }
}

}  // namespace

template <typename T, int HD>
int multi_simt(const MultiParams &p, int dev, cudaStream_t st) {
    const int grid = min(host::sm_count(dev) * 4, kMultiSimtCtas);
    const cudaError_t e = host::launch_dependent(multi_simt_kernel<T, HD>, grid, kThreads, 0, st, p);
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return launch_join<T, HD, Axis>(p, grid, st);
}

int launch_multi_simt(const MultiParams &p, int head_dim, int dev, cudaStream_t st) {
    return head_dim == 128 ? multi_simt<float, 128>(p, dev, st) : multi_simt<float, 64>(p, dev, st);
}

}  // namespace pa
