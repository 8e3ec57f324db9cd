// Cache write and read of the 4-bit cache for sm_103a (include/pa.h states the
// format and the quantisation).
//
// Both are one pass over the rows.  HD / 8 lanes share a head row; lane (w, g)
// of them owns 32-bit code word g * W + w, whose halves are the units of four
// values 16 w + g and 16 w + 8 + g.  So a lane loads two 8-byte (bf16) or
// 16-byte (fp32) pieces, a row's eight lanes of one w cover 64 consecutive
// bytes per load, and the group minimum and maximum are three shuffles over
// those eight lanes (the eight lanes of one w hold one group of 64 or two of
// 32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {
namespace {

constexpr int kQ4Threads = 256;

__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void put4(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void put4(__nv_bfloat16 *p, const float (&x)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    uint2 u;
    memcpy(&u.x, &lo, 4);
    memcpy(&u.y, &hi, 4);
    *reinterpret_cast<uint2 *>(p) = u;
}

struct Range {
    float lo, hi;
    bool bad;
};

// Minimum, maximum and "holds something not finite" over the eight lanes of one w.
__device__ __forceinline__ Range octet_range(Range r, int lane) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        r.lo = fminf(r.lo, __shfl_xor_sync(kFull, r.lo, o));
        r.hi = fmaxf(r.hi, __shfl_xor_sync(kFull, r.hi, o));
    }
    r.bad = ((__ballot_sync(kFull, r.bad) >> (lane & ~7)) & 0xffu) != 0u;
    return r;
}

__device__ __forceinline__ Range range_of(const float (&x)[4]) {
    Range r;
    r.lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
    r.hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    const float big = 0x1p126f;   // comparisons with NaN are false, so NaN is bad too
    r.bad = !(fabsf(x[0]) < big && fabsf(x[1]) < big && fabsf(x[2]) < big && fabsf(x[3]) < big);
    return r;
}

struct Group {
    float m, inv;
    uint32_t pair;
};

// The group's parameters.  Only this rounds in a direction: m down and s up,
// so that [m, m + 15 s] covers the group and no code needs a clamp.
__device__ __forceinline__ Group group_of(const Range &r) {
    Group g{0.f, 0.f, 0x7fc00000u};   // step 0, minimum NaN
    if (r.bad) return g;
    const uint32_t lo = __float_as_uint(r.lo);
    uint32_t m = lo & 0xffff0000u;
    if ((lo >> 31) && (lo & 0xffffu)) m += 0x10000u;   // negative: towards the larger magnitude
    g.m = __uint_as_float(m);
    const float far = __fsub_rn(r.hi, g.m);
    float s = 0.f;
    if (far > 0.f) {
        s = __uint_as_float((__float_as_uint(__fdiv_rn(far, 15.f)) + 0xffffu) & 0xffff0000u);
        s = fmaxf(s, 0x1p-126f);
        g.inv = __frcp_rn(s);
    }
    g.pair = m | (__float_as_uint(s) >> 16);
    return g;
}

// Codes of four values in the low 16 bits.  Adding 1.5 * 2^23 rounds to an
// integer, half to even, and leaves it in the low mantissa bits.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], const Group &g) {
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float t = __fadd_rn(__fmul_rn(__fsub_rn(x[j], g.m), g.inv), 12582912.f);
        u |= (__float_as_uint(t) & 15u) << (4 * j);
    }
    return u;
}

// grid (row tiles, 2): blockIdx.y selects K or V.
template <typename T, int HD, int G>
__global__ void __launch_bounds__(kQ4Threads)
    q4_write_kernel(const T *__restrict__ k, const T *__restrict__ v, uint8_t *__restrict__ k_cache,
                    uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slot_mapping, long long rows,
                    int num_kv_heads, int bs_shift, long long num_slots, int32_t *status) {
    using F = Q4Format<HD, G>;
    constexpr int LPR = HD / 8;
    const int lane = threadIdx.x & 31, li = threadIdx.x % LPR, w = li >> 3, g = li & 7;
    const long long r = (long long)blockIdx.x * (kQ4Threads / LPR) + threadIdx.x / LPR;
    const bool live = r < rows;
    const int64_t slot = live ? slot_mapping[r / num_kv_heads] : -1;
    const int h = static_cast<int>(r % num_kv_heads);
    const bool ok = slot >= 0 && slot < num_slots;
    if (slot >= num_slots && li == 0 && h == 0 && blockIdx.y == 0) flag_status(status, PA_STATUS_BAD_SLOT);

    const T *src = (blockIdx.y ? v : k) + (live ? r : 0) * HD + 64 * w + 4 * g;
    float a[4], b[4];
    load4(src, a);
    load4(src + 32, b);
    Range ra = range_of(a), rb = range_of(b);
    if (G == 64) {
        ra.lo = fminf(ra.lo, rb.lo);
        ra.hi = fmaxf(ra.hi, rb.hi);
        ra.bad |= rb.bad;
    }
    const Group ga = group_of(octet_range(ra, lane));
    const Group gb = G == 64 ? ga : group_of(octet_range(rb, lane));
    const bool bad_a = (ga.pair & 0xffff0000u) == 0x7fc00000u, bad_b = (gb.pair & 0xffff0000u) == 0x7fc00000u;
    const uint32_t word = (bad_a ? 0u : encode4(a, ga)) | (bad_b ? 0u : encode4(b, gb) << 16);
    if (!ok) return;
    const int bs = 1 << bs_shift;
    const int row = static_cast<int>(slot & (bs - 1));
    uint8_t *page = (blockIdx.y ? v_cache : k_cache) +
                    ((slot >> bs_shift) * num_kv_heads + h) * ((long long)F::ROW_BYTES << bs_shift);
    *reinterpret_cast<uint32_t *>(page + row * F::CODE_BYTES + (g * F::W + w) * 4) = word;
    uint32_t *par = reinterpret_cast<uint32_t *>(page + bs * F::CODE_BYTES + row * F::PARAM_BYTES);
    if (g == 0) {
        if (G == 64)
            par[w] = ga.pair;
        else
            *reinterpret_cast<uint2 *>(par + 2 * w) = make_uint2(ga.pair, gb.pair);
    }
}

template <typename T, int HD, int G>
__global__ void __launch_bounds__(kQ4Threads)
    q4_gather_kernel(T *__restrict__ k, T *__restrict__ v, const uint8_t *__restrict__ k_cache,
                     const uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slot_mapping, long long rows,
                     int num_kv_heads, int bs_shift, long long num_slots, int32_t *status) {
    using F = Q4Format<HD, G>;
    constexpr int LPR = HD / 8;
    const int li = threadIdx.x % LPR, w = li >> 3, g = li & 7;
    const long long r = (long long)blockIdx.x * (kQ4Threads / LPR) + threadIdx.x / LPR;
    if (r >= rows) return;
    const int64_t slot = slot_mapping[r / num_kv_heads];
    if (slot < 0) return;
    const int h = static_cast<int>(r % num_kv_heads);
    if (slot >= num_slots) {
        if (li == 0 && h == 0 && blockIdx.y == 0) flag_status(status, PA_STATUS_BAD_SLOT);
        return;
    }
    const int bs = 1 << bs_shift;
    const int row = static_cast<int>(slot & (bs - 1));
    const uint8_t *page = (blockIdx.y ? v_cache : k_cache) +
                          ((slot >> bs_shift) * num_kv_heads + h) * ((long long)F::ROW_BYTES << bs_shift);
    const uint32_t word = *reinterpret_cast<const uint32_t *>(page + row * F::CODE_BYTES + (g * F::W + w) * 4);
    const uint32_t *par = reinterpret_cast<const uint32_t *>(page + bs * F::CODE_BYTES + row * F::PARAM_BYTES);
    const uint32_t pa = G == 64 ? par[w] : par[2 * w], pb = G == 64 ? pa : par[2 * w + 1];
    float a[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // step * code is exact in fp32 (8 by 4 bits), so this rounds once
        a[j] = fmaf(static_cast<float>((word >> (4 * j)) & 15u), q4_step(pa), q4_min(pa));
        b[j] = fmaf(static_cast<float>((word >> (16 + 4 * j)) & 15u), q4_step(pb), q4_min(pb));
    }
    T *dst = (blockIdx.y ? v : k) + r * HD + 64 * w + 4 * g;
    put4(dst, a);
    put4(dst + 32, b);
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks shared by the two calls; PA_OK with *rows = 0 when there is nothing to do.
int check(const char *const (&msg)[5], const void *k, const void *v, const void *k_cache, const void *v_cache,
          const int64_t *slot_mapping, int num_tokens, int num_kv_heads, int head_dim, int block_size, int group_size,
          int num_blocks, int dtype, long long *rows) {
    *rows = 0;
    if (dtype != PA_F32 && dtype != PA_BF16) return pa_fail(PA_ERR_INVALID_ARG, msg[0]);
    if (num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0) return pa_fail(PA_ERR_INVALID_ARG, msg[1]);
    if (!q4_sizes_ok(head_dim, block_size, group_size)) return pa_fail(PA_ERR_UNSUPPORTED, msg[2]);
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !k_cache || !v_cache || !slot_mapping) return pa_fail(PA_ERR_INVALID_ARG, msg[3]);
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return pa_fail(PA_ERR_INVALID_ARG, msg[4]);
    // the grid counts tiles of at least 16 rows in 31 bits
    if (static_cast<long long>(num_tokens) * num_kv_heads > (1ll << 34))
        return pa_fail(PA_ERR_UNSUPPORTED, msg[1]);
    *rows = static_cast<long long>(num_tokens) * num_kv_heads;
    return PA_OK;
}

#define PA_Q4_MESSAGES(name)                                                                        \
    {name ": bad dtype", name ": bad sizes",                                                        \
     name ": head_dim must be 64 or 128, block_size 16 or 32, group_size 32 or 64", name ": null pointer", \
     name ": misaligned pointer"}

template <typename Launch>
int dispatch(int dtype, int head_dim, int group_size, Launch &&launch) {
    const bool wide = head_dim == 128, big = group_size == 64;
    if (dtype == PA_F32) {
        if (wide) big ? launch.template run<float, 128, 64>() : launch.template run<float, 128, 32>();
        else big ? launch.template run<float, 64, 64>() : launch.template run<float, 64, 32>();
    } else {
        if (wide) big ? launch.template run<__nv_bfloat16, 128, 64>() : launch.template run<__nv_bfloat16, 128, 32>();
        else big ? launch.template run<__nv_bfloat16, 64, 64>() : launch.template run<__nv_bfloat16, 64, 32>();
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PA_OK : pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
}

struct Call {
    void *k, *v, *k_cache, *v_cache;
    const int64_t *slot_mapping;
    long long rows, num_slots;
    int num_kv_heads, bs_shift;
    int32_t *status;
    cudaStream_t stream;
    template <int HD>
    dim3 grid() const {
        constexpr int per = kQ4Threads / (HD / 8);
        return dim3(static_cast<unsigned>((rows + per - 1) / per), 2);
    }
};

struct WriteLaunch : Call {
    template <typename T, int HD, int G>
    void run() const {
        q4_write_kernel<T, HD, G><<<grid<HD>(), kQ4Threads, 0, stream>>>(
            static_cast<const T *>(k), static_cast<const T *>(v), static_cast<uint8_t *>(k_cache),
            static_cast<uint8_t *>(v_cache), slot_mapping, rows, num_kv_heads, bs_shift, num_slots, status);
    }
};

struct GatherLaunch : Call {
    template <typename T, int HD, int G>
    void run() const {
        q4_gather_kernel<T, HD, G><<<grid<HD>(), kQ4Threads, 0, stream>>>(
            static_cast<T *>(k), static_cast<T *>(v), static_cast<const uint8_t *>(k_cache),
            static_cast<const uint8_t *>(v_cache), slot_mapping, rows, num_kv_heads, bs_shift, num_slots, status);
    }
};

}  // namespace
}  // namespace pa

extern "C" size_t pa_q4_page_bytes(int head_dim, int block_size, int group_size) {
    if (!pa::q4_sizes_ok(head_dim, block_size, group_size)) return 0;
    return static_cast<size_t>(block_size) * pa::q4_row_bytes(head_dim, group_size);
}

extern "C" int pa_reshape_and_cache_q4(const void *k, const void *v, void *k_cache, void *v_cache,
                                       const int64_t *slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
                                       int block_size, int group_size, int num_blocks, int dtype,
                                       int32_t *dev_status, void *stream) {
    PaTraceRange trace("pa_reshape_and_cache_q4");
    static const char *const msg[5] = PA_Q4_MESSAGES("pa_reshape_and_cache_q4");
    long long rows = 0;
    const int rc = pa::check(msg, k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim, block_size,
                             group_size, num_blocks, dtype, &rows);
    if (rc != PA_OK || rows == 0) return rc;
    pa::WriteLaunch l;
    static_cast<pa::Call &>(l) = {const_cast<void *>(k), const_cast<void *>(v), k_cache, v_cache, slot_mapping, rows,
                                  static_cast<long long>(num_blocks) * block_size, num_kv_heads,
                                  block_size == 32 ? 5 : 4, dev_status, static_cast<cudaStream_t>(stream)};
    return pa::dispatch(dtype, head_dim, group_size, l);
}

extern "C" int pa_gather_q4(void *k, void *v, const void *k_cache, const void *v_cache, const int64_t *slot_mapping,
                            int num_tokens, int num_kv_heads, int head_dim, int block_size, int group_size,
                            int num_blocks, int dtype, int32_t *dev_status, void *stream) {
    PaTraceRange trace("pa_gather_q4");
    static const char *const msg[5] = PA_Q4_MESSAGES("pa_gather_q4");
    long long rows = 0;
    const int rc = pa::check(msg, k, v, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim, block_size,
                             group_size, num_blocks, dtype, &rows);
    if (rc != PA_OK || rows == 0) return rc;
    pa::GatherLaunch l;
    static_cast<pa::Call &>(l) = {k, v, const_cast<void *>(k_cache), const_cast<void *>(v_cache), slot_mapping, rows,
                                  static_cast<long long>(num_blocks) * block_size, num_kv_heads,
                                  block_size == 32 ? 5 : 4, dev_status, static_cast<cudaStream_t>(stream)};
    return pa::dispatch(dtype, head_dim, group_size, l);
}
