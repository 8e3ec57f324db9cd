// Cache write and read of the 4-bit cache for sm_103a (include/pa.h states the
// format and the quantisation).
//
// Both are one pass over the rows.  Eight lanes take the K and the V row of one
// (token, head); lane g of them owns code words g * W .. g * W + W - 1 (W = HD /
// 64), whose halves are the units of four values 16 w + g and 16 w + 8 + g.  So
// a lane loads 2 W pieces of four values, the eight lanes' pieces of one unit
// row are contiguous, and a group is what the eight lanes hold of one word (64)
// or one half-word (32): its minimum and maximum are three shuffles.  bf16
// values are compared packed, two groups' extremes to a register.
//
// The write has about as many instructions to issue as bytes to move, so each
// group's parameters (a division and a reciprocal) are worked out by one lane
// (lane i K's group i, lane 4 + i V's) and handed round, and a code costs three
// instructions: subtract and multiply two at a time, add 1.5 * 2^23 (which rounds
// half to even and leaves the code in the low mantissa bits), and a multiply-add
// that packs it.  Measured on 30011 tokens x 8 heads of 128 bf16 values in groups
// of 32 (161 MB either way, 24 us at the copy peak): write 32.2 us (82.6 with
// sixteen lanes a row, every lane at the parameters and 64-bit divisions; 37 with
// 256 threads per CTA; 33.6 without packed fp32), read 28.4 us (50.6; packed fp32 and
// two or four rows a lane change nothing).  32 tokens: 1.9 and 1.7 us, the launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pa_internal.h"
#include "pa_q4.cuh"

namespace pa {
namespace {

constexpr int kQ4Threads = 128;

// r / d for r < 2^31 by a product: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d),
// m d - 2^(31 + s) < 2^s, so r m / 2^(31 + s) is over r / d by less than 1 / d.
struct Divisor {
    uint32_t m;
    int shift;   // s - 1; -1 for d = 1
    explicit Divisor(uint32_t d) {
        int s = 0;
        while ((1u << s) < d) ++s;
        m = static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d);
        shift = s - 1;
    }
    __device__ __forceinline__ uint32_t of(uint32_t r) const { return shift < 0 ? r : __umulhi(r, m) >> shift; }
};

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

__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint32_t min_nan(uint32_t a, uint32_t b) {   // of two bf16
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The extremes of a lane's (then an octet's) two half-words of one word w:
// element 0 the unit 16 w + g, element 1 the unit 16 w + 8 + g.  NaN where one
// of the values is.
template <typename T>
struct Extremes;

template <>
struct Extremes<float> {
    float lo[2], hi[2];
    __device__ __forceinline__ void take(const float *p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[4];
            load4(p + 32 * h, x);
            lo[h] = min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3]));
            hi[h] = max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
        }
    }
    __device__ __forceinline__ void join_octet() {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                lo[h] = min_nan(lo[h], __shfl_xor_sync(kFull, lo[h], o));
                hi[h] = max_nan(hi[h], __shfl_xor_sync(kFull, hi[h], o));
            }
    }
    // Both half-words as one group.
    __device__ __forceinline__ void join_halves() {
        lo[0] = min_nan(lo[0], lo[1]);
        hi[0] = max_nan(hi[0], hi[1]);
    }
    __device__ __forceinline__ float low(bool h) const { return h ? lo[1] : lo[0]; }
    __device__ __forceinline__ float high(bool h) const { return h ? hi[1] : hi[0]; }
};

template <>
struct Extremes<__nv_bfloat16> {
    uint32_t lo, hi;   // half h of each: half-word h
    __device__ __forceinline__ void take(const __nv_bfloat16 *p) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p), b = *reinterpret_cast<const uint2 *>(p + 32);
        const uint32_t la = min_nan(a.x, a.y), lb = min_nan(b.x, b.y);
        const uint32_t ha = max_nan(a.x, a.y), hb = max_nan(b.x, b.y);
        // each register holds two partial extremes of one unit: one of each unit instead
        lo = min_nan(__byte_perm(la, lb, 0x5410), __byte_perm(la, lb, 0x7632));
        hi = max_nan(__byte_perm(ha, hb, 0x5410), __byte_perm(ha, hb, 0x7632));
    }
    __device__ __forceinline__ void join_octet() {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(kFull, hi, o));
        }
    }
    __device__ __forceinline__ void join_halves() {
        lo = min_nan(lo, __byte_perm(lo, 0u, 0x1032));
        hi = max_nan(hi, __byte_perm(hi, 0u, 0x1032));
    }
    __device__ __forceinline__ float low(bool h) const { return __uint_as_float(h ? lo & 0xffff0000u : lo << 16); }
    __device__ __forceinline__ float high(bool h) const { return __uint_as_float(h ? hi & 0xffff0000u : hi << 16); }
};

struct Group {
    float m, inv;
    uint32_t pair;
};

// The group's parameters.  Only this rounds in a direction: m down and s up,
// so that [m, m + 15 s] covers the group and no code needs a clamp.  A group
// that holds something not finite (or 2^126 and more) has pair kBad, and the
// caller masks its codes off.
constexpr uint32_t kBad = 0x7fc00000u;   // step 0, minimum NaN

__device__ __forceinline__ Group group_of(float low, float high) {
    Group g{0.f, 0.f, kBad};
    if (!(low > -0x1p126f && high < 0x1p126f)) return g;   // NaN compares false
    const uint32_t lo = __float_as_uint(__fadd_rn(low, 0.f));   // -0 becomes +0
    uint32_t m = lo & 0xffff0000u;
    if ((lo >> 31) && (lo & 0xffffu)) m += 0x10000u;   // negative: towards the larger magnitude
    g.m = __uint_as_float(m);
    const float far = __fsub_rn(high, g.m);
    float s = 0.f;
    if (far > 0.f) {
        s = __uint_as_float((__float_as_uint(__fdiv_rn(far, 15.f)) + 0xffffu) & 0xffff0000u);
        s = fmaxf(s, 0x1p-126f);
        g.inv = __frcp_rn(s);
    }
    g.pair = m | (__float_as_uint(s) >> 16);
    return g;
}

// Codes of four values in the low 16 bits.  Each sum's bits are 0x4b400000 plus
// the code; the constant's low 22 bits are zero and stay so when multiplied.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float m, float inv) {
    const float2 less = make_float2(-m, -m), by = make_float2(inv, inv);
    const float2 a = __fmul2_rn(__fadd2_rn(make_float2(x[0], x[1]), less), by);
    const float2 b = __fmul2_rn(__fadd2_rn(make_float2(x[2], x[3]), less), by);
    constexpr float up = 12582912.f;   // added one at a time: a packed sum would be contracted with the product
    uint32_t u = __float_as_uint(__fadd_rn(b.y, up));
    u = u * 16u + __float_as_uint(__fadd_rn(b.x, up));
    u = u * 16u + __float_as_uint(__fadd_rn(a.y, up));
    return u * 16u + __float_as_uint(__fadd_rn(a.x, up));
}

// Eight lanes take the K and the V row of one (token, head).
template <typename T, int HD, int G>
__global__ void __launch_bounds__(kQ4Threads, sizeof(T) == 2 ? 12 : 8)
    q4_write_kernel(const T *__restrict__ k, const T *__restrict__ v, uint8_t *__restrict__ k_cache,
                    uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slot_mapping, uint32_t rows,
                    uint32_t num_kv_heads, const Divisor by_heads, int bs_shift, long long num_slots, int32_t *status) {
    using F = Q4Format<HD, G>;
    constexpr int W = F::W, NG = F::GROUPS;
    const int lane = threadIdx.x & 31, g = lane & 7;
    const uint32_t r = blockIdx.x * (kQ4Threads / 8) + threadIdx.x / 8;
    const bool live = r < rows;
    const uint32_t t = by_heads.of(live ? r : 0u), h = r - t * num_kv_heads;
    const int64_t slot = live ? slot_mapping[t] : -1;
    const bool ok = slot >= 0 && slot < num_slots;
    if (slot >= num_slots && g == 0 && h == 0) flag_status(status, PA_STATUS_BAD_SLOT);

    const long long at = static_cast<long long>(live ? r : 0u) * HD + 4 * g;
    const T *src[2] = {k + at, v + at};
    Extremes<T> ends[2][W];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 0; w < W; ++w) ends[c][w].take(src[c] + 64 * w);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            ends[c][w].join_octet();
            if constexpr (G == 64) ends[c][w].join_halves();
        }
    // Lane i of the octet's first four (modulo the groups) works out K's group
    // i, the last four V's.
    const bool of_v = g & 4, second = W == 2 && (g & (NG / 2)), upper = G == 32 && (g & 1);
    const Extremes<T> ek = second ? ends[0][W - 1] : ends[0][0], ev = second ? ends[1][W - 1] : ends[1][0];
    const Extremes<T> e = of_v ? ev : ek;
    const Group mine = group_of(e.low(upper), e.high(upper));
    const unsigned bads = __ballot_sync(kFull, mine.pair == kBad) >> (lane & ~7);
    uint32_t word[2][W];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            word[c][w] = 0;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int from = 4 * c + (G == 64 ? w : 2 * w + hf);
                const float m = __shfl_sync(kFull, mine.m, (lane & ~7) + from);
                const float inv = __shfl_sync(kFull, mine.inv, (lane & ~7) + from);
                float x[4];
                load4(src[c] + 64 * w + 32 * hf, x);   // again: in a register or the L1
                const uint32_t codes = encode4(x, m, inv) & ((bads >> from) & 1u ? 0u : 0xffffu);
                word[c][w] |= codes << (16 * hf);
            }
        }
    if (!ok) return;
    const int bs = 1 << bs_shift;
    const int row = static_cast<int>(slot & (bs - 1));
    const long long page = ((slot >> bs_shift) * num_kv_heads + h) * (static_cast<long long>(F::ROW_BYTES) << bs_shift);
    const long long code_at = page + row * F::CODE_BYTES + 4 * W * g;
    if constexpr (W == 2) {
        *reinterpret_cast<uint2 *>(k_cache + code_at) = make_uint2(word[0][0], word[0][W - 1]);
        *reinterpret_cast<uint2 *>(v_cache + code_at) = make_uint2(word[1][0], word[1][W - 1]);
    } else {
        *reinterpret_cast<uint32_t *>(k_cache + code_at) = word[0][0];
        *reinterpret_cast<uint32_t *>(v_cache + code_at) = word[1][0];
    }
    if ((g & 3) < NG)
        *reinterpret_cast<uint32_t *>((of_v ? v_cache : k_cache) + page + bs * F::CODE_BYTES + row * F::PARAM_BYTES +
                                      4 * (g & 3)) = mine.pair;
}

template <typename T, int HD, int G>
__global__ void __launch_bounds__(kQ4Threads)
    q4_gather_kernel(T *__restrict__ k, T *__restrict__ v, const uint8_t *__restrict__ k_cache,
                     const uint8_t *__restrict__ v_cache, const int64_t *__restrict__ slot_mapping, uint32_t rows,
                     uint32_t num_kv_heads, const Divisor by_heads, int bs_shift, long long num_slots, int32_t *status) {
    using F = Q4Format<HD, G>;
    constexpr int W = F::W, NG = F::GROUPS;
    const int g = threadIdx.x & 7;
    const uint32_t r = blockIdx.x * (kQ4Threads / 8) + threadIdx.x / 8;
    if (r >= rows) return;
    const uint32_t t = by_heads.of(r), h = r - t * num_kv_heads;
    const int64_t slot = slot_mapping[t];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (g == 0 && h == 0) flag_status(status, PA_STATUS_BAD_SLOT);
        return;
    }
    const int bs = 1 << bs_shift;
    const int row = static_cast<int>(slot & (bs - 1));
    const long long page = ((slot >> bs_shift) * num_kv_heads + h) * (static_cast<long long>(F::ROW_BYTES) << bs_shift);
    const long long code_at = page + row * F::CODE_BYTES + 4 * W * g, par_at = page + bs * F::CODE_BYTES + row * F::PARAM_BYTES;
    uint32_t word[2][W], pair[2][NG];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint8_t *cache = c ? v_cache : k_cache;
        if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(cache + code_at);
            word[c][0] = x.x;
            word[c][W - 1] = x.y;
        } else {
            word[c][0] = *reinterpret_cast<const uint32_t *>(cache + code_at);
        }
        if constexpr (NG == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(cache + par_at);
            pair[c][0] = x.x, pair[c][1] = x.y, pair[c][NG - 2] = x.z, pair[c][NG - 1] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < NG; ++i) pair[c][i] = reinterpret_cast<const uint32_t *>(cache + par_at)[i];
        }
    }
    const long long at = static_cast<long long>(r) * HD + 4 * g;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t p = pair[c][G == 64 ? w : 2 * w + hf], u = word[c][w];
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // 2^23 + code; step * code is exact in fp32 (8 by 4 bits), so the sum rounds once
                    const float code = __uint_as_float(((u >> (16 * hf + 4 * j)) & 15u) | 0x4b000000u) - 8388608.f;
                    x[j] = fmaf(code, q4_step(p), q4_min(p));
                }
                put4((c ? v : k) + at + 64 * w + 32 * hf, x);
            }
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
    // rows are counted in 31 bits
    if (static_cast<long long>(num_tokens) * num_kv_heads >= (1ll << 31))
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
    dim3 grid() const {
        constexpr int per = kQ4Threads / 8;
        return dim3(static_cast<unsigned>((rows + per - 1) / per));
    }
};

struct WriteLaunch : Call {
    template <typename T, int HD, int G>
    void run() const {
        q4_write_kernel<T, HD, G><<<grid(), kQ4Threads, 0, stream>>>(
            static_cast<const T *>(k), static_cast<const T *>(v), static_cast<uint8_t *>(k_cache),
            static_cast<uint8_t *>(v_cache), slot_mapping, static_cast<uint32_t>(rows),
            static_cast<uint32_t>(num_kv_heads), Divisor(num_kv_heads), bs_shift, num_slots, status);
    }
};

struct GatherLaunch : Call {
    template <typename T, int HD, int G>
    void run() const {
        q4_gather_kernel<T, HD, G><<<grid(), kQ4Threads, 0, stream>>>(
            static_cast<T *>(k), static_cast<T *>(v), static_cast<const uint8_t *>(k_cache),
            static_cast<const uint8_t *>(v_cache), slot_mapping, static_cast<uint32_t>(rows),
            static_cast<uint32_t>(num_kv_heads), Divisor(num_kv_heads), bs_shift, num_slots, status);
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
