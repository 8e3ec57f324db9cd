// The 4-bit cache's page layout and parameter pairs, shared by the kernels that
// write, read and attend over it (pa_cache_q4.cu, pa_decode_q4.cu).  include/pa.h
// states the format.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pa_internal.h"

namespace pa {

template <int HD, int G>
struct Q4Format {
    static constexpr int W = HD / 64;           // 32-bit words per lane octet member
    static constexpr int GROUPS = HD / G;       // parameter pairs per row
    static constexpr int CODE_BYTES = HD / 2;   // per row
    static constexpr int PARAM_BYTES = 4 * GROUPS;
    static constexpr int ROW_BYTES = CODE_BYTES + PARAM_BYTES;
};

// A parameter pair: step in the low bf16, minimum in the high one.  A bf16
// value is the upper half of the fp32 value with the same bits.
__device__ __forceinline__ float q4_step(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float q4_min(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

// D = A (16x16 fp16, row) * B (16x8 fp16, col) + C, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A B + C with C in registers of its own (or a constant).
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c));
}
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                               const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane (lane 4 r + c
// holds row r, columns 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

inline bool q4_sizes_ok(int head_dim, int block_size, int group_size) {
    return (head_dim == 64 || head_dim == 128) && (block_size == 16 || block_size == 32) &&
           (group_size == 32 || group_size == 64);
}

inline int q4_row_bytes(int head_dim, int group_size) { return head_dim / 2 + 4 * (head_dim / group_size); }

}  // namespace pa
