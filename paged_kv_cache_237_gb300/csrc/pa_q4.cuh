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

inline bool q4_sizes_ok(int head_dim, int block_size, int group_size) {
    return (head_dim == 64 || head_dim == 128) && (block_size == 16 || block_size == 32) &&
           (group_size == 32 || group_size == 64);
}

inline int q4_row_bytes(int head_dim, int group_size) { return head_dim / 2 + 4 * (head_dim / group_size); }

}  // namespace pa
