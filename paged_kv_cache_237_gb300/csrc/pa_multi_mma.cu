// pa_decode_tree and pa_decode_cross over bf16 caches, on tcgen05.
//
// An item is up to 256 rows (query tokens x the heads of one KV head) against a
// stretch of the sequence's cache in tiles of 128 tokens.  One CTA per SM runs
// two streams, each with its own 128 rows of scores S, its own sums O (both in
// tensor memory), running maximum and sum:
//   more than 128 rows: stream s has rows 128 s.. and both use every tile;
//   at most 128 rows: both have the same rows, stream s takes every second tile,
//   and the two are joined at the end of the item.
// So while one stream's softmax runs, the tensor core works for the other, and a
// decode step's few rows keep as many copies in flight as a prompt's many.
//
// Roles (warps): 0-3 and 4-7 the streams' softmax, a thread per row; 8 the
// copies; 9 the matrix instructions; 10 and 11 nothing (registers move between
// whole groups of four warps: 12 x 168 at launch, 8 x 224 + 4 x 56 then).
//   S = Q K^T      128 x 128 x head_dim, Q and K in shared memory (128-byte swizzle)
//   O += P V       128 x head_dim x 128, P in tensor memory over S, V in shared
//                  memory as it is cached (tokens x head_dim, the MN-major form)
//
// p enters as the sum of two bf16 parts (about 16 significant bits), as in pa_decode and
// in the pass for few rows: a sequence's result is as exact whatever shares its batch.
// One part alone would take a third of the matrix work away (32 contexts with trees 382
// us, 8 x 2000 queries 4.9 ms) and leave a row off by up to 2^-8 where
// its weights are alike, as much as the rounding of its result to bf16.
// Row maxima are references that only move when a tile's maximum is more than 2^8
// above: then the row's O and sum are rescaled (p stays below 2^8, and fp32 sums lose
// nothing by it).  O starts from zero every 64 steps, and its sums so far are kept in the
// workspace (kRun).
//
// What bounds it: the chain from a stream's scores to its weights: tensor memory read,
// maximum, exponentials and their parts, tensor memory written, three barrier operations;
// for long prompts, whose steps come one after the other, the tensor core nearly as much
// (70 % of a step's cycles, head_dim 128).  Short contexts pay
// each item's beginning and end besides (Q, results, 5 or 6 steps' time).  Measured: 8 x 2000
// queries of 64 / 8 heads of 128 over 4,000..16,384 tokens 6.2 to 7.1 ms, 0.91 to 1.04 PFLOP/s; 7
// contexts of up to 131,072 with 25 drafted tokens each 680 to 785 us, 3.6 to 4.2 TB/s; 32 lognormal
// contexts with trees of 16..64 nodes 443 to 465 us; prompts of 1..448 queries over 1..1500
// tokens, 20 heads of 64: 193 to 200 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_multi.cuh"

namespace pa {
namespace {

constexpr int kTile = 128;                 // tokens per tile, and rows per stream
constexpr int kMmaThreads = 384;

// Steps of a stream whose products meet in tensor memory.  The tensor core cuts a sum off where an addition rounds, 16 tokens
// and a part of the weights at a time: 2^-25 of it on average, 2^-15 in 64 steps and always towards zero.  So the sums of a
// run join those of the runs before it in the CTA's part of the workspace, by fp32 additions.  Measured, without runs / of
// 64 / of 32 steps: 32 lognormal contexts with trees 429 / 443 / 457 us, 7 contexts of up to 131,072 tokens 662 / 679 / 690 (results
// 1.7 / 0.4 / 0.2 hundredths of a bf16 step towards zero on average), 8 x 2000 queries 5930 / 6210 / 6440.
constexpr int kRun = 64;

// A tile for both streams takes twice as long as one for one of them where the
// softmax bounds both (head_dim 64), and no longer where the copies bound the second
// (128).  Measured, with the other weights in brackets, us: heads of 64, prompts of 1..448
// queries over inputs of 1..1500 204 (equal weights 235), of 100..448 over 200..1500 120 (128),
// 200 of 60..160 over 1..200 166 (189), trees with groups of 4 152 (155); heads of 128,
// trees of 16..64 nodes with groups of 8 429 (weights of two and one 524), of 4 194 (219), but
// prompts of 1..448 queries with a head each 308 (282).  A beginning and end take as long as
// 6 or 5 units (head_dim 64, 10 units: 212, 124, 179; 3: 241, 136, 167; head_dim 128, 11: 452
// and 198; 3: 458 and 206).
template <int HD>
using AxisOf = MultiAxis<kMultiMmaRows, HD == 64 ? kTile : kMultiMmaRows, kTile, HD == 64 ? 6 : 5>;

// ---------------------------------------------------------------- tcgen05 ---
__device__ __forceinline__ void tm_alloc(uint32_t dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_dealloc(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's lane.  The values are there after tm_wait_ld().
__device__ __forceinline__ void tm_ld32(uint32_t addr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(u[0]),
        "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]),
        "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tm_ld16(uint32_t addr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tm_ld2(uint32_t addr, float *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=f"(r[0]), "=f"(r[1]) : "r"(addr));
}
__device__ __forceinline__ void tm_st2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%2], {%0, %1};" ::"r"(a), "r"(b), "r"(addr) : "memory");
}

// One lane of the warp, always the same: its mask as the operand `lead` below.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes;
}

// Matrix instructions, executed by the whole warp and issued by its leading lane: a branch around them would take
// their operands out of the uniform registers that the instruction reads, and moving them back there takes longer
// than the instruction.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(lead)
        : "memory");
}
// Arrives at `bar` once every matrix instruction issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %1, 0;\n\t"
        "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
}
// Shared-memory operand in 128-byte swizzled rows; 8-row groups follow each other.
// K-major (Q, K): the row is along head_dim.  MN-major (V): the row is along
// head_dim too, but that is N, so the next 64 columns are `next` bytes away.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t next) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>((next >> 4) & 0x3fffu) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32, 128 rows, n columns.
constexpr __host__ __device__ uint32_t mma_idesc(int n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
           (static_cast<uint32_t>(128 / 16) << 24);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 32 sums join those that a row keeps in memory (times f), if there are any yet.
__device__ __forceinline__ void keep_sums(float4 *kept, int stride, const float *o, float f, bool any) {
    float4 y[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] = any ? __ldcg(kept + c * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        __stcg(kept + c * stride, make_float4(fmaf(y[c].x, f, o[4 * c]), fmaf(y[c].y, f, o[4 * c + 1]),
                                              fmaf(y[c].z, f, o[4 * c + 2]), fmaf(y[c].w, f, o[4 * c + 3])));
}

// Shared memory: Q (two tiles), rings of K and V tiles, then the small things.
template <int HD>
struct Smem {
    static constexpr int TILE = kTile * HD * 2, SLAB = kTile * 128;   // a slab: 64 columns of a tile
    static constexpr int NK = HD == 128 ? 3 : 6, NV = HD == 128 ? 2 : 6;
    static constexpr int K = 2 * TILE, V = K + NK * TILE, END = V + NV * TILE;
    static constexpr int BYTES = END + 1024;   // and room to align
};

struct Control {
    uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6], s_full[2], p_full[2][2], o_full[2], q_full, e_full;
    struct {
        MultiSpot spot;
        long long left;
    } walk[8];                 // of the softmax warps, out of their registers
    int dirty[2];          // number of the item whose drafted tokens have values that are not finite, by its parity
    int failed;
    uint32_t tmem;
    MultiSpot spot;
};

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    template <int N>
    __device__ __forceinline__ void advance() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Waits give up after about two seconds, or when another role has; every role
// then leaves its loop.
__device__ __forceinline__ bool await_slow(Control &c, uint32_t bar, uint32_t parity) {
    const uint64_t start = global_timer_ns();
#pragma unroll 1
    for (uint32_t spin = 1;; ++spin) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((spin & 63u) == 0) {
            if (*static_cast<volatile int *>(&c.failed)) return false;
            if (global_timer_ns() - start > kWaitLimitNs) {
                *static_cast<volatile int *>(&c.failed) = 1;
                return false;
            }
        }
    }
}

// For a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool await_warp(Control &c, uint64_t *bar, uint32_t parity) {
    const uint32_t b = smem_addr(bar);
    if (__all_sync(kFull, mbar_try_wait(b, parity))) return true;
    return __all_sync(kFull, await_slow(c, b, parity));
}

// For a warp and two barriers, the second only if it is needed.  A wait costs about
// 100 cycles even when there is nothing to wait for.  (All lanes look at the same.)
__device__ __forceinline__ bool await_two(Control &c, uint64_t *first, uint32_t parity_a, uint64_t *second,
                                          uint32_t parity_b, bool need_b) {
    const uint32_t a = smem_addr(first), b = smem_addr(second);
    const bool there_a = mbar_try_wait(a, parity_a);
    const bool there_b = !need_b || mbar_try_wait(b, parity_b);
    if (__all_sync(kFull, there_a && there_b)) return true;
    const bool ok = await_slow(c, a, parity_a) && (!need_b || await_slow(c, b, parity_b));
    return __all_sync(kFull, ok);
}

template <int HD>
__global__ void __launch_bounds__(kMmaThreads, 1)
    multi_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const MultiParams p) {
    using M = Smem<HD>;
    using Axis = AxisOf<HD>;
    constexpr uint32_t kIdescS = mma_idesc(kTile, false), kIdescO = mma_idesc(HD, true);
    extern __shared__ uint8_t smem_raw[];
    __shared__ Control ctl;
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *smem_p = smem_raw + (smem - smem_addr(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(smem_addr(&ctl.k_full[i]), 1);
            mbar_init(smem_addr(&ctl.k_empty[i]), 1);
            mbar_init(smem_addr(&ctl.v_full[i]), 1);
            mbar_init(smem_addr(&ctl.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.p_full[i][0]), 4);
            mbar_init(smem_addr(&ctl.p_full[i][1]), 4);
            mbar_init(smem_addr(&ctl.o_full[i]), 1);
            ctl.dirty[i] = 0;
        }
        mbar_init(smem_addr(&ctl.q_full), 8);
        mbar_init(smem_addr(&ctl.e_full), 8);
        ctl.failed = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 9) tm_alloc(smem_addr(&ctl.tmem), 512);
    griddep_wait();
    int flags = 0;
    const MultiLocator<Axis, kMmaThreads> loc(p, flags);
    if (flags && blockIdx.x == 0) flag_status(p.status, flags);
    const MultiSplit split(loc.total, gridDim.x);
    const bool idle = static_cast<int>(blockIdx.x) >= split.ctas;
    const long long unit = idle ? 0 : split.start(blockIdx.x);
    long long left = idle ? 0 : split.start(blockIdx.x + 1) - unit;
    if (!idle) loc.find(p, unit, &ctl.spot);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = ctl.tmem;
    MultiSpot spot = ctl.spot;
    MultiItem it;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8) {
            // ------------------------------------------------------- copies ---
            const int pages = kTile / p.block_size, box_bytes = p.block_size * 128;
            const uint64_t once = l2_evict_first_policy(), again = l2_normal_policy();
            Ring k, v;
            bool ok = true;
            while (ok && Axis::next(p, spot, left, it)) {
                const int seen = Axis::seen(p, it.s, it.m), rows = it.s.c * p.group - it.m * kMultiMmaRows;
                const int lag = rows > kTile ? 0 : 1;   // a V tile is needed after the next tile's K if the streams alternate
                const uint64_t policy = Axis::row_blocks(p, it.s) > 1 ? again : once;
                const int32_t *table = p.block_tables + static_cast<long long>(it.seq) * p.width;
                // Lane l holds page l of a window of 32 pages, as a row of the cache view.
                const auto page_row = [&](int page) {
                    const long long u = static_cast<long long>(page) * p.block_size;
                    if (u >= seen || page >= it.tile1 * pages) return p.total_rows;
                    const int b = table[page];
                    if (b < 0 || b >= p.num_blocks) {
                        flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                        return p.total_rows;
                    }
                    return static_cast<int>((static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size);
                };
                int window = it.tile0 * pages, now = page_row(window + lane), ahead = page_row(window + 32 + lane);
                int row = p.total_rows, row_v = p.total_rows;
                const auto issue = [&](const CUtensorMap *map, int r, uint32_t dst, uint64_t *full) {
                    if (lane == 0) mbar_arrive_expect_tx(smem_addr(full), M::TILE);
                    __syncwarp();
                    if (lane < pages)
    #pragma unroll
                        for (int h = 0; h < HD / 64; ++h)
                            tma_load_2d_hint(dst + h * M::SLAB + lane * box_bytes, map, h * 64, r, smem_addr(full), policy);
                };
                for (int t = it.tile0; t < it.tile1 + lag; ++t) {
                    if (lag) row_v = row;
                    if (t < it.tile1) {
                        if (t * pages >= window + 32) {
                            window += 32;
                            now = ahead;
                            ahead = page_row(window + 32 + lane);
                        }
                        row = __shfl_sync(kFull, now, (t * pages - window + lane) & 31);
                        if (!(ok = await_warp(ctl, &ctl.k_empty[k.slot], k.phase ^ 1))) break;
                        issue(&tmK, row, smem + M::K + k.slot * M::TILE, &ctl.k_full[k.slot]);
                        k.advance<M::NK>();
                    }
                    if (!lag) row_v = row;
                    if (t >= it.tile0 + lag) {
                        if (!(ok = await_warp(ctl, &ctl.v_empty[v.slot], v.phase ^ 1))) break;
                        issue(&tmV, row_v, smem + M::V + v.slot * M::TILE, &ctl.v_full[v.slot]);
                        v.advance<M::NV>();
                    }
                }
            }
        } else if (warp == 9) {
            // --------------------------------------------- matrix instructions ---
            // The whole warp walks, on values that the compiler can see to be the same in all lanes.
            const uint32_t tm = __shfl_sync(kFull, tmem, 0), lead = elect_one();
            Ring k, v;
            uint32_t items = 0, used = 0;   // used: the streams' phases of p_full, a bit each
            bool ok = true;
            while (ok && Axis::next(p, spot, left, it)) {
                const bool both = __shfl_sync(kFull, it.s.c * p.group - it.m * kMultiMmaRows > kTile, 0);
                const int tiles = __shfl_sync(kFull, it.tile1 - it.tile0, 0), count = both ? 2 * tiles : tiles;
                if (!(ok = await_warp(ctl, &ctl.q_full, items++ & 1))) break;
                tm_fence_after();
                // Products of step q, then scores of step q + 2.  The loops are kept short: this warp's instructions come
                // through the same cache as the softmax's many.
    #pragma unroll 1
                for (int q = -2; q < count; ++q) {
                    const int s = q & 1;
                    const bool more = q + 2 < count, last = !both || s == 1;
                    if (q >= 0) {
                        const uint32_t pt = tm + s * kTile, o = tm + 256 + s * kTile;
                        const uint64_t b = smem_desc(smem + M::V + v.slot * M::TILE, M::SLAB);
    #pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            // beside the weights: V for the first half, the next scores' K for the second
                            if (!(ok = await_two(ctl, &ctl.p_full[s][half], (used >> s) & 1u,
                                                 half == 0 ? &ctl.v_full[v.slot] : &ctl.k_full[k.slot],
                                                 half == 0 ? v.phase : k.phase, half == 0 || more)))
                                break;
                            tm_fence_after();
                            const uint64_t vb = b + half * (4 * 16 * 128 >> 4);
                            const uint32_t pa = pt + half * 32;
    #pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ts(o, pa + kk * 8, vb + kk * (16 * 128 >> 4), kIdescO, (q >> 1) % kRun > 0 || half + kk > 0, lead);
    #pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ts(o, pa + 64 + kk * 8, vb + kk * (16 * 128 >> 4), kIdescO, true, lead);
                        }
                        if (!ok) break;
                        used ^= 1u << s;
                        if (!more) mma_commit(smem_addr(&ctl.o_full[s]), lead);
                        if (last) {
                            mma_commit(smem_addr(&ctl.v_empty[v.slot]), lead);
                            v.advance<M::NV>();
                        }
                    } else if (more && !(ok = await_warp(ctl, &ctl.k_full[k.slot], k.phase))) {
                        break;
                    }
                    if (more) {
                        uint64_t a = smem_desc(smem + (both ? s * M::TILE : 0), 16);
                        uint64_t b = smem_desc(smem + M::K + k.slot * M::TILE, 16);
    #pragma unroll 1
                        for (int slab = 0; slab < HD / 64; ++slab, a += M::SLAB >> 4, b += M::SLAB >> 4)
    #pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ss(tm + s * kTile, a + 2 * kk, b + 2 * kk, kIdescS, slab + kk > 0, lead);
                        mma_commit(smem_addr(&ctl.s_full[s]), lead);
                        if (last) {
                            mma_commit(smem_addr(&ctl.k_empty[k.slot]), lead);
                            k.advance<M::NK>();
                        }
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ------------------------------------------------------- softmax ---
        const int s = warp >> 2, r = tid & (kTile - 1);   // stream, and row of its tile
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // first lane of this warp's quarter, in bits 16..
        const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + 256 + s * kTile;
        const float scale = fmaxf(fabsf(p.scale_log2), 1.2e-38f);   // the sign goes into Q; zero stays finite on -inf
        uint32_t step = 0, ends = 0;
        int item_no = 0;
        Ring v;
        bool ok = true;
        // 16 bytes c of this thread's row in its stream's tile of Q, where its results are staged too.
        const auto staged = [&](int row, int c) {
            return reinterpret_cast<uint4 *>(smem_p + s * M::TILE + (c / 8) * M::SLAB + row * 128 + (((c & 7) ^ (row & 7)) << 4));
        };
        const auto arrive = [&](uint64_t *bar) {
            tm_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(bar));
        };
        while (ok) {
            if (!Axis::next(p, spot, left, it)) break;
            __syncwarp();
            if (lane == 0) {
                ctl.walk[warp].spot = spot;
                ctl.walk[warp].left = left;
            }
            ++item_no;
            const int R0 = it.m * kMultiMmaRows, total = it.s.c * p.group - R0;
            const bool both = total > kTile;
            const int rows = both ? min(kTile, total - s * kTile) : total;   // of this stream's tile
            const int row0 = R0 + (both ? s * kTile : 0);
            const int tok = min(row0 + r, it.s.c * p.group - 1) / p.group;
            const int seen = Axis::seen(p, it.s, it.m);
            const int clear = Axis::clear(p, it.s, it.m);   // every row sees every position before
            // Where this row lies in q and out.
            const long long row_at = multi_row(p, it.s, it.kvh, min(row0 + r, it.s.c * p.group - 1), HD);
            if (both || s == 0) {
                // Q, a row per thread, zero behind the last one.
                const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
                const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + row_at);
                uint4 x[HD / 8];
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) x[c] = r < rows ? q[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    x[c].x ^= flip, x[c].y ^= flip, x[c].z ^= flip, x[c].w ^= flip;
                    *staged(r, c) = x[c];
                }
                fence_proxy_async_smem();
            }
            arrive(&ctl.q_full);
            const bool live = (warp & 3) * 32 < rows;   // this warp has rows
            float ref = -INFINITY, sum = 0.f;
            // Where this row's sums of earlier runs are kept, four columns next to the other rows' same: in the CTA's place for
            // this item's partial, which is not written before.
            const auto kept_row = [&] { return static_cast<long long>(it.slot(blockIdx.x)) * p.slot_rows + s * (p.slot_rows / 2); };
            const int tiles = it.tile1 - it.tile0;
            int mine = 0;   // steps of this stream
            for (int t = 0; t < tiles; ++t, v.advance<M::NV>()) {
                if (!both && (t & 1) != s) continue;
                const int u0 = (it.tile0 + t) * kTile;
                // First the scores: they were issued behind the products of this stream's tile before, so the
                // V ring's barrier is in the phase before the awaited one at least.
                if (!(ok = await_warp(ctl, &ctl.s_full[s], step & 1))) break;
                tm_fence_after();
                if (u0 + kTile > clear || u0 + kTile > seen) {
                    // Values that some row does not see: what lies behind the last seen token becomes zero, and
                    // so do values of drafted tokens that are not finite (added again where they are seen).
                    if (!(ok = await_warp(ctl, &ctl.v_full[v.slot], v.phase))) break;
                    uint8_t *vt = smem_p + M::V + v.slot * M::TILE;
                    const int from = max(0, min(kTile, clear - u0));
                    for (int i = from * (HD / 8) + r; i < kTile * (HD / 8); i += kTile) {
                        const int j = i / (HD / 8), c = i % (HD / 8);
                        uint4 *at = reinterpret_cast<uint4 *>(vt + (c / 8) * M::SLAB + j * 128 + (c & 7) * 16);
                        if (u0 + j >= seen) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            if (clear_not_finite(*at)) ctl.dirty[item_no & 1] = item_no;
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (live && mine > 0 && mine % kRun == 0) {
                    // O holds the products of a whole run: these scores were issued behind them.  The next ones start from zero.
                    const int stride = p.slot_rows / 2;
                    float4 *kept = reinterpret_cast<float4 *>(p.part_acc + kept_row() * HD) + r;
                    float *kept_ref = p.part_ml + 2 * (kept_row() + r), f = 0.f;
                    if (r < rows) {
                        if (mine > kRun) f = *kept_ref == ref ? 1.f : ex2(*kept_ref - ref);
                        *kept_ref = ref;
                    }
#pragma unroll 1
                    for (int g = 0; g < HD / 32; ++g, kept += 8 * stride) {
                        float o[32];
                        tm_ld32(to + g * 32, o);
                        tm_wait_ld();
                        if (r < rows) keep_sums(kept, stride, o, f, mine > kRun);
                    }
                }
                if (live) {
                    float x[kTile];
                    // the second half arrives while the first one's maximum is taken
#pragma unroll
                    for (int g = 0; g < 2; ++g) tm_ld32(ts + g * 32, x + g * 32);
                    tm_wait_ld();
#pragma unroll
                    for (int g = 2; g < 4; ++g) tm_ld32(ts + g * 32, x + g * 32);
                    const bool masked = u0 + kTile > clear;
                    const auto hide = [&](int g) {
                        const uint32_t bits = multi_seen_bits(p, it.s, tok, u0 + g * 32);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!((bits >> c) & 1u)) x[g * 32 + c] = -INFINITY;
                    };
                    if (masked) hide(0), hide(1);
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < kTile / 2; c += 2) top[c / 2 & 3] = fmaxf(fmaxf(top[c / 2 & 3], x[c]), x[c + 1]);
                    tm_wait_ld();
                    if (masked) hide(2), hide(3);
#pragma unroll
                    for (int c = kTile / 2; c < kTile; c += 2)
                        top[c / 2 & 3] = fmaxf(fmaxf(top[c / 2 & 3], x[c]), x[c + 1]);
                    const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
                    if (mine == 0) {
                        ref = best;
                    } else if (__any_sync(kFull, best > ref + 8.f)) {
                        const float now = fmaxf(ref, best);
                        const float f = now == ref ? 1.f : ex2(ref - now);
                        // O holds the products of the step before: these scores were issued behind them, and
                        // their barrier waits for every matrix instruction issued so far
#pragma unroll 1
                        for (int g = 0; g < HD / 16; ++g) {
                            float o[16];
                            uint32_t u[16];
                            tm_ld16(to + g * 16, o);
                            tm_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(o[c] * f);
                            tm_st16(to + g * 16, u);
                        }
                        sum *= f;
                        ref = now;
                    }
                    const float shift = ref == -INFINITY ? 0.f : -ref;
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float *a = x + g * 32 + 2 * c;
                            const float2 y = fma2(make_float2(a[0], a[1]), make_float2(scale, scale), make_float2(shift, shift));
                            const float2 w = make_float2(ex2(y.x), ex2(y.y));
                            part[c & 1] = add2(part[c & 1], w);
                            weight_parts(w, hi[c], lo[c]);
                        }
                        tm_st16(ts + g * 16, hi);
                        tm_st16(ts + 64 + g * 16, lo);
                        if (g == 1) {   // the products with the first 64 tokens may begin
                            tm_wait_st();
                            arrive(&ctl.p_full[s][0]);
                        }
                    }
                    const float2 both_parts = add2(part[0], part[1]);
                    sum += both_parts.x + both_parts.y;
                    tm_wait_st();
                } else {
                    arrive(&ctl.p_full[s][0]);
                }
                arrive(&ctl.p_full[s][1]);
                ++step;
                ++mine;
            }
            if (!ok) break;
            // The item's end: all products are in, and both streams say what they have, in tensor memory.  In other
            // columns than the item before: a stream without steps in this item does not wait for the other one, which
            // may still be reading there.
            if (mine > 0 && !(ok = await_warp(ctl, &ctl.o_full[s], ends++ & 1))) break;
            tm_fence_after();
            if (live && mine > kRun) {   // the earlier runs' sums join the last one's
                const int stride = p.slot_rows / 2;
                const float4 *kept = reinterpret_cast<const float4 *>(p.part_acc + kept_row() * HD) + r;
                float f = 0.f;
                if (r < rows) {
                    const float kept_ref = p.part_ml[2 * (kept_row() + r)];
                    f = kept_ref == ref ? 1.f : ex2(kept_ref - ref);
                }
#pragma unroll 1
                for (int g = 0; g < HD / 16; ++g, kept += 4 * stride) {
                    float o[16];
                    float4 y[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) y[c] = r < rows ? __ldcg(kept + c * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
                    tm_ld16(to + g * 16, o);
                    tm_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        u[4 * c] = __float_as_uint(fmaf(y[c].x, f, o[4 * c]));
                        u[4 * c + 1] = __float_as_uint(fmaf(y[c].y, f, o[4 * c + 1]));
                        u[4 * c + 2] = __float_as_uint(fmaf(y[c].z, f, o[4 * c + 2]));
                        u[4 * c + 3] = __float_as_uint(fmaf(y[c].w, f, o[4 * c + 3]));
                    }
                    tm_st16(to + g * 16, u);
                }
                tm_wait_st();
            }
            const uint32_t sums_at = 2 * (item_no & 1);
            if (!both) {
                tm_st2(ts + sums_at, __float_as_uint(ref), __float_as_uint(sum));
                tm_wait_st();
            }
            arrive(&ctl.e_full);
            if (!(ok = await_warp(ctl, &ctl.e_full, (item_no - 1) & 1))) break;
            tm_fence_after();
            if (live) {
                const bool dirty = ctl.dirty[item_no & 1] == item_no;
                float f[2] = {1.f, 1.f}, top = ref, all = sum;
                if (!both) {
                    float a[4];
                    tm_ld2(tmem + lanes + sums_at, a);
                    tm_ld2(tmem + lanes + kTile + sums_at, a + 2);
                    tm_wait_ld();
                    top = fmaxf(a[0], a[2]);
                    const float at = top == -INFINITY ? 0.f : top;
                    f[0] = ex2(a[0] - at);
                    f[1] = ex2(a[2] - at);
                    all = f[0] * a[1] + f[1] * a[3];
                }
                const bool second = !both && tiles > 1, whole = it.whole();
                if (whole) {
                    const float inv = all == 0.f ? 0.f : 1.f / all;
                    f[0] *= inv;
                    f[1] *= inv;
                }
                // 16 columns of the row's result, ready to be written.
                const auto result = [&](int g, float *o) {
                    tm_ld16((both ? to : tmem + lanes + 256) + g * 16, o);
                    float o1[16];
                    if (second) tm_ld16(tmem + lanes + 256 + kTile + g * 16, o1);
                    tm_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = second ? fmaf(o1[c], f[1], o[c] * f[0]) : o[c] * f[0];
                    if (dirty && r < rows)
                        for (int u = max(max(clear, 0), it.tile0 * kTile); u < min(seen, it.tile1 * kTile); ++u) {
                            if (!(multi_seen_bits(p, it.s, tok, u) & 1u)) continue;
                            const int b = p.block_tables[static_cast<long long>(it.seq) * p.width + u / p.block_size];
                            if (b < 0 || b >= p.num_blocks) continue;
                            const __nv_bfloat16 *vr =
                                static_cast<const __nv_bfloat16 *>(p.v_cache) +
                                ((static_cast<long long>(b) * p.num_kv_heads + it.kvh) * p.block_size + u % p.block_size) * HD;
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float y = __bfloat162float(vr[g * 16 + c]);
                                if (!isfinite(y)) o[c] += y;
                            }
                        }
                };
                // Rows go through the warp's own rows of its Q tile, so that they are written to memory in full lines.
                const int g0 = both ? 0 : s * (HD / 32), g1 = both ? HD / 16 : g0 + HD / 32;
                const auto flush = [&](char *dst, long long at, int chunks) {
                    __syncwarp();
                    const int per = 32 / chunks;   // rows per turn
                    for (int k = 0; k < 32; k += per) {
                        const int row = k + lane / chunks;
                        const long long to_row = __shfl_sync(kFull, at, row);
                        if ((warp & 3) * 32 + row < rows)
                            *reinterpret_cast<uint4 *>(dst + to_row + (lane % chunks) * 16) =
                                *staged((warp & 3) * 32 + row, lane % chunks);
                    }
                    __syncwarp();
                };
                if (whole) {
#pragma unroll 1
                    for (int g = g0; g < g1; ++g) {
                        float o[16];
                        result(g, o);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            *staged(r, (g - g0) * 2 + c) =
                                make_uint4(bf16_pair(o[8 * c], o[8 * c + 1]), bf16_pair(o[8 * c + 2], o[8 * c + 3]),
                                           bf16_pair(o[8 * c + 4], o[8 * c + 5]), bf16_pair(o[8 * c + 6], o[8 * c + 7]));
                    }
                    flush(static_cast<char *>(p.out) + g0 * 32, row_at * 2, (g1 - g0) * 2);
                } else {
                    const long long at = static_cast<long long>(it.slot(blockIdx.x)) * p.slot_rows + (both ? s * kTile : 0) + r;
#pragma unroll 1
                    for (int h = g0; h < g1; h += HD / 32) {   // as many columns as a staged row holds
#pragma unroll 1
                        for (int g = h; g < h + HD / 32; ++g) {
                            float o[16];
                            result(g, o);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                store4(reinterpret_cast<float *>(staged(r, (g - h) * 4 + c)),
                                       make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
                        }
                        flush(reinterpret_cast<char *>(p.part_acc) + h * 64, at * HD * 4, HD / 8);
                    }
                    if (r < rows && (both || s == 0))
                        *reinterpret_cast<float2 *>(p.part_ml + 2 * at) = make_float2(top, all);
                }
            }
            __syncwarp();
            spot = ctl.walk[warp].spot;
            left = ctl.walk[warp].left;
        }
    }

    griddep_launch_dependents();
    __syncwarp();
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    if (ctl.failed) {
        // A wait gave up: copies and products in flight get a millisecond to land.
        if (tid == 0) flag_status(p.status, PA_STATUS_WAIT_TIMEOUT);
        for (const uint64_t start = global_timer_ns(); global_timer_ns() - start < 1000000ull;) {
        }
        __syncthreads();
    }
    if (warp == 9) tm_dealloc(tmem, 512);
}

// A cache seen as [rows][HD], boxes of one block's rows x 64 columns with the
// 128-byte swizzle; rows past the end read as zeros.
bool block_map(CUtensorMap *map, const void *base, long long rows, int hd, int block_size) {
    const host::EncodeTiledFn enc = host::encode_tiled();
    if (!enc) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(hd) * 2};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(block_size)}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD>
int multi_mma(const MultiParams &p, int dev, cudaStream_t st) {
    static host::KernelSlot slot;
    auto kernel = multi_mma_kernel<HD>;
    if (host::ensure_kernel(kernel, slot, Smem<HD>::BYTES, dev, kMmaThreads) == 0)
        return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cannot configure the bf16 kernel");
    CUtensorMap mk, mv;
    if (!block_map(&mk, p.k_cache, p.total_rows, HD, p.block_size) ||
        !block_map(&mv, p.v_cache, p.total_rows, HD, p.block_size))
        return pa_fail(PA_ERR_CUDA, "pa_decode_tree/cross: cuTensorMapEncodeTiled failed");
    const int grid = min(host::sm_count(dev), kMultiMmaCtas);
    const cudaError_t e = host::launch_dependent(kernel, grid, kMmaThreads, Smem<HD>::BYTES, st, mk, mv, p);
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return launch_join<__nv_bfloat16, HD, AxisOf<HD>>(p, grid, st);
}

}  // namespace

int launch_multi_mma(const MultiParams &p, int head_dim, int dev, cudaStream_t st) {
    return head_dim == 128 ? multi_mma<128>(p, dev, st) : multi_mma<64>(p, dev, st);
}

}  // namespace pa
