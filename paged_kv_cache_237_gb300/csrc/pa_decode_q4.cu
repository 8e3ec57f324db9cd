// Decode attention over the 4-bit paged cache (include/pa.h states the
// format), partition pass for sm_103a.
//
// For a query row q and a token t with codes c, steps s_g and minima m_g:
//   q . K_t = sum_g s_g (sum_{d in g} q_d c_d) + m_g (sum_{d in g} q_d)
//   o_d     = sum_t p_t (s_g c_td + m_g)
// Work.  A row is one (sequence, KV head, head tile); laid end to end, the
// batch's rows are one axis of units of 32 tokens, and every warp takes an equal
// stretch of it, so that all finish together whatever the lengths.  A warp
// stores the rows that lie in its stretch whole, and one partial for a row that
// its stretch's beginning or end cuts; a second launch joins those.  No barrier
// and no counter: warps do not meet.
//
// The products run on fp16 tensor-core MMAs with tokens as rows of both: S = K
// Q^T has K's codes as its A operand, O^T = V^T W has V's.  With tokens as
// rows, up to eight query heads are one tile of columns.  For bf16 q and out, a
// code masked out of its word is already the fp16 subnormal code * 2^-24 (the
// next nibble up: code * 2^-20), so unpacking eight codes is one shift and four
// ands, and the powers of two are undone where they cost nothing, in q and in
// the output.  The tensor core aligns a subnormal's products by its nominal
// exponent, which leaves sums about 17 bits: plenty for a bf16 result (8), not
// for fp32.  It also cuts sums off towards zero, so V's codes are taken as c for
// the first eight tokens of a product's sixteen and as -(15 - c), with the sign in
// the weight and the maximum m + 15 s for the minimum, for the others: sums of both
// signs stay small, and what is cut off, or rounded off weights that are alike,
// does not add up (flat scores over values of mean zero are the worst case: the
// output is a small difference of large sums).  fp32 q and out take codes as the
// normal values c - 7.5 and the middle of the range for the minimum, s c + m =
// s (c - 7.5) + (m + 7.5 s), to the same end; two fp16 parts of q and of the
// weights, the second scaled up, since a small weight's second part would be
// subnormal; and each part's products in an accumulator of its own, added in fp32.
//
// What bounds it: 16 tokens of a head row of 128 are 2304 bytes and over 200 warp
// instructions (40 % on the ALU pipe, which takes two cycles each: 64 ands and 24
// permutes and shifts unpack the codes), so their issue and HBM are close, and every
// instruction taken out of the loop has counted.  Pages come by 16-byte
// asynchronous copies, 8 or 16 lanes a page: nine instructions for a stage, where a
// bulk copy per page takes a loop over the lanes that ask, a barrier and a fence
// (50.2 for 47.3 us on the lognormal batch below, 138.5 for 130.9 on the long one, 81.5
// for 72.6 with head_dim 64, when it was taken).
// Measured (graph replays): 256 sequences of 16..8192 tokens, GQA 64/8, 1.2 GB:
// 197.7 us, 0.91 of the copy peak (pass 190, 0.95; join 8); 32 lognormal sequences, 235
// MB: 47.6 us, 0.74 (about 5 are the pass' start and end, 4.6 the join); 7 sequences of
// up to 131072, groups of 32: 133.7 us, 0.88; head_dim 64 without head groups, window
// 2000: 72.1 us, 0.75 (the softmax and the parameters cost as much for half the bytes);
// fp32 q and out, 32 sequences of 1000..6000, GQA 64/8: 55.9 us with groups of 32, 50.0
// with 64, 0.39 (issue: 65 % of slots, and 8 warps per SM to hide latency with).  Of
// this the two signs of V's codes cost 0.5 to 3 %, the second set of sums 0.5 %, weights
// that keep their bits 0 to 4 % (fp32: 3; with 16 heads a group 8).  On plain FMAs, one
// token a warp: 5691, 1231, 3390 and 1508 us for the first four.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>

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

// 2^x to about 2^-22, results below the normals flushed to zero: weights are
// relative to one of 1, or more than 2^-5 once others have outgrown it.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The products of N values, and of a factor with each, or added to sums: PACKED,
// two at a time (Blackwell's packed fp32, each half rounded as by itself; 1 to 2 %
// of the whole for bf16, while fp32's kernels have no registers for the pairs).
template <bool PACKED, int N>
__device__ __forceinline__ void times(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += PACKED && N % 2 == 0 ? 2 : 1) {
        if constexpr (PACKED && N % 2 == 0) {
            const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
            d[i] = v.x, d[i + 1] = v.y;
        } else {
            d[i] = a[i] * b[i];
        }
    }
}
template <bool PACKED, int N>
__device__ __forceinline__ void times(float (&d)[N], float f, const float (&b)[N]) {
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = f;
    times<PACKED>(d, a, b);
}
template <bool PACKED, int N>
__device__ __forceinline__ void add_times(float (&d)[N], float f, const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += PACKED && N % 2 == 0 ? 2 : 1) {
        if constexpr (PACKED && N % 2 == 0) {
            const float2 v = __ffma2_rn(make_float2(f, f), make_float2(b[i], b[i + 1]), make_float2(d[i], d[i + 1]));
            d[i] = v.x, d[i + 1] = v.y;
        } else {
            d[i] = fmaf(f, b[i], d[i]);
        }
    }
}
template <bool PACKED, int N>
__device__ __forceinline__ void add_times(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += PACKED && N % 2 == 0 ? 2 : 1) {
        if constexpr (PACKED && N % 2 == 0) {
            const float2 v = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(d[i], d[i + 1]));
            d[i] = v.x, d[i + 1] = v.y;
        } else {
            d[i] = fmaf(a[i], b[i], d[i]);
        }
    }
}

// A token's steps and minima, or (NORMAL: codes less 7.5) the middles of its ranges.
template <int NG, bool NORMAL>
__device__ __forceinline__ void load_pairs(const uint8_t *at, float (&s)[NG], float (&m)[NG]) {
    uint32_t pair[NG];
    if constexpr (NG == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(at);
        pair[0] = x.x, pair[1] = x.y, pair[2] = x.z, pair[3] = x.w;
    } else if constexpr (NG == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(at);
        pair[0] = x.x, pair[1] = x.y;
    } else {
        pair[0] = *reinterpret_cast<const uint32_t *>(at);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        s[i] = q4_step(pair[i]);
        m[i] = NORMAL ? fmaf(7.5f, s[i], q4_min(pair[i])) : q4_min(pair[i]);
    }
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The two nibble pairs (a nibble of each half-word) at a time that make the
// codes of two units fp16 operands: values 0, 1, 2, 3 of both units.  NORMAL:
// code - 7.5, exactly, by way of 16 + code (whose mantissa holds the code in its
// upper bits).  Otherwise code * 2^-24, and code * 2^-20 for values 1 and 3.
template <bool NORMAL>
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t (&r)[4]) {
    if constexpr (NORMAL) {
        r[0] = x << 6;
        r[1] = x << 2;
        r[2] = x >> 2;
        r[3] = x >> 6;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = (r[i] & 0x03c003c0u) | 0x4c004c00u;
            asm("sub.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(0x4de04de0u));   // 23.5
        }
    } else {
        r[0] = x & 0x000f000fu;
        r[1] = x & 0x00f000f0u;
        x >>= 8;
        r[2] = x & 0x000f000fu;
        r[3] = x & 0x00f000f0u;
    }
}

// The same for V, whose products can be untangled in the output: not NORMAL,
// values 1 and 3 come as whole bytes, lower code * 2^-24 + code * 2^-20, which
// saves an and each.  UPPER: 15 - code in place of code.
template <bool NORMAL, bool UPPER>
__device__ __forceinline__ void codes_or_bytes_f16(uint32_t x, uint32_t (&r)[4]) {
    if constexpr (NORMAL) {
        codes_f16<true>(x, r);
    } else if constexpr (UPPER) {
        r[1] = ~x & 0x00ff00ffu;
        r[0] = ~x & 0x000f000fu;
        // 255 - byte as an fp16 subtraction (exact), which the FMA pipe takes
        asm("sub.f16x2 %0, %1, %2;" : "=r"(r[3]) : "r"(0x00ff00ffu), "r"(__byte_perm(x, 0u, 0x4341)));
        r[2] = r[3] & 0x000f000fu;
    } else {
        r[1] = x & 0x00ff00ffu;
        r[0] = x & 0x000f000fu;
        r[3] = __byte_perm(x, 0u, 0x4341);
        r[2] = r[3] & 0x000f000fu;
    }
}

// 16 bytes to shared memory, both addresses 16-byte aligned; a group of them; and
// the wait until at most `left` (up to MOST) of the newest groups are on their way.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int MOST>
__device__ __forceinline__ void copies_wait(uint32_t left) {
    if constexpr (MOST > 0) {
        if (left < MOST) return copies_wait<MOST - 1>(left);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(MOST) : "memory");
}

// The smallest power of two above x >= 0, within [2^-100, 2^120].
__device__ __forceinline__ float pow2_above(float x) {
    const float c = fminf(fmaxf(x, 0x1p-101f), 0x1p119f);
    return __uint_as_float((__float_as_uint(c) + 0x800000u) & 0x7f800000u);
}

// The largest weight when its scale is chosen, from below; and what the second
// fp16 part of a weight (fp32) is multiplied by, so that it has as many bits as
// the first down to the first's subnormals (their sum's steps end at 2^-36).
constexpr float kLift = 256.f, kPart = 2048.f;

constexpr int kQ4Warps = 4;   // per CTA; they are independent

// Launch shape: stages per warp, and the CTAs per SM the kernel is built for.
// The pass is bound by instruction issue, so it wants registers (163 of 168)
// before warps: 3 CTAs of 4 warps take 198 us on 256 sequences x 16..8192
// tokens (GQA 64/8, groups of 64), 4 CTAs at 128 registers 204.  Four warps per
// CTA keep the SM's four schedulers evenly loaded, which equal stretches need:
// 12 or 14 CTAs of one warp take 10 to 15 % longer.  fp32's kernels for head_dim 128
// (SPLIT) would spill at 168 registers: 2 CTAs, 53.7 us against 59.3 on 32 sequences,
// GQA 64/8, groups of 32.  Two tiles of heads (NT) fit 168 for bf16 and head_dim 64
// only: 27.7 us against 28.5 with 2 CTAs (64 sequences of 1000..6000, GQA 64/4).
template <int HD, int NT, bool SPLIT>
struct Q4Shape {
    static constexpr int NSTAGE = 2;   // 3 and 4 change nothing, or cost 2 % (head_dim 128)
    static constexpr int CPS = (NT == 2) + SPLIT + (HD == 128) >= 2 ? 2 : 3;
};

// Every kHoldBlocks blocks of 32 units (4096 tokens) a lane adds its running sums
// to a second set, in shared memory, and starts anew: whatever a row's length, no
// accumulator adds up more.  (An fp32 sum of n equal terms may be n 2^-25 off, a
// tensor core's more.)  q4_held: the sums of a lane, and q4_held_all: with the
// references and scales that they go by.
constexpr int kHoldBlocks = 4;

template <int HD, int G, int NT, int NC>
__host__ __device__ constexpr int q4_held() { return NT * (HD / 16 * 4 + NC * (HD / G) + NC); }
template <int HD, int G, int NT, int NC>
__host__ __device__ constexpr int q4_held_all() { return q4_held<HD, G, NT, NC>() + NT * NC + HD / G; }

constexpr int kUnit = 32;   // tokens per stage: one block of 32 or two of 16

// Where a warp stands on the axis, kept in shared memory.
struct Walk {
    uint32_t pos, begin, end;    // next place, and the warp's stretch
    uint32_t base, places;       // first place of sequence seq, places of each of its rows
    int seq, n, seen, skip, begins, index;
};

// Up to 32 units of one row, kept in shared memory.
struct Block {
    int seq, qh0, rows, n, skip, tok_begin, tok_end;
    int first, last;             // of the row's units in this stretch
    int begins, whole;           // the stretch holds the row's beginning; the whole row
    int index;                   // of the block in the row's part of this stretch
};

// The split-K state of a call, in its workspace.
struct Q4Split {
    uint32_t *share;             // places per warp
    uint32_t *bases;             // [S] first place of each sequence
    float *ml, *acc;             // [warps][2][rows][2] and [..][HD]: a row that the stretch
                                 // does not begin (0) or does not end (1)
    uint32_t stretches;          // that there is room for
};

__device__ __forceinline__ uint32_t row_units(int seen) { return seen > kUnit ? (seen + kUnit - 1) / kUnit : 1; }

// A row takes kRowCost more places on the axis than it has units, before them:
// what beginning and ending a row costs a warp, in units.
constexpr uint32_t kRowCost = 3;   // 256 sequences x 16..8192 tokens: 2 takes 200 us, 3 198, 4 198.5
__device__ __forceinline__ uint32_t row_places(int seen) { return row_units(seen) + kRowCost; }

// T: type of q and out.  fp32 splits q and the weights into two fp16 parts.
// NT: tiles of 8 query heads per row.  NC: columns of a tile that a lane looks
// after; 1 where a row has at most 4 heads, which then take the even columns and
// leave the lanes half the softmax (64 sequences, GQA 32/8: 132 us for 141; MHA of
// head_dim 64: 82 for 92).
// bs: block size.
template <typename T, int HD, int G, int NT, int NC, int bs>
__global__ void __launch_bounds__(kQ4Warps * 32, Q4Shape<HD, NT, sizeof(T) == 4>::CPS)
    decode_q4_kernel(const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache, const DecodeParams p,
                     const Q4Split split, uint32_t warps, uint32_t min_share) {
    using F = Q4Format<HD, G>;
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int PARTS = SPLIT ? 2 : 1;
    constexpr int NSTAGE = Q4Shape<HD, NT, sizeof(T) == 4>::NSTAGE;
    constexpr int W = F::W, NG = F::GROUPS;
    constexpr int HALF_BYTES = kUnit * F::ROW_BYTES;   // a stage's K, then its V
    constexpr int STAGE_BYTES = 2 * HALF_BYTES;
    constexpr int WARP_BYTES = NSTAGE * STAGE_BYTES;
    constexpr int ROWS = 4 * NC * NT;
    static_assert(NC == 2 || NT == 1);
    constexpr int OW = HD / 32;    // code words a lane feeds to one token row's products
    constexpr int MT = HD / 16;    // m-tiles of the output

    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t *wbuf = smem + warp * WARP_BYTES;
    // (volatile: one after the other, or the batch of them takes 15 registers that the loop needs)
    volatile float *const held = reinterpret_cast<float *>(smem + kQ4Warps * WARP_BYTES) + warp * 32 * q4_held_all<HD, G, NT, NC>() + lane;
    constexpr int HELD = q4_held<HD, G, NT, NC>();
    const uint32_t wbuf_s = smem_addr(wbuf);

    // Where the 16-token halves of a stage begin: two pages, or one of 32 rows.
    constexpr int bs_shift = bs == 32 ? 5 : 4;
    constexpr int page_bytes = bs * F::ROW_BYTES;
    constexpr int code_half = bs == 16 ? page_bytes : 16 * F::CODE_BYTES;
    constexpr int par_0 = bs * F::CODE_BYTES, par_half = bs == 16 ? page_bytes : 16 * F::PARAM_BYTES;
    // Token of matrix row g (row g + 8 is 8 further): neighbours swapped in
    // every other pair, so that a lane octet's reads of V hit both halves of
    // the banks.
    const int row_g = g ^ ((g >> 1) & 1);
    const int tok_a = (2 * t) ^ (t & 1), tok_b = (2 * t + 1) ^ (t & 1);   // matrix rows 2 t and 2 t + 1

    uint32_t n_issued = 0, n_done = 0;
    const uint64_t kv_policy = l2_evict_first_policy();
    griddep_wait();   // everything above touched only this warp's registers and shared memory

    // The warp's stretch.  Without a split (every row is short) it counts rows.
    const bool cut = split.share != nullptr;
    const uint32_t heads = p.num_kv_heads * p.head_tiles;
    __shared__ Walk s_walk[kQ4Warps];
    __shared__ Block s_blocks[kQ4Warps][2];
    Walk &walk = s_walk[warp];
    {
        const uint32_t me = blockIdx.x * kQ4Warps + warp;   // those past `warps` get nothing
        uint32_t total = p.num_seqs;
        if (cut) {
            total = 0;
            for (int s = lane; s < p.num_seqs; s += 32) total += row_places(seq_view<true>(p, s).seen);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) total += __shfl_xor_sync(kFull, total, o);
        }
        total *= heads;
        const uint32_t share = max((total + warps - 1) / warps, cut ? min_share : 1u);
        const uint32_t begin = min(total, me * share), end = min(total, begin + share);
        if (cut && me == 0 && lane == 0) *split.share = share;
        // The sequence that holds place `begin`, 32 lengths at a time.
        int seq = cut ? 0 : static_cast<int>(begin / heads);
        uint32_t base = cut ? 0 : seq * heads;
        while (cut && seq < p.num_seqs) {
            const int s = seq + lane;
            const uint32_t u = s < p.num_seqs ? row_places(seq_view<true>(p, s).seen) * heads : 0u;
            uint32_t incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned hit = __ballot_sync(kFull, begin < base + incl);
            if (hit) {
                const int at = __ffs(hit) - 1;
                base += __shfl_sync(kFull, incl - u, at);
                seq += at;
                break;
            }
            base += __shfl_sync(kFull, incl, 31);
            seq += 32;
        }
        if (lane == 0) {
            const SeqView view = begin < end ? seq_view<true>(p, seq) : SeqView{0, 0, 0};
            walk = Walk{begin, begin, end, base, cut ? row_places(view.seen) : 1u, seq, view.n, view.seen, view.skip, 0, 0};
        }
        __syncwarp();
    }
    // Takes up the next block of the stretch: its description into shared
    // memory, its pages into page_a and page_b (lane k holds unit k's first and,
    // with block size 16, second, as block * heads + head; -1 is a block id out
    // of range, -2 a page past the block's tokens).  Returns its units, at most
    // 32; -1 past the last.
    auto read_block = [&](Block &to, int &page_a, int &page_b) {
        page_a = page_b = -2;
        uint32_t pos = walk.pos;
        const uint32_t stretch_end = walk.end;
        if (pos >= stretch_end) return -1;
        int seq = walk.seq;
        uint32_t base = walk.base, rp = walk.places;
        SeqView view{walk.n, walk.seen, walk.skip};
        while (pos >= base + rp * heads) {
            base += rp * heads;
            view = seq_view<true>(p, ++seq);
            if (cut) rp = row_places(view.seen);
        }
        const uint32_t in_seq = pos - base, h = in_seq / rp, at = in_seq - h * rp;
        uint32_t u = 0, left = 1;      // the row's next unit, and how many follow in this stretch
        if (cut) {
            const uint32_t skipped = at < kRowCost ? kRowCost - at : 0u;
            u = at + skipped - kRowCost;
            pos += skipped;
            if (pos >= stretch_end) return -1;   // the row's units are all the next stretch's
            left = min(rp - at - skipped, stretch_end - pos);
        }
        const int units = cut ? static_cast<int>(min(left, 32u)) : static_cast<int>(row_units(view.seen));
        const bool first = u == 0 || pos == walk.begin, last = !cut || units == static_cast<int>(left);
        const bool begins = first ? u == 0 : walk.begins != 0;
        const int kvh = h / p.head_tiles, ht = h - kvh * p.head_tiles;
        const int begin = static_cast<int>(u) * kUnit, end = min(view.seen, begin + units * kUnit);
        const int index = first ? 0 : walk.index + 1;
        __syncwarp();   // the slot's last readers, and the walk's, are done
        if (lane == 0) {
            to = Block{seq, kvh * p.group + ht * ROWS, min(ROWS, p.group - ht * ROWS), view.n, view.skip, begin, end,
                       first, last, begins, begins && (!cut || u + units + kRowCost == rp), index};
            walk.pos = pos + (cut ? units : 1);
            walk.base = base;
            walk.places = rp;
            walk.seq = seq;
            walk.n = view.n;
            walk.seen = view.seen;
            walk.skip = view.skip;
            walk.begins = begins;
            walk.index = index;
            if (h == 0 && u == 0) {
                if (cut) split.bases[seq] = base;
                const int raw = p.context_lens[seq];
                if (raw < 0 || raw > p.ctx_cap) flag_status(p.status, PA_STATUS_BAD_CONTEXT_LEN);
            }
        }
        __syncwarp();
        auto page_of = [&](int v) {
            if (v >= end) return -2;
            const int pos = v >= p.sink_end ? v + view.skip : v;
            const int phys = p.block_tables[(long long)seq * p.max_blocks_per_seq + (pos >> bs_shift)];
            if (phys < 0 || phys >= p.num_blocks) {
                flag_status(p.status, PA_STATUS_BAD_BLOCK_ID);
                return -1;
            }
            return phys * p.num_kv_heads + kvh;
        };
        const int v = begin + lane * kUnit;
        page_a = page_of(v);
        if (bs == 16) page_b = page_of(v + 16);
        return units;
    };
    // A stage's copies: 8 lanes (block size 32: 16) take a page each, K's and V's and
    // with block size 16 those of the second half, 16 bytes a lane at a time.
    constexpr int LANES = bs == 16 ? 8 : 16, PIECES = page_bytes / 16;
    const int sub = lane % LANES;
    const bool of_v = (lane / LANES) & 1, of_b = bs == 16 && lane >= 16;
    const uint8_t *const from = (of_v ? v_cache : k_cache) + 16 * sub;
    const uint32_t to = wbuf_s + (of_v ? HALF_BYTES : 0) + (of_b ? page_bytes : 0) + 16 * sub;
    auto issue = [&](int page_a, int page_b, int k) {
        int page = __shfl_sync(kFull, page_a, k);
        if (bs == 16) {
            const int b = __shfl_sync(kFull, page_b, k);
            if (of_b) page = b;
        }
        if (page >= 0) {
            const uint8_t *src = from + (long long)page * page_bytes;
            const uint32_t dst = to + n_issued % NSTAGE * STAGE_BYTES;
#pragma unroll
            for (int i = 0; i < PIECES; i += LANES)
                if (PIECES - i >= LANES || sub < PIECES - i) copy16_async(dst + 16 * i, src + 16 * i, kv_policy);
        }
        copies_commit();
        ++n_issued;
    };

    // A row's state, carried from block to block.
    uint32_t qf[PARTS][NT][OW][4];
    float qs[NT][NC];           // per column (head): undoes q's scaling, times scale * log2(e)
    // Sums of q over a group, times scale * log2(e): by column and group, or
    // (bf16) group t's of head g as the coefficient of m in a B operand whose
    // A operand is a row's (s, m) pairs as they are, in two bf16 parts.
    float qsum[SPLIT ? NT : 1][NC][NG];
    uint32_t qm[NT][2];
    float o[MT][NT][4];         // [row g or g + 8][column]: sums of w * code, see below
    float om[NT][NC][NG];       // this lane's tokens' sum of p * m
    float less[NT][4], l[NT][NC];  // minus the columns' references, as an accumulator; sums of p
    // w = p * s * inv with inv = kLift / S, S a power of two; bf16: 15 steps are
    // fifteen times s inv
    float inv[NG], fifteen[NG];
    auto S = [&](int i) { return __uint_as_float(0x83000000u - __float_as_uint(inv[i])); };
    // f(sum, its place among the held, its tile and column, and of o its group)
    auto each_sum = [&](auto &&f) {
        int j = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                f(l[nt][c], j++, nt, c, -1);
#pragma unroll
                for (int i = 0; i < NG; ++i) f(om[nt][c][i], j++, nt, c, -1);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) f(o[mt][nt][c], j++, nt, c % NC, G == 64 ? mt / 4 : mt / 2);
        }
    };

    int slot = 0, page_a, page_b, next_a, next_b;
    int units = read_block(s_blocks[warp][0], page_a, page_b);
    int asked = 0, asked_next = 0;        // units of the two blocks that have been issued
    while (units >= 0) {
        const Block &it = s_blocks[warp][slot];
        for (; asked < units && n_issued - n_done < NSTAGE; ++asked) issue(page_a, page_b, asked);
        const int next_units = read_block(s_blocks[warp][slot ^ 1], next_a, next_b);
        const bool some_bad = __any_sync(kFull, page_a == -1 || page_b == -1);
        // Tokens from all_from to all_to are not masked.
        const int all_from = max(0, it.n - p.window) - it.skip, all_to = it.tok_end, tok_begin = it.tok_begin;
        const bool first = it.first;
        if (first) {

        // q as B operands: lane (g, t) holds head g of each tile, the units of
        // its code words, divided by a power of two that brings the row's
        // largest magnitude into [2^14, 2^15) (exact for bf16: 8 bits of an
        // fp16's 11), and by 16 where a code comes out 16 times too large.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = NC == 2 ? 8 * nt + g : g / 2;   // of column g
            const bool live = head < it.rows && (NC == 2 || g % 2 == 0);
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
            // To the columns of the accumulators: 2 t and 2 t + 1.
            const float back = p.scale_log2 * (SPLIT ? 1.f : 0x1p24f) * pow2i(e);
            float own = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                sum[i] *= p.scale_log2;
                if (t == i) own = sum[i];
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                qs[nt][c] = __shfl_sync(kFull, back, 4 * (2 * t + c));
                if constexpr (SPLIT)
#pragma unroll
                    for (int i = 0; i < NG; ++i) qsum[nt][c][i] = __shfl_sync(kFull, sum[i], 4 * (2 * t + c));
            }
            // two bf16 parts (16 bits), each over a zero that meets the step
            qm[nt][0] = __float_as_uint(own) & 0xffff0000u;
            qm[nt][1] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(own - __uint_as_float(qm[nt][0]))))
                        << 16;
        }

#pragma unroll
        for (int i = 0; i < NG; ++i) {
            inv[i] = kLift;
            fifteen[i] = 15.f / kLift;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)   // (a column without a head has no weights)
                less[nt][c] = 8 * nt + NC * t + (NC == 2 ? c % 2 : 0) < it.rows ? 0.f : -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                l[nt][c] = 0.f;
#pragma unroll
                for (int i = 0; i < NG; ++i) om[nt][c][i] = 0.f;
            }
        }

        }   // first

        for (int k = 0; k < units; ++k) {
            const int s = n_done % NSTAGE;
            copies_wait<NSTAGE - 1>(n_issued - n_done - 1);
            __syncwarp();   // every lane's copies, for all
            ++n_done;
            uint8_t *stage = wbuf + s * STAGE_BYTES;
            const int v0 = tok_begin + k * kUnit;
            uint32_t hidden = 0;   // bits of this lane's tokens: 2 half + row, set where masked
            const bool masked = some_bad || v0 < all_from || v0 + kUnit > all_to;
            if (masked) {
                // A block id out of range reads as zeros, and a masked token's
                // parameters become zeros (its codes are finite whatever they are).
                const bool bad[2] = {__shfl_sync(kFull, page_a, k) == -1, __shfl_sync(kFull, page_b, k) == -1};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (bad[half])
                        for (int i = lane * 4; i < page_bytes; i += 128) {
                            *reinterpret_cast<uint32_t *>(stage + half * page_bytes + i) = 0u;
                            *reinterpret_cast<uint32_t *>(stage + HALF_BYTES + half * page_bytes + i) = 0u;
                        }
                    const int v = v0 + 16 * half;
                    const uint32_t mask = window_mask(p, it.n, v >= p.sink_end ? v + it.skip : v, it.tok_end - v);
                    for (int i = lane; i < 16 * NG; i += 32)
                        if (!((mask >> (i / NG)) & 1u)) {
                            uint8_t *at = stage + par_0 + half * par_half + 4 * i;
                            *reinterpret_cast<uint32_t *>(at) = 0u;
                            *reinterpret_cast<uint32_t *>(at + HALF_BYTES) = 0u;
                        }
                    hidden |= ((~mask >> row_g) & 1u) << (2 * half) | ((~mask >> (row_g + 8)) & 1u) << (2 * half + 1);
                }
                __syncwarp();
            }

            // ---- S = K Q^T: rows are tokens, columns heads; one accumulator per group.
            float sc[2][NT][2 * NC];   // of row g + 8 r and column 2 t + c at NC r + c
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint8_t *Kc = stage + half * code_half, *Kp = stage + par_0 + half * par_half;
                float acc[NT][NG][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        if (SPLIT) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
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
                            if (!SPLIT && (G == 32 || (j & 1) == 0))   // the group's first
                                mma_f16_16816(acc[nt][i], a0, qf[q][nt][j][0], qf[q][nt][j][1], 0.f);
                            else
                                mma_f16_16816(acc[nt][i], a0, qf[q][nt][j][0], qf[q][nt][j][1]);
                            mma_f16_16816(acc[nt][i], a1, qf[q][nt][j][2], qf[q][nt][j][3]);
                        }
                }
                // sc: the scores less their references
                float y[NT][4];
                if constexpr (SPLIT) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) y[nt][c] = less[nt][c];
                } else {
                    const uint8_t *at = Kp + row_g * F::PARAM_BYTES + 4 * (t & (NG - 1));
                    const uint32_t a0 = *reinterpret_cast<const uint32_t *>(at);
                    const uint32_t a1 = *reinterpret_cast<const uint32_t *>(at + 8 * F::PARAM_BYTES);
                    const uint32_t a[4] = {a0, a1, a0, a1};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(y[nt], a, qm[nt][0], qm[nt][1], less[nt]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float ks[NG], km[NG];
                    load_pairs<NG, SPLIT>(Kp + (row_g + 8 * r) * F::PARAM_BYTES, ks, km);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int col = 0; col < NC; ++col) {
                            const int c = 2 * r + col;
                            float x = ks[0] * acc[nt][0][c];
                            if constexpr (SPLIT) y[nt][c] = fmaf(km[0], qsum[nt][col][0], y[nt][c]);
#pragma unroll
                            for (int i = 1; i < NG; ++i) {
                                x = fmaf(ks[i], acc[nt][i][c], x);
                                if constexpr (SPLIT) y[nt][c] = fmaf(km[i], qsum[nt][col][i], y[nt][c]);
                            }
                            sc[half][nt][NC * r + col] = fmaf(x, qs[nt][col], y[nt][c]);
                        }
                }
            }

            if (masked) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2 * NC; ++c)
                            if ((hidden >> (2 * half + c / NC)) & 1u) sc[half][nt][c] = -INFINITY;
            }

            // ---- weights.  w = p s inv in fp16 (inv = kLift / S, S a power of two)
            // carries the value's step, so that the codes enter the second product
            // as they are.  S is the power of two above the largest p s when it was
            // chosen: from 2^7, weights may grow to 2^15 before it is chosen anew, and
            // fall by 2^21 before fp16's subnormals cost them bits.  What would pass
            // that is seen by sums, which the FMA pipe has room for: this lane's p,
            // and its w.  (Not by s alone: a token without weight may have any step.)
            float pr[2][NT][2 * NC], sw[2][2][NG];   // p, and s inv of this lane's tokens
            float sum[NT][NC], most = 0.f, ws[NG] = {}, w_sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sum[nt][0] = sum[nt][NC - 1] = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint8_t *Vp = stage + HALF_BYTES + par_0 + half * par_half;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2 * NC; ++c) {
                        pr[half][nt][c] = ex2(sc[half][nt][c]);
                        sum[nt][c % NC] += pr[half][nt][c];
                    }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float sv[NG], mv[NG], p_all = 0.f;
                    load_pairs<NG, SPLIT>(Vp + (row_g + 8 * r) * F::PARAM_BYTES, sv, mv);
                    times<!SPLIT>(sw[half][r], sv, inv);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < NC; ++c) p_all += pr[half][nt][NC * r + c];
                    add_times<!SPLIT>(ws, p_all, sw[half][r]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) most = fmaxf(most, fmaxf(sum[nt][0], sum[nt][NC - 1]));   // passes NaN over
#pragma unroll
            for (int i = 0; i < NG; ++i) w_sum += ws[i];
            const bool fresh = first && k == 0;
            if (fresh || __any_sync(kFull, most > 32.f || !(w_sum <= 0x1p15f))) {   // (or NaN: 0 times infinity)
                // Raise the references to the running maxima (a row's first unit
                // sets them), choose S anew above every p s, and take p again.  Rare
                // after the first unit.
                float alpha[NT][NC], rise[NT][NC], keep = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        float mx = fmaxf(fmaxf(sc[0][nt][c], sc[0][nt][c + NC]), fmaxf(sc[1][nt][c], sc[1][nt][c + NC]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                        // by how much; a column of NaN alone stays where it is
                        rise[nt][c] = !fresh ? fmaxf(mx, 0.f) : mx == -INFINITY ? 0.f : mx;
                        alpha[nt][c] = !fresh && less[nt][c] != -INFINITY ? ex2(-rise[nt][c]) : 0.f;
                        less[nt][c] -= rise[nt][c];
                        less[nt][c + 2] = less[nt][c];
                        l[nt][c] *= alpha[nt][c];
                        keep = fmaxf(keep, alpha[nt][c]);
#pragma unroll
                        for (int i = 0; i < NG; ++i) om[nt][c][i] *= alpha[nt][c];
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    sum[nt][0] = sum[nt][NC - 1] = 0.f;
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int c = 0; c < 2 * NC; ++c) {
                            pr[half][nt][c] = ex2(sc[half][nt][c] - rise[nt][c % NC]);
                            sum[nt][c % NC] += pr[half][nt][c];
                        }
                }
                // (the steps once more: s inv may have overflowed)
                float top[NG];
#pragma unroll
                for (int i = 0; i < NG; ++i) top[i] = 0.5f * keep * S(i);   // S is above what it was chosen for
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float most_p = 0x1p-100f, mv[NG];   // (s inv stays below 2^109)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            most_p = fmaxf(most_p, fmaxf(pr[half][nt][NC * r], pr[half][nt][NC * r + NC - 1]));
                        load_pairs<NG, SPLIT>(stage + HALF_BYTES + par_0 + half * par_half +
                                                  (row_g + 8 * r) * F::PARAM_BYTES, sw[half][r], mv);
#pragma unroll
                        for (int i = 0; i < NG; ++i) top[i] = fmaxf(top[i], most_p * sw[half][r][i]);
                    }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    float mx = top[i];
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                    const float now = pow2_above(mx), ratio = fminf(S(i) / now, 0x1p126f);   // (finite: alpha may be 0)
                    inv[i] = kLift / now;
                    fifteen[i] = 15.f / kLift * now;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        sw[half][0][i] *= inv[i];
                        sw[half][1][i] *= inv[i];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        if ((G == 64 ? mt / 4 : mt / 2) == i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int c = 0; c < 4; ++c) o[mt][nt][c] *= alpha[nt][c % NC] * ratio;   // (NC 1: column 2 t + 1 is zero)
                }
            }

#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pb[PARTS][NT][NG][2];
                float sv[2][NG], mv[2][NG];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    load_pairs<NG, SPLIT>(stage + HALF_BYTES + par_0 + half * par_half +
                                              (row_g + 8 * r) * F::PARAM_BYTES, sv[r], mv[r]);
                if constexpr (!SPLIT) add_times<true>(mv[1], fifteen, sw[half][1]);   // rows 8 to 15 count codes from 15
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (half == 0) l[nt][c] += sum[nt][c];
                        add_times<!SPLIT>(om[nt][c], pr[half][nt][c + NC], mv[1]);
                        add_times<!SPLIT>(om[nt][c], pr[half][nt][c], mv[0]);
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float wx[NG], wy[NG] = {};
                        times<!SPLIT>(wx, pr[half][nt][NC * r], sw[half][r]);
                        if (NC == 2) times<!SPLIT>(wy, pr[half][nt][NC * r + NC - 1], sw[half][r]);
#pragma unroll
                        for (int i = 0; i < NG; ++i) {
                            const float x = !SPLIT && r == 1 ? -wx[i] : wx[i], y = !SPLIT && r == 1 ? -wy[i] : wy[i];
                            const uint32_t h = pack_f16(x, y);
                            pb[0][nt][i][r] = movmatrix_trans(h);
                            if constexpr (SPLIT) {
                                const float2 b = unpack_f16(h);
                                pb[PARTS - 1][nt][i][r] = movmatrix_trans(pack_f16((x - b.x) * kPart, (y - b.y) * kPart));
                            }
                        }
                    }
                }

                // ---- O += V^T W: rows are values, k is the tokens.
                const uint8_t *va = stage + HALF_BYTES + half * code_half + g * 4 * W;
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
                        codes_or_bytes_f16<SPLIT, false>(__byte_perm(x[0][wd], x[1][wd], sel), y);
                        codes_or_bytes_f16<SPLIT, true>(__byte_perm(x[2][wd], x[3][wd], sel), z);
                        const int i = G == 64 ? wd : 2 * wd + hf;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t a[4] = {y[2 * e], y[2 * e + 1], z[2 * e], z[2 * e + 1]};
                            const int mt = 4 * wd + 2 * hf + e;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
{
                                    if constexpr (SPLIT) {
                                        float d[4], rest[4];
                                        mma_f16_16816(d, a, pb[0][nt][i][0], pb[0][nt][i][1], 0.f);
                                        mma_f16_16816(rest, a, pb[PARTS - 1][nt][i][0], pb[PARTS - 1][nt][i][1], 0.f);
#pragma unroll
                                        for (int c = 0; c < 4; ++c) o[mt][nt][c] += fmaf(rest[c], 1.f / kPart, d[c]);
                                    } else {
                                        mma_f16_16816(o[mt][nt], a, pb[0][nt][i][0], pb[0][nt][i][1]);
                                    }
                                }
                        }
                    }
            }
            __syncwarp();
            if (asked < units)
                issue(page_a, page_b, asked++);
            else if (asked_next < next_units)
                issue(next_a, next_b, asked_next++);
        }

        const bool hold = !it.last && it.index % kHoldBlocks == kHoldBlocks - 1;
        if (it.index >= kHoldBlocks && (hold || it.last)) {
            // what the held sums' references and scales were then, against now
            float f[NT][NC], ratio[NG];
            int j = HELD;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < NC; ++c) f[nt][c] = ex2(less[nt][c] - held[32 * j++]);
#pragma unroll
            for (int i = 0; i < NG; ++i) ratio[i] = fminf(held[32 * j++] / S(i), 0x1p126f);   // (finite: f may be 0)
            each_sum([&](float &sum, int j, int nt, int c, int i) {
                sum = fmaf(held[32 * j], i < 0 ? f[nt][c] : f[nt][c] * ratio[i], sum);
            });
        }
        if (hold) {
            int j = HELD;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < NC; ++c) held[32 * j++] = less[nt][c];
#pragma unroll
            for (int i = 0; i < NG; ++i) held[32 * j++] = S(i);
            each_sum([&](float &sum, int j, int, int, int) {
                held[32 * j] = sum;
                sum = 0.f;
            });
        }

        // Undo the scalings, add the minima's part, and store: the final rows,
        // or the row's partial.
        if (it.last) {
        const bool whole = it.whole;
        const long long out0 = (long long)it.seq * p.num_q_heads + it.qh0;
        const long long part0 = ((blockIdx.x * kQ4Warps + warp) * 2ll + it.begins) * ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[nt][c] += __shfl_xor_sync(kFull, l[nt][c], d);
#pragma unroll
                    for (int i = 0; i < NG; ++i) om[nt][c][i] += __shfl_xor_sync(kFull, om[nt][c][i], d);
                }
                const int head = 8 * nt + NC * t + c;
                if (head >= it.rows) continue;
                // a row without a token has l = 0 and zero sums; NaN stays NaN
                const float norm = !whole ? 1.f : l[nt][c] == 0.f ? 0.f : 1.f / l[nt][c];
#pragma unroll
                for (int m2 = 0; m2 < MT / 2; ++m2) {   // a unit of four values: m-tiles 2 m2 and 2 m2 + 1
                    const int u = 16 * (m2 / 2) + 8 * (m2 % 2) + g;
                    const int i = G == 64 ? m2 / 2 : m2;
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float *acc = o[2 * m2 + e][nt];
                        y[2 * e] = fmaf(acc[c] * ((SPLIT ? 1.f : 0x1p24f) / kLift), S(i), om[nt][c][i]) * norm;
                        const float odd = SPLIT ? acc[c + 2] / kLift : (acc[c + 2] - acc[c]) * (0x1p20f / kLift);
                        y[2 * e + 1] = fmaf(odd, S(i), om[nt][c][i]) * norm;
                    }
                    const float4 v = make_float4(y[0], y[1], y[2], y[3]);
                    if (whole)
                        store4(static_cast<T *>(p.out) + (out0 + head) * HD + 4 * u, v);
                    else
                        store4(split.acc + (part0 + head) * HD + 4 * u, v);
                }
                if (!whole && g == 0)
                    *reinterpret_cast<float2 *>(split.ml + (part0 + head) * 2) = make_float2(-less[nt][c], l[nt][c]);
            }
        }   // last
        slot ^= 1;
        units = next_units;
        page_a = next_a;
        page_b = next_b;
        asked = asked_next;
        asked_next = 0;
    }
    griddep_launch_dependents();
}

// Joins the partials of every row that stretches cut.  out = sum_i 2^(m_i - M)
// acc_i / sum_i 2^(m_i - M) l_i.  PER warps per (sequence, query head).
constexpr int kJoinWarps = 4;

// A warp takes 8 partials at a time.  Where there are more for a row, four warps
// share them: the whole call takes 138.4 us rather than 141.6 on 7 sequences of up
// to 131072 tokens, 50.0 rather than 50.9 on 32 lognormal ones, 8.4 rather than 8.9
// on one of 777.  Not where there are fewer (64 sequences, GQA 32/8: 134.4 against
// 132.3) or rows enough to fill the GPU (64 sequences, GQA 64/4: 73.3 against 68.9).
bool join_by_four(long long stretches, long long rows, long long head_rows, int sms) {
    return stretches >= 8 * rows && head_rows <= 14ll * sms;
}

template <typename T, int HD, int PER>
__global__ void __launch_bounds__(kJoinWarps * 32) join_q4_kernel(const DecodeParams p, const Q4Split split, int rows) {
    static_assert(PER == 1 || PER == kJoinWarps);
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = PER == 1 ? 0 : warp;
    // (rows are counted in 31 bits, and partials' values too: kMaxStretches of them)
    const uint32_t me = PER == 1 ? blockIdx.x * kJoinWarps + warp : blockIdx.x;
    const uint32_t seq = me / static_cast<uint32_t>(p.num_q_heads), qh = me - seq * p.num_q_heads;
    if (seq >= static_cast<uint32_t>(p.num_seqs)) return;
    const uint32_t share = max(1u, *split.share), ru = row_units(seq_view<true>(p, seq).seen);
    const uint32_t kvh = qh / static_cast<uint32_t>(p.group), in_group = qh - kvh * p.group;
    const uint32_t ht = in_group / static_cast<uint32_t>(rows), r = in_group - ht * rows;
    const uint32_t begin = split.bases[seq] + (kvh * p.head_tiles + ht) * (ru + kRowCost) + kRowCost;
    const uint32_t w0 = begin / share, w1 = (begin + ru - 1) / share;
    // Equal: stored whole.  Past the room, or reversed: no pass has written the bases.
    if (w0 >= w1 || w1 >= split.stretches) return;
    const int parts = static_cast<int>(w1 - w0) + 1;
    // the stretch that begins the row keeps it in its second slot, the others in their first
    auto at = [&](int i) { return ((w0 + i) * 2 + (i == 0)) * rows + r; };
    constexpr int E = HD / 32;   // values per lane
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    // Partials on their way at a time (registers for 16 halve the warps per SM:
    // 256 sequences' 16384 rows 9.4 us against 7.2; 4 lengthen the longest rows).
    constexpr int FETCH = 8;
    float M = -INFINITY, L = 0.f;
    float acc[E] = {};
    for (int i0 = FETCH * mine; i0 < parts; i0 += FETCH * PER) {
        const int n = min(FETCH, parts - i0);
        const float2 ml = lane < n ? *reinterpret_cast<const float2 *>(split.ml + at(i0 + lane) * 2)
                                   : make_float2(-INFINITY, 0.f);
        Vec v[FETCH];
#pragma unroll
        for (int i = 0; i < FETCH; ++i)
            if (i < n) v[i] = *reinterpret_cast<const Vec *>(split.acc + at(i0 + i) * HD + lane * E);
        float top = ml.x;
#pragma unroll
        for (int o = 1; o < FETCH; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        top = __shfl_sync(kFull, top, 0);
        const float now = fmaxf(M, top), alpha = exp2f(M - now);   // the first M is -inf: alpha 0
        M = now;
        const float f = lane < n ? exp2f(ml.x - now) : 0.f;
        L = L * alpha + f * ml.y;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= alpha;
#pragma unroll
        for (int i = 0; i < FETCH; ++i) {
            if (i >= n) break;
            const float w = __shfl_sync(kFull, f, i);
            acc[0] = fmaf(w, v[i].x, acc[0]);
            acc[1] = fmaf(w, v[i].y, acc[1]);
            if constexpr (E == 4) {
                acc[E - 2] = fmaf(w, v[i].z, acc[E - 2]);
                acc[E - 1] = fmaf(w, v[i].w, acc[E - 1]);
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) L += __shfl_xor_sync(kFull, L, o);
    if constexpr (PER > 1) {   // the warps' sums, in their order (one without a partial has M = -inf and zeros)
        __shared__ float s_m[PER], s_l[PER];
        __shared__ Vec s_acc[PER][32];
        if (lane == 0) {
            s_m[warp] = M;
            s_l[warp] = L;
        }
        if constexpr (E == 4) s_acc[warp][lane] = make_float4(acc[0], acc[1], acc[E - 2], acc[E - 1]);
        else s_acc[warp][lane] = make_float2(acc[0], acc[1]);
        __syncthreads();
        if (warp != 0) return;
        float f[PER];
#pragma unroll
        for (int w = 1; w < PER; ++w) M = fmaxf(M, s_m[w]);
        L = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < PER; ++w) {
            f[w] = exp2f(s_m[w] - M);
            L = fmaf(f[w], s_l[w], L);
            const Vec v = s_acc[w][lane];
            acc[0] = fmaf(f[w], v.x, acc[0]);
            acc[1] = fmaf(f[w], v.y, acc[1]);
            if constexpr (E == 4) {
                acc[E - 2] = fmaf(f[w], v.z, acc[E - 2]);
                acc[E - 1] = fmaf(f[w], v.w, acc[E - 1]);
            }
        }
    }
    const float norm = L == 0.f ? 0.f : 1.f / L;
    T *to = static_cast<T *>(p.out) + static_cast<size_t>(me) * HD + lane * E;
    if constexpr (E == 4) {
        store4(to, make_float4(acc[0] * norm, acc[1] * norm, acc[E - 2] * norm, acc[E - 1] * norm));
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2 *>(to) = make_float2(acc[0] * norm, acc[1] * norm);
    } else {
        *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(acc[0] * norm, acc[1] * norm);
    }
}

using namespace host;

// Warps of the partition pass at most: the stretches that a workspace has room
// for (152 SMs x 16).
constexpr long long kMaxStretches = 2432;

// Stretches of a call, at most: rows of up to walk_cap tokens, cut no finer
// than P tokens.  1 or less: nothing is cut.
long long stretches(int num_seqs, long long heads, int walk_cap, int P) {
    if (walk_cap <= P) return 0;
    const long long units = static_cast<long long>(num_seqs) * heads * ((walk_cap + static_cast<long long>(kUnit) - 1) / kUnit);
    const long long n = (units + P / kUnit - 1) / (P / kUnit);
    return n < kMaxStretches ? n : kMaxStretches;
}

struct Q4Launch {
    const void *k_cache, *v_cache;
    Q4Split split;
    long long stretches;   // 0: rows are not cut
    int min_share, dev, phase;
    cudaStream_t stream;
};

template <typename T, int HD, int G, int NT, int NC, int bs>
int launch_one(const DecodeParams &p, const Q4Launch &c) {
    const long long rows = static_cast<long long>(p.num_seqs) * p.num_kv_heads * p.head_tiles;
    if (c.phase != PA_PHASE_REDUCE) {
        constexpr int NS = Q4Shape<HD, NT, sizeof(T) == 4>::NSTAGE;
        constexpr int SMEM = kQ4Warps * (NS * 2 * kUnit * Q4Format<HD, G>::ROW_BYTES + 128 * q4_held_all<HD, G, NT, NC>());
        static KernelSlot slot;
        auto kernel = decode_q4_kernel<T, HD, G, NT, NC, bs>;
        const int occ = ensure_kernel(kernel, slot, SMEM, c.dev, kQ4Warps * 32);
        if (occ == 0) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: cannot configure the kernel");
        long long warps = static_cast<long long>(sm_count(c.dev)) * occ * kQ4Warps;
        if (warps > kMaxStretches) warps = kMaxStretches;
        const long long most = c.stretches ? c.stretches : rows;
        if (warps > most) warps = most;
        const cudaError_t e = launch_dependent(kernel, static_cast<int>((warps + kQ4Warps - 1) / kQ4Warps),
                                               kQ4Warps * 32, SMEM, c.stream, static_cast<const uint8_t *>(c.k_cache),
                                               static_cast<const uint8_t *>(c.v_cache), p, c.split, static_cast<uint32_t>(warps),
                                               static_cast<uint32_t>(c.min_share));
        if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    }
    if (c.stretches && c.phase != PA_PHASE_PARTITIONS) {
        const long long all = static_cast<long long>(p.num_seqs) * p.num_q_heads;
        const bool four = join_by_four(c.stretches, rows, all, sm_count(c.dev));
        const long long ctas = four ? all : (all + kJoinWarps - 1) / kJoinWarps;
        const cudaError_t e = launch_dependent(four ? join_q4_kernel<T, HD, kJoinWarps> : join_q4_kernel<T, HD, 1>,
                                               static_cast<int>(ctas), kJoinWarps * 32, 0, c.stream, p, c.split,
                                               4 * NC * NT);
        if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    }
    return PA_OK;
}

template <typename T, int HD, int G, int bs>
int launch_tile(const DecodeParams &p, const Q4Launch &c) {
    if (p.group > 8) return launch_one<T, HD, G, 2, 2, bs>(p, c);
    return p.group > 4 ? launch_one<T, HD, G, 1, 2, bs>(p, c) : launch_one<T, HD, G, 1, 1, bs>(p, c);
}

template <typename T, int HD, int G>
int launch_block(const DecodeParams &p, const Q4Launch &c) {
    return p.block_size == 32 ? launch_tile<T, HD, G, 32>(p, c) : launch_tile<T, HD, G, 16>(p, c);
}

template <typename T>
int launch_any(const DecodeParams &p, const Q4Launch &c, int head_dim, int group_size) {
    if (head_dim == 128) return group_size == 64 ? launch_block<T, 128, 64>(p, c) : launch_block<T, 128, 32>(p, c);
    return group_size == 64 ? launch_block<T, 64, 64>(p, c) : launch_block<T, 64, 32>(p, c);
}

// Contexts of up to so many tokens are not split, others no finer.  Splitting
// costs the join (about 2 us) and is worth it where rows alone do not fill the
// GPU: of 8 x 300 tokens P = 64 takes 8.9 us, unsplit 12.1; of 512 x 300, 16.2
// and 12.7; of 8 x 100, 9.4 and 7.2; of 512 x 1000, 25 and 31.  (Between 8 and 512
// rows nothing was measured: where in between they cross is not known.)
int q4_partition(int partition_size, long long rows, int walk_cap) {
    if (partition_size != 0) return partition_size;
    return walk_cap <= 128 ? 128 : rows >= 512 && walk_cap <= 512 ? 512 : 64;
}

// Query heads per row: half a tile's columns, a tile, or two for larger groups.
int q4_tile(int group) { return group > 8 ? 16 : group > 4 ? 8 : 4; }

// Workspace: [header: the units per warp at byte 16] [first unit of each
// sequence] [(max, sum)] [accumulators], two rows of heads per stretch.
size_t workspace_bytes(int num_seqs, int tile, int head_dim, long long n, size_t *ml_at, size_t *acc_at) {
    if (n == 0) return 0;
    const size_t rows = static_cast<size_t>(n) * 2 * tile;
    *ml_at = kWorkspaceHeader + align256(static_cast<size_t>(num_seqs) * sizeof(uint32_t));
    *acc_at = *ml_at + align256(rows * 2 * sizeof(float));
    return *acc_at + align256(rows * head_dim * sizeof(float));
}

// A window's edges are rounded to whole blocks (so that a page is walked or
// left out as one); for sizing a workspace, to the largest.
constexpr int kQ4MaxBlock = 32;

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_q4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                              int max_context_len, int partition_size, int window, int num_sinks) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || head_dim <= 0 ||
        max_context_len <= 0 || window < 0 || num_sinks < 0 || (partition_size != 0 && partition_size < pa::kUnit))
        return 0;
    const int group = num_q_heads / num_kv_heads, tile = pa::q4_tile(group);
    const long long heads = static_cast<long long>(num_kv_heads) * ((group + tile - 1) / tile);
    const int walk = pa::host::seen_cap(max_context_len, window, num_sinks, pa::kQ4MaxBlock);
    const int P = pa::q4_partition(partition_size, num_seqs * heads, walk);
    size_t ml_at, acc_at;
    return pa::workspace_bytes(num_seqs, tile, head_dim, pa::stretches(num_seqs, heads, walk, P), &ml_at, &acc_at);
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
    if (a->partition_size != 0 && (a->partition_size < 32 || a->partition_size > 1024 || a->partition_size % 32 != 0))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: partition_size must be a multiple of 32 in [32, 1024]");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return pa_fail(PA_ERR_INVALID_ARG, "pa_decode_q4: out, q and caches must be 16-byte aligned");

    const long long table_cap = static_cast<long long>(a->max_blocks_per_seq) * block_size;
    const int ctx_cap = static_cast<int>(a->max_context_len < table_cap ? a->max_context_len : table_cap);
    // The walk the workspace is sized for, which also picks the split.
    const int sized_walk = seen_cap(a->max_context_len, window, num_sinks, pa::kQ4MaxBlock);
    // No window is one that no sequence outgrows; sinks past the end change nothing.
    if (window == 0 || window > ctx_cap) window = ctx_cap > 0 ? ctx_cap : 1;
    if (num_sinks > ctx_cap) num_sinks = ctx_cap;
    const int walk_cap = seen_cap(ctx_cap, window, num_sinks, block_size);
    pa::DecodeParams p{};
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
    p.ctx_cap = ctx_cap;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.window = window;
    p.num_sinks = num_sinks;
    p.view_gran = block_size;
    // pages are counted in 31 bits
    if (static_cast<long long>(a->num_blocks) * num_kv_heads >= INT_MAX)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_q4: cache has 2^31 or more pages");
    p.sink_end = round_up_int(num_sinks, block_size);
    const int tile = pa::q4_tile(p.group);
    p.tile_rows = p.group < tile ? p.group : tile;
    p.head_tiles = (p.group + tile - 1) / tile;
    // units are counted in 31 bits, and the join's CTAs too
    const long long heads = static_cast<long long>(num_kv_heads) * p.head_tiles;
    if (static_cast<long long>(a->num_seqs) * heads * (walk_cap / pa::kUnit + 1ll + pa::kRowCost) >= INT_MAX ||
        static_cast<long long>(a->num_seqs) * num_q_heads >= INT_MAX)
        return pa_fail(PA_ERR_UNSUPPORTED, "pa_decode_q4: 2^31 or more units of 32 tokens");
    const int P = pa::q4_partition(a->partition_size, a->num_seqs * heads, sized_walk);
    pa::Q4Launch c{k_cache, v_cache, {}, pa::stretches(a->num_seqs, heads, walk_cap, P), P / pa::kUnit, 0, a->phase,
                   static_cast<cudaStream_t>(a->stream)};
    if (c.stretches) {
        size_t ml_at, acc_at;
        const size_t need = pa::workspace_bytes(a->num_seqs, tile, head_dim, c.stretches, &ml_at, &acc_at);
        if (!a->workspace || a->workspace_bytes < need || !aligned16(a->workspace))
            return pa_fail(PA_ERR_WORKSPACE, "pa_decode_q4: workspace missing, unaligned or smaller than "
                                             "pa_decode_q4_workspace_size()");
        char *ws = static_cast<char *>(a->workspace);
        c.split = {reinterpret_cast<uint32_t *>(ws + 16), reinterpret_cast<uint32_t *>(ws + kWorkspaceHeader),
                   reinterpret_cast<float *>(ws + ml_at), reinterpret_cast<float *>(ws + acc_at),
                   static_cast<uint32_t>(c.stretches)};
    }
    if (cudaGetDevice(&c.dev) != cudaSuccess) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: no CUDA device");
    if (sm_count(c.dev) <= 0) return pa_fail(PA_ERR_CUDA, "pa_decode_q4: cannot query the SM count");
    const int rc = a->dtype == PA_F32 ? pa::launch_any<float>(p, c, head_dim, group_size)
                                      : pa::launch_any<__nv_bfloat16>(p, c, head_dim, group_size);
    if (rc != PA_OK) return rc;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return pa_fail(PA_ERR_CUDA, cudaGetErrorString(e));
    return PA_OK;
}
