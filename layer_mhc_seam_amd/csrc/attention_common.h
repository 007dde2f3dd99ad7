// attention_common.h -- what the two kernels of attention over the 4-bit cache
// share: the softmax's constants, where a row block lies, what a row sees, NaN
// that only some rows of a step see.
#pragma once

#include <hip/hip_runtime.h>

#include "cache_layout.h"
#include "half_ops.h"
#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.44269504089f;
constexpr float kLn2 = 0.69314718056f;

template <int DT> struct Softmax;
// exp(s - max) is kept times 2^kShift: fp16's smallest number is 2^-24
template <> struct Softmax<MHC_BF16> {
    static constexpr float kShift = 0.0f, kSlack = 8.0f;
};
template <> struct Softmax<MHC_F16> {
    static constexpr float kShift = 12.0f, kSlack = 3.0f;
};

// Over the lanes of equal c = l % 16, the same value in each
__device__ __forceinline__ float max_over_groups(float v)
{
    u32 x = __float_as_uint(v);
    auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    x = __float_as_uint(v);
    auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

__device__ __forceinline__ float sum_over_groups(float v)
{
    u32 x = __float_as_uint(v);
    auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    x = __float_as_uint(v);
    auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

__device__ __forceinline__ u32 or_over_groups(u32 x)
{
    auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = p[0] | p[1];
    auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return q[0] | q[1];
}

// Lengths, starts and tables, which no kernel writes: where the index is the
// wave's, it and what follows from it stay in scalar registers
typedef const __attribute__((address_space(4))) int32_t *Whole;

__device__ __forceinline__ Whole whole(const int32_t *p) { return (Whole)(uintptr_t)p; }

// Tokens [lo, hi) that query row i of n, the last of len tokens, sees
__device__ __forceinline__ void row_sees(const AttentionParams &P, int len, int n, int i, int *lo, int *hi)
{
    const int p = len - n + i;       // -2^31 < p < len < 2^31
    *hi = P.causal ? max(p + 1, 0) : len;
    *lo = P.window > 0 ? max(max(p, -1) + 1 - P.window, 0) : 0;
}

// First query row of sequence b, and past the last of b - 1
__device__ __forceinline__ int row_start(const AttentionParams &P, int b)
{
    return P.q_starts ? min(max(whole(P.q_starts)[b], 0), (int)P.T) : b;
}

__device__ __forceinline__ int length_of(const AttentionParams &P, int b)
{
    return (int)min((int64_t)max(whole(P.lens)[b], 0), P.max_len);
}

// Row blocks of `rows` rows: those of sequence b have the numbers from
// first_number on, of which there may be more than it has blocks.  Rows times
// heads of a kv head number below 2^31, and so do these.
__device__ __forceinline__ int first_number(const AttentionParams &P, int b, int start, int rows)
{
    return P.q_starts ? start * P.group / rows + b : b * ((P.group + rows - 1) / rows);
}

// The sequence that number `id` is one of, and its first number
__device__ __forceinline__ int sequence_of(const AttentionParams &P, int id, int rows, int *first)
{
    int low = 0, high = P.B;
    if (!P.q_starts) {
        low = id / ((P.group + rows - 1) / rows);
    } else {
        while (high - low > 1) {
            const int mid = (low + high) / 2;
            if (first_number(P, mid, row_start(P, mid), rows) <= id)
                low = mid;
            else
                high = mid;
        }
    }
    *first = first_number(P, low, row_start(P, low), rows);
    return low;
}

// How many numbers T rows in B sequences take
inline int64_t most_blocks(int64_t T, int B, int group, int rows, bool ragged)
{
    return ragged ? T * group / rows + B : (int64_t)B * ((group + rows - 1) / rows);
}

// Sum of v over the lanes up to this one: inside rows of 16, then over the rows
__device__ __forceinline__ int sum_upto(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // lanes 1, 2, 4, 8 before
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // lane 15 to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // lane 31 to the last two
    return v;
}

// Sum over the lanes of v, not negative and below 2^48
__device__ __forceinline__ int64_t sum_of_lanes(int64_t v)
{
    const int low = (int)read_lane((u32)sum_upto((int)(v & 0xffffff)), 63);
    return ((int64_t)(int)read_lane((u32)sum_upto((int)(v >> 24)), 63) << 24) + low;
}

// Which groups of 32 channels of a token's values are NaN, by their scales.  The
// token is there.
template <int D>
__device__ u32 nan_groups(const AttentionParams &P, Whole table, int32_t t, int head)
{
    int32_t page, at;
    if (!cache_page(P.c, table, t + 1, t / kCacheTile * kCacheTile, &page, &at))
        return 0;
    const uint8_t *vs = P.cache + cache_page_near(P.c, page, head, D) + cache_scales(P.c.page_size, D, 1) + at +
                        t % kCacheTile;
    u32 bits = 0;
    for (int j = 0; j < D / 32; ++j)
        bits |= (u32)(vs[j * P.c.page_size] == 255) << j;
    return bits;
}

// A page of a head, its loads by a lane's offset plus the wave's: the lanes'
// offsets stay as they are from page to page.  The long loads, of whole lines
// that nobody asks for again, go past the caches: a cache of 520 MB then reads
// at 5.9 TB/s for 4.7, and one that the last level holds no slower.  Short ones
// that share lines go through them (with all loads past them: 5.0).
struct Page {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ u32 load32(u32 lane, int wave) const
    {
        return __builtin_amdgcn_raw_buffer_load_b32(r, lane, wave, 0);
    }
    __device__ __forceinline__ u32x2 load64(u32 lane, int wave) const
    {
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, lane, wave, 0));
    }
    __device__ __forceinline__ u32x4 load128(u32 lane, int wave) const
    {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, wave, 2));
    }
    // the same through the caches, for what other workgroups read too
    __device__ __forceinline__ u32x4 load128_again(u32 lane, int wave) const
    {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane, wave, 0));
    }
};

template <int D> __device__ __forceinline__ Page page_of(const AttentionParams &P, int page, int head)
{
    const uint8_t *base = P.cache + cache_page_near(P.c, page, head, D);
    return {__builtin_amdgcn_make_buffer_rsrc((void *)base, 0, (int)cache_page_bytes(P.c.page_size, D), 0x00027000)};
}

// How scores are capped: not at all, by a cap up to kLowCap, by a higher one
enum Cap { kNoCap = 0, kLow = 1, kHigh = 2 };
constexpr float kLowCap = 64.0f;

inline Cap cap_of(float softcap) { return softcap == 0.0f ? kNoCap : softcap <= kLowCap ? kLow : kHigh; }

// N products q . k capped: their scores in base 2, c tanh(x) with x = s / c.
// tanh x = 1 - 2 / (exp 2|x| + 1), its sign x's, is off by up to 2^-21 of the cap, whatever
// the score: of a low cap that is 2^-15, an eighth of the rounding that the score's
// weight gets in fp16.  Under a higher one, scores up to a quarter of it are
// s tanh(x) / x by the Taylor series of tanh to the degree 9, whose next term is
// below 2^-26 there: they are off by a part of themselves, and a cap far above the
// scores changes nothing.  The low caps' kernels are apart because that takes longer
// where a step's scores lie on both sides (2048 rows over 8192 tokens, 40 heads on 8 of
// 64, 128 and 256 channels, a cap of 5: 525, 571 and 1131 us for 393, 463 and 923).
template <int N, int CAP> __device__ __forceinline__ void cap(const AttentionParams &P, float v[N])
{
    const float in = P.scale / P.softcap, f = P.scale * kLog2e, out = P.softcap * kLog2e, near = 0.25f;
    auto far = [&](float s) {
        const float e = __builtin_amdgcn_exp2f(fabsf(s * in) * (2.0f * kLog2e));
        return copysignf(out - 2.0f * out * __builtin_amdgcn_rcpf(e + 1.0f), s * in);
    };
    auto series = [&](float s) {
        const float x = s * in, t = x * x;
        float r = fmaf(t, 62.0f / 2835, -17.0f / 315);
        r = fmaf(t, r, 2.0f / 15);
        r = fmaf(t, r, -1.0f / 3);
        return s * f * fmaf(t, r, 1.0f);
    };
    if constexpr (CAP == kHigh) {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            most = fmaxf(most, fabsf(v[i]));
        if (!__any(most * fabsf(in) > near)) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = series(v[i]);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = CAP == kHigh && fabsf(v[i] * in) <= near ? series(v[i]) : far(v[i]);
}

}  // namespace
}  // namespace mhc
