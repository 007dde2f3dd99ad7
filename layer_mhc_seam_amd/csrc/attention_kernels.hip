// attention_kernels.hip -- attention over the 4-bit cache.
//
// One pass over the cache with a running maximum and sum.  A wave takes 32
// tokens a step, in registers from memory to the result:
//   S^T = K Q^T   v_mfma 16x16x32: lane (c, g), c = l % 16, g = l / 16, holds token
//                 c of a half of 16 and channels [g D/4, (g + 1) D/4), as does Q's
//                 lane of row c; gfx950 turns two codes into two values at once.
//                 The result's lane holds row c and tokens 4g .. 4g + 3.
//   softmax       in that lane, base 2.  The maximum moves only when a score
//                 passes it by kSlack, so most steps exchange nothing.
//   O^T += V^T P^T  P is the operand as it stands: its eight numbers are tokens
//                 4g .. 4g + 3 of both halves, and V's lane loads those tokens'
//                 D/16 channels from c D/16 on.  The order of tokens and of
//                 channels inside a product is free.
// The values' pairs of channels become pairs of tokens by two byte permutes.
#include <hip/hip_runtime.h>

#include "cache_layout.h"
#include "half_ops.h"
#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

constexpr int kRows = 16;                 // query rows a block: heads of one kv head, tokens in order
constexpr int kStep = 32;                 // tokens a wave's step
constexpr int kAttnWaves = 4;
constexpr int kQuantum = kStep * kAttnWaves;   // tokens that a workgroup's waves take side by side
constexpr int kMostBalanced = 1024;       // sequences whose lengths a worker adds up
constexpr int kLeastQuanta = 2;           // of a worker's share
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

// A sequence's share of the work: blocks of rows, and the quanta of tokens that
// some row of it sees, the same number for every block and kv head.
struct Sequence {
    int64_t first;      // its first query row
    int64_t rows;       // query rows times heads of a kv head
    int64_t n;          // query rows
    int64_t len;        // cached tokens
    int64_t lo;         // first quantum's first token
    int64_t blocks;     // of kRows rows
    int64_t quanta;
};

__device__ __forceinline__ Sequence sequence(const AttentionParams &P, int b)
{
    Sequence s;
    int64_t from = b, to = b + 1;
    if (P.q_starts) {
        from = min((int64_t)max(P.q_starts[b], 0), P.T);
        to = min((int64_t)max(P.q_starts[b + 1], 0), P.T);
    }
    s.first = from;
    s.n = max(to - from, (int64_t)0);
    s.rows = s.n * P.group;
    s.len = min((int64_t)max(P.lens[b], 0), P.max_len);
    s.lo = P.window > 0 ? max(s.len - s.n + 1 - P.window, (int64_t)0) / kStep * kStep : 0;
    s.blocks = (s.rows + kRows - 1) / kRows;
    s.quanta = max((s.len - s.lo + kQuantum - 1) / kQuantum, (int64_t)1);
    return s;
}

__device__ __forceinline__ int64_t wave_total(int64_t v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const u64 x = (u64)v;
        const u32 lo = __shfl_xor((u32)x, d), hi = __shfl_xor((u32)(x >> 32), d);
        v += (int64_t)((u64)hi << 32 | lo);
    }
    const u32 lo = read_lane((u32)(u64)v, 0), hi = read_lane((u32)((u64)v >> 32), 0);
    return (int64_t)((u64)hi << 32 | lo);
}

// All quanta of the batch: of each sequence blocks * kv heads * quanta, in that
// order of sequences, kv heads, blocks.
__device__ int64_t all_quanta(const AttentionParams &P)
{
    int64_t mine = 0;
    for (int b = threadIdx.x & 63; b < P.B; b += 64) {
        const Sequence s = sequence(P, b);
        mine += s.blocks * s.quanta;
    }
    return wave_total(mine) * P.c.heads;
}

// Sequence that quantum `at` (below the total) belongs to, and the first quantum of it
__device__ int find_sequence(const AttentionParams &P, int64_t at, int64_t *start)
{
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int b0 = 0; b0 < P.B; b0 += 64) {
        int64_t mine = 0;
        if (b0 + lane < P.B) {
            const Sequence s = sequence(P, b0 + lane);
            mine = s.blocks * s.quanta * P.c.heads;
        }
        int64_t upto = mine;             // sum over lanes 0 .. lane
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const u64 x = (u64)upto;
            const u32 lo = __shfl_up((u32)x, d), hi = __shfl_up((u32)(x >> 32), d);
            if (lane >= d)
                upto += (int64_t)((u64)hi << 32 | lo);
        }
        const u64 past = __ballot(before + upto > at);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            const int64_t first = before + upto - mine;
            const u32 lo = read_lane((u32)(u64)first, l), hi = read_lane((u32)((u64)first >> 32), l);
            *start = (int64_t)((u64)hi << 32 | lo);
            return b0 + l;
        }
        const u32 lo = read_lane((u32)(u64)upto, 63), hi = read_lane((u32)((u64)upto >> 32), 63);
        before += (int64_t)((u64)hi << 32 | lo);
    }
    *start = before;
    return P.B;
}

__device__ __forceinline__ int64_t share_start(int64_t total, int64_t workers, int64_t w)
{
    return total * w / workers;          // total < 2^40, workers < 2^13
}

__device__ __forceinline__ int64_t workers_for(int64_t total, int64_t most)
{
    return max(min((total + kLeastQuanta - 1) / kLeastQuanta, most), (int64_t)1);
}

// A partial result: kRows maxima, kRows sums, [kRows][D] weighted values.  A
// worker's share leaves at most two: of its first and of its last block.
template <int D> __device__ __forceinline__ float *record(const AttentionParams &P, int64_t worker, bool first)
{
    return P.workspace + (2 * worker + (first ? 0 : 1)) * (int64_t)(kRows * (D + 2));
}

template <int D> struct Tile {
    u32 k[2][D / 32];
    u32 ks[2][(D + 127) / 128];
    u32 v[8][(D + 127) / 128];
    u32 vs[2];
};

// The rows of a block as a lane of row c sees them
struct Rows {
    int64_t lo, hi;          // tokens that the lane's row sees
    int64_t most_lo, least_hi;   // that every row of the block sees
};

template <int DT, int D> struct Attention {
    typedef Half<DT> H;
    typedef Softmax<DT> S;
    static constexpr int KC = D / 32;        // products of a score: 8 channels a lane each
    static constexpr int VC = D / 16;        // channels of V a lane
    static constexpr int VB = VC / 2;        // bytes of them

    const AttentionParams &P;
    const int lane, c, g;
    u32x4 q[KC];
    f32x4 acc[VC];
    float top, sum;
    u32 nans;                // groups of V's channels that a NaN reaches in this lane's row

    __device__ Attention(const AttentionParams &p)
        : P(p), lane(threadIdx.x & 63), c(lane & 15), g(lane >> 4)
    {
    }

    __device__ void load_q(const Sequence &s, int64_t block, int head)
    {
        const int64_t r = block * kRows + c;
        const int64_t i = r / P.group;
        if (r < s.rows) {
            const uint16_t *at = P.q + (s.first + i) * P.q_token + (head * P.group + (r - i * P.group)) * P.q_head;
#pragma unroll
            for (int j = 0; j < KC; ++j)
                q[j] = *(const u32x4 *)(at + g * (D / 4) + j * 8);
        } else {
#pragma unroll
            for (int j = 0; j < KC; ++j)
                q[j] = u32x4{0, 0, 0, 0};
        }
    }

    __device__ Rows rows_of(const Sequence &s, int64_t block)
    {
        auto bounds = [&](int64_t r, int64_t *lo, int64_t *hi) {
            const int64_t p = s.len - s.n + r / P.group;
            *hi = P.causal ? max(min(p + 1, s.len), (int64_t)0) : s.len;
            *lo = P.window > 0 ? max(p + 1 - P.window, (int64_t)0) : 0;
        };
        Rows w;
        const int64_t first = block * kRows, last = min(first + kRows, s.rows) - 1;
        int64_t skip;
        bounds(first, &skip, &w.least_hi);
        bounds(last, &w.most_lo, &skip);
        if (first + c <= last)
            bounds(first + c, &w.lo, &w.hi);
        else
            w.lo = w.hi = 0;
        return w;
    }

    // Half h of the tile at t: page and place, or page 0, which no token of it is read from
    __device__ bool place(const int32_t *table, int64_t len, int64_t t, int64_t *page, int32_t *at)
    {
        const bool there = cache_tile(P.c, table, len, t, page, at);
        if (!there) {
            *page = 0;
            *at = 0;
        }
        return there;
    }

    __device__ void load(Tile<D> &x, bool there[2], const int32_t *table, int64_t len, int64_t t, int head)
    {
        const int ps = P.c.page_size;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int64_t page;
            int32_t at;
            there[h] = place(table, len, t + 16 * h, &page, &at);
            const uint8_t *base = P.cache + cache_page_at(P.c, page, head, D);
            const uint8_t *kc = base + (u32)((at + c) * (D / 2) + g * (D / 8));
            if constexpr (D == 64) {
                const u32x2 w = *(const u32x2 *)kc;
                x.k[h][0] = w[0];
                x.k[h][1] = w[1];
            } else {
#pragma unroll
                for (int j = 0; j < KC / 4; ++j) {
                    const u32x4 w = *(const u32x4 *)(kc + 16 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x.k[h][4 * j + i] = w[i];
                }
            }
            const uint8_t *ks = base + cache_scales(ps, D, 0) + (u32)(g * D / 128 * ps + at + c);
#pragma unroll
            for (int j = 0; j < (D + 127) / 128; ++j)
                x.ks[h][j] = ks[j * ps];
            const uint8_t *vc = base + cache_codes(ps, D, 1) + (u32)((at + 4 * g) * (D / 2) + c * VB);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint8_t *from = vc + j * (D / 2);
                if constexpr (D == 64) {
                    x.v[4 * h + j][0] = *(const uint16_t *)from;
                } else if constexpr (D == 128) {
                    x.v[4 * h + j][0] = *(const u32 *)from;
                } else {
                    const u32x2 w = *(const u32x2 *)from;
                    x.v[4 * h + j][0] = w[0];
                    x.v[4 * h + j][1] = w[1];
                }
            }
            x.vs[h] = *(const u32 *)(base + cache_scales(ps, D, 1) + (u32)(c * VC / 32 * ps + at + 4 * g));
        }
    }

    // Which groups of V's channels of a token are NaN, by their scales
    __device__ u32 nan_groups(const int32_t *table, int64_t t, int head)
    {
        int64_t page;
        int32_t at;
        cache_tile(P.c, table, t + 1, t / 16 * 16, &page, &at);
        const uint8_t *vs = P.cache + cache_page_at(P.c, page, head, D) + cache_scales(P.c.page_size, D, 1) + at + t % 16;
        u32 bits = 0;
        for (int j = 0; j < D / 32; ++j)
            bits |= (u32)(vs[j * P.c.page_size] == 255) << j;
        return bits;
    }

    template <bool MASKED>
    __device__ void step(Tile<D> &x, const bool there[2], const Rows &rows, int64_t len, const int32_t *table,
                         int64_t t0, int head)
    {
        f32x4 s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                const float f = scale_of(x.ks[h][D == 256 ? j / 4 : 0]);
                const u32 w = x.k[h][j];
                const u32x4 a = {H::template from_fp4<0>(w, f), H::template from_fp4<1>(w, f),
                                 H::template from_fp4<2>(w, f), H::template from_fp4<3>(w, f)};
                s[h] = H::mfma16(a, q[j], s[h]);
            }
        }
        float v[8];
        const float to_base2 = P.softcap > 0 ? 1.0f : P.scale * kLog2e;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = s[i / 4][i % 4] * to_base2;
        if (P.softcap > 0) {
            const float in = 2.0f * kLog2e * (P.scale / P.softcap), out = P.softcap * kLog2e;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float e = __builtin_amdgcn_exp2f(fabsf(v[i] * in));
                v[i] = copysignf(out - 2.0f * out * __builtin_amdgcn_rcpf(e + 1.0f), v[i] * in);
            }
        }
        if constexpr (MASKED) {
            u32 nan_tokens = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t t = t0 + 16 * (i / 4) + 4 * g + i % 4;
                const bool seen = there[i / 4] && t >= rows.lo && t < rows.hi;
                v[i] = seen ? v[i] : -__builtin_inff();
                // what no row sees may be anything; what some row does not see,
                // NaN: it then goes by `nans` to those that do
                const bool valid = there[i / 4] && t < len;
#pragma unroll
                for (int j = 0; j < (D + 127) / 128; ++j)
                    x.v[i][j] = valid ? x.v[i][j] : 0;
                const u32 byte = x.vs[i / 4] >> (8 * (i % 4)) & 255;
                if (byte == 255 || !valid)
                    x.vs[i / 4] &= ~(255u << (8 * (i % 4)));
                nan_tokens |= (u32)(byte == 255 && valid) << i;
            }
            if (__any(nan_tokens != 0)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t t = t0 + 16 * (i / 4) + 4 * g + i % 4;
                    if (there[i / 4] && t >= rows.lo && t < rows.hi)
                        nans |= nan_groups(table, t, head);
                }
            }
        }
        float most = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
        if (__any(most > top + S::kSlack)) {
            const float now = fmaxf(top, max_over_groups(most));
            const float a = __builtin_amdgcn_exp2f(top - now);
            top = now;
            sum *= a;
#pragma unroll
            for (int m = 0; m < VC; ++m)
                acc[m] *= a;
        }
        const float zero = top - S::kShift;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __builtin_amdgcn_exp2f(v[i] - zero);
        sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        const u32x4 p = {H::pack(v[0], v[1]), H::pack(v[2], v[3]), H::pack(v[4], v[5]), H::pack(v[6], v[7])};
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = scale_of(x.vs[i / 4] >> (8 * (i % 4)) & 255);
        values<0>(x, f, p);
        values<1>(x, f, p);
        if constexpr (VB > 2) {
            values<2>(x, f, p);
            values<3>(x, f, p);
        }
        if constexpr (VB > 4) {
            values<4>(x, f, p);
            values<5>(x, f, p);
            values<6>(x, f, p);
            values<7>(x, f, p);
        }
    }

    // Channels 2 BYTE and 2 BYTE + 1 of the lane's
    template <int BYTE> __device__ __forceinline__ void values(const Tile<D> &x, const float f[8], const u32x4 &p)
    {
        u32 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = H::template from_fp4<BYTE % 4>(x.v[i][BYTE / 4], f[i]);
        u32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100);
            hi[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302);
        }
        acc[2 * BYTE] = H::mfma16(lo, p, acc[2 * BYTE]);
        acc[2 * BYTE + 1] = H::mfma16(hi, p, acc[2 * BYTE + 1]);
    }

    // The wave's part of quanta [from, to) of the block
    __device__ void run(const Sequence &s, const Rows &rows, const int32_t *table, int head, int64_t from, int64_t to,
                        int wave)
    {
        top = kLowest;
        sum = 0.0f;
        nans = 0;
#pragma unroll
        for (int m = 0; m < VC; ++m)
            acc[m] = f32x4{0, 0, 0, 0};
        for (int64_t n = from; n < to; ++n) {
            const int64_t t = s.lo + n * kQuantum + wave * kStep;
            if (t >= s.len)
                break;
            Tile<D> x;
            bool there[2];
            load(x, there, table, s.len, t, head);
            if (t >= rows.most_lo && t + kStep <= rows.least_hi && there[0] && there[1])
                step<false>(x, there, rows, s.len, table, t, head);
            else
                step<true>(x, there, rows, s.len, table, t, head);
        }
    }
};

template <int D> struct Shared {
    float top[kAttnWaves][kRows], sum[kAttnWaves][kRows];
    float o[kAttnWaves][kRows][D + 4];
};

// Four channels of a finished row
template <int DT, int D>
__device__ void store(const AttentionParams &P, const Sequence &s, int64_t block, int head, int row, int d, float4 o,
                      float top, float sum)
{
    typedef Half<DT> H;
    const int64_t r = block * kRows + row;
    if (r >= s.rows)
        return;
    const int64_t i = r / P.group, at = (s.first + i) * P.q_heads + head * P.group + (r - i * P.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const u32x2 w = {H::pack(o.x * inv, o.y * inv), H::pack(o.z * inv, o.w * inv)};
    *(u32x2 *)(P.out + at * D + d) = w;
    if (P.lse && d == 0)
        P.lse[at] = sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum) - Softmax<DT>::kShift) * kLn2;
}

// BALANCED: the workers share all quanta evenly, and a block that several have
// parts of is put together by attention_join_kernel.  Otherwise a workgroup a block.
template <int DT, int D, bool BALANCED>
__global__ __launch_bounds__(64 * kAttnWaves) void attention_kernel(const AttentionParams P)
{
    __shared__ Shared<D> L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t at = 0, end = 0, start = 0, worker = 0;
    int b;
    if constexpr (BALANCED) {
        worker = block_id();
        const int64_t total = all_quanta(P), workers = workers_for(total, P.workers);
        if (worker >= workers || total == 0)
            return;
        at = share_start(total, workers, worker);
        end = share_start(total, workers, worker + 1);
        b = find_sequence(P, at, &start);
    } else {
        // row blocks of sequence b have numbers first * group / kRows + b on, or none
        const int64_t id = block_id() / P.c.heads;
        if (id >= P.blocks)
            return;
        int low = 0, high = P.B;
        if (P.q_starts) {
            while (high - low > 1) {
                const int mid = (low + high) / 2;
                const int64_t from = min((int64_t)max(P.q_starts[mid], 0), P.T);
                if (from * P.group / kRows + mid <= id)
                    low = mid;
                else
                    high = mid;
            }
            start = min((int64_t)max(P.q_starts[low], 0), P.T) * P.group / kRows + low;
        } else {
            const int each = (P.group + kRows - 1) / kRows;
            low = (int)(id / each);
            start = (int64_t)low * each;
        }
        b = low;
        const Sequence s = sequence(P, b);
        if (id < start || id - start >= s.blocks)
            return;
        // as if this block's quanta were a worker's share
        const int64_t head = block_id() % P.c.heads;
        at = (head * s.blocks + (id - start)) * s.quanta;
        end = at + s.quanta;
        start = 0;
    }
    Attention<DT, D> A(P);
    const int64_t begin = at;
    while (at < end) {
        Sequence s = sequence(P, b);
        while (at - start >= s.blocks * P.c.heads * s.quanta) {
            start += s.blocks * P.c.heads * s.quanta;
            s = sequence(P, ++b);
        }
        const int64_t index = (at - start) / s.quanta, from = at - start - index * s.quanta;
        const int head = (int)(index / s.blocks);
        const int64_t block = index - head * s.blocks;
        const int64_t to = min(s.quanta, from + (end - at));
        const Rows rows = A.rows_of(s, block);
        A.load_q(s, block, head);
        const int32_t *table = P.tables + b * P.table_stride;
        A.run(s, rows, table, head, from, to, wave);

        // the waves' parts, over their largest maximum
        const float sum = sum_over_groups(A.sum);
        const u32 nans = or_over_groups(A.nans);
        if (A.g == 0) {
            L.top[wave][A.c] = A.top;
            L.sum[wave][A.c] = sum;
        }
        __syncthreads();
        float top = kLowest;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w)
            top = fmaxf(top, L.top[w][A.c]);
        const float part = __builtin_amdgcn_exp2f(A.top - top);
#pragma unroll
        for (int m = 0; m < A.VC; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = (4 * A.g + i) * A.VC + m;
                L.o[wave][A.c][d] = nans >> (d / 32) & 1 ? __builtin_nanf("") : A.acc[m][i] * part;
            }
        __syncthreads();
        const bool whole = from == 0 && to == s.quanta;
        float *rec = record<D>(P, worker, at == begin);
        for (int e = threadIdx.x; e < kRows * D / 4; e += 64 * kAttnWaves) {
            const int row = e / (D / 4), d = e % (D / 4) * 4;
            float most = kLowest, all = 0.0f;
            float4 o = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w)
                most = fmaxf(most, L.top[w][row]);
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w) {
                all += L.sum[w][row] * __builtin_amdgcn_exp2f(L.top[w][row] - most);
                const float4 x = *(const float4 *)&L.o[w][row][d];
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
            }
            if (whole) {
                store<DT, D>(P, s, block, head, row, d, o, most, all);
            } else {
                *(float4 *)(rec + 2 * kRows + row * D + d) = o;
                if (d == 0) {
                    rec[row] = most;
                    rec[kRows + row] = all;
                }
            }
        }
        __syncthreads();
        at += to - from;
    }
}

// Puts together the block that begins in this worker's share and ends in another's
template <int DT, int D>
__global__ __launch_bounds__(64 * kAttnWaves) void attention_join_kernel(const AttentionParams P)
{
    const int64_t worker = block_id();
    const int64_t total = all_quanta(P), workers = workers_for(total, P.workers);
    if (worker + 1 >= workers || total == 0)
        return;
    const int64_t begin = share_start(total, workers, worker), end = share_start(total, workers, worker + 1);
    if (begin == end)
        return;
    int64_t start;
    const int b = find_sequence(P, end - 1, &start);
    const Sequence s = sequence(P, b);
    const int64_t index = (end - 1 - start) / s.quanta;
    const int64_t first = start + index * s.quanta, last = first + s.quanta;
    if (first < begin || last == end)
        return;
    int64_t upto = worker;       // the last worker with a part
    while (share_start(total, workers, upto + 1) < last)
        ++upto;
    const int head = (int)(index / s.blocks);
    const int64_t block = index - head * s.blocks;
    for (int e = threadIdx.x; e < kRows * D / 4; e += 64 * kAttnWaves) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        float most = kLowest, all = 0.0f;
        float4 o = {0, 0, 0, 0};
        for (int64_t w = worker; w <= upto; ++w) {
            const float *rec = record<D>(P, w, w > worker || first == begin);
            const float top = rec[row], now = fmaxf(most, top);
            const float old = __builtin_amdgcn_exp2f(most - now), part = __builtin_amdgcn_exp2f(top - now);
            const float4 x = *(const float4 *)(rec + 2 * kRows + row * D + d);
            all = all * old + rec[kRows + row] * part;
            o.x = o.x * old + x.x * part;
            o.y = o.y * old + x.y * part;
            o.z = o.z * old + x.z * part;
            o.w = o.w * old + x.w * part;
            most = now;
        }
        store<DT, D>(P, s, block, head, row, d, o, most, all);
    }
}

// Row blocks that T rows in B sequences may have, numbered as above
int64_t most_blocks(int64_t T, int B, int group, bool ragged)
{
    return ragged ? T * group / kRows + B : (int64_t)B * ((group + kRows - 1) / kRows);
}

int workers_of(int cus) { return cus * 3; }

template <int DT, int D> hipError_t launch(AttentionParams p, int cus, hipStream_t s)
{
    if (p.workspace) {
        attention_kernel<DT, D, true><<<grid_of(p.workers), 64 * kAttnWaves, 0, s>>>(p);
        attention_join_kernel<DT, D><<<grid_of(p.workers), 64 * kAttnWaves, 0, s>>>(p);
    } else {
        attention_kernel<DT, D, false><<<grid_of(p.blocks * p.c.heads), 64 * kAttnWaves, 0, s>>>(p);
    }
    return hipGetLastError();
}

template <int DT> hipError_t launch_width(const AttentionParams &p, int D, int cus, hipStream_t s)
{
    return D == 64 ? launch<DT, 64>(p, cus, s) : D == 128 ? launch<DT, 128>(p, cus, s) : launch<DT, 256>(p, cus, s);
}

// Whether a batch's quanta are shared out: not where there are blocks for every
// CU many times over, or more sequences than a worker adds up
bool balanced(int64_t T, int B, int q_heads, int kv_heads, int cus)
{
    return B <= kMostBalanced && most_blocks(T, B, q_heads / kv_heads, true) * kv_heads < (int64_t)cus * 16;
}

}  // namespace

uint64_t attention_workspace_floats(int64_t T, int B, int q_heads, int kv_heads, int head_dim, int cus)
{
    return balanced(T, B, q_heads, kv_heads, cus) ? (uint64_t)workers_of(cus) * 2 * kRows * (head_dim + 2) : 0;
}

hipError_t launch_attention(const AttentionParams &a, int head_dim, int dtype, int cus, hipStream_t s)
{
    AttentionParams p = a;
    p.blocks = most_blocks(p.T, p.B, p.group, p.q_starts != nullptr);
    p.workers = workers_of(cus);
    if (!balanced(p.T, p.B, p.q_heads, p.c.heads, cus))
        p.workspace = nullptr;
    return dtype == MHC_BF16 ? launch_width<MHC_BF16>(p, head_dim, cus, s)
                             : launch_width<MHC_F16>(p, head_dim, cus, s);
}

}  // namespace mhc
