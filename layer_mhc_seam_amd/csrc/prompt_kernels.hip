// prompt_kernels.hip -- attention over the 4-bit cache for many query rows a
// sequence: prompts and chunks of them.
//
// The matrix cores bound it, 4 D operations a row and token.  A workgroup holds
// kWaves * 32 * CT rows (query rows times heads of a kv head) and goes through
// the tokens in tiles of 64, once: keys and values are turned from 4 bits into
// the products' type on their way into LDS, by all waves for all of them, while
// the tile before is worked on.  A wave's products are 32 x 32 x 16:
//   S^T = K Q^T     lane (q, h), q = l % 32, h = l / 32, holds row q of Q, and of
//                   the result tokens 8 b + 4 h + r, b and r 0 .. 3
//   O^T += V^T P^T  P is the operand as it stands: k = 16 tokens, of which lane h
//                   has 4 h + r and 8 + 4 h + r.  V lies in LDS in those groups
//                   of eight tokens, for one channel after another.
#include "attention_common.h"

namespace mhc {
namespace {

constexpr int kTile = 64;                // tokens
constexpr int kGroups = kTile / 8;       // of tokens, as a product's lane has them

template <int D> struct PromptShared {
    u32x4 k[2][D / 8][kTile];            // eight channels of a token
    u32x2 v[2][kGroups][D][2];           // eight tokens of a channel; channel c D/16 + m at m 16 + c
    u32 nan[2][8];                       // whether a wave met a NaN among a tile's values
    u32 there[2][4];                     // whether a tile's 16 tokens have a page
};

// A thread's part of a tile on its way: units of 32 channels of a token's keys,
// and four tokens' values, D/16 channels.  Short loads are of four bytes that
// begin with theirs, for the compiler to have nothing to cut off behind them.
template <int D, int KU> struct Raw {
    u32x4 k[KU];
    u32 ks[KU];
    u32 v[4][(D + 127) / 128];
    u32 vs;
    bool k_there, v_there;
};

typedef u32 u32_any __attribute__((aligned(1)));

template <int DT, int D, int WAVES, int CT, bool CAP> struct Prompt {
    typedef Half<DT> H;
    typedef Softmax<DT> S;
    static constexpr int kThreads = 64 * WAVES, kRows = 32 * CT * WAVES;
    static constexpr int KC = D / 16, DC = D / 32;
    static constexpr int kUnits = kTile * (D / 32);                 // of keys
    static constexpr int KU = (kUnits + kThreads - 1) / kThreads;
    static constexpr int kFirstV = kThreads - 256;                  // threads from here on take values

    const AttentionParams &P;
    PromptShared<D> &L;
    const int lane, wave, q, h;
    f32x16 o[CT][DC];
    u32x4 qr[CT][KC];
    float top[CT], sum[CT];
    float factor;                        // of the products, to scores in base 2; not negative
    u32 nans[CT];
    int lo[CT], hi[CT];

    __device__ Prompt(const AttentionParams &p, PromptShared<D> &l)
        : P(p), L(l), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), q(lane & 31),
          h(lane >> 5)
    {
    }

    // ------------------------------------------------------- a tile's way in

    // Pages of the thread's tokens of a tile, as the table has them: of its keys'
    // and of its values'.  Nothing is done with them before they are used, a tile
    // later.
    struct Pages {
        int k, k_at, v, v_at;
    };

    __device__ __forceinline__ int value_group() const { return ((int)threadIdx.x - kFirstV) / 32; }
    // First of the 16 tokens that the thread's are of, in the tile.  Units u, u +
    // kThreads, .. of keys have one token: 64 divides kThreads.
    __device__ __forceinline__ int key_tile() const { return (int)(threadIdx.x % kTile) / 16 * 16; }
    __device__ __forceinline__ int value_tile() const { return max(value_group(), 0) / 2 * 16; }

    __device__ __forceinline__ Pages pages(const int32_t *table, int last, int t) const
    {
        int k, v;
        Pages g;
        cache_tile(P.c, t + key_tile(), &k, &g.k_at);
        cache_tile(P.c, t + value_tile(), &v, &g.v_at);
        g.k = table[min(k, last)];
        g.v = table[min(v, last)];
        return g;
    }

    // Whether that page is one, and tokens [t, t + 16) are of the sequence's: if
    // not, page 0 and its first tokens stand for them
    __device__ __forceinline__ bool there(int &page, int &at, int len, int t) const
    {
        const bool ok = t < len && (u32)page < (u32)P.c.pages;
        page = ok ? page : 0;
        at = ok ? at : 0;
        return ok;
    }

    __device__ __forceinline__ void load(Raw<D, KU> &x, Pages g, int len, int t, int head) const
    {
        const int ps = P.c.page_size;
        x.k_there = there(g.k, g.k_at, len, t + key_tile());
        x.v_there = there(g.v, g.v_at, len, t + value_tile());
        {
            const uint8_t *base = P.cache + cache_page_near(P.c, g.k, head, D);
            const u32 token = g.k_at + threadIdx.x % 16;
#pragma unroll
            for (int i = 0; i < KU; ++i) {
                const u32 unit = threadIdx.x + i * kThreads, part = unit / kTile;
                if (kUnits % kThreads == 0 || unit < kUnits) {
                    x.k[i] = *(const u32x4 *)(base + (token * (D / 2) + part * 16));
                    x.ks[i] = *(const u32_any *)(base + (cache_scales(ps, D, 0) + part * ps + token));
                }
            }
        }
        if (kFirstV == 0 || (int)threadIdx.x >= kFirstV) {
            const uint8_t *base = P.cache + cache_page_near(P.c, g.v, head, D);
            const u32 first = g.v_at + 4 * (value_group() & 1) + 8 * (threadIdx.x & 1), c = threadIdx.x / 2 % 16;
            const u32 code = cache_codes(ps, D, 1) + first * (D / 2) + c * (D / 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *from = base + code + i * (D / 2);
                if constexpr (D <= 128) {
                    x.v[i][0] = *(const u32_any *)from;
                } else {
                    const u32x2 w = *(const u32x2 *)from;
                    x.v[i][0] = w[0];
                    x.v[i][1] = w[1];
                }
            }
            x.vs = *(const u32 *)(base + (cache_scales(ps, D, 1) + c * (D / 16) / 32 * ps + first));
        }
    }

    // EDGE: some row sees only some of the tile's tokens.  A NaN among its values
    // is then left out, and noted.
    __device__ __forceinline__ void put(Raw<D, KU> &x, int buf, int len, int t, bool edge)
    {
#pragma unroll
        for (int i = 0; i < KU; ++i) {
            const int unit = threadIdx.x + i * kThreads, part = unit / kTile, token = threadIdx.x % kTile;
            if (kUnits % kThreads == 0 || unit < kUnits) {
                const float f = scale_of(x.ks[i] & 255);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    L.k[buf][part * 4 + j][token] =
                        u32x4{H::template from_fp4<0>(x.k[i][j], f), H::template from_fp4<1>(x.k[i][j], f),
                              H::template from_fp4<2>(x.k[i][j], f), H::template from_fp4<3>(x.k[i][j], f)};
                if (unit % 16 == 0 && unit < kTile)
                    L.there[buf][unit / 16] = x.k_there;
            }
        }
        u32 odd = 0;
        if (kFirstV == 0 || (int)threadIdx.x >= kFirstV) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32 byte = x.vs >> (8 * i) & 255;
                if (edge || !x.v_there) {
                    const bool valid = x.v_there && t + value_tile() + 4 * (value_group() & 1) +
                                                           8 * (int)(threadIdx.x & 1) + i < len;
                    odd |= (u32)(byte == 255 && valid);
#pragma unroll
                    for (int j = 0; j < (D + 127) / 128; ++j)
                        x.v[i][j] = valid ? x.v[i][j] : 0;
                    byte = byte == 255 || !valid ? 0 : byte;
                }
                f[i] = scale_of(byte);
            }
            values<0>(x, f, buf);
            values<1>(x, f, buf);
            if constexpr (D >= 128) {
                values<2>(x, f, buf);
                values<3>(x, f, buf);
            }
            if constexpr (D >= 256) {
                values<4>(x, f, buf);
                values<5>(x, f, buf);
                values<6>(x, f, buf);
                values<7>(x, f, buf);
            }
        }
        if (edge) {
            const u32 any = __any(odd != 0);
            if (lane == 0)
                L.nan[buf][wave] = any;
        }
    }

    template <int BYTE>
    __device__ __forceinline__ void values(const Raw<D, KU> &x, const float f[4], int buf)
    {
        const int group = value_group(), c = threadIdx.x / 2 % 16, half = threadIdx.x & 1;
        u32 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = H::template from_fp4<BYTE % 4>(x.v[i][BYTE / 4], f[i]);
        L.v[buf][group][(2 * BYTE) * 16 + c][half] = u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x05040100),
                                                           __builtin_amdgcn_perm(w[3], w[2], 0x05040100)};
        L.v[buf][group][(2 * BYTE + 1) * 16 + c][half] = u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x07060302),
                                                               __builtin_amdgcn_perm(w[3], w[2], 0x07060302)};
    }

    // ------------------------------------------------------------ a tile's work

    // Whether the tile's 16 tokens have their pages, a bit each
    __device__ __forceinline__ u32 pages_there(int buf) const
    {
        u32 there = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            there |= L.there[buf][j] << j;
        return __builtin_amdgcn_readfirstlane(there);
    }

    // Hides what the lane's row does not see of the tile: edge, by the rows'
    // bounds; there, for its page
    __device__ __forceinline__ void mask(float v[32], int i, int buf, int t, Whole table, int head, bool edge,
                                         u32 there)
    {
        u32 seen = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int token = t + 32 * (j / 16) + 8 * (j % 16 / 4) + 4 * h + j % 4;
            const bool sees = token >= lo[i] && token < hi[i] && (there >> (j / 8) & 1);
            seen |= (u32)sees << j;
            v[j] = sees ? v[j] : -__builtin_inff();
        }
        if (!edge)
            return;
        u32 odd = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            odd |= L.nan[buf][w];
        if (__builtin_amdgcn_readfirstlane(odd))
#pragma unroll 1
            for (int j = 0; j < 32; ++j)
                if (seen >> j & 1)
                    nans[i] |=
                        nan_groups<D>(P, table, t + 32 * (j / 16) + 8 * (j % 16 / 4) + 4 * h + j % 4, head);
    }

    __device__ __forceinline__ void work(int buf, int t, Whole table, int head, bool edge)
    {
        const u32 there = pages_there(buf);
        f32x16 s[CT][2];
#pragma unroll
        for (int i = 0; i < CT; ++i)
            s[i][0] = s[i][1] = f32x16{0};
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const u32x4 a = L.k[buf][2 * k + h][32 * tt + q];
#pragma unroll
                for (int i = 0; i < CT; ++i)
                    s[i][tt] = H::mfma32(a, qr[i][k], s[i][tt]);
            }
        u32x4 p[CT][4];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = s[i][j / 16][j % 16];
            if constexpr (CAP)
                cap<32>(P, v);
            if (edge || there != 15)
                mask(v, i, buf, t, table, head, edge, there);
            float most = v[0];
#pragma unroll
            for (int j = 1; j < 32; ++j)
                most = fmaxf(most, v[j]);
            most *= factor;
            if (__any(most > top[i] + S::kSlack)) {
                const u32 x = __float_as_uint(most);
                auto both = __builtin_amdgcn_permlane32_swap(x, x, false, false);
                const float now = fmaxf(top[i], fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])));
                const float a = __builtin_amdgcn_exp2f(top[i] - now);
                top[i] = now;
                sum[i] *= a;
#pragma unroll
                for (int d = 0; d < DC; ++d)
                    o[i][d] *= a;
            }
            const float zero = S::kShift - top[i];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = __builtin_amdgcn_exp2f(fmaf(v[j], factor, zero));
            float part[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 32; ++j)
                part[j % 4] += v[j];
            sum[i] += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                p[i][c] = u32x4{H::pack(v[8 * c], v[8 * c + 1]), H::pack(v[8 * c + 2], v[8 * c + 3]),
                                H::pack(v[8 * c + 4], v[8 * c + 5]), H::pack(v[8 * c + 6], v[8 * c + 7])};
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int d = 0; d < DC; ++d) {
                const u32x4 a = *(const u32x4 *)L.v[buf][2 * c + h][d * 32 + q];
#pragma unroll
                for (int i = 0; i < CT; ++i)
                    o[i][d] = H::mfma32(a, p[i][c], o[i][d]);
            }
    }
};

template <int DT, int D, int WAVES, int CT, bool CAP>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
void prompt_kernel(const AttentionParams P)
{
    typedef Prompt<DT, D, WAVES, CT, CAP> A_;
    typedef Half<DT> H;
    __shared__ PromptShared<D> L;
    constexpr int ROWS = A_::kRows;
    const int64_t id = block_id() / P.c.heads;
    const int head = (int)(block_id() - id * P.c.heads);
    if (id >= P.blocks)
        return;
    const int64_t number = P.blocks - 1 - id;        // a prompt's last rows have the most to do
    int64_t numbered;
    const int b = sequence_of(P, number, ROWS, &numbered);
    const int64_t first = row_start(P, b), n64 = row_start(P, b + 1) - first;
    const int n = (int)max(n64, (int64_t)0);
    const int64_t row = (number - numbered) * ROWS, rows = (int64_t)n * P.group;
    if (number < numbered || row >= rows)
        return;
    const int len = length_of(P, b);
    const Whole table = whole(P.tables + b * P.table_stride);
    const int i0 = (int)(row / P.group), skip = (int)(row - (int64_t)i0 * P.group);

    A_ A(P, L);
    // a negative scale's sign goes to the queries, one of 0 makes them 0: the
    // scores' order is that of their products, and -inf times the factor -inf
    const u32 sign = CAP || P.scale >= 0 ? 0 : 0x80008000u, keep = CAP || P.scale != 0 ? ~0u : 0;
    A.factor = CAP ? 1.0f : P.scale != 0 ? fabsf(P.scale) * kLog2e : 1.0f;
    // tokens that some row, and that every row, of the block sees
    int least_lo, most_lo, least_hi, most_hi;
    row_sees(P, len, n, i0, &least_lo, &least_hi);
    row_sees(P, len, n, min(i0 + (skip + ROWS - 1) / P.group, n - 1), &most_lo, &most_hi);
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        const int r = skip + (A.wave * CT + i) * 32 + A.q, over = r / P.group;
        row_sees(P, len, n, i0 + over, &A.lo[i], &A.hi[i]);
        if (i0 + over >= n)
            A.lo[i] = A.hi[i] = 0;
        const uint16_t *at = P.q + (first + min(i0 + over, n - 1)) * P.q_token +
                             (int64_t)(head * P.group + (r - over * P.group)) * P.q_head;
#pragma unroll
        for (int k = 0; k < A.KC; ++k)
            A.qr[i][k] = (*(const u32x4 *)(at + 16 * k + 8 * A.h) & keep) ^ sign;
        A.top[i] = kLowest;
        A.sum[i] = 0.0f;
        A.nans[i] = 0;
#pragma unroll
        for (int d = 0; d < A.DC; ++d)
            A.o[i][d] = f32x16{0};
    }

    int t = least_lo / kTile * kTile;
    if (t < most_hi) {
        auto is_edge = [&](int at) { return at < most_lo || at + kTile > least_hi; };
        Raw<D, A.KU> x;
        const int32_t *entries = P.tables + b * P.table_stride;
        int last, none;
        cache_tile(P.c, (len - 1) / kCacheTile * kCacheTile, &last, &none);
        typename A_::Pages g = A.pages(entries, last, t);
        A.load(x, g, len, t, head);
        g = A.pages(entries, last, t + kTile);
        A.put(x, 0, len, t, is_edge(t));
        __syncthreads();
        int buf = 0;
        while (true) {
            // the next tile is asked for, this one worked on, the next one put beside it
            const bool more = t + kTile < most_hi;
            if (more) {
                A.load(x, g, len, t + kTile, head);
                g = A.pages(entries, last, t + 2 * kTile);
            }
            A.work(buf, t, table, head, is_edge(t));
            if (!more)
                break;
            t += kTile;
            buf ^= 1;
            A.put(x, buf, len, t, is_edge(t));
            __syncthreads();
        }
    }

#pragma unroll
    for (int i = 0; i < CT; ++i) {
        const u32 s = __float_as_uint(A.sum[i]);
        auto sums = __builtin_amdgcn_permlane32_swap(s, s, false, false);
        const float sum = __uint_as_float(sums[0]) + __uint_as_float(sums[1]);
        auto odd = __builtin_amdgcn_permlane32_swap(A.nans[i], A.nans[i], false, false);
        const u32 nans = odd[0] | odd[1];
        const int r = skip + (A.wave * CT + i) * 32 + A.q, over = r / P.group;
        if (i0 + over >= n)
            continue;
        const int64_t at = (first + i0 + over) * P.q_heads + head * P.group + (r - over * P.group);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        // register i of product d is row r = 8 (i / 4) + 4 h + i % 4 of it, channel
        // r % 16 D/16 + 2 d + r / 16: D/16 channels side by side in two registers
        // of all the products
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c0 = (8 * j + 4 * A.h + e) * (D / 16);
                u32 w[A.DC];
#pragma unroll
                for (int d = 0; d < A.DC; ++d)
                    w[d] = H::pack(A.o[i][d][4 * j + e] * inv, A.o[i][d][4 * j + 8 + e] * inv);
                if (nans >> (c0 / 32) & 1)
#pragma unroll
                    for (int d = 0; d < A.DC; ++d)
                        w[d] = DT == MHC_BF16 ? 0x7fc07fc0u : 0x7e007e00u;
                uint16_t *to = P.out + at * D + c0;
                if constexpr (A.DC == 2) {
                    *(u32x2 *)to = u32x2{w[0], w[1]};
                } else {
#pragma unroll
                    for (int d = 0; d < A.DC; d += 4)
                        *(u32x4 *)(to + 2 * d) = u32x4{w[d], w[d + 1], w[d + 2], w[d + 3]};
                }
            }
        if (P.lse && A.h == 0)
            P.lse[at] = sum == 0.0f ? -__builtin_inff()
                                    : (A.top[i] + __builtin_amdgcn_logf(sum) - Softmax<DT>::kShift) * kLn2;
    }
}

template <int DT, int D, bool CAP> hipError_t launch_cap(const AttentionParams &p, hipStream_t s)
{
    constexpr int WAVES = 4, CT = 1;
    AttentionParams q = p;
    q.blocks = most_blocks(p.T, p.B, p.group, 32 * CT * WAVES, p.q_starts != nullptr);
    prompt_kernel<DT, D, WAVES, CT, CAP><<<grid_of(q.blocks * p.c.heads), 64 * WAVES, 0, s>>>(q);
    return hipGetLastError();
}

template <int DT, int D> hipError_t launch(const AttentionParams &p, hipStream_t s)
{
    return p.softcap > 0 ? launch_cap<DT, D, true>(p, s) : launch_cap<DT, D, false>(p, s);
}

template <int DT> hipError_t launch_width(const AttentionParams &p, int D, hipStream_t s)
{
    return D == 64 ? launch<DT, 64>(p, s) : D == 128 ? launch<DT, 128>(p, s) : launch<DT, 256>(p, s);
}

}  // namespace

hipError_t launch_prompt(const AttentionParams &p, int head_dim, int dtype, hipStream_t s)
{
    return dtype == MHC_BF16 ? launch_width<MHC_BF16>(p, head_dim, s) : launch_width<MHC_F16>(p, head_dim, s);
}

}  // namespace mhc
