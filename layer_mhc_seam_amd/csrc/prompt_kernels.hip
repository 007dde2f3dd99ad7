// prompt_kernels.hip -- attention over the 4-bit cache for many query rows a
// sequence: prompts and chunks of them.
//
// The matrix cores bound it, 4 D operations a row and token, and the clock under
// them: 4096 rows of 40 heads over 16384 tokens take 1150 to 1350 us, 0.89 to 1.04
// PFLOP/s where a large bf16 product reaches 1.44.  Of the 2.4 million cycles that a
// CU is busy matrix instructions take 48% and vector instructions 51%; six calls
// had the clock at 1.71 to 1.96 GHz.
// A workgroup holds 128 rows (query rows times heads of a kv head), 32 a wave (64 a
// wave, one workgroup a CU: 1551 us for 1323 then), and goes through the tokens in
// tiles of 64, once: keys and values are turned from 4 bits into the products' type
// on their way into LDS, by all waves for all of them, while the tile before is
// worked on (products of 4-bit by 8-bit operands, which would take the codes as they
// are, sum to 2^-12.9 of the sum of magnitudes only, and are not used).  The order of
// products, weights and LDS writes is written out: the compiler's own has all
// products first.  A wave's products are 32 x 32 x 16:
//   S^T = K Q^T     lane (q, h), q = l % 32, h = l / 32, holds row q of Q, and of
//                   the result tokens 8 b + 4 h + r, b and r 0 .. 3
//   O^T += V^T P^T  P is the operand as it stands: k = 16 tokens, of which lane h
//                   has 4 h + r and 8 + 4 h + r.  V lies in LDS in those groups
//                   of eight tokens, for one channel after another.
#include "attention_join.h"

namespace mhc {
namespace {

constexpr int kTile = 64;                // tokens
constexpr int kPromptWaves = 4, kPromptRows = 32 * kPromptWaves;
constexpr int kGroups = kTile / 8;       // of tokens, as a product's lane has them
constexpr int kLeastTiles = 4;           // of a worker's share, where a block has as many
constexpr int kSharedTokens = 2048;      // of sequences whose tiles are shared out

template <int D> struct PromptShared {
    u32x4 k[2][D / 8][kTile];            // eight channels of a token
    u32x2 v[2][kGroups][D][2];           // eight tokens of a channel; channel c D/16 + m at m 16 + c
    u32 nan[2][4];                       // whether a wave met a NaN among a tile's values
    u32 there[2][4];                     // whether a tile's 16 tokens have a page
};

template <int N> struct Number {
    static constexpr int value = N;
};

// f(Number<0>) .. f(Number<N - 1>)
template <int N, int I = 0, typename F> __device__ __forceinline__ void static_for(F f)
{
    if constexpr (I < N) {
        f(Number<I>{});
        static_for<N, I + 1>(f);
    }
}

// 16 tokens' keys on their way: a lane has units of 32 channels of a token
template <int D> struct RawKeys {
    u32x4 k[(D + 127) / 128];
    u32 scale[(D + 127) / 128];          // in the low byte
    bool there;
};

// 16 tokens' values: a lane has D/16 channels of four tokens
template <int D> struct RawValues {
    u32 v[4][(D + 127) / 128];           // D = 64: in the low half
    u32 scale;
    bool there;
};

template <int DT, int D, int CAP> struct Prompt {
    typedef Half<DT> H;
    typedef Softmax<DT> S;
    static constexpr int KC = D / 16, DC = D / 32, KU = (D + 127) / 128;

    const AttentionParams &P;
    PromptShared<D> &L;
    const int lane, wave, q, h;
    u32 at_k, at_ks, at_v, at_vs;        // the lane's bytes in the wave's 16 tokens
    f32x16 o[DC], s[2];                  // of the lane's row, as all below
    u32x4 qr[KC], p[4];
    float top, sum;
    u32 nans;                            // groups of channels that a NaN reaches
    int lo, hi;                          // tokens that it sees
    float factor;                        // of the products, to scores in base 2; not negative

    __device__ Prompt(const AttentionParams &p_, PromptShared<D> &l)
        : P(p_), L(l), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), q(lane & 31),
          h(lane >> 5)
    {
        const int ps = P.c.page_size;
        at_k = lane % 16 * (D / 2) + lane / 16 * 16;
        at_ks = cache_scales(ps, D, 0) + lane / 16 * ps + lane % 16;
        at_v = cache_codes(ps, D, 1) + value_token() * (D / 2) + value_chunk() * (D / 32);
        at_vs = cache_scales(ps, D, 1) + value_chunk() * (D / 16) / 32 * ps + value_token();
        if (D == 64 && lane >= 32)       // there are no third and fourth units: the first's once more
            at_k -= 32, at_ks -= 2 * ps;
    }

    // ------------------------------------------------------- a tile's way in
    //
    // Wave w brings tokens 16 w .. 16 w + 15 of each tile: one page.

    // The lane's values: four tokens from this one on, of the wave's 16; a lane's
    // eight tokens of a product are two lanes' halves
    __device__ __forceinline__ int value_token() const { return 4 * (lane >> 5) + 8 * (lane & 1); }
    __device__ __forceinline__ int value_chunk() const { return lane / 2 % 16; }

    // Page and place there of the wave's 16 tokens of the tile at t; page 0 for none
    __device__ __forceinline__ bool place(Whole table, int len, int t, int *page, int *at) const
    {
        return cache_page(P.c, table, len, t + 16 * wave, page, at);
    }

    __device__ __forceinline__ void load(RawKeys<D> &x, Whole table, int len, int t, int head) const
    {
        int page, at;
        x.there = place(table, len, t, &page, &at);
        const Page from = page_of<D>(P, page, head);
#pragma unroll
        for (int i = 0; i < KU; ++i) {
            x.k[i] = from.load128_again(at_k + 64 * i, at * (D / 2));
            x.scale[i] = from.load32(at_ks + 4 * i * P.c.page_size, at);
        }
    }

    __device__ __forceinline__ void load(RawValues<D> &x, Whole table, int len, int t, int head) const
    {
        int page, at;
        x.there = place(table, len, t, &page, &at);
        const Page from = page_of<D>(P, page, head);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D <= 128) {
                x.v[i][0] = from.load32(at_v + i * (D / 2), at * (D / 2));
            } else {
                const u32x2 w = from.load64(at_v + i * (D / 2), at * (D / 2));
                x.v[i][0] = w[0];
                x.v[i][1] = w[1];
            }
        }
        x.scale = from.load32(at_vs, at);
    }

    // Channels 8 j .. 8 j + 7 of the lane's unit i
    __device__ __forceinline__ void put_key(int i, int j, const RawKeys<D> &x, const float f[KU], int buf)
    {
        // D = 64: lanes l and l + 32 have the same and write it to the same place
        L.k[buf][(lane / 16 % (D < 128 ? 2 : 4) + 4 * i) * 4 + j][16 * wave + lane % 16] =
            u32x4{H::template from_fp4<0>(x.k[i][j], f[i]), H::template from_fp4<1>(x.k[i][j], f[i]),
                  H::template from_fp4<2>(x.k[i][j], f[i]), H::template from_fp4<3>(x.k[i][j], f[i])};
    }

    __device__ __forceinline__ void put(const RawKeys<D> &x, int buf)
    {
        float f[KU];
#pragma unroll
        for (int i = 0; i < KU; ++i)
            f[i] = scale_of(x.scale[i] & 255);
#pragma unroll
        for (int i = 0; i < KU; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                put_key(i, j, x, f, buf);
        if (lane == 0)
            L.there[buf][wave] = x.there;
    }

    // Where some row sees only some of the tile's tokens (edge) a NaN among its
    // values is left out and noted; tokens that are not there, or outside those
    // [from, to) that some row sees, are 0
    __device__ __forceinline__ void clean(RawValues<D> &x, int buf, int from, int to, int t, bool edge)
    {
        u32 odd = 0;
        if (edge || !x.there) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int token = t + 16 * wave + value_token() + i;
                const bool valid = x.there && token >= from && token < to;
                const u32 byte = x.scale >> (8 * i) & 255;
                odd |= (u32)(byte == 255 && valid);
#pragma unroll
                for (int j = 0; j < KU; ++j)
                    x.v[i][j] = valid ? x.v[i][j] : 0;
                if (byte == 255 || !valid)
                    x.scale &= ~(255u << (8 * i));
            }
            if (edge)
                L.nan[buf][wave] = __any(odd != 0);
        }
    }

    __device__ __forceinline__ void put(const RawValues<D> &x, int buf)
    {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = scale_of(x.scale >> (8 * i) & 255);
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

    template <int BYTE> __device__ __forceinline__ void values(const RawValues<D> &x, const float f[4], int buf)
    {
        const int group = 2 * wave + (lane >> 5), c = value_chunk(), half = lane & 1;
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

    __device__ __forceinline__ void products(int buf)
    {
        s[0] = s[1] = f32x16{0};
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s[i] = H::mfma32(L.k[buf][2 * k + h][32 * i + q], qr[k], s[i]);
    }

    // Token of the tile at t that register j of the scores is, 0 .. 31
    __device__ __forceinline__ int token(int t, int j) const
    {
        return t + 32 * (j / 16) + 8 * (j % 16 / 4) + 4 * h + j % 4;
    }

    // The products of the tile at t as scores to the factor, hidden where the
    // lane's row does not see them, and the maximum brought up to them
    __device__ __forceinline__ void settle(int buf, int t, bool edge)
    {
        if constexpr (CAP != kNoCap) {
            // the series leaves no registers for more than eight at once
            constexpr int N = CAP == kHigh ? 8 : 32;
#pragma unroll
            for (int j0 = 0; j0 < 32; j0 += N) {
                float v[N];
#pragma unroll
                for (int j = 0; j < N; ++j)
                    v[j] = s[(j0 + j) / 16][(j0 + j) % 16];
                cap<N, CAP>(P, v);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    s[(j0 + j) / 16][(j0 + j) % 16] = v[j];
            }
        }
        u32 there = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            there |= L.there[buf][j] << j;
        there = __builtin_amdgcn_readfirstlane(there);
        if (edge || there != 15) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const bool sees = token(t, j) >= lo && token(t, j) < hi && (there >> (j / 8) & 1);
                s[j / 16][j % 16] = sees ? s[j / 16][j % 16] : -__builtin_inff();
            }
        }
        float most = s[0][0];
#pragma unroll
        for (int j = 1; j < 32; ++j)
            most = fmaxf(most, s[j / 16][j % 16]);
        most *= factor;
        if (__any(most > top + S::kSlack)) {
            const u32 x = __float_as_uint(most);
            auto both = __builtin_amdgcn_permlane32_swap(x, x, false, false);
            const float now = fmaxf(top, fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])));
            const float a = __builtin_amdgcn_exp2f(top - now);
            top = now;
            sum *= a;
#pragma unroll
            for (int d = 0; d < DC; ++d)
                o[d] *= a;
        }
    }

    // Score j as a weight; every second one packs two
    __device__ __forceinline__ void weigh(int j, float v[2], float part[2], float zero)
    {
        v[j % 2] = __builtin_amdgcn_exp2f(fmaf(s[j / 16][j % 16], factor, zero));
        part[j % 2] += v[j % 2];
        if (j % 2) {
            u32 w = H::pack(v[0], v[1]);
            asm volatile("" : "+v"(w), "+v"(part[0]), "+v"(part[1]));    // here, and not behind all products
            p[j / 8][j % 8 / 2] = w;
        }
    }

    __device__ __forceinline__ void weights()
    {
        float part[2] = {0, 0}, v[2];
#pragma unroll
        for (int j = 0; j < 32; ++j)
            weigh(j, v, part, S::kShift - top);
        sum += part[0] + part[1];
    }

    __device__ __forceinline__ void add(int buf)
    {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int d = 0; d < DC; ++d)
                o[d] = H::mfma32(*(const u32x4 *)L.v[buf][2 * n + h][d * 32 + q], p[n], o[d]);
    }

    // The next tile's products with this one's weights beside them, product after
    // product: the compiler by itself puts all products first
    __device__ __forceinline__ void products_and_weights(f32x16 next[2], int buf)
    {
        constexpr int N = 2 * KC, EACH = 32 / N, AHEAD = 4;
        const float zero = S::kShift - top;
        float part[2] = {0, 0}, v[2];
        u32x4 a[AHEAD];
        auto read = [&](int n) { return L.k[buf][2 * (n / 2) + h][32 * (n % 2) + q]; };
        next[0] = next[1] = f32x16{0};
#pragma unroll
        for (int n = 0; n < AHEAD - 1; ++n)
            a[n] = read(n);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (n + AHEAD - 1 < N)
                a[(n + AHEAD - 1) % AHEAD] = read(n + AHEAD - 1);
            next[n % 2] = H::mfma32(a[n % AHEAD], qr[n / 2], next[n % 2]);
#pragma unroll
            for (int j = n * EACH; j < (n + 1) * EACH; ++j)
                weigh(j, v, part, zero);
            __builtin_amdgcn_sched_barrier(0);
        }
        sum += part[0] + part[1];
    }

    // Likewise this tile's values with what comes in
    __device__ __forceinline__ void values_and_puts(int buf, const RawValues<D> &vals, const RawKeys<D> &keys)
    {
        constexpr int N = 4 * DC, CHUNKS = D / 32 + 4 * KU, AHEAD = 4;
        u32x4 a[AHEAD];
        auto read = [&](int n) { return *(const u32x4 *)L.v[buf][2 * (n / DC) + h][n % DC * 32 + q]; };
        float f[4], fk[KU];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = scale_of(vals.scale >> (8 * i) & 255);
#pragma unroll
        for (int i = 0; i < KU; ++i)
            fk[i] = scale_of(keys.scale[i] & 255);
#pragma unroll
        for (int n = 0; n < AHEAD - 1; ++n)
            a[n] = read(n);
        if (lane == 0)
            L.there[buf][wave] = keys.there;
        static_for<N>([&](auto n_) {
            constexpr int n = n_.value;
            if constexpr (n + AHEAD - 1 < N)
                a[(n + AHEAD - 1) % AHEAD] = read(n + AHEAD - 1);
            o[n % DC] = H::mfma32(a[n % AHEAD], p[n / DC], o[n % DC]);
            if constexpr (n * CHUNKS / N != (n + 1) * CHUNKS / N) {
                constexpr int chunk = n * CHUNKS / N;
                if constexpr (chunk < D / 32)
                    values<chunk>(vals, f, buf ^ 1);
                else
                    put_key((chunk - D / 32) / 4, (chunk - D / 32) % 4, keys, fk, buf);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }

    // NaN that were left out of the tile's values, for the rows that see them
    __device__ __forceinline__ void note(int buf, Whole table, int t, int head)
    {
        u32 odd = 0;
#pragma unroll
        for (int w = 0; w < kPromptWaves; ++w)
            odd |= L.nan[buf][w];
        if (__builtin_amdgcn_readfirstlane(odd))
#pragma unroll 1
            for (int j = 0; j < 32; ++j)
                if (token(t, j) >= lo && token(t, j) < hi)
                    nans |= nan_groups<D>(P, table, token(t, j), head);
    }
};

// A block of rows and the tokens it sees
struct Block {
    int first;              // its sequence's first query row
    int b, n, len;
    int i0, skip;           // begins with head `skip` of the sequence's query row i0
    int rows;               // 0: the number is no block's
    int least_lo, most_lo, least_hi, most_hi;   // tokens that some row, and that every row sees
    int begin, tiles;       // the first tile's first token; 1 tile at least
};

__device__ __forceinline__ Block block_of(const AttentionParams &P, int number)
{
    constexpr int ROWS = kPromptRows;
    Block k;
    int numbered;
    k.rows = k.tiles = 0;
    k.b = sequence_of(P, number, ROWS, &numbered);
    k.first = row_start(P, k.b);
    k.n = max(row_start(P, k.b + 1) - k.first, 0);
    const int row = (number - numbered) * ROWS;          // of the sequence's
    const int rows = k.n * P.group;
    if (row < 0 || row >= rows)
        return k;
    k.rows = min(rows - row, ROWS);
    k.len = length_of(P, k.b);
    k.i0 = row / P.group;
    k.skip = row - k.i0 * P.group;
    row_sees(P, k.len, k.n, k.i0, &k.least_lo, &k.least_hi);
    row_sees(P, k.len, k.n, k.i0 + (k.skip + k.rows - 1) / P.group, &k.most_lo, &k.most_hi);
    k.begin = k.least_lo / kTile * kTile;
    k.tiles = max((k.most_hi - k.begin + kTile - 1) / kTile, 1);
    return k;
}

// SHARED: the workers share all tiles evenly: those of kv head after kv head, of
// block after block in it.  Worker w has the tiles from total * w / workers on,
// consecutive shares go to one XCD, and a block that several have parts of is
// put together by a join kernel.  Otherwise a workgroup a block, those of a
// prompt's last rows, which have the most to do, first.
template <int DT, int D, int CAP, bool SHARED>
__global__ __launch_bounds__(64 * kPromptWaves) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2)))
void prompt_kernel(const AttentionParams P)
{
    typedef Prompt<DT, D, CAP> A_;
    typedef Half<DT> H;
    __shared__ PromptShared<D> L;
    constexpr int ROWS = kPromptRows;
    const int blocks = (int)P.blocks;
    int head, number, worker = 0;
    int64_t at, end, start, total = 0, workers = 0;
    Parts *parts = nullptr;
    if constexpr (SHARED) {
        const int lane = threadIdx.x & 63, id = (int)block_id();
        if (id >= P.workers)
            return;
        worker = P.workers % 8 ? id : id % 8 * (P.workers / 8) + id / 8;
        // the block that begins in this share and ends in another's, if there is one
        parts = parts_of<D, ROWS>(P, worker);
        if (threadIdx.x == 0)
            parts->count = 0;
        int64_t mine = 0, shares = 0;
        for (int n = lane; n < blocks; n += 64) {
            const int tiles = block_of(P, n).tiles;
            mine += tiles;
            shares += (tiles + kLeastTiles - 1) / kLeastTiles;
        }
        const int64_t of_head = sum_of_lanes(mine);
        total = of_head * P.c.heads;
        workers = max(min(sum_of_lanes(shares) * P.c.heads, (int64_t)P.workers), (int64_t)1);
        if (worker >= workers || total == 0)
            return;
        at = total * worker / workers;
        end = total * (worker + 1) / workers;
        head = (int)(at / of_head);
        // the block that tile `at` is of, and its first tile
        number = 0;
        start = head * of_head;
        while (true) {
            const int tiles = number + lane < blocks ? block_of(P, number + lane).tiles : 0;
            const int upto = sum_upto(tiles);
            const u64 past = __ballot(start + upto > at);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                number += l;
                start += (int)read_lane((u32)(upto - tiles), l);
                break;
            }
            start += (int)read_lane((u32)upto, 63);
            number += 64;
        }
    } else {
        const int64_t id = block_id(), behind = id / P.c.heads;
        if (behind >= blocks)
            return;
        head = (int)(id - behind * P.c.heads);
        number = blocks - 1 - (int)behind;
        at = start = 0;
        end = block_of(P, number).tiles;
    }
    const int64_t begin = at;

    A_ A(P, L);
    // a negative scale's sign goes to the queries, one of 0 makes them 0: the
    // scores' order is that of their products, and -inf times the factor -inf
    const u32 sign = CAP != kNoCap || P.scale >= 0 ? 0 : 0x80008000u, keep = CAP != kNoCap || P.scale != 0 ? ~0u : 0;
    A.factor = CAP != kNoCap ? 1.0f : P.scale != 0 ? fabsf(P.scale) * kLog2e : 1.0f;
    while (at < end) {
        Block k = block_of(P, number);
        while (k.tiles == 0 || at - start >= k.tiles) {
            start += k.tiles;
            if (++number >= blocks) {
                number = 0;
                ++head;
            }
            k = block_of(P, number);
        }
        const int from = (int)(at - start), to = (int)min((int64_t)k.tiles, from + (end - at));
        const Whole table = whole(P.tables + k.b * P.table_stride);
        const int r = A.wave * 32 + A.q, over = (k.skip + r) / P.group;
        row_sees(P, k.len, k.n, k.i0 + over, &A.lo, &A.hi);
        if (k.i0 + over >= k.n)
            A.lo = A.hi = 0;
        const uint16_t *from_q = P.q + (int64_t)(k.first + min(k.i0 + over, k.n - 1)) * P.q_token +
                                 (int64_t)(head * P.group + (k.skip + r - over * P.group)) * P.q_head;
#pragma unroll
        for (int i = 0; i < A.KC; ++i)
            A.qr[i] = (*(const u32x4 *)(from_q + 16 * i + 8 * A.h) & keep) ^ sign;
        A.top = kLowest;
        A.sum = 0.0f;
        A.nans = 0;
#pragma unroll
        for (int d = 0; d < A.DC; ++d)
            A.o[d] = f32x16{0};

        int t = k.begin + from * kTile;
        const int past = min(k.most_hi, k.begin + to * kTile);
        if (t < past) {
            auto is_edge = [&](int x) { return x < k.most_lo || x + kTile > k.least_hi; };
            RawKeys<D> keys;
            RawValues<D> vals;
            A.load(keys, table, k.len, t, head);
            A.load(vals, table, k.len, t, head);
            __syncthreads();             // the block before is done with LDS
            A.put(keys, 0);
            A.clean(vals, 0, k.least_lo, k.most_hi, t, is_edge(t));
            A.put(vals, 0);
            A.load(keys, table, k.len, t + kTile, head);
            A.put(keys, 1);
            A.load(keys, table, k.len, t + 2 * kTile, head);
            A.load(vals, table, k.len, t + kTile, head);
            __syncthreads();
            A.products(0);
            A.settle(0, t, is_edge(t));
            __syncthreads();
            int buf = 0;
            // A step has the weights and values of the tile at t and the products of
            // the next one: these while the weights are taken, the values while what
            // comes in, the one after's keys and the next one's values, goes to LDS.
            while (t + kTile < past) {
                if (is_edge(t))
                    A.note(buf, table, t, head);
                A.clean(vals, buf ^ 1, k.least_lo, k.most_hi, t + kTile, is_edge(t + kTile));
                f32x16 next[2];
                A.products_and_weights(next, buf ^ 1);
                A.values_and_puts(buf, vals, keys);
                t += kTile;
                buf ^= 1;
                A.load(keys, table, k.len, t + 2 * kTile, head);
                A.load(vals, table, k.len, t + kTile, head);
                A.s[0] = next[0];
                A.s[1] = next[1];
                A.settle(buf, t, is_edge(t));
                __syncthreads();
            }
            if (is_edge(t))
                A.note(buf, table, t, head);
            A.weights();
            A.add(buf);
        }

        const bool all = !SHARED || (from == 0 && to == k.tiles);
        float *rec = SHARED ? record<D, ROWS>(P, worker, at == begin) : nullptr;
        const u32 bits = __float_as_uint(A.sum);
        auto sums = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
        const float sum = __uint_as_float(sums[0]) + __uint_as_float(sums[1]);
        auto odd = __builtin_amdgcn_permlane32_swap(A.nans, A.nans, false, false);
        const u32 nans = odd[0] | odd[1];
        if (r < k.rows) {
            const int64_t row = (int64_t)(k.first + k.i0 + over) * P.q_heads + head * P.group + (k.skip + r - over * P.group);
            const float inv = !all ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
            // register i of product d is row x = 8 (i / 4) + 4 h + i % 4 of it, channel
            // x % 16 D/16 + 2 d + x / 16: D/16 channels side by side in two registers
            // of all the products
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c0 = (8 * j + 4 * A.h + e) * (D / 16);
                    const float nan = nans >> (c0 / 32) & 1 ? __builtin_nanf("") : 0.0f;
                    float v[2 * A.DC];
#pragma unroll
                    for (int d = 0; d < A.DC; ++d) {
                        v[2 * d] = A.o[d][4 * j + e] * inv + nan;
                        v[2 * d + 1] = A.o[d][4 * j + 8 + e] * inv + nan;
                    }
                    if (!all) {
                        float *out = rec + 2 * ROWS + r * D + c0;
#pragma unroll
                        for (int d = 0; d < 2 * A.DC; d += 4)
                            *(float4 *)(out + d) = float4{v[d], v[d + 1], v[d + 2], v[d + 3]};
                        continue;
                    }
                    uint16_t *out = P.out + row * D + c0;
#pragma unroll
                    for (int d = 0; d < 2 * A.DC; d += 4)
                        *(u32x2 *)(out + d) = u32x2{H::pack(v[d], v[d + 1]), H::pack(v[d + 2], v[d + 3])};
                }
            if (A.h == 0) {
                if (!all) {
                    rec[r] = A.top;
                    rec[ROWS + r] = sum;
                } else if (P.lse) {
                    P.lse[row] = sum == 0.0f
                                     ? -__builtin_inff()
                                     : (A.top + __builtin_amdgcn_logf(sum) - Softmax<DT>::kShift) * kLn2;
                }
            }
        }
        if (SHARED && from == 0 && threadIdx.x == 0) {
            Join *j = join_of<D, ROWS>(P, number, head);
            j->from = worker;
            j->parts = 0;
            if (!all) {
                j->parts = (int)((workers * (at + k.tiles) - 1) / total) - worker + 1 |
                           (at == begin ? kWholeShare : 0);
                parts->row = (int64_t)(k.first + k.i0) * P.q_heads + head * P.group;
                parts->skip = k.skip;
                parts->rows = k.rows;
                parts->count = j->parts;
            }
        }
        at += to - from;
    }
}

int prompt_workers(int cus, int D) { return cus * (D == 256 ? 1 : 2); }

template <int DT, int D, int CAP> hipError_t launch_cap(const AttentionParams &p, hipStream_t s)
{
    if (!p.workspace) {
        prompt_kernel<DT, D, CAP, false><<<grid_of(p.blocks * p.c.heads), 64 * kPromptWaves, 0, s>>>(p);
        return hipGetLastError();
    }
    prompt_kernel<DT, D, CAP, true><<<grid_of(p.workers), 64 * kPromptWaves, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_join_shares<DT, D, kPromptRows>(p, s);
}

template <int DT, int D> hipError_t launch(const AttentionParams &p, hipStream_t s)
{
    const Cap cap = cap_of(p.softcap);
    return cap == kNoCap ? launch_cap<DT, D, kNoCap>(p, s)
           : cap == kLow ? launch_cap<DT, D, kLow>(p, s)
                         : launch_cap<DT, D, kHigh>(p, s);
}

template <int DT> hipError_t launch_width(const AttentionParams &p, int D, hipStream_t s)
{
    return D == 64 ? launch<DT, 64>(p, s) : D == 128 ? launch<DT, 128>(p, s) : launch<DT, 256>(p, s);
}

}  // namespace

uint64_t prompt_workspace_floats(int64_t T, int B, int q_heads, int kv_heads, int head_dim, int cus, int64_t max_len)
{
    const int workers = prompt_workers(cus, head_dim);
    const int64_t blocks = most_blocks(T, B, q_heads / kv_heads, kPromptRows, true) * kv_heads;
    // Tiles are shared out where blocks are few and sequences may be long: joining
    // costs as much as ten tiles (one sequence, 8 kv heads of 5 heads of 128
    // channels: 640 rows over 1024 tokens 32 us by blocks, 47 shared, 700 over 2048
    // 53 and 61, 512 over 4096 95 and 73, over 16384 353 and 193, 2000 over 16384 785
    // and 660).  More than two blocks for every place of a workgroup fill the chip by
    // themselves, the longest first (4096 rows over 16384 tokens: 1323 and 1360).
    // With a share of at least 1, 4 or 12 tiles 64 rows over 4096 tokens of a table of
    // 65536 take 41, 37 and 46 us.
    if (blocks > 2 * workers || max_len <= kSharedTokens)
        return 0;
    return join_floats(workers, blocks, kPromptRows, head_dim) + parts_floats(workers);
}

hipError_t launch_prompt(const AttentionParams &a, int head_dim, int dtype, int cus, hipStream_t s)
{
    AttentionParams p = a;
    p.blocks = most_blocks(p.T, p.B, p.group, kPromptRows, p.q_starts != nullptr);
    p.workers = prompt_workers(cus, head_dim);
    return dtype == MHC_BF16 ? launch_width<MHC_BF16>(p, head_dim, s) : launch_width<MHC_F16>(p, head_dim, s);
}

}  // namespace mhc
