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
//
// Bytes bound it, D + D/16 a token and kv head: 520 MB of cache are read at 5.9 TB/s
// (a large copy: 6.05), 64 sequences of up to 8192 tokens, 8 kv heads of 128
// channels, 268 MB, in 45 us and 5.5 to join; short sequences are bound by latency, 4.4
// us for one token, 0.35 us each 128 tokens more.  Eight waves a block instead of four
// are no faster there (one token 4.8 us, 1003 tokens 8.2 for 8.3).
#include <hip/hip_runtime.h>

#include "attention_join.h"

namespace mhc {
namespace {

constexpr int kRows = 16;                 // query rows a block: heads of one kv head, tokens in order
constexpr int kStep = 32;                 // tokens a wave's step
constexpr int kAttnWaves = 4;             // of a workgroup
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kQuantum = kStep * kAttnWaves;   // tokens that a workgroup's waves take side by side
constexpr int kMostBalanced = 1024;       // sequences whose lengths a worker adds up
constexpr int kLeastQuanta = 4;           // of a worker's share, where a block has as many
constexpr int kAloneTokens = 2048;        // of sequences whose blocks a workgroup each has alone
constexpr int kAloneBlocks = 8;           // a CU, of which each has a workgroup alone
constexpr int64_t kPromptWork = 3 << 23;  // rows times heads times tokens

// A sequence's share of the work: blocks of rows, and the quanta of tokens that
// some row of it sees, the same number for every block and kv head.
struct Sequence {
    int first;          // its first query row
    int n;              // query rows
    int rows;           // times heads of a kv head
    int len;            // cached tokens
    int lo;             // first quantum's first token
    int blocks;         // of kRows rows
    int quanta;
};

__device__ __forceinline__ Sequence sequence(const AttentionParams &P, int b)
{
    Sequence s;
    s.first = row_start(P, b);
    s.n = max(row_start(P, b + 1) - s.first, 0);
    s.rows = s.n * P.group;
    s.len = length_of(P, b);
    int hi;
    row_sees(P, s.len, s.n, 0, &s.lo, &hi);
    s.lo = s.lo / kStep * kStep;
    s.blocks = (s.rows + kRows - 1) / kRows;
    s.quanta = max((s.len - s.lo + kQuantum - 1) / kQuantum, 1);
    return s;
}

// A worker's share of all quanta, which are those of sequence after sequence, of
// kv head after kv head in it, of block after block.  Their number is below 2^31,
// unless starts fall: then nobody has any.
struct Share {
    int begin, end;
    int each, over;     // quanta of a worker; workers that have one more
    int b;              // the sequence of quantum `begin`
    int start;          // that sequence's first quantum
};

__device__ __forceinline__ int quanta_of(const AttentionParams &P, int b, int *shares)
{
    if (b >= P.B)
        return 0;
    const Sequence s = sequence(P, b);
    *shares += s.blocks * P.c.heads * ((s.quanta + kLeastQuanta - 1) / kLeastQuanta);
    return s.blocks * s.quanta * P.c.heads;
}

// The first `over` workers have one quantum more than the others' `each`
__device__ __forceinline__ int share_start(const Share &h, int w) { return w * h.each + min(w, h.over); }

// The worker whose share holds that quantum
__device__ __forceinline__ int share_of(const Share &h, int quantum)
{
    const int more = h.over * (h.each + 1);
    return quantum < more ? quantum / (h.each + 1) : h.over + (quantum - more) / h.each;
}

__device__ Share share(const AttentionParams &P, int worker)
{
    const int lane = threadIdx.x & 63;
    Share h;
    // A worker for kLeastQuanta quanta of a block, if there are as many: with 1, 4 and
    // 12 a sequence of 32768 tokens takes 20, 17 and 21 us, one of 4096 9.8, 11.1 and 18
    int shares = 0, own = quanta_of(P, lane, &shares), upto = sum_upto(own);
    int total = (int)read_lane((u32)upto, 63), many = own >> 12;
    for (int b0 = 64; b0 < P.B; b0 += 64) {
        const int next = quanta_of(P, b0 + lane, &shares);
        total = (int)((u32)total + read_lane((u32)sum_upto(next), 63));
        many += next >> 12;
    }
    shares = (int)read_lane((u32)sum_upto(shares), 63);
    // a lane's `many` is below 2^23; with their sum at most 2^19 the total is below
    // 2^31 + 2^12 kMostBalanced
    if ((int)read_lane((u32)sum_upto(many), 63) > 1 << 19 || total < 0)
        total = 0;
    const int workers = max(min(shares, P.workers), 1);
    h.each = total / workers;
    h.over = total - h.each * workers;
    h.begin = worker < workers ? share_start(h, worker) : total;
    h.end = worker < workers ? share_start(h, worker + 1) : total;
    h.b = h.start = 0;
    if (h.begin == h.end)
        return h;
    int before = 0;
    for (int b0 = 0;; b0 += 64) {
        if (b0 > 0) {
            own = quanta_of(P, b0 + lane, &shares);
            upto = sum_upto(own);
        }
        const u64 past = __ballot(before + upto > h.begin);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            h.b = b0 + l;
            h.start = before + (int)read_lane((u32)(upto - own), l);
            return h;
        }
        before += (int)read_lane((u32)upto, 63);
    }
}

// 32 tokens of a kv head as a lane holds them
template <int D> struct Tile {
    u32 k[2][D / 32];                    // token c of each half, its channels' piece g and, D = 256, g + 4
    u32 ks[2][(D + 127) / 128];
    u32 v[8][(D + 127) / 128];           // tokens 4g .. 4g + 3 of each half, chunk c of the channels
    u32 vs[2];
    bool there[2];
};

// The rows of a block as a lane of row c sees them
struct Rows {
    int lo, hi;              // tokens that the lane's row sees
    int most_lo, least_hi;   // that every row of the block sees
    int least_lo, most_hi;   // that some row of it sees
};

template <int DT, int D, int CAP> struct Attention {
    typedef Half<DT> H;
    typedef Softmax<DT> S;
    static constexpr int KC = D / 32;        // products of a score: 8 channels a lane each
    static constexpr int VC = D / 16;        // channels of V a lane
    static constexpr int VB = VC / 2;        // bytes of them

    const AttentionParams &P;
    const int c, g;
    u32 at_k, at_v, at_ks, at_vs;            // the lane's bytes in a tile
    u32x4 q[KC];
    f32x4 acc[VC];
    float top, sum;
    u32 nans;                // groups of V's channels that a NaN reaches in this lane's row

    __device__ Attention(const AttentionParams &p) : P(p), c(threadIdx.x & 15), g(threadIdx.x >> 4 & 3)
    {
        const int ps = P.c.page_size;
        at_k = c * (D / 2) + g * (D == 64 ? 8 : 16);
        at_v = cache_codes(ps, D, 1) + 4 * g * (D / 2) + c * VB;
        at_ks = cache_scales(ps, D, 0) + (D == 64 ? g / 2 : g) * ps + c;
        at_vs = cache_scales(ps, D, 1) + c * VC / 32 * ps + 4 * g;
    }

    // Rows of the block that begins with head `skip` of the sequence's query row
    // i0: the lane's query row, counted in the sequence, and head
    __device__ void load_q(const Sequence &s, int i0, int skip, int head)
    {
        const int over = (skip + c) / P.group, i = i0 + over;
        if (i < s.n) {
            const uint16_t *at =
                P.q + (int64_t)(s.first + i) * P.q_token + (int64_t)(head * P.group + (skip + c - over * P.group)) * P.q_head;
#pragma unroll
            for (int j = 0; j < KC; ++j)
                q[j] = *(const u32x4 *)(at + (D == 64 ? 16 * g + 8 * j : 32 * (g + 4 * (j / 4)) + 8 * (j % 4)));
        } else {
#pragma unroll
            for (int j = 0; j < KC; ++j)
                q[j] = u32x4{0, 0, 0, 0};
        }
    }

    __device__ Rows rows_of(const Sequence &s, int i0, int skip)
    {
        Rows w;
        const int i = i0 + (skip + c) / P.group, last = min(i0 + (skip + kRows - 1) / P.group, s.n - 1);
        row_sees(P, s.len, s.n, i0, &w.least_lo, &w.least_hi);
        row_sees(P, s.len, s.n, last, &w.most_lo, &w.most_hi);
        row_sees(P, s.len, s.n, i, &w.lo, &w.hi);
        if (i >= s.n)
            w.lo = w.hi = 0;
        return w;
    }

    __device__ __forceinline__ void load(Tile<D> &x, Whole table, int len, int t, int head)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int32_t page, at;
            x.there[h] = cache_page(P.c, table, len, t + 16 * h, &page, &at);
            const Page from = page_of<D>(P, page, head);
            const int codes = at * (D / 2);
            if constexpr (D == 64) {
                const u32x2 w = from.load64(at_k, codes);
                x.k[h][0] = w[0];
                x.k[h][1] = w[1];
            } else {
#pragma unroll
                for (int j = 0; j < KC / 4; ++j) {
                    const u32x4 w = from.load128(at_k + 64 * j, codes);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x.k[h][4 * j + i] = w[i];
                }
            }
#pragma unroll
            for (int j = 0; j < (D + 127) / 128; ++j)
                x.ks[h][j] = from.load32(at_ks, at + 4 * j * P.c.page_size);      // its low byte
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32 v = at_v + j * (D / 2);
                if constexpr (D == 64) {
                    x.v[4 * h + j][0] = from.load32(v, codes);      // its low half
                } else if constexpr (D == 128) {
                    x.v[4 * h + j][0] = from.load32(v, codes);
                } else {
                    const u32x2 w = from.load64(v, codes);
                    x.v[4 * h + j][0] = w[0];
                    x.v[4 * h + j][1] = w[1];
                }
            }
            x.vs[h] = from.load32(at_vs, at);
        }
    }

    // Hides what the lane's row does not see of the 32 tokens at t0
    __device__ void mask(Tile<D> &x, float v[8], const Rows &rows, Whole table, int t0, int head)
    {
        u32 nan_tokens = 0, seen = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = t0 + 16 * (i / 4) + 4 * g + i % 4;
            const bool sees = x.there[i / 4] && t >= rows.lo && t < rows.hi;
            seen |= (u32)sees << i;
            v[i] = sees ? v[i] : -__builtin_inff();
            // what no row sees may be anything, infinite too; a NaN that only
            // some rows see goes by `nans` to those
            const bool valid = x.there[i / 4] && t >= rows.least_lo && t < rows.most_hi;
#pragma unroll
            for (int j = 0; j < (D + 127) / 128; ++j)
                x.v[i][j] = valid ? x.v[i][j] : 0;
            const u32 byte = x.vs[i / 4] >> (8 * (i % 4)) & 255;
            if (byte == 255 || !valid)
                x.vs[i / 4] &= ~(255u << (8 * (i % 4)));
            nan_tokens |= (u32)(byte == 255 && valid);
        }
        if (__any(nan_tokens != 0))
#pragma unroll 1
            for (int i = 0; i < 8; ++i)
                if (seen >> i & 1)
                    nans |= nan_groups<D>(P, table, t0 + 16 * (i / 4) + 4 * g + i % 4, head);
    }

    __device__ __forceinline__ void step(Tile<D> &x, const Rows &rows, Whole table, int t0, int head)
    {
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 s = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                const float f = scale_of(x.ks[h][D == 256 ? j / 4 : 0] & 255);
                const u32 w = x.k[h][j];
                const u32x4 a = {H::template from_fp4<0>(w, f), H::template from_fp4<1>(w, f),
                                 H::template from_fp4<2>(w, f), H::template from_fp4<3>(w, f)};
                s = H::mfma16(a, q[j], s);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[4 * h + i] = s[i];
        }
        if constexpr (CAP != kNoCap) {
            cap<8, CAP>(P, v);
        } else {
            const float f = P.scale * kLog2e;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= f;
        }
        if (!(t0 >= rows.most_lo && t0 + kStep <= rows.least_hi && x.there[0] && x.there[1]))
            mask(x, v, rows, table, t0, head);
        const float most =
            fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
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

    // The wave's part of quanta [from, to) of the block: each step's tokens are
    // asked for before the step before
    __device__ void run(const Sequence &s, const Rows &rows, Whole table, int head, int from, int to, int wave)
    {
        top = kLowest;
        sum = 0.0f;
        nans = 0;
#pragma unroll
        for (int m = 0; m < VC; ++m)
            acc[m] = f32x4{0, 0, 0, 0};
        int t = s.lo + from * kQuantum + wave * kStep;
        const int end = min(s.len - s.lo, to * kQuantum) + s.lo;
        if (t >= end)
            return;
        // no branch stands about the loads, so that each wait is for one step's
        // and not for those behind it; past the end they read page 0
        Tile<D> a, b;
        load(a, table, s.len, t, head);
        while (true) {
            load(b, table, s.len, t + kQuantum, head);
            step(a, rows, table, t, head);
            t += kQuantum;
            if (t >= end)
                break;
            load(a, table, s.len, t + kQuantum, head);
            step(b, rows, table, t, head);
            t += kQuantum;
            if (t >= end)
                break;
        }
    }
};

template <int D> struct Shared {
    float top[kAttnWaves][kRows], sum[kAttnWaves][kRows];
    float o[kAttnWaves][kRows][D + 4];
};

// BALANCED: the workers share all quanta evenly, and a block that several have
// parts of is put together by attention_join_kernel.  Otherwise a workgroup a block.
template <int DT, int D, int CAP, bool BALANCED>
__global__ __launch_bounds__(kAttnThreads)
    __attribute__((amdgpu_waves_per_eu(2))) void attention_kernel(const AttentionParams P)
{
    __shared__ Shared<D> L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = block_id();
    Sequence s;
    Share h;
    int at, end, start = 0, b, block = 0, head = 0;
    if constexpr (BALANCED) {
        if (id >= P.workers)
            return;
        h = share(P, (int)id);
        at = h.begin;
        end = h.end;
        b = h.b;
        start = h.start;
        if (at == end)
            return;
        s = sequence(P, b);
    } else {
        const int64_t behind = id / P.c.heads;
        if (behind >= P.blocks)
            return;
        const int number = (int)behind;
        int first;
        b = sequence_of(P, number, kRows, &first);
        s = sequence(P, b);
        if (number < first || number - first >= s.blocks)
            return;
        head = (int)(id - behind * P.c.heads);
        block = number - first;
        at = 0;
        end = s.quanta;
    }
    Attention<DT, D, CAP> A(P);
    const int begin = at;
    while (at < end) {
        int from = 0;
        if constexpr (BALANCED) {
            while (at - start >= s.blocks * P.c.heads * s.quanta) {
                start += s.blocks * P.c.heads * s.quanta;
                s = sequence(P, ++b);
            }
            const int index = (at - start) / s.quanta;
            from = at - start - index * s.quanta;
            head = index / s.blocks;
            block = index - head * s.blocks;
        }
        const int to = min(s.quanta, from + (end - at));
        const int row = block * kRows, i0 = row / P.group, skip = row - i0 * P.group;
        const Rows rows = A.rows_of(s, i0, skip);
        A.load_q(s, i0, skip, head);
        A.run(s, rows, whole(P.tables + b * P.table_stride), head, from, to, wave);

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
        const int count = min(s.rows - row, kRows);
        float *rec = record<D, kRows>(P, id, at == begin);
        for (int e = threadIdx.x; e < count * (D / 4); e += kAttnThreads) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            float most = kLowest, all = 0.0f;
            float4 o = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w)
                most = fmaxf(most, L.top[w][r]);
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w) {
                all += L.sum[w][r] * __builtin_amdgcn_exp2f(L.top[w][r] - most);
                const float4 x = *(const float4 *)&L.o[w][r][d];
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
            }
            if (whole) {
                store<DT, D>(P, s.first + i0, skip + r, head, d, o, most, all);
            } else {
                *(float4 *)(rec + 2 * kRows + r * D + d) = o;
                if (d == 0) {
                    rec[r] = most;
                    rec[kRows + r] = all;
                }
            }
        }
        if constexpr (BALANCED)
            if (from == 0 && threadIdx.x == 0) {
                Join *j = join_of<D, kRows>(P, first_number(P, b, s.first, kRows) + block, head);
                j->from = (int)id;
                j->parts = whole ? 0
                                 : (share_of(h, at + s.quanta - 1) - (int)id + 1) |
                                       (at == begin ? kWholeShare : 0);
            }
        __syncthreads();
        at += to - from;
    }
}

// As many as have room.  Two a CU are faster where all lengths are alike (64
// sequences of 8192 tokens 109 us for 120), slower where they are not (of 1 .. 8192
// 72 for 68, 32 of 1 .. 4096 38 for 31); one is slower still there (90, 45).
int workers_of(int cus, int D) { return cus * (D == 256 ? 2 : 3); }

template <int DT, int D, int CAP> hipError_t launch_cap(const AttentionParams &p, hipStream_t s)
{
    const int64_t segments = p.blocks * p.c.heads;
    if (p.workspace)
        attention_kernel<DT, D, CAP, true><<<grid_of(p.workers), kAttnThreads, 0, s>>>(p);
    else
        attention_kernel<DT, D, CAP, false><<<grid_of(segments), kAttnThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT, int D> hipError_t launch(const AttentionParams &p, hipStream_t s)
{
    const Cap cap = cap_of(p.softcap);
    const hipError_t e = cap == kNoCap ? launch_cap<DT, D, kNoCap>(p, s)
                         : cap == kLow ? launch_cap<DT, D, kLow>(p, s)
                                       : launch_cap<DT, D, kHigh>(p, s);
    if (e != hipSuccess || !p.workspace)
        return e;
    return launch_join<DT, D, kRows>(p, s);
}

template <int DT> hipError_t launch_width(const AttentionParams &p, int D, hipStream_t s)
{
    return D == 64 ? launch<DT, 64>(p, s) : D == 128 ? launch<DT, 128>(p, s) : launch<DT, 256>(p, s);
}

// Whether it is prompt_kernel's: sequences of 64 rows on average (64 sequences of
// 4096 tokens, 8 kv heads of 128 channels: at 40 rows each 144 us by blocks of 16
// rows and 162 by 128, at 80 243 and 213), and work enough for its tiles of 128
// rows to fill the chip, rows times heads times tokens (8 kv heads, 5 heads each: 64
// rows over 1024 tokens 11 and 29 us, 512 31.3 and 30.8; 64 over 4096 30 and 37, 256
// 59 and 57; 32 over 16384 40.7 and 40.4; 8 times 64 over 1024 30.8 and 31.3).  One
// kernel for the whole call: single rows beside a prompt fill a block of 128 rows with
// their heads (63 of them beside 2048 rows, each over 8192 tokens, 703 us; the two as
// calls of their own 370 and 105).
bool prompts(int64_t T, int B, int q_heads, int group, int64_t max_len)
{
    return T * group >= (int64_t)B * 64 && T * q_heads >= kPromptWork / max_len;
}

}  // namespace

uint64_t attention_workspace_floats(int64_t T, int B, int q_heads, int kv_heads, int head_dim, int cus,
                                    int64_t max_len)
{
    const int group = q_heads / kv_heads;
    if (max_len == 0)
        return 0;
    if (prompts(T, B, q_heads, group, max_len))
        return prompt_workspace_floats(T, B, q_heads, kv_heads, head_dim, cus, max_len);
    // Quanta are shared out but where a workgroup a block does better:
    // - short sequences: a second launch and its parts cost as much as 1500 tokens
    //   (one sequence, 2 kv heads of 128 channels: 1024 tokens 9.6 us alone and 11.0
    //   shared, 2048 14.8 and 11.1);
    // - longer ones, if there is a block for every CU (64 sequences of 4096 tokens,
    //   8 kv heads: 51 and 63 us; of 1 .. 4096 34 and 44; of 8192 107 and 120; one of
    //   8192 among 63 of 512 49 and 21, for which they end at 4096);
    // - many blocks for every CU (300 sequences of 2304 tokens: 141 and 156; 40 heads on
    //   8, 256 of 5000 tokens 221 and 254, of 1 .. 8192 212 and 225).  That holds for
    //   lengths alike: of 512 .. 65536, even over their logarithm, 732 and 582, and one
    //   long sequence among 255 of 512 is one workgroup's way through it, one of 8192
    //   71 and 50, of 32768 195 and 55, of 131072 699 and 73;
    // and where there are more sequences than a worker adds up.
    const int64_t blocks = most_blocks(T, B, group, kRows, true) * kv_heads;
    if (B > kMostBalanced || blocks >= (int64_t)cus * kAloneBlocks ||
        max_len <= (blocks < cus ? kAloneTokens : 2 * kAloneTokens))
        return 0;
    return join_floats(workers_of(cus, head_dim), blocks, kRows, head_dim);
}

hipError_t launch_attention(const AttentionParams &a, int head_dim, int dtype, int cus, hipStream_t s)
{
    if (prompts(a.T, a.B, a.q_heads, a.group, a.seen))
        return launch_prompt(a, head_dim, dtype, cus, s);
    AttentionParams p = a;
    p.blocks = most_blocks(p.T, p.B, p.group, kRows, p.q_starts != nullptr);
    p.workers = workers_of(cus, head_dim);
    // quanta are counted in 31 bits; a window's first token may lie inside one
    if (p.blocks * p.c.heads * (p.seen / kQuantum + 2) > INT32_MAX)
        p.workspace = nullptr;
    return dtype == MHC_BF16 ? launch_width<MHC_BF16>(p, head_dim, s) : launch_width<MHC_F16>(p, head_dim, s);
}

}  // namespace mhc
