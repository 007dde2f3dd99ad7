// route_kernels.hip -- routing of tokens to experts from their logits.
//
// For each token, with logits l [E], an optional bias b [E] that balances
// the experts' load, and G groups of E / G consecutive experts:
//   s   = softmax(l)  or  1 / (1 + exp(-l))
//   key = s + b, or l without a bias (the scores' order, told apart also
//   where scores are equal in binary64)
//   the `keep` groups whose best key (top 1), or whose two best s + b together
//   (top 2), are the largest stay open; of their experts the k of the largest
//   keys are chosen, largest first
//   w   = s of the chosen, divided by their sum (renorm), times scale
// Equal keys, and equal sums of groups, go to the lowest index.  The bias
// steers the choice only, never the weights.
//
// Keys are held in binary64.  Two experts' binary32 scores are equal or in
// the wrong order whenever they lie within a few units of the last place,
// which at 256 experts happens somewhere in almost every batch; the choice
// would then hang on the rounding of exp and on the order of the softmax's
// sum.  In binary64 it is the definition's for all but bit-equal scores.
//
// Masks: a logit of -inf, or a bias of -inf, takes an expert out.  A key
// missing from a sum of two counts as -1e30: groups with more experts left
// come first.  Where fewer than k experts are left the other slots hold id -1,
// weight 0; a row with none left has nothing else.  A NaN logit (and +inf under
// softmax) is taken out likewise and turns the row's weights to NaN, so ids
// always lie in -1 .. E - 1 and are distinct but for -1.
//
// Reading the logits would take 2.8 us at T = 16384, E = 256 (8 groups,
// sigmoid, bias), the launch 2.  With a wave a token in binary64 it took 34 us;
// four tokens a wave 12.0 to 12.3.  Past that instructions bound it: 1027
// vector ones a wave, and each 16384 tokens more cost 6.2 to 7.2 us, about what
// these take issued back to back (T = 32768 19 us, 65536 33, 131072 58).  Below
// it is latency: 6.0 us at T = 1, 7.3 at T = 4096.  At 16384 all waves, four a
// SIMD, are resident at once and wait for their logits together, so that first
// wait and the last stores are not hidden behind another wave's instructions.
// A row that has to be done again in binary64 costs 3 us by itself: with those
// whose groups were close done so, T = 4160 took 9.6 where it then took 7.6.
// Where a mask sends many rows there, it shows: T = 16384 with one of the eight
// groups out in every row 48 us; without groups, with 30% of the rows short of
// experts 31, and softmax over logits with 30% of them at -1e9 43 for 9.
#include <hip/hip_runtime.h>

#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

typedef uint32_t u32;
typedef uint64_t u64;

constexpr double kMissing = -1e30;

template <class T>
__device__ __forceinline__ float logit(const void *p, int64_t i)
{
    return (float)static_cast<const T *>(p)[i];
}

// LDS writes of the wave's lanes before its reads that follow
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------- in binary64 --
//
// One wave a token; lane l holds experts EPL l .. EPL l + EPL - 1.  Groups of
// any size go through LDS (`keys`, the wave's own).
template <class T, int EPL>
__device__ __forceinline__ void route_token(const RouteParams &P, int64_t t, int lane,
                                            double *keys)
{
    const int E = P.E;
    const double inf = __builtin_inf();
    double l[EPL], s[EPL], key[EPL];
    bool bad = false;
    double top = -inf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = EPL * lane + j;
        const float v = e < E ? logit<T>(P.logits, t * E + e) : -__builtin_inff();
        const bool nan = v != v || (!P.sigmoid && v == __builtin_inff());
        bad |= nan;
        l[j] = nan ? -inf : (double)v;
        top = fmax(top, l[j]);
    }
    bad = __ballot(bad) != 0;
    if (P.sigmoid) {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            s[j] = 1.0 / (1.0 + exp(-l[j]));
    } else {
        top = wave_max(top);
        double total = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            s[j] = l[j] == -inf ? 0.0 : exp(l[j] - top);
            total += s[j];
        }
        total = wave_sum(total);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            s[j] = total > 0.0 ? s[j] / total : 0.0;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = EPL * lane + j;
        key[j] = !P.bias ? l[j] : e < E ? s[j] + (double)P.bias[e] : -inf;
        if (l[j] == -inf || key[j] != key[j])
            key[j] = -inf;
    }
    if (P.groups > 1) {
        const int size = E / P.groups;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            keys[EPL * lane + j] = P.bias || P.top == 1 || l[j] == -inf ? key[j] : s[j];
        wave_fence();
        double first = -inf, second = -inf;
        if (lane < P.groups)
            for (int i = 0; i < size; ++i) {
                const double v = keys[lane * size + i];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
        const double sum = P.top == 1 ? first
                                      : (first == -inf ? kMissing : first) +
                                            (second == -inf ? kMissing : second);
        wave_fence();
        keys[lane] = sum;
        wave_fence();
        int rank = 0;
        for (int g = 0; g < P.groups; ++g)
            rank += keys[g] > sum || (keys[g] == sum && g < lane);
        const u64 open = __ballot(lane < P.groups && rank < P.keep);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = EPL * lane + j;
            if (e < E && !(open >> (e / size) & 1))
                key[j] = -inf;
        }
    }
    // lane i keeps the i-th chosen expert and its score
    int id = -1;
    double w = 0.0, sum = 0.0;
    for (int i = 0; i < P.k; ++i) {
        double mine = key[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j)
            mine = fmax(mine, key[j]);
        const double best = wave_max(mine);
        if (best == -inf)
            break;
        const int from = __builtin_ctzll(__ballot(mine == best));
        int at = 0;
        double score = 0.0;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j)
            if (key[j] == best) {
                at = EPL * lane + j;
                score = s[j];
            }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane == from && EPL * lane + j == at)
                key[j] = -inf;
        at = __shfl(at, from);
        score = __shfl(score, from);
        sum += score;
        if (lane == i) {
            id = at;
            w = score;
        }
    }
    if (lane < P.k) {
        if (P.renorm)
            w = sum > 0.0 ? w / sum : 0.0;
        P.weights[t * P.k + lane] = bad ? __builtin_nanf("") : (float)(w * (double)P.scale);
        P.ids[t * P.k + lane] = id;
    }
}

template <class T, int EPL>
__global__ __launch_bounds__(64) void route_kernel(RouteParams P, int64_t tokens)
{
    __shared__ double keys[EPL * 64];
    const int64_t t = block_id();
    if (t < tokens)
        route_token<T, EPL>(P, t, threadIdx.x, keys);
}

// ----------------------------------------------------- four tokens a wave --
//
// The choice from binary32 keys wherever they prove it right.  A row of 16
// lanes takes a token, up to EPL experts a lane; each group has a power of two
// of the lanes, as many as there are for all.  A key is a whole number: the
// score's place between the row's lowest and highest, below 2^22, above the
// expert's index (inverted, so that the lowest index of a place is the largest
// number); place 0 is no expert.  One maximum then gives place and index at
// once.
//
// Each lane sorts out its four largest keys (76 minima and maxima for 16);
// its two largest give the groups' sums, and the choice takes the largest
// head of the row's lanes and moves that lane on, 12 instructions a chosen
// expert.  Only where a lane runs out of its four does the wave look through
// all keys again for every next one.
//
// Scores are binary32 with an error of at most `delta`, so two keys further
// apart than `need` places are in the order of the binary64 ones.  Where
// neighbours among the k largest are nearer than that, or the k-th and the
// next (then the choice goes on, up to 16, to a gap that is wide enough), the
// binary64 keys of those chosen are compared; where groups are too close on
// both sides of the border (one row in 4000 at 256 experts in 8 groups), their
// binary64 sums, if the experts that make them are certain.  What is left (it
// is not, some experts are but fewer than asked for, infinities, NaN) goes
// through route_token afterwards, which keeps its wave for 3 us.  Without a
// bias the order is the logits' own: bf16 and fp16 logits fit a place whole,
// and no row is too close to call (equal logits are common there and are
// ties).
//
// Weights are binary64 of the k chosen.
constexpr int kIndexBits = 9;
constexpr u32 kIndexMask = (1u << kIndexBits) - 1;
constexpr float kSpan = 0x3p20f, kPlaces = 0x1p22f - 1.0f;   // of the places; the last one
constexpr int kRowWaves = 4;

template <class T>
struct Whole {   // low bits of a binary32 value that T's have zero
    static constexpr int kShift = 0;
};
template <>
struct Whole<__bf16> {
    static constexpr int kShift = 16;
};
template <>
struct Whole<_Float16> {
    static constexpr int kShift = 13;
};

// binary32 bits in the order of the values, -0 with +0
__device__ __forceinline__ u32 in_order(float v)
{
    const u32 b = __float_as_uint(v + 0.0f);
    return b ^ ((u32)((int)b >> 31) | 0x80000000u);
}

// The first `count` of EPL values, the rest as `none`; four at a time
template <class T, int EPL>
__device__ __forceinline__ void load_row(const T *p, int count, float none, float (&v)[EPL])
{
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T4 T4_any __attribute__((aligned(sizeof(T))));
    T4 q[EPL / 4];
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
        if (j + 4 <= count) {
            q[j / 4] = *reinterpret_cast<const T4_any *>(p + j);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j + i < count)
                    q[j / 4][i] = p[j + i];
        }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        v[j] = j < count ? (float)q[j / 4][j % 4] : none;
}

__device__ __forceinline__ void sort2(u32 &a, u32 &b)
{
    const u32 hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// The four largest keys, largest first: sorted fours, joined two at a time
template <int EPL>
__device__ __forceinline__ void four_largest(const u32 (&key)[EPL], u32 (&h)[4])
{
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
        u32 a = key[j], b = key[j + 1], c = key[j + 2], d = key[j + 3];
        sort2(a, b);
        sort2(c, d);
        sort2(a, c);
        sort2(b, d);
        sort2(b, c);
        if (j == 0) {
            h[0] = a, h[1] = b, h[2] = c, h[3] = d;
        } else {
            h[0] = max(h[0], d), h[1] = max(h[1], c), h[2] = max(h[2], b), h[3] = max(h[3], a);
            sort2(h[0], h[2]);
            sort2(h[1], h[3]);
            sort2(h[0], h[1]);
            sort2(h[2], h[3]);
        }
    }
}

// Lanes of a row that hold each of up to 16 groups: a power of two
__host__ __device__ __forceinline__ int lanes_of(int groups)
{
    return groups == 1 ? 16 : groups == 2 ? 8 : groups <= 4 ? 4 : groups <= 8 ? 2 : 1;
}

template <class T, int EPL>
__global__ __launch_bounds__(64 * kRowWaves) void route_rows_kernel(RouteParams P, int64_t tokens)
{
    static_assert(EPL % 4 == 0 && 16 * EPL <= (int)kIndexMask + 1, "indexes fit a key");
    __shared__ double keys_of[kRowWaves][EPL / 4 * 64];
    const int lane = threadIdx.x & 63, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first_token = (block_id() * kRowWaves + wave) * 4;
    if (first_token >= tokens)
        return;
    const int64_t own = first_token + (lane >> 4);
    const int64_t t = own < tokens ? own : tokens - 1;
    const T *row = static_cast<const T *>(P.logits) + t * P.E;
    const int lanes = lanes_of(P.groups), size = P.E / P.groups;   // of a group
    const bool idle = c / lanes >= P.groups;
    const int per = (size + lanes - 1) / lanes, sub = (c % lanes) * per;
    const int start = idle ? 0 : c / lanes * size + sub;
    const int count = idle ? 0 : max(0, min(per, size - sub));
    const float inf = __builtin_inff();
    float v[EPL], b[EPL];
    load_row<T, EPL>(row + start, count, -inf, v);
    if (P.bias)
        load_row<float, EPL>(P.bias + start, count, 0.0f, b);
    float top = -inf, bottom = inf;
    bool odd = false;   // the row is for route_token
#pragma unroll
    for (int j = 0; j < EPL; j += 2) {
        top = fmaxf(fmaxf(top, v[j]), v[j + 1]);
        bottom = fminf(fminf(bottom, v[j]), v[j + 1]);
        odd |= __builtin_isunordered(v[j], v[j + 1]);
    }
    top = row_max(top);
    // every expert masked, as in a padded batch's rows
    const bool none = top == -inf && (__ballot(odd) >> (lane & 48) & 0xffff) == 0;
    odd |= !(top < inf && top > -inf);
    // The factor of exp(l - top): 1 over the sum of all experts' in a softmax,
    // or 1 where it cancels, in renormalized weights and in keys without a
    // bias.  Keys with one, of a renormalized softmax, need it only where
    // experts or groups are close.
    double share = 1.0;
    auto share_of_all = [&] {
        double all = 0.0;
#pragma unroll 4
        for (int j = 0; j < count; ++j)
            all += exp((double)(float)row[start + j] - (double)top);
        return 1.0 / row_sum(all);
    };
    if (!P.sigmoid && !P.renorm) {
        double all = 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            all += exp((double)v[j] - (double)top);
        share = 1.0 / row_sum(all);
    }
    double key_share = share;
    bool known = P.sigmoid || !P.renorm || !P.bias;
    auto score = [&](double l, double part) {
        return P.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) * part;
    };
    const bool by_group = P.groups > P.keep;
    u32 key[EPL];
    u32 need = 0;
    if (Whole<T>::kShift > 0 && !P.bias && (!by_group || P.top == 1)) {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            key[j] = v[j] == -inf ? 0u
                                  : (in_order(v[j]) >> Whole<T>::kShift) << kIndexBits |
                                        (kIndexMask - (u32)(start + j));
    } else {
        // scores with their error, then their places between lowest and highest
        float delta = 0.0f;
        const bool gaps = __ballot(bottom == -inf) != 0;   // absent or masked experts
        if (P.bias || (by_group && P.top == 2)) {
            const float log2e = 1.44269504f;
            float s[EPL], most = 1.0f;
            if (P.sigmoid) {
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    s[j] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v[j] * log2e));
            } else {
                float total = 0.0f;
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    s[j] = __builtin_amdgcn_exp2f((v[j] - top) * log2e);
                    total += s[j];
                }
                most = __builtin_amdgcn_rcpf(row_sum(total));
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    s[j] *= most;
            }
            if (P.bias)
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    s[j] += b[j];
            if (gaps)
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    s[j] = v[j] == -inf ? -inf : s[j];
            // In units of 2^-24: a sigmoid's exponent, exp2, sum and
            // reciprocal, weighted with s (1 - s) or s, come to less than 8;
            // a softmax's exponent, exp2, sum of 36 terms, reciprocal and
            // product to less than 48 of its largest score.
            delta = P.sigmoid ? 0x1p-21f : 0x1p-18f * most;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                v[j] = s[j];
        }
        float hi = -inf, lo = inf;
        if (gaps) {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                lo = fminf(lo, v[j] == -inf ? inf : v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                lo = fminf(lo, v[j]);
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            hi = fmaxf(hi, v[j]);
        hi = row_max(hi);
        lo = -row_max(-lo);
        if (P.bias) {
            // a bias of -inf may have left lo at it
            const bool masked = lo == -inf;
            if (__ballot(masked)) {
                lo = inf;
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    lo = fminf(lo, v[j] == -inf ? inf : v[j]);
                lo = -row_max(-lo);
            }
            // the rounding of score + bias
            delta += 0x1p-24f * fmaxf(fabsf(hi), fabsf(lo));
        }
        // Places to the nearest, from the low bits of a sum with 2^23.  What
        // is the same for all of them (scale, base) keeps their order; the
        // product and the sum round each by less than 5 / 8.  The lowest place
        // is above `need`, so that no expert is as far from every one.
        const float scale = kSpan / (hi - lo), from = -lo * scale;
        const float slack = 2.0f * delta * scale + 0x1p-22f * fabsf(from) + 2.0f;
        odd |= !(hi - lo > 0.0f) || !(scale < 0x1p100f) || !(slack < 0x1p18f);
        need = (u32)fminf(slack, 0x1p18f) + 1u;
        const float base = from + (2.0f * slack + 2.0f);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float place = fminf(fmaxf(__builtin_fmaf(v[j], scale, base), 0.0f), kPlaces);
            key[j] = __float_as_uint(place + 0x1p23f) << kIndexBits | (kIndexMask - (u32)(start + j));
        }
    }
    u32 h[4];
    four_largest<EPL>(key, h);
    if (by_group) {
        u32 first = h[0], second = h[1];
        auto join = [&](u32 f, u32 s) {
            second = max(max(second, s), min(first, f));
            first = max(first, f);
        };
        if (lanes >= 2)
            join(row_swap<kXor1>(first), row_swap<kXor1>(second));
        if (lanes >= 4)
            join(row_swap<kXor2>(first), row_swap<kXor2>(second));
        if (lanes >= 8)
            join(row_swap<kXor4>(first), row_swap<kXor4>(second));
        u32 mine = first;
        if (P.top == 2) {
            odd |= !idle && second <= kIndexMask;
            mine = (first >> kIndexBits) + (second >> kIndexBits);
        }
        // groups that come before this lane's
        int before = 0;
#define OTHER_GROUPS(COUNT)                                                                 \
    if (lanes == 1) {                                                                       \
        COUNT(1) COUNT(3) COUNT(5) COUNT(7) COUNT(9) COUNT(11) COUNT(13) COUNT(15)          \
    }                                                                                       \
    if (lanes <= 2) {                                                                       \
        COUNT(2) COUNT(6) COUNT(10) COUNT(14)                                               \
    }                                                                                       \
    if (lanes <= 4) {                                                                       \
        COUNT(4) COUNT(12)                                                                  \
    }                                                                                       \
    COUNT(8)
#define COUNT(N) before += row_ror<N>(mine) > mine;
        OTHER_GROUPS(COUNT)
#undef COUNT
        bool open = !idle && before < P.keep;
        const int shift = P.top == 2 ? 0 : kIndexBits;
        const u32 last = ~row_max(open ? ~(mine >> shift) : 0u);
        const u32 next = row_max(open ? 0u : mine >> shift);
        // equal sums: more groups open than there should be
        const bool near = (next > 0 && last - next < need * (u32)P.top) ||
                          (need > 0 && __builtin_popcountll(__ballot(open) >> (lane & 48) &
                                                            0xffff) != P.keep * lanes);
        if (__ballot(near)) {
            // the sums in binary64, where the keys tell for certain of what
            u32 third = h[0] < second ? h[0] : h[1] < second ? h[1] : h[2];
            if (lanes >= 2)
                third = max(third, row_swap<kXor1>(third));
            if (lanes >= 4)
                third = max(third, row_swap<kXor2>(third));
            if (lanes >= 8)
                third = max(third, row_swap<kXor4>(third));
            const u32 least = P.top == 2 ? second : first, rest = P.top == 2 ? third : second;
            odd |= near && !idle && (least >> kIndexBits) - (rest >> kIndexBits) < need;
            if (!known) {
                key_share = share_of_all();
                known = true;
            }
            double sum = idle ? -(double)inf : 0.0;
#pragma unroll 1
            for (int i = 0; i < P.top; ++i) {
                const u32 k = i == 0 ? first : second;
                const int e = min((int)(kIndexMask - (k & kIndexMask)), P.E - 1);
                const double l = (double)(float)row[e];
                const double s = P.bias || P.top == 2 ? score(l, key_share) : l;
                sum += k <= kIndexMask ? -(double)inf : P.bias ? s + (double)P.bias[e] : s;
            }
            before = 0;
#define COUNT(N)                                                                            \
    {                                                                                       \
        const double other = row_ror<N>(sum);                                               \
        before += other > sum || (other == sum && ((c - N) & 15) < c);                      \
    }
            OTHER_GROUPS(COUNT)
#undef COUNT
            open = near ? !idle && before < P.keep : open;
        }
#undef OTHER_GROUPS
        if (!open) {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                key[j] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = 0;
        }
    }
    // `chosen`: the c-th of the row.  `sure`: how many of them are a set that
    // is certain, k where the gap after the k-th is wide enough.  `close`: some
    // of them are nearer to each other than `need`.
    u32 best = row_max(h[0]), chosen = best;
    int sure = 0, popped = 0;
    bool close = false, all_keys = false;
    for (int i = 1; i <= 16; ++i) {
        odd |= i <= P.k && best <= kIndexMask;
        const bool here = h[0] == best;
        popped += here;
        h[0] = here ? h[1] : h[0];
        h[1] = here ? h[2] : h[1];
        h[2] = here ? h[3] : h[2];
        h[3] = here ? 0u : h[3];
        u32 next;
        all_keys |= __ballot(popped >= 4) != 0;
        if (!all_keys) {
            next = row_max(h[0]);
        } else {
            // the largest key below `best`: modulo 2^32 only those wrap around
            u32 step = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                step = max(step, key[j] - best);
            step = row_max(step);
            next = (int)step < 0 ? best + step : 0u;
        }
        const bool wide = (best >> kIndexBits) - (next >> kIndexBits) >= need;
        if (i < P.k)
            close |= !wide;
        else if (sure == 0) {
            sure = wide ? i : 0;
            close |= !wide;
        }
        if (i >= P.k && __ballot(sure == 0 && !odd) == 0)
            break;
        best = next;
        chosen = c == i ? best : chosen;
    }
    odd |= sure == 0;
    int id = (int)(kIndexMask - (chosen & kIndexMask)), rank = c;
    const double l = (double)(float)row[min(id, P.E - 1)];
    double w = score(l, share);
    if (__ballot(close)) {
        double mine = l;
        if (P.bias) {
            if (!known)
                key_share = share_of_all();
            const double part = P.sigmoid || !P.renorm ? 1.0 : key_share;   // of w
            mine = w * part + (double)P.bias[min(id, P.E - 1)];
        }
        if (c >= sure)
            mine = -__builtin_inf();
        int before = 0;
#define COUNT(N)                                                                            \
    {                                                                                       \
        const double other = row_ror<N>(mine);                                              \
        const int other_id = (int)row_ror<N>((u32)id);                                      \
        before += other > mine || (other == mine && other_id < id);                         \
    }
        COUNT(1) COUNT(2) COUNT(3) COUNT(4) COUNT(5) COUNT(6) COUNT(7) COUNT(8)
        COUNT(9) COUNT(10) COUNT(11) COUNT(12) COUNT(13) COUNT(14) COUNT(15)
#undef COUNT
        rank = close && c < sure ? before : c;
    }
    const bool has = rank < P.k && c < (close ? sure : P.k);
    const double sum = row_sum(has ? w : 0.0);
    if (P.renorm)
        w = sum > 0.0 ? w / sum : 0.0;
    // a row's lanes agree on `odd` once they have all been asked
    const u64 lanes_odd = __ballot(odd);
    if (has && own < tokens && (lanes_odd >> (lane & 48) & 0xffff) == 0) {
        P.weights[t * P.k + rank] = (float)(w * (double)P.scale);
        P.ids[t * P.k + rank] = id;
    }
    const u64 lanes_none = __ballot(none);
    if (none && own < tokens && c < P.k) {
        P.weights[t * P.k + c] = 0.0f * P.scale;
        P.ids[t * P.k + c] = -1;
    }
    for (int r = 0; r < 4; ++r) {
        const int64_t tt = first_token + r;
        if (((lanes_odd & ~lanes_none) >> (16 * r) & 0xffff) && tt < tokens)
            route_token<T, EPL / 4>(P, tt, lane, keys_of[wave]);
    }
}

template <class T>
hipError_t launch(const RouteParams &p, int64_t tokens, hipStream_t s)
{
    // Four tokens a wave where groups, experts and the chosen fit a row of 16
    // lanes and 32 experts each; a wave a token, in binary64, past that (T =
    // 16384, 512 experts without groups 18 us, 768 84, 1024 89; 256 experts in 8
    // groups 12 and in 32 groups 34; 32 chosen of 256 71)
    const int lanes = p.groups <= 16 ? lanes_of(p.groups) : 1, size = p.E / p.groups;
    const int per = (size + lanes - 1) / lanes;
    if (p.groups <= 16 && per <= 32 && p.k <= 16) {
        const int a_block = 4 * kRowWaves;
        const dim3 grid = grid_of((tokens + a_block - 1) / a_block), block(64 * kRowWaves);
        if (per <= 4)
            hipLaunchKernelGGL((route_rows_kernel<T, 4>), grid, block, 0, s, p, tokens);
        else if (per <= 8)
            hipLaunchKernelGGL((route_rows_kernel<T, 8>), grid, block, 0, s, p, tokens);
        else if (per <= 16)
            hipLaunchKernelGGL((route_rows_kernel<T, 16>), grid, block, 0, s, p, tokens);
        else
            hipLaunchKernelGGL((route_rows_kernel<T, 32>), grid, block, 0, s, p, tokens);
        return hipGetLastError();
    }
    const dim3 grid = grid_of(tokens), block(64);
    if (p.E <= 64)
        hipLaunchKernelGGL((route_kernel<T, 1>), grid, block, 0, s, p, tokens);
    else if (p.E <= 128)
        hipLaunchKernelGGL((route_kernel<T, 2>), grid, block, 0, s, p, tokens);
    else if (p.E <= 256)
        hipLaunchKernelGGL((route_kernel<T, 4>), grid, block, 0, s, p, tokens);
    else if (p.E <= 512)
        hipLaunchKernelGGL((route_kernel<T, 8>), grid, block, 0, s, p, tokens);
    else
        hipLaunchKernelGGL((route_kernel<T, 16>), grid, block, 0, s, p, tokens);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteParams &p, int64_t tokens, int dtype, hipStream_t s)
{
    if (tokens == 0)
        return hipSuccess;
    if (dtype == MHC_F32)
        return launch<float>(p, tokens, s);
    return dtype == MHC_BF16 ? launch<__bf16>(p, tokens, s) : launch<_Float16>(p, tokens, s);
}

}  // namespace mhc
