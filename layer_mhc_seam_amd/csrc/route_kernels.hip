// route_kernels.hip -- routing of tokens to experts from their logits.
//
// For each token, with logits l [E], an optional bias b [E] that balances
// the experts' load, and G groups of E / G consecutive experts:
//   s   = softmax(l)  or  1 / (1 + exp(-l))
//   key = s + b                        (s without a bias)
//   the `keep` groups whose sums of their best `top` (1 or 2) keys are the
//   largest stay open; of their experts the k of the largest keys are chosen,
//   largest first
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
// Masks: a logit of -inf, or a bias of -inf, takes an expert out.  A group's
// missing keys count as -1e30, so groups with more experts left come first.
// Where fewer than k experts are left the other slots hold id -1, weight 0; a
// row with none left has nothing else.  A NaN logit (and +inf under softmax)
// is taken out likewise and turns the row's weights to NaN, so ids always lie
// in -1 .. E - 1 and are distinct but for -1.
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

// One wave a token; lane l holds experts EPL l .. EPL l + EPL - 1.
template <class T, int EPL>
__global__ __launch_bounds__(64) void route_kernel(RouteParams P)
{
    __shared__ double keys[EPL * 64];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x, E = P.E;
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
        key[j] = s[j] + (P.bias && e < E ? (double)P.bias[e] : 0.0);
        if (l[j] == -inf || key[j] != key[j])
            key[j] = -inf;
    }
    if (P.groups > 1) {
        const int size = E / P.groups;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            keys[EPL * lane + j] = key[j];
        __syncthreads();
        double first = -inf, second = -inf;
        if (lane < P.groups)
            for (int i = 0; i < size; ++i) {
                const double v = keys[lane * size + i];
                second = fmax(second, fmin(first, v));
                first = fmax(first, v);
            }
        double sum = first == -inf ? kMissing : first;
        if (P.top == 2)
            sum += second == -inf ? kMissing : second;
        __syncthreads();
        keys[lane] = sum;
        __syncthreads();
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

template <class T>
hipError_t launch(const RouteParams &p, int64_t tokens, hipStream_t s)
{
    const dim3 grid((unsigned)tokens), block(64);
    if (p.E <= 64)
        hipLaunchKernelGGL((route_kernel<T, 1>), grid, block, 0, s, p);
    else if (p.E <= 128)
        hipLaunchKernelGGL((route_kernel<T, 2>), grid, block, 0, s, p);
    else if (p.E <= 256)
        hipLaunchKernelGGL((route_kernel<T, 4>), grid, block, 0, s, p);
    else if (p.E <= 512)
        hipLaunchKernelGGL((route_kernel<T, 8>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((route_kernel<T, 16>), grid, block, 0, s, p);
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
