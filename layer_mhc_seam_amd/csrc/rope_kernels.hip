// rope_kernels.hip -- rotary positions of queries and keys.
//
// Pair i of a token turns by theta = p f_i.  In turns, theta / 2 pi = p (f_i /
// 2 pi) is taken in binary64, four times that is split into a whole number k of
// quarters and d in [-1/2, 1/2], still in binary64, and sine and cosine of d pi/2
// come from their Taylor series to degrees 9 and 10, whose next terms are below
// 2^-28 there.  So a position of 2^20 costs no more bits than one of 3: the two
// products and the constant are off by 3 2^-53 of the angle, and p by one more past
// 2^53.
//
// Bytes bound it: each value is read and written once, 16384 tokens of 48 heads of
// 128 channels inside a product's rows, 403 MB, in 69 us into the same output again
// and again, 88 into outputs in turn (a copy of as many bytes: 73).  A thread keeps
// the sines and cosines of NP pairs and turns them in several heads: with two heads a
// thread instead of eight that takes 106 us; with the next head's loads before this
// one's stores, or a grid that stays, 87 to 99.
#include <hip/hip_runtime.h>

#include "half_ops.h"
#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

constexpr int kRopeThreads = 256;

template <int N> struct alignas(2 * N) Vec {
    uint16_t v[N];
};

__device__ __forceinline__ void sin_cos_of_turns(double turns, float *sine, float *cosine)
{
    const double magic = 6755399441055744.0;     // 1.5 * 2^52: a sum's low bits are the whole number
    const double quarters = turns * 4.0, shifted = quarters + magic;
    const u32 k = (u32)__builtin_bit_cast(u64, shifted);
    const float z = (float)(quarters - (shifted - magic)) * 1.57079632679f;
    const float q = z * z;
    const float s = z * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
    const float c = fmaf(
        q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const float a = k & 1 ? c : s, b = k & 1 ? s : c;
    *sine = k & 2 ? -a : a;
    *cosine = (k + 1) & 2 ? -b : b;
}

template <int DT> __device__ __forceinline__ float value(uint16_t v)
{
    return Half<DT>::low(v);
}

template <int DT> __device__ __forceinline__ uint16_t half_of(float v)
{
    return __builtin_bit_cast(uint16_t, (typename Half<DT>::type)v);
}

// Long vectors past the caches: T = 16384, 48 heads of 128 channels 6% faster
template <int N> __device__ __forceinline__ void store(uint16_t *to, const Vec<N> &v)
{
    if constexpr (N == 8)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), (u32x4 *)to);
    else
        *(Vec<N> *)to = v;
}

// A thread's unit: NP pairs, or 2 NP channels past the rotary ones to copy.
template <int DT, int NP, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(const RopeParams P)
{
    const int64_t id = block_id() * kRopeThreads + threadIdx.x;
    const int64_t row = id / P.units;
    const int unit = (int)(id - row * P.units);
    const int64_t t = row / P.head_steps;
    const int first = (int)(row - t * P.head_steps);
    if (t >= P.T)
        return;
    const int half = P.rotary / 2, turning = half / NP;
    const bool turns = unit < turning;
    const int pair = unit * NP;
    int at0, at1;           // of the two chunks of NP channels
    if (turns) {
        at0 = INTER ? 2 * pair : pair;
        at1 = INTER ? at0 + NP : pair + half;
    } else {
        at0 = P.rotary + (unit - turning) * 2 * NP;
        at1 = at0 + NP;
    }
    float sine[NP], cosine[NP];
    if (turns) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int i = pair + j;
            const int axis = (int)(P.axis[i / 16] >> (i % 16 * 2)) & 3;
            const int64_t from = axis * P.position_axis + t;
            const double p = P.position_bytes == 8 ? (double)((const int64_t *)P.positions)[from]
                                                   : (double)((const int32_t *)P.positions)[from];
            sin_cos_of_turns(p * (double)P.inv_freq[i] * 0.15915494309189533577, &sine[j], &cosine[j]);
            sine[j] *= P.inverse ? -P.scale : P.scale;
            cosine[j] *= P.scale;
        }
    }
    const bool second = turns || at1 < P.head_dim;
    for (int h = first; h < P.q_heads + P.k_heads; h += P.head_steps) {
        const bool is_k = h >= P.q_heads;
        const int hh = is_k ? h - P.q_heads : h;
        const uint16_t *src = is_k ? P.k + t * P.k_token + hh * P.k_head : P.q + t * P.q_token + hh * P.q_head;
        uint16_t *dst =
            is_k ? P.k_out + t * P.k_out_token + hh * P.k_out_head : P.q_out + t * P.q_out_token + hh * P.q_out_head;
        Vec<NP> a = *(const Vec<NP> *)(src + at0), b{};
        if (second)
            b = *(const Vec<NP> *)(src + at1);
        if (turns) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                uint16_t &x = INTER ? (2 * j < NP ? a.v[2 * j % NP] : b.v[2 * j % NP]) : a.v[j];
                uint16_t &y = INTER ? (2 * j + 1 < NP ? a.v[(2 * j + 1) % NP] : b.v[(2 * j + 1) % NP]) : b.v[j];
                const float u = value<DT>(x), w = value<DT>(y);
                x = half_of<DT>(rounded(fmaf(u, cosine[j], -(w * sine[j]))));
                y = half_of<DT>(rounded(fmaf(w, cosine[j], u * sine[j])));
            }
        }
        store(dst + at0, a);
        if (second)
            store(dst + at1, b);
    }
}

template <int DT, int NP> hipError_t launch(const RopeParams &p, bool interleaved, hipStream_t s)
{
    const dim3 grid = grid_of((p.T * p.head_steps * p.units + kRopeThreads - 1) / kRopeThreads);
    if (interleaved)
        rope_kernel<DT, NP, true><<<grid, kRopeThreads, 0, s>>>(p);
    else
        rope_kernel<DT, NP, false><<<grid, kRopeThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT> hipError_t launch_vector(const RopeParams &p, int vector, bool interleaved, hipStream_t s)
{
    return vector == 8   ? launch<DT, 8>(p, interleaved, s)
           : vector == 4 ? launch<DT, 4>(p, interleaved, s)
           : vector == 2 ? launch<DT, 2>(p, interleaved, s)
                         : launch<DT, 1>(p, interleaved, s);
}

}  // namespace

hipError_t launch_rope(RopeParams p, int dtype, int vector, bool interleaved, bool in_place, int cus, hipStream_t s)
{
    // channels past the rotary ones are copied, or stay where they are
    p.units = p.rotary / 2 / vector;
    if (!in_place)
        p.units += (p.head_dim - p.rotary + 2 * vector - 1) / (2 * vector);
    // up to 8 heads a thread, fewer where that leaves under four waves a SIMD
    const int heads = p.q_heads + p.k_heads;
    int each = 8;
    while (each > 1 && p.T * p.units * ((heads + each - 1) / each) < (int64_t)cus * 16 * 64)
        each /= 2;
    p.head_steps = (heads + each - 1) / each;
    return dtype == MHC_BF16 ? launch_vector<MHC_BF16>(p, vector, interleaved, s)
                             : launch_vector<MHC_F16>(p, vector, interleaved, s);
}

}  // namespace mhc
