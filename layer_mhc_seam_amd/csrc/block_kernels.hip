// block_kernels.hip -- the one-stream block boundary and its int8 quantiser.
//
// Block norm: what stands between two sub-layers of a model with an ordinary
// residual stream x [T][H], given the sub-layer's output y [T][H]:
//   p    = y rstd(y) gamma_post                            (or p = y)
//   r    = round_x( residual_scale x + branch_scale (p gate) )   -> residual_out
//   norm = round_e( r rstd(r) gamma )                      -> norm
//   rstd(v) = f32( 1 / sqrt( mean_h v^2 + eps ) )
// and the norm's int8 form (below).  Every product and sum of the
// elementwise chains is rounded to binary32 on its own, in the order written
// (-ffp-contract=off).  The sums of squares are held in binary64: squares of
// binary32 values are exact there and the error of a row's sum is below
// H 2^-53 of it, so rstd does not depend on how the row is dealt out to lanes,
// and neither do the norm's last bits or the codes on either side of a
// rounding border.
//
// Int8 form of a row v (of the norm as rounded, or any row in quantise):
//   a = max( max_h |v|, 2^-119 ),  scale = a / 127,  code = rint( v (127 / a) )
// The floor keeps 127 / a finite and scale normal; a zero row gives zero
// codes.  |v| 127 / a is at most 127 (1 + 2^-23), so no code leaves +-127.  A
// row holding an infinity or NaN gets codes 0 and scale NaN: every product
// taken with it is NaN.
//
// One pass over memory: a workgroup owns a row and keeps it in registers
// between the two (or three) reductions, so each input is read once and each
// output written once.  The row's bytes bound it: T = 16384, H = 5120, bf16,
// both norms, a gate for each element, norm and codes (923 MB) take 153 us at
// best, 6.05 TB/s, which is what a copy reaches, and 157 to 161 call after
// call; the quantiser alone 42 us (6.0 TB/s).  Vector instructions are next,
// 638 a wave of 1024 values, 85 us of them issued back to back: hence the
// cheap roundings and maxima below.  (With 802, of a quotient and a square
// root in binary64 a wave and masks for each value, the best was 163 us.)
// Asking for the gammas ahead of the sums changes nothing (157 to 161 us; T = 4
// 5.0 for 4.9).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

typedef uint32_t u32;
typedef uint64_t u64;
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef u32 u32x2 __attribute__((ext_vector_type(2)));
typedef u32 u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // at any element

constexpr float kTinyMax = 0x1p-119f;

struct Bf16 {
    typedef __bf16 type;
};
struct F16 {
    typedef _Float16 type;
};
struct F32 {
    typedef float type;
};

// Eight consecutive elements of a row, `at` .. at + 7, of which those from
// `from` to `to` - 1 exist (the rest read as zero).  Chunks end where memory
// has a multiple of 8 elements, so that whole ones are aligned in every tensor
// of the row's layout whatever the width; the first and last of a row may be
// partial.  (Chunks counted from the row's first element took 8% longer at
// T = 16384, H = 5117, bf16 with int8.  With these it takes 160 us where H =
// 5120 takes 125: 558 vector instructions a wave for 457, of the partial
// chunks' code, and six waves a row for five, since a row spans up to 642
// chunks; the bytes written are 4% more.)
template <bool RAGGED>
struct Span {
    int at, from, to;
    bool inside;   // all eight lie inside the tensor, in this row or its neighbours
    __device__ __forceinline__ bool whole() const { return to - from == 8; }
    // some of the eight exist, or, in a row of whole chunks, none
    __device__ __forceinline__ bool part() const { return RAGGED && !whole(); }
    __device__ __forceinline__ bool has(int i) const { return i >= from && i < to; }
};

template <bool RAGGED>
__device__ __forceinline__ Span<RAGGED> span_of(int64_t row, int64_t rows, int H, int chunk)
{
    if (!RAGGED) {
        const bool whole = 8 * chunk < H;
        return {8 * chunk, 0, whole ? 8 : 0, whole};
    }
    const int at = 8 * chunk - (int)(row * H & 7), from = max(0, -at);
    const int to = max(from, min(8, H - at));
    return {at, from, to, to > from && row * H + at + 8 <= rows * H};
}

template <class E>
__device__ __forceinline__ void unpack8(const u32x4 &v, float (&f)[8])
{
    typedef typename E::type e8 __attribute__((ext_vector_type(8)));
    const e8 h = __builtin_bit_cast(e8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = (float)h[i];
}

template <class E>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    typedef typename E::type e8 __attribute__((ext_vector_type(8)));
    e8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = (typename E::type)rounded(f[i]);   // to nearest even
    return __builtin_bit_cast(u32x4, h);
}

// A chunk of a row as it lies in memory
template <class E>
struct Chunk {
    u32x4 v;
};
template <>
struct Chunk<F32> {
    u32x4 v, w;
};

// The span's elements of a row of a tensor.  A partial chunk is read whole
// too, and what belongs to the rows beside it dropped, but for one that ends
// past the tensor.
template <class E, bool RAGGED>
__device__ __forceinline__ void load_chunk(Chunk<E> &c, const void *row, const Span<RAGGED> &s)
{
    typedef typename E::type T;
    const T *p = static_cast<const T *>(row) + s.at;
    if (s.inside) {
        c.v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
        if constexpr (sizeof(T) == 4)
            c.w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p) + 1);
    } else if (RAGGED) {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = s.has(i) ? p[i] : (T)0.0f;
        __builtin_memcpy(&c, e, sizeof c);
    } else {
        __builtin_memset(&c, 0, sizeof c);
    }
}

// The span's elements of a vector over the channels
template <class E, bool RAGGED>
__device__ __forceinline__ void load_channels(Chunk<E> &c, const void *v, const Span<RAGGED> &s)
{
    typedef typename E::type T;
    const T *p = static_cast<const T *>(v) + s.at;
    if (s.whole()) {
        c.v = *reinterpret_cast<const u32x4_any *>(p);
        if constexpr (sizeof(T) == 4)
            c.w = reinterpret_cast<const u32x4_any *>(p)[1];
    } else if (RAGGED) {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = s.has(i) ? p[i] : (T)0.0f;
        __builtin_memcpy(&c, e, sizeof c);
    } else {
        __builtin_memset(&c, 0, sizeof c);
    }
}

// zeros for the elements of c that do not exist
template <class E, bool RAGGED>
__device__ __forceinline__ void keep_own(Chunk<E> &c, const Span<RAGGED> &s)
{
    typedef typename E::type T;
    if (!s.part())
        return;
    T e[8];
    __builtin_memcpy(e, &c, sizeof c);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        e[k] = s.has(k) ? e[k] : (T)0.0f;
    __builtin_memcpy(&c, e, sizeof c);
}

template <class E>
__device__ __forceinline__ void unpack(const Chunk<E> &c, float (&f)[8])
{
    if constexpr (sizeof(typename E::type) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __uint_as_float(c.v[i]);
            f[4 + i] = __uint_as_float(c.w[i]);
        }
    } else {
        unpack8<E>(c.v, f);
    }
}

// f rounded to E, in memory and back in f
template <class E, bool RAGGED>
__device__ __forceinline__ Chunk<E> store_round(void *row, const Span<RAGGED> &s, float (&f)[8])
{
    typedef typename E::type T;
    T *p = static_cast<T *>(row) + s.at;
    Chunk<E> c;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c.v[i] = __float_as_uint(f[i]);
            c.w[i] = __float_as_uint(f[4 + i]);
        }
    } else {
        c.v = pack8<E>(f);
        unpack8<E>(c.v, f);
    }
    if (!row)
        return c;
    if (s.whole()) {
        __builtin_nontemporal_store(c.v, reinterpret_cast<u32x4 *>(p));
        if constexpr (sizeof(T) == 4)
            __builtin_nontemporal_store(c.w, reinterpret_cast<u32x4 *>(p) + 1);
    } else if (RAGGED) {
        T e[8];
        __builtin_memcpy(e, &c, sizeof c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s.has(i))
                p[i] = e[i];
    }
    return c;
}

// Codes of eight values, four to a word: in the low byte of the product's sum
// with 1.5 x 2^23, which rounds it to a whole number, ties to even.
template <bool RAGGED>
__device__ __forceinline__ void store_codes(int8_t *row, const Span<RAGGED> &s, const float (&f)[8],
                                            float inv)
{
    int8_t *p = row + s.at;
    u32 b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i] = __float_as_uint(f[i] * inv + 0x1.8p23f);
    u32x2 c;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const u32 lo = __builtin_amdgcn_perm(b[4 * w + 1], b[4 * w], 0x0c0c0400u);
        const u32 hi = __builtin_amdgcn_perm(b[4 * w + 3], b[4 * w + 2], 0x04000c0cu);
        c[w] = lo | hi;
    }
    if (s.whole()) {
        __builtin_nontemporal_store(c, reinterpret_cast<u32x2 *>(p));
    } else if (RAGGED) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s.has(i))
                p[i] = (int8_t)(c[i / 4] >> (8 * (i % 4)));
    }
}

// Largest magnitudes of a chunk's even and odd elements, joined to `m`: bit
// patterns without their sign, of which any NaN's is above infinity's.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void join_max(u16x2 &m, const u32x4 &v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
}

// the larger of both as binary32 bits
template <class E>
__device__ __forceinline__ u32 max_bits(const u16x2 &m)
{
    const unsigned short v = m[0] > m[1] ? m[0] : m[1];
    return __float_as_uint((float)__builtin_bit_cast(typename E::type, v));
}

// Workgroup reductions: each wave's value in LDS, one barrier, every thread
// joins them in wave order.  `slot` is used for this reduction alone.
__device__ __forceinline__ double block_sum(double v, double *slot, int waves)
{
    v = wave_sum(v);
    if (waves == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        slot[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = slot[0];
    for (int w = 1; w < waves; ++w)
        s += slot[w];
    return s;
}

__device__ __forceinline__ u32 block_max(u32 v, u32 *slot, int waves)
{
    v = wave_max(v);
    if (waves == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        slot[threadIdx.x >> 6] = v;
    __syncthreads();
    u32 m = slot[0];
    for (int w = 1; w < waves; ++w)
        m = max(m, slot[w]);
    return m;
}

// 1 / sqrt(sum / H + eps), rounded once to binary32: the hardware's estimate
// (24 bits or more) and two steps of Newton's iteration, each of which squares
// the error, in a tenth of the instructions of a square root and a quotient.
__device__ __forceinline__ float rstd_of(double sum, double inv_H, float eps)
{
    const double x = __builtin_fma(sum, inv_H, (double)eps);
    double y = __builtin_amdgcn_rsq(x);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double h = 0.5 * y;
        y = __builtin_fma(h, __builtin_fma(-x * y, y, 1.0), y);
    }
    return x == __builtin_inf() ? 0.0f : (float)y;
}

// The row's scale and the factor its codes are made with.  amax: the largest
// magnitude's bits (any NaN's are above infinity's).
__device__ __forceinline__ void int8_scale(u32 amax, float &scale, float &inv)
{
    const bool fine = amax < 0x7f800000u;
    const float a = fmaxf(fine ? __uint_as_float(amax) : 1.0f, kTinyMax);
    scale = fine ? a / 127.0f : __uint_as_float(0x7fc00000u);
    inv = fine ? 127.0f / a : 0.0f;
}

constexpr int kMaxWaves = 16, kWaveRows = 4;

// Who works on a row: a workgroup, or (WAVE) one of its kWaveRows waves.
// Thread i holds the row's chunks i, i + stride, ...
template <bool WAVE>
struct RowPlace {
    int64_t row;
    int index, stride, waves;
    __device__ __forceinline__ RowPlace()
    {
        if (WAVE) {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            row = block_id() * kWaveRows + wave;
            index = threadIdx.x & 63;
            stride = 64;
            waves = 1;
        } else {
            row = block_id();
            index = threadIdx.x;
            stride = blockDim.x;
            waves = blockDim.x >> 6;
        }
    }
};

template <int NC, bool WAVE>
constexpr int max_threads()
{
    return WAVE ? 64 * kWaveRows : NC == 4 ? 1024 : 512;
}

template <class E, class X, int NC, bool WAVE, bool RAGGED>
__global__ __launch_bounds__((max_threads<NC, WAVE>())) void block_norm_kernel(BlockNormParams P)
{
    __shared__ double sum_y[kMaxWaves], sum_r[kMaxWaves];
    __shared__ u32 max_n[kMaxWaves];
    typedef typename E::type T;
    typedef typename X::type TX;
    const RowPlace<WAVE> me;
    const int64_t t = me.row;
    if (t >= P.T)
        return;
    const int H = P.H, waves = me.waves;
    Span<RAGGED> span[NC];
    Chunk<X> cx[NC];
    Chunk<E> cy[NC], cg[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        span[i] = span_of<RAGGED>(t, P.T, H, me.index + i * me.stride);
        load_chunk<X>(cx[i], static_cast<const TX *>(P.x) + t * H, span[i]);
        if (P.y)
            load_chunk<E>(cy[i], static_cast<const T *>(P.y) + t * H, span[i]);
        if (P.gate_kind == MHC_GATE_ELEMENT)
            load_chunk<E>(cg[i], static_cast<const T *>(P.gate) + t * H, span[i]);
    }
    float r[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        keep_own<X>(cx[i], span[i]);
        unpack<X>(cx[i], r[i]);
    }
    if (P.y) {
        float p[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            keep_own<E>(cy[i], span[i]);
            unpack<E>(cy[i], p[i]);
        }
        if (P.gamma_post) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s = __builtin_fma((double)p[i][e], (double)p[i][e], s);
            const float rs = rstd_of(block_sum(s, sum_y, waves), P.inv_H, P.eps);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                Chunk<E> c;
                float g[8];
                load_channels<E>(c, P.gamma_post, span[i]);
                unpack<E>(c, g);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p[i][e] = (p[i][e] * rs) * g[e];
            }
        }
        if (P.gate_kind != MHC_GATE_NONE) {
            const float token = P.gate_kind == MHC_GATE_TOKEN ? static_cast<const float *>(P.gate)[t]
                                                              : 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float g[8];
                if (P.gate_kind == MHC_GATE_ELEMENT) {
                    unpack<E>(cg[i], g);
                } else if (P.gate_kind == MHC_GATE_CHANNEL) {
                    Chunk<F32> c;
                    load_channels<F32>(c, P.gate, span[i]);
                    unpack<F32>(c, g);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        g[e] = token;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    p[i][e] = p[i][e] * g[e];
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[i][e] = P.residual_scale * r[i][e] + P.branch_scale * p[i][e];
            store_round<X>(static_cast<TX *>(P.residual_out) + t * H, span[i], r[i]);
        }
        // what does not exist adds nothing, whatever rstd made of its zeros
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (!span[i].whole())
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    r[i][e] = span[i].has(e) ? r[i][e] : 0.0f;
    }
    if (!P.gamma)
        return;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s = __builtin_fma((double)r[i][e], (double)r[i][e], s);
    const float rs = rstd_of(block_sum(s, sum_r, waves), P.inv_H, P.eps);
    u16x2 amax = {0, 0};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        Chunk<E> c;
        float g[8];
        load_channels<E>(c, P.gamma, span[i]);
        unpack<E>(c, g);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[i][e] = (r[i][e] * rs) * g[e];
        c = store_round<E>(P.norm ? static_cast<T *>(P.norm) + t * H : nullptr, span[i], r[i]);
        keep_own<E>(c, span[i]);   // a NaN rstd makes NaN of zeros
        if (RAGGED || span[i].whole())
            join_max(amax, c.v);
    }
    if (!P.codes)
        return;
    float scale, inv;
    int8_scale(block_max(max_bits<E>(amax), max_n, waves), scale, inv);
    const bool fine = inv != 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if (!fine)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[i][e] = 0.0f;
        store_codes(P.codes + t * H, span[i], r[i], inv);
    }
    if (me.index == 0)
        P.scales[t] = scale;
}

template <class E, int NC, bool WAVE, bool RAGGED>
__global__ __launch_bounds__((max_threads<NC, WAVE>())) void int8_quantize_kernel(
    const void *src, int64_t rows, int H, int8_t *codes, float *scales)
{
    __shared__ u32 max_n[kMaxWaves];
    typedef typename E::type T;
    const RowPlace<WAVE> me;
    const int64_t t = me.row;
    if (t >= rows)
        return;
    Span<RAGGED> span[NC];
    Chunk<E> c[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        span[i] = span_of<RAGGED>(t, rows, H, me.index + i * me.stride);
        load_chunk<E>(c[i], static_cast<const T *>(src) + t * H, span[i]);
    }
    u16x2 amax = {0, 0};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        keep_own<E>(c[i], span[i]);
        join_max(amax, c[i].v);
    }
    float scale, inv;
    int8_scale(block_max(max_bits<E>(amax), max_n, me.waves), scale, inv);
    const bool fine = inv != 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float v[8];
        unpack<E>(c[i], v);
        if (!fine)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = 0.0f;
        store_codes(codes + t * H, span[i], v, inv);
    }
    if (me.index == 0)
        scales[t] = scale;
}

// Rows of up to 128 chunks (H = 1024) take a wave each, four in a workgroup,
// without barriers (bf16, both norms, element gate, int8, in a wave and in a
// workgroup: H = 512 17.8 and 20.5 us at T = 16384, 2.7 and 3.3 at T = 4; H =
// 1024 no difference; H = 2048 64.3 and 63.0, 5.0 and 4.0).  Longer ones take a
// workgroup of up to 512 threads with two chunks each (H = 5120 with one, two
// and four a thread: 186, 157 and 158 us at T = 16384; 4.4, 4.9 and 5.7 at T =
// 4, channel gate), the longest up to 1024 with four.
template <class F>
hipError_t with_shape(int64_t rows, int H, F &&f)
{
    const bool ragged = H % 8 != 0;
    const int chunks = ragged ? H / 8 + 2 : H / 8;   // the most a row spans
    auto go = [&](auto nc, auto wave, dim3 grid, dim3 block) {
        return ragged ? f(nc, wave, std::true_type{}, grid, block)
                      : f(nc, wave, std::false_type{}, grid, block);
    };
    auto wave = [&](auto nc) {
        return go(nc, std::true_type{}, grid_of((rows + kWaveRows - 1) / kWaveRows),
                  dim3(64 * kWaveRows));
    };
    auto block = [&](auto nc) {
        const int threads = ((chunks + nc() - 1) / nc() + 63) / 64 * 64;
        return go(nc, std::false_type{}, grid_of(rows), dim3(threads));
    };
    if (chunks <= 64)
        return wave(std::integral_constant<int, 1>{});
    if (chunks <= 128)
        return wave(std::integral_constant<int, 2>{});
    if (chunks <= 1024)
        return block(std::integral_constant<int, 2>{});
    return block(std::integral_constant<int, 4>{});
}

template <class E, class X>
hipError_t launch_norm(const BlockNormParams &p, hipStream_t s)
{
    return with_shape(p.T, p.H, [&](auto nc, auto wave, auto ragged, dim3 grid, dim3 block) {
        hipLaunchKernelGGL((block_norm_kernel<E, X, nc(), wave(), ragged()>), grid, block, 0, s, p);
        return hipGetLastError();
    });
}

template <class E>
hipError_t launch_quant(const void *src, int64_t rows, int H, int8_t *codes, float *scales,
                        hipStream_t s)
{
    return with_shape(rows, H, [&](auto nc, auto wave, auto ragged, dim3 grid, dim3 block) {
        hipLaunchKernelGGL((int8_quantize_kernel<E, nc(), wave(), ragged()>), grid, block, 0, s,
                           src, rows, H, codes, scales);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_block_norm(const BlockNormParams &p, int dtype, int x_dtype, hipStream_t s)
{
    if (p.T == 0)
        return hipSuccess;
    const bool wide = x_dtype == MHC_F32;
    if (dtype == MHC_BF16)
        return wide ? launch_norm<Bf16, F32>(p, s) : launch_norm<Bf16, Bf16>(p, s);
    return wide ? launch_norm<F16, F32>(p, s) : launch_norm<F16, F16>(p, s);
}

hipError_t launch_int8_quantize(const void *src, int dtype, int64_t rows, int H, int8_t *codes,
                                float *scales, hipStream_t s)
{
    if (rows == 0)
        return hipSuccess;
    return dtype == MHC_BF16 ? launch_quant<Bf16>(src, rows, H, codes, scales, s)
                             : launch_quant<F16>(src, rows, H, codes, scales, s);
}

}  // namespace mhc
