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
// output written once.  The row's bytes bound it.
#include <hip/hip_runtime.h>

#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

typedef uint32_t u32;
typedef uint64_t u64;
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef u32 u32x2 __attribute__((ext_vector_type(2)));
// rows of a width that is no multiple of 8 start at any element
typedef u32 u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef u32 u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

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

// 8 consecutive elements of a row as binary32.  `n` of them exist: 8, or
// fewer in the last chunk of a ragged row (the rest read as zero).
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

template <class E>
__device__ __forceinline__ void load_chunk(Chunk<E> &c, const void *row, int at, int n)
{
    typedef typename E::type T;
    const T *p = static_cast<const T *>(row) + at;
    if (n == 8) {
        c.v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
        if constexpr (sizeof(T) == 4)
            c.w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p) + 1);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = i < n ? p[i] : (T)0.0f;
        __builtin_memcpy(&c, e, sizeof c);
    }
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
template <class E>
__device__ __forceinline__ void store_round(void *row, int at, int n, float (&f)[8])
{
    typedef typename E::type T;
    T *p = static_cast<T *>(row) + at;
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
        return;
    if (n == 8) {
        __builtin_nontemporal_store(c.v, reinterpret_cast<u32x4_any *>(p));
        if constexpr (sizeof(T) == 4)
            __builtin_nontemporal_store(c.w, reinterpret_cast<u32x4_any *>(p) + 1);
    } else {
        T e[8];
        __builtin_memcpy(e, &c, sizeof c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = e[i];
    }
}

__device__ __forceinline__ void store_codes(int8_t *p, int n, const float (&f)[8], float inv)
{
    u32x2 c = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i / 4] |= ((u32)(int)__builtin_rintf(f[i] * inv) & 0xffu) << (8 * (i % 4));
    if (n == 8) {
        __builtin_nontemporal_store(c, reinterpret_cast<u32x2_any *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = (int8_t)(c[i / 4] >> (8 * (i % 4)));
    }
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

__device__ __forceinline__ float rstd_of(double sum, int H, float eps)
{
    return (float)(1.0 / __builtin_sqrt(sum / (double)H + (double)eps));
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

constexpr int kMaxWaves = 16;

// NC chunks of 8 elements a thread, thread t holds chunks t, t + threads, ...
template <class E, class X, int NC>
__global__ __launch_bounds__(1024) void block_norm_kernel(BlockNormParams P)
{
    __shared__ double sum_y[kMaxWaves], sum_r[kMaxWaves];
    __shared__ u32 max_n[kMaxWaves];
    typedef typename E::type T;
    typedef typename X::type TX;
    const int64_t t = blockIdx.x;
    const int H = P.H, waves = blockDim.x >> 6;
    const TX *x = static_cast<const TX *>(P.x) + t * H;
    int at[NC], n[NC];
    Chunk<X> cx[NC];
    Chunk<E> cy[NC], cg[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        at[i] = 8 * (threadIdx.x + i * blockDim.x);
        n[i] = max(0, min(8, H - at[i]));
        load_chunk<X>(cx[i], x, at[i], n[i]);
        if (P.y)
            load_chunk<E>(cy[i], static_cast<const T *>(P.y) + t * H, at[i], n[i]);
        if (P.gate_kind == MHC_GATE_ELEMENT)
            load_chunk<E>(cg[i], static_cast<const T *>(P.gate) + t * H, at[i], n[i]);
    }
    float r[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
        unpack<X>(cx[i], r[i]);
    if (P.y) {
        float p[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            unpack<E>(cy[i], p[i]);
        if (P.gamma_post) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s = __builtin_fma((double)p[i][e], (double)p[i][e], s);
            const float rs = rstd_of(block_sum(s, sum_y, waves), H, P.eps);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                Chunk<E> c;
                float g[8];
                load_chunk<E>(c, P.gamma_post, at[i], n[i]);
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
                    load_chunk<F32>(c, P.gate, at[i], n[i]);
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
            store_round<X>(static_cast<TX *>(P.residual_out) + t * H, at[i], n[i], r[i]);
        }
    }
    if (!P.gamma)
        return;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s = e < n[i] ? __builtin_fma((double)r[i][e], (double)r[i][e], s) : s;
    const float rs = rstd_of(block_sum(s, sum_r, waves), H, P.eps);
    u32 amax = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        Chunk<E> c;
        float g[8];
        load_chunk<E>(c, P.gamma, at[i], n[i]);
        unpack<E>(c, g);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[i][e] = (r[i][e] * rs) * g[e];
        store_round<E>(P.norm ? static_cast<T *>(P.norm) + t * H : nullptr, at[i], n[i], r[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            amax = max(amax, e < n[i] ? __float_as_uint(r[i][e]) & 0x7fffffffu : 0u);
    }
    if (!P.codes)
        return;
    float scale, inv;
    int8_scale(block_max(amax, max_n, waves), scale, inv);
    const bool fine = inv != 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if (!fine)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[i][e] = 0.0f;
        store_codes(P.codes + t * H + at[i], n[i], r[i], inv);
    }
    if (threadIdx.x == 0)
        P.scales[t] = scale;
}

template <class E, int NC>
__global__ __launch_bounds__(1024) void int8_quantize_kernel(const void *src, int H, int8_t *codes,
                                                             float *scales)
{
    __shared__ u32 max_n[kMaxWaves];
    typedef typename E::type T;
    const int64_t t = blockIdx.x;
    const int waves = blockDim.x >> 6;
    const T *row = static_cast<const T *>(src) + t * H;
    int at[NC], n[NC];
    Chunk<E> c[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        at[i] = 8 * (threadIdx.x + i * blockDim.x);
        n[i] = max(0, min(8, H - at[i]));
        load_chunk<E>(c[i], row, at[i], n[i]);
    }
    float v[NC][8];
    u32 amax = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        unpack<E>(c[i], v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            amax = max(amax, __float_as_uint(v[i][e]) & 0x7fffffffu);
    }
    float scale, inv;
    int8_scale(block_max(amax, max_n, waves), scale, inv);
    const bool fine = inv != 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if (!fine)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = 0.0f;
        store_codes(codes + t * H + at[i], n[i], v[i], inv);
    }
    if (threadIdx.x == 0)
        scales[t] = scale;
}

// Chunks a thread holds and threads a row: whole rows in registers, 64 to
// 1024 threads.
struct RowShape {
    int nc, threads;
};

RowShape row_shape(int H)
{
    const int chunks = (H + 7) / 8;
    const int nc = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
    return {nc, ((chunks + nc - 1) / nc + 63) / 64 * 64};
}

template <class E, class X>
hipError_t launch_norm(const BlockNormParams &p, int64_t T, hipStream_t s)
{
    const RowShape g = row_shape(p.H);
    const dim3 grid((unsigned)T), block(g.threads);
    if (g.nc == 1)
        hipLaunchKernelGGL((block_norm_kernel<E, X, 1>), grid, block, 0, s, p);
    else if (g.nc == 2)
        hipLaunchKernelGGL((block_norm_kernel<E, X, 2>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((block_norm_kernel<E, X, 4>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <class E>
hipError_t launch_quant(const void *src, int64_t rows, int H, int8_t *codes, float *scales,
                        hipStream_t s)
{
    const RowShape g = row_shape(H);
    const dim3 grid((unsigned)rows), block(g.threads);
    if (g.nc == 1)
        hipLaunchKernelGGL((int8_quantize_kernel<E, 1>), grid, block, 0, s, src, H, codes, scales);
    else if (g.nc == 2)
        hipLaunchKernelGGL((int8_quantize_kernel<E, 2>), grid, block, 0, s, src, H, codes, scales);
    else
        hipLaunchKernelGGL((int8_quantize_kernel<E, 4>), grid, block, 0, s, src, H, codes, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const BlockNormParams &p, int64_t T, int dtype, int x_dtype,
                             hipStream_t s)
{
    if (T == 0)
        return hipSuccess;
    const bool wide = x_dtype == MHC_F32;
    if (dtype == MHC_BF16)
        return wide ? launch_norm<Bf16, F32>(p, T, s) : launch_norm<Bf16, Bf16>(p, T, s);
    return wide ? launch_norm<F16, F32>(p, T, s) : launch_norm<F16, F16>(p, T, s);
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
