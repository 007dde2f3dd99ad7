// lane_ops.h -- what the block operators' kernels share: launches of any
// number of workgroups, wave-wide reductions, a rounding barrier.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mhc {
namespace {

// Grid of that many workgroups and, past 2^21, up to 2^21 - 1 more: a grid's
// threads along x stay below 2^32 whatever the workgroup.  Workgroups past the
// number asked for have nothing to do.
inline dim3 grid_of(int64_t blocks)
{
    const int64_t x = blocks < (int64_t(1) << 21) ? blocks : int64_t(1) << 21;
    return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

__device__ __forceinline__ int64_t block_id()
{
    return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// v as its own rounding left it: keeps the compiler from folding the product
// or sum that made it into the conversion to fp16 that follows (one rounding
// in place of two, where the other types round twice)
__device__ __forceinline__ float rounded(float v)
{
    asm("" : "+v"(v));
    return v;
}

// Value of lane (l - N) mod 16 of the lane's row of 16
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xf, 0xf, true);
}

template <int N>
__device__ __forceinline__ double row_ror(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = row_ror<N>((uint32_t)b), hi = row_ror<N>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ uint32_t read_lane(uint32_t v, int l)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}

__device__ __forceinline__ double read_lane(double v, int l)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = read_lane((uint32_t)b, l), hi = read_lane((uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Reductions over a row of 16 lanes (all active), the same value in each.
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, row_ror<8>(v));
    v = max(v, row_ror<4>(v));
    v = max(v, row_ror<2>(v));
    return max(v, row_ror<1>(v));
}

template <int N>
__device__ __forceinline__ float row_ror(float v)
{
    return __uint_as_float(row_ror<N>(__float_as_uint(v)));
}

__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, row_ror<8>(v));
    v = fmaxf(v, row_ror<4>(v));
    v = fmaxf(v, row_ror<2>(v));
    return fmaxf(v, row_ror<1>(v));
}

__device__ __forceinline__ float row_sum(float v)
{
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    return v + row_ror<1>(v);
}

__device__ __forceinline__ double row_sum(double v)
{
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    return v + row_ror<1>(v);
}

// Value of lane l ^ 1, l ^ 2; and of lane l ^ 7, which stands for l ^ 4 once
// the lanes of each four hold one value.
enum { kXor1 = 0xb1, kXor2 = 0x4e, kXor4 = 0x141 };

template <int CTRL>
__device__ __forceinline__ uint32_t row_swap(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}

// Reductions over the wave's 64 lanes (all active), the same value in every
// lane: four rotations inside the rows of 16, then the four rows.
__device__ __forceinline__ double wave_sum(double v)
{
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    v += row_ror<1>(v);
    return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

__device__ __forceinline__ double wave_max(double v)
{
    v = fmax(v, row_ror<8>(v));
    v = fmax(v, row_ror<4>(v));
    v = fmax(v, row_ror<2>(v));
    v = fmax(v, row_ror<1>(v));
    return fmax(fmax(read_lane(v, 0), read_lane(v, 16)), fmax(read_lane(v, 32), read_lane(v, 48)));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, row_ror<8>(v));
    v = max(v, row_ror<4>(v));
    v = max(v, row_ror<2>(v));
    v = max(v, row_ror<1>(v));
    return max(max(read_lane(v, 0), read_lane(v, 16)), max(read_lane(v, 32), read_lane(v, 48)));
}

}  // namespace
}  // namespace mhc
