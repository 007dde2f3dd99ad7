// int8_kernels.hip -- matrix product of int8 codes with a scale for each
// token (row of a) and each channel (row of b).
//
//   out[t][n] = round( f32( sum_k a[t][k] b[n][k] ) sa[t] sb[n] (+ bias[n]) )
//
// a [T][K] and b [N][K] int8, K contiguous in both; sa [T], sb [N] and bias
// [N] binary32; out bf16, fp16 or binary32.  The sum is exact: int32 holds
// 128 x 128 x K for every K the entry takes.  It is rounded once to binary32
// (exact below 2^24), then each product and the sum with the bias is rounded
// to binary32, then the result to the output's type.
//
// gfx950's v_mfma_i32_16x16x64_i8: lane l of an operand holds 16 consecutive
// bytes of row (A) or column (B) l % 16, and lane l of the result holds rows
// 4 (l / 16) + e of column l % 16.  Both operands are read with the same
// assignment of K to lanes and bytes, and a sum of integers does not depend
// on its order, so the assignment itself is free: here the 16-byte pieces
// l / 16 and l / 16 + 4 of a 128-wide step.
#include <hip/hip_runtime.h>

#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

typedef uint32_t u32;
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;   // K per step of the tiled kernels

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void *lds_ptr;

__device__ __forceinline__ rsrc_t make_rsrc(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes,
                                             0x00020000);
}

// 16 bytes a lane from memory into LDS: lane l's at byte 16 l of `to`.  (The
// host pass does not know the 16-byte form.)
__device__ __forceinline__ void load_lds(rsrc_t src, void *to, int offset, int step)
{
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_ptr)to, 16, offset, step, 0, 0);
#endif
}

// Waits until all but the last N of this wave's loads have completed.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// The workgroup barrier alone, without a fence that would wait for the
// stages' loads in flight: a wave's LDS reads have completed before it comes
// here, since its products have used them.
__device__ __forceinline__ void block_barrier()
{
    asm volatile("s_barrier" ::: "memory");
}

// ------------------------------------------------------------ tiled kernel --
//
// A workgroup of (TM / WM)(TN / WN) waves computes a TM x TN block, each wave
// WM x WN of it, in 128-wide K steps.  A step's rows go from memory straight
// into LDS (16 bytes a lane, 1 KB a wave and instruction: 8 rows of 128
// bytes); S stages keep S - 1 steps' loads in flight.  Piece c of row R lies
// in slot c ^ ((R >> 1) & 7) of its row, which puts the 16 lanes of a read
// phase on different banks.
template <int TM_, int TN_, int WM_, int WN_, int S_>
struct Tile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, S = S_;
    static constexpr int NW = (TM / WM) * (TN / WN);
    static constexpr int kThreads = 64 * NW;
    static constexpr int kRunsA = TM / 8 / NW, kRunsB = TN / 8 / NW;   // 1 KB runs per wave and step
    static constexpr int kLoads = kRunsA + kRunsB;
    static_assert(kRunsA * 8 * NW == TM && kRunsB * 8 * NW == TN, "whole runs per wave");
    static_assert(S >= 2 && (S - 1) * kLoads < 64, "the loads in flight fit the vmcnt counter");
};

template <class C>
struct StageT {
    int8_t a[C::TM * kStep];
    int8_t b[C::TN * kStep];
};

// Buffer resources based at the block's first rows, so that offsets fit 32
// bits whatever T K and N K, and this lane's offsets in them.  Rows past the
// end re-read the last.  In a last step that K does not fill, a row's pieces
// past K hold the next row's bytes (past the last row the resource ends and
// nothing outside is read); the products leave them out.
template <class C>
struct SrcT {
    rsrc_t a, b;
    int oa[C::kRunsA], ob[C::kRunsB];
};

template <class C>
__device__ __forceinline__ SrcT<C> src_tile(const Int8GemmParams &P, int m_blk, int n_blk, int wave,
                                           int lane)
{
    const int ra = min(C::TM, P.T - m_blk), rb = min(C::TN, P.N - n_blk);
    SrcT<C> s;
    s.a = make_rsrc(P.a + (size_t)m_blk * P.K, (uint32_t)(ra * P.K));
    s.b = make_rsrc(P.b + (size_t)n_blk * P.K, (uint32_t)(rb * P.K));
    const int slot = lane & 7;
#pragma unroll
    for (int i = 0; i < C::kRunsA; ++i) {
        const int row = 8 * (wave * C::kRunsA + i) + (lane >> 3);
        s.oa[i] = min(row, ra - 1) * P.K + 16 * (slot ^ ((row >> 1) & 7));
    }
#pragma unroll
    for (int i = 0; i < C::kRunsB; ++i) {
        const int row = 8 * (wave * C::kRunsB + i) + (lane >> 3);
        s.ob[i] = min(row, rb - 1) * P.K + 16 * (slot ^ ((row >> 1) & 7));
    }
    return s;
}

template <class C>
__device__ __forceinline__ void fetch_step(const SrcT<C> &s, int ks, StageT<C> &st, int wave)
{
#pragma unroll
    for (int i = 0; i < C::kRunsA; ++i)
        load_lds(s.a, st.a + 1024 * (wave * C::kRunsA + i), s.oa[i], ks * kStep);
#pragma unroll
    for (int i = 0; i < C::kRunsB; ++i)
        load_lds(s.b, st.b + 1024 * (wave * C::kRunsB + i), s.ob[i], ks * kStep);
}

// Block order: consecutive workgroups go to the 8 XCDs in turn, and XCD x
// takes the x-th eighth of the blocks, 4 row blocks by all column blocks at
// a time, so that the workgroups resident on an XCD share rows in its L2.
constexpr int kGroupRows = 4;

__device__ __forceinline__ bool block_of(int w, int mb, int nb, int &m, int &n)
{
    const int total = mb * nb, per_xcd = (total + 7) / 8;
    const int L = (w % 8) * per_xcd + w / 8;
    if (L >= total)
        return false;
    const int group = L / (kGroupRows * nb), first = group * kGroupRows;
    const int gm = min(mb - first, kGroupRows), in = L % (kGroupRows * nb);
    m = first + in % gm;
    n = in / gm;
    return true;
}

template <class O>
__device__ __forceinline__ O finish(int acc, float sa, float sb, float bias, bool has_bias)
{
    const float v = ((float)acc * sa) * sb;
    return (O)rounded(has_bias ? v + bias : v);
}

template <class C, class O>
__global__ __launch_bounds__(C::kThreads, 1) void int8_gemm_tile_kernel(Int8GemmParams P)
{
    constexpr int MI = C::WM / 16, NJ = C::WN / 16, S = C::S;
    __shared__ StageT<C> st[S];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int T = P.T, N = P.N;
    int mi, ni;
    if (!block_of(blockIdx.x, (T + C::TM - 1) / C::TM, (N + C::TN - 1) / C::TN, mi, ni))
        return;
    const int m_blk = mi * C::TM, n_blk = ni * C::TN;
    const int wm = (wave / (C::TN / C::WN)) * C::WM, wn = (wave % (C::TN / C::WN)) * C::WN;
    const int g = lane >> 4, r = lane & 15;
    const int p0 = 16 * (g ^ (r >> 1)), p1 = p0 ^ 64;   // slots of pieces g and g + 4 of row r
    i32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    const int steps = (P.K + kStep - 1) / kStep;
    const int pieces = (P.K - (steps - 1) * kStep) / 16;   // of the last step
    const SrcT<C> src = src_tile<C>(P, m_blk, n_blk, wave, lane);
    // Steps past the end re-read the last into a free stage: every step has
    // the same loads in flight, so the waits are constants.
#pragma unroll
    for (int p = 0; p < S - 1; ++p)
        fetch_step<C>(src, min(p, steps - 1), st[p], wave);
    int cur_s = 0, next_s = S - 1;
    for (int ks = 0; ks < steps; ++ks) {
        wait_vm<(S - 2) * C::kLoads>();   // this wave's loads of step ks are in LDS
        block_barrier();                   // every wave's are, and step ks - 1's stage is free
        fetch_step<C>(src, min(ks + S - 1, steps - 1), st[next_s], wave);
        __builtin_amdgcn_sched_barrier(0);
        const StageT<C> &cur = st[cur_s];
        const bool ragged = ks == steps - 1 && pieces < 8;
        i32x4 b0[NJ], b1[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int8_t *p = cur.b + (wn + 16 * j + r) * kStep;
            b0[j] = *reinterpret_cast<const i32x4 *>(p + p0);
            b1[j] = *reinterpret_cast<const i32x4 *>(p + p1);
            if (ragged) {   // integers: a zero on one side leaves the product out
                if (g >= pieces)
                    b0[j] = i32x4{0, 0, 0, 0};
                if (g + 4 >= pieces)
                    b1[j] = i32x4{0, 0, 0, 0};
            }
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int8_t *p = cur.a + (wm + 16 * i + r) * kStep;
            const i32x4 a0 = *reinterpret_cast<const i32x4 *>(p + p0);
            const i32x4 a1 = *reinterpret_cast<const i32x4 *>(p + p1);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, b0[j], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, b1[j], acc[i][j], 0, 0, 0);
        }
        __builtin_amdgcn_s_setprio(0);
        cur_s = cur_s == S - 1 ? 0 : cur_s + 1;
        next_s = next_s == S - 1 ? 0 : next_s + 1;
    }
    wait_vm<0>();      // the re-reads past the end have landed
    __syncthreads();   // and every wave is done with the stages
    O *out = static_cast<O *>(P.out);
    float sb[NJ], bias[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int col = min(n_blk + wn + 16 * j + r, N - 1);
        sb[j] = P.sb[col];
        bias[j] = P.bias ? P.bias[col] : 0.0f;
    }
    if constexpr (sizeof(O) == 4) {
        // 16 lanes store 64 consecutive bytes
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = m_blk + wm + 16 * i + 4 * g + e;
                if (row >= T)
                    continue;
                const float sa = P.sa[row];
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int col = n_blk + wn + 16 * j + r;
                    if (col < N)
                        out[(size_t)row * N + col] =
                            finish<O>(acc[i][j][e], sa, sb[j], bias[j], P.bias != nullptr);
                }
            }
    } else {
        // the block in LDS, then 16-byte row pieces to memory
        static_assert(sizeof(O) == 4 || S * sizeof(StageT<C>) >= C::TM * C::TN * sizeof(O),
                      "the output block fits the stages");
        O *ot = reinterpret_cast<O *>(&st[0]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = wm + 16 * i + 4 * g + e;
                const float sa = P.sa[min(m_blk + row, T - 1)];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    ot[row * C::TN + wn + 16 * j + r] =
                        finish<O>(acc[i][j][e], sa, sb[j], bias[j], P.bias != nullptr);
            }
        __syncthreads();
        const bool whole = N % 8 == 0;
        for (int c = tid; c < C::TM * C::TN / 8; c += C::kThreads) {
            const int row = c / (C::TN / 8), col = (c % (C::TN / 8)) * 8;
            const int gr = m_blk + row, gc = n_blk + col;
            if (gr >= T || gc >= N)
                continue;
            O *dst = out + (size_t)gr * N + gc;
            const O *e8 = ot + row * C::TN + col;
            if (whole) {
                *reinterpret_cast<u32x4 *>(dst) = *reinterpret_cast<const u32x4 *>(e8);
            } else {
                for (int e = 0; e < 8 && gc + e < N; ++e)
                    dst[e] = e8[e];
            }
        }
    }
}

using BigTile = Tile<256, 256, 64, 128, 2>;
using MidTile = Tile<128, 128, 64, 64, 3>;
using SmallTile = Tile<64, 64, 32, 32, 3>;
using Tile32 = Tile<32, 32, 16, 16, 6>;

template <class C, class O>
hipError_t launch_tile(const Int8GemmParams &p, hipStream_t s)
{
    const int64_t total = (int64_t)((p.T + C::TM - 1) / C::TM) * ((p.N + C::TN - 1) / C::TN);
    if (total > INT32_MAX / 2)
        return hipErrorInvalidValue;
    const int grid = (int)((total + 7) / 8 * 8);   // whole rounds of the 8 XCDs
    hipLaunchKernelGGL((int8_gemm_tile_kernel<C, O>), dim3(grid), dim3(C::kThreads), 0, s, p);
    return hipGetLastError();
}

template <class O>
hipError_t launch_shape(const Int8GemmParams &p, const GemmBlocks &g, hipStream_t s)
{
#define SHAPE(C)                                                                            \
    if (g.tm == C::TM && g.tn == C::TN)                                                     \
        return launch_tile<C, O>(p, s);
    SHAPE(BigTile)
    SHAPE(MidTile)
    SHAPE(SmallTile)
    SHAPE(Tile32)
#undef SHAPE
    return hipErrorInvalidValue;
}

}  // namespace

GemmBlocks int8_gemm_blocks(int64_t T, int N, int cus)
{
    auto blocks = [&](int tm, int tn) {
        return ((T + tm - 1) / tm) * (int64_t)((N + tn - 1) / tn);
    };
    if (blocks(256, 256) >= cus)
        return {256, 256, 2};
    if (blocks(128, 128) >= cus)
        return {128, 128, 3};
    if (blocks(64, 64) >= cus)
        return {64, 64, 3};
    return {32, 32, 6};
}

hipError_t launch_int8_gemm(const Int8GemmParams &p, int out_dtype, int cus, hipStream_t s)
{
    if (p.T == 0)
        return hipSuccess;
    const GemmBlocks g = int8_gemm_blocks(p.T, p.N, cus);
    if (out_dtype == MHC_F32)
        return launch_shape<float>(p, g, s);
    return out_dtype == MHC_BF16 ? launch_shape<__bf16>(p, g, s) : launch_shape<_Float16>(p, g, s);
}

}  // namespace mhc
