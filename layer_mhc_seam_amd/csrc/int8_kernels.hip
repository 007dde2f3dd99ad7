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
// l / 16 + 4 q of a step.
//
// What bounds it, at N = K = 5120 (times in a graph of such products over four
// sets of operands in turn, beyond the L2, within the 256 MB behind it): T = 1
// the weights' bytes, 6.4 us, 2 of them the launch (4.1 TB/s; a bare read of
// them takes 5.4); T = 384 the rows' way from L2 into LDS, 17.3 to 18.0 us
// (983 KB a CU, 17 TB/s in all; these loads alone, without products, take
// 12.8; larger wave tiles with half the LDS reads, LDS reads moved between the
// products, steps begun elsewhere in each block took as long), and 19.9 to
// 20.5 at K = 5136, whose rows do not start on 128 bytes, so that a piece
// touches three lines for two; T = 16384 the clock under the products and the
// loads: 340 us at best (2.53 PFLOP/s), 380 to 395 call after call (2.2), the
// loads alone 295 and the products alone 235 (4.0 PFLOP/s is the instruction's
// own rate over Gaussian codes, 4.7 over zeros).
// Operands straight into registers, without LDS: 9 us at T = 1, since 64-byte
// pieces of rows come at two thirds of the rate of 128-byte ones.
#include <hip/hip_runtime.h>

#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

typedef uint32_t u32;
typedef u32 u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

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

// The workgroup barrier with this wave's LDS reads complete, and without a
// fence, which would wait for the stages' loads in flight too.
__device__ __forceinline__ void block_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// ------------------------------------------------------------ tiled kernel --
//
// A workgroup of KW (TM / WM)(TN / WN) waves computes a TM x TN block, each wave
// WM x WN of it over a KW-th of every step of KS = 128, 256 or 512 of K; sums
// of the KW parts are joined at the end.  (Small blocks wait for a step's chain
// of LDS reads and products more than for its bytes.  T = 4, N = 256, K = 5120
// with 16 x 32 and KW 1, 2 and 4, then 16 x 16 and 8: 5.6, 5.0, 4.8, 4.4 us; T =
// 32, N = 5120 with 32 x 32 and KW 1 and 2: 7.7 and 7.2; blocks of 64 x 64 and
// more gain nothing.)  A step's rows go from
// memory straight into LDS (16 bytes a lane, 1 KB a wave and instruction:
// 1024 / KS rows of KS bytes); S stages keep S - 1 steps' loads in flight.
// Piece c of row R lies in slot c ^ turn(R) of its row, which puts the 16
// lanes of a read phase (16 rows, one piece each) on different banks: two
// rows of 128 bytes, or 256 of a row, cover the banks once.
template <int TM_, int TN_, int WM_, int WN_, int S_, int KS_ = 128, int KW_ = 1>
struct Tile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, S = S_, KS = KS_, KW = KW_;
    static constexpr int kTiles = (TM / WM) * (TN / WN), NW = kTiles * KW;
    static constexpr int kThreads = 64 * NW;
    static constexpr int kPieces = KS / 16, kRunRows = 1024 / KS;   // of a row; of a 1 KB run
    static constexpr int kRunsA = TM / kRunRows / NW, kRunsB = TN / kRunRows / NW;   // a wave's
    static constexpr int kLoads = kRunsA + kRunsB;
    static constexpr int kFactors = (TM + 2 * TN + kThreads - 1) / kThreads;   // a thread's
    static_assert(KS == 128 || KS == 256 || KS == 512, "turn() is for these");
    static_assert(kRunsA * kRunRows * NW == TM && kRunsB * kRunRows * NW == TN,
                  "whole runs per wave");
    static_assert(S >= 2 && (S - 1) * kLoads + kFactors < 64,
                  "the loads in flight fit the vmcnt counter");
    static_assert(S * (TM + TN) * KS >= TM * TN * 2, "16-bit results fit the stages");
    static_assert(S * (TM + TN) * KS >= (KW - 1) * TM * TN * 4, "and the parts' sums do");
    static_assert(KS / 64 % KW == 0, "whole products per part");
    static __device__ __forceinline__ int turn(int row)
    {
        return KS == 128 ? row >> 1 & 7 : row & 15;
    }
};

template <class C>
struct StageT {
    alignas(16) int8_t a[C::TM * C::KS];
    alignas(16) int8_t b[C::TN * C::KS];
};

// A workgroup's LDS.  (One object: beside a second one the compiler waits for
// every load in flight before it reads the first.)
template <class C>
struct TileLds {
    StageT<C> st[C::S];
    float factor[C::TM + 2 * C::TN];   // the block's sa, sb and bias
};

// Buffer resources based at the block's first rows, so that offsets fit 32
// bits whatever T K and N K, and this lane's offsets in them.  Rows past the
// end re-read the last.  In a last step that K does not fill, a row's pieces
// past K hold the next row's bytes (past the last row the resource ends and
// nothing outside is read); zero_tail leaves them out.
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
    const int slot = lane % C::kPieces, sub = lane / C::kPieces;
#pragma unroll
    for (int i = 0; i < C::kRunsA; ++i) {
        const int row = C::kRunRows * (wave * C::kRunsA + i) + sub;
        s.oa[i] = min(row, ra - 1) * P.K + 16 * (slot ^ C::turn(row));
    }
#pragma unroll
    for (int i = 0; i < C::kRunsB; ++i) {
        const int row = C::kRunRows * (wave * C::kRunsB + i) + sub;
        s.ob[i] = min(row, rb - 1) * P.K + 16 * (slot ^ C::turn(row));
    }
    return s;
}

template <class C>
__device__ __forceinline__ void fetch_step(const SrcT<C> &s, int ks, StageT<C> &st, int wave)
{
#pragma unroll
    for (int i = 0; i < C::kRunsA; ++i)
        load_lds(s.a, st.a + 1024 * (wave * C::kRunsA + i), s.oa[i], ks * C::KS);
#pragma unroll
    for (int i = 0; i < C::kRunsB; ++i)
        load_lds(s.b, st.b + 1024 * (wave * C::kRunsB + i), s.ob[i], ks * C::KS);
}

// Block order: consecutive workgroups go to the 8 XCDs in turn, and XCD x
// takes the x-th eighth of the blocks, 4 row blocks by all column blocks at
// a time, so that the workgroups resident on an XCD share rows in its L2.
constexpr int kGroupRows = 4;

__device__ __forceinline__ bool block_of(int w, int mb, int nb, int &m, int &n)
{
    const int total = mb * nb, per_xcd = (total + 7) / 8;
    const int L = (w % 8) * per_xcd + w / 8;
    if (w >= 8 * per_xcd || L >= total)
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

// The block's results from a wave's sums: binary32 straight to memory (16
// lanes store 64 consecutive bytes), 16-bit types by way of LDS (`ot`, free by
// now) to 16-byte pieces of rows, or single elements, 64 in a row, where rows
// do not start on 16 bytes.  factor: the block's sa, sb and bias.  The first
// of the KW parts' waves hold the sums.
template <class C, class O>
__device__ __forceinline__ void store_block(const Int8GemmParams &P, int m_blk, int n_blk, int wm,
                                            int wn, const i32x4 (&acc)[C::WM / 16][C::WN / 16],
                                            const float *factor, O *ot)
{
    constexpr int MI = C::WM / 16, NJ = C::WN / 16;
    const int tid = threadIdx.x, g = tid >> 4 & 3, r = tid & 15;
    const int T = P.T, N = P.N;
    O *out = static_cast<O *>(P.out);
    float sb[NJ], bias[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        sb[j] = factor[C::TM + wn + 16 * j + r];
        bias[j] = factor[C::TM + C::TN + wn + 16 * j + r];
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4 && (C::KW == 1 || tid < 64 * C::kTiles); ++e) {
            const int row = wm + 16 * i + 4 * g + e;
            const float sa = factor[row];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int col = wn + 16 * j + r;
                const O v = finish<O>(acc[i][j][e], sa, sb[j], bias[j], P.bias != nullptr);
                if constexpr (sizeof(O) == 2)
                    ot[row * C::TN + col] = v;
                else if (m_blk + row < T && n_blk + col < N)
                    out[(size_t)(m_blk + row) * N + n_blk + col] = v;
            }
        }
    if constexpr (sizeof(O) == 2) {
        __syncthreads();
        const int rows = min(C::TM, T - m_blk), cols = min(C::TN, N - n_blk);
        O *to = out + (size_t)m_blk * N + n_blk;
        if (N % 8 == 0) {
            for (int c = tid; c < C::TM * C::TN / 8; c += C::kThreads) {
                const int row = c / (C::TN / 8), col = c % (C::TN / 8) * 8;
                if (row < rows && col < cols)
                    *reinterpret_cast<u32x4 *>(to + (size_t)row * N + col) =
                        *reinterpret_cast<const u32x4 *>(ot + row * C::TN + col);
            }
        } else {
            for (int c = tid; c < C::TM * C::TN; c += C::kThreads) {
                const int row = c / C::TN, col = c % C::TN;
                if (row < rows && col < cols)
                    to[(size_t)row * N + col] = ot[c];
            }
        }
    }
}

// sa, sb or bias of the block's i-th factor
template <class C>
__device__ __forceinline__ float factor_of(const Int8GemmParams &P, int m_blk, int n_blk, int i)
{
    const int col = i - C::TM;
    return i < C::TM           ? P.sa[min(m_blk + i, P.T - 1)]
           : col < C::TN       ? P.sb[min(n_blk + col, P.N - 1)]
           : P.bias != nullptr ? P.bias[min(n_blk + col - C::TN, P.N - 1)]
                               : 0.0f;
}

// A last step that K does not fill: zeros in B's pieces past K leave the
// products out, whatever A's rows hold there.
template <class C>
__device__ __forceinline__ void zero_tail(int8_t *b, int pieces)
{
    const int rest = C::kPieces - pieces;
    for (int i = threadIdx.x; i < C::TN * rest; i += C::kThreads) {
        const int row = i / rest, piece = pieces + i % rest;
        *reinterpret_cast<i32x4 *>(b + row * C::KS + 16 * (piece ^ C::turn(row))) =
            i32x4{0, 0, 0, 0};
    }
    __syncthreads();
}

template <class C, class O>
__global__ __launch_bounds__(C::kThreads, 1) void int8_gemm_tile_kernel(Int8GemmParams P)
{
    constexpr int MI = C::WM / 16, NJ = C::WN / 16, S = C::S;
    __shared__ TileLds<C> lds;
    StageT<C>(&st)[S] = lds.st;
    float(&factor)[C::TM + 2 * C::TN] = lds.factor;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int T = P.T, N = P.N;
    int mi, ni;
    if (!block_of((int)block_id(), (T - 1) / C::TM + 1, (N - 1) / C::TN + 1, mi, ni))
        return;
    const int m_blk = mi * C::TM, n_blk = ni * C::TN;
    const int part = wave / C::kTiles, tile = wave % C::kTiles;
    const int wm = (tile / (C::TN / C::WN)) * C::WM, wn = (tile % (C::TN / C::WN)) * C::WN;
    const int g = lane >> 4, r = lane & 15;
    constexpr int Q = C::KS / 64 / C::KW;   // products of a step: pieces g + 4 q of row r
    int at[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        at[q] = r * C::KS + 16 * ((g + 4 * (part * Q + q)) ^ C::turn(r));
    i32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    // The factors are asked for first: their way from memory is as long as
    // several steps, and the first rows' follows on its heels.
    float f[C::kFactors];
#pragma unroll
    for (int i = 0; i < C::kFactors; ++i)
        f[i] = factor_of<C>(P, m_blk, n_blk, min(tid + i * C::kThreads, C::TM + 2 * C::TN - 1));
    __builtin_amdgcn_sched_barrier(0);
    const int steps = (P.K + C::KS - 1) / C::KS;
    const int pieces = (P.K - (steps - 1) * C::KS) / 16;   // of the last step
    const SrcT<C> src = src_tile<C>(P, m_blk, n_blk, wave, lane);
    // Steps past the end re-read the last into a free stage: every step has
    // the same loads in flight, so the waits are constants.
#pragma unroll
    for (int p = 0; p < S - 1; ++p)
        fetch_step<C>(src, min(p, steps - 1), st[p], wave);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C::kFactors; ++i)
        if (tid + i * C::kThreads < C::TM + 2 * C::TN)
            factor[tid + i * C::kThreads] = f[i];
    int cur_s = 0, next_s = S - 1;
    for (int ks = 0; ks < steps; ++ks) {
        wait_vm<(S - 2) * C::kLoads>();   // this wave's loads of step ks are in LDS
        block_barrier();                   // every wave's are, and step ks - 1's stage is free
        fetch_step<C>(src, min(ks + S - 1, steps - 1), st[next_s], wave);
        __builtin_amdgcn_sched_barrier(0);
        const StageT<C> &cur = st[cur_s];
        if (ks == steps - 1 && pieces < C::kPieces)
            zero_tail<C>(st[cur_s].b, pieces);
        i32x4 b[NJ][Q];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int q = 0; q < Q; ++q)
                b[j][q] = *reinterpret_cast<const i32x4 *>(cur.b + (wn + 16 * j) * C::KS + at[q]);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            i32x4 a[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q)
                a[q] = *reinterpret_cast<const i32x4 *>(cur.a + (wm + 16 * i) * C::KS + at[q]);
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[q], b[j][q], acc[i][j], 0,
                                                                      0, 0);
        }
        __builtin_amdgcn_s_setprio(0);
        cur_s = cur_s == S - 1 ? 0 : cur_s + 1;
        next_s = next_s == S - 1 ? 0 : next_s + 1;
    }
    wait_vm<0>();      // the re-reads past the end have landed
    __syncthreads();   // and every wave is done with the stages
    if constexpr (C::KW > 1) {
        constexpr int kEach = 64 * MI * NJ;
        i32x4 *sums = reinterpret_cast<i32x4 *>(&st[0]) + tile * kEach + lane;
#pragma unroll
        for (int i = 0; i < MI * NJ; ++i)
            if (part > 0)
                sums[(part - 1) * C::kTiles * kEach + 64 * i] = acc[i / NJ][i % NJ];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < C::KW - 1; ++k)
#pragma unroll
            for (int i = 0; i < MI * NJ; ++i)
                if (part == 0)
                    acc[i / NJ][i % NJ] += sums[k * C::kTiles * kEach + 64 * i];
        __syncthreads();
    }
    store_block<C, O>(P, m_blk, n_blk, wm, wn, acc, factor, reinterpret_cast<O *>(&st[0]));
}

// --------------------------------------------------------- 256 x 256 blocks --
//
// The largest block, for many rows: 8 waves of 64 x 128 and 128-wide steps,
// whose loads, LDS reads and products overlap in each wave.  A step's products
// take two halves of 64 of K.  While one half's are issued, the other half's
// fragments (or the next step's first) come from LDS into registers, one read
// for two products.  In the middle of a step all of its rows are in
// registers; after a barrier there the loads of later steps overwrite them.
// LDS holds five half steps (A or B rows, 32 KB each, 160 KB in all) in a
// ring: when a step's rows have to be there, the A rows of the one after it
// are still on their way, so loads never run dry.
using RingTile = Tile<256, 256, 64, 128, 2>;

template <class O>
__global__ __launch_bounds__(RingTile::kThreads, 1) void int8_gemm_ring_kernel(Int8GemmParams P)
{
    using C = RingTile;
    constexpr int MI = C::WM / 16, NJ = C::WN / 16, kSlots = 5, kSlot = C::TM * C::KS;
    constexpr int kHalf = C::kRunsA;   // loads of a half step, a wave's
    static_assert(C::TM == C::TN, "A and B rows share the slots");
    static_assert(kSlots * kSlot >= C::TM * C::TN * 2 + 4 * (C::TM + 2 * C::TN),
                  "16-bit results and the factors fit");
    __shared__ alignas(16) int8_t lds[kSlots * kSlot];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int mi, ni;
    if (!block_of((int)block_id(), (P.T - 1) / C::TM + 1, (P.N - 1) / C::TN + 1, mi, ni))
        return;
    const int m_blk = mi * C::TM, n_blk = ni * C::TN;
    const int wm = (wave / (C::TN / C::WN)) * C::WM, wn = (wave % (C::TN / C::WN)) * C::WN;
    const int g = lane >> 4, r = lane & 15;
    const int at[2] = {r * C::KS + 16 * (g ^ C::turn(r)), r * C::KS + 16 * ((g + 4) ^ C::turn(r))};
    i32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    const int steps = (P.K + C::KS - 1) / C::KS;
    const int pieces = (P.K - (steps - 1) * C::KS) / 16;   // of the last step
    const bool ragged = pieces < C::kPieces;
    const SrcT<C> src = src_tile<C>(P, m_blk, n_blk, wave, lane);
    // steps past the end re-read the last, so that waits are constants
    auto fetch_a = [&](int ks, int slot) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
            load_lds(src.a, lds + slot * kSlot + 1024 * (wave * kHalf + i), src.oa[i],
                     min(ks, steps - 1) * C::KS);
    };
    auto fetch_b = [&](int ks, int slot) {
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
            load_lds(src.b, lds + slot * kSlot + 1024 * (wave * kHalf + i), src.ob[i],
                     min(ks, steps - 1) * C::KS);
    };
    i32x4 a0[MI], b0[NJ], a1[MI], b1[NJ];   // fragments of a step's halves
    auto read = [&](i32x4(&a)[MI], i32x4(&b)[NJ], int slot_a, int slot_b, int half) {
        const int8_t *pa = lds + slot_a * kSlot + wm * C::KS + at[half];
        const int8_t *pb = lds + slot_b * kSlot + wn * C::KS + at[half];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            b[j] = *reinterpret_cast<const i32x4 *>(pb + 16 * C::KS * j);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            a[i] = *reinterpret_cast<const i32x4 *>(pa + 16 * C::KS * i);
    };
    // the products, two for each of the reads asked for before them
    auto multiply = [&](const i32x4(&a)[MI], const i32x4(&b)[NJ]) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < MI + NJ; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);   // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, MI * NJ - 2 * (MI + NJ), 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    fetch_a(0, 0);
    fetch_b(0, 1);
    fetch_a(1, 2);
    fetch_b(1, 3);
    fetch_a(2, 4);
    wait_vm<3 * kHalf>();
    block_barrier();
    if (ragged && steps == 1)
        zero_tail<C>(lds + kSlot, pieces);
    int slot_a = 0, slot_b = 1;
    float f[C::kFactors] = {};
    read(a0, b0, slot_a, slot_b, 0);
    for (int ks = 0; ks < steps; ++ks) {
        const int next_a = slot_a >= kSlots - 2 ? slot_a - (kSlots - 2) : slot_a + 2;
        const int next_b = slot_b >= kSlots - 2 ? slot_b - (kSlots - 2) : slot_b + 2;
        read(a1, b1, slot_a, slot_b, 1);
        multiply(a0, b0);
        wait_vm<kHalf>();   // the next step's rows are in LDS, the A rows after them may not be
        block_barrier();    // and this step's in every wave's registers
        if (ragged && ks + 1 == steps - 1)
            zero_tail<C>(lds + next_b * kSlot, pieces);
        fetch_b(ks + 2, slot_a);
        fetch_a(ks + 3, slot_b);
        if (ks == steps - 1)
#pragma unroll
            for (int i = 0; i < C::kFactors; ++i)
                f[i] = factor_of<C>(P, m_blk, n_blk, min(tid + i * C::kThreads,
                                                         C::TM + 2 * C::TN - 1));
        __builtin_amdgcn_sched_barrier(0);
        read(a0, b0, next_a, next_b, 0);
        multiply(a1, b1);
        slot_a = next_a;
        slot_b = next_b;
    }
    wait_vm<0>();      // the re-reads past the end have landed
    __syncthreads();   // and every wave is done with the slots
    float *factor = reinterpret_cast<float *>(lds + C::TM * C::TN * 2);
#pragma unroll
    for (int i = 0; i < C::kFactors; ++i)
        if (tid + i * C::kThreads < C::TM + 2 * C::TN)
            factor[tid + i * C::kThreads] = f[i];
    __syncthreads();
    store_block<C, O>(P, m_blk, n_blk, wm, wn, acc, factor, reinterpret_cast<O *>(lds));
}

// The shapes a launch chooses from, smallest first, with what a round of the
// CUs costs: measured times of one workgroup a CU at K = 5120 less the
// launch's 2 us, in units of half a microsecond.  K is not asked for: the
// prologue, the re-reads and the store weigh more at short depths than these
// costs say.  Few rows of K a step leave the small blocks waiting at barriers
// (16 x 32 with KW 1 in steps of 128, 256 and 512: 7.7, 6.7 and 6.4 us at T = 1,
// N = K = 5120); from 128 x 128 on LDS has no room for more than 128.
template <class F>
void int8_shapes(F &&f)
{
    f(Tile<16, 16, 16, 16, 4, 512, 8>(), 5);
    f(Tile<16, 32, 16, 16, 3, 512, 2>(), 10);
    f(Tile<32, 32, 16, 16, 4, 256, 2>(), 11);
    f(Tile<32, 64, 16, 32, 4, 256, 2>(), 15);
    f(Tile<64, 64, 16, 32, 3, 256>(), 21);
    f(Tile<96, 64, 48, 16, 3, 256>(), 28);
    f(Tile<128, 64, 32, 32, 3, 256>(), 32);
    f(Tile<128, 128, 32, 32, 4, 128>(), 45);
    f(Tile<128, 192, 32, 96, 3, 128>(), 62);
    f(Tile<128, 256, 64, 64, 3, 128>(), 75);
    f(Tile<192, 256, 96, 64, 2, 128>(), 100);
    f(RingTile(), 122);
}

template <class C, class O>
hipError_t launch_tile(const Int8GemmParams &p, hipStream_t s)
{
    const int64_t total = (int64_t)((p.T - 1) / C::TM + 1) * ((p.N - 1) / C::TN + 1);
    if (total > INT32_MAX / 2)
        return hipErrorInvalidValue;
    const dim3 grid = grid_of((total + 7) / 8 * 8), block(C::kThreads);   // rounds of the XCDs
    if constexpr (C::TM == RingTile::TM)
        hipLaunchKernelGGL(int8_gemm_ring_kernel<O>, grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((int8_gemm_tile_kernel<C, O>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <class O>
hipError_t launch_shape(const Int8GemmParams &p, const GemmBlocks &g, hipStream_t s)
{
    hipError_t e = hipErrorInvalidValue;
    int8_shapes([&](auto shape, int) {
        using C = decltype(shape);
        if (g.tm == C::TM && g.tn == C::TN)
            e = launch_tile<C, O>(p, s);
    });
    return e;
}

}  // namespace

// The shape whose rounds of the CUs cost least, the larger on a tie.
GemmBlocks int8_gemm_blocks(int64_t T, int N, int cus)
{
    GemmBlocks best{};
    int64_t least = INT64_MAX;
    int8_shapes([&](auto shape, int cost) {
        using C = decltype(shape);
        const int64_t blocks = ((T + C::TM - 1) / C::TM) * (int64_t)((N + C::TN - 1) / C::TN);
        const int64_t total = (blocks + cus - 1) / cus * cost;
        if (total <= least) {
            least = total;
            best = {C::TM, C::TN, C::S};
        }
    });
    return best;
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
