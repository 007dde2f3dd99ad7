// attention_join.h -- parts of attention's row blocks, of several workers, put
// together: what each leaves, where, and the kernel.
#pragma once

#include "attention_common.h"

namespace mhc {
namespace {

constexpr int kJoinWaves = 4;

// A partial result of a block of ROWS rows: maxima, sums, [ROWS][D] weighted
// values.  A worker's share leaves at most two: of its first and of its last block.
template <int D, int ROWS> __device__ __forceinline__ float *record(const AttentionParams &P, int64_t worker, bool first)
{
    return P.workspace + (2 * worker + (first ? 0 : 1)) * (int64_t)(ROWS * (D + 2));
}

// What is to be joined of a block: its parts are those of workers `from` on.
// parts is 0 where one worker has all of it.
struct alignas(8) Join {
    int from;
    int parts;          // below 2^13; its top bit: the first part is all of its worker's share
};

constexpr int kWholeShare = 1 << 30;

// Of the block with that number and that kv head
template <int D, int ROWS>
__device__ __forceinline__ Join *join_of(const AttentionParams &P, int number, int head)
{
    return (Join *)(P.workspace + 2 * (int64_t)P.workers * (ROWS * (D + 2))) + (int64_t)number * P.c.heads + head;
}

// What is to be joined of the block that begins in a worker's share and ends in
// another's: its first part is that worker's, the others the next ones'.
// count is as Join's parts.
struct alignas(16) Parts {
    int64_t row;        // the block's first output row, a head's of a query row
    int skip, rows;     // its first head in that query row's group; how many rows
    int count, none[3];
};

// Behind the joins of all blocks, as many as the batch may have
template <int D, int ROWS> __device__ __forceinline__ Parts *parts_of(const AttentionParams &P, int worker)
{
    const int64_t joins = 2 * P.blocks * P.c.heads;
    return (Parts *)(P.workspace + 2 * (int64_t)P.workers * (ROWS * (D + 2)) + (joins + 3) / 4 * 4) + worker;
}

inline uint64_t parts_floats(int workers) { return (uint64_t)workers * sizeof(Parts) / 4 + 4; }

// Four channels of a finished row of the output
template <int DT, int D>
__device__ __forceinline__ void store_row(const AttentionParams &P, int64_t at, int d, float4 o, float top, float sum)
{
    typedef Half<DT> H;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const u32x2 w = {H::pack(o.x * inv, o.y * inv), H::pack(o.z * inv, o.w * inv)};
    *(u32x2 *)(P.out + at * D + d) = w;
    if (P.lse && d == 0)
        P.lse[at] = sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum) - Softmax<DT>::kShift) * kLn2;
}

// The same, head `skip` behind those of query row i
template <int DT, int D>
__device__ __forceinline__ void store(const AttentionParams &P, int64_t i, int skip, int head, int d, float4 o,
                                      float top, float sum)
{
    const int over = skip / P.group;
    store_row<DT, D>(P, (i + over) * P.q_heads + head * P.group + (skip - over * P.group), d, o, top, sum);
}

// Puts together the blocks that several workers have parts of.  WAVES waves a
// row, D/4 lanes a part, eight parts a lane at once.
template <int DT, int D, int BLOCK, int WAVES>
__global__ __launch_bounds__(64 * kJoinWaves) void attention_join_kernel(const AttentionParams P)
{
    constexpr int ROWS = kJoinWaves / WAVES, LANES = D / 4, AT_ONCE = 64 / LANES * WAVES, BATCH = WAVES > 1 ? 8 : 2;
    __shared__ float4 L[kJoinWaves][LANES];
    __shared__ float2 M[kJoinWaves];
    const int64_t id = block_id(), segment = id / (BLOCK / ROWS), behind = segment / P.c.heads;
    if (behind >= P.blocks)
        return;
    const int number = (int)behind, head = (int)(segment - behind * P.c.heads);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int row = (int)(id % (BLOCK / ROWS)) * ROWS + wave / WAVES;
    // starts that fall give a block to two workers, or to none: in range all the same
    Join j = *join_of<D, BLOCK>(P, number, head);
    j.from = min(max(j.from, 0), P.workers - 1);
    int first;
    const int b = sequence_of(P, number, BLOCK, &first);
    const int from = row_start(P, b), rows = (row_start(P, b + 1) - from) * P.group;
    // every block's Join has been written, those of numbers that no block has not
    if (number < first || (number - first) * BLOCK >= rows)
        return;
    const int parts = min(j.parts & (kWholeShare - 1), P.workers - j.from);
    const int at = (number - first) * BLOCK;
    if (parts == 0 || (WAVES > 1 && at + row >= rows))      // the workgroup's all
        return;
    const int d = lane % LANES * 4;
    float most = kLowest, all = 0.0f;
    float4 o = {0, 0, 0, 0};
    if (at + row < rows)
        for (int i0 = wave % WAVES * (64 / LANES) + lane / LANES; i0 < parts; i0 += AT_ONCE * BATCH) {
            float top[BATCH], sum[BATCH];
            float4 x[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                // past the last: the last once more, with a weight of 0
                const int i = min(i0 + k * AT_ONCE, parts - 1);
                const float *rec = record<D, BLOCK>(P, j.from + i, i > 0 || (j.parts & kWholeShare));
                top[k] = rec[row];
                sum[k] = rec[BLOCK + row];
                x[k] = *(const float4 *)(rec + 2 * BLOCK + row * D + d);
            }
            float now = most;
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                now = fmaxf(now, top[k]);
            const float old = __builtin_amdgcn_exp2f(most - now);
            most = now;
            all *= old;
            o = {o.x * old, o.y * old, o.z * old, o.w * old};
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (i0 + k * AT_ONCE >= parts)
                    continue;
                const float w = __builtin_amdgcn_exp2f(top[k] - now);
                all += sum[k] * w;
                o = {o.x + x[k].x * w, o.y + x[k].y * w, o.z + x[k].z * w, o.w + x[k].w * w};
            }
        }
    auto add = [&](float top, float sum, const float4 &x) {
        const float now = fmaxf(most, top);
        const float a = __builtin_amdgcn_exp2f(most - now), c = __builtin_amdgcn_exp2f(top - now);
        most = now;
        all = all * a + sum * c;
        o = {o.x * a + x.x * c, o.y * a + x.y * c, o.z * a + x.z * c, o.w * a + x.w * c};
    };
#pragma unroll
    for (int x = LANES; x < 64; x <<= 1) {
        const float top = __shfl_xor(most, x), sum = __shfl_xor(all, x);
        const float4 v = {__shfl_xor(o.x, x), __shfl_xor(o.y, x), __shfl_xor(o.z, x), __shfl_xor(o.w, x)};
        add(top, sum, v);
    }
    if constexpr (WAVES > 1) {
        if (lane < LANES)
            L[wave][lane] = o;
        if (lane == 0)
            M[wave] = {most, all};
        __syncthreads();
        if (wave > 0)
            return;
        for (int w = 1; w < WAVES; ++w)
            add(M[w].x, M[w].y, L[w][lane % LANES]);
    }
    if (lane < LANES && at + row < rows) {
        const int i = at / P.group;
        store<DT, D>(P, from + i, at - i * P.group + row, head, d, o, most, all);
    }
}

// The same where most blocks have few parts: D/4 lanes a row, 16 rows a workgroup
template <int DT, int D, int BLOCK>
__global__ __launch_bounds__(256) void attention_join_shares_kernel(const AttentionParams P)
{
    constexpr int LANES = D / 4, ROWS = 256 / LANES, BATCH = 4, GROUP = 16;
    const int64_t id = block_id();
    const int worker = (int)(id / (BLOCK / GROUP));
    if (worker >= P.workers)
        return;
    const Parts j = *parts_of<D, BLOCK>(P, worker);
    const int count = j.count & ~kWholeShare, d = threadIdx.x % LANES * 4;
    if (count == 0)
        return;
    const int first = (int)(id % (BLOCK / GROUP)) * GROUP;
    for (int row = first + threadIdx.x / LANES; row < min(first + GROUP, j.rows); row += ROWS) {
        float most = kLowest, all = 0.0f;
        float4 o = {0, 0, 0, 0};
        for (int i0 = 0; i0 < count; i0 += BATCH) {
            float top[BATCH], sum[BATCH];
            float4 x[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = min(i0 + k, count - 1);
                const float *rec = record<D, BLOCK>(P, worker + i, i > 0 || (j.count & kWholeShare));
                top[k] = rec[row];
                sum[k] = rec[BLOCK + row];
                x[k] = *(const float4 *)(rec + 2 * BLOCK + row * D + d);
            }
            float now = most;
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                now = fmaxf(now, top[k]);
            const float old = __builtin_amdgcn_exp2f(most - now);
            most = now;
            all *= old;
            o = {o.x * old, o.y * old, o.z * old, o.w * old};
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (i0 + k >= count)
                    continue;
                const float w = __builtin_amdgcn_exp2f(top[k] - now);
                all += sum[k] * w;
                o = {o.x + x[k].x * w, o.y + x[k].y * w, o.z + x[k].z * w, o.w + x[k].w * w};
            }
        }
        const int over = (j.skip + row) / P.group;
        store_row<DT, D>(P, j.row + (int64_t)over * P.q_heads + (j.skip + row - over * P.group), d, o, most, all);
    }
}

// Floats of workspace for that many workers and blocks of `rows` rows
inline uint64_t join_floats(int workers, int64_t blocks, int rows, int D)
{
    return (uint64_t)workers * 2 * rows * (D + 2) + (uint64_t)blocks * sizeof(Join) / 4;
}

template <int DT, int D, int BLOCK> hipError_t launch_join(const AttentionParams &p, hipStream_t s)
{
    const int64_t segments = p.blocks * p.c.heads;
    if (segments * 4 <= p.workers)      // few blocks have many parts each
        attention_join_kernel<DT, D, BLOCK, kJoinWaves><<<grid_of(segments * BLOCK), 64 * kJoinWaves, 0, s>>>(p);
    else
        attention_join_kernel<DT, D, BLOCK, 1>
            <<<grid_of(segments * (BLOCK / kJoinWaves)), 64 * kJoinWaves, 0, s>>>(p);
    return hipGetLastError();
}

// Few blocks may have many parts each: the kernel for those
template <int DT, int D, int BLOCK> hipError_t launch_join_shares(const AttentionParams &p, hipStream_t s)
{
    const int64_t segments = p.blocks * p.c.heads;
    if (segments * 8 <= p.workers)
        attention_join_kernel<DT, D, BLOCK, kJoinWaves><<<grid_of(segments * BLOCK), 64 * kJoinWaves, 0, s>>>(p);
    else
        attention_join_shares_kernel<DT, D, BLOCK><<<grid_of((int64_t)p.workers * (BLOCK / 16)), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace
}  // namespace mhc
