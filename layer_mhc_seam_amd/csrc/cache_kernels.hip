// cache_kernels.hip -- keys and values into the 4-bit cache and out of it.
//
// A group of 32 channels shares the scale 2^e, e the smallest whole number
// with 6 * 2^e >= the group's largest magnitude a: with a = f 2^E, 1 <= f < 2,
// that is E - 2 where f <= 1.5 and E - 1 above.  The codes are the nearest
// e2m1 values of v 2^-e, ties to the even code, which gfx950 converts two at a
// time; e is held where every value of the grid is exact in the tensors' type.
#include <hip/hip_runtime.h>

#include "cache_layout.h"
#include "half_ops.h"
#include "lane_ops.h"
#include "seam_internal.h"

namespace mhc {
namespace {

constexpr int kCacheThreads = 256;

__device__ __forceinline__ int64_t slot_of(const CacheParams &P, int64_t t)
{
    return P.slot_bytes == 8 ? ((const int64_t *)P.slots)[t] : ((const int32_t *)P.slots)[t];
}

// D/8 lanes a row of 8 channels each, four lanes a group; a workgroup takes
// 2048 / D tokens of one head, keys or values: their codes lie side by side
// where the slots follow each other.
template <int DT, int D>
__global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(const CacheParams P)
{
    typedef Half<DT> H;
    constexpr int LANES = D / 8, ROWS = kCacheThreads / LANES;
    const int64_t id = block_id();
    const int kind = (int)(id & 1), row = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int64_t rest = id >> 1, block = rest / P.c.heads;
    const int head = (int)(rest - block * P.c.heads);
    const int64_t t = block * ROWS + row;
    if (t >= P.T)      // whole groups of four lanes leave together
        return;
    int64_t page;
    int32_t at;
    if (!cache_slot(P.c, slot_of(P, t), &page, &at))
        return;
    const uint16_t *src = kind ? (const uint16_t *)P.v + t * P.v_token + head * P.v_head
                               : (const uint16_t *)P.k + t * P.k_token + head * P.k_head;
    const u32x4 w = *(const u32x4 *)(src + lane * 8);
    u32 most = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        most = max(most, max(w[j] & 0x7fff, (w[j] >> 16) & 0x7fff));
    }
    most = max(most, row_swap<kXor1>(most));
    most = max(most, row_swap<kXor2>(most));
    const bool fine = most < H::kInf;
    const u32 bits = __float_as_uint(H::low(most));
    int e = (int)(bits >> 23) - 127 - ((bits & 0x7fffff) <= 0x400000 ? 2 : 1);
    e = min(max(e, H::kLow), H::kHigh);
    const u32 byte = fine ? (u32)(e + 127) : 255;
    const float scale = scale_of((u32)(e + 127));
    u32 codes = H::template to_fp4<0>(0, w[0], scale);
    codes = H::template to_fp4<1>(codes, w[1], scale);
    codes = H::template to_fp4<2>(codes, w[2], scale);
    codes = H::template to_fp4<3>(codes, w[3], scale);
    uint8_t *base = P.cache + cache_page_at(P.c, page, head, D);
    *(u32 *)(base + cache_codes(P.c.page_size, D, kind) + at * (D / 2) + lane * 4) = fine ? codes : 0;
    if (lane % 4 == 0)
        base[cache_scales(P.c.page_size, D, kind) + (lane / 4) * P.c.page_size + at] = (uint8_t)byte;
}

// Lanes as above; a workgroup takes 2048 / D * UNROLL tokens of one head, keys
// and values.
template <int DT, int D>
__global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(const CacheParams P)
{
    typedef Half<DT> H;
    constexpr int LANES = D / 8, ROWS = kCacheThreads / LANES, UNROLL = 4;
    const int row = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int64_t id = block_id(), block = id / P.c.heads;
    const int head = (int)(id - block * P.c.heads);
    const int64_t t0 = block * (ROWS * UNROLL) + row;
    if (t0 >= P.T)
        return;
    u32 w[UNROLL][2], byte[UNROLL][2];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int64_t t = t0 + i * ROWS;
        int64_t page;
        int32_t at;
        const bool there = t < P.T && cache_slot(P.c, slot_of(P, t), &page, &at);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            w[i][kind] = byte[i][kind] = 0;
            if (there && (kind ? P.v : P.k)) {
                const uint8_t *base = P.cache + cache_page_at(P.c, page, head, D);
                w[i][kind] = *(const u32 *)(base + cache_codes(P.c.page_size, D, kind) + at * (D / 2) + lane * 4);
                byte[i][kind] = base[cache_scales(P.c.page_size, D, kind) + (lane / 4) * P.c.page_size + at];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        const int64_t t = t0 + i * ROWS;
        if (t >= P.T)
            break;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const float s = scale_of(byte[i][kind]);
            const u32x4 v = {H::template from_fp4<0>(w[i][kind], s), H::template from_fp4<1>(w[i][kind], s),
                             H::template from_fp4<2>(w[i][kind], s), H::template from_fp4<3>(w[i][kind], s)};
            uint16_t *to = kind ? (uint16_t *)P.v : (uint16_t *)P.k;
            if (to)
                *(u32x4 *)(to + t * (kind ? P.v_token : P.k_token) + head * (kind ? P.v_head : P.k_head) +
                           lane * 8) = v;
        }
    }
}

template <int DT, int D> hipError_t launch(const CacheParams &p, bool write, hipStream_t s)
{
    constexpr int rows = kCacheThreads / (D / 8);
    if (write)
        cache_write_kernel<DT, D><<<grid_of((p.T + rows - 1) / rows * p.c.heads * 2), kCacheThreads, 0, s>>>(p);
    else
        cache_read_kernel<DT, D><<<grid_of((p.T + 4 * rows - 1) / (4 * rows) * p.c.heads), kCacheThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT> hipError_t launch_width(const CacheParams &p, int D, bool write, hipStream_t s)
{
    return D == 64 ? launch<DT, 64>(p, write, s) : D == 128 ? launch<DT, 128>(p, write, s) : launch<DT, 256>(p, write, s);
}

}  // namespace

hipError_t launch_cache(const CacheParams &p, int D, int dtype, bool write, hipStream_t s)
{
    return dtype == MHC_BF16 ? launch_width<MHC_BF16>(p, D, write, s) : launch_width<MHC_F16>(p, D, write, s);
}

}  // namespace mhc
