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
constexpr int kCacheBlocks = 2;           // workgroups a CU, at most

__device__ __forceinline__ int64_t slot_of(const CacheParams &P, int64_t t)
{
    return P.slot_bytes == 8 ? ((const int64_t *)P.slots)[t] : ((const int32_t *)P.slots)[t];
}

// Bytes bound both directions.  D/8 lanes hold a row, 8 channels each, four lanes
// a group of 32.  A wave takes all heads of a token, ROWS * UNROLL of them a step,
// then the token that lies the number of waves behind it: so the waves together
// go through k and v in one narrow band, 131072 tokens of 8 heads of 128
// channels read in 132 us at two workgroups a CU (5.2 TB/s; 180 us at four or more;
// tokens or heads dealt out in blocks 170 us).  A step's loads are issued before the
// last step's stores: loads and stores come back in one order, and behind the
// stores they would wait for them (206 us).  A token's place costs ten products of 32
// bits; lane l finds that of the wave's l-th token.
struct Place {
    int64_t page_at;         // first byte of the page's first head; below 0: no place
    int32_t at;
};

__device__ __forceinline__ Place place_of(const CacheParams &P, int64_t t, int D)
{
    int64_t page = 0;
    Place p{-1, 0};
    if (t < P.T && cache_slot(P.c, slot_of(P, t), &page, &p.at))
        p.page_at = cache_page_at(P.c, page, 0, D);
    return p;
}

__device__ __forceinline__ Place of_lane(const Place &p, int l)
{
    return {(int64_t)((u64)read_lane((u32)((u64)p.page_at >> 32), l) << 32 | read_lane((u32)(u64)p.page_at, l)),
            (int32_t)read_lane((u32)p.at, l)};
}

// The wave's steps: heads from h on of token t, which lies at place
template <int D> struct Walk {
    const CacheParams &P;
    int64_t waves, t;
    int h, step, l;
    Place mine, place;
    __device__ __forceinline__ Walk(const CacheParams &P, int step) : P(P), h(0), step(step), l(0)
    {
        waves = (int64_t)gridDim.x * (kCacheThreads / 64);
        // workgroups go to the 8 dies in turn: neighbouring tokens, which share
        // cache lines of codes and scales, to one die (write, 16384 tokens: 3% faster)
        const u32 b = gridDim.x % 8 == 0 ? blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
        t = (int64_t)b * (kCacheThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        mine = place_of(P, t + (threadIdx.x & 63) * waves, D);
        place = of_lane(mine, 0);
    }
    __device__ __forceinline__ bool more() const { return t < P.T; }
    __device__ __forceinline__ void next()
    {
        if ((h += step) < P.c.heads)
            return;
        h = 0;
        t += waves;
        if (++l == 64) {
            l = 0;
            mine = place_of(P, t + (threadIdx.x & 63) * waves, D);
        }
        place = of_lane(mine, l);
    }
};

template <int DT, int D> __global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(const CacheParams P)
{
    typedef Half<DT> H;
    constexpr int LANES = D / 8, ROWS = 64 / LANES, UNROLL = 2;
    const int lane = threadIdx.x & 63, row = lane / LANES, part = lane % LANES, ps = P.c.page_size;
    const u32 each = cache_page_bytes(ps, D);
    Walk<D> walk(P, ROWS * UNROLL);
    u32x4 w[UNROLL][2];
    auto load = [&]() {
        // behind the last token and where it has no place: the last token's, not stored
        const int64_t t = min(walk.t, P.T - 1);
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int head = min(walk.h + row + i * ROWS, P.c.heads - 1);
            w[i][0] = *(const u32x4 *)((const uint16_t *)P.k + t * P.k_token + head * P.k_head + part * 8);
            w[i][1] = *(const u32x4 *)((const uint16_t *)P.v + t * P.v_token + head * P.v_head + part * 8);
        }
    };
    if (!walk.more())
        return;
    load();
    while (walk.more()) {
        u32 codes[UNROLL][2], byte[UNROLL][2];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                u32 most = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    most = max(most, max(w[i][kind][j] & 0x7fff, (w[i][kind][j] >> 16) & 0x7fff));
                most = max(most, row_swap<kXor1>(most));
                most = max(most, row_swap<kXor2>(most));
                const bool fine = most < H::kInf;
                const u32 bits = __float_as_uint(H::low(most));
                int e = (int)(bits >> 23) - 127 - ((bits & 0x7fffff) <= 0x400000 ? 2 : 1);
                e = min(max(e, H::kLow), H::kHigh);
                byte[i][kind] = fine ? (u32)(e + 127) : 255;
                const float scale = scale_of((u32)(e + 127));
                u32 c = H::template to_fp4<0>(0, w[i][kind][0], scale);
                c = H::template to_fp4<1>(c, w[i][kind][1], scale);
                c = H::template to_fp4<2>(c, w[i][kind][2], scale);
                c = H::template to_fp4<3>(c, w[i][kind][3], scale);
                codes[i][kind] = fine ? c : 0;
            }
        const Place p = walk.place;
        const int h = walk.h + row;
        walk.next();
        load();
        if (p.page_at < 0)
            continue;
        uint8_t *page = P.cache + p.page_at;
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind)
                if (h + i * ROWS < P.c.heads) {
                    const u32 to = (h + i * ROWS) * each;
                    *(u32 *)(page + (to + cache_codes(ps, D, kind) + part * 4 + p.at * (D / 2))) = codes[i][kind];
                    if (part % 4 == 0)
                        page[to + cache_scales(ps, D, kind) + part / 4 * ps + p.at] = (uint8_t)byte[i][kind];
                }
    }
}

template <int DT, int D> __global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(const CacheParams P)
{
    typedef Half<DT> H;
    constexpr int LANES = D / 8, ROWS = 64 / LANES, UNROLL = 2;
    const int lane = threadIdx.x & 63, row = lane / LANES, part = lane % LANES, ps = P.c.page_size;
    const u32 each = cache_page_bytes(ps, D);
    uint16_t *const out[2] = {(uint16_t *)P.k, (uint16_t *)P.v};
    Walk<D> walk(P, ROWS * UNROLL);
    u32 w[UNROLL][2], byte[UNROLL][2];
    auto load = [&]() {
        // a token without a place reads the cache's first row, and is given zeros
        const bool none = walk.place.page_at < 0;
        const uint8_t *page = P.cache + (none ? 0 : walk.place.page_at);
        const int at = none ? 0 : walk.place.at;
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                const u32 from = min(walk.h + row + i * ROWS, P.c.heads - 1) * each;
                w[i][kind] = *(const u32 *)(page + (from + cache_codes(ps, D, kind) + part * 4 + at * (D / 2)));
                byte[i][kind] = page[from + cache_scales(ps, D, kind) + part / 4 * ps + at];
            }
    };
    if (!walk.more())
        return;
    load();
    while (walk.more()) {
        const bool none = walk.place.page_at < 0;
        u32x4 o[UNROLL][2];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {
                const float s = scale_of(none ? 0 : byte[i][kind]);
                const u32 c = none ? 0 : w[i][kind];
                o[i][kind] = {H::template from_fp4<0>(c, s), H::template from_fp4<1>(c, s),
                              H::template from_fp4<2>(c, s), H::template from_fp4<3>(c, s)};
            }
        const int64_t t = walk.t;
        const int h = walk.h + row;
        walk.next();
        load();
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
#pragma unroll
            for (int kind = 0; kind < 2; ++kind)
                // past the caches: 5% faster where they would be full of it
                if (h + i * ROWS < P.c.heads && out[kind])
                    __builtin_nontemporal_store(
                        o[i][kind], (u32x4 *)(out[kind] + t * (kind ? P.v_token : P.k_token) +
                                              (h + i * ROWS) * (kind ? P.v_head : P.k_head) + part * 8));
    }
}

template <int DT, int D> hipError_t launch(const CacheParams &p, bool write, int cus, hipStream_t s)
{
    const int64_t all = (p.T + kCacheThreads / 64 - 1) / (kCacheThreads / 64), most = (int64_t)cus * kCacheBlocks;
    const dim3 grid((unsigned)(all < most ? all : most));
    if (write)
        cache_write_kernel<DT, D><<<grid, kCacheThreads, 0, s>>>(p);
    else
        cache_read_kernel<DT, D><<<grid, kCacheThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT> hipError_t launch_width(const CacheParams &p, int D, bool write, int cus, hipStream_t s)
{
    return D == 64    ? launch<DT, 64>(p, write, cus, s)
           : D == 128 ? launch<DT, 128>(p, write, cus, s)
                      : launch<DT, 256>(p, write, cus, s);
}

}  // namespace

hipError_t launch_cache(const CacheParams &p, int D, int dtype, bool write, int cus, hipStream_t s)
{
    return dtype == MHC_BF16 ? launch_width<MHC_BF16>(p, D, write, cus, s)
                             : launch_width<MHC_F16>(p, D, write, cus, s);
}

}  // namespace mhc
