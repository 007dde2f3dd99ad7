// cache_layout.h -- where a token's codes and scales lie in the 4-bit cache
// u8 [pages][heads][page_size * (D + D/16)]: of each page and head the keys'
// codes [page_size][D/2], the values' codes, the keys' scales
// [D/32][page_size], the values' scales.  Plain C++, for the kernels and for
// host code alike.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define MHC_BOTH __host__ __device__ __forceinline__
#else
#define MHC_BOTH inline
#endif

namespace mhc {

constexpr int kCacheTile = 16;       // tokens that never straddle two pages
constexpr int kCacheMaxPage = 512;   // tokens a page

struct CacheLayout {
    int64_t pages;
    int32_t heads;
    int32_t page_size;
    uint64_t magic;                  // ceil(2^63 / (page_size / 16))
    uint32_t magic32, whole;         // ceil(2^32 / (page_size / 16)), or 0 and 1
};

MHC_BOTH CacheLayout cache_layout(int64_t pages, int32_t heads, int32_t page_size)
{
    const uint64_t tiles = (uint64_t)page_size / kCacheTile;
    return {pages, heads, page_size, ((uint64_t(1) << 63) + tiles - 1) / tiles,
            (uint32_t)(((uint64_t(1) << 32) + tiles - 1) / tiles), tiles == 1};
}

MHC_BOTH uint64_t high_product(uint64_t a, uint64_t b)
{
#if defined(__HIP_DEVICE_COMPILE__)
    return __umul64hi(a, b);
#else
    return (uint64_t)((unsigned __int128)a * b >> 64);
#endif
}

// Bytes of one head's page, and where its four parts begin
MHC_BOTH constexpr uint32_t cache_page_bytes(int ps, int D) { return (uint32_t)(ps * (D + D / 16)); }
MHC_BOTH constexpr uint32_t cache_codes(int ps, int D, int kind) { return (uint32_t)(kind * ps * (D / 2)); }
MHC_BOTH constexpr uint32_t cache_scales(int ps, int D, int kind)
{
    return (uint32_t)(ps * D + kind * ps * (D / 32));
}

// Page of token (or slot) t and its place there.  The quotient is exact: with
// d = page_size / 16 <= 32 and u = t / 16 < 2^36, magic exceeds 2^63 / d by
// less than 1, so 2u magic / 2^64 exceeds u / d by less than 2^-26 < 1 / d.
MHC_BOTH void cache_place(const CacheLayout &c, uint64_t t, int64_t *page, int32_t *at)
{
    const uint64_t p = high_product((t / kCacheTile) * 2, c.magic);
    *page = (int64_t)p;
    *at = (int32_t)(t - p * (uint64_t)c.page_size);
}

// Place of a slot; false for one that is not in the cache
MHC_BOTH bool cache_slot(const CacheLayout &c, int64_t slot, int64_t *page, int32_t *at)
{
    if (slot < 0 || slot >= c.pages * c.page_size)
        return false;
    cache_place(c, (uint64_t)slot, page, at);
    return true;
}

// First byte of a head's page
MHC_BOTH int64_t cache_page_at(const CacheLayout &c, int64_t page, int head, int D)
{
    return (page * c.heads + head) * (int64_t)cache_page_bytes(c.page_size, D);
}

// The same where pages * heads < 2^31
MHC_BOTH uint64_t cache_page_near(const CacheLayout &c, int32_t page, int head, int D)
{
    return (uint64_t)(uint32_t)(page * c.heads + head) * cache_page_bytes(c.page_size, D);
}

// The page of a sequence, and the place there, that its tokens [t, t + 16), t a
// multiple of 16 below 2^31, lie on.  Exact: u = t / 16 < 2^27 times magic32's
// excess, below page_size / 16 <= 32, is below 2^32.
MHC_BOTH void cache_tile(const CacheLayout &c, int32_t t, int32_t *index, int32_t *at)
{
    const uint32_t u = (uint32_t)t / kCacheTile;
    const uint32_t i = (uint32_t)((uint64_t)u * c.magic32 >> 32) + u * c.whole;
    *index = (int32_t)i;
    *at = (int32_t)((uint32_t)t - i * (uint32_t)c.page_size);
}

// That tile's page and place there.  Where the sequence of `len` tokens has none
// at t, or the table names a page that there is not: false, and page 0.  The
// table is read at no place but those of the sequence's own tokens; len > 0.
template <typename Table>
MHC_BOTH bool cache_page(const CacheLayout &c, Table table, int32_t len, int32_t t, int32_t *page, int32_t *at)
{
    int32_t index, last, skip;
    cache_tile(c, t, &index, at);
    cache_tile(c, (len - 1) / kCacheTile * kCacheTile, &last, &skip);
    *page = table[index < last ? index : last];
    const bool there = t < len && *page >= 0 && *page < c.pages;
    if (!there)
        *page = *at = 0;
    return there;
}

}  // namespace mhc
