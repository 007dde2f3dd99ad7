// Walks the 4-bit cache's addresses on the CPU, in memory of exactly the
// cache's and the table's size: every slot, slots outside, tables with bad pages,
// lengths past a table.  Prints "ok" or what is wrong; run under the address
// sanitizer it ends at the first byte outside.
#include <stdint.h>
#include <stdio.h>
#include <vector>

#include "../layer_mhc_seam_amd/csrc/cache_layout.h"

using namespace mhc;

static int bad(const char *what, long long a, long long b)
{
    printf("%s %lld %lld\n", what, a, b);
    return 1;
}

int main()
{
    // the quotient, against a division, at the ends of every page of large caches
    for (int ps = 16; ps <= kCacheMaxPage; ps += 16) {
        const CacheLayout c = cache_layout((int64_t(1) << 40) / ps - 1, 1, ps);
        for (int64_t p : {int64_t(0), int64_t(1), int64_t(12345), (int64_t(1) << 31) / ps, (int64_t(1) << 33) + 7,
                          c.pages - 1}) {
            if (p >= c.pages)
                continue;
            for (int32_t at : {0, 1, 15, 16, ps - 1}) {
                int64_t page;
                int32_t place;
                if (at < ps && (!cache_slot(c, p * ps + at, &page, &place) || page != p || place != at))
                    return bad("place", ps, p);
            }
        }
    }
    // and of a sequence's tokens, up to the last that there can be
    for (int ps = 16; ps <= kCacheMaxPage; ps += 16) {
        const CacheLayout c = cache_layout(1, 1, ps);
        for (int64_t t0 : {int64_t(0), int64_t(1) << 20, int64_t(1234567) * 16, INT32_MAX - int64_t(5) * ps})
            for (int64_t t = t0 / 16 * 16; t < t0 + 4 * ps; t += 16) {
                int32_t index, at;
                cache_tile(c, (int32_t)t, &index, &at);
                if (index != t / ps || at != t % ps)
                    return bad("index", ps, t);
            }
    }
    for (int D : {64, 128, 256})
        for (int ps : {16, 48, 512})
            for (int heads : {1, 3}) {
                const CacheLayout c = cache_layout(3, heads, ps);
                std::vector<uint8_t> cache((size_t)3 * heads * cache_page_bytes(ps, D));
                // each slot's parts: every byte of the cache belongs to one of them, once
                for (int64_t slot = -2; slot < 3 * ps + 2; ++slot) {
                    int64_t page;
                    int32_t at;
                    const bool there = cache_slot(c, slot, &page, &at);
                    if (there != (slot >= 0 && slot < 3 * ps))
                        return bad("slot", slot, ps);
                    for (int h = 0; there && h < heads; ++h)
                        for (int kind = 0; kind < 2; ++kind) {
                            uint8_t *base = cache.data() + cache_page_at(c, page, h, D);
                            for (int j = 0; j < D / 2; ++j)
                                ++base[cache_codes(ps, D, kind) + at * (D / 2) + j];
                            for (int j = 0; j < D / 32; ++j)
                                ++base[cache_scales(ps, D, kind) + j * ps + at];
                        }
                }
                for (uint8_t v : cache)
                    if (v != 1)
                        return bad("bytes", D, ps);
                // tiles of a sequence: tables of exactly their width, with bad pages
                const std::vector<int32_t> table{2, -1, 0, 3, INT32_MAX, INT32_MIN, 1};
                const int capacity = (int)table.size() * ps;
                for (int len : {1, 15, 16, 17, ps, 2 * ps + 1, capacity})
                    for (int t = 0; t < capacity + 64; t += kCacheTile) {
                        int32_t page, at;
                        const bool there = cache_page(c, table.data(), len, t, &page, &at);
                        const bool want = t < len && table[t / ps] >= 0 && table[t / ps] < 3;
                        if (there != want || (there ? page != table[t / ps] || at != t % ps : page || at))
                            return bad("tile", len, t);
                        // its last token's last bytes, also where it is not there
                        for (int kind = 0; kind < 2; ++kind) {
                            uint8_t *base = cache.data() + cache_page_at(c, page, heads - 1, D);
                            ++base[cache_codes(ps, D, kind) + (at + 15) * (D / 2) + D / 2 - 1];
                            ++base[cache_scales(ps, D, kind) + (D / 32 - 1) * ps + at + 15];
                        }
                    }
                // a table that holds no more than the sequence's pages
                for (int len = 1; len < 3 * ps; ++len) {
                    const std::vector<int32_t> own((len + ps - 1) / ps, 1);
                    for (int t = 0; t < len + 4 * ps; t += kCacheTile) {
                        int32_t page, at;
                        if (cache_page(c, own.data(), len, t, &page, &at) != (t < len))
                            return bad("own", len, t);
                    }
                }
            }
    printf("ok\n");
    return 0;
}
