// cache_runtime.cpp -- C ABI of the rotary positions, the 4-bit cache and the
// attention over it.  Argument rules only; each call is checked in full before
// any device call is made, but for the attention's workspace, whose size goes by
// the device's compute units and which is checked before the launch.

#include <cmath>
#include <cstdint>

#include "arg_checks.h"

using namespace mhc;

namespace {

constexpr int kMaxHeads = 4096, kMaxRopeDim = 512;

bool width_known(int D) { return D == 64 || D == 128 || D == 256; }

bool page_known(int ps) { return ps >= 16 && ps <= kCacheMaxPage && ps % 16 == 0; }

bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

// A tensor [T][heads][D] of 2-byte elements, token and head strides in elements
struct Rows {
    const void *p;
    int64_t T, heads, D, token, head;
    int64_t row() const { return (heads - 1) * head + D; }                 // of one token, end to end
    int64_t extent() const { return T > 0 ? (T - 1) * token + row() : 0; }
    Range range() const { return {p, 2 * extent()}; }
    // Strides above 0 and sizes whose products stay in 64 bits
    bool small() const
    {
        return token > 0 && head > 0 && token < kMaxElements && head < kMaxElements && T <= INT32_MAX &&
               (T <= 1 || token <= (kMaxElements - 1) / T) && head <= (kMaxElements - 1) / heads &&
               extent() < kMaxElements;
    }
    // And heads apart from each other inside a token, or tokens apart inside a head
    bool apart() const
    {
        if (!small())
            return false;
        const bool tokens_outside = (heads == 1 || head >= D) && (T == 1 || token >= row());
        const bool heads_outside = (T == 1 || token >= D) && (heads == 1 || head >= (T - 1) * token + D);
        return tokens_outside || heads_outside;
    }
    bool same(const Rows &o) const { return p == o.p && token == o.token && head == o.head; }
};

// Whether two such tensors share an element, as far as their rows tell: rows
// side by side in one wider row do not
bool overlap(const Rows &a, const Rows &b)
{
    if (!overlap(a.range(), b.range()))
        return false;
    if (a.token == b.token && a.row() <= a.token && b.row() <= b.token) {
        const int64_t step = 2 * a.token;
        const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
        const int64_t r = ((d % step) + step) % step;      // b's row behind a's, in the wider row
        if (r >= 2 * a.row() && r + 2 * b.row() <= step)
            return false;
    }
    return true;
}

int check_cache(const mhc_cache_args *a, bool write)
{
    const char *what = write ? "cache write" : "cache read";
    if (!a)
        return fail(MHC_SEAM_INVALID_ARG, "args is NULL");
    if (a->T < 0 || a->T > INT32_MAX)
        return fail(MHC_SEAM_INVALID_ARG, "%s needs 0 <= T < 2^31", what);
    if (!width_known(a->head_dim) || !page_known(a->page_size))
        return fail(MHC_SEAM_INVALID_ARG,
                    "%s: head_dim is 64, 128 or 256, page_size a multiple of 16 up to %d", what, kCacheMaxPage);
    if (!half_type(a->dtype))
        return fail(MHC_SEAM_INVALID_ARG, "%s takes bf16 or f16", what);
    if (a->heads < 1 || a->heads > kMaxHeads || a->pages < 1 ||
        a->pages >= kMaxElements / ((int64_t)a->heads * a->page_size) || a->T * a->heads >= (int64_t(1) << 34))
        return fail(MHC_SEAM_INVALID_ARG, "%s needs 1 .. %d heads, pages > 0, pages*heads*page_size < 2^40 and "
                    "T*heads < 2^34", what, kMaxHeads);
    if (a->slot_bytes != 4 && a->slot_bytes != 8)
        return fail(MHC_SEAM_INVALID_ARG, "slot_bytes must be 4 or 8");
    if (a->reserved)
        return fail(MHC_SEAM_INVALID_ARG, "reserved fields must be zero");
    if (a->T == 0)
        return MHC_SEAM_OK;
    if (!a->cache || !a->slots || (write ? !a->k || !a->v : !a->k && !a->v))
        return fail(MHC_SEAM_INVALID_ARG, "%s needs cache, slots, k and v", what);
    if (!aligned16(a->cache) || !aligned16(a->k) || !aligned16(a->v) || !aligned_to(a->slots, a->slot_bytes))
        return fail(MHC_SEAM_INVALID_ARG, "cache, k and v must be 16-byte aligned, slots to their elements");
    const Rows k{a->k, a->T, a->heads, a->head_dim, a->k_token, a->k_head};
    const Rows v{a->v, a->T, a->heads, a->head_dim, a->v_token, a->v_head};
    for (const Rows &x : {k, v})
        if (x.p && (!x.apart() || x.token % 8 || x.head % 8))
            return fail(MHC_SEAM_INVALID_ARG,
                        "strides of k and v are positive multiples of 8 that keep heads and tokens apart");
    const Range cache{a->cache, a->pages * a->heads * (int64_t)cache_page_bytes(a->page_size, a->head_dim)};
    const Range slots{a->slots, a->T * a->slot_bytes};
    const Range kr = k.p ? k.range() : Range{nullptr, 0}, vr = v.p ? v.range() : Range{nullptr, 0};
    if (write ? clash({cache}, {kr, vr, slots})
              : clash({kr}, {cache, slots}) || clash({vr}, {cache, slots}) || (k.p && v.p && overlap(k, v)))
        return fail(MHC_SEAM_INVALID_ARG, "an output overlaps an input or the other output");
    return MHC_SEAM_OK;
}

int run_cache(const mhc_cache_args *a, bool write, void *stream)
{
    const int status = check_cache(a, write);
    if (status != MHC_SEAM_OK || a->T == 0)
        return status;
    CacheParams p;
    p.c = cache_layout(a->pages, a->heads, a->page_size);
    p.T = a->T;
    p.slot_bytes = a->slot_bytes;
    p.k_token = a->k_token;
    p.k_head = a->k_head;
    p.v_token = a->v_token;
    p.v_head = a->v_head;
    p.cache = (uint8_t *)a->cache;
    p.slots = a->slots;
    p.k = a->k;
    p.v = a->v;
    int cus = 0;
    hipError_t e = compute_units(&cus);
    if (e != hipSuccess)
        return hip_fail(e, "device attributes");
    e = launch_cache(p, a->head_dim, a->dtype, write, cus, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return hip_fail(e, write ? "cache write launch" : "cache read launch");
    return MHC_SEAM_OK;
}

bool attention_sizes(int64_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t D)
{
    return T >= 0 && T <= INT32_MAX && B >= 0 && B <= 65535 && kv_heads >= 1 && q_heads >= kv_heads &&
           q_heads <= kMaxHeads && q_heads % kv_heads == 0 && width_known(D) &&
           T * (q_heads / kv_heads) + 128 * (int64_t)B < INT32_MAX && T * q_heads < (int64_t(1) << 34);
}

}  // namespace

extern "C" {

int mhc_rope(const mhc_rope_args *a, void *stream)
{
    if (!a)
        return fail(MHC_SEAM_INVALID_ARG, "args is NULL");
    const int64_t T = a->T, D = a->head_dim;
    if (T < 0 || T > INT32_MAX || D < 2 || D > kMaxRopeDim || a->rotary < 2 || a->rotary > D || a->rotary % 2)
        return fail(MHC_SEAM_INVALID_ARG,
                    "rope needs 0 <= T < 2^31, head_dim up to %d and an even rotary in 2 .. head_dim", kMaxRopeDim);
    if (a->q_heads < 1 || a->q_heads > kMaxHeads || a->k_heads < 0 || a->k_heads > kMaxHeads)
        return fail(MHC_SEAM_INVALID_ARG, "rope needs 1 .. %d q_heads and 0 .. %d k_heads", kMaxHeads, kMaxHeads);
    if (!half_type(a->dtype))
        return fail(MHC_SEAM_INVALID_ARG, "rope takes bf16 or f16");
    if (a->position_bytes != 4 && a->position_bytes != 8)
        return fail(MHC_SEAM_INVALID_ARG, "position_bytes must be 4 or 8");
    if (a->axes < 1 || a->axes > 4)
        return fail(MHC_SEAM_INVALID_ARG, "rope takes 1 to 4 axes");
    if ((a->interleaved != 0 && a->interleaved != 1) || (a->inverse != 0 && a->inverse != 1))
        return fail(MHC_SEAM_INVALID_ARG, "interleaved and inverse must be 0 or 1");
    if (!std::isfinite(a->scale))
        return fail(MHC_SEAM_INVALID_ARG, "scale must be finite");
    if (a->pair_axis)
        for (int i = 0; i < a->rotary / 2; ++i)
            if (a->pair_axis[i] >= a->axes)
                return fail(MHC_SEAM_INVALID_ARG, "pair_axis[%d] is no axis", i);
    if (T == 0)
        return MHC_SEAM_OK;
    const bool has_k = a->k_heads > 0;
    if (!a->q || !a->q_out || !a->positions || !a->inv_freq || has_k != !!a->k || has_k != !!a->k_out)
        return fail(MHC_SEAM_INVALID_ARG,
                    "rope needs q, q_out, positions and inv_freq, k and k_out exactly with k_heads");
    if (a->axes > 1 && (a->position_axis < T || a->position_axis >= kMaxElements))
        return fail(MHC_SEAM_INVALID_ARG, "position_axis must be T at least");
    if (!aligned_to(a->positions, a->position_bytes) || !aligned4(a->inv_freq) || !aligned_to(a->q, 2) ||
        !aligned_to(a->k, 2) || !aligned_to(a->q_out, 2) || !aligned_to(a->k_out, 2))
        return fail(MHC_SEAM_INVALID_ARG, "rope's tensors must be aligned to their elements");
    const Rows in[2] = {{a->q, T, a->q_heads, D, a->q_token, a->q_head}, {a->k, T, a->k_heads, D, a->k_token, a->k_head}};
    const Rows out[2] = {{a->q_out, T, a->q_heads, D, a->q_out_token, a->q_out_head},
                         {a->k_out, T, a->k_heads, D, a->k_out_token, a->k_out_head}};
    const int tensors = has_k ? 2 : 1;
    bool in_place = true;
    const Range others[2] = {{a->positions, (int64_t)a->position_bytes * ((a->axes - 1) * a->position_axis + T)},
                             {a->inv_freq, 2 * (int64_t)a->rotary}};
    for (int i = 0; i < tensors; ++i) {
        if (!in[i].apart() || !out[i].apart())
            return fail(MHC_SEAM_INVALID_ARG, "rope's strides are positive and keep heads and tokens apart");
        in_place = in_place && in[i].same(out[i]);
    }
    for (int i = 0; i < tensors; ++i)
        if (clash({out[i].range()}, {others[0], others[1]}) || (!in[i].same(out[i]) && overlap(in[i], out[i])) ||
            (has_k && overlap(out[i], in[1 - i])))
            return fail(MHC_SEAM_INVALID_ARG, "an output overlaps an input");
    if (has_k && overlap(out[0], out[1]))
        return fail(MHC_SEAM_INVALID_ARG, "the outputs overlap");
    // the longest vector that every chunk starts on
    int vector = 8;
    auto divides = [&](int n) {
        if (a->rotary / 2 % n || (D - a->rotary) % n)
            return false;
        for (int i = 0; i < tensors; ++i)
            for (const Rows &x : {in[i], out[i]})
                if (x.token % n || x.head % n || !aligned_to(x.p, 2 * n))
                    return false;
        return true;
    };
    while (vector > 1 && !divides(vector))
        vector /= 2;
    int cus = 0;
    hipError_t e = compute_units(&cus);
    if (e != hipSuccess)
        return hip_fail(e, "device attributes");
    RopeParams p{};
    p.T = T;
    p.q_heads = a->q_heads;
    p.k_heads = a->k_heads;
    p.head_dim = a->head_dim;
    p.rotary = a->rotary;
    p.inverse = a->inverse;
    p.position_bytes = a->position_bytes;
    p.scale = a->scale;
    p.position_axis = a->position_axis;
    p.q_token = a->q_token;
    p.q_head = a->q_head;
    p.k_token = a->k_token;
    p.k_head = a->k_head;
    p.q_out_token = a->q_out_token;
    p.q_out_head = a->q_out_head;
    p.k_out_token = a->k_out_token;
    p.k_out_head = a->k_out_head;
    p.q = (const uint16_t *)a->q;
    p.k = (const uint16_t *)a->k;
    p.positions = a->positions;
    p.inv_freq = a->inv_freq;
    p.q_out = (uint16_t *)a->q_out;
    p.k_out = (uint16_t *)a->k_out;
    if (a->pair_axis)
        for (int i = 0; i < a->rotary / 2; ++i)
            p.axis[i / 16] |= (uint32_t)a->pair_axis[i] << (i % 16 * 2);
    e = launch_rope(p, a->dtype, vector, a->interleaved, in_place, cus, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return hip_fail(e, "rope launch");
    return MHC_SEAM_OK;
}

int mhc_cache_write(const mhc_cache_args *a, void *stream) { return run_cache(a, true, stream); }

int mhc_cache_read(const mhc_cache_args *a, void *stream) { return run_cache(a, false, stream); }

int mhc_cache_attention_workspace(int64_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                  int32_t cu_count, int64_t max_len, uint64_t *bytes)
{
    if (!attention_sizes(T, B, q_heads, kv_heads, head_dim) || cu_count < 1 || cu_count > 4096 || max_len < 0 ||
        max_len > (1 << 30) || !bytes)
        return fail(MHC_SEAM_INVALID_ARG, "workspace of cache attention: sizes out of range");
    *bytes = T && B ? 4 * attention_workspace_floats(T, B, q_heads, kv_heads, head_dim, cu_count, max_len) : 0;
    return MHC_SEAM_OK;
}

int mhc_cache_attention(const mhc_cache_attention_args *a, void *stream)
{
    if (!a)
        return fail(MHC_SEAM_INVALID_ARG, "args is NULL");
    const int64_t T = a->T, D = a->head_dim;
    if (!attention_sizes(T, a->B, a->q_heads, a->kv_heads, a->head_dim))
        return fail(MHC_SEAM_INVALID_ARG,
                    "cache attention needs 0 <= T < 2^31, 0 <= B < 2^16, kv_heads that divide q_heads (up to %d), "
                    "head_dim 64, 128 or 256, T*q_heads/kv_heads + 128*B < 2^31, T*q_heads < 2^34", kMaxHeads);
    if (!half_type(a->dtype))
        return fail(MHC_SEAM_INVALID_ARG, "cache attention takes bf16 or f16");
    if (!page_known(a->page_size) || a->pages < 1 || a->pages > INT32_MAX / a->kv_heads || a->table_width < 1 ||
        (int64_t)a->table_width * a->page_size > (1 << 30))
        return fail(MHC_SEAM_INVALID_ARG,
                    "cache attention: page_size is a multiple of 16 up to %d, pages > 0, pages*kv_heads < 2^31, "
                    "0 < table_width*page_size <= 2^30", kCacheMaxPage);
    if (a->max_len < 0 || a->window < 0 || (a->causal != 0 && a->causal != 1))
        return fail(MHC_SEAM_INVALID_ARG, "max_len and window must not be negative, causal 0 or 1");
    if (!std::isfinite(a->scale) || !std::isfinite(a->softcap) || a->softcap < 0 ||
        (a->softcap > 0 && !std::isfinite(a->scale / a->softcap)))
        return fail(MHC_SEAM_INVALID_ARG, "scale, softcap and their quotient must be finite, softcap not negative");
    if (a->reserved)
        return fail(MHC_SEAM_INVALID_ARG, "reserved fields must be zero");
    if (!a->q_starts && T != a->B)
        return fail(MHC_SEAM_INVALID_ARG, "without q_starts there is one query row a sequence: T == B");
    if (T == 0 || a->B == 0)
        return MHC_SEAM_OK;
    if (!a->q || !a->cache || !a->tables || !a->lens || !a->out)
        return fail(MHC_SEAM_INVALID_ARG, "cache attention needs q, cache, tables, lens and out");
    if (!aligned16(a->q) || !aligned16(a->cache) || !aligned16(a->out) || !aligned4(a->tables) ||
        !aligned4(a->lens) || !aligned4(a->q_starts) || !aligned4(a->lse) || !aligned16(a->workspace))
        return fail(MHC_SEAM_INVALID_ARG,
                    "q, cache, out and workspace must be 16-byte aligned, the others to their elements");
    const Rows q{a->q, T, a->q_heads, D, a->q_token, a->q_head};
    if (!q.apart() || q.token % 8 || q.head % 8)
        return fail(MHC_SEAM_INVALID_ARG, "q's strides are positive multiples of 8 that keep heads and tokens apart");
    if (a->B > 1 && (a->table_stride < a->table_width || a->table_stride >= kMaxElements))
        return fail(MHC_SEAM_INVALID_ARG, "table_stride must be table_width at least");
    const Range ins[5] = {q.range(),
                          {a->cache, a->pages * a->kv_heads * (int64_t)cache_page_bytes(a->page_size, a->head_dim)},
                          {a->tables, 4 * ((a->B - 1) * a->table_stride + a->table_width)},
                          {a->lens, 4 * (int64_t)a->B},
                          {a->q_starts, 4 * (int64_t)(a->B + 1)}};
    const Range out{a->out, 2 * T * a->q_heads * D}, lse{a->lse, 4 * T * a->q_heads};
    if (clash({out, lse}, {ins[0], ins[1], ins[2], ins[3], ins[4]}))
        return fail(MHC_SEAM_INVALID_ARG, "an output overlaps an input or the other output");
    int cus = 0;
    hipError_t e = compute_units(&cus);
    if (e != hipSuccess)
        return hip_fail(e, "device attributes");
    int64_t max_len = (int64_t)a->table_width * a->page_size;
    if (a->max_len > 0 && a->max_len < max_len)
        max_len = a->max_len;
    const uint64_t floats = attention_workspace_floats(T, a->B, a->q_heads, a->kv_heads, a->head_dim, cus, max_len);
    // A window leaves a sequence's rows window + n - 1 tokens, which choose the
    // kernel as sequences of that length would (16 sequences' 5 rows over 4099 tokens,
    // a window of 1024, 4 kv heads of 256 channels: 18.5 us, shared out 23.1).
    int64_t seen = max_len;
    if (a->window > 0 && a->window + T < seen)
        seen = a->window + T;
    uint64_t used = attention_workspace_floats(T, a->B, a->q_heads, a->kv_heads, a->head_dim, cus, seen);
    if (used > floats) {
        seen = max_len;
        used = floats;
    }
    if (floats && (!a->workspace || a->workspace_bytes < 4 * floats))
        return fail(MHC_SEAM_INVALID_ARG, "cache attention needs a workspace of %llu bytes",
                    (unsigned long long)(4 * floats));
    const Range space{floats ? a->workspace : nullptr, 4 * (int64_t)floats};
    if (clash({space}, {ins[0], ins[1], ins[2], ins[3], ins[4], out, lse}))
        return fail(MHC_SEAM_INVALID_ARG, "the workspace overlaps an input or an output");
    AttentionParams p{};
    p.c = cache_layout(a->pages, a->kv_heads, a->page_size);
    p.T = T;
    p.max_len = max_len;
    p.q_token = a->q_token;
    p.q_head = a->q_head;
    p.table_stride = a->table_stride;
    p.B = a->B;
    p.q_heads = a->q_heads;
    p.group = a->q_heads / a->kv_heads;
    p.causal = a->causal;
    p.window = a->window;
    p.scale = a->scale;
    p.softcap = a->softcap;
    p.q = (const uint16_t *)a->q;
    p.cache = a->cache;
    p.tables = a->tables;
    p.lens = a->lens;
    p.q_starts = a->q_starts;
    p.out = (uint16_t *)a->out;
    p.lse = a->lse;
    p.workspace = used ? (float *)a->workspace : nullptr;
    p.seen = seen;
    e = launch_attention(p, a->head_dim, a->dtype, cus, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return hip_fail(e, "cache attention launch");
    return MHC_SEAM_OK;
}

}  // extern "C"
