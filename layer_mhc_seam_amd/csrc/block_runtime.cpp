// block_runtime.cpp -- C ABI of the one-stream block operators: the block
// norm, the int8 quantiser and product, and expert routing.  Argument rules
// only; each call is checked in full before any device call is made.

#include <atomic>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "seam_internal.h"

using mhc::aligned16;
using mhc::fail;
using mhc::hip_fail;

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 40;
// Widths whose rows fit a workgroup's registers: 4096 chunks of 8, of which a
// row that starts and ends inside one spans two more than it fills
bool width_fits(int64_t H) { return H >= 1 && H <= (H % 8 ? 32752 : 32768); }
constexpr int kMaxDepth = 131056;    // 128 * 128 * K < 2^31
constexpr int kMaxRoute = 1024, kMaxGroups = 64, kMaxChosen = 64;

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool half_type(int d) { return d == MHC_BF16 || d == MHC_F16; }

int64_t size_of(int d) { return d == MHC_F32 ? 4 : 2; }

struct Range {
    const void *p;
    int64_t bytes;
};

bool overlap(const Range &a, const Range &b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0)
        return false;
    const uintptr_t al = reinterpret_cast<uintptr_t>(a.p), bl = reinterpret_cast<uintptr_t>(b.p);
    return al < bl + (uintptr_t)b.bytes && bl < al + (uintptr_t)a.bytes;
}

// Whether an output overlaps an input or another output
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins)
{
    for (const Range *o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &i : ins)
            if (overlap(*o, i))
                return true;
        for (const Range *q = outs.begin(); q != o; ++q)
            if (overlap(*o, *q))
                return true;
    }
    return false;
}

// Compute units of the current device, asked for once per device
hipError_t compute_units(int *cus)
{
    static std::atomic<int> known[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    if (dev >= 0 && dev < 64 && (*cus = known[dev].load(std::memory_order_relaxed)) > 0)
        return hipSuccess;
    e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e == hipSuccess && dev >= 0 && dev < 64)
        known[dev].store(*cus, std::memory_order_relaxed);
    return e;
}

}  // namespace

extern "C" {

int mhc_block_norm(const mhc_block_norm_args *a, void *stream)
{
    if (!a)
        return fail(MHC_SEAM_INVALID_ARG, "args is NULL");
    const int64_t T = a->T, H = a->H;
    if (T < 0 || T > INT32_MAX || !width_fits(H) || T * H >= kMaxElements)
        return fail(MHC_SEAM_INVALID_ARG,
                    "block norm needs 0 <= T < 2^31, 1 <= H <= 32768 (32752 if no multiple of 8) "
                    "and T*H < 2^40");
    if (!half_type(a->dtype) || (a->x_dtype != a->dtype && a->x_dtype != MHC_F32))
        return fail(MHC_SEAM_INVALID_ARG,
                    "block norm: dtype is bf16 or f16, x_dtype the same or f32");
    if (a->gate_kind < MHC_GATE_NONE || a->gate_kind > MHC_GATE_ELEMENT)
        return fail(MHC_SEAM_INVALID_ARG, "unknown gate_kind %d", a->gate_kind);
    if (!(a->eps >= 0.0f) || a->eps > 1.0f)
        return fail(MHC_SEAM_INVALID_ARG, "eps must be in [0, 1] (0 selects 1e-6)");
    if (!std::isfinite(a->residual_scale) || !std::isfinite(a->branch_scale))
        return fail(MHC_SEAM_INVALID_ARG, "residual_scale and branch_scale must be finite");
    if (a->reserved)
        return fail(MHC_SEAM_INVALID_ARG, "reserved fields must be zero");
    if (T == 0)
        return MHC_SEAM_OK;
    if (!a->x)
        return fail(MHC_SEAM_INVALID_ARG, "x is required");
    if (!a->y && !a->gamma)
        return fail(MHC_SEAM_INVALID_ARG, "block norm needs y, gamma or both");
    if (!a->y != !a->residual_out)
        return fail(MHC_SEAM_INVALID_ARG, "y and residual_out come together");
    if (!a->y && (a->gamma_post || a->gate_kind != MHC_GATE_NONE || a->residual_scale != 1.0f ||
                  a->branch_scale != 1.0f))
        return fail(MHC_SEAM_INVALID_ARG,
                    "without y there is no gamma_post, no gate and no scale but 1");
    if (!a->gate != (a->gate_kind == MHC_GATE_NONE))
        return fail(MHC_SEAM_INVALID_ARG, "gate is required exactly when gate_kind is set");
    if (!a->codes != !a->scales)
        return fail(MHC_SEAM_INVALID_ARG, "codes and scales come together");
    if (!a->gamma != (!a->norm && !a->codes))
        return fail(MHC_SEAM_INVALID_ARG,
                    "gamma is required exactly when norm or codes are written");
    const int64_t e = size_of(a->dtype), xb = T * H * size_of(a->x_dtype), eb = T * H * e;
    for (const void *p : {a->x, a->y, a->gamma_post, a->gate, a->gamma,
                          (const void *)a->residual_out, (const void *)a->norm,
                          (const void *)a->codes})
        if (!aligned16(p))
            return fail(MHC_SEAM_INVALID_ARG, "block norm's tensors must be 16-byte aligned");
    if (!aligned4(a->scales))
        return fail(MHC_SEAM_INVALID_ARG, "scales must be 4-byte aligned");
    const int64_t gate_bytes = a->gate_kind == MHC_GATE_TOKEN     ? 4 * T
                               : a->gate_kind == MHC_GATE_CHANNEL ? 4 * H
                                                                  : eb;
    const bool in_place = a->residual_out == a->x;
    const Range x{a->x, xb}, y{a->y, eb}, gp{a->gamma_post, H * e}, gate{a->gate, gate_bytes},
        gamma{a->gamma, H * e};
    const Range r{a->residual_out, xb}, norm{a->norm, eb}, codes{a->codes, T * H},
        scales{a->scales, 4 * T};
    if (clash({r, norm, codes, scales}, {y, gp, gate, gamma}) || clash({norm, codes, scales}, {x}) ||
        (!in_place && overlap(r, x)))
        return fail(MHC_SEAM_INVALID_ARG, "an output overlaps an input or another output");
    mhc::BlockNormParams p;
    p.T = T;
    p.H = a->H;
    p.inv_H = 1.0 / (double)a->H;
    p.gate_kind = a->gate_kind;
    p.eps = a->eps > 0.0f ? a->eps : 1e-6f;
    p.residual_scale = a->residual_scale;
    p.branch_scale = a->branch_scale;
    p.x = a->x;
    p.y = a->y;
    p.gamma_post = a->gamma_post;
    p.gate = a->gate;
    p.gamma = a->gamma;
    p.residual_out = a->residual_out;
    p.norm = a->norm;
    p.codes = a->codes;
    p.scales = a->scales;
    hipError_t err = mhc::launch_block_norm(p, a->dtype, a->x_dtype,
                                            reinterpret_cast<hipStream_t>(stream));
    if (err != hipSuccess)
        return hip_fail(err, "block norm launch");
    return MHC_SEAM_OK;
}

int mhc_int8_quantize(const void *src, int32_t dtype, int64_t rows, int32_t H, int8_t *codes,
                      float *scales, void *stream)
{
    if (rows < 0 || rows > INT32_MAX || !width_fits(H) || rows * H >= kMaxElements)
        return fail(MHC_SEAM_INVALID_ARG,
                    "int8 quantize needs 0 <= rows < 2^31, 1 <= H <= 32768 (32752 if no multiple "
                    "of 8) and rows*H < 2^40");
    if (!half_type(dtype))
        return fail(MHC_SEAM_INVALID_ARG, "int8 quantize takes bf16 or f16");
    if (rows == 0)
        return MHC_SEAM_OK;
    if (!src || !codes || !scales)
        return fail(MHC_SEAM_INVALID_ARG, "int8 quantize needs src, codes and scales");
    if (!aligned16(src) || !aligned16(codes) || !aligned4(scales))
        return fail(MHC_SEAM_INVALID_ARG,
                    "src and codes must be 16-byte aligned, scales 4-byte aligned");
    if (clash({{codes, rows * H}, {scales, 4 * rows}}, {{src, rows * H * size_of(dtype)}}))
        return fail(MHC_SEAM_INVALID_ARG, "an output overlaps src or the other output");
    hipError_t e = mhc::launch_int8_quantize(src, dtype, rows, H, codes, scales,
                                             reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return hip_fail(e, "int8 quantize launch");
    return MHC_SEAM_OK;
}

int mhc_int8_gemm(const int8_t *a, const float *a_scales, const int8_t *b, const float *b_scales,
                  const float *bias, int64_t T, int32_t N, int32_t K, int32_t out_dtype, void *out,
                  void *stream)
{
    if (T < 0 || T > INT32_MAX || N <= 0 || K <= 0 || K % 16 || K > kMaxDepth)
        return fail(MHC_SEAM_INVALID_ARG,
                    "int8 gemm needs 0 <= T < 2^31, N > 0 and K a positive multiple of 16, at "
                    "most %d", kMaxDepth);
    if (T * N >= kMaxElements || T * K >= kMaxElements || (int64_t)N * K >= kMaxElements)
        return fail(MHC_SEAM_INVALID_ARG, "int8 gemm sizes too large");
    if (out_dtype != MHC_F32 && !half_type(out_dtype))
        return fail(MHC_SEAM_INVALID_ARG, "int8 gemm writes bf16, f16 or f32");
    if (T == 0)
        return MHC_SEAM_OK;
    if (!a || !a_scales || !b || !b_scales || !out)
        return fail(MHC_SEAM_INVALID_ARG, "int8 gemm needs a, a_scales, b, b_scales and out");
    if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned4(a_scales) ||
        !aligned4(b_scales) || !aligned4(bias))
        return fail(MHC_SEAM_INVALID_ARG,
                    "a, b and out must be 16-byte aligned, scales and bias 4-byte aligned");
    if (clash({{out, T * N * size_of(out_dtype)}},
              {{a, T * K}, {a_scales, 4 * T}, {b, (int64_t)N * K}, {b_scales, 4 * (int64_t)N},
               {bias, 4 * (int64_t)N}}))
        return fail(MHC_SEAM_INVALID_ARG, "out overlaps an input");
    int cus = 0;
    hipError_t e = compute_units(&cus);
    if (e != hipSuccess)
        return hip_fail(e, "device attributes");
    const mhc::Int8GemmParams p{a, a_scales, b, b_scales, bias, out, (int)T, N, K};
    e = mhc::launch_int8_gemm(p, out_dtype, cus, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return hip_fail(e, "int8 gemm launch");
    return MHC_SEAM_OK;
}

int mhc_int8_gemm_blocks(int64_t T, int32_t N, int32_t cu_count, int32_t *tm, int32_t *tn)
{
    if (T <= 0 || T > INT32_MAX || N <= 0 || cu_count <= 0 || !tm || !tn)
        return fail(MHC_SEAM_INVALID_ARG,
                    "gemm blocks need T in 1..2^31-1, N > 0, cu_count > 0 and two outputs");
    const mhc::GemmBlocks g = mhc::int8_gemm_blocks(T, N, cu_count);
    *tm = g.tm;
    *tn = g.tn;
    return MHC_SEAM_OK;
}

int mhc_route(const mhc_route_args *a, void *stream)
{
    if (!a)
        return fail(MHC_SEAM_INVALID_ARG, "args is NULL");
    const int64_t T = a->T, E = a->E;
    if (T < 0 || T > INT32_MAX || E < 1 || E > kMaxRoute || T * E >= kMaxElements)
        return fail(MHC_SEAM_INVALID_ARG, "route needs 0 <= T < 2^31 and 1 <= E <= %d", kMaxRoute);
    if (a->dtype != MHC_F32 && !half_type(a->dtype))
        return fail(MHC_SEAM_INVALID_ARG, "route takes bf16, f16 or f32 logits");
    if (a->scoring != MHC_SOFTMAX && a->scoring != MHC_SIGMOID)
        return fail(MHC_SEAM_INVALID_ARG, "unknown scoring %d", a->scoring);
    if (a->groups < 1 || a->groups > kMaxGroups || E % a->groups)
        return fail(MHC_SEAM_INVALID_ARG, "groups must divide E and be in 1 .. %d", kMaxGroups);
    const int64_t size = E / a->groups;
    if (a->topk_groups < 1 || a->topk_groups > a->groups)
        return fail(MHC_SEAM_INVALID_ARG, "topk_groups must be in 1 .. groups");
    if (a->group_top < 1 || a->group_top > 2 || a->group_top > size ||
        (a->groups == 1 && a->group_top != 1))
        return fail(MHC_SEAM_INVALID_ARG,
                    "group_top must be 1 or 2, at most E / groups, and 1 without groups");
    if (a->k < 1 || a->k > kMaxChosen || a->k > a->topk_groups * size)
        return fail(MHC_SEAM_INVALID_ARG,
                    "k must be in 1 .. %d and at most the experts of topk_groups groups",
                    kMaxChosen);
    if (a->renormalize != 0 && a->renormalize != 1)
        return fail(MHC_SEAM_INVALID_ARG, "renormalize must be 0 or 1");
    if (!std::isfinite(a->scale))
        return fail(MHC_SEAM_INVALID_ARG, "scale must be finite");
    if (a->reserved)
        return fail(MHC_SEAM_INVALID_ARG, "reserved fields must be zero");
    if (T == 0)
        return MHC_SEAM_OK;
    if (!a->logits || !a->weights || !a->ids)
        return fail(MHC_SEAM_INVALID_ARG, "route needs logits, weights and ids");
    const uintptr_t unit = (uintptr_t)size_of(a->dtype) - 1;
    if ((reinterpret_cast<uintptr_t>(a->logits) & unit) || !aligned4(a->bias) ||
        !aligned4(a->weights) || !aligned4(a->ids))
        return fail(MHC_SEAM_INVALID_ARG, "route's tensors must be aligned to their elements");
    const int64_t out = 4 * T * a->k;
    if (clash({{a->weights, out}, {a->ids, out}},
              {{a->logits, T * E * size_of(a->dtype)}, {a->bias, 4 * E}}))
        return fail(MHC_SEAM_INVALID_ARG, "an output overlaps an input or the other output");
    mhc::RouteParams p;
    p.logits = a->logits;
    p.bias = a->bias;
    p.weights = a->weights;
    p.ids = a->ids;
    p.E = a->E;
    p.k = a->k;
    p.groups = a->groups;
    p.keep = a->topk_groups;
    p.top = a->group_top;
    p.sigmoid = a->scoring == MHC_SIGMOID;
    p.renorm = a->renormalize;
    p.scale = a->scale;
    hipError_t e = mhc::launch_route(p, T, a->dtype, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess)
        return hip_fail(e, "route launch");
    return MHC_SEAM_OK;
}

}  // extern "C"
