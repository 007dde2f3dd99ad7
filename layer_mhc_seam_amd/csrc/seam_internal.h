// seam_internal.h -- shared between the HIP kernels and the host runtime of
// libmhc_seam.so (not part of the public C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mhc_seam.h"
#include "cache_layout.h"

namespace mhc {

// Set the calling thread's error message and return the status
// (seam_runtime.cpp).
int fail(int status, const char *fmt, ...) __attribute__((visibility("hidden")));
int hip_fail(hipError_t e, const char *what) __attribute__((visibility("hidden")));
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kBlockTokens = 16;   // tokens per block: the MFMA M dimension
constexpr int kWaves = 8;          // waves per workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kChunk = 32;         // columns per quantiser group / MFMA K step
constexpr int kSeg = 64;           // columns per segment (one 128-byte line per row)
constexpr int kPartFloats = 32;    // per (block, split, token) partial record
constexpr int kMaxSplits = 128;    // splits per block (<= H/64 for H <= 8192)

// kCollapse: x collapsed with pre, its sums of squares and the norm only
// (no post-mix, no gate projection): the second launch of the unshifted
// ordering, whose gates the first launch computed
enum Form { kPost = 0, kNoPost = 1, kCollapse = 2 };
enum Out { kBf16 = 0, kFp8Grid = 1, kMxfp8 = 2, kMxfp8G128 = 3 };

struct SeamParams {
    int T, H, nchunks, nseg;
    int nblocks, ksplit, segs_per_split;
    int rows_blocks;          // blocks [0, rows_blocks) whole-row, the rest split
    float eps;
    int iters;
    int identity_pre;
    int skip_norm;            // post-mix and gates only (no collapse output)
    int skip_gates;           // collapse, norm and quantiser only (no gates)
    const uint16_t *x;
    const uint16_t *y;
    const float *pre;
    const float *post;
    const float *res;
    const void *fnp;          // packed fn: [nchunks][4][3][64] x 16 bytes
    const uint16_t *gamma;
    const float *bias;
    uint16_t *resid;
    uint16_t *norm;
    uint16_t *grid;
    uint8_t *codes;
    uint8_t *scales;
    float *pre_out;
    float *post_out;
    float *res_out;
    // split-mode scratch; partials and u cover the split blocks only (blocks
    // rows_blocks .. nblocks-1, tokens 16*rows_blocks .. T-1)
    float *part;              // [nblocks - rows_blocks][ksplit][16][kPartFloats]
    uint16_t *uscr;           // [T - 16*rows_blocks][H] bf16 u of handed-off splits
    int *sync;                // [nblocks - rows_blocks][sync_stride]: arrival counter, two
                              // hand-off mask sets
    int sync_stride;          // ints per block (one 128-byte line)
    int spin_limit;           // polls a waiting split makes before handing off
};

// bytes of the packed fn for width H
inline size_t fn_pack_bytes(int H) { return (size_t)(H / kChunk) * 4 * 3 * 64 * 16; }

// whole-row kernels are compiled for nseg == 8 * rs with these rs
bool row_segs_instance(int rs);

hipError_t launch_fn_pack(const float *fn, int H, void *pack, hipStream_t s);
hipError_t launch_seam(const SeamParams &p, int form, int out, int row_segs,
                       int grid, hipStream_t s);
hipError_t launch_copy(void *dst, const void *src, size_t bytes, int cus, hipStream_t s);
hipError_t launch_stream_mix(void *dst, size_t dst_bytes, const void *src, size_t src_bytes,
                             int cus, hipStream_t s);
// The MXFP8 GEMM's output blocks for T x N on cus CUs: TM x TN and the
// number of LDS stages (host only; the launch takes exactly this shape)
struct GemmBlocks {
    int tm, tn, stages;
};
GemmBlocks gemm_blocks(int64_t T, int N, int cus);
hipError_t launch_mxfp8_gemm(const uint8_t *a, const uint8_t *sa, const uint8_t *b,
                             const uint8_t *sb, int T, int N, int K, uint16_t *out, int cus,
                             hipStream_t s);
hipError_t launch_head_reduce(const uint16_t *x, const float *w, int64_t T, int H, uint16_t *out,
                              int cus, hipStream_t s);

// The one-stream block norm (block_kernels.hip); P.y, gamma_post, gate,
// gamma, norm and codes are null where the call has none
struct BlockNormParams {
    int64_t T;
    int H;
    int gate_kind;            // mhc_gate
    float eps, residual_scale, branch_scale;
    double inv_H;             // 1 / H
    const void *x;
    const void *y;
    const void *gamma_post;
    const void *gate;
    const void *gamma;
    void *residual_out;
    void *norm;
    int8_t *codes;
    float *scales;
};
hipError_t launch_block_norm(const BlockNormParams &p, int dtype, int x_dtype, hipStream_t s);
hipError_t launch_int8_quantize(const void *src, int dtype, int64_t rows, int H, int8_t *codes,
                                float *scales, hipStream_t s);

// int8 product (int8_kernels.hip)
struct Int8GemmParams {
    const int8_t *a;
    const float *sa;
    const int8_t *b;
    const float *sb;
    const float *bias;        // null without one
    void *out;
    int T, N, K;
};
GemmBlocks int8_gemm_blocks(int64_t T, int N, int cus);
hipError_t launch_int8_gemm(const Int8GemmParams &p, int out_dtype, int cus, hipStream_t s);

// Expert routing (route_kernels.hip)
struct RouteParams {
    const void *logits;
    const float *bias;        // null without one
    float *weights;
    int32_t *ids;
    int E, k, groups, keep, top;
    int sigmoid, renorm;
    float scale;
};
hipError_t launch_route(const RouteParams &p, int64_t tokens, int dtype, hipStream_t s);

// Rotary positions (rope_kernels.hip)
struct RopeParams {
    int64_t T;
    int q_heads, k_heads, head_dim, rotary;
    int inverse, position_bytes;
    float scale;
    int units;                // of a head: pairs by the vector, and channels to copy
    int head_steps;           // threads that share a unit of a token, heads dealt out in turn
    int64_t position_axis;
    int64_t q_token, q_head, k_token, k_head, q_out_token, q_out_head, k_out_token, k_out_head;
    const uint16_t *q;
    const uint16_t *k;
    const void *positions;
    const float *inv_freq;
    uint16_t *q_out;
    uint16_t *k_out;
    uint32_t axis[16];        // two bits a pair
};
hipError_t launch_rope(RopeParams p, int dtype, int vector, bool interleaved, bool in_place, int cus, hipStream_t s);

// The 4-bit cache (cache_kernels.hip)
struct CacheParams {
    CacheLayout c;
    int64_t T;
    int slot_bytes;
    int64_t k_token, k_head, v_token, v_head;
    uint8_t *cache;
    const void *slots;
    void *k;
    void *v;
};
hipError_t launch_cache(const CacheParams &p, int head_dim, int dtype, bool write, int cus, hipStream_t s);

// Attention over it (attention_kernels.hip)
struct AttentionParams {
    CacheLayout c;
    int64_t T, max_len;       // max_len: no more than the tables hold
    int64_t seen;             // as much of it as a window leaves a sequence's rows
    int64_t q_token, q_head, table_stride;
    int B, q_heads, group;    // group: query heads a kv head
    int causal, window;
    float scale, softcap;
    const uint16_t *q;
    const uint8_t *cache;
    const int32_t *tables;
    const int32_t *lens;
    const int32_t *q_starts;
    uint16_t *out;
    float *lse;
    float *workspace;
    int workers;
    int64_t blocks;           // row blocks that the batch may have
};
// Floats of workspace, 0 for none, and the launch, which takes them as a plan
uint64_t attention_workspace_floats(int64_t T, int B, int q_heads, int kv_heads, int head_dim, int cus,
                                    int64_t max_len);
hipError_t launch_attention(const AttentionParams &p, int head_dim, int dtype, int cus, hipStream_t s);
// The same for many query rows a sequence (prompt_kernels.hip)
uint64_t prompt_workspace_floats(int64_t T, int B, int q_heads, int kv_heads, int head_dim, int cus, int64_t max_len);
hipError_t launch_prompt(const AttentionParams &p, int head_dim, int dtype, int cus, hipStream_t s);

hipError_t launch_quantize(const uint16_t *src, int rows, int H, int group, uint8_t *codes,
                           uint8_t *scales, uint16_t *grid, hipStream_t s);

}  // namespace mhc
