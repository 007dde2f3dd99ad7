// The argument checks of the cache operators' C entries on sizes and strides
// at the ends of their types, built for the host with overflow checks that trap:
// each call is refused, and no product overflows on the way.  Nothing is
// launched: the functions behind the checks are stand-ins that end the program.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../layer_mhc_seam_amd/csrc/cache_runtime.cpp"

namespace mhc {

int fail(int status, const char *, ...) { return status; }
int hip_fail(hipError_t, const char *) { return MHC_SEAM_HIP_ERROR; }
hipError_t launch_rope(RopeParams, int, int, bool, bool, int, hipStream_t) { abort(); }
hipError_t launch_cache(const CacheParams &, int, int, bool, int, hipStream_t) { abort(); }
hipError_t launch_attention(const AttentionParams &, int, int, int, hipStream_t) { abort(); }
uint64_t attention_workspace_floats(int64_t, int, int, int, int, int, int64_t) { return 0; }

}  // namespace mhc

// no device: what passes all checks that come before one ends here
extern "C" hipError_t hipGetDevice(int *) { return hipErrorNoDevice; }
extern "C" hipError_t hipDeviceGetAttribute(int *, hipDeviceAttribute_t, int) { return hipErrorNoDevice; }

static char *at(int k) { return (char *)(uintptr_t)0x7f0000000000 + ((uintptr_t)k << 36); }

static int bad;

static void refused(const char *what, int64_t v, int status)
{
    if (status != MHC_SEAM_INVALID_ARG) {
        std::printf("%s = %lld: status %d\n", what, (long long)v, status);
        ++bad;
    }
}

int main()
{
    mhc_rope_args rope{4, 8, 2, 128, 128, 0, 4, 1, 0, 0, 1.0f, 4, 1024, 128, 256, 128, 1024, 128, 256, 128,
                       at(0), at(1), at(2), (float *)at(3), nullptr, at(4), at(5)};
    mhc_cache_args cache{4, 8, 64, 2, 128, 0, 8, 0, 256, 128, 256, 128, at(0), at(1), at(2), at(3)};
    mhc_cache_attention_args attention{};
    attention.T = attention.B = 4;
    attention.pages = 8;
    attention.q_token = 1024;
    attention.q_head = attention.head_dim = 128;
    attention.table_stride = attention.table_width = 4;
    attention.q_heads = 8;
    attention.kv_heads = 2;
    attention.page_size = 64;
    attention.causal = 1;
    attention.scale = 0.1f;
    attention.q = at(0);
    attention.cache = (uint8_t *)at(1);
    attention.tables = (int32_t *)at(2);
    attention.lens = (int32_t *)at(3);
    attention.out = at(5);
    attention.workspace = at(7);
    // as they stand these pass: only the device is missing
    if (mhc_rope(&rope, nullptr) != MHC_SEAM_HIP_ERROR || mhc_cache_write(&cache, nullptr) != MHC_SEAM_HIP_ERROR ||
        mhc_cache_read(&cache, nullptr) != MHC_SEAM_HIP_ERROR ||
        mhc_cache_attention(&attention, nullptr) != MHC_SEAM_HIP_ERROR)
        std::printf("a call that is right was refused\n"), ++bad;
    for (const int64_t v : {INT64_MAX, INT64_MIN, INT64_MAX / 2 + 1, INT64_MIN / 4 - 1, INT64_MAX / 4 + 9, int64_t(-1)}) {
        for (int64_t mhc_rope_args::*m :
             {&mhc_rope_args::T, &mhc_rope_args::q_token, &mhc_rope_args::q_head, &mhc_rope_args::k_token,
              &mhc_rope_args::k_head, &mhc_rope_args::q_out_token, &mhc_rope_args::q_out_head,
              &mhc_rope_args::k_out_token, &mhc_rope_args::k_out_head, &mhc_rope_args::position_axis}) {
            mhc_rope_args a = rope;
            a.axes = 2;
            a.*m = v;
            refused("rope", v, mhc_rope(&a, nullptr));
        }
        for (int64_t mhc_cache_args::*m :
             {&mhc_cache_args::T, &mhc_cache_args::pages, &mhc_cache_args::k_token, &mhc_cache_args::k_head,
              &mhc_cache_args::v_token, &mhc_cache_args::v_head}) {
            mhc_cache_args a = cache;
            a.*m = v;
            refused("write", v, mhc_cache_write(&a, nullptr));
            refused("read", v, mhc_cache_read(&a, nullptr));
        }
        for (int64_t mhc_cache_attention_args::*m :
             {&mhc_cache_attention_args::T, &mhc_cache_attention_args::pages, &mhc_cache_attention_args::q_token,
              &mhc_cache_attention_args::q_head, &mhc_cache_attention_args::table_stride}) {
            mhc_cache_attention_args a = attention;
            a.*m = v;
            refused("attention", v, mhc_cache_attention(&a, nullptr));
        }
        uint64_t bytes;
        refused("workspace", v, mhc_cache_attention_workspace(v, 4, 8, 2, 128, 256, 1000, &bytes));
        refused("workspace's length", v, mhc_cache_attention_workspace(4, 4, 8, 2, 128, 256, v, &bytes));
    }
    if (!bad)
        std::puts("ok");
    return bad != 0;
}
