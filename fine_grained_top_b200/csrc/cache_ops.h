// cache_ops.h -- launchers of the cache append and of the attention over an
// 8-bit cache, and what they share.
#pragma once

#include "internal.h"

namespace sa {

constexpr int kAppendMaxT = 131072;   // tokens a sequence and call into an 8-bit cache (see append_page)

struct AppendArgs {
    const uint16_t *q, *k, *v, *kI;
    int64_t ld_q, ld_k, ld_v, ld_kI;
    uint16_t *q_out;
    const int32_t *n_valid, *page_table;
    int max_pages, pool_pages, S_max;   // S_max: cached tokens a sequence can hold
    int B, T, Hq, d, D_I;
    const float *inv_freq;
    int rot_dim;
    bool interleaved, q8, kI_e4m3;
    void *k_cache, *v_cache, *kI_cache;
    float *k_scale, *v_scale;
    int scale_block;
    int *dev_status;
};
sa_status launch_append(const AppendArgs &a, cudaStream_t st);

struct AttnQ8Args {
    const uint16_t *q;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    int scale_block;
    const int32_t *page_table;
    int max_pages, pool_pages, S_max;   // S_max: cached tokens a sequence can hold
    const int32_t *n_valid, *topk;
    int K, W, B, T, Hq, d;
    float scale;
    uint16_t *out;
    float *lse;
    int *dev_status;
};
sa_status launch_attn_q8(const AttnQ8Args &a, cudaStream_t st);
// The same with `ctas` CTAs a row, whose waits give up after limit_ns, one for an MMA that never comes (d 128, Hq <= 16).
sa_status launch_attn_q8_check(const AttnQ8Args &a, int ctas, int lost, unsigned long long limit_ns, cudaStream_t st);

// A cached scale as a number in [2^-64, 2^64]; NaN -> 2^-64.
__device__ __forceinline__ float clamp_scale(float s) {
    return fminf(fmaxf(s, 5.421010862427522e-20f), 1.8446744073709552e19f);
}

// Cache rules shared by the append and the 8-bit attention: SA_OK when the
// cache's sizes are within limits.
inline sa_status check_cache_shape(const int32_t *page_table, int max_pages, int pool_pages, int page_size,
                                   int S_max, int B, int scale_block) {
    if (scale_block < 1 || scale_block > 64 || (scale_block & (scale_block - 1))) return SA_ERR_UNSUPPORTED;
    if (page_table) {
        if (page_size != 64) return SA_ERR_UNSUPPORTED;
        if (max_pages <= 0 || pool_pages <= 0) return SA_ERR_INVALID_ARG;
        if ((int64_t)pool_pages * 64 > INT32_MAX || (int64_t)max_pages * 64 > INT32_MAX) return SA_ERR_UNSUPPORTED;
    } else {
        if (S_max < 0 || S_max % scale_block) return SA_ERR_INVALID_ARG;
        if ((int64_t)B * S_max > INT32_MAX) return SA_ERR_UNSUPPORTED;
    }
    return SA_OK;
}

}  // namespace sa
