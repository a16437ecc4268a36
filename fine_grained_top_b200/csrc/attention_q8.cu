// attention_q8.cu -- exact softmax attention over the selected keys of an
// 8-bit cache with a scale for each block of tokens.
//
//   S(r) = {s in TopK(r) : s <= p - W}  U  {max(0, p-W+1) .. p}
//   O[r,h] = sum_{s in S(r)} softmax_s(q[r,h] . kc[s] ks[s] scale) vs[s] vc[s]
//
// One warp computes one head of one row: d / 32 dims a lane, the keys one after
// another with a running maximum and sum.
#include <math_constants.h>

#include "internal.h"
#include "ptx.cuh"

namespace sa {

namespace {

template <int D>
__global__ void __launch_bounds__(128) attn_q8_simple_kernel(AttnQ8Args P) {
    constexpr int NV = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.x, h = blockIdx.y * 4 + warp, b = r / P.T;
    if (h >= P.Hq) return;
    const bool first = h == 0;
    int p = P.n_valid[r] - 1;
    if (p < -1 || p >= P.S_max) {
        if (first && lane == 0) report(P.dev_status, SA_DEV_INDEX);
        p = -1;
    }
    const float sl2 = P.scale * 1.4426950408889634f;
    float q[NV], o[NV], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        q[e] = __uint_as_float((uint32_t)P.q[((int64_t)r * P.Hq + h) * D + lane * NV + e] << 16);
        o[e] = 0.f;
    }
    auto code = [](uint8_t c) {
        uint32_t hh;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"((unsigned short)c));
        float f;
        asm("{ .reg .b16 l, u; mov.b32 {l, u}, %1; cvt.f32.f16 %0, l; }" : "=f"(f) : "r"(hh));
        return f;
    };
    auto sc = [](float s) { return fminf(fmaxf(s, 5.421010862427522e-20f), 1.8446744073709552e19f); };
    auto add = [&](int pos) {
        int64_t row;
        if (P.page_table) {
            const int page = P.page_table[(int64_t)b * P.max_pages + (pos >> 6)];
            if (page < 0 || page >= P.pool_pages) {
                if (first && lane == 0) report(P.dev_status, SA_DEV_INDEX);
                return;
            }
            row = (int64_t)page * 64 + (pos & 63);
        } else {
            row = (int64_t)b * P.S_max + pos;
        }
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < NV; ++e) dot = fmaf(q[e], code(P.k[row * D + lane * NV + e]), dot);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
        const float x = dot * sc(P.k_scale[row / P.scale_block]) * sl2;
        const float mn = fmaxf(m, x), f = exp2f(m - mn), w = exp2f(x - mn), vs = sc(P.v_scale[row / P.scale_block]);
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < NV; ++e) o[e] = o[e] * f + w * vs * code(P.v[row * D + lane * NV + e]);
        m = mn;
    };
    const int32_t *top = P.topk + (int64_t)r * P.K;
    int prev = -1;
    for (int i = 0; i < P.K; ++i) {
        const int e = top[i];
        if (e >= 0 && i > 0 && !(prev >= 0 && prev < e) && first && lane == 0) report(P.dev_status, SA_DEV_ORDER);
        if (e > p && p >= 0 && first && lane == 0) report(P.dev_status, SA_DEV_INDEX);
        prev = e;
        if (e >= 0 && e <= p - P.W) add(e);
    }
    for (int s = max(0, p - P.W + 1); s <= p; ++s) add(s);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const __nv_bfloat16 v = __float2bfloat16_rn(l > 0.f ? o[e] / l : (l == 0.f ? 0.f : l));
        P.out[((int64_t)r * P.Hq + h) * D + lane * NV + e] = *reinterpret_cast<const uint16_t *>(&v);
    }
    if (P.lse && lane == 0)
        P.lse[(int64_t)r * P.Hq + h] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

sa_status launch_attn_q8(const AttnQ8Args &a, cudaStream_t st) {
    const dim3 grid((unsigned)(a.B * a.T), (unsigned)((a.Hq + 3) / 4));
    if (a.d == 128) attn_q8_simple_kernel<128><<<grid, 128, 0, st>>>(a);
    else attn_q8_simple_kernel<64><<<grid, 128, 0, st>>>(a);
    return cuda_ok(cudaGetLastError());
}

}  // namespace sa
