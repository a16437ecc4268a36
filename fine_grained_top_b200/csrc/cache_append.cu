// cache_append.cu -- fill the caches that the indexer, the top-K and the
// attention read: rotate new keys (and queries) to their positions, round or
// quantise them, and store them in their slots.
//
//   x'_first  = x_first cos a_i - x_second sin a_i,   a_i = p * inv_freq[i]
//   x'_second = x_second cos a_i + x_first sin a_i
//
// The angle p * inv_freq[i] (a position below 2^31 times 24 bits: 55) is an fp64
// product and what it rounds off, its turns likewise, with 1 / (2 pi) in two parts;
// their fraction is taken in fp64 and only then handed to fp32 sine and cosine, so
// that positions far out lose nothing.
//
// The step is bound by its bytes (the queries of all heads make nearly all of
// them) at prompt lengths, and by one launch's latency for single tokens: 8192
// rows of 64 heads into 8 bits 55 us (5.0 TB/s), 2 x 2048 rows of 16 heads into 16
// bits 11.6 us (3.3 TB/s), 16 single tokens 3.4 us, 64 into 16 bits 2.4 us, 7 x 333
// ragged rows with blocks of 16 into 8 bits 5.3 us.
// Two kinds of CTAs share one launch:
//   rows:  a few rows each, one 16-byte chunk (or the two halves of a pair of
//          chunks) per thread and turn; cosines and sines once a row in shared
//          memory, used by all of its heads.  With a 16-bit cache the key is one
//          more head of the row, value and index key are copied beside it.
//   pages: (8-bit caches) the new keys or values of one 64-token page, or of a
//          part of one, so that every scale block has one owner: a warp holds a
//          token in registers (d / 32 values a lane, pair partners exchanged by
//          shuffles), block maxima meet in shared memory, and codes are made
//          from the registers once the scales are known.
#include <algorithm>

#include "cache_ops.h"
#include "ptx.cuh"

namespace sa {

namespace {

constexpr int kAThreads = 256;
constexpr int kARowsMax = 8;        // rows of one row CTA
constexpr int kAPage = 64;

struct AppendParams {
    AppendArgs a;
    int n_page_ctas;     // CTAs of the page kind, first in the grid (8-bit caches)
    int unit;            // tokens of a page CTA: a page, or a part of one that whole scale blocks make
    int jobs;            // such units a sequence
    int rows;            // rows per row CTA
    int heads;           // heads a row CTA rotates: Hq, and the key with a 16-bit cache
    int u_rot, u_head;   // rotating chunks (or chunk pairs) and all units of a head
    int u_row;           // units of a row
    uint32_t m_head, m_row;   // ceil(2^16 / u_head), ceil(2^24 / u_row)
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// cos and sin of p * f (see the head of the file).  FAR: with what the products round off,
// under 2^-31 of a turn below kNear.  (The registers for it spill with 16-bit caches: 2 x 2048
// rows of 16 heads 14.1 us with, 12.8 without, so that a launch takes it by the cache's length.)
constexpr int kNear = 1 << 24;
template <bool FAR>
__device__ __forceinline__ float2 turn(int p, float f) {
    const double turn = 0.15915494309189535, turn_lo = -9.839338337591243e-18;   // 1 / (2 pi)
    const double a = (double)p * (double)f, t = a * turn;
    double part = t - rint(t);
    if (FAR) part += fma(a, turn, -t) + fma(a, turn_lo, fma((double)p, (double)f, -a) * turn);
    const float x = (float)(2.0 * part);   // the angle in half turns, -1 .. 1
    float2 cs;
    sincospif(x, &cs.y, &cs.x);
    return cs;
}

// Cache row of position p (within the cache) of sequence b; -1 for a bad page id.
__device__ __forceinline__ int64_t cache_slot(const AppendArgs &a, int b, int p) {
    if (!a.page_table) return (int64_t)b * a.S_max + p;
    const int page = a.page_table[(int64_t)b * a.max_pages + p / kAPage];
    if (page < 0 || page >= a.pool_pages) return -1;
    return (int64_t)page * kAPage + p % kAPage;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)c));
    float2 f;
    asm("{ .reg .b16 l, u; mov.b32 {l, u}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, u; }" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
__device__ __forceinline__ uint2 e4m3_of8(const uint4 &u) {
    uint2 o;
    o.x = e4m3x2(bf_lo(u.x), bf_hi(u.x)) | e4m3x2(bf_lo(u.y), bf_hi(u.y)) << 16;
    o.y = e4m3x2(bf_lo(u.z), bf_hi(u.z)) | e4m3x2(bf_lo(u.w), bf_hi(u.w)) << 16;
    return o;
}

// The smallest 2^e, -64 <= e <= 64, with amax <= 448 * 2^e (448 = 0.875 * 2^9).
__device__ __forceinline__ float scale_for(float amax) {
    if (!(amax > 0.f)) return 5.421010862427522e-20f;   // 2^-64
    int x;
    const float m = frexpf(amax, &x);
    const int e = min(64, max(-64, m <= 0.875f ? x - 9 : x - 8));
    return __int_as_float((e + 127) << 23);
}

// ------------------------------------------------------------------ rows
// One chunk pair (halves) or chunk (interleaved) of 8 values, rotated.
template <bool INTER>
__device__ __forceinline__ void rotate8(uint4 &a, uint4 &b, const float2 *cs) {
    uint32_t *x = reinterpret_cast<uint32_t *>(&a), *y = reinterpret_cast<uint32_t *>(&b);
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = bf_lo(x[i]), v = bf_hi(x[i]);
            x[i] = pack_bf16(u * cs[i].x - v * cs[i].y, v * cs[i].x + u * cs[i].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u0 = bf_lo(x[i]), u1 = bf_hi(x[i]), v0 = bf_lo(y[i]), v1 = bf_hi(y[i]);
            const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
            x[i] = pack_bf16(u0 * c0.x - v0 * c0.y, u1 * c1.x - v1 * c1.y);
            y[i] = pack_bf16(v0 * c0.x + u0 * c0.y, v1 * c1.x + u1 * c1.y);
        }
    }
}

template <bool INTER, bool FAR>
__device__ __forceinline__ void append_rows(const AppendParams &P, int cta, float2 (*cs)[64], int64_t *slot, int *pos) {
    const AppendArgs &a = P.a;
    const int R = a.B * a.T, r0 = cta * P.rows, nr = min(P.rows, R - r0), half = a.rot_dim / 2, tid = threadIdx.x;
    const int u_heads = P.heads * P.u_head, n_units = nr * P.u_row;
    // unit i: a chunk of 8 values (x), or the two halves of a pair of chunks (x, y)
    struct Unit {
        int rl, h, c;   // row; head, or P.heads: value and index key; chunk
    };
    auto unit = [&](int i) {
        Unit t;
        t.rl = (int)(((uint64_t)i * P.m_row) >> 24);
        const int u = i - t.rl * P.u_row;
        t.h = u < u_heads ? (int)((u * P.m_head) >> 16) : P.heads;
        t.c = u - t.h * P.u_head;
        return t;
    };
    auto load = [&](const Unit &t, uint4 &x, uint4 &y) {
        const int64_t r = r0 + t.rl;
        y = make_uint4(0, 0, 0, 0);
        if (t.h < P.heads) {
            const uint16_t *src = t.h == a.Hq ? a.k + r * a.ld_k : a.q + r * a.ld_q + t.h * a.d;
            const bool rot = t.c < P.u_rot;
            x = __ldcs(reinterpret_cast<const uint4 *>(src + (rot ? t.c * 8 : a.rot_dim + (t.c - P.u_rot) * 8)));
            if (!INTER && rot) y = __ldcs(reinterpret_cast<const uint4 *>(src + half + t.c * 8));
        } else {
            const int c = t.c * 8;
            x = c < a.d ? *reinterpret_cast<const uint4 *>(a.v + r * a.ld_v + c)
                        : *reinterpret_cast<const uint4 *>(a.kI + r * a.ld_kI + (c - a.d));
        }
    };
    // two units a turn; the first turn's values are on their way while the angles are computed
    Unit t[2] = {};
    uint4 x[2] = {}, y[2] = {};
    auto load2 = [&](int i) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (i + k * kAThreads < n_units) load(t[k] = unit(i + k * kAThreads), x[k], y[k]);
    };
    load2(tid);
    for (int i = tid; i < nr * half; i += kAThreads) {
        const int rl = i / half, f = i - rl * half, n = __ldg(a.n_valid + r0 + rl);
        if (n > 0) cs[rl][f] = turn<FAR>(n - 1, __ldg(a.inv_freq + f));
    }
    if (tid >= kAThreads - 32 && tid - (kAThreads - 32) < nr) {   // (the angles rarely reach the last warp)
        const int rl = tid - (kAThreads - 32), r = r0 + rl, n = __ldg(a.n_valid + r);
        int p = n - 1;
        int64_t s = -1;
        if (n < 0 || n > a.S_max) {
            report(a.dev_status, SA_DEV_INDEX);
            p = -1;
        } else if (p >= 0 && !a.q8) {
            s = cache_slot(a, r / a.T, p);
            if (s < 0) report(a.dev_status, SA_DEV_INDEX);
        }
        pos[rl] = p;
        slot[rl] = s;
    }
    __syncthreads();
    for (int i = tid; i < n_units;) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Unit &w = t[k];
            const bool is_k = w.h == a.Hq && w.h < P.heads;   // the row's key (16-bit cache)
            const int64_t r = r0 + w.rl, sl = slot[w.rl];
            if (i + k * kAThreads >= n_units || pos[w.rl] < 0 || (w.h >= a.Hq && sl < 0)) continue;   // (padding, no slot)
            if (w.h < P.heads) {
                uint16_t *dst = is_k ? static_cast<uint16_t *>(a.k_cache) + sl * a.d : a.q_out + (r * a.Hq + w.h) * a.d;
                if (w.c < P.u_rot) {
                    rotate8<INTER>(x[k], y[k], &cs[w.rl][INTER ? 4 * w.c : 8 * w.c]);
                    *reinterpret_cast<uint4 *>(dst + w.c * 8) = x[k];
                    if (!INTER) *reinterpret_cast<uint4 *>(dst + half + w.c * 8) = y[k];
                } else {
                    *reinterpret_cast<uint4 *>(dst + a.rot_dim + (w.c - P.u_rot) * 8) = x[k];
                }
            } else {
                const int c = w.c * 8;
                if (c < a.d)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.v_cache) + sl * a.d + c) = x[k];
                else if (a.kI_e4m3)
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.kI_cache) + sl * a.D_I + (c - a.d)) = e4m3_of8(x[k]);
                else
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.kI_cache) + sl * a.D_I + (c - a.d)) = x[k];
            }
        }
        i += 2 * kAThreads;
        load2(i);
    }
}

// ------------------------------------------------------------------ pages
// The scale and codes of one side (keys or values) of the page's new tokens.
template <int NV>
__device__ __forceinline__ void store_codes(uint8_t *dst, int lane, const float (&x)[NV], float s) {
    if (NV == 4)
        *reinterpret_cast<uint32_t *>(dst + lane * 4) =
            e4m3x2(__fdiv_rn(x[0], s), __fdiv_rn(x[1], s)) | e4m3x2(__fdiv_rn(x[NV - 2], s), __fdiv_rn(x[NV - 1], s)) << 16;
    else
        *reinterpret_cast<uint16_t *>(dst + lane * 2) = (uint16_t)e4m3x2(__fdiv_rn(x[0], s), __fdiv_rn(x[1], s));
}

__device__ __forceinline__ uint32_t finite_abs(float x) {   // bits of |x|, 0 for infinities and NaN
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// One side of a page, or of a part of it: its new keys (rotated) or values.
template <int D, bool INTER, bool KEYS, bool FAR>
__device__ __forceinline__ void append_page(const AppendParams &P, int job, uint32_t *amax, float *scale, int *red, float *ratio) {
    constexpr int NV = D / 32, NW = kAThreads / 32, NT = kAPage / NW;   // values a lane, warps, tokens a warp
    const AppendArgs &a = P.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = job / P.jobs, j = job - b * P.jobs;
    const int32_t *nv = a.n_valid + (int64_t)b * a.T;

    // The sequence's run of valid rows, checked.  Each unit reads all T numbers, from L2: next
    // to nothing at prompt lengths, but it grows with T^2 / 64, hence the limit kAppendMaxT.
    if (tid < kAPage) amax[tid] = 0;
    if (tid == 0) *ratio = 1.f;
    int first = 0, count, err = 0, n0;   // n0: n_valid of the run's first row
    if (a.T == 1) {
        n0 = __ldg(nv);
        count = n0 > 0;
        if (n0 < 0 || n0 > a.S_max) err = SA_DEV_INDEX;
        __syncthreads();
    } else {   // red: first, last, count, errors
        if (tid < 4) red[tid] = tid == 0 ? a.T : (tid == 1 ? -1 : 0);
        __syncthreads();
        int last = -1;
        first = a.T;
        count = 0;
        for (int t = tid; t < a.T; t += kAThreads) {
            const int n = __ldg(nv + t);
            if (n < 0 || n > a.S_max) err |= SA_DEV_INDEX;
            if (n > 0) {
                const int before = t > 0 ? __ldg(nv + t - 1) : 0;
                if (before > 0 && n != before + 1) err |= SA_DEV_ORDER;
                first = min(first, t);
                last = max(last, t);
                ++count;
            }
        }
        if (last >= 0) {
            atomicMin(&red[0], first);
            atomicMax(&red[1], last);
            atomicAdd(&red[2], count);
        }
        if (err) atomicOr(&red[3], err);
        __syncthreads();
        first = red[0];
        count = red[2];
        err = red[3];
        if (count > 0 && red[1] - first + 1 != count) err |= SA_DEV_ORDER;   // a gap
        n0 = count > 0 ? __ldg(nv + first) : 0;
    }
    if (err & SA_DEV_INDEX) err = SA_DEV_INDEX;   // a number out of range is no successor either: one error
    if (err || count == 0) {
        if (err && j == 0 && tid == 0) report(a.dev_status, err);
        return;
    }
    const int p0 = n0 - 1, o_p0 = p0 & (P.unit - 1);   // first position, its place in its unit
    const int at = max(j * P.unit - o_p0, 0), m = min((j + 1) * P.unit - o_p0, count) - at;   // the unit's tokens of the run
    if (m <= 0) return;
    const int begin = p0 + at, o0 = begin & (P.unit - 1), sb = a.scale_block;
    const int64_t base = cache_slot(a, b, begin - o0);   // the unit's first slot
    const int64_t row0 = (int64_t)b * a.T + first + at;
    const uint16_t *src = KEYS ? a.k : a.v;
    const int64_t ld = KEYS ? a.ld_k : a.ld_v;
    uint8_t *cache = static_cast<uint8_t *>(KEYS ? a.k_cache : a.v_cache);

    // this warp's tokens warp, warp + NW, ...
    const int half = a.rot_dim / 2, hl = half / NV;      // lanes of one half of the rotated dims
    const int d0 = lane * NV;                            // this lane's first dim
    const bool rot = d0 < a.rot_dim;
    const int partner = INTER ? lane : (lane < hl ? lane + hl : (lane < 2 * hl ? lane - hl : lane));
    const bool upper = !INTER && lane >= hl;
    uint32_t w[NT][NV / 2];   // the values as they came, in bf16
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int tok = i * NW + warp;
        if (tok >= m) break;   // the same for the whole warp
#pragma unroll
        for (int e = 0; e < NV / 2; ++e)
            w[i][e] = __ldg(reinterpret_cast<const uint32_t *>(src + (row0 + tok) * ld + d0) + e);
    }
    if (base < 0) {
        if (tid == 0) report(a.dev_status, SA_DEV_INDEX);
        return;
    }
    // the old scale of a block that holds earlier tokens (the first one, if any)
    const int blk0 = o0 / sb, blk1 = (o0 + m - 1) / sb;
    float *scales = (KEYS ? a.k_scale : a.v_scale) + base / sb;
    const bool partial = blk0 * sb < o0;
    const float was = partial && tid == 0 ? scales[blk0] : 0.f;
    float x[NT][NV];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int tok = i * NW + warp;
        if (tok >= m) break;
        float y[NV];
#pragma unroll
        for (int e = 0; e < NV; ++e) x[i][e] = y[e] = e & 1 ? bf_hi(w[i][e / 2]) : bf_lo(w[i][e / 2]);
        if (KEYS && INTER) {
#pragma unroll
            for (int e = 0; e < NV / 2; ++e) {
                const float2 c = rot ? turn<FAR>(begin + tok, __ldg(a.inv_freq + d0 / 2 + e)) : make_float2(1.f, 0.f);
                if (rot) {
                    x[i][2 * e] = y[2 * e] * c.x - y[2 * e + 1] * c.y;
                    x[i][2 * e + 1] = y[2 * e + 1] * c.x + y[2 * e] * c.y;
                }
            }
        } else if (KEYS) {
            // the pair's two lanes need the same NV angles: each takes half of them
            const int f0 = (upper ? d0 - half : d0);
            float2 mine[NV / 2];
#pragma unroll
            for (int e = 0; e < NV / 2; ++e)
                mine[e] = rot ? turn<FAR>(begin + tok, __ldg(a.inv_freq + f0 + (upper ? NV / 2 : 0) + e)) : make_float2(1.f, 0.f);
#pragma unroll
            for (int e = 0; e < NV / 2; ++e) {
                const float2 other = make_float2(__shfl_sync(0xffffffffu, mine[e].x, partner),
                                                 __shfl_sync(0xffffffffu, mine[e].y, partner));
                const float2 c0 = upper ? other : mine[e], c1 = upper ? mine[e] : other;   // angles e and NV / 2 + e
                const float y0 = __shfl_sync(0xffffffffu, y[e], partner);
                const float y1 = __shfl_sync(0xffffffffu, y[NV / 2 + e], partner);
                const float s0 = upper ? c0.y : -c0.y, s1 = upper ? c1.y : -c1.y;
                if (rot) {
                    x[i][e] = y[e] * c0.x + y0 * s0;
                    x[i][NV / 2 + e] = y[NV / 2 + e] * c1.x + y1 * s1;
                }
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < NV; ++e) top = max(top, finite_abs(x[i][e]));
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) atomicMax(&amax[(o0 + tok) / sb], top);   // non-negative floats order as their bits
    }
    if (!KEYS && a.kI) {   // index keys beside the values
        const int nc = a.D_I / 8;
        for (int i = tid; i < m * nc; i += kAThreads) {
            const int tok = i / nc, c = (i - tok * nc) * 8;
            const uint4 v = *reinterpret_cast<const uint4 *>(a.kI + (row0 + tok) * a.ld_kI + c);
            const int64_t o = (base + o0 + tok) * a.D_I + c;
            if (a.kI_e4m3)
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.kI_cache) + o) = e4m3_of8(v);
            else
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.kI_cache) + o) = v;
        }
    }
    __syncthreads();
    if (tid <= blk1 - blk0) {   // the touched blocks' scales
        float s = scale_for(__uint_as_float(amax[blk0 + tid]));
        if (tid == 0 && partial) {
            const float old = clamp_scale(was);
            s = fmaxf(s, old);
            if (s != old) *ratio = __fdiv_rn(old, s);   // what the earlier tokens' codes shrink by
        }
        scale[blk0 + tid] = s;
        scales[blk0 + tid] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int tok = i * NW + warp;
        if (tok >= m) break;
        store_codes<NV>(cache + (base + o0 + tok) * D, lane, x[i], scale[(o0 + tok) / sb]);
    }
    const float f = *ratio;
    if (f != 1.f) {
        uint32_t *words = reinterpret_cast<uint32_t *>(cache + (base + blk0 * sb) * D);
        for (int i = tid; i < (o0 - blk0 * sb) * (D / 4); i += kAThreads) {
            const uint32_t c = words[i];
            const float2 lo = from_e4m3x2(c & 0xFFFFu), hi = from_e4m3x2(c >> 16);
            words[i] = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
        }
    }
}

// CTAs an SM: the row CTAs hold two units a thread in flight, and the more CTAs
// share an SM the better they cover each other (8192 rows of 64 heads: 92 us with the
// two that fit unbounded, 57 with four, 55 with five, which spill 28 to 40 bytes with 128
// dims; six spill 112 to 180).  With 16 bits eight spill 104 bytes with halves as pairs,
// none with neighbours (2 x 2048 rows 12.8 us with eight, 14.3 with six).
template <int D, bool INTER, bool Q8, bool FAR>
__global__ void __launch_bounds__(kAThreads, Q8 ? 5 : 8) append_kernel(AppendParams P) {
    __shared__ float2 cs[kARowsMax][64];
    __shared__ int64_t slot[kARowsMax];
    __shared__ int pos[kARowsMax];
    if constexpr (Q8) {
        const int job = (int)blockIdx.x;
        if (job < P.n_page_ctas) {
            __shared__ uint32_t amax[kAPage];
            __shared__ float scale[kAPage], ratio;
            __shared__ int red[4];
            if (job & 1) append_page<D, INTER, false, FAR>(P, job >> 1, amax, scale, red, &ratio);
            else append_page<D, INTER, true, FAR>(P, job >> 1, amax, scale, red, &ratio);
            return;
        }
    }
    append_rows<INTER, FAR>(P, (int)blockIdx.x - P.n_page_ctas, cs, slot, pos);
}

template <int D, bool INTER, bool FAR>
void launch_append_kernel(const AppendParams &P, unsigned grid, cudaStream_t st) {
    if (P.a.q8) append_kernel<D, INTER, true, FAR><<<grid, kAThreads, 0, st>>>(P);
    else append_kernel<D, INTER, false, FAR><<<grid, kAThreads, 0, st>>>(P);
}
template <int D, bool INTER>
void launch_append_kernel(const AppendParams &P, unsigned grid, cudaStream_t st) {
    if (P.a.S_max > kNear) launch_append_kernel<D, INTER, true>(P, grid, st);
    else launch_append_kernel<D, INTER, false>(P, grid, st);
}

}  // namespace

sa_status launch_append(const AppendArgs &a, cudaStream_t st) {
    AppendParams P;
    P.a = a;
    const int64_t R = (int64_t)a.B * a.T;
    // Smaller units shorten a page CTA's chain, but each reads all T lengths.  Blocks of 16,
    // one sequence, units of 16 / 32 / 64 tokens: 64 rows 4.1 / 5.1 / 6.9 us, 1024 rows 5.0 /
    // 5.4 / 7.0, 4096 rows 8.7 / 8.0 / 9.3, 16384 rows 42 / 28 / 23.
    P.unit = a.T <= 1024 ? std::max(a.scale_block, 16) : a.T <= 4096 ? std::max(a.scale_block, 32) : kAPage;
    P.jobs = (a.T + P.unit - 2) / P.unit + 1;   // units that T consecutive tokens can touch
    const int64_t n_page = a.q8 ? 2 * (int64_t)a.B * P.jobs : 0;   // keys and values apart
    P.heads = a.q8 ? a.Hq : a.Hq + 1;
    P.u_rot = a.interleaved ? a.rot_dim / 8 : a.rot_dim / 16;
    P.u_head = P.u_rot + (a.d - a.rot_dim) / 8;
    P.u_row = P.heads * P.u_head + (a.q8 ? 0 : (a.d + a.D_I) / 8);
    P.rows = P.u_row > 0 ? std::min(kARowsMax, std::max(1, kAThreads / P.u_row)) : 1;
    P.m_head = (65536u + P.u_head - 1) / P.u_head;
    P.m_row = P.u_row > 0 ? ((1u << 24) + P.u_row - 1) / P.u_row : 0;
    const int64_t n_rows = P.u_row > 0 ? (R + P.rows - 1) / P.rows : 0;
    if (n_page + n_rows > INT32_MAX) return SA_ERR_UNSUPPORTED;
    P.n_page_ctas = (int)n_page;
    const unsigned grid = (unsigned)(n_page + n_rows);
    if (grid == 0) return SA_OK;
    if (a.d == 128) {
        if (a.interleaved) launch_append_kernel<128, true>(P, grid, st);
        else launch_append_kernel<128, false>(P, grid, st);
    } else {
        if (a.interleaved) launch_append_kernel<64, true>(P, grid, st);
        else launch_append_kernel<64, false>(P, grid, st);
    }
    return cuda_ok(cudaGetLastError());
}

}  // namespace sa
