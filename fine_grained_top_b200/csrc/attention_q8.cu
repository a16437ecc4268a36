// attention_q8.cu -- exact softmax attention over the selected keys of an
// 8-bit cache with a scale for each block of tokens (one new token or a chunk
// of tokens a sequence, contiguous or paged).
//
//   S(r) = {s in TopK(r) : s <= p - W}  U  {max(0, p-W+1) .. p}
//   x_s = (q[r,h] . kc[s]) ks[s] scale,   O[r,h] = sum_s softmax(x)_s vs[s] vc[s]
//
// The codes go into the tensor cores as they lie in the cache (tcgen05
// kind::f8f6f4, e4m3 x e4m3 products are exact, fp32 sums): nothing is
// widened on the way, so a key costs 2 d bytes of gather and no conversions.
// The 16-bit operands are split instead: q = (q_hi + q_lo) 2^e and P = P_hi +
// P_lo, two e4m3 parts each, put side by side on the MMA's N dimension.  Four
// significant bits and four of the rest hold a bf16 q exactly down to 2^-10 of
// the row's largest value (2^-18 of it is the error below), and P to 2^-8 of
// its value; the scales stay out of the products: in
//   S^T = K Q^T        M = 128 keys, N = 2 x heads, K = d            -> TMEM
//   P^T                softmax over keys, one thread per key lane
//   O^T += V^T P^T     M = d, N = 2 x heads, K = 128 keys            -> TMEM
// a key is a lane, so ks and vs are one number per thread: with
//   e = (S_hi + S_lo) ks scale log2e + log2 vs - m,    P = 2^e
// the running maximum m is of the contributions p vs (so P fills e4m3's range
// whatever the scales), and the row sum takes P / vs.  After a raise the
// largest P is 2^6; it may grow to 2^8.75 (e4m3 ends at 448) before the next.
//
// CTAs (one per SM) stream their tiles through a pipeline of warp roles:
//   scan (one warp): row after row: its length, the prefix of its top-K in
//               front of the window (SA_DEV_INDEX / SA_DEV_ORDER), its Q split
//               into shared memory; rows without keys are written here
//   index builder (one warp): each tile's cache rows (page table two tiles
//               ahead) and its scales (4-byte cp.async)
//   gather (two warps a side): 16-byte cp.async of the K and V rows into
//               swizzled tiles of separate rings; slots without a key are
//               zero-filled, so nothing that was not selected is ever read
//   S issuer, P V issuer (one thread each)
//   softmax (HQP / HG groups of four warps, HG heads each)
// Many rows: persistent CTAs take whole rows.  Few rows: a thread-block
// cluster shares a row, each CTA a run of its tiles, and the partial (m, l, O)
// meet through distributed shared memory.  Every wait is bounded
// (SA_DEV_TIMEOUT).
#include <math_constants.h>

#include <algorithm>

#include "gather_pipe.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sa {

namespace {

constexpr int kTile = 128;                  // keys per tile (MMA M)
constexpr int kGW = 2;                      // gather warps per side
constexpr int kGKeys = kTile / kGW;         // keys of a tile per gather warp
constexpr int kWarpSmx = 2 * kGW;           // first softmax warp
constexpr int kRing = 6;                    // row-index tiles the builder runs ahead
constexpr int kInfo = 8;                    // tile records and scales in flight
constexpr int kRows = 4;                    // rows the scan runs ahead
constexpr int kPB = 3;                      // P buffers in shared memory
constexpr float kTop = 6.f, kRaise = 8.75f; // log2 of the largest P after a raise, and before the next
constexpr float kLowest = -1e30f;           // running maximum of a row that has met no key yet
constexpr size_t kSmemLimit = 232448;
// At least this much shared memory, so that two CTAs of these kernels never
// share an SM: a CTA waiting for TMEM columns that another cluster's CTA holds
// could wait for good.
constexpr size_t kSmemLeast = 118784;

struct Params {
    AttnQ8Args a;
    int G;                // CTAs a row (cluster size); 1: persistent CTAs
    int n_units;          // persistent CTAs, or clusters
    int sb_shift;         // log2 of the tokens a scale
    float scale_log2;
};

struct RowInfo {
    int end, r, b, n_top, n_keys, w0, i0, i1;
};
struct TileRec {
    int end, r, j, first, last, full;
    uint32_t vmask[4];    // slots that hold a key
};

template <int D_, int HQP_>
struct Cfg {
    static constexpr int D = D_, HQP = HQP_;
    static constexpr int N2 = 2 * HQP;                    // MMA N: hi and lo columns
    static constexpr int NG = HQP == 64 ? 4 : 2;          // softmax groups
    static constexpr int HG = HQP / NG;                   // heads of a group
    static constexpr int kWarpS = kWarpSmx + 4 * NG, kWarpBuild = kWarpS + 1, kWarpPV = kWarpS + 2, kWarpScan = kWarpS + 3;
    static constexpr int kThreads = (kWarpScan + 1) * 32;
    static constexpr int SB = HQP == 64 ? 2 : 4;          // S buffers in TMEM
    static constexpr int kKV = kTile * D, kQ = N2 * D, kP = kTile * N2;
    static constexpr int kSoft = 4 * NG;                  // softmax warps
    static constexpr int kBarFixed = 2 * kRing + 2 * kInfo + 2 * kRows + 2 * SB + kPB + 2 * 5;
    static constexpr size_t fixed() {
        return 1024 + 2 * (size_t)kQ + kPB * (size_t)kP + kRing * (kTile * 4 + sizeof(TileRec)) +
               kInfo * (2 * kTile * 4 + sizeof(TileRec)) + kRows * sizeof(RowInfo) + 8 * 4 +
               (2 * 4 * HQP + 4 * HQP + 2 * 2 * HQP) * 4 + 2 * 16 * HQP * 4 + (kBarFixed + 4 * 6) * 8 + 64;
    }
    static constexpr int ring() {
        int n = 6;
        while (n > 2 && fixed() + 2 * (size_t)n * kKV > kSmemLimit) --n;
        return n;
    }
    static constexpr int NK = ring(), NV = NK;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + NK * kKV;
    static constexpr int kOffQ = kOffV + NV * kKV;
    static constexpr int kOffP = kOffQ + 2 * kQ;
    static constexpr int kOffRows = kOffP + kPB * kP;                         // [kRing][128] cache rows
    static constexpr int kOffScale = kOffRows + kRing * kTile * 4;            // [kInfo][2][128] ks, vs
    static constexpr int kOffRed = kOffScale + kInfo * 2 * kTile * 4;         // maxima [4][HQP], sums [4][HQP]
    static constexpr int kOffNegM = kOffRed + 2 * 4 * HQP * 4;                // [softmax warp][HG] minus the running maxima
    static constexpr int kOffEpi = kOffNegM + 4 * HQP * 4;                    // m, l of two rows [2][2][HQP]
    static constexpr int kOffMerge = kOffEpi + 2 * 2 * HQP * 4;               // [2][HQP * 16] every CTA's m, l (clusters)
    static constexpr int kOffRingRec = kOffMerge + 2 * 16 * HQP * 4;          // [kRing] TileRec
    static constexpr int kOffRec = kOffRingRec + kRing * (int)sizeof(TileRec);
    static constexpr int kOffRow = kOffRec + kInfo * (int)sizeof(TileRec);    // [kRows] RowInfo
    static constexpr int kOffQs = kOffRow + kRows * (int)sizeof(RowInfo);     // [8] q scales
    static constexpr int kOffBar = (kOffQs + 8 * 4 + 7) & ~7;
    static constexpr int kNumBar = kBarFixed + 2 * NK + 2 * NV;
    static constexpr size_t kUsed = 1024 + (size_t)kOffBar + kNumBar * 8 + 16;
    static constexpr size_t kSmem = kUsed > kSmemLeast ? kUsed : kSmemLeast;
    static constexpr int kCols = (SB + 2) * N2;
    static constexpr uint32_t kTmemCols = kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512 && kSmem <= kSmemLimit, "TMEM or shared memory");
    static_assert(NK * kKV >= HQP * D * 4, "the partial O of a cluster's CTA lies in the K ring");
};

// ------------------------------------------------------------------ helpers
typedef unsigned long long f2;   // a pair of f32 (one 64-bit register pair)
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 pku(uint32_t lo, uint32_t hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 up(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float redux_max(float x) {   // NaN counts as absent
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
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
__device__ __forceinline__ void cp_async4(void *smem_dst, const void *gsrc) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gsrc) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(void *smem_dst, const void *gsrc, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(gsrc), "r"(some ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ float clamp_scale(float s) {   // into [2^-64, 2^64]; NaN -> 2^-64
    return fminf(fmaxf(s, 5.421010862427522e-20f), 1.8446744073709552e19f);
}
__device__ __forceinline__ float dsmem_ld_f32(const void *local, uint32_t rank) {
    return __uint_as_float(dsmem_ld_u32(local, rank));
}
__device__ __forceinline__ float4 dsmem_ld_f4(const void *local, uint32_t rank) {
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}
// Byte offset of 16-byte chunk `ch` of row `r` in a tile of D-byte rows with
// the D-byte swizzle (128 or 64).
template <int D>
__device__ __forceinline__ uint32_t sw(int r, int ch) {
    return (uint32_t)(r * D + ((D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4));
}
// MN-major operand of D-byte K rows with the D-byte swizzle.  D = 64: the MMA's
// upper 64 M rows read the same 64 dims again (a stride of 0 between the MN
// chunks); their results are not used.
template <int D>
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((8 * D) >> 4) << 32;      // 8-row K groups
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
    return d;
}

template <int D, int HQP>
__global__ void __launch_bounds__(Cfg<D, HQP>::kThreads, 1) attn_q8_kernel(Params P) {
    using C = Cfg<D, HQP>;
    constexpr int NK = C::NK, NV = C::NV, N2 = C::N2, SB = C::SB, HG = C::HG, NG = C::NG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int32_t *rows = reinterpret_cast<int32_t *>(sm + C::kOffRows);
    float *scales = reinterpret_cast<float *>(sm + C::kOffScale);
    float *redmax = reinterpret_cast<float *>(sm + C::kOffRed), *redsum = redmax + 4 * HQP;
    float *epi_m = reinterpret_cast<float *>(sm + C::kOffEpi), *epi_l = epi_m + 2 * HQP;   // [2 rows][HQP]
    TileRec *rrec = reinterpret_cast<TileRec *>(sm + C::kOffRingRec), *rec = reinterpret_cast<TileRec *>(sm + C::kOffRec);
    RowInfo *rinfo = reinterpret_cast<RowInfo *>(sm + C::kOffRow);
    float *qscale = reinterpret_cast<float *>(sm + C::kOffQs);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
    uint64_t *k_full = bar, *k_empty = k_full + NK, *v_full = k_empty + NK, *v_empty = v_full + NV;
    uint64_t *row_full = v_empty + NV, *row_empty = row_full + kRing, *rec_full = row_empty + kRing, *rec_empty = rec_full + kInfo;
    uint64_t *ri_full = rec_empty + kInfo, *ri_empty = ri_full + kRows, *s_full = ri_empty + kRows, *p_full = s_full + SB;
    uint64_t *p_empty = p_full + SB, *o_full = p_empty + kPB, *o_empty = o_full + 2, *q_full = o_empty + 2, *q_empty = q_full + 2;
    uint64_t *drain = q_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + C::kNumBar);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *merge_row = reinterpret_cast<int *>(tmem_slot + 2);

    const AttnQ8Args &A = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = A.B * A.T;
    const int rank = P.G > 1 ? (int)cluster_rank() : 0, unit = P.G > 1 ? (int)blockIdx.x / P.G : (int)blockIdx.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 32 * kGW);   // one cp.async arrival per K-side thread
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 32 * kGW);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&row_full[i], 1);
            mbar_init(&row_empty[i], 2 * kGW);
        }
        for (int i = 0; i < kInfo; ++i) {
            mbar_init(&rec_full[i], 33);       // the record, and the scale copies of 32 lanes
            mbar_init(&rec_empty[i], 1);
        }
        for (int i = 0; i < kRows; ++i) {
            mbar_init(&ri_full[i], 1);
            mbar_init(&ri_empty[i], 1);
        }
        for (int i = 0; i < SB; ++i) {
            mbar_init(&s_full[i], 2);          // the products' commit, and the issuer itself
            mbar_init(&p_full[i], C::kSoft);
        }
        for (int i = 0; i < kPB; ++i) mbar_init(&p_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], C::kSoft);
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&drain[i], 1);
        }
        *abort_flag = 0;
        *merge_row = -1;
        fence_mbar_init();
    }
    // both Q buffers start as zeros: heads >= Hq stay zero
    for (int i = threadIdx.x; i < 2 * C::kQ / 16; i += C::kThreads)
        reinterpret_cast<uint4 *>(sm + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < 2 * HQP; i += C::kThreads) {
        epi_m[i] = kLowest;   // a cluster's CTA without tiles
        epi_l[i] = 0.f;
    }
    fence_async_smem();
    if (warp == C::kWarpS) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;   // S buffers of N2 columns, then two O buffers

    if (warp == C::kWarpScan) {
        // ------------------------------------------------------------ rows and their Q
        bool ok = true;
        int j = 0;   // rows handed over
        for (int u = unit; u < R && ok; u += P.n_units) {
            const int r = R - 1 - u;
            const int nv = __ldg(A.n_valid + r);
            int p = nv - 1;
            if (nv < 0 || nv > A.S_max) {
                if (lane == 0 && rank == 0) report(A.dev_status, SA_DEV_INDEX);
                p = -1;
            }
            const int lim = p - A.W;   // top-K entries <= lim are taken; the window covers the rest
            const int32_t *trow = A.topk + (int64_t)r * A.K;
            int first_out = A.K;
            bool bad_idx = false, bad_ord = false;
            if (p >= 0) {
                int prev_last = -1;   // the entry in front of the batch
                auto check = [&](int k, int e, int before) {
                    if (e > p) bad_idx = true;
                    if (e >= 0 && k > 0 && !(before >= 0 && before < e)) bad_ord = true;
                    if (!(e >= 0 && e <= lim)) first_out = min(first_out, k);
                };
                if ((A.K & 3) == 0 && (reinterpret_cast<uintptr_t>(A.topk) & 15u) == 0) {
                    for (int base = 0; base < A.K; base += 128 * 8) {
                        int4 e[8];
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const int k = base + 128 * v + 4 * lane;
                            e[v] = k < A.K ? __ldg(reinterpret_cast<const int4 *>(trow + k)) : make_int4(-1, -1, -1, -1);
                        }
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const int k = base + 128 * v + 4 * lane;
                            int before = __shfl_up_sync(0xffffffffu, e[v].w, 1);
                            if (lane == 0) before = prev_last;
                            prev_last = __shfl_sync(0xffffffffu, e[v].w, 31);
                            if (k < A.K) {
                                check(k, e[v].x, before);
                                check(k + 1, e[v].y, e[v].x);
                                check(k + 2, e[v].z, e[v].y);
                                check(k + 3, e[v].w, e[v].z);
                            }
                        }
                    }
                } else {
                    for (int base = 0; base < A.K; base += 32 * 8) {
                        int e[8];
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const int k = base + 32 * v + lane;
                            e[v] = k < A.K ? __ldg(trow + k) : -1;
                        }
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const int k = base + 32 * v + lane;
                            int before = __shfl_up_sync(0xffffffffu, e[v], 1);
                            if (lane == 0) before = prev_last;
                            prev_last = __shfl_sync(0xffffffffu, e[v], 31);
                            if (k < A.K) check(k, e[v], before);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, bad_idx) && lane == 0 && rank == 0) report(A.dev_status, SA_DEV_INDEX);
                if (__any_sync(0xffffffffu, bad_ord) && lane == 0 && rank == 0) report(A.dev_status, SA_DEV_ORDER);
            }
            const int n_top = p >= 0 ? (int)__reduce_min_sync(0xffffffffu, (unsigned)first_out) : 0;
            const int w0 = max(0, p - A.W + 1);
            const int n_keys = p >= 0 ? n_top + (p - w0 + 1) : 0;
            if (n_keys == 0) {   // no keys: out 0, lse -infinity
                if (rank == 0) {
                    uint4 *o = reinterpret_cast<uint4 *>(A.out + (int64_t)r * A.Hq * D);
                    for (int i = lane; i < A.Hq * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
                    if (A.lse)
                        for (int i = lane; i < A.Hq; i += 32) A.lse[(int64_t)r * A.Hq + i] = -CUDART_INF_F;
                }
                continue;
            }
            if (P.G > 1 && lane == 0) *merge_row = r;
            const int n_tiles = (n_keys + kTile - 1) / kTile;
            const int i0 = (int)((int64_t)n_tiles * rank / P.G), i1 = (int)((int64_t)n_tiles * (rank + 1) / P.G);
            if (i0 == i1) continue;   // (a cluster's CTA without a share of the row)
            ok = __all_sync(0xffffffffu, gwait(&ri_empty[j % kRows], ((uint32_t)(j / kRows) & 1u) ^ 1u, abort_flag));
            if (!ok) break;
            if (lane == 0) {
                RowInfo f;
                f.end = 0; f.r = r; f.b = r / A.T; f.n_top = n_top; f.n_keys = n_keys; f.w0 = w0; f.i0 = i0; f.i1 = i1;
                rinfo[j % kRows] = f;
                mbar_arrive(&ri_full[j % kRows]);
            }
            // Q of the row: largest finite value, then both parts of q 2^-e, 16 dims a lane
            const uint16_t *qrow = A.q + (int64_t)r * A.Hq * D;
            uint32_t mx = 0;
#pragma unroll 4
            for (int i = lane; i < A.Hq * D / 8; i += 32) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(qrow) + i);
                const uint32_t u4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t t = u4[k] & 0x7FFF7FFFu;
                    mx = __vmaxu2(mx, t & __vcmpltu2(t, 0x7F807F80u));
                }
            }
            mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
            // the largest value's power of two, so that it lies in (224, 448]; at least 2^-120
            const float amax = __uint_as_float(mx << 16);
            int ex;
            const float mant = frexpf(amax, &ex);
            const int e2 = amax > 0.f ? max(-120, mant <= 0.875f ? ex - 9 : ex - 8) : 0;
            const float down = __int_as_float((127 - e2) << 23), upw = __int_as_float((e2 + 127) << 23);
            if (j >= 2)   // Q buffer j % 2, once the S products of row j - 2 are done
                ok = __all_sync(0xffffffffu, gwait(&q_empty[j & 1], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag));
            if (!ok) break;
            if (lane == 0) qscale[j & 7] = upw;
            uint8_t *sq = sm + C::kOffQ + (j & 1) * C::kQ;
#pragma unroll 2
            for (int i = lane; i < A.Hq * (D / 16); i += 32) {
                const int h = i / (D / 16), ch = i % (D / 16);
                const uint4 *src = reinterpret_cast<const uint4 *>(qrow) + 2 * i;
                const uint4 w0q = __ldg(src), w1q = __ldg(src + 1);
                const uint32_t w[8] = {w0q.x, w0q.y, w0q.z, w0q.w, w1q.x, w1q.y, w1q.z, w1q.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t hh[2], ll[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float x = __uint_as_float(w[2 * k + s] << 16) * down;
                        float y = __uint_as_float(w[2 * k + s] & 0xFFFF0000u) * down;
                        // an infinite q makes NaN scores, as the formula does
                        if (!(fabsf(x) <= 448.f)) x = CUDART_NAN_F;
                        if (!(fabsf(y) <= 448.f)) y = CUDART_NAN_F;
                        hh[s] = e4m3x2(x, y);
                        const float2 b = from_e4m3x2(hh[s]);
                        ll[s] = e4m3x2(x - b.x, y - b.y);
                    }
                    hi[k] = hh[0] | hh[1] << 16;
                    lo[k] = ll[0] | ll[1] << 16;
                }
                *reinterpret_cast<uint4 *>(sq + sw<D>(h, ch)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(sq + sw<D>(HQP + h, ch)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[j & 1]);
            ++j;
        }
        if (ok) {
            ok = __all_sync(0xffffffffu, gwait(&ri_empty[j % kRows], ((uint32_t)(j / kRows) & 1u) ^ 1u, abort_flag));
            if (ok && lane == 0) {
                rinfo[j % kRows].end = 1;
                mbar_arrive(&ri_full[j % kRows]);
            }
        }
        __syncwarp();
    } else if (warp == C::kWarpBuild) {
        // ------------------------------------------------------------ index builder
        int g = 0;
        bool ok = true;
        for (int j = 0; ok; ++j) {
            ok = __all_sync(0xffffffffu, gwait(&ri_full[j % kRows], (uint32_t)(j / kRows) & 1u, abort_flag));
            if (!ok) break;
            const RowInfo f = rinfo[j % kRows];
            __syncwarp();
            if (lane == 0) mbar_arrive(&ri_empty[j % kRows]);
            if (f.end) break;
            const int32_t *trow = A.topk + (int64_t)f.r * A.K;
            const int32_t *pt = A.page_table ? A.page_table + (int64_t)f.b * A.max_pages : nullptr;
            // positions (-1: none) and pages of a tile's keys, lane + 32 u
            auto positions = [&](int i, int (&pos)[4]) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int kk = i * kTile + u * 32 + lane;
                    pos[u] = kk < f.n_top ? __ldg(trow + kk) : (kk < f.n_keys ? f.w0 + (kk - f.n_top) : -1);
                }
            };
            auto pages = [&](const int (&pos)[4], int (&page)[4]) {
#pragma unroll
                for (int u = 0; u < 4; ++u) page[u] = pos[u] >= 0 && pt ? __ldg(pt + (pos[u] >> 6)) : 0;
            };
            int pos0[4], pos1[4], pg0[4];
            positions(f.i0, pos0);
            pages(pos0, pg0);
            if (f.i0 + 1 < f.i1) positions(f.i0 + 1, pos1);
            for (int i = f.i0; i < f.i1; ++i, ++g) {
                int pg1[4], pos2[4];
                if (i + 1 < f.i1) pages(pos1, pg1);
                if (i + 2 < f.i1) positions(i + 2, pos2);
                const int slot = g % kRing, rs = g % kInfo;
                bool w = gwait(&row_empty[slot], ((uint32_t)(g / kRing) & 1u) ^ 1u, abort_flag);
                if (w && g >= kInfo) w = gwait(&rec_empty[rs], ((uint32_t)(g / kInfo) & 1u) ^ 1u, abort_flag);
                ok = __all_sync(0xffffffffu, w);
                if (!ok) break;
                uint32_t vm[4];
                bool bad = false;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    int row = -1;
                    if (pos0[u] >= 0) {
                        if (pt) {
                            if (pg0[u] < 0 || pg0[u] >= A.pool_pages) bad = true;
                            else row = pg0[u] * 64 + (pos0[u] & 63);
                        } else {
                            row = f.b * A.S_max + pos0[u];
                        }
                    }
                    vm[u] = __ballot_sync(0xffffffffu, row >= 0);
                    // in the order the gather lanes read them: key kt of the tile belongs to
                    // gather warp kt / kGKeys, whose lane group `sub` takes every RPI-th key
                    constexpr int RPI = 512 / D, NIT = kGKeys / RPI;   // rows a warp copies at once, turns
                    const int kt = u * 32 + lane, kw = kt % kGKeys;
                    rows[slot * kTile + (kt / kGKeys) * kGKeys + (kw % RPI) * NIT + kw / RPI] = row;
                    if (row >= 0) {
                        float *sc = scales + rs * 2 * kTile + kt;
                        cp_async4(sc, A.k_scale + (row >> P.sb_shift));
                        cp_async4(sc + kTile, A.v_scale + (row >> P.sb_shift));
                    }
                }
                if (__any_sync(0xffffffffu, bad) && lane == 0) report(A.dev_status, SA_DEV_INDEX);
                cp_async_arrive_noinc(&rec_full[rs]);
                if (lane == 0) {
                    TileRec h;
                    h.end = 0; h.r = f.r; h.j = j; h.first = i == f.i0; h.last = i == f.i1 - 1;
                    h.full = (vm[0] & vm[1] & vm[2] & vm[3]) == 0xFFFFFFFFu;
#pragma unroll
                    for (int u = 0; u < 4; ++u) h.vmask[u] = vm[u];
                    rrec[slot] = h;
                    rec[rs] = h;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&row_full[slot]);
                    mbar_arrive(&rec_full[rs]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    pos0[u] = pos1[u]; pos1[u] = pos2[u]; pg0[u] = pg1[u];
                }
            }
        }
        if (ok) {   // end marker
            const int slot = g % kRing, rs = g % kInfo;
            bool w = gwait(&row_empty[slot], ((uint32_t)(g / kRing) & 1u) ^ 1u, abort_flag);
            if (w && g >= kInfo) w = gwait(&rec_empty[rs], ((uint32_t)(g / kInfo) & 1u) ^ 1u, abort_flag);
            if (__all_sync(0xffffffffu, w)) {
                cp_async_arrive_noinc(&rec_full[rs]);
                if (lane == 0) {
                    TileRec h = {};
                    h.end = 1;
                    rrec[slot] = h;
                    rec[rs] = h;
                    mbar_arrive(&row_full[slot]);
                    mbar_arrive(&rec_full[rs]);
                }
            }
        }
        cp_async_wait_all();
        __syncwarp();
    } else if (warp < kWarpSmx) {
        // ------------------------------------------------------------ gather
        // The first kGW warps copy K rows, the next kGW copy V rows, each side on
        // its own ring: K(g) waits only for S(g - NK), V(g) only for P V(g - NV).
        constexpr int LPR = D / 16, RPI = 32 / LPR, NIT = kGKeys / RPI;   // lanes a row, rows a turn, turns
        const bool kside = warp < kGW;
        const int pw = warp % kGW, sub = lane / LPR, ch = lane % LPR;
        const uint8_t *base = (kside ? A.k : A.v) + ch * 16;
        bool ok = true;
        for (int g = 0; ok; ++g) {
            const int slot = g % kRing;
            ok = gwait(&row_full[slot], (uint32_t)(g / kRing) & 1u, abort_flag);
            if (!ok) break;
            const int end = rrec[slot].end, full = rrec[slot].full;
            if (!end) {
                ok = kside ? gwait(&k_empty[g % NK], ((uint32_t)(g / NK) & 1u) ^ 1u, abort_flag)
                           : gwait(&v_empty[g % NV], ((uint32_t)(g / NV) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                uint8_t *dst = sm + (kside ? C::kOffK + (g % NK) * C::kKV : C::kOffV + (g % NV) * C::kKV);
                const int4 *rr = reinterpret_cast<const int4 *>(rows + slot * kTile + pw * kGKeys + sub * NIT);
                int ro[NIT];
#pragma unroll
                for (int q = 0; q < NIT / 4; ++q) {
                    const int4 o = rr[q];
                    ro[4 * q] = o.x; ro[4 * q + 1] = o.y; ro[4 * q + 2] = o.z; ro[4 * q + 3] = o.w;
                }
                if (full) {
#pragma unroll
                    for (int it = 0; it < NIT; ++it)
                        cp_async16(dst + sw<D>(pw * kGKeys + RPI * it + sub, ch), base + (int64_t)ro[it] * D);
                } else {
#pragma unroll
                    for (int it = 0; it < NIT; ++it)
                        cp_async16_or_zero(dst + sw<D>(pw * kGKeys + RPI * it + sub, ch), base + (int64_t)max(ro[it], 0) * D,
                                           ro[it] >= 0);
                }
                cp_async_arrive_noinc(kside ? &k_full[g % NK] : &v_full[g % NV]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&row_empty[slot]);
            if (end) break;
        }
        cp_async_wait_all();
    } else if (warp == C::kWarpS) {
        // ------------------------------------------------------------ S issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(128, N2);
            const uint64_t k_d = smem_desc(smem_u32(sm + C::kOffK), 8 * D, D == 128 ? 2 : 4);
            const uint64_t q_d = smem_desc(smem_u32(sm + C::kOffQ), 8 * D, D == 128 ? 2 : 4);
            for (int g = 0;; ++g) {
                bool ok = iwait(&rec_full[g % kInfo], (uint32_t)(g / kInfo) & 1u, abort_flag);
                if (!ok) break;
                struct { int end, j, first, last; } h = {rec[g % kInfo].end, rec[g % kInfo].j, rec[g % kInfo].first, rec[g % kInfo].last};
                if (h.end) break;
                ok = iwait(&k_full[g % NK], (uint32_t)(g / NK) & 1u, abort_flag);
                if (ok && h.first) ok = iwait(&q_full[h.j & 1], (uint32_t)(h.j >> 1) & 1u, abort_flag);
                if (ok && g >= SB)   // S buffer g % SB, read by the softmax of tile g - SB
                    ok = iwait(&p_full[g % SB], ((uint32_t)(g / SB) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                fence_async_smem();
                tc_fence_after();
                const uint32_t dt = tmem + (uint32_t)((g % SB) * N2);
                const uint64_t kd = k_d + (uint64_t)(((g % NK) * C::kKV) >> 4);
                const uint64_t qd = q_d + (uint64_t)(((h.j & 1) * C::kQ) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    tc_mma_f8(dt, kd + (uint64_t)((kk * 32) >> 4), qd + (uint64_t)((kk * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
                tc_commit(&s_full[g % SB]);
                mbar_arrive(&s_full[g % SB]);   // passes on what this thread has seen: scales and Q's
                tc_commit(&k_empty[g % NK]);
                if (h.last) tc_commit(&q_empty[h.j & 1]);
            }
            tc_commit(&drain[0]);
            volatile int no_abort = 0;
            iwait(&drain[0], 0, &no_abort);
        }
        __syncwarp();
    } else if (warp == C::kWarpPV) {
        // ------------------------------------------------------------ P V issuer
        if (lane == 0) {
            // A (V^T) and B (P^T) both MN-major
            constexpr uint32_t idesc = idesc_e4m3_f32(128, N2) | (1u << 15) | (1u << 16);
            const uint64_t v_d = desc_v<D>(smem_u32(sm + C::kOffV));
            const uint64_t p_d = desc_mn_plain(smem_u32(sm + C::kOffP), N2 * 8, 128);
            for (int g = 0;; ++g) {
                bool ok = iwait(&rec_full[g % kInfo], (uint32_t)(g / kInfo) & 1u, abort_flag);
                if (!ok) break;
                struct { int end, j, first, last; } h = {rec[g % kInfo].end, rec[g % kInfo].j, rec[g % kInfo].first, rec[g % kInfo].last};
                if (h.end) break;
                ok = iwait(&p_full[g % SB], (uint32_t)(g / SB) & 1u, abort_flag);
                if (!ok) break;
                mbar_arrive(&rec_empty[g % kInfo]);   // every reader of the record and the scales is done with them
                ok = iwait(&v_full[g % NV], (uint32_t)(g / NV) & 1u, abort_flag);
                if (ok && h.first && h.j >= 2)   // O buffer read by the epilogue of row j - 2
                    ok = iwait(&o_empty[h.j & 1], ((uint32_t)(h.j >> 1) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                fence_async_smem();
                tc_fence_after();
                const uint32_t dt = tmem + (uint32_t)((SB + (h.j & 1)) * N2);
                const uint64_t vd = v_d + (uint64_t)(((g % NV) * C::kKV) >> 4);
                const uint64_t pd = p_d + (uint64_t)(((g % kPB) * C::kP) >> 4);
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)   // 32 keys: four 8-key groups
                    tc_mma_f8(dt, vd + (uint64_t)((kk * 32 * D) >> 4), pd + (uint64_t)((kk * 4 * N2 * 8) >> 4), idesc,
                              (h.first && kk == 0) ? 0u : 1u);
                tc_commit(&p_empty[g % kPB]);
                tc_commit(&v_empty[g % NV]);
                if (h.last) tc_commit(&o_full[h.j & 1]);
            }
            tc_commit(&drain[1]);
            volatile int no_abort = 0;
            iwait(&drain[1], 0, &no_abort);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        const int quad = warp & 3, hg = (warp - kWarpSmx) >> 2, h0 = hg * HG;
        const int bar_red = 2 + 2 * hg, bar_x = 3 + 2 * hg;   // this group's named barriers
        const int key = quad * 32 + lane;                     // TMEM lane: key (S^T) or head dim (O^T)
        const uint32_t lane_t = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)h0;
        float *gmax = redmax + hg * 4 * HG, *gsum = redsum + hg * 4 * HG;
        float *negm = reinterpret_cast<float *>(sm + C::kOffNegM) + (hg * 4 + quad) * HG;   // this warp's copy
        f2 l[HG / 2];
#pragma unroll
        for (int i = 0; i < HG / 2; ++i) l[i] = 0;
        if (lane < HG) negm[lane] = 0.f;
        __syncwarp();
        // both parts of this group's columns `col`.. of a TMEM buffer, added
        auto tload = [&](uint32_t col, f2 (&x)[HG / 2]) {
#pragma unroll
            for (int c = 0; c < HG; c += 8) {
                uint32_t u[8], v[8];
                tmem_ld_x8(lane_t + col + (uint32_t)c, u);
                tmem_ld_x8(lane_t + col + (uint32_t)(HQP + c), v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[c / 2 + e] = add2(pku(u[2 * e], u[2 * e + 1]), pku(v[2 * e], v[2 * e + 1]));
            }
        };
        int pend_j = -1, pend_r = 0, pend_g = 0;
        // The epilogue of a row runs kPB tiles after its last one, when that tile's
        // P V is known to be done, or at the next row's last tile, or at the end.
        auto epilogue = [&]() -> bool {
            if (pend_j < 0) return true;
            const int jb = pend_j & 1;
            if (!bar_and(bar_red, 128, gwait(&o_full[jb], (uint32_t)(pend_j >> 1) & 1u, abort_flag))) return false;
            tc_fence_after();
            f2 o[HG / 2];
            tload((uint32_t)((SB + jb) * N2), o);
            if (P.G > 1) {
                // a part of the row: unnormalised, for the merge (the K ring is idle by now)
                float *part = reinterpret_cast<float *>(sm + C::kOffK);
                if (D == 128 || key < D) {
#pragma unroll
                    for (int i = 0; i < HG / 2; ++i) {
                        const float2 v = up(o[i]);
                        part[(h0 + 2 * i) * D + key] = v.x;
                        part[(h0 + 2 * i + 1) * D + key] = v.y;
                    }
                }
            } else {
                if (D == 128 || key < D) {
                    uint16_t *orow = A.out + (int64_t)pend_r * A.Hq * D;
#pragma unroll
                    for (int i = 0; i < HG / 2; ++i) {
                        const float2 v = up(o[i]);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int h = h0 + 2 * i + s;
                            if (h < A.Hq) {
                                const float L = epi_l[jb * HQP + h];
                                const __nv_bfloat16 ob = __float2bfloat16_rn((s ? v.y : v.x) * (L == 0.f ? 0.f : 1.f / L));
                                orow[(int64_t)h * D + key] = *reinterpret_cast<const uint16_t *>(&ob);
                            }
                        }
                    }
                }
                if (A.lse && quad == 0 && lane < HG && h0 + lane < A.Hq) {
                    const float L = epi_l[jb * HQP + h0 + lane];
                    A.lse[(int64_t)pend_r * A.Hq + h0 + lane] =
                        L == 0.f ? -CUDART_INF_F : (epi_m[jb * HQP + h0 + lane] + log2f(L)) * 0.69314718055994531f;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[jb]);
            pend_j = -1;
            return true;
        };
        bool ok = true;
        for (int g = 0; ok; ++g) {
            const int sb = g % SB, pb = g % kPB, rs = g % kInfo;
            bool w = gwait(&rec_full[rs], (uint32_t)(g / kInfo) & 1u, abort_flag);
            struct { int end, r, j, first, last; uint32_t vmask; } h = {};
            if (w) {
                h.end = rec[rs].end; h.r = rec[rs].r; h.j = rec[rs].j; h.first = rec[rs].first; h.last = rec[rs].last;
                h.vmask = rec[rs].vmask[quad];
                if (!h.end) w = gwait(&s_full[sb], (uint32_t)(g / SB) & 1u, abort_flag);
                if (!h.end && w && g >= kPB) w = gwait(&p_empty[pb], ((uint32_t)(g / kPB) & 1u) ^ 1u, abort_flag);
            }
            // One vote per tile decides the common case: nobody stopped and no head
            // needs a new maximum.  (After a failed wait the S read below returns
            // whatever TMEM holds; the vote discards it.)
            const bool stop = !w || h.end;
            tc_fence_after();
            f2 x[HG / 2];
            tload((uint32_t)(sb * N2), x);
            // this lane's key: score factor, log2 of the value scale and its reciprocal
            const bool some = (h.vmask >> lane) & 1u;
            float c1 = 0.f, lv = -CUDART_INF_F, iv = 0.f;
            if (some) {
                const float vs = clamp_scale(scales[rs * 2 * kTile + kTile + key]);
                c1 = clamp_scale(scales[rs * 2 * kTile + key]) * qscale[h.j & 7] * P.scale_log2;
                lv = __log2f(vs);
                iv = __frcp_rn(vs);
            }
            const f2 c2 = pk(c1, c1), lv2 = pk(lv, lv), iv2 = pk(iv, iv);
            const f2 *nm = reinterpret_cast<const f2 *>(negm);
            f2 e[HG / 2];
            float emax = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < HG / 2; ++i) {
                e[i] = fma2(x[i], c2, add2(lv2, nm[i]));
                const float2 v = up(e[i]);
                emax = fmaxf(emax, fmaxf(v.x, v.y));
            }
            bool need = h.first || emax > kRaise;
            if (!bar_or(bar_red, 128, need || stop)) {
                need = false;
            } else if (bar_or(bar_red, 128, stop)) {
                ok = bar_and(bar_red, 128, w);   // every wait succeeded: the end marker for all
                if (ok) ok = epilogue();
                break;
            } else {
                need = true;
            }
            if (need) {
                // exact tile maximum of every head over the 128 key lanes
#pragma unroll
                for (int i = 0; i < HG / 2; ++i) {
                    const float2 v = up(fma2(x[i], c2, lv2));
                    const float a = redux_max(v.x), b = redux_max(v.y);
                    if (lane == 0) *reinterpret_cast<float2 *>(gmax + quad * HG + 2 * i) = make_float2(a, b);
                }
                bar_sync_n(bar_x, 128);
                // the new maxima, one head a lane (every warp for its own copy)
                float f = 1.f, nm_new = 0.f;
                if (lane < HG) {
                    const float tm = fmaxf(fmaxf(gmax[lane], gmax[HG + lane]), fmaxf(gmax[2 * HG + lane], gmax[3 * HG + lane]));
                    const float old = -negm[lane];
                    nm_new = old;
                    if (h.first) {
                        nm_new = fmaxf(tm - kTop, kLowest);
                    } else if (tm > old + kRaise) {
                        nm_new = tm - kTop;
                        f = ex2f(old - nm_new);
                    }
                }
                const bool resc = __any_sync(0xffffffffu, f != 1.f);
                __syncwarp();
                if (lane < HG) negm[lane] = -nm_new;
                __syncwarp();
                if (h.first) {
#pragma unroll
                    for (int i = 0; i < HG / 2; ++i) l[i] = 0;
                } else if (resc) {
                    // O holds the row's earlier tiles: wait for P V of tile g - 1
                    ok = bar_and(bar_red, 128, gwait(&p_empty[(g - 1) % kPB], (uint32_t)((g - 1) / kPB) & 1u, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t ot = lane_t + (uint32_t)((SB + (h.j & 1)) * N2);
#pragma unroll
                    for (int c = 0; c < HG; c += 8) {
                        float fc[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) fc[k] = __shfl_sync(0xffffffffu, f, c + k);
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            uint32_t o[8];
                            tmem_ld_x8(ot + (uint32_t)(part * HQP + c), o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fc[k]);
                            tmem_st8(ot + (uint32_t)(part * HQP + c), o);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) l[c / 2 + k] = fma2(l[c / 2 + k], pk(fc[2 * k], fc[2 * k + 1]), 0);
                    }
                    tmem_st_wait_all();
                }
#pragma unroll
                for (int i = 0; i < HG / 2; ++i) e[i] = fma2(x[i], c2, add2(lv2, nm[i]));
            }
            // P^T as an MN-major operand without swizzle: 16-byte rows of 16 heads, the
            // rows of 8 keys 16 bytes apart, the head chunks of a key group 128 bytes
            // apart (first all high parts, then the low ones), key groups N2 * 8 bytes apart
            uint32_t hi[HG / 4], lo[HG / 4];
            const f2 minus1 = pk(-1.f, -1.f);
#pragma unroll
            for (int i = 0; i < HG / 4; ++i) {
                uint32_t ph[2], pl[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float2 v = up(e[2 * i + s]);
                    const float p0 = ex2f(v.x), p1 = ex2f(v.y);
                    const f2 p2 = pk(p0, p1);
                    l[2 * i + s] = fma2(p2, iv2, l[2 * i + s]);
                    // four significant bits, rounded to nearest; the rest exactly
                    const uint32_t a = (__float_as_uint(p0) + 0x80000u) & 0xFFF00000u;
                    const uint32_t b = (__float_as_uint(p1) + 0x80000u) & 0xFFF00000u;
                    const float2 d = up(fma2(pku(a, b), minus1, p2));
                    ph[s] = e4m3x2(__uint_as_float(a), __uint_as_float(b));
                    pl[s] = e4m3x2(d.x, d.y);
                }
                hi[i] = ph[0] | ph[1] << 16;
                lo[i] = pl[0] | pl[1] << 16;
            }
            uint8_t *pbuf = sm + C::kOffP + pb * C::kP + (key >> 3) * (N2 * 8) + (key & 7) * 16;
            uint8_t *ph = pbuf + (h0 >> 4) * 128 + (h0 & 15), *pl = pbuf + ((HQP + h0) >> 4) * 128 + (h0 & 15);
            if (HG == 16) {
                *reinterpret_cast<uint4 *>(ph) = make_uint4(hi[0], hi[1], hi[HG / 4 - 2], hi[HG / 4 - 1]);
                *reinterpret_cast<uint4 *>(pl) = make_uint4(lo[0], lo[1], lo[HG / 4 - 2], lo[HG / 4 - 1]);
            } else {
                *reinterpret_cast<uint2 *>(ph) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(pl) = make_uint2(lo[0], lo[1]);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[sb]);
            // a pending epilogue, now that this tile is handed over
            if (pend_j >= 0 && (g - pend_g >= kPB || h.last))
                if (!(ok = epilogue())) break;
            if (h.last) {
                // the row's sums over all 128 key lanes and its maxima, kept for its epilogue
#pragma unroll
                for (int i = 0; i < HG / 2; ++i) {
                    float2 v = up(l[i]);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
                        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
                    }
                    if (lane == 0) *reinterpret_cast<float2 *>(gsum + quad * HG + 2 * i) = v;
                }
                bar_sync_n(bar_x, 128);
                if (quad == 0 && lane < HG) {
                    const int jb = h.j & 1;
                    epi_l[jb * HQP + h0 + lane] = (gsum[lane] + gsum[HG + lane]) + (gsum[2 * HG + lane] + gsum[3 * HG + lane]);
                    epi_m[jb * HQP + h0 + lane] = -negm[lane];
                }
                bar_sync_n(bar_x, 128);   // epi_* written before any warp's epilogue reads them
                pend_j = h.j;
                pend_r = h.r;
                pend_g = g;
            }
        }
    }
    // Every role is past its last TMEM access and its last copy.
    tc_fence_before();
    bar_sync_n(1, C::kThreads);
    if (warp == C::kWarpS) {
        if (lane == 0 && *abort_flag) report(A.dev_status, SA_DEV_TIMEOUT);
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (P.G > 1) {
        // join the parts: this CTA takes the heads rank * hpr .., 4 dims a thread
        cluster_sync();
        const int r = *merge_row, G = P.G, hpr = (A.Hq + G - 1) / G, hb = rank * hpr, nh = max(0, min(hpr, A.Hq - hb));
        float *gm = reinterpret_cast<float *>(sm + C::kOffMerge), *gl = gm + 16 * HQP;   // [head][CTA]
        if (r >= 0) {
            for (int i = threadIdx.x; i < nh * G; i += C::kThreads) {
                const int h = i / G, c = i % G;
                gm[i] = dsmem_ld_f32(epi_m + hb + h, (uint32_t)c);
                gl[i] = dsmem_ld_f32(epi_l + hb + h, (uint32_t)c);
            }
        }
        __syncthreads();
        if (r >= 0) {
            const float *part = reinterpret_cast<const float *>(sm + C::kOffK);
            for (int i = threadIdx.x; i < nh * (D / 4); i += C::kThreads) {
                const int h = i / (D / 4), d4 = i % (D / 4);
                float m = kLowest, L = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = 0; c < G; ++c)
                    if (gl[h * G + c] != 0.f) m = fmaxf(m, gm[h * G + c]);
#pragma unroll 4
                for (int c = 0; c < G; ++c) {
                    const float lc = gl[h * G + c];
                    if (lc == 0.f) continue;   // no share of the row
                    const float f = ex2f(gm[h * G + c] - m);
                    const float4 v = dsmem_ld_f4(part + (hb + h) * D + 4 * d4, (uint32_t)c);
                    L = fmaf(f, lc, L);
                    o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
                }
                const float s = L == 0.f ? 0.f : 1.f / L;
                uint2 b;
                b.x = pack_bf16(o.x * s, o.y * s);
                b.y = pack_bf16(o.z * s, o.w * s);
                *reinterpret_cast<uint2 *>(A.out + ((int64_t)r * A.Hq + hb + h) * D + 4 * d4) = b;
                if (A.lse && d4 == 0)
                    A.lse[(int64_t)r * A.Hq + hb + h] = L == 0.f ? -CUDART_INF_F : (m + log2f(L)) * 0.69314718055994531f;
            }
        }
        cluster_sync();   // nobody leaves while its parts are read
    }
}

template <int D, int HQP>
sa_status launch_q8(const AttnQ8Args &a, cudaStream_t st) {
    using C = Cfg<D, HQP>;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SA_ERR_CUDA;
    Params p;
    p.a = a;
    const int R = a.B * a.T;
    const int tiles = (int)std::min<int64_t>(((int64_t)a.K + a.W + kTile - 1) / kTile, ((int64_t)a.S_max + kTile - 1) / kTile);
    p.G = std::max(1, std::min({16, tiles, sms / R}));
    p.n_units = p.G > 1 ? R : std::min(R, sms);
    p.sb_shift = 0;
    while ((1 << p.sb_shift) < a.scale_block) ++p.sb_shift;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    if (prepare_kernel<attn_q8_kernel<D, HQP>>(C::kSmem, p.G > 8) != cudaSuccess) return SA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_units * p.G));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)p.G;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = p.G > 1 ? 1 : 0;
    return cuda_ok(cudaLaunchKernelEx(&cfg, attn_q8_kernel<D, HQP>, p));
}

template <int D>
sa_status launch_q8_heads(const AttnQ8Args &a, cudaStream_t st) {
    if (a.Hq <= 16) return launch_q8<D, 16>(a, st);
    if (a.Hq <= 32) return launch_q8<D, 32>(a, st);
    return launch_q8<D, 64>(a, st);
}

}  // namespace

sa_status launch_attn_q8(const AttnQ8Args &a, cudaStream_t st) {
    return a.d == 128 ? launch_q8_heads<128>(a, st) : launch_q8_heads<64>(a, st);
}

}  // namespace sa
