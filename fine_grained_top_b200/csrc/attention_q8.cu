// attention_q8.cu -- exact softmax attention over the selected keys of an
// 8-bit cache with a scale for each block of tokens (one new token or a chunk
// of tokens a sequence, contiguous or paged).
//
//   S(r) = {s in TopK(r) : s <= p - W}  U  {max(0, p-W+1) .. p}
//   x_s = (q[r,h] . kc[s]) ks[s] scale,   O[r,h] = sum_s softmax(x)_s vs[s] vc[s]
//
// Two products on the tensor cores, each with fp32 sums:
//   S^T = K Q^T        M = 128 keys, N = heads, K = d            -> TMEM
//   P^T                softmax over keys, one thread per key lane
//   O^T += V^T P^T     M = d, N = heads, K = 128 keys            -> TMEM
// S takes the codes as they lie in the cache (tcgen05 kind::f8f6f4, e4m3 x e4m3
// products are exact) and q split into two e4m3 parts: q 2^-e = q_hi + q_lo (exact for
// a bf16 q down to 2^-10 of the row's largest value, below it off by 2^-18 of that).  If
// heads lie more than 2^6 apart each has its own e, and its scores are brought to the row's
// in TMEM before they are read (a row of such heads takes longer, the others 1 to 4 percent
// for the question).
// P V is a product of fp16 (kind::f16): V's codes are widened on the way (exactly), and
// P is rounded once.  P has to keep its precision over many orders of magnitude: a key
// that takes most of the weight with next to no value of its own (an attention sink)
// leaves the output to keys 2^-10 to 2^-20 of it.  (Two e4m3 parts of P, which let V go in
// as it is, end at 2^-14: such a head's output was off by up to its whole size.)
// The scales stay out of the products: in S^T a key is a lane, so ks and vs are one
// number per thread: with
//   e = (S_hi + S_lo) ks 2^e scale log2e + log2 vs - m,    P = 2^e
// the running maximum m is of the contributions p vs (so P fills fp16's range whatever
// the scales), and the row sum takes P / vs.  P's largest is 2^8 after the first tile; it
// may grow to 2^15.75 (fp16 ends at 2^16) before m goes up, by 2^8: so a head's largest is
// always at least 2^7.75, and a P is off by 2^-11 of its value and, where fp16 runs out of
// exponents, by 2^-25, which is 2^-32 of that largest.
//
// A CTA takes one row, or (few rows: the cost rule in launch_q8_rows) one run of
// a row's tiles: a thread-block cluster shares the row, and the partial m, l, O
// meet through distributed shared memory.  A tile is 128 keys.  The warps:
//   4 loader warps   one key a thread looked up ahead (selection entry four tiles
//                    ahead, page three, scales two).  V's codes are loaded into registers a
//                    tile ahead and widened into the V tile as soon as P V(t-1) lets go of
//                    it; K(t+2) is copied with 16-byte cp.async as soon as S(t+1) lets go of
//                    the single K tile (a slot without a key is zero-filled: nothing that
//                    was not selected is ever read).  Both fly while P V(t) runs
//   4 or 8 softmax   one key a lane, 16 heads a thread with up to 16 heads, else 32
//     warps          (two groups with 64): a vote on raises, the exponentials, P^T
//                    into the single P tile.  32 heads keep their sums in registers
//                    and read the scores from TMEM twice; 64 a thread spill, and 16
//                    with four groups read each key's factors twice as often
//   1 MMA warp       issues P V(t), then S(t+2) (two S buffers), is the only one that
//                    polls their mbarriers, and passes each end on over a named
//                    barrier: polling warps take issue slots from the softmax
// and one barrier of the CTA a tile hands P(t), V(t) and the next factors over.
// Two (from 17 heads) or three CTAs share an SM and fill each other's waits.  (A
// persistent CTA of 16 to 24 warps in roles, a row after another, spent its time on
// instruction-cache misses and single-warp latencies: three times as long for 2048 rows.)
//
// What bounds it.  Few rows: the launch and the chain row start -> lookups -> gather ->
// S -> P -> P V -> join, of code that each CTA runs once: one row of 1152 keys 6.4 us, 8
// rows of 2560 keys and 64 heads 11.0, 16 such paged rows 15.3.  Alone on an SM a CTA's
// tile takes 1.0 (16 heads) to 1.4 us (64): P V, V's widening, the barrier, P V; while its
// MMAs run neither the lookups nor reads of the scores get on, hence the order in the MMA
// warp.  Many rows: that same chain, two or three CTAs an SM deep, as many as V in fp16
// leaves room for.  2048 rows of 1152 keys and 16 heads 104 us, of which the rows' starts and
// ends are 23 (issue slots 56 percent); 4 x 1024 padded rows of up to 2560 keys and 64
// heads 389 us (397 TFLOP/s), bound to 72 registers a thread.  V's codes in a stage of
// their own in shared memory instead of registers took 6 and 0 percent longer, with both
// copies before the barrier of the tile 7 and 4.  Every wait is bounded (SA_DEV_TIMEOUT).
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "cache_ops.h"
#include "ptx.cuh"

namespace sa {

namespace {

constexpr int kTile = 128;                  // keys per tile (MMA M)
constexpr float kTop = 8.f, kRaise = 15.75f; // log2 of a row's largest P at first, and of what it may grow to
constexpr float kStep = 8.f;                // how far a head's reference goes up then
constexpr float kSmallV = -30.f;            // log2 of the value scales from which P may vanish before the weight does
constexpr float kLowest = -3.4028235e38f;   // running maximum of a head that has met no finite score yet
constexpr float kCoarse = 8388608.f;        // a reference from 2^23 on is not moved by steps
constexpr int kSmemSm = 233472;             // shared memory of an SM, 1 KB of it reserved per CTA

struct Params {
    AttnQ8Args a;
    int G;                // CTAs a row (cluster size)
    uint32_t inv_G;       // ceil(2^20 / G): n / G is n inv_G >> 20 for n <= 2^16 + 2^6
    int hpr;              // heads that a CTA of a cluster joins
    int sb_shift;         // log2 of the tokens a scale
    float scale_log2;
    unsigned long long limit_ns;   // health check: of every wait
    int lost;                      // health check: S (even) or P V (odd) of this half of a tile of row 0 never comes
};

template <int D_, int HQP_>
struct Cfg {
    static constexpr int D = D_, HQP = HQP_;
    static constexpr int N2 = 2 * HQP;                    // MMA N: hi and lo columns
    static constexpr int HG = HQP == 16 ? 16 : 32;        // heads a softmax thread handles
    static constexpr int NG = HQP / HG;                   // softmax groups of 128 threads
    static constexpr int kThreads = 128 + 128 * NG + 32;  // loader warps, softmax warps, the MMA warp
    static constexpr int kWarpMma = 4 + 4 * NG;
    static constexpr int kKV = kTile * D, kQ = N2 * D, kP = kTile * HQP * 2;
    static constexpr int kOffK = 0;
    // Q's parts: one after the other into the same columns of S, or with 16 heads side
    // by side (half the MMAs, which are all of the least size, for one more addition)
    static constexpr bool kSide = HQP == 16;
    static constexpr int SN = kSide ? N2 : HQP;           // columns of an S buffer
    static constexpr int kOffV = kOffK + kKV;            // V in fp16: halves of 64 dims, 128 bytes a key
    static constexpr int kOffQ = kOffV + 2 * kKV;
    static constexpr int kOffP = kOffQ + kQ;
    static constexpr int kOffSc = kOffP + kP;                         // [2][2][128] score factor, log2 vs
    static constexpr int kOffMax = kOffSc + 2 * 2 * kTile * 4;           // [4][HQP] maxima or sums of the quads
    static constexpr int kOffNegM = kOffMax + 4 * HQP * 4;            // [softmax warp][HG] minus the running maxima
    static constexpr int kOffEpi = kOffNegM + 4 * HQP * 4;            // a part's m and l [HQP][2]
    static constexpr int kOffFlags = kOffEpi + 2 * HQP * 4;  // [group][4] heads to raise, by eights
    static constexpr int kOffQs = kOffFlags + NG * 16;                // [HQP] the heads' factors
    static constexpr int kOffMisc = kOffQs + HQP * 4;
    static constexpr int kUsed = kOffMisc + 64 + 16 * 16;
    static constexpr uint32_t kTmemCols = 2 * SN + HQP <= 64 ? 64 : (2 * SN + HQP <= 128 ? 128 : 256);   // two S buffers, O
    // CTAs wait for TMEM columns while others of their cluster wait for them, so
    // whatever shares an SM must fit its 512 columns: shared memory in proportion.
    static constexpr int kLeast = (int)(kTmemCols * (kSmemSm / 512)) - 1024;
    static constexpr int kSmem = kUsed > kLeast ? kUsed : kLeast;
    // CTAs an SM, by their shared memory and registers (with 64 dims and 16 heads a fourth
    // would fit, and spill: 2048 rows 80 us with three, 93 with four)
    static constexpr int kPerSm = std::min(kSmemSm / (kSmem + 1024), HQP == 16 ? 3 : 2);
    static_assert(3 * kKV >= HQP * D * 4, "O lies in the K and V tiles when a row or its part is done");
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
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Arrive at barrier `id` of `n` threads without waiting for it; wait for it; wait and return the OR of a predicate.
__device__ __forceinline__ void bar_arrive_n(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_sync_n(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int n, bool p) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred a, b; setp.ne.u32 a, %1, 0; bar.red.or.pred b, %2, %3, a; selp.u32 %0, 1, 0, b; }"
        : "=r"(r)
        : "r"((uint32_t)p), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait_all() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// MN-major operand without swizzle: 8 x 16-byte core matrices (8 K rows of 8
// MN elements, 128 contiguous bytes); K groups of 8 rows `kgroup` bytes apart,
// MN chunks of 8 elements `mnchunk` bytes apart.  (For this layout the
// descriptor's leading offset is the K-group stride and its stride offset the
// MN-chunk stride.)
__device__ __forceinline__ uint64_t desc_mn_plain(uint32_t addr, uint32_t kgroup, uint32_t mnchunk) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((kgroup >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)((mnchunk >> 4) & 0x3FFF) << 32;
    d |= (uint64_t)1 << 46;   // layout type 0 (no swizzle) in bits 61-63
    return d;
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[8]) { tmem_ld_x8(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_x16(taddr, r); }
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; .reg .b32 d; elect.sync d|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ float redux_max(float x) {   // NaN counts as absent
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void cp_async16_or_zero(void *smem_dst, const void *gsrc, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(gsrc), "r"(some ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_x2(uint32_t taddr, uint32_t (&r)[2]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
}
// Two f32 rounded to f16 (lo in the low half), and f16 pairs to and from e4m3.
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4_of_f16(uint32_t a, uint32_t b) {   // a's pair in the low half
    uint32_t r;
    asm("{ .reg .b16 x, y; cvt.rn.satfinite.e4m3x2.f16x2 x, %1; cvt.rn.satfinite.e4m3x2.f16x2 y, %2; mov.b32 %0, {x, y}; }"
        : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void f16_of_e4m3x4(uint32_t c, uint32_t &a, uint32_t &b) {
    asm("{ .reg .b16 x, y; mov.b32 {x, y}, %2; cvt.rn.f16x2.e4m3x2 %0, x; cvt.rn.f16x2.e4m3x2 %1, y; }" : "=r"(a), "=r"(b) : "r"(c));
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // NaN counts as absent
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The address of this CTA's shared memory `local` in CTA `rank` of the cluster, and loads from such.
__device__ __forceinline__ uint32_t in_cta(const void *local, uint32_t rank) {
    uint32_t remote;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    return remote;
}
__device__ __forceinline__ void dsmem_ld(uint32_t at, float (&v)[2]) {
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void dsmem_ld(uint32_t at, float (&v)[4]) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint32_t cluster_id() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
// Byte offset of 16-byte chunk `ch` of row `r` in a tile of D-byte rows with
// the D-byte swizzle (128 or 64).
template <int D>
__device__ __forceinline__ uint32_t sw(int r, int ch) {
    return (uint32_t)(r * D + ((D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4));
}
// Byte offset of 16-byte chunk `ch` (8 dims) of key `r` in the fp16 V tile: 128-byte
// swizzled rows of 64 dims, two halves of them with 128 dims.
__device__ __forceinline__ uint32_t sw_v(int r, int ch) {
    return (uint32_t)((ch >> 3) * (kTile * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}
// The MN-major operand of that tile: 8-row K groups 1024 bytes apart.  D = 64: the MMA's
// upper 64 M rows read the same 64 dims again (a stride of 0 between the MN chunks);
// their results are not used.
template <int D>
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)(((D == 128 ? kTile * 128 : 0) >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;   // 128-byte swizzle
    return d;
}
// Instruction descriptor, kind::f16 with both operands fp16 (format code 0), f32
// accumulate, both MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_mn(int M, int N) {
    return (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// CL: a cluster shares the row (the two forms are apart to keep the code, and the
// instruction cache it needs, small).
// Wait (with a limit) for every MMA that this warp has issued.  (Out of line: between the
// others it costs 3 percent of a chunk's time.)
__device__ __noinline__ void drain_mmas(uint64_t *bar) {
    if (elect_one()) tc_commit(bar);
    __syncwarp();
    int none = 0;
    mbar_wait(bar, 0, &none);
}

// CHECK: the health check's form, whose waits take their limit from the call and one of
// whose MMAs is not issued.
template <int D, int HQP, bool CL, bool CHECK = false>
__global__ void __launch_bounds__(Cfg<D, HQP>::kThreads, Cfg<D, HQP>::kPerSm) attn_q8_kernel(Params P) {
    using C = Cfg<D, HQP>;
    constexpr int NT = C::kThreads, HG = C::HG, SN = C::SN;
    extern __shared__ __align__(1024) uint8_t sm[];   // (no static shared memory: it begins 1024-byte aligned)
    float *sc = reinterpret_cast<float *>(sm + C::kOffSc);
    float2 *part_ml = reinterpret_cast<float2 *>(sm + C::kOffEpi);   // a part's m and l
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::kOffMisc);
    uint64_t *bar_s = bar, *bar_pv = bar + 2, *bar_drain = bar + 3;   // S(t) done, one for each S buffer; P V(t) done; all MMAs
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 4);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    uint4 *found = reinterpret_cast<uint4 *>(sm + C::kOffMisc + 64);   // a warp's first entry not taken, its heads' largest and least |q|

    const AttnQ8Args &A = P.a;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int G = CL ? P.G : 1, rank = CL ? (int)cluster_rank() : 0;
    const int r = CL ? (int)cluster_id() : (int)blockIdx.x, b = A.T == 1 ? r : r / A.T;
    auto by_G = [&](int n) { return CL ? (int)(((uint64_t)n * P.inv_G) >> 20) : n; };   // n / G

    // ------------------------------------------------------------ the row
    // Loads that wait for nothing go first: its length, its Q (16 dims a thread and turn),
    // the start of its top-K row (16 bytes a thread and turn), and the selection's entries
    // of this CTA's first three tiles if the top-K row is full, as most are.  The pages of
    // those follow as soon as the length is there.  (Each after the barrier that makes it
    // certain costs 4 percent.  The second turn over the top-K row pays with the longer rows
    // that go with 64 heads.)
    const int nv = __ldg(A.n_valid + r);
    const int32_t *trow = A.topk + (int64_t)r * A.K;
    const int32_t *pt = A.page_table ? A.page_table + (int64_t)b * A.max_pages : nullptr;
    const bool loader = warp < 4;
    constexpr int CPH = D / 16;   // 16-dim chunks of a head
    constexpr int NQ = (HQP * CPH + NT - 1) / NT;   // chunks a thread
    constexpr int NE = HQP == 64 ? 2 : 1, NP = 3;   // turns over the top-K row that go first, tiles looked up
    const bool vec = (A.K & 3) == 0 && (reinterpret_cast<uintptr_t>(A.topk) & 15u) == 0;
    auto entries = [&](int k) {   // k .. k + 3 of the top-K row
        int4 v = make_int4(-1, -1, -1, -1);
        if (vec) {
            if (k < A.K) v = __ldg(reinterpret_cast<const int4 *>(trow + k));
        } else {
            if (k < A.K) v.x = __ldg(trow + k);
            if (k + 1 < A.K) v.y = __ldg(trow + k + 1);
            if (k + 2 < A.K) v.z = __ldg(trow + k + 2);
            if (k + 3 < A.K) v.w = __ldg(trow + k + 3);
        }
        return v;
    };
    auto entry_before = [&](int k) { return lane == 0 && k > 0 && k <= A.K ? __ldg(trow + k - 1) : -1; };   // (others ask their neighbour)
    int4 ent[NE];
    int before[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        ent[i] = entries(4 * (tid + i * NT));
        before[i] = entry_before(4 * (tid + i * NT));
    }
    const int g0 = by_G((A.K + A.W + kTile - 1) / kTile * rank);   // this CTA's first tile, if so
    int pos_g[NP], page_g[NP];
#pragma unroll
    for (int t = 0; t < NP; ++t) {
        const int kk = (g0 + t) * kTile + tid;
        pos_g[t] = loader && kk < A.K ? __ldg(trow + kk) : -1;
    }
    uint4 qv[2 * NQ];
    uint32_t q_head[NQ] = {};   // the largest |q| of each chunk's head
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int c = tid + i * NT;
        qv[2 * i] = qv[2 * i + 1] = make_uint4(0, 0, 0, 0);
        if (c < A.Hq * CPH) {
            const uint4 *src = reinterpret_cast<const uint4 *>(A.q + (int64_t)r * A.Hq * D) + 2 * c;
            qv[2 * i] = __ldg(src);
            qv[2 * i + 1] = __ldg(src + 1);
        }
    }
    if (tid == 0) {
        mbar_init(bar_s, 1);
        mbar_init(bar_s + 1, 1);
        mbar_init(bar_pv, 1);
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    int p = nv - 1;
    if (nv < 0 || nv > A.S_max) {
        if (tid == 0 && rank == 0) report(A.dev_status, SA_DEV_INDEX);
        p = -1;
    }
    auto no_keys = [&]() {   // out 0, lse -infinity
        uint4 *o = reinterpret_cast<uint4 *>(A.out + (int64_t)r * A.Hq * D);
        for (int i = tid; i < A.Hq * D / 8; i += NT) o[i] = make_uint4(0, 0, 0, 0);
        if (A.lse)
            for (int i = tid; i < A.Hq; i += NT) A.lse[(int64_t)r * A.Hq + i] = -CUDART_INF_F;
    };
    if (p < 0 && !CL) {   // a padding row
        no_keys();
        return;
    }
    if (warp == C::kWarpMma) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    const int w0 = max(0, p - A.W + 1);
#pragma unroll
    for (int t = 0; t < NP; ++t) {
        const int kk = (g0 + t) * kTile + tid;
        if (kk >= A.K) pos_g[t] = w0 + (kk - A.K);
        page_g[t] = loader && pt && pos_g[t] >= 0 && pos_g[t] <= p ? __ldg(pt + (pos_g[t] >> 6)) : 0;
    }

    const int lim = p - A.W;   // top-K entries <= lim are taken; the window covers the rest
    if (p >= 0) {
        int first_out = A.K;
        bool bad_idx = false, bad_ord = false;
        auto check = [&](int k, const int4 &v, int first) {
            int e[5];   // entries k - 1 .. k + 3
            e[0] = __shfl_up_sync(0xffffffffu, v.w, 1);
            if (lane == 0) e[0] = first;
            e[1] = v.x; e[2] = v.y; e[3] = v.z; e[4] = v.w;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (e[u + 1] > p) bad_idx = true;
                if (e[u + 1] >= 0 && k + u > 0 && !(e[u] >= 0 && e[u] < e[u + 1])) bad_ord = true;
                if (!(e[u + 1] >= 0 && e[u + 1] <= lim)) first_out = min(first_out, k + u);
            }
        };
        for (int k = 4 * tid;;) {
            check(k, ent[0], before[0]);
            k += 4 * NT;
            if (k - 4 * lane >= A.K) break;   // (whole warps)
#pragma unroll
            for (int i = 0; i + 1 < NE; ++i) {
                ent[i] = ent[i + 1];
                before[i] = before[i + 1];
            }
            ent[NE - 1] = entries(k + 4 * (NE - 1) * NT);
            before[NE - 1] = entry_before(k + 4 * (NE - 1) * NT);
        }
        if (rank == 0 && bad_idx) report(A.dev_status, SA_DEV_INDEX);
        if (rank == 0 && bad_ord) report(A.dev_status, SA_DEV_ORDER);
        first_out = (int)__reduce_min_sync(0xffffffffu, (unsigned)first_out);
        // the heads' largest |q| in bf16 bits, a head's chunks lying side by side; `below`: of those under it
        auto largest_q = [&](int i, uint32_t below) {
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 v = qv[2 * i + j];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t t = w[k] & 0x7FFF7FFFu;
                    if (below) t &= __vcmpltu2(t, below);
                    mx = __vmaxu2(mx, t);
                }
            }
            mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
            for (int o = 1; o < CPH; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            return mx;
        };
        uint32_t most = 0, least = 0xFFFFu, odd = 0;   // over the warp's heads with values
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            q_head[i] = largest_q(i, 0);
            if (__any_sync(0xffffffffu, q_head[i] >= 0x7F80u)) {   // an infinite or NaN one: the largest finite
                odd = 1;
                q_head[i] = largest_q(i, 0x7F807F80u);
            }
            most = max(most, q_head[i]);
            if (q_head[i]) least = min(least, q_head[i]);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) found[warp] = make_uint4((unsigned)first_out, most, least, odd);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);   // two S buffers (SN columns each), O (HQP columns)
    const uint4 part = found[min(lane, NT / 32 - 1)];
    const int n_top = p >= 0 ? (int)__reduce_min_sync(0xffffffffu, part.x) : 0;
    const uint32_t q_max = __reduce_max_sync(0xffffffffu, part.y), q_odd = __any_sync(0xffffffffu, part.w);
    // Heads 2^6 apart: each has an exponent of its own then, and its scores a factor
    const bool mixed = __reduce_min_sync(0xffffffffu, part.z) + (6u << 7) < q_max;
    const int n_keys = p >= 0 ? n_top + (p - w0 + 1) : 0;
    const int n_tiles = (n_keys + kTile - 1) / kTile;
    const int i0 = by_G(n_tiles * rank), i1 = by_G(n_tiles * (rank + 1));
    if (n_keys == 0 && rank == 0) no_keys();

    // softmax warps: TMEM lane quadrant, group, first head
    const int quad = warp & 3, hg = loader ? 0 : (warp >> 2) - 1, h0 = hg * HG;
    const int key = quad * 32 + lane;                     // TMEM lane: key (S^T) or head dim (O^T)
    const uint32_t lane_t = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)h0;
    float *negm = reinterpret_cast<float *>(sm + C::kOffNegM) + (hg * 4 + quad) * HG;   // this warp's copy
    float *q_scale = reinterpret_cast<float *>(sm + C::kOffQs);   // (mixed) the heads' exponents against the row's

    if (i0 < i1) {
        // the largest value's power of two, so that it lies in (224, 448] (a mantissa beyond
        // 1.75 carries into the exponent); at least 2^-120
        auto exponent_of = [](uint32_t q) { return max(-120, (int)(((q << 16) + 0x1FFFFFu) >> 23) - 135); };
        const int e2 = exponent_of(q_max);
        const float factor = __int_as_float((e2 + 127) << 23) * P.scale_log2;

        constexpr int RPT = 32 / CPH, NIT = 32 / RPT;   // rows that a loader warp copies at once, turns for its 32
        // lookups of the loader threads, one key each: position (-1: none), page, cache row, scales
        auto position = [&](int t) {
            const int kk = t * kTile + tid;
            return t < i1 && kk < n_keys ? (kk < n_top ? __ldg(trow + kk) : w0 + (kk - n_top)) : -1;
        };
        auto page_of = [&](int pos) { return pos >= 0 && pt ? __ldg(pt + (pos >> 6)) : 0; };
        auto row_of = [&](int pos, int page) {
            if (pos < 0) return -1;
            if (!pt) return b * A.S_max + pos;
            if (page >= 0 && page < A.pool_pages) return page * 64 + (pos & 63);
            report(A.dev_status, SA_DEV_INDEX);
            return -1;
        };
        auto put_scale = [&](int t, int row, float ks, float vs) {
            vs = clamp_scale(vs);
            float *o = sc + (t & 1) * 2 * kTile + tid;
            o[0] = row >= 0 ? clamp_scale(ks) * factor : 0.f;
            o[kTile] = row >= 0 ? __log2f(vs) : -CUDART_INF_F;
        };
        int pos3 = -1;   // the position of tile t + 3's key
        int row[NP] = {-1, -1, -1};   // the cache rows of tiles t, t + 1 and t + 2's
        if (loader) {
            if (n_top != A.K || i0 != g0) {   // it came otherwise
#pragma unroll
                for (int t = 0; t < NP; ++t) pos_g[t] = position(i0 + t);
#pragma unroll
                for (int t = 0; t < NP; ++t) page_g[t] = page_of(pos_g[t]);
            }
            pos3 = position(i0 + 3);
#pragma unroll
            for (int t = 0; t < NP; ++t)
                row[t] = row_of(i0 + t < i1 && (i0 + t) * kTile + tid < n_keys ? pos_g[t] : -1, page_g[t]);
        }

        // Copies of a warp's 32 keys, D / 16 threads a row: K into its swizzled tile; V's codes
        // to where the thread that copied them finds them again.
        const int key_l = (tid & 96) + lane / CPH, ch_l = lane % CPH;   // turn 0's key and chunk
        auto gather_k = [&](int row) {
#pragma unroll
            for (int i = 0; i < NIT; ++i) {
                const int id = __shfl_sync(0xffffffffu, row, i * RPT + lane / CPH);
                cp_async16_or_zero(sm + C::kOffK + sw<D>(key_l + i * RPT, ch_l), A.k + (int64_t)max(id, 0) * D + ch_l * 16, id >= 0);
            }
        };
        uint4 vc[NIT];   // V's codes
        auto gather_v = [&](int row) {
#pragma unroll
            for (int i = 0; i < NIT; ++i) {
                const int id = __shfl_sync(0xffffffffu, row, i * RPT + lane / CPH);
                vc[i] = make_uint4(0, 0, 0, 0);
                if (id >= 0) vc[i] = __ldg(reinterpret_cast<const uint4 *>(A.v + (int64_t)id * D + ch_l * 16));
            }
        };
        // V(t)'s codes to fp16 (exact).  With 128 dims the threads of a row's upper half write
        // their two chunks in the other order: in one go the two halves would meet in the banks.
        auto widen_v = [&]() {
            const bool flip = D == 128 && ch_l >= 4;
#pragma unroll
            for (int i = 0; i < NIT; ++i) {
                const uint4 c = vc[i];
                uint4 a, b;
                f16_of_e4m3x4(flip ? c.z : c.x, a.x, a.y);
                f16_of_e4m3x4(flip ? c.w : c.y, a.z, a.w);
                f16_of_e4m3x4(flip ? c.x : c.z, b.x, b.y);
                f16_of_e4m3x4(flip ? c.y : c.w, b.z, b.w);
                uint8_t *to = sm + C::kOffV;
                const int key = key_l + i * RPT, ch = 2 * ch_l + (flip ? 1 : 0);
                *reinterpret_cast<uint4 *>(to + sw_v(key, ch)) = a;
                *reinterpret_cast<uint4 *>(to + sw_v(key, ch ^ 1)) = b;
            }
        };
        float ks0 = 0.f, vs0 = 0.f;
        if (loader) {
            gather_k(row[0]);
            cp_async_commit();
            if (row[0] >= 0) {
                ks0 = __ldg(A.k_scale + (row[0] >> P.sb_shift));
                vs0 = __ldg(A.v_scale + (row[0] >> P.sb_shift));
            }
        }
        // both parts of this thread's chunks of Q, while the copies fly (heads >= Hq are zeros)
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int c = tid + i * NT;
            if (c >= HQP * CPH) break;
            const int eh = mixed ? exponent_of(q_head[i]) : e2;
            const float down = __int_as_float((127 - eh) << 23);
            if (mixed && c % CPH == 0) q_scale[c / CPH] = eh - e2 < -126 ? 0.f : __int_as_float((eh - e2 + 127) << 23);
            const uint4 q0 = qv[2 * i], q1 = qv[2 * i + 1];
            const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t y[2], h[2];   // scaled q in fp16: exact but for what is 2^-23 of the largest
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t x = w[2 * k + j];
                    y[j] = f16x2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down);
                }
                hi[k] = e4m3x4_of_f16(y[0], y[1]);
                f16_of_e4m3x4(hi[k], h[0], h[1]);
                lo[k] = e4m3x4_of_f16(hsub2(y[0], h[0]), hsub2(y[1], h[1]));
                if (q_odd) {   // an infinite q makes NaN scores, as the formula does
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (((w[2 * k + j / 2] >> (16 * (j & 1))) & 0x7F80u) == 0x7F80u) hi[k] |= 0x7Fu << (8 * j);
                }
            }
            *reinterpret_cast<uint4 *>(sm + C::kOffQ + sw<D>(c / CPH, c % CPH)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(sm + C::kOffQ + sw<D>(HQP + c / CPH, c % CPH)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (loader) put_scale(i0, row[0], ks0, vs0);
        cp_async_wait<0>();   // the K tile
        fence_async_smem();
        __syncthreads();

        auto lost = [&](int t, int what) { return CHECK && r == 0 && rank == 0 && P.lost == 2 * (t - i0) + what; };
        auto issue_s = [&](int t) {   // both parts of Q into the same columns
            if (lost(t, 0)) return;
            constexpr uint32_t idesc = idesc_e4m3_f32(128, SN);
            const uint64_t kd = smem_desc(smem_u32(sm + C::kOffK), 8 * D, D == 128 ? 2 : 4);
            const uint64_t qd = smem_desc(smem_u32(sm + C::kOffQ), 8 * D, D == 128 ? 2 : 4);
            const uint32_t dt = tmem + (uint32_t)(((t - i0) & 1) * SN);
#pragma unroll
            for (int part = 0; part < (C::kSide ? 1 : 2); ++part)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    tc_mma_f8(dt, kd + (uint64_t)((kk * 32) >> 4), qd + (uint64_t)((part * HQP * D + kk * 32) >> 4), idesc,
                              part + kk > 0 ? 1u : 0u);
            tc_commit(bar_s + ((t - i0) & 1));
        };
        auto issue_pv = [&](int t) {   // A (V^T) and B (P^T) both MN-major
            if (lost(t, 1)) return;
            constexpr uint32_t idesc = idesc_f16_mn(128, HQP);
            const uint64_t vd = desc_v<D>(smem_u32(sm + C::kOffV));
            const uint64_t pd = desc_mn_plain(smem_u32(sm + C::kOffP), HQP * 16, 128);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)   // 16 keys: two 8-key groups
                tc_mma_f16(tmem + 2 * SN, vd + (uint64_t)((kk * 2048) >> 4), pd + (uint64_t)((kk * 2 * HQP * 16) >> 4), idesc,
                           (t == i0 && kk == 0) ? 0u : 1u);
            tc_commit(bar_pv);
        };
        bool ok = true;
        // P V(t) is phase t - i0 of its barrier; S(t) may end while some warp still looks for
        // the end of S(t - 1), so each S buffer has a barrier of its own
        // A wait that runs out first waits for all MMAs that were issued (with a limit again):
        // what comes after it reuses their tiles and gives their TMEM back.  None is issued then.
        auto waited = [&](uint64_t *which, uint32_t parity) {
            const unsigned long long limit = CHECK ? P.limit_ns : kWaitLimitNs;
            if (__all_sync(0xffffffffu, mbar_wait(which, parity, abort_flag, limit))) return true;
            drain_mmas(bar_drain);
            return false;
        };
        auto wait_s = [&](int t) { return waited(bar_s + ((t - i0) & 1), (uint32_t)((t - i0) >> 1) & 1u); };
        auto wait_pv = [&](int t) { return waited(bar_pv, (uint32_t)(t - i0) & 1u); };
        // Only the MMA warp polls: warps that poll take issue slots from those that compute,
        // and warps that wait at a barrier do not.  It tells the loader warps when P V(t - 1) and
        // S(t + 1) are done, and the softmax warps when P V(t - 1) is.
        constexpr int kBarSoft = 6, kBarVote = 8, kSoft = C::kThreads - 128, kBarV = 1, kBarK = 7, kBarKIn = 9, kLoad = 160;
        if (warp == C::kWarpMma) {
            // ------------------------------------------------------------ MMA warp
            if (elect_one()) issue_s(i0);
            __syncwarp();
            ok = wait_s(i0);
            bar_arrive_n(kBarSoft, kSoft);   // the first tile's scores
            if (i0 + 1 < i1) {
                bar_arrive_n(kBarK, kLoad);  // the K tile is free
                bar_sync_n(kBarV, kLoad);    // K(i0 + 1) is there
                if (elect_one() && ok) issue_s(i0 + 1);
                __syncwarp();
                ok = ok && wait_s(i0 + 1);
                if (i0 + 2 < i1) bar_arrive_n(kBarK, kLoad);
            }
            for (int t = i0; t < i1; ++t) {
                if (__syncthreads_or(!ok)) {   // a wait ran out: everybody leaves here
                    bar_arrive_n(kBarSoft, kSoft);
                    break;
                }
                if (elect_one()) {
                    tc_fence_after();
                    issue_pv(t);
                }
                __syncwarp();
                ok = wait_pv(t);
                bar_arrive_n(kBarSoft, kSoft);
                if (t + 1 < i1) bar_arrive_n(kBarV, kLoad);
                if (t + 2 < i1) {
                    // Not before the vote on tile t + 1 has read its scores: reads that meet MMAs
                    // wait.  (Behind P V's end 7 percent more for 4 x 1024 rows of 64 heads.)
                    bar_sync_n(kBarVote, kSoft);
                    bar_sync_n(kBarKIn, kLoad);   // K(t + 2) is there
                    if (elect_one() && ok) issue_s(t + 2);
                    __syncwarp();
                    ok = ok && wait_s(t + 2);
                    if (t + 3 < i1) bar_arrive_n(kBarK, kLoad);
                }
            }
            if (!ok && lane == 0) report(A.dev_status, SA_DEV_TIMEOUT);
        } else if (loader) {
            // ------------------------------------------------------------ loader warps
            gather_v(row[0]);
            if (row[1] >= 0) {
                ks0 = __ldg(A.k_scale + (row[1] >> P.sb_shift));
                vs0 = __ldg(A.v_scale + (row[1] >> P.sb_shift));
            }
            if (i0 + 1 < i1) {
                bar_sync_n(kBarK, kLoad);   // S(i0) is done: the K tile is free
                gather_k(row[1]);
                cp_async_wait_all();
                fence_async_smem();
                bar_arrive_n(kBarV, kLoad);
            }
            for (int t = i0; t < i1; ++t) {
                // lookups ahead: the page of tile t + 3's key, the scales of tile t + 2's
                const int pg3 = page_of(pos3);
                const float ks1 = ks0, vs1 = vs0;
                if (row[2] >= 0) {
                    ks0 = __ldg(A.k_scale + (row[2] >> P.sb_shift));
                    vs0 = __ldg(A.v_scale + (row[2] >> P.sb_shift));
                }
                const int pos4 = position(t + 4);
                if (t > i0) bar_sync_n(kBarV, kLoad);   // P V(t - 1) is done: V(t) over V(t - 1)
                widen_v();
                if (t + 1 < i1) put_scale(t + 1, row[1], ks1, vs1);
                fence_async_smem();
                if (__syncthreads_or(false)) {   // a wait ran out
                    if (t + 2 < i1) bar_sync_n(kBarK, kLoad);
                    break;
                }
                // the next copies fly while P V(t) runs
                if (t + 1 < i1) gather_v(row[1]);
                if (t + 2 < i1) {
                    bar_sync_n(kBarK, kLoad);   // S(t + 1) is done: K(t + 2) over K(t + 1)
                    gather_k(row[2]);
                }
                row[1] = row[2];
                row[2] = row_of(pos3, pg3);
                pos3 = pos4;
                cp_async_wait_all();
                if (t + 2 < i1) {
                    fence_async_smem();
                    bar_arrive_n(kBarKIn, kLoad);
                }
            }
        } else {
            // ------------------------------------------------------------ softmax warps
            f2 l[HG / 2];
#pragma unroll
            for (int i = 0; i < HG / 2; ++i) l[i] = 0;
            float *gmax = reinterpret_cast<float *>(sm + C::kOffMax) + h0 * 4;   // [quad][HG]
            uint32_t *flags = reinterpret_cast<uint32_t *>(sm + C::kOffFlags) + 4 * hg;   // [quad]
            uint8_t *pbuf = sm + C::kOffP + (key >> 3) * (HQP * 16) + (key & 7) * 16 + (h0 / 8) * 128;
            float m = kLowest;   // a head a lane: its running maximum
            float l_small = 0.f; // (clusters) and its sum over this warp's keys of small value scales
            if (lane < HG) negm[lane] = -m;
            bool fresh = true;                         // no key yet
            bar_sync_n(kBarSoft, kSoft);               // S(i0) is done
            for (int t = i0; t < i1; ++t) {
                // S(t) is done: the MMA warp waited for it before it met the last barrier
                tc_fence_after();
                const uint32_t s_t = lane_t + (uint32_t)(((t - i0) & 1) * SN);
                const float *kf = sc + (t & 1) * 2 * kTile + key;
                const float lv = kf[kTile], iv = lv >= kSmallV ? ex2f(-lv) : 0.f;
                const f2 c2 = pk(kf[0], kf[0]), lv2 = pk(lv, lv), iv2 = pk(iv, iv);
                if (mixed) {   // S in the row's exponent, in place (unrolled: a loop here costs the whole one registers)
#pragma unroll
                    for (int c = 0; c < (C::kSide ? 2 : 1) * HG; c += 8) {
                        uint32_t u[8];
                        tmem_ld_x8(s_t + (uint32_t)c, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * q_scale[h0 + (c + i) % HG]);
                        tmem_st8(s_t + (uint32_t)c, u);
                    }
                    tmem_st_wait_all();
                }
                // Scores of N heads: read from TMEM for the vote and again for P (of 32 heads the
                // second half: keeping all of them beside 32 sums spills).
                auto scores = [&](int c, auto &x) {
                    constexpr int N = 2 * sizeof(x) / sizeof(f2);
                    uint32_t u[N], v[N];
                    tmem_ld_cols(s_t + (uint32_t)c, u);
                    if (C::kSide) tmem_ld_cols(s_t + (uint32_t)(HQP + c), v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        x[i] = pku(u[2 * i], u[2 * i + 1]);
                        if (C::kSide) x[i] = add2(x[i], pku(v[2 * i], v[2 * i + 1]));
                    }
                };
                // e: log2 of P
                auto exponents = [&](int c, auto &x) {
                    constexpr int N = 2 * sizeof(x) / sizeof(f2);
                    scores(c, x);
#pragma unroll
                    for (int i = 0; i < N / 4; ++i) {
                        const ulonglong2 n2 = reinterpret_cast<const ulonglong2 *>(negm + c)[i];
                        // (the largest one's difference to m is exact, however large both are)
                        x[2 * i] = add2(fma2(x[2 * i], c2, lv2), n2.x);
                        x[2 * i + 1] = add2(fma2(x[2 * i + 1], c2, lv2), n2.y);
                    }
                };
                // the exact maxima over the tile's keys, a head a lane
                auto maxima = [&]() {
                    float tm = -CUDART_INF_F;
#pragma unroll
                    for (int c = 0; c < HG; c += 8) {
                        f2 x[4];
                        scores(c, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = up(fma2(x[i], c2, lv2));
                            const float a = redux_max(f.x), b = redux_max(f.y);
                            if (lane == c + 2 * i) tm = a;
                            if (lane == c + 2 * i + 1) tm = b;
                        }
                    }
                    if (lane < HG) gmax[quad * HG + lane] = tm;
                    const bool any_key = bar_or(3 + 2 * hg, 128, lv > -CUDART_INF_F);
                    if (lane < HG) tm = fmaxf(fmaxf(gmax[lane], gmax[HG + lane]), fmaxf(gmax[2 * HG + lane], gmax[3 * HG + lane]));
                    fresh = fresh && !any_key;
                    return tm;
                };
                if (fresh) {   // the row's first keys: references by which the largest P is 2^kTop
                    const float tm = maxima();
                    if (lane < HG) {
                        if (tm > kLowest) m = __fsub_ru(tm, kTop);   // (up: among large numbers it is tm itself)
                        negm[lane] = -m;
                    }
                    __syncwarp();
                }
                // One vote of the group a tile: does any head need a new reference?
                // (KEEP: the first 16 heads' e is kept for P, where registers allow: with 64
                // heads it spills, 412 us for the padded chunk instead of 393.)
                constexpr bool KEEP = !CL && HQP == 16;
                f2 e0[8];
                exponents(0, e0);
                float top = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = up(e0[i]);
                    top = max3(top, f.x, f.y);
                }
#pragma unroll
                for (int c = 16; c < HG; c += 16) {
                    f2 e[8];
                    exponents(c, e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = up(e[i]);
                        top = max3(top, f.x, f.y);
                    }
                }
                if (t > i0 && t + 1 < i1) bar_arrive_n(kBarVote, kSoft);
                const bool raise = bar_or(2 + 2 * hg, 128, top > kRaise);
                if (t > i0) bar_sync_n(kBarSoft, kSoft);   // P V(t - 1) is done: O is whole, the P tile is free
                tc_fence_after();
                if (raise) {
                    uint32_t heads = 0;   // those with an e above kRaise, for any key of the tile
                    if (__any_sync(0xffffffffu, top > kRaise)) {
#pragma unroll
                        for (int c = 0; c < HG; c += 16) {
                            f2 e[8];
                            if (c > 0 || !KEEP) exponents(c, e);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 f = up(c > 0 || !KEEP ? e[i] : e0[i]);
                                if (f.x > kRaise) heads |= 1u << (c + 2 * i);
                                if (f.y > kRaise) heads |= 2u << (c + 2 * i);
                            }
                        }
                        heads = __reduce_or_sync(0xffffffffu, heads);
                    }
                    if (lane == 0) flags[quad] = heads;
                    // They go up by kStep: nothing but a bit a head has to be known of the other
                    // keys.  Where that is not enough, or lost in a large reference's rounding, to
                    // what takes the largest P back to 2^kTop.
                    const bool far = bar_or(3 + 2 * hg, 128, top > kRaise + kStep || (lane < HG && fabsf(m) > kCoarse));
                    const uint4 fl = *reinterpret_cast<const uint4 *>(flags);
                    heads = fl.x | fl.y | fl.z | fl.w;
                    const bool mine = (heads >> lane) & 1u;
                    float to = m + kStep, f = 1.f;
                    if (far) to = __fsub_ru(maxima(), kTop);
                    if (mine) {
                        // What the row's earlier tiles made of the head shrinks by f^2: the step may be
                        // that of two value scales, 2^128, and the sum is not of contributions but weights.
                        f = ex2f(0.5f * (m - to));
                        if (CL) l_small *= f * f;
                        m = to;
                        negm[lane] = -m;
                    }
#pragma unroll
                    for (int c = 0; c < HG; c += 8) {
                        if (!((heads >> c) & 0xFFu)) continue;
                        float fc[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) fc[i] = __shfl_sync(0xffffffffu, f, c + i);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f2 f2i = pk(fc[2 * i], fc[2 * i + 1]);
                            l[c / 2 + i] = mul2(mul2(l[c / 2 + i], f2i), f2i);
                        }
                        if (t > i0) {
                            uint32_t o[8];
                            tmem_ld_x8(lane_t + (uint32_t)(2 * SN + c), o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fc[k] * fc[k]);
                            tmem_st8(lane_t + (uint32_t)(2 * SN + c), o);
                        }
                    }
                    tmem_st_wait_all();
                    __syncwarp();
                    if (KEEP && (heads & 0xFFFFu)) exponents(0, e0);
                }
                // P^T as an MN-major operand without swizzle: 16-byte rows of 8 heads, the
                // rows of 8 keys 16 bytes apart, the head chunks of a key group 128 bytes
                // apart, key groups HQP * 16 bytes apart
#pragma unroll
                for (int c = 0; c < HG; c += 16) {
                    f2 e[8];
                    if (KEEP && c == 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) e[i] = e0[i];
                    } else {
                        exponents(c, e);
                    }
                    uint32_t p16[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {   // two heads
                        const float2 f = up(e[i]);
                        const float p0 = ex2f(f.x), p1 = ex2f(f.y);
                        l[c / 2 + i] = fma2(pk(p0, p1), iv2, l[c / 2 + i]);
                        p16[i] = f16x2(p0, p1);
                    }
                    *reinterpret_cast<uint4 *>(pbuf + c * 16) = make_uint4(p16[0], p16[1], p16[2], p16[3]);
                    *reinterpret_cast<uint4 *>(pbuf + c * 16 + 128) = make_uint4(p16[4], p16[5], p16[6], p16[7]);
                }
                // A key of a small value scale: its P may be next to nothing beside those of large
                // ones (down to 2^-128), its weight not, so that one is computed by itself.
                // (Rare, but its code has to be chosen: in a cluster, where each CTA runs the loop's
                // body a few times, a short one, a head a lane; else one that takes no register.
                // 16 paged rows of 2560 keys 14.5 us, the other way 16.8; padded chunk 381 and 483.)
                const bool small = lv > -CUDART_INF_F && lv < kSmallV;
                if (__any_sync(0xffffffffu, small)) {
                    if constexpr (CL) {
#pragma unroll 1
                        for (int c = 0; c < HG; c += 2) {
                            uint32_t u[2][2] = {};
                            tmem_ld_x2(s_t + (uint32_t)c, u[0]);
                            if (C::kSide) tmem_ld_x2(s_t + (uint32_t)(HQP + c), u[1]);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float w = __uint_as_float(u[0][i]);
                                if (C::kSide) w += __uint_as_float(u[1][i]);
                                w = small ? ex2f(fmaf(w, kf[0], lv) + negm[c + i] - lv) : 0.f;
#pragma unroll
                                for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
                                if (lane == c + i) l_small += w;
                            }
                        }
                    } else {
                        const float off = small ? lv : CUDART_INF_F;
#pragma unroll
                        for (int c = 0; c < HG; c += 8) {
                            f2 e[4];
                            exponents(c, e);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 f = up(e[i]);
                                l[c / 2 + i] = add2(l[c / 2 + i], pk(ex2f(f.x - off), ex2f(f.y - off)));
                            }
                        }
                    }
                }
                fence_async_smem();
                tc_fence_before();
                if (__syncthreads_or(false)) break;   // a wait ran out
            }
            // the row's sums over this warp's keys, each step on half as many heads as the
            // last: a lane ends with the sum of one head (HG = 16: of one half of the lanes)
            float v[HG];
#pragma unroll
            for (int i = 0; i < HG / 2; ++i) {
                const float2 f = up(l[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
#pragma unroll
            for (int o = HG / 2; o > 0; o >>= 1) {
                const bool high = lane & o;
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const float give = high ? v[i] : v[i + o], keep = high ? v[i + o] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            if (HG == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
            if (lane < HG) gmax[quad * HG + lane] = CL ? v[0] + l_small : v[0];
            bar_sync_n(3 + 2 * hg, 128);
            if (lane < HG) {
                const float L = (gmax[lane] + gmax[HG + lane]) + (gmax[2 * HG + lane] + gmax[3 * HG + lane]);
                const int h = h0 + lane;
                if (CL) {
                    if (quad == 0) part_ml[h] = make_float2(m, L);
                } else {
                    negm[lane] = L == 0.f ? 0.f : rcp(L);
                    if (A.lse && quad == 0 && h < A.Hq)
                        A.lse[(int64_t)r * A.Hq + h] = L == 0.f ? -CUDART_INF_F : (m + log2f(L)) * 0.69314718055994531f;
                }
            }
            bar_sync_n(kBarSoft, kSoft);   // P V of the last tile is done
            tc_fence_after();
            // A part of a row as it is into shared memory (the K and V tiles are idle by
            // now), for the join; a row normalised and out, 64 bytes of a head a store (staged
            // for 16-byte stores it took 4 percent longer)
            float *part = reinterpret_cast<float *>(sm + C::kOffK) + h0 * D;
            uint16_t *out = A.out + ((int64_t)r * A.Hq + h0) * D + key;
#pragma unroll
            for (int c = 0; c < HG; c += 8) {
                uint32_t u[8];
                tmem_ld_x8(lane_t + (uint32_t)(2 * SN + c), u);
                tmem_ld_wait();
                if (D == 128 || key < D) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float o = __uint_as_float(u[k]);
                        if (CL) {
                            part[(c + k) * D + key] = o;
                        } else {
                            const __nv_bfloat16 ob = __float2bfloat16_rn(o * negm[c + k]);
                            if (h0 + c + k < A.Hq) out[(c + k) * D] = *reinterpret_cast<const uint16_t *>(&ob);
                        }
                    }
                }
            }
        }
    } else if (CL && tid < HQP) {   // no share of the row
        part_ml[tid] = make_float2(kLowest, 0.f);
    }
    tc_fence_before();
    if (CL) cluster_sync();
    else __syncthreads();
    if (warp == C::kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (CL) {
        // Join the parts of the heads rank * hpr ..: a warp a head, D / 32 dims a lane, so that a
        // load takes a whole row of one CTA's memory.  (16 paged rows of 2560 keys and 64 heads
        // 15 us; with each lane of four taking every fourth part of 4 dims, so that a load went
        // to four CTAs, 16.1.)
        constexpr int V = D / 32, AT = 10;   // dims a lane, parts on their way at once
        const int hb = rank * P.hpr, nh = n_keys > 0 ? max(0, min(P.hpr, A.Hq - hb)) : 0;
        for (int h = hb + warp; h < hb + nh; h += NT / 32) {
            float v[AT][V];
            const uint32_t off = C::kOffK + (h * D + lane * V) * 4;
            auto fetch = [&](int c0) {
#pragma unroll
                for (int u = 0; u < AT; ++u)
                    if (c0 + u < G) dsmem_ld(in_cta(sm, (uint32_t)(c0 + u)) + off, v[u]);
            };
            float ml[2] = {kLowest, 0.f};   // part `lane`: its reference and sum
            if (lane < G) dsmem_ld(in_cta(sm, (uint32_t)lane) + C::kOffEpi + h * 8, ml);
            fetch(0);
            const bool some = ml[1] != 0.f;   // (a part without keys wrote nothing)
            const float m = redux_max(some ? ml[0] : kLowest), fh = some ? ex2f(0.5f * (ml[0] - m)) : 0.f;   // (as in a raise)
            float L = some ? fh * ml[1] * fh : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
            const float w = L == 0.f ? 0.f : fh * rcp(L) * fh;
            float o[V] = {};
            for (int c0 = 0; c0 < G; c0 += AT) {
                if (c0 > 0) fetch(c0);
#pragma unroll
                for (int u = 0; u < AT; ++u) {
                    const float wu = __shfl_sync(0xffffffffu, w, c0 + u);
                    if (wu != 0.f) {   // (0 for c0 + u >= G)
#pragma unroll
                        for (int k = 0; k < V; ++k) o[k] = fmaf(wu, v[u][k], o[k]);
                    }
                }
            }
            uint32_t *out = reinterpret_cast<uint32_t *>(A.out + ((int64_t)r * A.Hq + h) * D) + lane * (V / 2);
            if constexpr (V == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
            else *out = pack_bf16(o[0], o[1]);
            if (A.lse && lane == 0) A.lse[(int64_t)r * A.Hq + h] = L == 0.f ? -CUDART_INF_F : (m + log2f(L)) * 0.69314718055994531f;
        }
        cluster_sync();   // nobody leaves while its parts are read
    }
}

template <int D, int HQP, bool CL, bool CHECK = false>
sa_status launch_q8(const Params &p, int R, cudaStream_t st) {
    using C = Cfg<D, HQP>;
    if (prepare_kernel<attn_q8_kernel<D, HQP, CL, CHECK>>(C::kSmem, CL) != cudaSuccess) return SA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)R * (unsigned)p.G);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)p.G;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = CL ? 1 : 0;
    return cuda_ok(cudaLaunchKernelEx(&cfg, attn_q8_kernel<D, HQP, CL, CHECK>, p));
}

// What follows from the call and p.G.
void fill(Params &p, const AttnQ8Args &a) {
    p.a = a;
    p.inv_G = ((1u << 20) + p.G - 1) / p.G;
    p.hpr = (a.Hq + p.G - 1) / p.G;
    p.sb_shift = 0;
    while ((1 << p.sb_shift) < a.scale_block) ++p.sb_shift;
    p.scale_log2 = a.scale * 1.4426950408889634f;
}

// How many clusters of G of these CTAs the device runs at once, one CTA an SM
// (asked once for each device and size; clusters do not span GPCs, so it is
// less than SMs / G: 33 of 4, 15 of 8 or 9, 11 of 10, 7 of 12 to 16 on 148 SMs).
template <int D, int HQP>
int active_clusters(int dev, int sms, int G) {
    if (G == 1) return sms;
    static std::atomic<int> known[64][17];
    const int k = dev < 64 ? known[dev][G].load(std::memory_order_relaxed) : 0;
    if (k > 0) return k;
    using C = Cfg<D, HQP>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)G);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)G;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, attn_q8_kernel<D, HQP, true>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 0;
    }
    n = std::min(n, sms / G);
    if (dev < 64) known[dev][G].store(n, std::memory_order_relaxed);
    return n;
}

template <int D, int HQP>
sa_status launch_q8_rows(const AttnQ8Args &a, cudaStream_t st) {
    using C = Cfg<D, HQP>;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SA_ERR_CUDA;
    Params p = {};
    const int R = a.B * a.T;
    const int tiles = (int)std::min<int64_t>(((int64_t)a.K + a.W + kTile - 1) / kTile, ((int64_t)a.S_max + kTile - 1) / kTile);
    // CTAs a row.  In units of one tile's time in a cluster (1.0 us with 16 heads, 1.9
    // with 64), alone on an SM, a cluster takes 5.4 for its row's start and join and 1 a
    // tile, a single CTA 3.2 and 0.85; another CTA on the SM costs all of them 24 percent
    // with up to 32 heads, 33 with 64 (over rows of 2 to 40 tiles, 1 to 304 rows, it is 0.5
    // percent off the best on average, 15 at worst: 8 rows of 20 tiles and 64 heads 10.5 us
    // with 10 CTAs a row, 33.5 with one, 14.5 with 4; 112 such rows 34 with one, 40 with 4).
    p.G = 1;
    double best = 0;
    if (prepare_kernel<attn_q8_kernel<D, HQP, true>>(C::kSmem, true) != cudaSuccess) return SA_ERR_CUDA;
    for (int G = 1; G <= std::min(16, tiles); ++G) {
        if (G > 1 && (R >= 2 * sms || (tiles + G - 1) / G == (tiles + G - 2) / (G - 1))) continue;
        const int at_once = active_clusters<D, HQP>(dev, sms, G);
        if (at_once < 1) continue;
        const int n = (R + at_once - 1) / at_once, t = (tiles + G - 1) / G;
        const double cost = (G == 1 ? 3.2 + 0.85 * t : 5.4 + t) * (1.0 + (HQP == 64 ? 0.33 : 0.24) * (std::min(n, C::kPerSm) - 1)) *
                            ((n + C::kPerSm - 1) / C::kPerSm);
        if (G == 1 || cost < best) {
            best = cost;
            p.G = G;
        }
    }
    fill(p, a);
    return p.G > 1 ? launch_q8<D, HQP, true>(p, R, st) : launch_q8<D, HQP, false>(p, R, st);
}

template <int D>
sa_status launch_q8_heads(const AttnQ8Args &a, cudaStream_t st) {
    if (a.Hq <= 16) return launch_q8_rows<D, 16>(a, st);
    if (a.Hq <= 32) return launch_q8_rows<D, 32>(a, st);
    return launch_q8_rows<D, 64>(a, st);
}

}  // namespace

sa_status launch_attn_q8_check(const AttnQ8Args &a, int ctas, int lost, unsigned long long limit_ns, cudaStream_t st) {
    Params p = {};
    p.G = ctas;
    fill(p, a);
    p.limit_ns = limit_ns;
    p.lost = lost;
    return ctas > 1 ? launch_q8<128, 16, true, true>(p, a.B, st) : launch_q8<128, 16, false, true>(p, a.B, st);
}

sa_status launch_attn_q8(const AttnQ8Args &a, cudaStream_t st) {
    return a.d == 128 ? launch_q8_heads<128>(a, st) : launch_q8_heads<64>(a, st);
}

}  // namespace sa
