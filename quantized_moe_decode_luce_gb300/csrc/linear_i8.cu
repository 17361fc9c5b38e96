// linear_i8.cu -- the dense int8 product with scales per token and per output
// channel (luce_linear_i8), with its C-ABI entry point.
//
//   out[t][n] = isum[t][n] * (x_scale[t] * w_scale[n]) (+ bias[n]),
//   isum[t][n] = sum_k xq[t][k] wq[n][k], an exact int32 sum
//   (K <= 65,536: |isum| <= 2^16 2^14 = 2^30).
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include <cuda.h> // CUtensorMap and its enums (the encoder is reached through the runtime's entry-point query)
#include <cuda_bf16.h>

#include "common.cuh"

LUCE_DEFINE_FAULT_WORD(luce_internal_fault_linear)

namespace {

using namespace luce;

// The epilogue of every kernel of this file: four roundings to fp32 at most,
// then the output type's, so that all of them give the same bits.
__device__ __forceinline__ float epilogue(int isum, float xs, float ws, const float *bias, int n)
{
    float v = __fmul_rn((float)isum, __fmul_rn(xs, ws));
    if (bias)
        v = __fadd_rn(v, bias[n]);
    return v;
}
__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(__half *p, float v) { *p = __float2half_rn(v); }

// One warp per output channel and up to TPW tokens: the lanes walk K in
// 16-byte steps with dp4a, then a butterfly.
constexpr int WARPS = 8;
constexpr int TPW = 8;

template <typename TO>
__global__ void __launch_bounds__(WARPS * 32)
    k_linear_i8_rows(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int T,
                     int N, int K, TO *out, int64_t ldo)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int t0 = blockIdx.y * TPW, nt = min(TPW, T - t0);
    const int K16 = K >> 4;
    for (int64_t n = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); n < N; n += (int64_t)gridDim.x * WARPS) {
        int acc[TPW] = {};
        const int4 *wr = reinterpret_cast<const int4 *>(wq + (size_t)n * K);
        for (int i = lane; i < K16; i += 32) {
            const int4 w = wr[i];
#pragma unroll
            for (int t = 0; t < TPW; t++) {
                if (t < nt) {
                    const int4 v = reinterpret_cast<const int4 *>(xq + (size_t)(t0 + t) * K)[i];
                    acc[t] = __dp4a(w.x, v.x, acc[t]);
                    acc[t] = __dp4a(w.y, v.y, acc[t]);
                    acc[t] = __dp4a(w.z, v.z, acc[t]);
                    acc[t] = __dp4a(w.w, v.w, acc[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TPW; t++) {
            const int s = warp_sum_i(acc[t]);
            if (lane == 0 && t < nt)
                store_out(out + (size_t)(t0 + t) * ldo + n, epilogue(s, xs[t0 + t], ws[n], bias, (int)n));
        }
    }
}

// ---------------------------------------------------------------------------
// The product on the tensor cores (more than a few tokens).
//
// Exactness.  tcgen05.mma has no int8 kind on this GPU, so the codes go in as
// fp16: every code is an exact fp16 number, and the partial sums of up to 1024
// products (at most 1024 * 2^14 = 2^24) are exact fp32 integers.  Every CHUNK
// stages the accumulator is read back, converted to int32 and added to the
// int32 sums that the worker threads hold, and the next chunk starts from
// zero: the result is the int32 sum, bit for bit.
//
// Operands.  A = 128 weight rows per CTA, converted into tensor memory (a
// thread writes its own lane's row); B = the tokens, converted into shared
// memory in the tensor core's 128-byte-swizzled K-major layout; D[channel,
// token].  Weights cross HBM and shared memory as int8 and are converted once
// per token tile.  With CG = 2 a CTA pair shares one 256-channel tile: each
// CTA converts its own 128 weight rows and half of the tokens, so the tokens'
// shared-memory traffic per MMA halves, which is what bounds wide tiles (per
// 64 values of K a CTA moves 8 + 8 KB of weights and, for 128 of its own
// token rows, 8 + 8 + 16 + 16 KB of tokens through a 128 B/clock shared
// memory, 512 clocks against the MMAs' 536).
//
// HALVES = 2 splits a tile of up to 256 tokens in two accumulators whose
// chunks end at different stages, so that one is read back while the MMAs of
// the other run; with HALVES = 1 (up to 128 tokens) the two accumulator slots
// alternate chunk by chunk.
//
// Few tiles: SK CTA groups of one cluster split K among them and add their
// int32 sums through distributed shared memory (any split gives the same
// bits).
//
// Roles: warps 0-15 convert (warp w: lane quarter w & 3, a quarter of the
// stage's K; a share of the token rows), read accumulators back and store;
// warp 16 issues the TMA tiles, warp 17 the MMAs (of the pair, in its leader).
// Every wait is bounded: a role that gives up raises LUCE_FAULT_TIMEOUT and
// the CTA's abort flag, the others leave at their next wait, copies and MMAs
// in flight are waited for (bounded) and tensor memory is freed.
constexpr int SK_MAX = 8;          // CTAs of one cluster at most
constexpr int KS = 128;            // K values of one stage
constexpr int CHUNK = 1024 / KS;   // stages whose sums fit fp32
constexpr int RM = 128;            // weight rows per CTA
constexpr int WORKERS = 16;        // warps
constexpr int TMA_WARP = WORKERS, MMA_WARP = WORKERS + 1;
constexpr int TC_THREADS = (WORKERS + 2) * 32;
constexpr uint32_t TMEM_COLS = 512;
constexpr int RA = 4;              // converted stages: A slots of 64 columns in tensor memory, B slots in shared memory
constexpr uint32_t D_COL = RA * 64;
constexpr int LAG = 2;             // stages converted past a chunk's end before it is read back (at most RB)

template <int CG_, int HALVES_, int ROWS_, int NS_, int RB_> struct Cfg {
    static constexpr int CG = CG_, HALVES = HALVES_;
    static constexpr int ROWS = ROWS_;           // token rows per half and CTA, at most
    static constexpr int NS = NS_, RB = RB_;     // raw stages, converted stages (A and B slots)
    static constexpr int DCOLS = ROWS * CG;      // columns of one accumulator slot
    static constexpr int CPW = DCOLS / 4;        // accumulator columns per worker warp
    static constexpr int RAW_W = RM * KS;        // raw weights of a stage
    static constexpr int RAW_X = HALVES * ROWS * KS;
    static constexpr int RAW = RAW_W + RAW_X;
    static constexpr int ATOM = ROWS * 128;      // 64 K values of one half's rows
    static constexpr int BST = HALVES * 2 * ATOM;
    static constexpr int SMEM = NS * RAW + RB * BST + 1024;
    static constexpr int PART = HALVES * DCOLS * RM * 4; // the int32 sums of a CTA
    static_assert(LAG <= RB && RB <= RA && D_COL + 2 * DCOLS <= TMEM_COLS, "tensor memory");
    static_assert(RAW % 1024 == 0 && BST % 1024 == 0 && ATOM % 1024 == 0, "swizzle atoms");
    static_assert(PART <= NS * RAW + RB * BST && SMEM <= 232448, "shared memory");
    static_assert(CPW == 16 || CPW == 32, "accumulator columns");
};

struct TcArgs {
    CUtensorMap tw, tx; // int8 [N][K], box 128 x 128; int8 [T][K], box (nh / CG) x 128; 128-byte swizzle
    const float *xs, *ws, *bias;
    void *out;
    int64_t ldo;
    int T, N, stages; // stages of the whole K
    int nh;           // tokens per half (a multiple of 16 CG)
    int mt, tiles;    // channel tiles, tiles in all (channel tiles fastest)
    int sk;           // CTA groups along K
};

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 128-byte swizzle, K-major, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(16u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

template <int CG> __device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                     "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                     "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
}

// One arrival on `bar` (in both CTAs of the pair) once every MMA issued so far has completed.
template <int CG> __device__ __forceinline__ void mma_commit(uint64_t *bar, uint16_t pair_mask)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(smem_addr(bar)), "h"(pair_mask)
                     : "memory");
}

// The same on this CTA's barrier alone.
template <int CG> __device__ __forceinline__ void mma_commit_here(uint64_t *bar)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Sixteen int8 codes -> sixteen fp16 numbers: bias to unsigned (c + 128),
// place each byte under the exponent of 1024, subtract 1152.  Exact.
__device__ __forceinline__ void codes16(const uint4 w, uint32_t (&h)[8])
{
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t u = in[i] ^ 0x80808080u;
        uint32_t a, b;
        asm("prmt.b32 %0, %1, %2, 0x4140;" : "=r"(a) : "r"(u), "r"(0x64646464u));
        asm("prmt.b32 %0, %1, %2, 0x4342;" : "=r"(b) : "r"(u), "r"(0x64646464u));
        const __half2 ha = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
        const __half2 hb = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
        h[2 * i] = *reinterpret_cast<const uint32_t *>(&ha);
        h[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&hb);
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Waits.  Barriers that the peer CTA arrives on need the cluster's scope.
template <bool CLUSTER> __device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity, uint32_t ns)
{
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_addr(bar)), "r"(parity), "r"(ns)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_addr(bar)), "r"(parity), "r"(ns)
                     : "memory");
    return ok != 0;
}

template <bool CLUSTER> __device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    if (try_wait<CLUSTER>(bar, parity, 0))
        return true;
    const unsigned long long t0 = global_timer_ns();
    for (;;) {
        if (try_wait<CLUSTER>(bar, parity, 10000))
            return true;
        if (*abort_flag)
            return false;
        if (global_timer_ns() - t0 > WAIT_LIMIT_NS) {
            *abort_flag = 1;
            atomicOr(&g_fault_word, LUCE_FAULT_TIMEOUT);
            return false;
        }
    }
}

// The same for a whole warp, one answer for every lane (.sync.aligned instructions follow).
__device__ __forceinline__ bool tc_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(0xffffffffu, tc_wait<false>(bar, parity, abort_flag));
}

// One arrival on the barrier at `bar` of cluster CTA `rank`.
template <int CG> __device__ __forceinline__ void arrive_on(uint64_t *bar, uint32_t rank)
{
    if constexpr (CG == 1) {
        mbar_arrive(bar);
    } else {
        uint32_t remote;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(bar)), "r"(rank));
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
    }
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int R> struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == R) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Whether an accumulator's chunk starts, or ends, at stage i of n: half 0
// restarts every CHUNK stages, half 1 half a chunk earlier.
template <int HALVES> __device__ __forceinline__ bool chunk_starts(int h, int i)
{
    const int o = HALVES == 2 && h == 1 ? CHUNK / 2 : 0;
    return i == 0 || (i + o) % CHUNK == 0;
}
template <int HALVES> __device__ __forceinline__ bool chunk_ends(int h, int i, int n)
{
    return i == n - 1 || chunk_starts<HALVES>(h, i + 1);
}

template <class C, typename TO> __global__ void __launch_bounds__(TC_THREADS, 1) k_linear_i8_tc(const __grid_constant__ TcArgs a)
{
    constexpr int CG = C::CG, HALVES = C::HALVES, NS = C::NS, RB = C::RB, CPW = C::CPW;
    extern __shared__ uint8_t smraw[];
    __shared__ uint64_t full[NS], rfree[NS], afull[RB], sfree[RB], dfull[2], dfree[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const uint32_t sm = (smem_addr(smraw) + 1023u) & ~1023u;
    const uint32_t smb = sm + NS * C::RAW;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int csize = CG * a.sk;
    const uint32_t rank = csize > 1 ? cluster_rank() : 0;
    const uint32_t pr = rank % CG, leader = rank - pr; // place in the pair, the pair's leader
    const int kg = (int)rank / CG;                      // place along K
    const uint16_t pair_mask = (uint16_t)(3u << leader);

    if (tid == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&rfree[i], WORKERS);
        }
        for (int i = 0; i < RB; i++) {
            mbar_init(&afull[i], WORKERS * CG);
            mbar_init(&sfree[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dfree[i], WORKERS * CG);
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                         "r"(TMEM_COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                         "r"(TMEM_COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (csize > 1)
        cluster_sync_all(); // the peers' barriers are initialised before any remote arrival
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    // this CTA's tiles: cluster c takes tiles c, c + clusters, ...; its share of K
    const int c0 = (int)(blockIdx.x / (unsigned)csize), cstep = (int)(gridDim.x / (unsigned)csize);
    const int s0 = (int)((long long)a.stages * kg / a.sk), s1 = (int)((long long)a.stages * (kg + 1) / a.sk);
    const int ns = s1 - s0; // (the host keeps sk <= stages, so that ns >= 1)
    const int nh = a.nh, xr = nh / CG;

    if (warp == TMA_WARP) {
        if (lane == 0) {
            const uint32_t bytes = (uint32_t)(C::RAW_W + HALVES * xr * KS);
            Ring<NS> r;
            int issued = 0;
            auto load_x = [&](uint32_t slot, int st, int tile) {
                const int t0 = (tile / a.mt) * (nh * HALVES);
#pragma unroll
                for (int h = 0; h < HALVES; h++)
                    tma_2d(sm + slot * C::RAW + C::RAW_W + h * (C::ROWS * KS), &a.tx, (s0 + st) * KS,
                           t0 + h * nh + (int)pr * xr, &full[slot]);
            };
            // the first tile's weights do not depend on the previous kernel
            const int early = c0 < a.tiles ? min(ns, NS) : 0;
            for (int st = 0; st < early; st++) {
                mbar_arrive_expect_tx(&full[st], bytes);
                tma_2d(sm + st * C::RAW, &a.tw, (s0 + st) * KS, ((c0 % a.mt) * CG + (int)pr) * RM, &full[st]);
            }
            pdl_wait();
            for (int st = 0; st < early; st++)
                load_x((uint32_t)st, st, c0);
            bool ok = true;
            for (int tile = c0; tile < a.tiles && ok; tile += cstep) {
                for (int st = 0; st < ns; st++, r.next(), issued++) {
                    if (issued < early)
                        continue;
                    if (!(ok = tc_wait<false>(&rfree[r.slot], r.phase ^ 1, abort_flag)))
                        break;
                    mbar_arrive_expect_tx(&full[r.slot], bytes);
                    tma_2d(sm + r.slot * C::RAW, &a.tw, (s0 + st) * KS, ((tile % a.mt) * CG + (int)pr) * RM, &full[r.slot]);
                    load_x(r.slot, st, tile);
                }
            }
            if (!ok || *abort_flag) {
                // the copies in flight land before the CTA leaves: the last NS stages issued
                for (int g = max(0, issued - NS); g < issued; g++) {
                    const unsigned long long t = global_timer_ns();
                    while (!try_wait<false>(&full[g % NS], (uint32_t)(g / NS) & 1, 1000) &&
                           !try_wait<false>(&full[g % NS], ((uint32_t)(g / NS) & 1) ^ 1, 0) &&
                           global_timer_ns() - t < WAIT_LIMIT_NS)
                        ;
                }
            }
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        pdl_wait();
        if (lane == 0 && pr == 0) {
            const uint32_t idesc = (1u << 4) | ((uint32_t)(nh >> 3) << 17) | ((uint32_t)(RM * CG >> 4) << 24);
            Ring<RB> ar;
            uint32_t dphase = 0;         // bit s: phase of accumulator slot s
            uint32_t slot = 0;           // (one half: the slots alternate)
            bool ok = true;
            for (int tile = c0; tile < a.tiles && ok; tile += cstep) {
                for (int st = 0; st < ns && ok; st++, ar.next()) {
                    if (!(ok = tc_wait<CG == 2>(&afull[ar.slot], ar.phase, abort_flag)))
                        break;
                    tc_fence_after();
                    const uint32_t bs = smb + ar.slot * C::BST, as = tmem + ar.slot * 64;
                    // the half whose accumulator is being read back goes second
                    const int first = HALVES == 2 && (chunk_starts<HALVES>(0, st) && st > 0) ? 1 : 0;
#pragma unroll
                    for (int hh = 0; hh < HALVES; hh++) {
                        const int h = HALVES == 2 ? hh ^ first : 0;
                        const bool fresh = chunk_starts<HALVES>(h, st);
                        const uint32_t ds = HALVES == 2 ? (uint32_t)h : slot;
                        if (fresh) {
                            if (!(ok = tc_wait<CG == 2>(&dfree[ds], ((dphase >> ds) & 1) ^ 1, abort_flag)))
                                break;
                            tc_fence_after();
                            dphase ^= 1u << ds;
                        }
#pragma unroll
                        for (int k = 0; k < KS / 16; k++)
                            mma_ts<CG>(tmem + D_COL + ds * C::DCOLS, as + 8 * k,
                                       sw128_desc(bs + h * 2 * C::ATOM + (k >> 2) * C::ATOM + (k & 3) * 32), idesc,
                                       !(fresh && k == 0));
                        if (chunk_ends<HALVES>(h, st, ns)) {
                            mma_commit<CG>(&dfull[ds], pair_mask);
                            if (HALVES == 1)
                                slot ^= 1;
                        }
                    }
                    if (ok)
                        mma_commit<CG>(&sfree[ar.slot], pair_mask);
                }
            }
            // every MMA issued has completed before the tensor memory is freed
            mma_commit_here<CG>(&drain);
            const unsigned long long t = global_timer_ns();
            while (!try_wait<false>(&drain, 0, 10000) && global_timer_ns() - t < WAIT_LIMIT_NS)
                ;
        }
        __syncwarp();
    } else {
        pdl_wait();
        const int q = warp & 3, kq = warp >> 2; // lane quarter; quarter of a stage's K, of an accumulator's columns
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        const int row = 32 * q + lane;
        // weights: 16-byte chunks 2 kq and 2 kq + 1 of this row, swizzled by the TMA
        const uint32_t w0 = (uint32_t)(row * KS + (((2 * kq) ^ (row & 7)) << 4));
        const uint32_t w1 = (uint32_t)(row * KS + (((2 * kq + 1) ^ (row & 7)) << 4));
        // tokens: a unit is 8 rows x 64 values; a quarter-warp takes rows p and
        // p ^ 5 and four chunks, which touches all banks once in the raw tile
        // and once in the converted one
        const int xrow = ((lane >> 2) & 1) ? ((lane >> 3) ^ 5) : (lane >> 3), xc = lane & 3;
        const int units = HALVES * (xr >> 3) * 2;
        Ring<NS> rr;
        Ring<RB> ar;
        int acc[HALVES][CPW];
        uint32_t dph = 0; // bit s: phase of accumulator slot s
        uint32_t slot = 0;
        const int lag = min(LAG, ns);
        int done_tile = -1; // tile whose last chunks are still to be read back
        bool ok = true;

        // reads accumulator `ds` back into acc[h] (set, or added to)
        auto read_back = [&](int h, uint32_t ds, bool set) {
            if (!tc_wait_warp(&dfull[ds], (dph >> ds) & 1, abort_flag))
                return false;
            tc_fence_after();
            dph ^= 1u << ds;
#pragma unroll
            for (int c = 0; c < CPW; c += 16) {
                uint32_t v[16];
                tmem_ld16(tl + D_COL + ds * C::DCOLS + kq * CPW + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int x = __float2int_rn(__uint_as_float(v[i]));
                    if (h == 0 || HALVES == 1)
                        acc[0][c + i] = set ? x : acc[0][c + i] + x;
                    else
                        acc[HALVES - 1][c + i] = set ? x : acc[HALVES - 1][c + i] + x;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_on<CG>(&dfree[ds], leader);
            return true;
        };
        auto store_tile = [&](int tile) {
            const int n = ((tile % a.mt) * CG + (int)pr) * RM + row;
            const int t0 = (tile / a.mt) * (nh * HALVES);
            if (n < a.N) {
                const float wsn = a.ws[n];
                TO *o = static_cast<TO *>(a.out) + n;
#pragma unroll
                for (int h = 0; h < HALVES; h++)
#pragma unroll
                    for (int c = 0; c < CPW; c++) {
                        const int j = kq * CPW + c, t = t0 + h * nh + j;
                        if (j < nh && t < a.T)
                            store_out(o + (size_t)t * a.ldo, epilogue(acc[h][c], __ldg(a.xs + t), wsn, a.bias, n));
                    }
            }
        };
        // the chunks that ended at stage i of a tile (n stages)
        auto read_backs = [&](int i) {
#pragma unroll
            for (int h = 0; h < HALVES; h++)
                if (chunk_ends<HALVES>(h, i, ns)) {
                    const int start = HALVES == 2 && h == 1 ? CHUNK / 2 : CHUNK;
                    if (!read_back(h, HALVES == 2 ? (uint32_t)h : slot, i < start))
                        return false;
                    if (HALVES == 1)
                        slot ^= 1;
                }
            return true;
        };

        for (int tile = c0; tile < a.tiles && ok; tile += cstep) {
            for (int st = 0; st < ns; st++, rr.next(), ar.next()) {
                if (!(ok = tc_wait_warp(&full[rr.slot], rr.phase, abort_flag)))
                    break;
                if (!(ok = tc_wait_warp(&sfree[ar.slot], ar.phase ^ 1, abort_flag)))
                    break;
                tc_fence_after();
                const uint32_t raw = sm + rr.slot * C::RAW, bst = smb + ar.slot * C::BST;
                {
                    const uint4 v0 = lds128(raw + w0), v1 = lds128(raw + w1);
                    uint32_t h8[8];
                    codes16(v0, h8);
                    tmem_st8(tl + ar.slot * 64 + kq * 16, h8);
                    codes16(v1, h8);
                    tmem_st8(tl + ar.slot * 64 + kq * 16 + 8, h8);
                }
                for (int u = warp; u < units; u += WORKERS) {
                    const int at = u & 1, grp = u >> 1;              // 64-value atom, 8-row group
                    const int h = HALVES == 2 ? grp / (xr >> 3) : 0; // half
                    const int r8 = (HALVES == 2 ? grp % (xr >> 3) : grp) * 8;
                    const uint32_t src = raw + C::RAW_W + h * (C::ROWS * KS) + (r8 + xrow) * KS +
                                         (((4 * at + xc) ^ xrow) << 4);
                    const uint32_t dst = bst + h * 2 * C::ATOM + at * C::ATOM + (r8 + xrow) * 128;
                    uint32_t h8[8];
                    codes16(lds128(src), h8);
                    sts128(dst + (((2 * xc) ^ xrow) << 4), h8[0], h8[1], h8[2], h8[3]);
                    sts128(dst + (((2 * xc + 1) ^ xrow) << 4), h8[4], h8[5], h8[6], h8[7]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // the tensor core reads the tokens
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    arrive_on<CG>(&afull[ar.slot], leader);
                    mbar_arrive(&rfree[rr.slot]);
                }
                // what ended `lag` stages ago, so that the MMAs have converted stages ahead of them meanwhile
                if (st >= lag) {
                    if (!(ok = read_backs(st - lag)))
                        break;
                } else if (done_tile >= 0) {
                    if (!(ok = read_backs(ns - lag + st)))
                        break;
                    if (st == lag - 1)
                        store_tile(done_tile);
                }
            }
            done_tile = tile;
        }
        for (int i = ns - lag; i < ns && ok && done_tile >= 0; i++)
            ok = read_backs(i);
        if (ok && done_tile >= 0) {
            if (a.sk == 1) {
                store_tile(done_tile);
            } else {
                // the int32 sums, [half][token][channel], where the stages were
                int *part = reinterpret_cast<int *>(smraw + (sm - smem_addr(smraw)));
#pragma unroll
                for (int h = 0; h < HALVES; h++)
#pragma unroll
                    for (int c = 0; c < CPW; c++)
                        part[(h * C::DCOLS + kq * CPW + c) * RM + row] = acc[h][c];
            }
        }
    }

    if (a.sk > 1) {
        // every group's sums are in shared memory; each group adds its share of the tokens
        __syncwarp();
        cluster_sync_all();
        const int tile = c0; // (one tile per cluster)
        const int n0 = ((tile % a.mt) * CG + (int)pr) * RM, t0 = (tile / a.mt) * (nh * HALVES);
        const int nt = min(nh * HALVES, a.T - t0);
        const int quads = RM / 4;
        if (!abort_word) {
            for (int i = tid; i < ((nt - kg + a.sk - 1) / a.sk) * quads; i += TC_THREADS) {
                const int j = kg + (i / quads) * a.sk, r4 = (i % quads) * 4; // token of the tile, four channels
                const int col = HALVES == 2 && j >= nh ? C::DCOLS + j - nh : j;
                int4 s = make_int4(0, 0, 0, 0);
                for (int g = 0; g < a.sk; g++) {
                    uint32_t remote;
                    int4 v;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                 : "=r"(remote)
                                 : "r"(sm + (uint32_t)((col * RM + r4) * 4)), "r"((uint32_t)(g * CG) + pr));
                    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(remote)
                                 : "memory");
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                const int t = t0 + j, n = n0 + r4;
                const float xst = a.xs[t];
                TO *o = static_cast<TO *>(a.out) + (size_t)t * a.ldo + n;
                const int sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (n + e < a.N)
                        store_out(o + e, epilogue(sv[e], xst, a.ws[n + e], a.bias, n + e));
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (csize > 1)
        cluster_sync_all(); // no CTA leaves while a peer reads its memory or signals its barriers
    tc_fence_after();
    if (warp == MMA_WARP) {
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
    }
}

using CfgSmall = Cfg<1, 1, 64, 6, 4>; // up to 64 tokens to a tile, one CTA
using CfgPair = Cfg<2, 1, 64, 6, 4>;  // up to 128, a CTA pair
using CfgWide = Cfg<2, 2, 64, 4, 3>;  // up to 256, a CTA pair

// ---------------------------------------------------------------------------
// Host side.
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else
            (void)cudaGetLastError();
    });
    return fn;
}

// int8 rows [rows][K]; box = 128 values x `box_rows`, 128-byte swizzle (what lies outside reads as zero).
bool map_codes(CUtensorMap *m, const int8_t *base, int rows, int K, int box_rows)
{
    EncodeTiledFn f = encode_tiled();
    if (!f)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {KS, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C, typename TO>
luce_status launch_tc(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int T,
                      int N, int K, TO *out, int64_t ldo, int nh, int sk, cudaStream_t stream)
{
    static luce_host::SmemLimit limit;
    auto kern = k_linear_i8_tc<C, TO>;
    TcArgs a;
    a.xs = xs;
    a.ws = ws;
    a.bias = bias;
    a.out = out;
    a.ldo = ldo;
    a.T = T;
    a.N = N;
    a.stages = (K + KS - 1) / KS;
    a.nh = nh;
    a.mt = (N + RM * C::CG - 1) / (RM * C::CG);
    const int64_t tt = ((int64_t)T + nh * C::HALVES - 1) / (nh * C::HALVES);
    if (a.mt * tt > INT_MAX / SK_MAX)
        return LUCE_ERR_UNSUPPORTED;
    a.tiles = (int)(a.mt * tt);
    a.sk = sk;
    if (!map_codes(&a.tw, wq, N, K, RM) || !map_codes(&a.tx, xq, T, K, nh / C::CG))
        return LUCE_ERR_CUDA;
    if (limit.raise(kern, C::SMEM) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_UNSUPPORTED;
    }
    const int csize = C::CG * sk;
    const int clusters = sk > 1 ? a.tiles : std::min(a.tiles, luce_host::sm_count() / C::CG);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    luce_host::make_config(cfg, attr, dim3((unsigned)(clusters * csize)), dim3(TC_THREADS), C::SMEM, stream);
    if (csize > 1) {
        cudaLaunchAttribute &c = attr[cfg.numAttrs++];
        c.id = cudaLaunchAttributeClusterDimension;
        c.val.clusterDim.x = (unsigned)csize;
        c.val.clusterDim.y = c.val.clusterDim.z = 1;
    }
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        (void)cudaGetLastError();
        limit.forget();
        return LUCE_ERR_CUDA;
    }
    return LUCE_OK;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

template <typename TO>
luce_status run_linear(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int T,
                       int N, int K, TO *out, int64_t ldo, cudaStream_t stream)
{
    if (T > TPW) {
        // token tiles of at most 64, 128 or 256, all of one width
        const int stages = (K + KS - 1) / KS;
        auto width = [](int tokens, int most) { // tokens of a tile, a multiple of 16, all tiles alike
            const int n = (tokens + most - 1) / most;
            return ((tokens + n - 1) / n + 15) & ~15;
        };
        auto split = [&](int64_t ctas, int cg) { // groups along K while SMs are idle
            int sk = 1;
            while (sk * 2 * cg <= SK_MAX && ctas * sk * 2 <= luce_host::sm_count() && sk * 2 <= stages)
                sk *= 2;
            return sk;
        };
        const int64_t mt = ((int64_t)N + RM - 1) / RM;
        if (T <= 64) {
            const int nh = width(T, 64);
            return launch_tc<CfgSmall>(xq, xs, wq, ws, bias, T, N, K, out, ldo, nh, split(mt, 1), stream);
        }
        if (T <= 128) {
            const int nh = width(T, 128);
            return launch_tc<CfgPair>(xq, xs, wq, ws, bias, T, N, K, out, ldo, nh, split((mt + 1) / 2 * 2, 2), stream);
        }
        const int nh = (width(T, 256) / 2 + 15) & ~15, tt = (T + 2 * nh - 1) / (2 * nh);
        return launch_tc<CfgWide>(xq, xs, wq, ws, bias, T, N, K, out, ldo, nh, split((mt + 1) / 2 * 2 * tt, 2), stream);
    }
    const int64_t nb = ((int64_t)N + WARPS - 1) / WARPS;
    // tokens in slices of at most 65,535 tiles, the grid's limit in y
    for (int t0 = 0; t0 < T;) {
        const int n = std::min(T - t0, 65535 * TPW);
        const luce_status st =
            luce_host::launch(k_linear_i8_rows<TO>, dim3((unsigned)nb, (unsigned)((n + TPW - 1) / TPW)),
                              dim3(WARPS * 32), 0, stream, xq + (size_t)t0 * K, xs + t0, wq, ws, bias, n, N, K,
                              out + (size_t)t0 * ldo, ldo);
        if (st != LUCE_OK)
            return st;
        t0 += n;
    }
    return LUCE_OK;
}

} // namespace

extern "C" luce_status luce_linear_i8(const int8_t *xq, const float *x_scale, const int8_t *wq, const float *w_scale,
                                      const float *bias, int T, int N, int K, void *out, luce_dtype out_dtype,
                                      int64_t ld_out, void *stream)
{
    using luce_host::aligned;
    if (T < 0 || T >= (1 << 24) || N < 1 || N >= (1 << 24) || K < 16 || K > 65536 || K % 16 != 0 || ld_out < N ||
        ld_out > ((int64_t)1 << 32) ||
        (out_dtype != LUCE_F32 && out_dtype != LUCE_BF16 && out_dtype != LUCE_F16))
        return LUCE_ERR_INVALID_ARG;
    if (T == 0)
        return LUCE_OK;
    const size_t es = out_dtype == LUCE_F32 ? 4 : 2;
    if (!xq || !x_scale || !wq || !w_scale || !out || !aligned(xq, 16) || !aligned(wq, 16) || !aligned(x_scale, 4) ||
        !aligned(w_scale, 4) || (bias && !aligned(bias, 4)) || !aligned(out, es))
        return LUCE_ERR_INVALID_ARG;
    const size_t no = ((size_t)(T - 1) * ld_out + N) * es;
    if (overlap(out, no, xq, (size_t)T * K) || overlap(out, no, wq, (size_t)N * K) ||
        overlap(out, no, x_scale, (size_t)T * 4) || overlap(out, no, w_scale, (size_t)N * 4) ||
        (bias && overlap(out, no, bias, (size_t)N * 4)))
        return LUCE_ERR_INVALID_ARG;
    cudaStream_t st = luce_host::as_stream(stream);
    switch (out_dtype) {
    case LUCE_F32:
        return run_linear(xq, x_scale, wq, w_scale, bias, T, N, K, (float *)out, ld_out, st);
    case LUCE_BF16:
        return run_linear(xq, x_scale, wq, w_scale, bias, T, N, K, (__nv_bfloat16 *)out, ld_out, st);
    case LUCE_F16:
        return run_linear(xq, x_scale, wq, w_scale, bias, T, N, K, (__half *)out, ld_out, st);
    }
    return LUCE_ERR_INVALID_ARG;
}
