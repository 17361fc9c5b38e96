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
__device__ __forceinline__ float epilogue(float isum, float xs, float ws, bool add, float bias)
{
    const float v = __fmul_rn(isum, __fmul_rn(xs, ws));
    return add ? __fadd_rn(v, bias) : v;
}
__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(__half *p, float v) { *p = __float2half_rn(v); }

// ---------------------------------------------------------------------------
// Few tokens (T of them at a time): a stream of the weights through dp4a.
//
// What bounds it is the weights' way from HBM, and for small matrices the
// latency of getting there.  A warp takes VR channels and a slice of K, 16
// bytes a lane and load; the wk warps of a row group split K and add their
// int32 sums through shared memory (exact, so any split gives the same bits).
// Slices are one batch of VU x VR loads wherever eight warps are enough for K:
// every load is then in flight at once, and without the registers for a next
// batch four CTAs fit an SM instead of two (1 x 129280 x 4096: 74.0 us, 7.16
// TB/s; with slices of 4096 and the next batch requested ahead, which longer
// rows still do, 79.3 us; 1 x 4096 x 4096: 4.7 against 6.2 us).  The tokens'
// codes come through L1 (VR channels share each load).
constexpr int VR = 4;      // channels of a warp
constexpr int V_WARPS = 8; // warps of a CTA

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Sums over a warp's lanes of V values (a power of two): each step sends half
// of the values one way and keeps the other half.  Lane l ends with the sum of
// value l >> log2(32 / V), in every lane that shares it.
template <int V> __device__ __forceinline__ int warp_sums(int (&v)[V], int lane)
{
    int o = 16;
#pragma unroll
    for (int n = V; n > 1; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; i++) {
            const int keep = up ? v[i + n / 2] : v[i], give = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    int s = v[0];
    for (; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <int T, int VU, bool MORE, typename TO>
__global__ void __launch_bounds__(V_WARPS * 32)
    k_linear_i8_vec(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int nt,
                    int N, int K, int wk, TO *out, int64_t ldo)
{
    constexpr int V = VR * T;
    __shared__ int part[V_WARPS][V];
    const int t0 = (int)blockIdx.y * T; // this CTA's tokens
    xq += (size_t)t0 * K;
    xs += t0;
    out += (size_t)t0 * ldo;
    nt = min(nt - t0, T);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = V_WARPS / wk, kw = warp % wk; // row groups of the CTA, this warp's place along K
    const int64_t n0 = ((int64_t)blockIdx.x * groups + warp / wk) * VR;
    const int slice = ((K >> 4) + wk - 1) / wk << 4;
    const int k1 = min(K, (kw + 1) * slice);
    const int8_t *w[VR];
#pragma unroll
    for (int r = 0; r < VR; r++)
        w[r] = wq + (size_t)min(n0 + r, (int64_t)N - 1) * K;
    uint4 cur[VU][VR];
    auto load = [&](uint4 (&b)[VU][VR], int k) {
#pragma unroll
        for (int u = 0; u < VU; u++)
#pragma unroll
            for (int r = 0; r < VR; r++)
                b[u][r] = k + 512 * u < k1 ? ldg_stream(w[r] + k + 512 * u) : make_uint4(0, 0, 0, 0);
    };
    pdl_wait(); // (the weights too may be the previous kernel's: luce_quantize_i8 writes them)
    pdl_trigger();
    load(cur, kw * slice + 16 * lane);
    int acc[V] = {};
    auto use = [&](int k) {
#pragma unroll
        for (int u = 0; u < VU; u++) {
            if (k + 512 * u < k1) {
#pragma unroll
                for (int t = 0; t < T; t++) {
                    const int4 x = *reinterpret_cast<const int4 *>(xq + (size_t)min(t, nt - 1) * K + k + 512 * u);
#pragma unroll
                    for (int r = 0; r < VR; r++) {
                        int s = acc[r * T + t];
                        s = __dp4a((int)cur[u][r].x, x.x, s);
                        s = __dp4a((int)cur[u][r].y, x.y, s);
                        s = __dp4a((int)cur[u][r].z, x.z, s);
                        acc[r * T + t] = __dp4a((int)cur[u][r].w, x.w, s);
                    }
                }
            }
        }
    };
    if constexpr (MORE) {
        for (int k0 = kw * slice; k0 < k1; k0 += 512 * VU) {
            const int k = k0 + 16 * lane;
            uint4 next[VU][VR];
            load(next, k + 512 * VU);
            use(k);
#pragma unroll
            for (int u = 0; u < VU; u++)
#pragma unroll
                for (int r = 0; r < VR; r++)
                    cur[u][r] = next[u][r];
        }
    } else {
        use(kw * slice + 16 * lane);
    }
    const int s = warp_sums<V>(acc, lane);
    if (lane % (32 / V) == 0)
        part[warp][lane / (32 / V)] = s;
    __syncthreads();
    // value r T + t of each row group, in its order along the output row
    for (int i = threadIdx.x; i < groups * V; i += V_WARPS * 32) {
        const int t = i / (groups * VR), c = i % (groups * VR), g = c / VR, r = c % VR;
        const int64_t n = ((int64_t)blockIdx.x * groups + g) * VR + r;
        if (n < N && t < nt) {
            int sum = 0;
            for (int j = 0; j < wk; j++)
                sum += part[g * wk + j][r * T + t];
            store_out(out + (size_t)t * ldo + n, epilogue(sum, xs[t], ws[n], bias != nullptr, bias ? bias[n] : 0.0f));
        }
    }
}

// ---------------------------------------------------------------------------
// The product on the tensor cores (more than a few tokens).
//
// Exactness.  tcgen05.mma has no int8 kind on this GPU, so the codes go in as
// fp16: every code is an exact fp16 number, and the partial sums of up to 1024
// products (at most 1024 * 2^14 = 2^24) are exact fp32 integers.  Every CHUNK
// units an accumulator is read back, converted to int32 and added to the
// int32 sums that the epilogue warps hold, and the next chunk starts from
// zero: the result is the int32 sum, bit for bit.
//
// Operands.  A = 128 weight rows per CTA, converted into tensor memory (a
// thread writes its own lane's row); B = the tokens, converted into shared
// memory in the tensor core's 128-byte-swizzled K-major layout; D[channel,
// token].  Codes cross HBM and L2 as int8 and are converted once per tile.
// What bounds a tile is the 128 B/clock of shared memory: per 64 values of K,
// 8 + 8 KB of weights in and out, and 8 + 8 + 16 + 16 KB for 128 token rows
// (raw in and out, converted in and out to the tensor core).  A CTA pair
// (CG = 2) shares a tile of 256 channels, so that each CTA holds only half of
// the tokens: 512 clocks for 256 tokens, whose MMAs take 512 too, and 320 for
// up to 128 tokens, where the weights' 8 KB take 356 clocks of HBM.
//
// Reading an accumulator back takes 64 to 128 values per thread, bound by the
// float-to-int conversions (16 a clock and SM: about 1000 clocks for 128
// columns), so it overlaps MMAs: up to 128 tokens the two accumulator slots
// alternate chunk by chunk; beyond, a tile has two halves of up to 128 tokens
// (HALVES = 2), a slot each, whose chunks end half a chunk apart, and the MMAs
// go through blocks of BLOCK units one half at a time, in an order that leaves
// two blocks of the other half between a chunk's end and its slot's next use.
//
// Few tiles: sk CTA groups of one cluster split K among them and add their
// int32 sums through distributed shared memory (any split gives the same
// bits).
//
// Roles: warp 0 issues the TMA tiles, warp 1 the MMAs (of the pair, in its
// leader); GROUPS groups of four warps convert, every GROUPS-th unit each (a
// warp its lane quarter of A and a quarter of B); eight epilogue warps read
// accumulators back (lane quarter w & 3, half of the columns) and store, while
// the next tile's products run.  The epilogue's sums need more registers than
// an even share, so warpgroups trade them with setmaxnreg; the shares add up
// to no more than the launch's (static_assert below).
// Every wait is bounded: a role that gives up raises LUCE_FAULT_TIMEOUT and
// the CTA's abort flag, the others leave at their next wait, copies and MMAs
// in flight are waited for (bounded) and tensor memory is freed.
constexpr int SK_MAX = 8;        // CTAs of one cluster at most
constexpr int EARLY = 2;         // stages of the first tile requested ahead of the CTA's other preparations
constexpr int KU = 128;          // K values of a unit: a TMA stage, what a group converts, and eight MMAs per half
constexpr int CHUNK = 1024 / KU; // units whose sums fit fp32
constexpr int BLOCK = 2;         // (half a chunk is two blocks)
constexpr int RM = 128;          // weight rows per CTA
constexpr int ROWS = 64;         // token rows per half and CTA, at most
constexpr int TMA_WARP = 0, MMA_WARP = 1, CONV_WARP0 = 4, EPI_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512;
constexpr int ACOLS = KU / 2;    // tensor-memory columns of a unit of A
constexpr uint32_t D_COL = 256;
constexpr int REGS_MISC = 40;
constexpr int PITCH = RM + 4;    // of the int32 sums [token][channel] in shared memory, without bank conflicts

template <int CG_, int HALVES_, int GROUPS_, int NS_, int RB_, int LAUNCH_REGS, int REGS_CONV_, int REGS_EPI_> struct Cfg {
    static constexpr int CG = CG_, HALVES = HALVES_, GROUPS = GROUPS_;
    static constexpr int NS = NS_, RB = RB_; // raw stages, converted units (A and B slots)
    static constexpr int REGS_CONV = REGS_CONV_, REGS_EPI = REGS_EPI_;
    static constexpr int EPI_WARP0 = CONV_WARP0 + 4 * GROUPS;
    static constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
    static constexpr int DCOLS = ROWS * CG;  // columns of an accumulator slot
    static constexpr int ECOLS = DCOLS / 2;  // of an epilogue warp
    static constexpr int RAW_W = RM * KU, RAW_X = ROWS * KU;
    static constexpr int RAW = RAW_W + HALVES * RAW_X;
    static constexpr int BATOM = ROWS * 128; // 64 values of K of one half's tokens, fp16
    static constexpr int BHALF = 2 * BATOM;
    static constexpr int BST = HALVES * BHALF;
    static constexpr int SMEM = NS * RAW + RB * BST + 1024;
    static_assert(RB * ACOLS <= (int)D_COL && D_COL + 2 * DCOLS <= TMEM_COLS, "tensor memory");
    static_assert(RAW % 1024 == 0 && BHALF % 1024 == 0, "swizzle atoms");
    static_assert(HALVES * DCOLS * PITCH * 4 <= NS * RAW + RB * BST && SMEM <= 232448, "shared memory");
    static_assert(NS > GROUPS && RB > GROUPS && (HALVES == 1 || RB >= 2 * BLOCK), "slots");
    static_assert(128 * REGS_MISC + 128 * GROUPS * REGS_CONV + 256 * REGS_EPI <= THREADS * LAUNCH_REGS &&
                      THREADS * LAUNCH_REGS <= 65536,
                  "register shares");
};

struct TcArgs {
    CUtensorMap tw, tx; // int8 [N][K], box 128 x 128; int8 [T][K], box 128 x rows; 128-byte swizzle
    const float *xs, *ws, *bias;
    void *out;
    int64_t ldo;
    int T, N, units;  // units of the whole K
    int xbox;         // token rows of a box
    int nb, nh[2];    // tokens of a tile, and of its halves (multiples of 16, of 32 for a pair)
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

// Waits.  Barriers that the peer CTA arrives on need the cluster's scope.  A
// poll parks the thread in hardware for a while; the timer, which is slow to
// read, is looked at every 64 polls only.
template <bool CLUSTER> __device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_addr(bar)), "r"(parity)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_addr(bar)), "r"(parity)
                     : "memory");
    return ok != 0;
}

template <bool CLUSTER> __device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    unsigned long long t0 = 0;
    for (uint32_t i = 1;; i++) {
        if (try_wait<CLUSTER>(bar, parity))
            return true;
        if ((i & 63u) == 0) {
            if (*abort_flag)
                return false;
            const unsigned long long t = global_timer_ns();
            if (t0 == 0)
                t0 = t;
            if (t - t0 > WAIT_LIMIT_NS) {
                *abort_flag = 1;
                atomicOr(&g_fault_word, LUCE_FAULT_TIMEOUT);
                return false;
            }
        }
    }
}

// A wait for what is in flight when the CTA leaves: bounded, whatever the abort flag says.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity)
{
    const unsigned long long t0 = global_timer_ns();
    while (!try_wait<false>(bar, parity) && global_timer_ns() - t0 < WAIT_LIMIT_NS)
        ;
}

// The same for a whole warp, one answer for every lane (.sync.aligned instructions follow).
template <bool CLUSTER = false>
__device__ __forceinline__ bool tc_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(0xffffffffu, tc_wait<CLUSTER>(bar, parity, abort_flag));
}

// One arrival on the barrier at `bar` of cluster CTA `rank`, of the cluster's
// scope where that may be another one.  What it orders is this CTA's shared
// memory (tensor memory has the tcgen05 fences), so the fence is restricted to
// that: a release of everything takes 4093 x 4096 x 4096 from 87.9 to 110.7 us.
template <int CG> __device__ __forceinline__ void arrive_on(uint64_t *bar, uint32_t rank)
{
    if constexpr (CG == 1) {
        mbar_arrive(bar);
    } else {
        uint32_t remote;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(bar)), "r"(rank));
        asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
    }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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

// Whether half h's chunk starts, or ends, at unit u of nu: half 0 restarts
// every CHUNK units, half 1 half a chunk earlier.
template <int HALVES> __device__ __forceinline__ bool chunk_starts(int h, int u)
{
    return u == 0 || ((u + (HALVES == 2 && h == 1 ? CHUNK / 2 : 0)) & (CHUNK - 1)) == 0;
}
template <int HALVES> __device__ __forceinline__ bool chunk_ends(int h, int u, int nu)
{
    return u == nu - 1 || chunk_starts<HALVES>(h, u + 1);
}

template <class C, typename TO>
__global__ void __launch_bounds__(C::THREADS, 1) k_linear_i8_tc(const __grid_constant__ TcArgs a)
{
    constexpr int CG = C::CG, HALVES = C::HALVES, GROUPS = C::GROUPS, NS = C::NS, RB = C::RB, ECOLS = C::ECOLS;
    extern __shared__ uint8_t smraw[];
    __shared__ uint64_t full[NS], rfree[NS], afull[RB], sfree[RB], dfull[2], dfree[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const uint32_t sm = (smem_addr(smraw) + 1023u) & ~1023u;
    const uint32_t smb = sm + NS * C::RAW;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int csize = CG * a.sk;
    const uint32_t rank = csize > 1 ? cluster_rank() : 0;
    const uint32_t pr = rank % CG, leader = rank - pr; // place in the pair, the pair's leader
    const int kg = (int)rank / CG;                      // place along K
    const uint16_t pair_mask = (uint16_t)(3u << leader);

    // this CTA's tiles: cluster c takes tiles c, c + clusters, ...; its share of K
    const int c0 = (int)(blockIdx.x / (unsigned)csize), cstep = (int)(gridDim.x / (unsigned)csize);
    const int u0 = (int)((long long)a.units * kg / a.sk), u1 = (int)((long long)a.units * (kg + 1) / a.sk);
    const int nu = u1 - u0; // (the host keeps sk <= units, so that nu >= 1)
    auto w_row = [&](int tile) { return ((tile % a.mt) * CG + (int)pr) * RM; };
    auto x_tile = [&](int tile) { return (tile / a.mt) * a.nb; };
    const uint32_t bytes = (uint32_t)(C::RAW_W + HALVES * a.xbox * KU);
    auto load_w = [&](uint32_t slot, int st, int wr) {
        mbar_arrive_expect_tx(&full[slot], bytes);
        tma_2d(sm + slot * C::RAW, &a.tw, (u0 + st) * KU, wr, &full[slot]);
    };
    auto load_x = [&](uint32_t slot, int st, int xt) {
        tma_2d(sm + slot * C::RAW + C::RAW_W, &a.tx, (u0 + st) * KU, xt + (int)pr * (a.nh[0] / CG), &full[slot]);
        if constexpr (HALVES == 2)
            tma_2d(sm + slot * C::RAW + C::RAW_W + C::RAW_X, &a.tx, (u0 + st) * KU,
                   xt + a.nh[0] + (int)pr * (a.nh[1] / CG), &full[slot]);
    };
    const int early = c0 < a.tiles ? min(nu, EARLY) : 0; // stages requested before anything else is set up

    if (warp == TMA_WARP) {
        // the first stages: their barriers are this CTA's own; weights and tokens
        // alike may be the previous kernel's
        if (elect_one()) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.tw)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.tx)) : "memory");
            for (int i = 0; i < NS; i++)
                mbar_init(&full[i], 1);
            fence_mbar_init();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        pdl_wait();
        if (elect_one())
            for (int st = 0; st < early; st++) {
                load_w((uint32_t)st, st, w_row(c0));
                load_x((uint32_t)st, st, x_tile(c0));
            }
    }
    if (tid == CONV_WARP0 * 32) {
        for (int i = 0; i < NS; i++)
            mbar_init(&rfree[i], 4);
        for (int i = 0; i < RB; i++) {
            mbar_init(&afull[i], 4 * CG);
            mbar_init(&sfree[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dfree[i], EPI_WARPS * CG);
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
    // the cluster's CTAs run and their barriers are initialised (made visible by
    // fence.mbarrier_init) before any remote access: each role waits for that
    // where it first needs it
    if (csize > 1)
        cluster_arrive_relaxed();
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    if (warp < CONV_WARP0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_MISC));
        // Both loops run warp-wide, with uniform control flow, and elect one lane
        // where something is issued: the operands then stay in uniform registers.
        if (warp == TMA_WARP) {
            Ring<NS> r;
            int issued = 0;
            bool ok = true;
            for (int tile = c0; tile < a.tiles && ok; tile += cstep) {
                const int wr = w_row(tile), xt = x_tile(tile);
                for (int st = 0; st < nu; st++, r.next(), issued++) {
                    if (issued < early)
                        continue;
                    if (!(ok = tc_wait_warp(&rfree[r.slot], r.phase ^ 1, abort_flag)))
                        break;
                    if (elect_one()) {
                        load_w(r.slot, st, wr);
                        load_x(r.slot, st, xt);
                    }
                }
            }
            if (!ok || *abort_flag) {
                // the copies in flight land before the CTA leaves: the last NS stages issued
                for (int g = max(0, issued - NS); g < issued; g++)
                    wait_out(&full[g % NS], (uint32_t)(g / NS) & 1);
            }
        } else if (warp == MMA_WARP && pr == 0) {
            if constexpr (CG == 2)
                cluster_wait();
            constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(RM * CG >> 4) << 24); // fp16 x fp16 -> fp32
            const uint32_t idesc0 = IDESC | ((uint32_t)(a.nh[0] >> 3) << 17), idesc1 = IDESC | ((uint32_t)(a.nh[1] >> 3) << 17);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t desc0 = sw128_desc(smb);
            uint32_t pos = 0, phase = 0; // ring position of the block's first unit
            uint32_t dphase = 3;         // bit s: parity of slot s's next wait
            uint32_t slot = 0;           // (one half: the slots alternate)
            bool ok = true;
            for (int tile = c0; tile < a.tiles && ok; tile += cstep) {
                for (int b = 0; b * BLOCK < nu && ok; b++) {
                    const int n = min(BLOCK, nu - b * BLOCK);
                    // half 0 restarts at blocks 0, 4, 8 .., half 1 at 2, 6 ..: the half that does not goes first
                    const int first = HALVES == 2 && b > 0 && (b & 3) < 2 ? 1 : 0;
#pragma unroll 1
                    for (int hh = 0; hh < HALVES && ok; hh++) {
                        const int h = HALVES == 2 ? hh ^ first : 0;
                        const uint32_t idesc = h ? idesc1 : idesc0;
                        uint32_t at = pos, ph = phase;
#pragma unroll 1
                        for (int j = 0; j < n; j++) {
                            const int u = b * BLOCK + j;
                            const bool fresh = chunk_starts<HALVES>(h, u);
                            const uint32_t ds = HALVES == 2 ? (uint32_t)h : slot;
                            if (fresh) {
                                if (!(ok = tc_wait_warp<CG == 2>(&dfree[ds], (dphase >> ds) & 1, abort_flag)))
                                    break;
                                dphase ^= 1u << ds;
                            }
                            if (hh == 0 && !(ok = tc_wait_warp<CG == 2>(&afull[at], ph, abort_flag)))
                                break;
                            tc_fence_after();
                            const uint32_t as = tm + at * ACOLS, dd = tm + D_COL + ds * C::DCOLS;
                            const uint64_t bd = desc0 + ((at * C::BST + (uint32_t)h * C::BHALF) >> 4);
                            const bool ends = chunk_ends<HALVES>(h, u, nu);
                            if (elect_one()) {
                                mma_ts<CG>(dd, as, bd, idesc, !fresh);
#pragma unroll
                                for (int k = 1; k < KU / 16; k++)
                                    mma_ts<CG>(dd, as + 8 * k, bd + ((k >> 2) * C::BATOM >> 4) + 2 * (k & 3), idesc, true);
                                if (hh == HALVES - 1)
                                    mma_commit<CG>(&sfree[at], pair_mask);
                                if (ends)
                                    mma_commit<CG>(&dfull[ds], pair_mask);
                            }
                            if (HALVES == 1 && ends)
                                slot ^= 1;
                            if (++at == RB) {
                                at = 0;
                                ph ^= 1;
                            }
                        }
                        if (hh == HALVES - 1) {
                            pos = at;
                            phase = ph;
                        }
                    }
                }
            }
            // every MMA issued has completed before the tensor memory is freed
            if (elect_one())
                mma_commit_here<CG>(&drain);
            wait_out(&drain, 0);
        }
        __syncwarp();
        if (csize > 1 && !(CG == 2 && warp == MMA_WARP && pr == 0))
            cluster_wait();
        if (a.sk > 1)
            cluster_sync_all(); // (the epilogue's exchange)
    } else if (warp < C::EPI_WARP0) {
        // ------------------------------------------------------------ converters
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONV));
        const int q = warp & 3, grp = (warp - CONV_WARP0) >> 2;
        const int row = 32 * q + lane;
        const uint32_t ta = tmem + ((uint32_t)(32 * q) << 16);
        // tokens: a warp's step is 8 rows x 128 values; a quarter-warp takes rows
        // p and p ^ 5 and four 16-byte chunks, which touches every bank once in
        // the raw tile and once in the converted one
        const int xrow = ((lane >> 2) & 1) ? ((lane >> 3) ^ 5) : (lane >> 3), xc = lane & 3;
        const uint32_t x_d0 = (uint32_t)(xrow * 128 + (((2 * xc) ^ xrow) << 4));
        const uint32_t x_d1 = (uint32_t)(xrow * 128 + (((2 * xc + 1) ^ xrow) << 4));
        const int mytiles = c0 < a.tiles ? (a.tiles - c0 + cstep - 1) / cstep : 0;
        const int total = mytiles * nu; // units of all tiles, in order
        bool peers_ready = csize == 1;
        uint32_t rslot = (uint32_t)grp, rphase = 0, aslot = (uint32_t)grp, aphase = 1;
        for (int g = grp; g < total; g += GROUPS) {
            // A parity names a phase only to who knows the one before it to be over.
            // The slot's last stage belonged to this group only if GROUPS divides NS;
            // else it may still be on its way (TMA tiles land out of order), so its
            // conversion is waited for first.  (That of the stage before it is over:
            // the stage this group converted last was requested after it.)
            if (NS % GROUPS != 0 && !tc_wait_warp(&rfree[rslot], rphase ^ 1, abort_flag))
                break;
            if (!tc_wait_warp(&full[rslot], rphase, abort_flag) || !tc_wait_warp<CG == 2>(&sfree[aslot], aphase, abort_flag))
                break;
            tc_fence_after();
            const uint32_t raw = sm + rslot * C::RAW, bst = smb + aslot * C::BST;
#pragma unroll
            for (int c0 = 0; c0 < 8; c0 += 4) {
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; c++)
                    v[c] = lds128(raw + row * KU + (((c0 + c) ^ (row & 7)) << 4));
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    uint32_t h8[8];
                    codes16(v[c], h8);
                    tmem_st8(ta + aslot * ACOLS + 8 * (c0 + c), h8);
                }
            }
#pragma unroll
            for (int h = 0; h < HALVES; h++) {
                const int steps = a.nh[h] / (8 * CG);
#pragma unroll 1
                for (int v = q; v < steps; v += 4) {
                    const uint32_t s = raw + C::RAW_W + h * C::RAW_X + v * (8 * KU) + (uint32_t)(xrow * KU);
                    const uint32_t d = bst + h * C::BHALF + v * 1024;
                    const uint4 v0 = lds128(s + ((xc ^ xrow) << 4)), v1 = lds128(s + (((4 + xc) ^ xrow) << 4));
                    uint32_t h8[8];
                    codes16(v0, h8);
                    sts128(d + x_d0, h8[0], h8[1], h8[2], h8[3]);
                    sts128(d + x_d1, h8[4], h8[5], h8[6], h8[7]);
                    codes16(v1, h8);
                    sts128(d + C::BATOM + x_d0, h8[0], h8[1], h8[2], h8[3]);
                    sts128(d + C::BATOM + x_d1, h8[4], h8[5], h8[6], h8[7]);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // the tensor core reads the tokens
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (!peers_ready) {
                cluster_wait();
                peers_ready = true;
            }
            if (lane == 0) {
                arrive_on<CG>(&afull[aslot], leader);
                mbar_arrive(&rfree[rslot]);
            }
            if ((rslot += GROUPS) >= NS) {
                rslot -= NS;
                rphase ^= 1;
            }
            if ((aslot += GROUPS) >= RB) {
                aslot -= RB;
                aphase ^= 1;
            }
        }
        __syncwarp();
        if (!peers_ready)
            cluster_wait();
        if (a.sk > 1)
            cluster_sync_all();
    } else {
        // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_EPI));
        pdl_wait();
        if (csize > 1)
            cluster_wait();
        const int q = warp & 3, eh = (warp - C::EPI_WARP0) >> 2;
        const int row = 32 * q + lane, col0 = eh * ECOLS;
        const uint32_t td = tmem + ((uint32_t)(32 * q) << 16) + D_COL + col0;
        uint32_t dphase = 0, slot = 0;
        bool ok = true;
        int acc[HALVES][ECOLS];
        // K of one chunk: the accumulators are the sums, and stay floats (1860 x 113600 x
        // 128: 186 us, converted to int32 and back 220; no gain for two halves)
        constexpr bool AS_FLOATS = HALVES == 1; // sums are stored as floats
        const bool raw = AS_FLOATS && a.sk == 1 && nu <= CHUNK;
        // accumulator slot `ds` into the sums of half h (set, or added to)
        auto read_back = [&](int (&s)[ECOLS], uint32_t ds, bool set) {
            if (!tc_wait_warp<CG == 2>(&dfull[ds], (dphase >> ds) & 1, abort_flag))
                return false;
            tc_fence_after();
            dphase ^= 1u << ds;
#pragma unroll
            for (int c = 0; c < ECOLS; c += 16) {
                uint32_t v[16];
                tmem_ld16(td + ds * C::DCOLS + c, v);
                tmem_wait_ld();
                if (raw) {
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        s[c + i] = __float_as_int(__fadd_rn(__uint_as_float(v[i]), 0.0f)); // (no -0, as of an int32)
                } else if (set) {
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        s[c + i] = __float2int_rn(__uint_as_float(v[i]));
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        s[c + i] += __float2int_rn(__uint_as_float(v[i]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_on<CG>(&dfree[ds], leader);
            return true;
        };
        for (int tile = c0; tile < a.tiles && ok; tile += cstep) {
            // the scales, requested before the sums are waited for
            const int n = w_row(tile) + row;
            const bool live = a.sk == 1 && n < a.N;
            const float wsn = live ? a.ws[n] : 0.0f, bn = live && a.bias ? a.bias[n] : 0.0f;
            float xl[HALVES][ECOLS / 32];
#pragma unroll
            for (int h = 0; h < HALVES; h++)
#pragma unroll
                for (int c = 0; c < ECOLS; c += 32) {
                    const int t = h * a.nh[0] + col0 + c + lane; // (of the tile)
                    xl[h][c / 32] = a.sk == 1 && col0 + c + lane < a.nh[h] && x_tile(tile) + t < a.T ? a.xs[x_tile(tile) + t] : 0.0f;
                }
            // the chunks in the order in which they end
            if constexpr (HALVES == 1) {
                for (int u = 0; u < nu && ok; u += CHUNK, slot ^= 1)
                    ok = read_back(acc[0], slot, u == 0);
            } else {
                for (int u = CHUNK / 2 - 1; u < nu - 1 && ok; u += CHUNK / 2) {
                    if ((u & (CHUNK - 1)) == CHUNK - 1)
                        ok = read_back(acc[0], 0, u == CHUNK - 1);
                    else
                        ok = read_back(acc[HALVES - 1], 1, u == CHUNK / 2 - 1);
                }
                ok = ok && read_back(acc[0], 0, nu <= CHUNK) && read_back(acc[HALVES - 1], 1, nu <= CHUNK / 2);
            }
            if (!ok)
                break;
            if (a.sk > 1) {
                // (one tile per cluster) the int32 sums, where the stages were
#pragma unroll
                for (int h = 0; h < HALVES; h++)
#pragma unroll
                    for (int c = 0; c < ECOLS; c++)
                        asm volatile("st.shared.s32 [%0], %1;" ::"r"(sm + ((h * C::DCOLS + col0 + c) * PITCH + row) * 4),
                                     "r"(acc[h][c])
                                     : "memory");
            } else {
                // a thread holds tokens of one channel: a warp stores 32 channels of
                // a token; the tokens' scales come from the lanes that loaded them
                const bool add = a.bias != nullptr;
                if (AS_FLOATS && !raw) {
#pragma unroll
                    for (int h = 0; h < HALVES; h++)
#pragma unroll
                        for (int c = 0; c < ECOLS; c++)
                            acc[h][c] = __float_as_int((float)acc[h][c]);
                }
#pragma unroll
                for (int h = 0; h < HALVES; h++) {
                    const int t0 = x_tile(tile) + h * a.nh[0] + col0, nt = min(a.nh[h] - col0, a.T - t0);
                    TO *o = static_cast<TO *>(a.out) + (size_t)t0 * a.ldo + n;
#pragma unroll
                    for (int c0 = 0; c0 < ECOLS; c0 += 32) {
                        if (c0 >= nt)
                            break;
#pragma unroll
                        for (int c = 0; c < 32; c++) {
                            const int s = acc[h][c0 + c];
                            const float v = epilogue(AS_FLOATS ? __int_as_float(s) : (float)s,
                                                     __shfl_sync(0xffffffffu, xl[h][c0 / 32], c), wsn, add, bn);
                            if (live && c0 + c < nt)
                                store_out(o, v);
                            o += a.ldo;
                        }
                    }
                }
            }
        }
        if (a.sk > 1) {
            // every group's sums are in shared memory: each group adds its share of
            // the tile's tokens, a thread four channels (its scales are requested
            // before the wait for the other groups)
            constexpr int QUADS = RM / 4, STEP = EPI_WARPS * 32 / QUADS; // tokens at once
            const int e0 = tid - C::EPI_WARP0 * 32, n = w_row(c0) + 4 * (e0 % QUADS), t0 = x_tile(c0);
            const int nt = min(a.nb, a.T - t0);
            float wsn[4], bn[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                wsn[e] = n + e < a.N ? a.ws[n + e] : 0.0f;
                bn[e] = a.bias && n + e < a.N ? a.bias[n + e] : 0.0f;
            }
            int t = kg + (e0 / QUADS) * a.sk;
            float xst = t < nt ? a.xs[t0 + t] : 0.0f;
            __syncwarp();
            cluster_sync_all();
            for (; t < nt && ok; t += STEP * a.sk) {
                const int col = HALVES == 2 && t >= a.nh[0] ? C::DCOLS + t - a.nh[0] : t;
                const uint32_t at = sm + (uint32_t)(col * PITCH + 4 * (e0 % QUADS)) * 4;
                int4 v[SK_MAX / CG];
#pragma unroll
                for (int g = 0; g < SK_MAX / CG; g++) { // (all in flight together)
                    v[g] = make_int4(0, 0, 0, 0);
                    if (g < a.sk) {
                        uint32_t remote;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                     : "=r"(remote)
                                     : "r"(at), "r"((uint32_t)(g * CG) + pr));
                        asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(v[g].x), "=r"(v[g].y), "=r"(v[g].z), "=r"(v[g].w)
                                     : "r"(remote)
                                     : "memory");
                    }
                }
                const float xnow = xst;
                if (t + STEP * a.sk < nt)
                    xst = a.xs[t0 + t + STEP * a.sk];
                int s[4] = {0, 0, 0, 0};
#pragma unroll
                for (int g = 0; g < SK_MAX / CG; g++) {
                    s[0] += v[g].x;
                    s[1] += v[g].y;
                    s[2] += v[g].z;
                    s[3] += v[g].w;
                }
                TO *o = static_cast<TO *>(a.out) + (size_t)(t0 + t) * a.ldo + n;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (n + e < a.N)
                        store_out(o + e, epilogue(s[e], xnow, wsn[e], a.bias != nullptr, bn[e]));
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

using CfgOne = Cfg<1, 1, 3, 6, 4, 80, 56, 104>;  // up to 64 tokens to a tile, one CTA
using CfgPair = Cfg<2, 1, 3, 6, 4, 80, 56, 136>; // up to 128, a CTA pair
using CfgWide = Cfg<2, 2, 2, 3, 4, 96, 48, 168>; // up to 256, a CTA pair

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
    const cuuint32_t box[2] = {KU, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What is asked of the runtime once per kernel and device.
template <class C, typename TO> struct Tc {
    static inline luce_host::SmemLimit limit;
    static inline std::atomic<int> resident[64][SK_MAX + 1]; // clusters of a size that a device holds at once, plus one
    static bool prepare()
    {
        if (limit.raise(k_linear_i8_tc<C, TO>, C::SMEM) == cudaSuccess)
            return true;
        (void)cudaGetLastError();
        return false;
    }
    static int clusters_at_once(int dev, int csize)
    {
        const bool keep = dev >= 0 && dev < 64;
        int n = keep ? resident[dev][csize].load(std::memory_order_relaxed) : 0;
        if (n > 0)
            return n - 1;
        if (!prepare())
            return 0;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        luce_host::make_config(cfg, attr, dim3((unsigned)csize), dim3(C::THREADS), C::SMEM, nullptr);
        cudaLaunchAttribute &cluster = attr[cfg.numAttrs++];
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim.x = (unsigned)csize;
        cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
        if (cudaOccupancyMaxActiveClusters(&n, k_linear_i8_tc<C, TO>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        if (keep)
            resident[dev][csize].store(n + 1, std::memory_order_relaxed);
        return n;
    }
    // Groups along K, while all tiles' clusters are resident at once: a second
    // round costs more than the split gains (100 x 4096 x 4096: clusters of 8 CTAs, of
    // which not all 16 fit, 24.7 us; clusters of 4 16.9 us; pairs alone 18.5 us).
    // Any number of groups that shortens the longest share (61 x 5120 x 5120, 40 tiles:
    // three groups 12.6 us, two 14.7).
    static int split(int dev, int sms, int64_t tiles, int units)
    {
        int sk = 1;
        for (int s = 2; s * C::CG <= SK_MAX && s <= units && tiles * s * C::CG <= sms; s++)
            if ((units + s - 1) / s < (units + sk - 1) / sk && tiles <= clusters_at_once(dev, s * C::CG))
                sk = s;
        return sk;
    }
};

// The tile of the tensor-core kernel for a product: its configuration (1, 2 or 4:
// CfgOne, CfgPair, CfgWide) and the tokens that it covers.  What a choice takes
// is estimated in microseconds: setup and last stores, the units that a CTA goes
// through, its tiles' sums.  The figures are fits to 45 products of 16 to 8192
// tokens with every choice timed, COST_WIDE.setup to 21 more (COST_WIDE.split, a time below zero, is what the
// fit gave, not a mechanism).  On 48 products that no fit had seen, of 9 to 3841
// tokens, what they choose took 0.6% longer than the best choice on average, 13% at
// most (5.08 for 4.49 us).  Tiles of 256 tokens for all products
// above 128, before, took 228 us for 8192 x 4096 x 4096 (now 159), 12.8 for 512 x
// 1024 x 1024 (7.4) and 9.5 for 137 x 88 x 800 (6.1).
struct Plan {
    float us = INFINITY;
    int cfg = 0, tokens = 0; // configuration 0 is the stream
};
// Where a tile's last round is not full: the channels of the whole rounds, by
// themselves, and a guess of the time with the rest spread over all SMs.
struct Part {
    float guess = INFINITY;
    Plan plan;
    int channels = 0;
};
struct Cost {
    float setup, unit, unit_token, token; // of a launch; of a unit; a unit's share per token of the tile; its sums per token
    float split, split_token, round;      // of the exchange between groups, per token; of a further tile of a CTA
};
constexpr Cost COST_ONE{3.83f, 0.333f, 0.0006f, 0.0302f, 1.09f, 0.0f, 0.38f};
constexpr Cost COST_PAIR{5.19f, 0.346f, 0.0f, 0.0201f, 0.07f, 0.0128f, 0.54f};
constexpr Cost COST_WIDE{6.53f, 0.616f, 0.0f, 0.0147f, -1.5f, 0.0142f, 1.7f};

// The same of the stream, eight tokens at a time: setup, and a megabyte of the
// weights as its warps go through them (fits to ten weights of 0.1 to 8 MB and 9 to
// 250 tokens: 16 x 1024 x 1024 2.5 us, tensor cores 6.0; 64 x 148 x 3376 3.2 and 6.8;
// 64 x 2048 x 2048 11.8 and 8.1).
constexpr float VUS_SETUP = 2.2f, VUS_MB = 0.28f;
constexpr float SECOND_LAUNCH = 0.95f; // what two launches may take of one's time

// Warps along K, as many as leave a slice of one batch, and the slice.
struct VecSplit {
    int wk, slice;
};
VecSplit vec_split(int K, int vu)
{
    int wk = 1;
    while (wk < V_WARPS && K / wk > 512 * vu)
        wk *= 2;
    return {wk, ((K >> 4) + wk - 1) / wk << 4};
}

template <class C, typename TO>
void consider(Plan &best, Part &part, int dev, int sms, int T, int N, int K, const Cost &c, int id, int first, int last, int step)
{
    const int units = (K + KU - 1) / KU;
    const int64_t mt = ((int64_t)N + RM * C::CG - 1) / (RM * C::CG);
    for (int w = first; w <= last && w - step < T; w += step) {
        const int64_t tt = (T + w - 1) / w, tiles = mt * tt;
        const int sk = Tc<C, TO>::split(dev, sms, tiles, units), at_once = sms / C::CG;
        const int64_t rounds = sk > 1 ? 1 : (tiles + at_once - 1) / at_once;
        const float share = (float)((units + sk - 1) / sk) * (c.unit + c.unit_token * (float)w);
        auto time = [&](float r) {
            return c.setup + r * share + c.token * (float)w + (r - 1.0f) * c.round +
                   (sk > 1 ? c.split + c.split_token * (float)w : 0.0f);
        };
        if (time((float)rounds) < best.us)
            best = Plan{time((float)rounds), id, w};
        const int64_t full = tiles / at_once * at_once / tt; // channel tiles of the whole rounds
        if (rounds > 1 && full > 0 && full < mt) {
            const float us = time((float)(rounds - 1)), rest = (float)((mt - full) * tt) / (float)at_once;
            if (us + c.setup + rest * share < part.guess)
                part = Part{us + c.setup + rest * share, Plan{us, id, w}, (int)full * RM * C::CG};
        }
    }
}

template <typename TO> Plan plan_product(int dev, int sms, int T, int N, int K, Part &part)
{
    Plan best;
    consider<CfgOne, TO>(best, part, dev, sms, T, N, K, COST_ONE, 1, 16, ROWS, 16);
    consider<CfgPair, TO>(best, part, dev, sms, T, N, K, COST_PAIR, 2, ROWS, 2 * ROWS, 32);
    if (T > 2 * ROWS)
        consider<CfgWide, TO>(best, part, dev, sms, T, N, K, COST_WIDE, 4, 2 * ROWS + 32, 4 * ROWS, 32);
    const VecSplit vs = vec_split(K, 1);
    const float mb = (float)N * (float)(vs.wk * ((vs.slice + 511) / 512 * 512)) / 1e6f;
    const float us = VUS_SETUP + VUS_MB * (float)((T + 7) / 8) * mb;
    if (us < best.us && T <= 8 * 65535)
        best = Plan{us, 0, 8};
    return best;
}

template <class C, typename TO>
luce_status launch_tc(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int T,
                      int N, int K, TO *out, int64_t ldo, int tile_tokens, int dev, int sms, cudaStream_t stream)
{
    auto kern = k_linear_i8_tc<C, TO>;
    TcArgs a;
    a.xs = xs;
    a.ws = ws;
    a.bias = bias;
    a.out = out;
    a.ldo = ldo;
    a.T = T;
    a.N = N;
    a.units = (K + KU - 1) / KU;
    a.nb = tile_tokens;
    a.nh[0] = C::HALVES == 2 ? std::min(tile_tokens, C::DCOLS) : tile_tokens;
    a.nh[1] = tile_tokens - a.nh[0];
    a.xbox = a.nh[0] / C::CG; // (the second half's box reads rows that no MMA uses when it is narrower)
    const int64_t mt = ((int64_t)N + RM * C::CG - 1) / (RM * C::CG);
    const int64_t tt = ((int64_t)T + tile_tokens - 1) / tile_tokens;
    if (mt * tt > INT_MAX / SK_MAX)
        return LUCE_ERR_UNSUPPORTED;
    a.mt = (int)mt;
    a.tiles = (int)(mt * tt);
    if (!map_codes(&a.tw, wq, N, K, RM) || !map_codes(&a.tx, xq, T, K, a.xbox))
        return LUCE_ERR_CUDA;
    if (!Tc<C, TO>::prepare())
        return LUCE_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    luce_host::make_config(cfg, attr, dim3((unsigned)C::CG), dim3(C::THREADS), C::SMEM, stream);
    cudaLaunchAttribute &cluster = attr[cfg.numAttrs];
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    a.sk = Tc<C, TO>::split(dev, sms, a.tiles, a.units);
    const int csize = C::CG * a.sk;
    const int clusters = a.sk > 1 ? a.tiles : std::min(a.tiles, sms / C::CG);
    cfg.gridDim = dim3((unsigned)(clusters * csize));
    cluster.val.clusterDim.x = (unsigned)csize;
    cfg.numAttrs += csize > 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        (void)cudaGetLastError();
        Tc<C, TO>::limit.forget();
        return LUCE_ERR_CUDA;
    }
    return LUCE_OK;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

template <int T, int VU, typename TO>
luce_status launch_vec(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int nt,
                       int N, int K, TO *out, int64_t ldo, cudaStream_t stream)
{
    const int64_t rows = ((int64_t)N + VR - 1) / VR;
    const VecSplit vs = vec_split(K, VU);
    const int wk = vs.wk, slice = vs.slice, groups = V_WARPS / wk;
    const dim3 grid((unsigned)((rows + groups - 1) / groups), (unsigned)((nt + T - 1) / T)), block(V_WARPS * 32);
    auto run = [&](auto kern) {
        return luce_host::launch(kern, grid, block, 0, stream, xq, xs, wq, ws, bias, nt, N, K, wk, out, ldo);
    };
    // (a slice of one batch: without the registers for the next, more CTAs to an SM)
    return slice > 512 * VU ? run(k_linear_i8_vec<T, VU, true, TO>) : run(k_linear_i8_vec<T, VU, false, TO>);
}

// The launches of a product: one, or the channels of the whole rounds of tiles
// and the rest.
struct Launches {
    Plan plan[2];
    int channels[2] = {0, 0};
};

template <typename TO> Launches choose(int dev, int sms, int T, int N, int K)
{
    Launches c;
    Part part, none;
    const Plan plan = plan_product<TO>(dev, sms, T, N, K, part);
    // a round that few tiles are left for: a launch of its own, whose tiles split K
    // (9 x 21891 x 10240, 171 tiles: 46.8 us, in one launch 59.8; 512 x 5120 x 13824: 57.7 and 70.2)
    if (part.guess < SECOND_LAUNCH * plan.us) {
        const Plan rest = plan_product<TO>(dev, sms, T, N - part.channels, K, none);
        if (part.plan.us + rest.us < SECOND_LAUNCH * plan.us) {
            c.plan[0] = part.plan;
            c.plan[1] = rest;
            c.channels[0] = part.channels;
            c.channels[1] = N - part.channels;
            return c;
        }
    }
    c.plan[0] = plan;
    c.channels[0] = N;
    return c;
}

// Tokens that a warp of the stream takes at once where the stream serves all
// products, else 0: up to four tokens, and up to eight while the weights are
// few: beyond 40 MB the sums of eight tokens bound it (8 x 8192 x 4096: 11.8 us,
// tensor cores 12.9; 8 x 16384 x 4096: 21.1 against 17.2).
int stream_tokens(int T, int N, int K)
{
    return T <= 2 ? T : T <= 4 ? 4 : T <= 8 && (int64_t)N * K <= (int64_t)40 << 20 ? 8 : 0;
}

template <typename TO>
luce_status run_linear(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int T,
                       int N, int K, TO *out, int64_t ldo, cudaStream_t stream)
{
    switch (stream_tokens(T, N, K)) {
    case 1:
        return launch_vec<1, 2>(xq, xs, wq, ws, bias, T, N, K, out, ldo, stream);
    case 2:
        return launch_vec<2, 2>(xq, xs, wq, ws, bias, T, N, K, out, ldo, stream);
    case 4:
        return launch_vec<4, 2>(xq, xs, wq, ws, bias, T, N, K, out, ldo, stream);
    case 8:
        return launch_vec<8, 1>(xq, xs, wq, ws, bias, T, N, K, out, ldo, stream);
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const int sms = luce_host::sm_count();
    auto run = [&](const Plan &plan, int n0, int n) { // channels n0 .. n0 + n - 1
        const int8_t *w = wq + (size_t)n0 * K;
        const float *s = ws + n0, *b = bias ? bias + n0 : nullptr;
        switch (plan.cfg) {
        case 0:
            return launch_vec<8, 1>(xq, xs, w, s, b, T, n, K, out + n0, ldo, stream);
        case 1:
            return launch_tc<CfgOne>(xq, xs, w, s, b, T, n, K, out + n0, ldo, plan.tokens, dev, sms, stream);
        case 2:
            return launch_tc<CfgPair>(xq, xs, w, s, b, T, n, K, out + n0, ldo, plan.tokens, dev, sms, stream);
        default:
            return launch_tc<CfgWide>(xq, xs, w, s, b, T, n, K, out + n0, ldo, plan.tokens, dev, sms, stream);
        }
    };
    const Launches c = choose<TO>(dev, sms, T, N, K);
    const luce_status st = run(c.plan[0], 0, c.channels[0]);
    return st == LUCE_OK && c.channels[1] ? run(c.plan[1], c.channels[0], c.channels[1]) : st;
}

// What luce_linear_i8_plan says of one launch.
template <typename TO> void describe(const Plan &plan, int channels, int dev, int sms, int T, int K, int *d)
{
    const int units = (K + KU - 1) / KU;
    auto tiles = [&](int rows) { return (((int64_t)channels + rows - 1) / rows) * (((int64_t)T + plan.tokens - 1) / plan.tokens); };
    d[0] = plan.cfg;
    d[1] = plan.tokens;
    d[2] = plan.cfg == 0   ? vec_split(K, 1).wk
           : plan.cfg == 1 ? Tc<CfgOne, TO>::split(dev, sms, tiles(RM), units)
           : plan.cfg == 2 ? Tc<CfgPair, TO>::split(dev, sms, tiles(2 * RM), units)
                           : Tc<CfgWide, TO>::split(dev, sms, tiles(2 * RM), units);
    d[3] = channels;
}

template <typename TO> luce_status describe_product(int T, int N, int K, int *d)
{
    if (const int n = stream_tokens(T, N, K)) {
        d[1] = n;
        d[2] = vec_split(K, n == 8 ? 1 : 2).wk;
        d[3] = N;
        return LUCE_OK;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const int sms = luce_host::sm_count();
    const Launches c = choose<TO>(dev, sms, T, N, K);
    for (int i = 0; i < 2 && c.channels[i]; i++)
        describe<TO>(c.plan[i], c.channels[i], dev, sms, T, K, d + 4 * i);
    return LUCE_OK;
}

bool bad_sizes(int T, int N, int K, luce_dtype out_dtype)
{
    return T < 0 || T >= (1 << 24) || N < 1 || N >= (1 << 24) || K < 16 || K > 65536 || K % 16 != 0 ||
           (out_dtype != LUCE_F32 && out_dtype != LUCE_BF16 && out_dtype != LUCE_F16);
}

} // namespace

extern "C" luce_status luce_linear_i8(const int8_t *xq, const float *x_scale, const int8_t *wq, const float *w_scale,
                                      const float *bias, int T, int N, int K, void *out, luce_dtype out_dtype,
                                      int64_t ld_out, void *stream)
{
    using luce_host::aligned;
    if (bad_sizes(T, N, K, out_dtype) || ld_out < N || ld_out > ((int64_t)1 << 32))
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

extern "C" luce_status luce_linear_i8_plan(int T, int N, int K, luce_dtype out_dtype, int *plan)
{
    if (!plan || bad_sizes(T, N, K, out_dtype))
        return LUCE_ERR_INVALID_ARG;
    std::fill_n(plan, 8, 0);
    if (T == 0)
        return LUCE_OK;
    switch (out_dtype) {
    case LUCE_F32:
        return describe_product<float>(T, N, K, plan);
    case LUCE_BF16:
        return describe_product<__nv_bfloat16>(T, N, K, plan);
    case LUCE_F16:
        return describe_product<__half>(T, N, K, plan);
    }
    return LUCE_ERR_INVALID_ARG;
}
