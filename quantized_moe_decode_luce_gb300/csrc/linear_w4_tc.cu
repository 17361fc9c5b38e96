// linear_w4_tc.cu -- products with 4-bit weights on the tensor cores
// (tcgen05), for more tokens than the stream of linear_w4.cu takes.
//
// A tile is 128 channels by up to 96 columns, K goes through it in chunks of
// 128.  A chunk's codes, less their zero points, become the A operand in tensor
// memory (a thread a channel); the activations are B in shared memory
// (128-byte swizzle, K-major); D[channel][column] holds one group's sums, which
// the epilogue multiplies by the channel's scale and adds in fp32 registers.
// What a chunk needs of each kind of activations:
//   bf16, and fp16 for 16-bit outputs   nothing: TMA puts them where B is.
//     The codes less their zero points become numbers of the same type.  A group's
//     sum is what the tensor cores make of it: each of its MMAs may cut off 2^-22 of
//     the sizes added so far.  For bf16 this holds for fp32 outputs too: fixed point
//     would keep sums exact as it does for fp16, but takes 24 tokens of 129280 x
//     4096 from 73 to 215 us, 300 of 8192 x 4096 from 49 to 175.
//   int8                                converted to fp16, exact sums.
//   fp32, and fp16 for fp32 outputs     two columns of whole numbers and a
//     factor per chunk (see linear_w4.cu), exact sums.
// What bounds a tile is instruction issue, 9 to 11 instructions for eight codes
// and one multiply-add per column and group in the epilogue, and for few
// columns the weights' way from HBM.
//
// Few tiles: sk CTAs of a cluster split K and add their sums through
// distributed shared memory, in the order of their ranks.  Where the last round
// of many tiles leaves most SMs without one, its tiles are split in that way too,
// by a launch of their own.
// 300 bf16 tokens of 8192 x 4096 in groups of 64: 48.7 us; 61 fp16 ones of 4096 x
// 14336 in groups of 128: 18.5 us.
//
// Roles: warp 0 issues the TMA tiles of codes, warp 1 the MMAs, warp 2 the TMA
// tiles of activations; groups of four warps convert codes, a chunk of each
// stage of two (or of every second stage); four warps convert activations where
// they need it; eight or sixteen warps are the epilogue (lane quarter w & 3, every
// second or fourth block of 16 columns).  A wait costs the
// warp that issues the MMAs some 250 clocks even where there is nothing to wait
// for, and a stage of two chunks about 700 in all: so operands change hands by
// the stage, A and B behind one barrier, and as many groups' sums as tensor
// memory holds twice (28672 x 4096 with one token, a barrier for each operand,
// chunk and group: 49 us).  Warpgroups trade
// registers with setmaxnreg; the shares add up to no more than the launch's.
// Every wait is bounded: a role that gives up raises LUCE_FAULT_TIMEOUT and the
// CTA's abort flag, the others leave at their next wait, copies and MMAs in
// flight are waited for (bounded) and tensor memory is freed.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda.h> // CUtensorMap and its enums (the encoder is reached through the runtime's entry-point query)

#include "w4.cuh"

LUCE_DEFINE_FAULT_WORD(luce_internal_fault_linear_w4)

namespace {

using namespace luce;
using namespace w4;

enum Mode { BF16 = 0, F16 = 1, I8 = 2, WHOLE = 3 };

constexpr int RM = 128;                  // channels of a tile
constexpr int STAGE = RM * 128;          // bytes of a stage of codes: two chunks
constexpr int NS_MAX = 12, XS = 2, RS = 2, DS_MAX = 8, FR = 32;
constexpr int NB_MAX = 96;               // columns of a tile
constexpr int SK_MAX = 8;                // CTAs of one cluster at most
constexpr int W_WARP = 0, MMA_WARP = 1, X_WARP = 2, CONV_WARP0 = 4;
constexpr uint32_t TMEM_COLS = 512, ACOLS = CHUNK / 2, D_COL = RS * 2 * ACOLS;
constexpr int PITCH = RM + 4;            // floats between the columns of a tile's sums in shared memory
constexpr size_t SMEM = 224 * 1024;

// Warps of a kind of activations (NBLK: pairs of blocks of 16 columns in a
// tile, at most), and their registers, which the warpgroups share out again.
// Where TMA writes B, no warps do: few columns leave the conversion of codes the
// longest part, more the epilogue, and the warps go there.
template <int MODE, int NBLK> struct Roles {
    static constexpr bool RAW = MODE == BF16 || MODE == F16; // operands as they come
    static constexpr int GROUPS = RAW && NBLK == 1 ? 4 : 2;  // of four warps that convert codes
    static constexpr int EPI = RAW && NBLK > 1 ? 4 : 2;      // of the epilogue
    static constexpr int B_WARP0 = CONV_WARP0 + 4 * GROUPS, EPI_WARP0 = B_WARP0 + (RAW ? 0 : 4), WARPS = EPI_WARP0 + 4 * EPI;
    static constexpr int THREADS = WARPS * 32, EPI_THREADS = EPI * 128;
    static constexpr int LAUNCH = RAW ? 72 : 80, REGS_MISC = 40, REGS_CONV = 56, REGS_B = 88, REGS_EPI = EPI == 4 ? 88 : 120;
    static_assert(128 * (REGS_MISC + GROUPS * REGS_CONV + (RAW ? 0 : REGS_B) + EPI * REGS_EPI) <= THREADS * LAUNCH && THREADS * LAUNCH <= 65536, "register shares");
};

struct TcArgs {
    CUtensorMap tw, tx;
    W4Args a;
    int whole_groups;      // groups of a row that one load may take: 8, 2 or 1
    int nb, tokens;        // columns (a multiple of 16) and tokens of a tile
    int rt, tt;            // tiles of channels, of tokens (fastest)
    int tile0, tiles;      // of this launch: the first, and the end
    int chunks, stages;    // of a row
    int sk;
    int ns, ds;            // stages of codes, slots of D
    uint32_t off_b, off_x, off_f, xbytes; // in shared memory; bytes of a chunk's activations as they come
};

// ---------------------------------------------------------------------------
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
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
}
// One arrival on `bar` once every MMA issued so far has completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts64(uint32_t a, const uint2 &v)
{
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A wait of a whole warp, one answer for every lane (.sync.aligned instructions
// follow).  A poll parks the thread in hardware for a while; the timer, which is
// slow to read, is looked at every 64 polls only.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    bool ok = true;
    unsigned long long t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); i++) {
        if ((i & 63u) == 0) {
            if (*abort_flag) {
                ok = false;
                break;
            }
            const unsigned long long t = global_timer_ns();
            if (t0 == 0)
                t0 = t;
            if (t - t0 > WAIT_LIMIT_NS) {
                *abort_flag = 1;
                atomicOr(&g_fault_word, LUCE_FAULT_TIMEOUT);
                ok = false;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}
// A wait for what is in flight when the CTA leaves: bounded, whatever the abort flag says.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity)
{
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < WAIT_LIMIT_NS)
        ;
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
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(int n)
    {
        if ((int)++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// The eight codes of a word less z, in their order, exact.  A code placed under
// the exponent of 128 (bf16) or 1024 (fp16) is 128 + q or 1024 + q; four places
// higher in an fp16 it counts sixteenfold.
template <bool BF> __device__ __forceinline__ void centred(uint32_t w, uint32_t z, uint32_t *h)
{
    if constexpr (BF) {
        const uint32_t zz = (0x4300u + z) * 0x10001u; // 128 + z
#pragma unroll
        for (int i = 0; i < 4; i++)
            h[i] = sub_bf16x2(and_or(w >> (4 * i), LO, 0x43004300u), zz);
    } else {
        const uint32_t zl = (0x6400u + z) * 0x10001u, zh = (0xD400u + 16u * z) * 0x10001u, w8 = w >> 8; // 1024 + z, -(64 + z)
        h[0] = sub_f16x2(and_or(w, LO, 0x64006400u), zl);
        h[1] = fma_f16x2(and_or(w, HI, 0x64006400u), 0x2C002C00u, zh); // a sixteenth
        h[2] = sub_f16x2(and_or(w8, LO, 0x64006400u), zl);
        h[3] = fma_f16x2(and_or(w8, HI, 0x64006400u), 0x2C002C00u, zh);
    }
}

// Sixteen int8 codes -> sixteen fp16 numbers: bias to unsigned (c + 128), place
// each byte under the exponent of 1024, subtract 1152.  Exact.
__device__ __forceinline__ void codes16(const uint4 &v, uint4 (&h)[2])
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t u = in[i] ^ 0x80808080u;
        o[2 * i] = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
        o[2 * i + 1] = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
    }
    h[0] = make_uint4(o[0], o[1], o[2], o[3]);
    h[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// The nearest whole number of a value below 2^22, as a float.
__device__ __forceinline__ float nearest(float v) { return __fadd_rn(__fadd_rn(v, 12582912.0f), -12582912.0f); }

// Four values of a chunk that a warp holds -> two columns of whole numbers of
// twelve bits, the second 2^-12 of the first, and the factor of the chunk's sums.
__device__ __forceinline__ float whole4(const float4 &v, uint2 &o0, uint2 &o1)
{
    const uint32_t most = __reduce_max_sync(0xffffffffu, max(max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu),
                                                             max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu)));
    const uint32_t e = max(most >> 23, 15u);            // 2^(e - 127) <= most < 2^(e - 126)
    const float up = __uint_as_float((264u - e) << 23); // to below 2^11
    const float x[4] = {v.x * up, v.y * up, v.z * up, v.w * up};
    float p[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        p[i] = nearest(x[i]);
        r[i] = nearest((x[i] - p[i]) * 4096.0f);
    }
    const __half2 h[4] = {__floats2half2_rn(p[0], p[1]), __floats2half2_rn(p[2], p[3]), __floats2half2_rn(r[0], r[1]), __floats2half2_rn(r[2], r[3])};
    o0 = make_uint2(*reinterpret_cast<const uint32_t *>(&h[0]), *reinterpret_cast<const uint32_t *>(&h[1]));
    o1 = make_uint2(*reinterpret_cast<const uint32_t *>(&h[2]), *reinterpret_cast<const uint32_t *>(&h[3]));
    return __uint_as_float((e - 10u) << 23); // 2^(e - 137)
}

// The scales and zero points of a row's groups 8 b .. 8 b + 7 (16 and 8 bits
// each), those beyond the row's G as zero.  Lanes hold rows, so that a load
// touches 32 lines however little it reads: one for eight groups where rows are
// aligned for it (1024 x 16384, 128 tokens: 18.9 us
// with a load a chunk, 16.1).
__device__ __forceinline__ uint4 load_scales(const TcArgs &t, int64_t row, int b)
{
    const uint16_t *s = reinterpret_cast<const uint16_t *>(t.a.ws) + row * t.a.G + 8 * b;
    const int left = t.a.G - 8 * b;
    if (t.whole_groups == 8)
        return left > 0 ? __ldg(reinterpret_cast<const uint4 *>(s)) : make_uint4(0, 0, 0, 0);
    uint32_t v[4] = {};
    if (t.whole_groups == 2) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (2 * i < left)
                v[i] = __ldg(reinterpret_cast<const uint32_t *>(s) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < left)
                v[i / 2] |= (uint32_t)__ldg(s + i) << (16 * (i & 1));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint2 load_zeros(const TcArgs &t, int64_t row, int b)
{
    const uint8_t *z = t.a.zeros + row * t.a.G + 8 * b;
    const int left = t.a.G - 8 * b;
    if (t.whole_groups == 8)
        return left > 0 ? __ldg(reinterpret_cast<const uint2 *>(z)) : make_uint2(0, 0);
    uint32_t v[2] = {};
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (i < left)
            v[i / 4] |= (uint32_t)__ldg(z + i) << (8 * (i & 3));
    return make_uint2(v[0], v[1]);
}
__device__ __forceinline__ float scale_of(uint32_t bits16, bool bf)
{
    return bf ? __uint_as_float(bits16 << 16) : half_bits_to_float(bits16);
}

// Groups of a slot of D: what leaves room for two slots of NBLK blocks of 16
// columns per epilogue warp.
template <int GPC, int NBLK> constexpr int GB = NBLK == 1 ? (GPC == 1 ? 2 : 4) : NBLK == 2 ? 2 : 1;

// GPC: groups of a chunk.  NBLK: pairs of blocks of 16 columns, at most.
template <int MODE, int GPC, int NBLK> __global__ void __launch_bounds__(Roles<MODE, NBLK>::THREADS, 1) k_linear_w4_tc(const __grid_constant__ TcArgs t)
{
    using R = Roles<MODE, NBLK>;
    constexpr bool RAW = R::RAW;
    constexpr int B_WARP0 = R::B_WARP0, EPI_WARP0 = R::EPI_WARP0, EPI_THREADS = R::EPI_THREADS;
    constexpr int EB = (2 * NBLK + R::EPI - 1) / R::EPI; // blocks of an epilogue warp, at most
    constexpr int GROUPS = 2 * GPC; // of a stage
    extern __shared__ uint8_t smraw[];
    __shared__ uint64_t wfull[NS_MAX], wfree[NS_MAX], full[RS], freed[RS], xfull[XS], xfree[XS], dfull[DS_MAX], dfree[DS_MAX], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const uint32_t sm = (smem_addr(smraw) + 1023u) & ~1023u;
    const uint32_t smb = sm + t.off_b, smx = sm + t.off_x;
    float *factors = reinterpret_cast<float *>(smraw + (sm - smem_addr(smraw)) + t.off_f); // [FR][token]
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t batom = (uint32_t)t.nb * 128u, bchunk = 2 * batom, bslot = 2 * bchunk; // 64 values of the columns, a chunk, a stage
    constexpr int gb = GB<GPC, NBLK>;

    if (tid == 0) {
        for (int i = 0; i < t.ns; i++) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wfree[i], 8);
        }
        for (int i = 0; i < RS; i++) {
            mbar_init(&full[i], 8 + (RAW ? 1 : 4)); // the codes' warps, and the activations' or their TMA
            mbar_init(&freed[i], 1);
        }
        for (int i = 0; i < XS; i++) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xfree[i], 4);
        }
        for (int i = 0; i < t.ds; i++) {
            mbar_init(&dfull[i], 2); // the MMAs' completion, and the issuing warp itself (for what it has seen)
            mbar_init(&dfree[i], EPI_THREADS / 32);
        }
        mbar_init(&drain, 1);
        abort_word = 0;
        fence_mbar_init();
        fence_async();
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "r"(TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait(); // (weights too may be the previous kernel's: luce_quantize_w4 writes them)
    pdl_trigger();

    // this CTA's tiles (cluster c takes tiles c, c + clusters, ...) and its share
    // of K: stages st0 .. st1 - 1.  A last stage's second chunk may lie behind the
    // row: it reads as zeros and has scales of zero.
    const int kg = t.sk > 1 ? (int)cluster_rank() : 0;
    const int first = t.tile0 + (int)(blockIdx.x / (unsigned)t.sk), step = (int)(gridDim.x / (unsigned)t.sk), tiles = t.tiles;
    const int st0 = (int)((long long)t.stages * kg / t.sk), st1 = (int)((long long)t.stages * (kg + 1) / t.sk);
    const int my_tiles = first < tiles ? (tiles - first + step - 1) / step : 0;
    const int total = my_tiles * (st1 - st0); // stages of all tiles, in order (the host keeps sk <= stages)

    if (warp < CONV_WARP0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::REGS_MISC));
        if (warp == W_WARP) {
            Ring r;
            int issued = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                const int row = tile / t.tt * RM;
                for (int st = st0; st < st1; st++, r.next(t.ns), issued++) {
                    if (!(ok = wait_warp(&wfree[r.slot], r.phase ^ 1, abort_flag)))
                        break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&wfull[r.slot], STAGE);
                        tma_2d(sm + r.slot * STAGE, &t.tw, st * 128, row, &wfull[r.slot]);
                    }
                }
            }
            if (!ok || *abort_flag) // the copies in flight land before the CTA leaves
                for (int g = max(0, issued - t.ns); g < issued; g++)
                    wait_out(&wfull[g % t.ns], (uint32_t)(g / t.ns) & 1);
        } else if (warp == X_WARP) {
            // activations: boxes of 64 values where TMA writes the operand itself, else chunks as they are
            int issued = 0; // (stages, or chunks)
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                const int token = tile % t.tt * t.tokens;
                for (int st = st0; st < st1 && ok; st++) {
                    if constexpr (RAW) {
                        const uint32_t slot = (uint32_t)issued % RS;
                        if (!(ok = wait_warp(&freed[slot], ((uint32_t)issued / RS & 1) ^ 1, abort_flag)))
                            break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&full[slot], bslot);
#pragma unroll
                            for (int h = 0; h < 4; h++)
                                tma_2d(smb + slot * bslot + (uint32_t)h * batom, &t.tx, st * (2 * CHUNK) + 64 * h, token, &full[slot]);
                        }
                        issued++;
                    } else {
                        for (int h = 0; h < 2; h++, issued++) {
                            const uint32_t slot = (uint32_t)issued % XS;
                            if (!(ok = wait_warp(&xfree[slot], ((uint32_t)issued / XS & 1) ^ 1, abort_flag)))
                                break;
                            if (elect_one()) {
                                mbar_arrive_expect_tx(&xfull[slot], t.xbytes);
                                tma_2d(smx + slot * t.xbytes, &t.tx, st * (2 * CHUNK) + h * CHUNK, token, &xfull[slot]);
                            }
                        }
                    }
                }
            }
            if (!ok || *abort_flag) {
                // (a slot that codes never reached stays open: the wait for it runs out)
                constexpr int N = RAW ? RS : XS;
                for (int g = max(0, issued - N); g < issued; g++)
                    wait_out(RAW ? &full[g % N] : &xfull[g % N], (uint32_t)(g / N) & 1);
            }
        } else if (warp == MMA_WARP) {
            // fp16 x fp16, or bf16 x bf16, to fp32; 128 rows, nb columns
            const uint32_t idesc = (1u << 4) | (MODE == BF16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(RM >> 4) << 24) |
                                   ((uint32_t)(t.nb >> 3) << 17);
            // (warp-wide loops with uniform control flow that elect a lane where something is
            // issued: the operands stay in uniform registers)
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), nb = (uint32_t)t.nb;
            const uint64_t desc0 = sw128_desc(smb);
            const uint32_t atom = batom >> 4;
            constexpr int STEPS = CHUNK / 16 / GPC; // MMAs of a group
            Ring rd;
            bool ok = true;
#pragma unroll 1
            for (int n = 0; n < total && ok; n++) {
                const uint32_t slot = (uint32_t)n % RS;
                if (!(ok = wait_warp(&full[slot], (uint32_t)n / RS & 1, abort_flag)))
                    break;
                const uint32_t as = tm + slot * (2 * ACOLS);
                const uint64_t bd = desc0 + (slot * bslot >> 4);
#pragma unroll
                for (int g = 0; g < GROUPS; g += gb) { // a slot of D
                    if (!(ok = wait_warp(&dfree[rd.slot], rd.phase ^ 1, abort_flag)))
                        break;
                    tc_fence_after();
                    const uint32_t dd = tm + D_COL + rd.slot * (uint32_t)gb * nb;
                    if (elect_one()) {
                        // (the groups in turn: an MMA waits for the sums of the one before it)
#pragma unroll
                        for (int k = 0; k < STEPS; k++)
#pragma unroll
                            for (int i = 0; i < gb; i++) {
                                const int kk = (g + i) * STEPS + k;
                                mma_ts(dd + (uint32_t)i * nb, as + 8 * kk, bd + (kk >> 2) * atom + 2 * (kk & 3), idesc, k > 0);
                            }
                        if (g + gb == GROUPS)
                            mma_commit(&freed[slot]);
                        mma_commit(&dfull[rd.slot]);
                        mbar_arrive(&dfull[rd.slot]);
                    }
                    rd.next(t.ds);
                }
            }
            // every MMA issued has completed before the tensor memory is freed
            if (elect_one())
                mma_commit(&drain);
            wait_out(&drain, 0);
        }
    } else if (warp < B_WARP0) {
        // ------------------------------------------------------------ codes
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::REGS_CONV));
        // (a group takes one chunk of every stage, or of every second one: each slot of codes then has
        // the same group's every time, their number being even)
        constexpr int EVERY = R::GROUPS / 2;
        const int q = warp & 3, g = ((warp - CONV_WARP0) >> 2) & 1, row = 32 * q + lane; // lane quarter, chunk of a stage, row
        const uint32_t ta = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)g * ACOLS;
        uint32_t n = (uint32_t)(warp - CONV_WARP0) >> 3;
        int tile = first, st = st0;
        auto advance = [&](int by) { // by stages
            st += by;
            while (st >= st1) {
                st -= st1 - st0;
                tile += step;
            }
        };
        advance((int)n);
        Ring r;
        r.slot = n;
        // the zero points of eight groups, of the chunk to come; loaded early
        uint2 zs = make_uint2(0x08080808u, 0x08080808u);
        int held = -1, held_tile = -1;
        auto zeros_of = [&] {
            const int block = (2 * st + g) * GPC / 8;
            if (t.a.zeros && (block != held || tile != held_tile)) {
                zs = load_zeros(t, min((int64_t)(tile / t.tt) * RM + row, (int64_t)t.a.N - 1), block);
                held = block;
                held_tile = tile;
            }
        };
        if ((int)n < total)
            zeros_of();
        for (; (int)n < total; n += EVERY) {
            if (!wait_warp(&wfull[r.slot], r.phase, abort_flag))
                break;
            uint4 v[4];
            const uint32_t raw = sm + r.slot * STAGE + (uint32_t)row * 128u;
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = lds128(raw + (((uint32_t)(4 * g + i) ^ (uint32_t)(row & 7)) << 4));
            const int at = (2 * st + g) * GPC % 8;
            const uint32_t zc = (at & 4 ? zs.y : zs.x) >> (8 * (at & 3));
            if ((int)n + EVERY < total) {
                advance(EVERY);
                zeros_of();
            }
            const uint32_t slot = n % RS;
            if (!wait_warp(&freed[slot], (n / RS & 1) ^ 1, abort_flag))
                break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t zg = (zc >> (8 * (GPC == 4 ? j : GPC == 2 ? j >> 1 : 0))) & 15u;
                uint32_t h[16];
#pragma unroll
                for (int i = 0; i < 4; i++)
                    centred<MODE == BF16>(j == 0 ? v[i].x : j == 1 ? v[i].y : j == 2 ? v[i].z : v[i].w, zg, h + 4 * i);
                tmem_st16(ta + slot * (2 * ACOLS) + 16 * j, h);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[slot]);
                mbar_arrive(&wfree[r.slot]);
            }
            r.slot += EVERY;
            if ((int)r.slot >= t.ns) {
                r.slot -= (uint32_t)t.ns;
                r.phase ^= 1;
            }
        }
    } else if (warp < EPI_WARP0) {
        // ------------------------------------------------------------ activations
        if constexpr (!RAW) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::REGS_B));
            const int q = warp - B_WARP0;
            bool ok = true;
            for (int n = 0; n < total && ok; n++) {
                const uint32_t slot = (uint32_t)n % RS;
                if (!(ok = wait_warp(&freed[slot], ((uint32_t)n / RS & 1) ^ 1, abort_flag)))
                    break;
                for (int ch = 0; ch < 2; ch++) { // (XS = 2: slot ch of the raw chunks, a phase per stage)
                    if (!(ok = wait_warp(&xfull[ch], (uint32_t)n & 1, abort_flag)))
                        break;
                    const uint32_t src = smx + (uint32_t)ch * t.xbytes, dst = smb + slot * bslot + (uint32_t)ch * bchunk;
                    if constexpr (MODE == I8) {
                        // a warp's step is 8 tokens x 128 values; a quarter-warp takes rows p and p ^ 5 and
                        // four 16-byte pieces, which touches every bank once in the raw tile and once in the converted one
                        const int xrow = ((lane >> 2) & 1) ? ((lane >> 3) ^ 5) : (lane >> 3), xc = lane & 3;
                        const uint32_t d0 = (uint32_t)(xrow * 128 + (((2 * xc) ^ xrow) << 4));
                        const uint32_t d1 = (uint32_t)(xrow * 128 + (((2 * xc + 1) ^ xrow) << 4));
#pragma unroll 1
                        for (int v = q; v < t.nb / 8; v += 4) {
                            const uint32_t s = src + (uint32_t)(v * 1024 + xrow * 128), d = dst + (uint32_t)v * 1024u;
                            const uint4 v0 = lds128(s + ((xc ^ xrow) << 4)), v1 = lds128(s + (((4 + xc) ^ xrow) << 4));
                            uint4 h[2];
                            codes16(v0, h);
                            sts128(d + d0, h[0]);
                            sts128(d + d1, h[1]);
                            codes16(v1, h);
                            sts128(d + batom + d0, h[0]);
                            sts128(d + batom + d1, h[1]);
                        }
                    } else {
                        // a warp a token, four values to a lane; token i has columns 2 i and 2 i + 1
                        const bool wide = t.a.x_dtype == LUCE_F32;
                        float *f = factors + (2 * n + ch) % FR * (NB_MAX / 2);
                        const uint32_t d = dst + (uint32_t)(lane >> 4) * batom + (uint32_t)(lane & 1) * 8u, u = (uint32_t)(lane & 15) >> 1;
#pragma unroll 4
                        for (int tok = q; tok < t.nb / 2; tok += 4) {
                            float4 v;
                            if (wide) {
                                const uint4 b = lds128(src + (uint32_t)(tok * 512 + lane * 16));
                                v = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
                            } else {
                                const uint2 b = lds64(src + (uint32_t)(tok * 256 + lane * 8));
                                v = make_float4(half_bits_to_float(b.x), half_bits_to_float(b.x >> 16), half_bits_to_float(b.y), half_bits_to_float(b.y >> 16));
                            }
                            uint2 o0, o1;
                            const float fac = whole4(v, o0, o1);
                            if (lane == 0)
                                f[tok] = fac;
                            const uint32_t col = (uint32_t)(2 * tok);
                            sts64(d + col * 128 + ((u ^ (col & 7)) << 4), o0);
                            sts64(d + (col + 1) * 128 + ((u ^ ((col + 1) & 7)) << 4), o1);
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&xfree[ch]);
                }
                if (!ok)
                    break;
                fence_async(); // the tensor core reads what was written
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[slot]);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::REGS_EPI));
        constexpr int BT = MODE == WHOLE ? 8 : 16; // tokens of a block of 16 columns
        const int q = warp & 3, e = (warp - EPI_WARP0) >> 2, row = 32 * q + lane;
        const uint32_t td = tmem + ((uint32_t)(32 * q) << 16) + D_COL;
        const int blocks = t.nb / 16;
        Ring rd;
        bool ok = true;
        uint32_t n = 0;
        float acc[EB][BT];
        // a block's sums of a group into the tokens'
        auto add = [&](float (&to)[BT], const uint32_t (&v)[16], float s, const float *f) {
            if constexpr (MODE == WHOLE) {
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 ff = *reinterpret_cast<const float4 *>(f + j);
                    const float fs[4] = {ff.x, ff.y, ff.z, ff.w};
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        to[j + k] = fmaf(s * fs[k], fmaf(__uint_as_float(v[2 * (j + k) + 1]), 1.0f / 4096.0f, __uint_as_float(v[2 * (j + k)])), to[j + k]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; j++)
                    to[j] = fmaf(s, __uint_as_float(v[j]), to[j]);
            }
        };
        for (int tile = first; tile < tiles && ok; tile += step) {
            const int chan = tile / t.tt * RM + row, token0 = tile % t.tt * t.tokens;
            const int64_t crow = min(chan, t.a.N - 1);
            const bool live = chan < t.a.N;
            constexpr int PER = 8 / GROUPS; // stages of eight groups
            uint4 sc = load_scales(t, crow, st0 / PER), next = make_uint4(0, 0, 0, 0);
            if (st0 / PER < (st1 - 1) / PER)
                next = load_scales(t, crow, st0 / PER + 1);
            auto shift = [&] { // a stage's scales out of sc
                if constexpr (GPC == 1)
                    sc = make_uint4(sc.y, sc.z, sc.w, 0);
                else
                    sc = make_uint4(sc.z, sc.w, 0, 0);
            };
            for (int i = 0; i < st0 % PER; i++)
                shift();
#pragma unroll
            for (int i = 0; i < EB; i++)
#pragma unroll
                for (int j = 0; j < BT; j++)
                    acc[i][j] = 0.0f;
            for (int st = st0; st < st1 && ok; st++, n++) {
                float s[GROUPS];
#pragma unroll
                for (int g = 0; g < GROUPS; g++) {
                    const uint32_t v = g < 2 ? sc.x : g < 4 ? sc.y : g < 6 ? sc.z : sc.w;
                    s[g] = scale_of(g & 1 ? v >> 16 : v & 0xffffu, t.a.ws_bf16);
                }
                if ((st + 1) % PER != 0) {
                    shift();
                } else {
                    sc = next;
                    if ((st + 1) / PER < (st1 - 1) / PER)
                        next = load_scales(t, crow, (st + 1) / PER + 1);
                }
                const float *f[2] = {factors + 2 * n % FR * (NB_MAX / 2), factors + (2 * n + 1) % FR * (NB_MAX / 2)};
#pragma unroll
                for (int g = 0; g < GROUPS; g += gb) {
                    if (!(ok = wait_warp(&dfull[rd.slot], rd.phase, abort_flag)))
                        break;
                    tc_fence_after();
                    // the slot's sums into registers, and the slot back
                    uint32_t v[gb][EB][16];
#pragma unroll
                    for (int i = 0; i < gb; i++)
#pragma unroll
                        for (int b = 0; b < EB; b++)
                            if (R::EPI * b + e < blocks)
                                tmem_ld16(td + (rd.slot * gb + i) * (uint32_t)t.nb + 16 * (R::EPI * b + e), v[i][b]);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&dfree[rd.slot]);
                    rd.next(t.ds);
#pragma unroll
                    for (int b = 0; b < EB; b++)
                        if (R::EPI * b + e < blocks)
#pragma unroll
                            for (int i = 0; i < gb; i++)
                                add(acc[b], v[i][b], s[g + i], f[(g + i) / GPC] + BT * (R::EPI * b + e));
                }
            }
            if (!ok)
                break;
            const int nt = min(t.tokens, t.a.T - token0);
            if (t.sk > 1) { // (one tile per cluster) the sums, where the stages were
#pragma unroll
                for (int i = 0; i < EB; i++)
#pragma unroll
                    for (int j = 0; j < BT; j++) {
                        const int tok = (R::EPI * i + e) * BT + j;
                        if (tok < nt)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sm + (uint32_t)(tok * PITCH + row) * 4u), "f"(acc[i][j]) : "memory");
                    }
            } else {
                const float bn = live && t.a.bias ? t.a.bias[chan] : 0.0f;
#pragma unroll
                for (int i = 0; i < EB; i++)
#pragma unroll
                    for (int j = 0; j < BT; j++) {
                        const int tok = (R::EPI * i + e) * BT + j;
                        if (tok < nt && live) {
                            float v = acc[i][j];
                            if (MODE == I8)
                                v = __fmul_rn(v, t.a.xs[token0 + tok]);
                            if (t.a.bias)
                                v = __fadd_rn(v, bn);
                            store_as(t.a.out, t.a.out_dtype, (int64_t)(token0 + tok) * t.a.ldo + chan, v);
                        }
                    }
            }
        }
        if (t.sk > 1) {
            // every CTA's sums are in its shared memory: each adds its share of the
            // tile's tokens, a thread four channels
            __syncwarp();
            cluster_sync_all();
            const int e0 = tid - EPI_WARP0 * 32, chan = first / t.tt * RM + 4 * (e0 % 32), token0 = first % t.tt * t.tokens;
            const int nt = min(t.tokens, t.a.T - token0);
            for (int tok = kg + (e0 / 32) * t.sk; tok < nt && ok; tok += EPI_THREADS / 32 * t.sk) {
                const uint32_t at = sm + (uint32_t)(tok * PITCH + 4 * (e0 % 32)) * 4u;
                float4 v[SK_MAX];
#pragma unroll
                for (int g = 0; g < SK_MAX; g++) { // (all in flight together)
                    v[g] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (g < t.sk) {
                        uint32_t remote;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"((uint32_t)g));
                        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(v[g].x), "=f"(v[g].y), "=f"(v[g].z), "=f"(v[g].w)
                                     : "r"(remote)
                                     : "memory");
                    }
                }
                float s[4] = {};
#pragma unroll
                for (int g = 0; g < SK_MAX; g++)
                    s[0] += v[g].x, s[1] += v[g].y, s[2] += v[g].z, s[3] += v[g].w;
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (chan + k < t.a.N) {
                        float x = s[k];
                        if (MODE == I8)
                            x = __fmul_rn(x, t.a.xs[token0 + tok]);
                        if (t.a.bias)
                            x = __fadd_rn(x, t.a.bias[chan + k]);
                        store_as(t.a.out, t.a.out_dtype, (int64_t)(token0 + tok) * t.a.ldo + chan + k, x);
                    }
            }
        }
    }
    __syncwarp();
    if (t.sk > 1 && warp < EPI_WARP0)
        cluster_sync_all(); // (the epilogue's exchange)
    tc_fence_before();
    __syncthreads();
    if (t.sk > 1)
        cluster_sync_all(); // no CTA leaves while a peer reads its memory
    tc_fence_after();
    if (warp == MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

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
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else
            (void)cudaGetLastError();
    });
    return fn;
}

// Rows `stride` bytes apart; a box of `inner` elements by `rows` (what lies outside reads as zero).
bool map_rows(CUtensorMap *m, CUtensorMapDataType type, const void *base, int64_t cols, int64_t rows, int64_t stride, int inner, int box,
              bool swizzle)
{
    EncodeTiledFn f = encode_tiled();
    if (!f)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t boxes[2] = {(cuuint32_t)inner, (cuuint32_t)box}, estr[2] = {1, 1};
    return f(m, type, 2, const_cast<void *>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Mode mode_of(const W4Args &a)
{
    return a.x_dtype == LUCE_I8 ? I8 : a.x_dtype == LUCE_BF16 ? BF16 : a.x_dtype == LUCE_F16 && a.out_dtype != LUCE_F32 ? F16 : WHOLE;
}

// Clocks of a stage, about (8192 x 4096 in groups of 64: 64 columns 2000, 80, whose slots of D take one group, 2900).
int stage_cost(int gpc, int nb) { return 1000 + nb * (gpc == 1 ? 7 : gpc == 2 ? 16 : 30) + (gpc > 1 && nb > 64 ? 500 : 0); }
constexpr int LAUNCH_COST = 8000; // clocks of a launch
// CTAs along K that `tiles` tiles, fewer than SMs, leave room for.
int split(int tiles, int stages, int sms) { return std::min({SK_MAX, stages, sms / tiles}); }
// Whether the tiles behind the last whole round get a launch of their own, split along K.
bool tail_apart(int tiles, int stages, int cost, int sms)
{
    const int rest = tiles % sms, sk = rest ? split(rest, stages, sms) : 1;
    return tiles > sms && sk > 1 && (stages + sk - 1) / sk * (int64_t)cost + LAUNCH_COST < stages * (int64_t)cost;
}
int64_t tiles_cost(int64_t tiles, int stages, int cost, int sms)
{
    const int rest = (int)(tiles % sms), sk = rest ? split(rest, stages, sms) : 1;
    const int64_t whole = tiles / sms * stages * (int64_t)cost;
    if (rest == 0)
        return whole;
    if (tiles < sms)
        return (stages + sk - 1) / sk * (int64_t)cost;
    return whole + (tail_apart((int)tiles, stages, cost, sms) ? (stages + sk - 1) / sk * (int64_t)cost + LAUNCH_COST : stages * (int64_t)cost);
}

template <int MODE, int GPC, int NBLK> luce_status launch_tc(TcArgs &t, cudaStream_t stream)
{
    static luce_host::SmemLimit limit;
    static std::atomic<int> resident[64][SK_MAX + 1]; // clusters of a size that a device holds at once, plus one
    const auto kern = k_linear_w4_tc<MODE, GPC, NBLK>;
    // (warpgroups take registers up from the launch's: with fewer of those they would wait for ever)
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, kern) == cudaSuccess)
            regs.store(at.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < Roles<MODE, NBLK>::LAUNCH || limit.raise(kern, SMEM) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const int sms = luce_host::sm_count(), tiles = t.tiles - t.tile0;
    auto config = [&](cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, int grid, int sk) {
        luce_host::make_config(cfg, attr, dim3((unsigned)grid), dim3(Roles<MODE, NBLK>::THREADS), SMEM, stream);
        if (sk > 1) {
            cudaLaunchAttribute &cluster = attr[cfg.numAttrs++];
            cluster.id = cudaLaunchAttributeClusterDimension;
            cluster.val.clusterDim.x = (unsigned)sk;
            cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
        }
    };
    auto at_once = [&](int sk) {
        const bool keep = dev >= 0 && dev < 64;
        int n = keep ? resident[dev][sk].load(std::memory_order_relaxed) : 0;
        if (n > 0)
            return n - 1;
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        config(cfg, attr, sk, sk);
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        if (keep)
            resident[dev][sk].store(n + 1, std::memory_order_relaxed);
        return n;
    };
    // CTAs along K, while all tiles' clusters are resident at once, as many as shorten the longest share
    t.sk = 1;
    for (int s = 2; s <= SK_MAX && s <= t.stages && (int64_t)tiles * s <= sms; s++)
        if ((t.stages + s - 1) / s < (t.stages + t.sk - 1) / t.sk && tiles <= at_once(s))
            t.sk = s;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(cfg, attr, t.sk > 1 ? tiles * t.sk : std::min(tiles, sms), t.sk);
    if (cudaLaunchKernelEx(&cfg, kern, t) != cudaSuccess) {
        (void)cudaGetLastError();
        limit.forget();
        return LUCE_ERR_CUDA;
    }
    return LUCE_OK;
}

template <int MODE, int GPC> luce_status launch_blocks(TcArgs &t, cudaStream_t stream)
{
    auto run = [&](auto nblk) {
        constexpr int NBLK = decltype(nblk)::value;
        t.ds = std::min(DS_MAX, (int)(TMEM_COLS - D_COL) / (GB<GPC, NBLK> * t.nb));
        // whole rounds of tiles, and what is left
        t.tile0 = 0;
        t.tiles = t.rt * t.tt;
        const int sms = luce_host::sm_count(), rest = t.tiles % sms;
        if (tail_apart(t.tiles, t.stages, stage_cost(GPC, t.nb), sms)) {
            t.tiles -= rest;
            const luce_status st = launch_tc<MODE, GPC, NBLK>(t, stream);
            if (st != LUCE_OK)
                return st;
            t.tile0 = t.tiles;
            t.tiles += rest;
        }
        return launch_tc<MODE, GPC, NBLK>(t, stream);
    };
    return t.nb <= 32 ? run(std::integral_constant<int, 1>()) : t.nb <= 64 ? run(std::integral_constant<int, 2>()) : run(std::integral_constant<int, 3>());
}

template <int MODE> luce_status launch_groups(TcArgs &t, int gpc, cudaStream_t stream)
{
    return gpc == 1 ? launch_blocks<MODE, 1>(t, stream) : gpc == 2 ? launch_blocks<MODE, 2>(t, stream) : launch_blocks<MODE, 4>(t, stream);
}

} // namespace

namespace w4 {

luce_status tc_product(const W4Args &a, int group, cudaStream_t stream)
{
    TcArgs t{};
    const Mode mode = mode_of(a);
    t.a = a;
    const int gpc = CHUNK / group;
    t.whole_groups = a.G % 8 == 0 && luce_host::aligned(a.ws, 16) && (!a.zeros || luce_host::aligned(a.zeros, 8)) ? 8
                     : a.G % 2 == 0 && luce_host::aligned(a.ws, 4) ? 2 : 1;
    t.chunks = (a.K + CHUNK - 1) / CHUNK;
    t.stages = (t.chunks + 1) / 2;
    const int parts = mode == WHOLE ? 2 : 1, most = NB_MAX / parts;
    t.rt = (a.N + RM - 1) / RM;
    const int sms = luce_host::sm_count();
    if ((int64_t)t.rt * ((a.T + most / 2 - 1) / (most / 2)) > INT_MAX / 2)
        return LUCE_ERR_UNSUPPORTED;
    // the tokens' tiles that take the least time (300 tokens of 8192 x 4096 in groups of 64: four of 75 53.6 us, five of 60 48.7)
    int64_t best = INT64_MAX;
    for (int cols = NB_MAX; cols >= NB_MAX / 2; cols -= 16) {
        const int tt = (a.T + cols / parts - 1) / (cols / parts), tokens = (a.T + tt - 1) / tt, nb = (tokens * parts + 15) / 16 * 16;
        const int64_t cost = tiles_cost((int64_t)t.rt * tt, t.stages, stage_cost(gpc, nb), sms);
        if (cost < best)
            best = cost, t.tt = tt, t.tokens = tokens, t.nb = nb;
    }
    t.tt = (a.T + t.tokens - 1) / t.tokens; // (none empty)
    // shared memory: stages of codes, operands of columns, activations as they come, factors
    const uint32_t es = a.x_dtype == LUCE_F32 ? 4 : a.x_dtype == LUCE_I8 ? 1 : 2, b = RS * (uint32_t)t.nb * 512u;
    const int box = mode == WHOLE ? t.nb / 2 : t.nb;
    t.xbytes = mode == I8 || mode == WHOLE ? (uint32_t)box * CHUNK * es : 0;
    const uint32_t rest = b + XS * t.xbytes + (mode == WHOLE ? FR * (NB_MAX / 2) * 4 : 0); // (every part a multiple of 1024)
    t.ns = (int)std::min<uint32_t>(NS_MAX, ((uint32_t)SMEM - 1024 - rest) / STAGE) & ~1;
    t.off_b = (uint32_t)t.ns * STAGE;
    t.off_x = t.off_b + b;
    t.off_f = t.off_x + XS * t.xbytes;
    const CUtensorMapDataType xt = a.x_dtype == LUCE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : a.x_dtype == LUCE_I8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                                          : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const int64_t xstride = a.T > 1 ? a.ldx * es : ((int64_t)a.K * es + 15) / 16 * 16;
    if (!map_rows(&t.tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq, (int64_t)t.chunks * CHUNK_BYTES, a.N, (int64_t)t.chunks * CHUNK_BYTES, 128, RM, true) ||
        !map_rows(&t.tx, xt, a.x, a.K, a.T, xstride, mode == WHOLE || mode == I8 ? CHUNK : 64, box, mode != WHOLE))
        return LUCE_ERR_CUDA;
    switch (mode) {
    case BF16:
        return launch_groups<BF16>(t, gpc, stream);
    case F16:
        return launch_groups<F16>(t, gpc, stream);
    case I8:
        return launch_groups<I8>(t, gpc, stream);
    default:
        return launch_groups<WHOLE>(t, gpc, stream);
    }
}

} // namespace w4
