// sample.cu -- a token per row of logits, drawn with a temperature, top-k,
// top-p and min-p from a given random number (luce_sample), with its C-ABI
// entry point.
//
// A cluster of CTAs takes a row: every CTA keeps a slice of it in shared
// memory, in the logits' own type, so the row is read from memory once and
// everything after the first pass runs on the chip.  What bounds a row is the
// way from barrier to barrier (top-k 50 with top-p of 129280 logits, clusters of
// 16: 10.6 us; 64 rows of 32000, all kinds: 40.5), for many rows how many clusters
// run at once and the passes over all logits (256 bf16 rows of 129280 with top-k
// 64 and top-p: 50.3 us; 128 fp32 rows of 151936 with top-p alone: 140).
//
// Both filters look for the token at which those before it, by falling logits,
// reach a count (top-k) or a weight (top-p).  A histogram over the logits'
// distance from the largest finds the bin that holds it: nine bits of the
// distance at a time (ten in CTAs of 512 threads), the CTAs' histograms added
// through distributed shared memory by every CTA for itself.  Few logits enter it.  For top-k the warps'
// largest lanes bound the k-th from below: with W warps in the cluster, k tokens
// are at or above the least of the warps' ceil(k / W)-th largest lane maxima.
// For top-p only those within 2^-24 of the largest weight are binned; if they do
// not reach the share, all are.  Up to MOST tokens up to the bin's end go to the
// first CTA, which sorts them, cuts, and draws.  More than those stay where they
// are: the bin's own tokens go to the first CTA, which finds the last to stay,
// and the draw adds the weights that stay in the order of ids: lanes, warps,
// CTAs.  A bin with too many tokens is divided further; what three rounds do not
// tell apart, by the bits of the logits, and equal ones by id.
//
// Weights are whole numbers.  2^-z is looked up for the first eight bits
// behind the binary point of z = (M - l) log2(e) / temperature and corrected by
// three terms of the exponential series for the rest, which is below 2^-9, in
// fixed point; z itself is carried in two floats, for a rounding of z would
// shift the borders between tokens by 2^-24 of the row's weight.  Sums of whole
// numbers have no order: atomics give the same bits every time.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace {

using namespace luce;
namespace cg = cooperative_groups;

constexpr int CL_MAX = 16, CL_PORTABLE = 8; // CTAs of a cluster at most, and without asking for more
constexpr float NEAR = 24.0f;            // octaves of weight whose tokens are binned for top-p at first
constexpr int64_t V_MAX = 393216;        // fp32 slices of eight CTAs within shared memory
constexpr uint32_t TOO_MANY = 1u << 20;  // tokens: above V_MAX, and for 1024 bins below 2^32
typedef unsigned long long u64;

struct SampleArgs {
    const void *logits;
    int64_t ld;
    int V, slice; // slice: elements of a CTA, whole vectors of every warp
    int sh;       // the largest weight is 2^(31 + sh)
    const float *u, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int32_t *idx;
    float *prob;
};

// 2^(31 - j / 256), rounded.
struct Powers {
    uint32_t v[256];
};
constexpr Powers powers()
{
    // the 256th root of 1/2 by eight square roots (Newton's iteration)
    double r = 0.5;
    for (int i = 0; i < 8; i++) {
        double s = 1.0;
        for (int k = 0; k < 60; k++)
            s = 0.5 * (s + r / s);
        r = s;
    }
    Powers p{};
    double x = 2147483648.0;
    for (int j = 0; j < 256; j++, x *= r)
        p.v[j] = (uint32_t)(x + 0.5);
    return p;
}
__device__ constexpr Powers POWERS = powers();

// ---------------------------------------------------------------------------
// Logits as whole numbers of the same order; both zeros are one.  Everything
// at or below the key of -infinity counts as -infinity (NaN never gets here).
template <typename TL> struct Key;
template <> struct Key<float> {
    static constexpr uint32_t NONE = 0x007fffffu;
    static __device__ __forceinline__ uint32_t of(float v)
    {
        const uint32_t b = __float_as_uint(v + 0.0f);
        return b & 0x80000000u ? ~b : b | 0x80000000u;
    }
    static __device__ __forceinline__ float value(uint32_t k)
    {
        return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
    }
    static __device__ __forceinline__ uint32_t at_least(float v) { return of(v); } // the smallest key of a logit >= v
};
struct Key16 {
    static __device__ __forceinline__ uint32_t of_bits(uint32_t b)
    {
        b = b == 0x8000u ? 0u : b;
        return b & 0x8000u ? b ^ 0xffffu : b | 0x8000u;
    }
    static __device__ __forceinline__ uint16_t bits(uint32_t k) { return (uint16_t)(k & 0x8000u ? k & 0x7fffu : k ^ 0xffffu); }
};
template <> struct Key<__half> : Key16 {
    static constexpr uint32_t NONE = 0x03ffu;
    static __device__ __forceinline__ uint32_t of(__half v) { return of_bits(__half_as_ushort(v)); }
    static __device__ __forceinline__ float value(uint32_t k) { return __half2float(__ushort_as_half(bits(k))); }
    static __device__ __forceinline__ uint32_t at_least(float v) { return of(__float2half_ru(v)); }
};
template <> struct Key<__nv_bfloat16> : Key16 {
    static constexpr uint32_t NONE = 0x007fu;
    static __device__ __forceinline__ uint32_t of(__nv_bfloat16 v) { return of_bits(__bfloat16_as_ushort(v)); }
    static __device__ __forceinline__ float value(uint32_t k) { return __bfloat162float(__ushort_as_bfloat16(bits(k))); }
    static __device__ __forceinline__ uint32_t at_least(float v) { return of(__float2bfloat16_ru(v)); }
};
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
// The greatest of logits; NaN where one is.
__device__ __forceinline__ float greatest(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ __half greatest(__half a, __half b) { return __hmax_nan(a, b); }
__device__ __forceinline__ __nv_bfloat16 greatest(__nv_bfloat16 a, __nv_bfloat16 b) { return __hmax_nan(a, b); }
__device__ __forceinline__ float greatest(const float (&v)[4]) { return greatest(greatest(v[0], v[1]), greatest(v[2], v[3])); }
template <typename TL> __device__ __forceinline__ TL greatest(const TL (&v)[8]) // two at a time
{
    using T2 = typename std::conditional<std::is_same<TL, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 *p = reinterpret_cast<const T2 *>(v);
    const T2 m = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
    return __hmax_nan(m.x, m.y);
}
template <typename TL> __device__ __forceinline__ TL minus_infinity();
template <> __device__ __forceinline__ float minus_infinity<float>() { return -INFINITY; }
template <> __device__ __forceinline__ __half minus_infinity<__half>() { return __ushort_as_half(0xfc00); }
template <> __device__ __forceinline__ __nv_bfloat16 minus_infinity<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }

// The weight of a logit at most 66 octaves of weight below M: 2^(31 + sh - z),
// z = (M - l) c, c = log2(e) / temperature, in whole numbers.  z is split into a
// multiple n of 2^-8 and a rest r.  Where c M is below 2^14, n is c M - c l
// rounded, and r = (A1 - n) - l c + A2, with c M = A1 + A2 and A1 a multiple of
// 2^-7: A1 - n is exact, and the difference with l c, below 2^-7, is rounded
// once.  Beyond (small temperatures) M - l is kept in two floats (as quarters, so
// that it cannot overflow).
struct Weigh {
    float c_hi, c_lo; // c in two floats
    float cM, A1, A2;
    float M4, c4_hi, c4_lo; // M / 4, 4 c
    int sh;
    bool small;
    const uint2 *table; // 2^(31 - j / 256) as a whole number and as a float
    __device__ __forceinline__ u64 operator()(float l) const { return small ? of<true>(l) : of<false>(l); }
    template <bool SMALL> __device__ __forceinline__ u64 of(float l) const
    {
        const float magic = 49152.0f; // steps of 2^-8 at 2^15
        float t, r;
        if constexpr (!SMALL) {
            t = fmaf(-l, c_hi, cM) + magic;
            r = fmaf(-l, c_hi, A1 - (t - magic)) + fmaf(-l, c_lo, A2);
        } else {
            const float b = -0.25f * l, d = M4 + b, bp = d - M4, e = (M4 - (d - bp)) + (b - bp); // M4 + b = d + e
            const float zh = __fmul_rn(d, c4_hi), zl = fmaf(d, c4_hi, -zh) + fmaf(d, c4_lo, e * c4_hi);
            t = zh + magic;
            r = (zh - (t - magic)) + zl;
        }
        const uint32_t n = __float_as_uint(t); // (the last eight bits of magic, and ten before them, are zero)
        const float p = r * fmaf(r, fmaf(r, -0.055504109f, 0.24022651f), -0.69314718f); // ln(2)^3 / 6, ln(2)^2 / 2, ln(2)
        const uint2 q = table[n & 255];
        const uint32_t m = q.x + (uint32_t)(__float_as_int(fmaf(__uint_as_float(q.y), p, 12582912.0f)) - 0x4B400000);
        u64 w;
        asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"((u64)m << sh), "r"(n >> 8 & 1023)); // (by 64 and more: zero)
        return w;
    }
};

template <typename T> __device__ __forceinline__ T warp_add(T v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <typename T> __device__ __forceinline__ T warp_scan(T v, int lane) // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += a;
    }
    return v;
}

template <int THREADS> struct Shared {
    static constexpr int WARPS = THREADS / 32;
    static constexpr int BINS = 2 * THREADS, DIGIT = THREADS == 256 ? 9 : 10;
    static constexpr int MOST = 2 * THREADS; // tokens that one CTA sorts
    static_assert(BINS == 1 << DIGIT, "bins");
    struct Hist {
        uint32_t lo[BINS], hi[BINS]; // weights in two halves, or counts
    };
    uint2 table[256];
    union {
        Hist hist[2];     // (alternating: a level's readers have passed the next level's barrier before it is zeroed)
        alignas(16) u64 sorted[MOST]; // (while no histogram is in use)
    };
    alignas(16) u64 list[MOST]; // the first CTA's tokens: key, and id from the last
    static constexpr int NEAR_MOST = 512;
    u64 near[NEAR_MOST];     // this CTA's candidates for top-k, the same
    u64 exchange[2][CL_MAX]; // (alternating, for the same reason)
    u64 warp[WARPS], part[64];
    u64 found[5];
    u64 sum[2];                  // (alternating with the histograms)
    float edge[2];
    uint32_t wtop[WARPS], wbound[WARPS];
    uint32_t count, near_count, cut;
    int last;
};

// f x, f in [0, 1), rounded down, or up: exact.
__device__ __forceinline__ u64 share(float f, u64 x, bool up)
{
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const u64 m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int s = 150 - (int)max(e, 1u); // f = m 2^-s, s >= 24
    const u64 hi = __umul64hi(x, m), lo = x * m;
    u64 q = s < 64 ? hi << (64 - s) | lo >> s : s < 128 ? hi >> (s - 64) : 0;
    if (up) { // the ceiling
        const u64 back_lo = s < 64 ? q << s : 0, back_hi = s < 64 ? q >> (64 - s) : s < 128 ? q << (s - 64) : 0;
        q += back_lo != lo || back_hi != hi;
    }
    return q;
}

// The largest key of a warp's lanes, and their j-th largest (j from 1; 0 where j is not asked for).
__device__ __forceinline__ uint32_t largest(uint32_t key, int j, int lane, uint32_t &jth)
{
    jth = 0;
    const uint32_t top = __reduce_max_sync(0xffffffffu, key);
    if (j == 1) {
        jth = top;
    } else if (j > 1) { // (warp-uniform)
        // bitonic, falling
#pragma unroll
        for (int k = 2; k <= 32; k *= 2)
#pragma unroll
            for (int d = k / 2; d > 0; d /= 2) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, key, d);
                const bool low = (lane & d) == 0, falling = (lane & k) == 0;
                key = low == falling ? max(key, other) : min(key, other);
            }
        jth = __shfl_sync(0xffffffffu, key, j - 1);
    }
    return top;
}

template <typename TL, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    k_sample(const SampleArgs a)
{
    using S = Shared<THREADS>;
    constexpr int VEC = 16 / sizeof(TL), WARPS = S::WARPS, BINS = S::BINS, DIGIT = S::DIGIT, MOST = S::MOST;
    constexpr int QBITS = 3 * DIGIT; // of a distance from the largest logit
    struct __align__(16) Vec { TL v[VEC]; };
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ S s;
    TL *buf = reinterpret_cast<TL *>(smem_raw);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), CL = (int)cl.num_blocks(), row = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    cl.barrier_arrive(); // (waited for before the first write to another CTA: every CTA runs)
    pdl_wait();
    pdl_trigger();
    const float temp = a.temperature ? a.temperature[row] : 1.0f;
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const float top_p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f, u = a.u[row];
    const bool greedy = !(temp > 0.0f), by_k = !greedy && top_k > 0 && top_k < a.V, by_p = !greedy && top_p < 1.0f;

    // The row's slice.  Place j of the row is its element j - first, so that
    // vectors of places start 16-byte aligned; places without an element hold -infinity.
    const TL *logits = reinterpret_cast<const TL *>(a.logits) + (int64_t)row * a.ld;
    const int first = (int)((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(TL));
    const int seg = a.slice / WARPS, id0 = rank * a.slice - first; // places of a warp; the id at the CTA's first place
    const int i0 = warp * seg, i1 = i0 + seg;                      // this warp's places, counted from the CTA's first
    TL most_v = minus_infinity<TL>(); // (NaN where there is one)
    constexpr int BATCH = 8;          // vectors requested together
    for (int ib = i0; ib < i1; ib += BATCH * 32 * VEC) {
        Vec v[BATCH];
#pragma unroll
        for (int x = 0; x < BATCH; x++) {
            const int i = ib + (x * 32 + lane) * VEC, e = id0 + i;
            if (i < i1) {
                if (e >= 0 && e + VEC <= a.V) {
                    v[x] = *reinterpret_cast<const Vec *>(logits + e);
                } else {
#pragma unroll
                    for (int k = 0; k < VEC; k++)
                        v[x].v[k] = e + k >= 0 && e + k < a.V ? logits[e + k] : minus_infinity<TL>();
                }
            }
        }
#pragma unroll
        for (int x = 0; x < BATCH; x++) {
            const int i = ib + (x * 32 + lane) * VEC;
            if (i < i1) {
                *reinterpret_cast<Vec *>(buf + i) = v[x];
                most_v = greatest(most_v, greatest(v[x].v));
            }
        }
    }
    const bool bad = __any_sync(0xffffffffu, !(to_float(most_v) < INFINITY)); // NaN or +infinity
    uint32_t top = bad ? 0xffffffffu : Key<TL>::of(most_v);                    // (no logit of a good row has this key)
    for (int i = tid; i < 256; i += THREADS)
        s.table[i] = make_uint2(POWERS.v[i], __float_as_uint((float)POWERS.v[i]));
    if (tid == 0)
        s.count = s.near_count = 0;
    const int nth = by_k ? (top_k + WARPS * CL - 1) / (WARPS * CL) : 0; // lane of every warp, by size, that bounds the k-th token
    uint32_t bound;
    top = largest(top, nth <= 32 ? nth : 0, lane, bound);
    if (lane == 0) {
        s.wtop[warp] = top;
        s.wbound[warp] = bound;
    }
    __syncthreads();
    cl.barrier_wait();

    // A value of each CTA to all of them; their sum, and the sum of those before this one.
    int phase = 0, level = 0;
    auto send = [&](u64 v) {
        phase ^= 1;
        if (tid < CL)
            cl.map_shared_rank(s.exchange[phase], tid)[rank] = v;
        cl.sync();
    };
    auto add_up = [&](u64 v, u64 &before) {
        send(v);
        const u64 x = lane < CL ? s.exchange[phase][lane] : 0, upto = warp_scan(x, lane);
        before = __shfl_sync(0xffffffffu, upto - x, rank);
        return __shfl_sync(0xffffffffu, upto, 31);
    };
    {
        uint32_t t = __reduce_max_sync(0xffffffffu, s.wtop[lane % WARPS]), b = __reduce_min_sync(0xffffffffu, s.wbound[lane % WARPS]);
        send((u64)t << 32 | b);
        const u64 x = s.exchange[phase][lane % CL]; // (a power of two)
        top = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32));
        bound = __reduce_min_sync(0xffffffffu, (uint32_t)x);
    }
    if (top == 0xffffffffu || top <= Key<TL>::NONE) {
        if (rank == 0 && tid == 0) {
            a.idx[row] = 0;
            if (a.prob)
                a.prob[row] = top == 0xffffffffu ? __int_as_float(0x7fffffff) : 0.0f;
        }
        return;
    }

    // Logits of `least` and more, with their ids.
    auto each = [&](float least, auto &&f) {
#pragma unroll 2
        for (int i = i0 + lane * VEC; i < i1; i += 32 * VEC) {
            const Vec v = *reinterpret_cast<const Vec *>(buf + i);
            if (to_float(greatest(v.v)) >= least) {
#pragma unroll
                for (int k = 0; k < VEC; k++) {
                    const float l = to_float(v.v[k]);
                    if (l >= least)
                        f(l, id0 + i + k);
                }
            }
        }
    };
    // All logits, with their ids.
    auto every = [&](auto &&f) {
        for (int i = i0 + lane * VEC; i < i1; i += 32 * VEC) {
            const Vec v = *reinterpret_cast<const Vec *>(buf + i);
#pragma unroll
            for (int k = 0; k < VEC; k++)
                f(to_float(v.v[k]), id0 + i + k);
        }
    };
    if (greedy) {
        uint32_t id = 0xffffffffu;
        each(Key<TL>::value(top), [&](float, int i) { id = min(id, (uint32_t)i); });
        id = __reduce_min_sync(0xffffffffu, id);
        if (lane == 0)
            s.wtop[warp] = id;
        __syncthreads();
        id = __reduce_min_sync(0xffffffffu, s.wtop[lane % WARPS]);
        send(id);
        if (rank == 0 && tid == 0) {
            for (int c = 0; c < CL; c++)
                id = min(id, (uint32_t)s.exchange[phase][c]);
            a.idx[row] = (int)id;
            if (a.prob)
                a.prob[row] = 1.0f;
        }
        return;
    }

    const float M = Key<TL>::value(top);
    // 4 log2(e) / temperature in two floats (temperatures below 1e-37 count as that)
    const float t = fmaxf(temp, 1e-37f), c_hi = __fdiv_rn(5.77078009f, t);
    const float c_lo = t < INFINITY ? __fdiv_rn(fmaf(-c_hi, t, 5.77078009f) + 7.703852e-08f, t) : 0.0f;
    Weigh weigh;
    weigh.c4_hi = c_hi, weigh.c4_lo = c_lo, weigh.c_hi = 0.25f * c_hi, weigh.c_lo = 0.25f * c_lo;
    weigh.M4 = 0.25f * M, weigh.sh = a.sh, weigh.table = s.table;
    weigh.cM = M * weigh.c_hi;
    weigh.small = !(fabsf(weigh.cM) < 16384.0f) || c_hi < 1e-30f;
    weigh.A1 = (weigh.cM + 98304.0f) - 98304.0f; // (a multiple of 2^-7)
    weigh.A2 = (weigh.cM - weigh.A1) + fmaf(M, weigh.c_lo, fmaf(M, weigh.c_hi, -weigh.cM));
    const u64 most = weigh(M); // 2^(31 + sh), or a few units of 2^sh off

    // logits below `low` weigh nothing (45 > 64 ln(2), by more than the roundings); weights below `least` fail min-p
    const float low = fmaxf(M - 45.0f * t, -3.4028235e38f);
    const u64 least = min_p > 0.0f ? (min_p < 1.0f ? share(min_p, most, true) : most) : 0;

    auto block_sum = [&](u64 v) { // of the warps' sums, which stay in s.warp
        v = warp_add(v);
        __syncthreads();
        if (lane == 0)
            s.warp[warp] = v;
        __syncthreads();
        return warp_add(lane < WARPS ? s.warp[lane] : 0);
    };

    // What stays: logits above `cut`, and of those at it the ids up to `last`.
    float cut = low;
    int last = INT_MAX;
    auto stays = [&](float l, int id) { return l > cut || (l == cut && id <= last); };

    // -------------------------------------------------------------- the first CTA's part
    // Each part is made for the whole CTA and (ONE) for one warp, which takes up to 64
    // tokens without a barrier.
    // s.list, n entries, by size into s.sorted, the largest first (no two are equal).
    auto sort = [&](auto one, int n) {
        constexpr bool ONE = decltype(one)::value;
        if constexpr (ONE) { // the place of each is the number of larger ones
            __syncwarp();
            const u64 x = lane < n ? s.list[lane] : 0, y = lane + 32 < n ? s.list[lane + 32] : 0;
            int to_x = 0, to_y = 0;
#pragma unroll 4
            for (int j = 0; j < n; j++) {
                const u64 v = s.list[j];
                to_x += v > x;
                to_y += v > y;
            }
            if (lane < n)
                s.sorted[to_x] = x;
            if (lane + 32 < n)
                s.sorted[to_y] = y;
            __syncwarp();
            return;
        }
        __syncthreads();
        if (n <= THREADS / 2) { // the same, with several threads to an entry
            int parts = 1;
            while (2 * parts * n <= THREADS && parts < 32)
                parts *= 2;
            const int e = tid / parts;
            const u64 mine = e < n ? s.list[e] : 0;
            int larger = 0;
            for (int j = tid % parts; j < n; j += parts)
                larger += s.list[j] > mine;
            for (int d = 1; d < parts; d *= 2)
                larger += __shfl_xor_sync(0xffffffffu, larger, d);
            if (e < n && tid % parts == 0)
                s.sorted[larger] = mine;
            __syncthreads();
            return;
        }
        // bitonic, falling, two neighbours a thread: exchanged by shuffles within 64 places, beyond through
        // shared memory (s.list and s.sorted in turn)
        const int size = n <= THREADS ? THREADS : 2 * THREADS, p0 = 2 * tid;
        const bool live = p0 < size; // (whole warps)
        ulonglong2 *at = reinterpret_cast<ulonglong2 *>(s.sorted), *next = reinterpret_cast<ulonglong2 *>(s.list);
        u64 e[2] = {p0 < n ? s.list[p0] : 0, p0 + 1 < n ? s.list[p0 + 1] : 0};
        for (int k = 2; k <= size; k *= 2) {
            const bool falling = (p0 & k) == 0;
            for (int d = k / 2; d > 1; d /= 2) {
                u64 o[2] = {0, 0};
                if (d <= 32) {
                    if (live)
#pragma unroll
                        for (int i = 0; i < 2; i++)
                            o[i] = __shfl_xor_sync(0xffffffffu, e[i], d / 2);
                } else { // (a buffer's readers have passed the next one's barrier before it is written again)
                    if (live)
                        at[tid] = make_ulonglong2(e[0], e[1]);
                    __syncthreads();
                    if (live) {
                        const ulonglong2 v = at[tid ^ (d / 2)];
                        o[0] = v.x, o[1] = v.y;
                    }
                    ulonglong2 *const was = at;
                    at = next, next = was;
                }
                const bool larger = ((p0 & d) == 0) == falling;
#pragma unroll
                for (int i = 0; i < 2; i++)
                    e[i] = larger == (o[i] > e[i]) ? o[i] : e[i];
            }
            if (falling == (e[0] < e[1])) {
                const u64 x = e[0];
                e[0] = e[1], e[1] = x;
            }
        }
        __syncthreads(); // (s.list's and s.sorted's last readers)
        if (live)
            reinterpret_cast<ulonglong2 *>(s.sorted)[tid] = make_ulonglong2(e[0], e[1]);
        __syncthreads();
    };
    auto key_of = [&](u64 entry) { return (uint32_t)(entry >> 32); };
    auto id_of = [&](u64 entry) { return (int)(0xffffffffu - (uint32_t)entry); };
    auto sync = [&](auto one) {
        if constexpr (decltype(one)::value)
            __syncwarp();
        else
            __syncthreads();
    };
    // Values of two neighbours a thread: what stands before the first, and the total.
    auto scan = [&](auto one, u64 x, u64 y, u64 &before) {
        const u64 upto = warp_scan(x + y, lane);
        before = upto - x - y;
        if constexpr (decltype(one)::value)
            return __shfl_sync(0xffffffffu, upto, 31);
        __syncthreads();
        if (lane == 31)
            s.warp[warp] = upto;
        __syncthreads();
        const u64 v = lane < WARPS ? s.warp[lane] : 0, sums = warp_scan(v, lane);
        before += __shfl_sync(0xffffffffu, sums - v, warp);
        return __shfl_sync(0xffffffffu, sums, 31);
    };
    // The draw from the n tokens of the list, of which the first `keep` and those that
    // reach a weight of `want` stay (0: top_p of theirs).
    auto draw_few = [&](auto one, int n, int keep, u64 want) {
        sort(one, n);
        const int p0 = 2 * tid;
        u64 w[2], before;
        uint32_t key[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (p0 + i < keep)
                key[i] = key_of(s.sorted[p0 + i]);
            w[i] = p0 + i < keep ? weigh(Key<TL>::value(key[i])) : 0;
        }
        const u64 all = scan(one, w[0], w[1], before);
        if (by_p && want == 0)
            want = top_p > 0.0f ? max(share(top_p, all, true), (u64)1) : (u64)1;
        int stay = 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const bool in = p0 + i < keep && (!by_p || before + (i ? w[0] : 0) < want) && w[i] >= least;
            if constexpr (decltype(one)::value) // (the first one always stays)
                stay += __popc(__ballot_sync(0xffffffffu, in));
            else
                stay += __syncthreads_count(in);
        }
        // those that stay, in the order of ids: the id, and the weight's place
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (p0 + i < stay)
                s.list[p0 + i] = (u64)(uint32_t)s.sorted[p0 + i] << 32 | (uint32_t)(p0 + i);
        sort(one, stay);
        int at[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            at[i] = p0 + i < stay ? (int)(uint32_t)s.sorted[p0 + i] : -1;
        // (the weights come from the threads that hold them)
        sync(one);
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (p0 + i < stay)
                s.list[p0 + i] = w[i];
        sync(one);
#pragma unroll
        for (int i = 0; i < 2; i++)
            w[i] = at[i] >= 0 ? s.list[at[i]] : 0;
        const u64 total = scan(one, w[0], w[1], before);
        const u64 target = u > 0.0f ? (u < 1.0f ? share(u, total, false) : total - 1) : 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (target >= before && target < before + w[i]) {
                a.idx[row] = (int)(0xffffffffu - (uint32_t)(s.sorted[p0 + i] >> 32));
                if (a.prob)
                    a.prob[row] = __fdiv_rn(__ull2float_rn(w[i]), __ull2float_rn(total));
            }
            before += w[i];
        }
    };
    // Of the n tokens in the list, the last to stay where `above` stands before them and
    // `want` is to be reached: `cut` and `last`, to every CTA.
    auto cut_list = [&](auto one, int n, bool by_weight, u64 above, u64 want) {
        sort(one, n);
        const int p0 = 2 * tid;
        u64 w[2], before;
#pragma unroll
        for (int i = 0; i < 2; i++)
            w[i] = p0 + i >= n ? 0 : by_weight ? weigh(Key<TL>::value(key_of(s.sorted[p0 + i]))) : (u64)1;
        scan(one, w[0], w[1], before);
        before += above;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (before < want && want <= before + w[i])
                for (int c = 0; c < CL; c++) {
                    *cl.map_shared_rank(&s.cut, c) = key_of(s.sorted[p0 + i]);
                    *cl.map_shared_rank(&s.last, c) = id_of(s.sorted[p0 + i]);
                }
            before += w[i];
        }
    };
    // f(whether one warp is to do it) in the first CTA, for n tokens.
    auto by_first = [&](int n, auto &&f) {
        if (n > 64)
            f(std::integral_constant<bool, false>());
        else if (warp == 0)
            f(std::integral_constant<bool, true>());
    };

    // -------------------------------------------------------------- sets of tokens
    // Tokens that stay, of logits from `from` to below `to`, into the first CTA's list (at
    // most MOST).  `noted`: those of this CTA are all in s.near, and `among` says which they are.
    auto collect = [&](bool noted, auto &&among, float from, float to) {
        u64 *list = cl.map_shared_rank(s.list, 0);
        uint32_t *count = cl.map_shared_rank(&s.count, 0);
        if (noted) {
            const int near = (int)s.near_count;
            for (int i = tid; i < near; i += THREADS) {
                const u64 entry = s.near[i];
                if (among(Key<TL>::value((uint32_t)(entry >> 32))))
                    list[min(atomicAdd(count, 1u), (uint32_t)MOST - 1)] = entry;
            }
        } else {
            each(from, [&](float l, int id) {
                if (l < to && (l > cut || id <= last))
                    list[min(atomicAdd(count, 1u), (uint32_t)MOST - 1)] = (u64)Key<TL>::at_least(l) << 32 | (0xffffffffu - (uint32_t)id);
            });
        }
        cl.sync();
    };
    // The id of tie number m (from 1) at `cut`, in the order of ids.
    auto locate = [&](u64 m) {
        uint32_t n = 0;
        each(cut, [&](float l, int) { n += l == cut; });
        u64 before;
        const u64 mine = block_sum(n);
        add_up(mine, before);
        if (m > before && m <= before + mine) {
            u64 rest = m - before; // among this CTA's
            int w = 0;
            while (rest > s.warp[w])
                rest -= s.warp[w++];
            if (warp == w) {
                for (int i = i0 + lane * VEC; i - lane * VEC < i1; i += 32 * VEC) {
                    uint32_t mask = 0;
                    if (i < i1)
                        for (int k = 0; k < VEC; k++)
                            mask |= (uint32_t)(to_float(buf[i + k]) == cut) << k;
                    const u64 upto = warp_scan((uint32_t)__popc(mask), lane);
                    if (upto >= rest && upto - __popc(mask) < rest) {
                        for (u64 t = rest - (upto - __popc(mask)); t > 1; t--)
                            mask &= mask - 1;
                        for (int c = 0; c < CL; c++)
                            *cl.map_shared_rank(&s.last, c) = id0 + i + __ffs(mask) - 1;
                    }
                    const u64 here = __shfl_sync(0xffffffffu, upto, 31);
                    if (here >= rest)
                        break;
                    rest -= here;
                }
            }
        }
        cl.sync();
        return s.last;
    };

    // A histogram over the tokens that stay, of logits from `from` to below `to`, and in
    // it the bin at which what stands before it reaches `want`.  (fresh: over all that stay,
    // those of a bin below zero apart; and the weight of all, for want_of.)
    struct Found {
        uint32_t bin;
        u64 above, in; // before the bin, in it
        u64 total;     // in all bins
        uint32_t upto, inside; // tokens up to the bin's end, and in it, at most
    };
    auto find = [&](bool by_weight, bool fresh, float from, float to, u64 above, auto &&want_of, auto &&bin, auto &&lightest) {
        level ^= 1;
        auto &h = s.hist[level];
        for (int i = tid; i < BINS; i += THREADS)
            h.lo[i] = h.hi[i] = 0;
        __syncthreads();
        u64 sum = 0;
        auto into = [&](int b, u64 w) {
            const uint32_t wl = (uint32_t)w, old = atomicAdd(&h.lo[b], wl);
            const uint32_t wh = (uint32_t)(w >> 32) + (old + wl < old);
            if (wh)
                atomicAdd(&h.hi[b], wh);
        };
        if (by_weight && fresh) {
            auto pass = [&](auto small, auto ties) {
                every([&](float l, int id) {
                    const bool in = decltype(ties)::value ? stays(l, id) : l >= cut;
                    const u64 w = weigh.template of<decltype(small)::value>(in ? l : cut);
                    sum += in ? w : 0;
                    const int b = bin(l);
                    if (in && b >= 0)
                        into(b, w);
                });
            };
            if (weigh.small)
                pass(std::true_type(), std::true_type());
            else if (last != INT_MAX)
                pass(std::false_type(), std::true_type());
            else
                pass(std::false_type(), std::false_type());
        } else if (fresh) { // (few, where the k-th is bounded well: noted, then counted)
            each(from, [&](float l, int id) {
                const uint32_t at = atomicAdd(&s.near_count, 1u);
                if (at < S::NEAR_MOST)
                    s.near[at] = (u64)Key<TL>::at_least(l) << 32 | (0xffffffffu - (uint32_t)id);
            });
            __syncthreads();
            const int near = (int)s.near_count;
            if (near <= S::NEAR_MOST) {
                for (int i = tid; i < near; i += THREADS)
                    atomicAdd(&h.lo[bin(Key<TL>::value((uint32_t)(s.near[i] >> 32)))], 1u);
            } else {
                each(from, [&](float l, int) { atomicAdd(&h.lo[bin(l)], 1u); });
            }
        } else {
            each(from, [&](float l, int id) {
                if (l < to && (l > cut || id <= last)) {
                    const int b = bin(l);
                    if (by_weight)
                        into(b, weigh(l));
                    else
                        atomicAdd(&h.lo[b], 1u);
                }
            });
        }
        if (by_weight && fresh) {
            sum = block_sum(sum);
            if (tid == 0)
                s.sum[level] = sum;
        }
        cl.sync();
        constexpr int PER = BINS / THREADS; // neighbouring bins of a thread
        static_assert(PER == 2, "two bins a thread");
        u64 w[PER] = {0, 0};
        sum = 0;
        for (int c0 = 0; c0 < CL; c0 += 4) { // (four CTAs' in flight)
            uint2 lo[4], hi[4];
            u64 one[4];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                lo[c] = hi[c] = make_uint2(0, 0);
                one[c] = 0;
                if (c0 + c < CL) {
                    const auto *r = cl.map_shared_rank(&h, c0 + c);
                    lo[c] = reinterpret_cast<const uint2 *>(r->lo)[tid];
                    if (by_weight) {
                        hi[c] = reinterpret_cast<const uint2 *>(r->hi)[tid];
                        if (fresh)
                            one[c] = *cl.map_shared_rank(&s.sum[level], c0 + c);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < 4; c++) {
                w[0] += (u64)hi[c].x << 32 | lo[c].x;
                w[1] += (u64)hi[c].y << 32 | lo[c].y;
                sum += one[c];
            }
        }
        // The tokens of a bin: no more than its weight over the lightest of them, which the rounding to whole units may
        // leave one below its real weight.  Where that is no unit at all they may be any number, and the bin is divided
        // further.
        uint32_t n[PER] = {(uint32_t)w[0], (uint32_t)w[1]};
        if (by_weight)
#pragma unroll
            for (int i = 0; i < PER; i++) {
                const float units = lightest(tid * PER + i) - 1.0f;
                n[i] = w[i] == 0 ? 0u : units >= 1.0f ? (uint32_t)fminf(__fmul_ru(__ull2float_ru(w[i]), __frcp_ru(units)), (float)TOO_MANY) : TOO_MANY;
            }
        const u64 all = w[0] + w[1], in_warp = warp_scan(all, lane);
        const uint32_t count = n[0] + n[1], n_warp = warp_scan(count, lane);
        if (lane == 31) {
            s.warp[warp] = in_warp;
            s.part[warp] = n_warp;
        }
        __syncthreads();
        const u64 v = lane < WARPS ? s.warp[lane] : 0, sums = warp_scan(v, lane);
        const uint32_t vn = lane < WARPS ? (uint32_t)s.part[lane] : 0, sums_n = warp_scan(vn, lane);
        u64 at = in_warp - all + __shfl_sync(0xffffffffu, sums - v, warp);
        const u64 total = __shfl_sync(0xffffffffu, sums, 31);
        uint32_t n_at = n_warp - count + __shfl_sync(0xffffffffu, sums_n - vn, warp);
        const u64 want = want_of(sum);
        at += above;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            n_at += n[i];
            if (at < want && want <= at + w[i]) {
                s.found[0] = tid * PER + i;
                s.found[1] = at;
                s.found[2] = w[i];
                s.found[3] = n_at;
                s.found[4] = n[i];
            }
            at += w[i];
        }
        __syncthreads();
        return Found{(uint32_t)s.found[0], s.found[1], s.found[2], total, (uint32_t)s.found[3], (uint32_t)s.found[4]};
    };
    // The cut at which the tokens that stay reach `want` (a weight of 0: a share top_p of
    // theirs).  True: they were few, and the first CTA has drawn from them.
    auto search = [&](bool by_weight, u64 want) {
        bool all_in = !by_weight; // whether every token that stays is binned
        while (true) {
            // distances as whole numbers of QBITS bits, the same order as the keys' (equal for logits that are near)
            const float range = all_in ? weigh.M4 - 0.25f * cut : NEAR * 0.69314718f * 0.25f * fminf(temp, 1e30f);
            constexpr float FULL = (float)(1 << QBITS);
            const float scale = range > 0.0f ? fminf(FULL / range, 1e38f) : 0.0f;
            auto place = [&](float l) {
                const float x = (weigh.M4 - 0.25f * l) * scale;
                return x < FULL ? (int)x : all_in ? (1 << QBITS) - 1 : -1;
            };
            // the weight at the end of a stretch of `bits` bits (less a hundredth, for all roundings), not yet in whole units
            const float octaves = scale > 0.0f ? c_hi / scale : 0.0f;
            auto end_weight = [&](uint32_t stretch, int bits) {
                return scale > 0.0f ? 0.99f * exp2f((float)(31 + a.sh) - octaves * ((float)stretch + 1.0f) * (float)(1 << bits)) : 0.0f;
            };
            // the smallest logits at a distance below q0 (from 1), and below q1 (0: none):
            // two warps find them, 32 keys at a time
            auto edges = [&](int q0, int q1, float &l0, float &l1) {
                if (warp < 2) {
                    const int q = warp ? q1 : q0;
                    uint32_t lo = Key<TL>::at_least(cut), hi = top; // hi is near enough
                    while (q > 0 && lo < hi) {
                        const uint32_t step = (hi - lo + 31) / 32, k = lo + (uint32_t)lane * step;
                        const int at = k < hi ? place(Key<TL>::value(k)) : 0;
                        const int f = __ffs((int)__ballot_sync(0xffffffffu, at >= 0 && at < q)) - 1; // the first lane that is (none: hi)
                        if (f >= 0)
                            hi = min(hi, lo + (uint32_t)f * step);
                        lo = f == 0 ? hi : min(hi, lo + (uint32_t)(f < 0 ? 31 : f - 1) * step + 1);
                    }
                    if (lane == 0)
                        s.edge[warp] = q > 0 ? Key<TL>::value(hi) : INFINITY;
                }
                __syncthreads();
                l0 = s.edge[0], l1 = s.edge[1]; // (written again behind find's barriers)
            };
            uint32_t prefix = 0;
            u64 above = 0;
            float from = cut, to = INFINITY;
            bool again = false;
            for (int bits = QBITS - DIGIT; bits >= 0; bits -= DIGIT) {
                const bool fresh = bits == QBITS - DIGIT;
                const Found f = find(by_weight, fresh, from, to, above,
                                     [&](u64 sum) {
                                         if (fresh && by_weight && want == 0)
                                             want = top_p > 0.0f ? max(share(top_p, sum, true), (u64)1) : (u64)1;
                                         return want;
                                     },
                                     [&](float l) {
                                         const int q = place(l);
                                         return q < 0 ? -1 : q >> bits & (BINS - 1);
                                     },
                                     [&](uint32_t b) { return end_weight(prefix << DIGIT | b, bits); });
                if (fresh && want > f.total) {
                    if (all_in)
                        return false; // all stay
                    again = all_in = true;
                    break;
                }
                prefix = prefix << DIGIT | f.bin;
                above = f.above;
                // (a CTA that has noted its candidates tells them by their distance)
                const bool few = fresh && f.upto <= MOST, noted = fresh && !by_weight && s.near_count <= S::NEAR_MOST;
                auto among = [&](float l) {
                    const uint32_t b = (uint32_t)place(l) >> bits;
                    return few ? b <= prefix : b == prefix;
                };
                if (!noted || !(few || f.inside <= MOST))
                    edges((int)((prefix + 1) << bits), (int)(prefix << bits), from, to);
                if (few) {
                    collect(noted, among, from, INFINITY);
                    if (rank == 0) {
                        const int n = min((int)s.count, MOST);
                        by_first(n, [&](auto one) { draw_few(one, n, by_weight ? n : min(top_k, n), by_weight ? want : 0); });
                    }
                    return true;
                }
                if (f.inside <= MOST) {
                    collect(noted, among, from, to);
                    if (rank == 0) {
                        const int n = min((int)s.count, MOST);
                        by_first(n, [&](auto one) { cut_list(one, n, by_weight, above, want); });
                        __syncthreads();
                        if (tid == 0)
                            s.count = 0;
                    }
                    cl.sync();
                    cut = Key<TL>::value(s.cut);
                    last = s.last;
                    return false;
                }
            }
            if (again)
                continue;
            // many logits of one distance: by their bits, then by id
            uint32_t hi = to < INFINITY ? Key<TL>::at_least(to) - 1 : top, lo = Key<TL>::at_least(from);
            while (true) {
                const int shift = max(0, 32 - __clz(hi - lo) - DIGIT);
                const Found f = find(by_weight, false, Key<TL>::value(lo), hi == top ? INFINITY : Key<TL>::value(hi + 1), above,
                                     [&](u64) { return want; }, [&](float l) { return (int)((hi - Key<TL>::at_least(l)) >> shift); },
                                     [&](uint32_t) { return 0.0f; });
                above = f.above;
                hi -= f.bin << shift;
                if (shift == 0) { // one key: how many of its ties stay
                    const float at = Key<TL>::value(hi);
                    const u64 each_one = by_weight ? weigh(at) : (u64)1, need = (want - above + each_one - 1) / each_one;
                    if (at != cut) // (at the same one, those that stayed so far do)
                        last = INT_MAX;
                    cut = at;
                    if (need * each_one < f.in)
                        last = locate(need);
                    return false;
                }
                lo = max(lo, hi - min(hi, (1u << shift) - 1));
            }
        }
    };

    if (by_k) {
        cut = bound > Key<TL>::NONE ? fmaxf(low, Key<TL>::value(bound)) : low;
        if (search(false, (u64)top_k))
            return;
    }
    if (by_p && search(true, 0))
        return;

    // -------------------------------------------------------------- the draw
    auto weight_of = [&](TL v, int id) {
        const float l = to_float(v);
        const u64 w = stays(l, id) ? weigh(l) : 0;
        return w >= least ? w : 0;
    };
    u64 mine = 0, before;
    auto pass = [&](auto small) {
        auto add = [&](float l, int id) {
            const bool in = stays(l, id);
            const u64 w = weigh.template of<decltype(small)::value>(in ? l : cut);
            mine += in && w >= least ? w : 0;
        };
        if (by_k || by_p)
            each(cut, add);
        else
            every(add);
    };
    if (weigh.small)
        pass(std::true_type());
    else
        pass(std::false_type());
    const u64 here = block_sum(mine);
    const u64 total = add_up(here, before);
    const u64 target = u > 0.0f ? (u < 1.0f ? share(u, total, false) : total - 1) : 0;
    if (target >= before && target < before + here) {
        u64 rest = target - before;
        int w = 0;
        while (rest >= s.warp[w])
            rest -= s.warp[w++];
        // that warp's places again, a warp for every 32 vectors
        const int steps = (seg + 32 * VEC - 1) / (32 * VEC);
        for (int x = warp; x < steps; x += WARPS) {
            const int i = w * seg + (x * 32 + lane) * VEC;
            u64 sum = 0;
            if (i < (w + 1) * seg)
#pragma unroll
                for (int k = 0; k < VEC; k++)
                    sum += weight_of(buf[i + k], id0 + i + k);
            sum = warp_add(sum);
            if (lane == 0)
                s.part[x] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            int x = 0;
            while (rest >= s.part[x])
                rest -= s.part[x++];
            const int i = w * seg + (x * 32 + lane) * VEC;
            u64 part[VEC], sum = 0;
#pragma unroll
            for (int k = 0; k < VEC; k++) {
                part[k] = i < (w + 1) * seg ? weight_of(buf[i + k], id0 + i + k) : 0;
                sum += part[k];
            }
            u64 upto = warp_scan(sum, lane) - sum;
#pragma unroll
            for (int k = 0; k < VEC; k++) {
                if (rest >= upto && rest < upto + part[k]) {
                    a.idx[row] = id0 + i + k;
                    if (a.prob)
                        a.prob[row] = __fdiv_rn(__ull2float_rn(part[k]), __ull2float_rn(total));
                }
                upto += part[k];
            }
        }
    }
}

constexpr size_t SMEM_CTA = 227 * 1024;
static_assert(sizeof(Shared<512>) + (V_MAX / CL_PORTABLE + 64) * sizeof(float) <= SMEM_CTA, "a slice of the longest rows");

template <typename TL, int THREADS> luce_host::SmemLimit &smem_limit()
{
    static luce_host::SmemLimit limit;
    return limit;
}

void cluster_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, int cl, int R, int threads, size_t smem, cudaStream_t stream)
{
    luce_host::make_config(cfg, attr, dim3((unsigned)cl, (unsigned)R), dim3((unsigned)threads), smem, stream);
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)cl;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    cfg.numAttrs++;
}

template <typename TL, int THREADS> luce_status launch_sample(SampleArgs a, int R, int cl, cudaStream_t stream)
{
    luce_host::SmemLimit &limit = smem_limit<TL, THREADS>();
    const auto kern = k_sample<TL, THREADS>;
    const size_t smem = (size_t)a.slice * sizeof(TL);
    if (smem + sizeof(Shared<THREADS>) > 48 * 1024 && limit.raise(kern, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    cluster_config(cfg, attr, cl, R, THREADS, smem, stream);
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        (void)cudaGetLastError();
        limit.forget();
        return LUCE_ERR_CUDA;
    }
    return LUCE_OK;
}

// Places of a CTA where n of them share a row of V logits, in whole vectors of every warp.
template <typename TL> int slice_of(int64_t V, int n, int warps)
{
    constexpr int VEC = 16 / sizeof(TL);
    const int unit = VEC * warps;
    return (int)((V + VEC - 1 + n - 1) / n + unit - 1) / unit * unit;
}
constexpr size_t QUARTER = 56 * 1024; // of an SM's shared memory

// Whether the current device holds a cluster of CL_MAX CTAs with so much shared memory.
template <typename TL, int THREADS> bool holds_wide(size_t smem)
{
    const auto kern = k_sample<TL, THREADS>;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    cluster_config(cfg, attr, CL_MAX, 1, THREADS, smem, nullptr);
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        smem_limit<TL, THREADS>().raise(kern, smem) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    return n > 0;
}

// Whether it takes them with the largest slices that they may have (asked once per device).
template <typename TL> bool wide_clusters()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return false;
    }
    int w = known[dev].load(std::memory_order_acquire);
    if (w == 0) {
        w = holds_wide<TL, 256>(QUARTER - sizeof(Shared<256>)) && holds_wide<TL, 512>(slice_of<TL>(V_MAX, CL_MAX, 16) * sizeof(TL)) ? 1 : -1;
        known[dev].store(w, std::memory_order_release);
    }
    return w > 0;
}

template <typename TL> luce_status run_sample(SampleArgs a, int R, cudaStream_t stream)
{
    // Few rows: as many CTAs to a row as there are SMs for, 1024 logits to a CTA at
    // least.  More: as many as fill every SM four times, or keep a slice small enough
    // for that; but clusters of more than eight CTAs find less room (at most 21
    // of 16 of them at once).  Slices too large for four CTAs to an SM get CTAs of
    // twice the threads (128 x 151936 fp32).
    const int sms = luce_host::sm_count();
    int cl = 1;
    while (cl < CL_PORTABLE && (int64_t)R * cl < 4 * sms && a.V > 1024 * cl)
        cl *= 2;
    if (cl == CL_PORTABLE && R * CL_MAX <= sms && a.V > 1024 * cl && wide_clusters<TL>())
        cl = CL_MAX;
    while (cl < CL_PORTABLE && slice_of<TL>(a.V, cl, 8) * sizeof(TL) > QUARTER - sizeof(Shared<256>))
        cl *= 2;
    const bool narrow = slice_of<TL>(a.V, cl, 8) * sizeof(TL) <= QUARTER - sizeof(Shared<256>);
    a.slice = slice_of<TL>(a.V, cl, narrow ? 8 : 16);
    return narrow ? launch_sample<TL, 256>(a, R, cl, stream) : launch_sample<TL, 512>(a, R, cl, stream);
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

} // namespace

extern "C" luce_status luce_sample(const void *logits, luce_dtype dtype, int R, int64_t V, int64_t ld_logits, const float *u,
                                   const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                                   int32_t *idx, float *prob, void *stream)
{
    using luce_host::aligned;
    if (R < 0 || R > 65535 || V < 1 || V >= ((int64_t)1 << 31) || ld_logits < V || ld_logits > ((int64_t)1 << 33) ||
        (dtype != LUCE_F32 && dtype != LUCE_BF16 && dtype != LUCE_F16))
        return LUCE_ERR_INVALID_ARG;
    if (V > V_MAX)
        return LUCE_ERR_UNSUPPORTED;
    if (R == 0)
        return LUCE_OK;
    const size_t es = dtype == LUCE_F32 ? 4 : 2, n = (size_t)R * 4;
    if (!logits || !u || !idx || !aligned(logits, es) || !aligned(idx, 4) || (prob && (!aligned(prob, 4) || overlap(prob, n, idx, n))))
        return LUCE_ERR_INVALID_ARG;
    const size_t nl = ((size_t)(R - 1) * ld_logits + V) * es;
    if (overlap(idx, n, logits, nl) || (prob && overlap(prob, n, logits, nl)))
        return LUCE_ERR_INVALID_ARG;
    const void *const rows[] = {u, temperature, top_k, top_p, min_p};
    for (const void *p : rows)
        if (p && (!aligned(p, 4) || overlap(p, n, idx, n) || (prob && overlap(p, n, prob, n))))
            return LUCE_ERR_INVALID_ARG;
    int bits = 0; // ceil(log2 V)
    while (((int64_t)1 << bits) < V)
        bits++;
    SampleArgs a{logits, ld_logits, (int)V, 0, 32 - bits, u, temperature, top_k, top_p, min_p, idx, prob};
    a.sh = std::min(a.sh, 31);
    cudaStream_t st = luce_host::as_stream(stream);
    return dtype == LUCE_F32 ? run_sample<float>(a, R, st)
         : dtype == LUCE_BF16 ? run_sample<__nv_bfloat16>(a, R, st)
                              : run_sample<__half>(a, R, st);
}
