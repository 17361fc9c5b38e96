// sample.cu -- a token per row of logits, drawn with a temperature, top-k,
// top-p and min-p from a given random number (luce_sample), with its C-ABI
// entry point.
//
// A cluster of CTAs takes a row: every CTA keeps a slice of it in shared
// memory, in the logits' own type, so the row is read from memory once and
// everything after the first pass runs on the chip.
//
// Both filters come down to a few candidates, as a rule.  For top-k the warps'
// largest lanes bound the key (a logit as a whole number of the same order) of
// the k-th token from below: with W warps in the cluster, k tokens are at or
// above the least of the warps' ceil(k / W)-th largest lane maxima.  For top-p
// the pass that adds all weights also adds those at four distances from the
// largest, and the first that reaches the share bounds the set.  Up to MOST
// candidates go to the first CTA, in the order of ids, which sorts them by
// logit, cuts, and draws.
// Larger sets are cut where they are: the key that divides those that stay from
// the rest is found digit by digit, a histogram of counts or weights over ten bits
// of the keys in question at a time, the CTAs' histograms added through
// distributed shared memory by every CTA for itself (one cluster barrier a
// level); ties at that key stay in the order of ids.  The draw then adds the
// weights that stay in the order of ids: lanes, warps, CTAs.
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

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"

namespace {

using namespace luce;
namespace cg = cooperative_groups;

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int CL_MAX = 16, CL_PORTABLE = 8; // CTAs of a cluster at most, and without asking for more
constexpr int MOST = 2 * THREADS;        // candidates that one CTA sorts
constexpr int DIGIT = 10, BINS = 1 << DIGIT;
constexpr int64_t V_MAX = 393216;        // fp32 slices of eight CTAs within shared memory
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
template <typename TL> __device__ __forceinline__ TL minus_infinity();
template <> __device__ __forceinline__ float minus_infinity<float>() { return -INFINITY; }
template <> __device__ __forceinline__ __half minus_infinity<__half>() { return __ushort_as_half(0xfc00); }
template <> __device__ __forceinline__ __nv_bfloat16 minus_infinity<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }

// The weight of a logit: 2^(31 + sh - z), z = (M - l) c, in whole numbers.
// (M and l are taken as quarters, so that their difference cannot overflow.)
struct Weigh {
    float M4, c_hi, c_lo; // M / 4, 4 c in two floats
    int sh;
    const uint2 *table; // 2^(31 - j / 256) as a whole number and as a float
    __device__ __forceinline__ u64 operator()(float l) const
    {
        const float b = -0.25f * l, d = M4 + b;
        const float bp = d - M4, e = (M4 - (d - bp)) + (b - bp); // M4 + b = d + e
        const float zh = fminf(d * c_hi, 64.0f);
        const float zl = fmaf(d, c_hi, -zh) + fmaf(d, c_lo, e * c_hi);
        const float magic = 49152.0f; // steps of 2^-8 at 2^15
        const float t = zh + magic;
        const int n = __float_as_int(t) - __float_as_int(magic);
        const float r = (zh - (t - magic)) + zl;
        const float p = r * fmaf(r, fmaf(r, -0.055504109f, 0.24022651f), -0.69314718f); // ln(2)^3 / 6, ln(2)^2 / 2, ln(2)
        const uint2 q = table[n & 255];
        const uint32_t m = q.x + (uint32_t)(__float_as_int(fmaf(__uint_as_float(q.y), p, 12582912.0f)) - 0x4B400000);
        return n < 64 * 256 ? ((u64)m << sh) >> (n >> 8) : 0;
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

constexpr int LEVELS = 4; // distances from the largest logit at which weights are added, in octaves of weight
__device__ constexpr float OCTAVES[LEVELS] = {3.0f, 6.0f, 10.0f, 16.0f};

struct Shared {
    uint2 table[256];
    union {
        u64 hist[2][BINS];                  // (alternating: a level's readers have passed the next level's barrier before it is zeroed)
        struct {
            u64 sorted[MOST];               // key and place of candidates, largest key first
            uint32_t key[MOST];             // candidates in the order of ids
            int id[MOST];
        } few;
    };
    u64 gather[2][CL_MAX][2 * LEVELS + 2]; // (alternating, for the same reason)
    u64 warp[WARPS];
    u64 found[4];
    uint32_t wtop[WARPS], wbound[WARPS];
    uint32_t tie;
};

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

template <typename TL>
__global__ void __launch_bounds__(THREADS, 2)
    k_sample(const SampleArgs a)
{
    constexpr int VEC = 16 / sizeof(TL);
    struct __align__(16) Vec { TL v[VEC]; };
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ Shared s;
    TL *buf = reinterpret_cast<TL *>(smem_raw);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), CL = (int)cl.num_blocks(), row = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 256; i += THREADS)
        s.table[i] = make_uint2(POWERS.v[i], __float_as_uint((float)POWERS.v[i]));
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
    const int seg = a.slice / WARPS, j0 = rank * a.slice; // places of a warp; the CTA's first
    const int i0 = warp * seg, i1 = i0 + seg;             // this warp's places, counted from the CTA's first
    uint32_t top = 0;
    bool bad = false;
#pragma unroll 4
    for (int i = i0 + lane * VEC; i < i1; i += 32 * VEC) {
        const int e = j0 + i - first; // (element)
        Vec v;
        if (e >= 0 && e + VEC <= a.V) {
            v = *reinterpret_cast<const Vec *>(logits + e);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; k++)
                v.v[k] = e + k >= 0 && e + k < a.V ? logits[e + k] : minus_infinity<TL>();
        }
        *reinterpret_cast<Vec *>(buf + i) = v;
#pragma unroll
        for (int k = 0; k < VEC; k++) {
            bad |= !(to_float(v.v[k]) < INFINITY); // NaN or +infinity
            top = max(top, Key<TL>::of(v.v[k]));
        }
    }
    const int nth = by_k ? (top_k + WARPS * CL - 1) / (WARPS * CL) : 0; // lane of every warp, by size, that bounds the k-th token
    uint32_t bound;
    top = largest(top, nth <= 32 ? nth : 0, lane, bound);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        s.wtop[warp] = bad ? 0xffffffffu : top; // (no logit of a good row has this key)
        s.wbound[warp] = bound;
    }
    __syncthreads();
    cl.sync(); // every CTA runs: its shared memory may be written

    // Values of each CTA to all of them; `mine` of a thread below N is its value number.
    int phase = 0, level = 0;
    auto exchange = [&](int n, auto &&value) {
        phase ^= 1;
        if (tid < CL * n)
            cl.map_shared_rank(&s.gather[phase][rank][0], tid / n)[tid % n] = value(tid % n);
        cl.sync();
    };
    // The sum over the CTAs of value i of each, and of those before this one.
    auto sum_of = [&](int i, u64 &before) {
        u64 all = 0;
        before = 0;
        for (int c = 0; c < CL; c++) {
            if (c == rank)
                before = all;
            all += s.gather[phase][c][i];
        }
        return all;
    };
    {
        uint32_t t = __reduce_max_sync(0xffffffffu, s.wtop[lane % WARPS]), b = __reduce_min_sync(0xffffffffu, s.wbound[lane % WARPS]);
        exchange(1, [&](int) { return (u64)t << 32 | b; });
        t = 0, b = 0xffffffffu;
        for (int c = 0; c < CL; c++) {
            t = max(t, (uint32_t)(s.gather[phase][c][0] >> 32));
            b = min(b, (uint32_t)s.gather[phase][c][0]);
        }
        top = t, bound = b;
    }
    if (top == 0xffffffffu || top <= Key<TL>::NONE) {
        if (rank == 0 && tid == 0) {
            a.idx[row] = 0;
            if (a.prob)
                a.prob[row] = top == 0xffffffffu ? __int_as_float(0x7fffffff) : 0.0f;
        }
        return;
    }

    const float M = Key<TL>::value(top);
    Weigh weigh{0.25f * M, 0.0f, 0.0f, a.sh, s.table};
    uint32_t low = Key<TL>::NONE + 1, least = 0; // keys below weigh nothing; those below `least` fail min-p
    if (!greedy) {
        const double c = fmin(4.0 * 1.4426950408889634 / (double)temp, 1e38);
        weigh.c_hi = (float)c;
        weigh.c_lo = (float)(c - (double)weigh.c_hi);
        const double reach = (double)M - 44.5 * (double)temp; // 44.5 > 64 ln(2)
        if (reach > -3e38)
            low = max(low, Key<TL>::at_least(__double2float_rd(reach)));
        if (min_p > 0.0f) {
            const double l = (double)M + (double)temp * log(fmin((double)min_p, 1.0));
            if (l > -3e38)
                least = min(top, Key<TL>::at_least(__double2float_ru(l)));
        }
    }

    auto block_sum = [&](u64 v) { // of the warps' sums, which stay in s.warp
        v = warp_add(v);
        __syncthreads();
        if (lane == 0)
            s.warp[warp] = v;
        __syncthreads();
        u64 t = 0;
        for (int i = 0; i < WARPS; i++)
            t += s.warp[i];
        return t;
    };

    // What stays: keys above `cut`, and of those at it the places up to `last`.
    uint32_t cut = low;
    int last = INT_MAX;
    auto stays = [&](uint32_t key, int i) { return key > cut || (key == cut && j0 + i <= last); };
    auto each = [&](auto &&f) {
        for (int i = i0 + lane * VEC; i < i1; i += 32 * VEC) {
            const Vec v = *reinterpret_cast<const Vec *>(buf + i);
#pragma unroll
            for (int k = 0; k < VEC; k++)
                f(v.v[k], i + k);
        }
    };

    // The draw from n candidates of the first CTA, in the order of ids, where the
    // weights to reach are `want` of (0: top_p of those that top-k leaves).
    auto draw_few = [&](int n, u64 want) {
        int size = 64; // a power of two, candidates two to a thread
        while (size < n)
            size *= 2;
        for (int i = tid; i < size; i += THREADS)
            s.few.sorted[i] = i < n ? (u64)s.few.key[i] << 32 | (0xffffffffu - (uint32_t)i) : 0;
        __syncthreads();
        for (int k = 2; k <= size; k *= 2)
            for (int d = k / 2; d > 0; d /= 2) {
                if (tid < size / 2) {
                    const int i = 2 * tid - (tid & (d - 1)); // (its partner is d further on)
                    const u64 x = s.few.sorted[i], y = s.few.sorted[i + d];
                    if ((x < y) == ((i & k) == 0)) {
                        s.few.sorted[i] = y;
                        s.few.sorted[i + d] = x;
                    }
                }
                if (d > 32 || (d == 1 && k >= 64)) // (up to a distance of 32 a warp stays within its 64 places)
                    __syncthreads();
                else
                    __syncwarp();
            }
        // two neighbours a thread
        auto scan = [&](u64 x, u64 y, u64 &before) {
            const u64 upto = warp_scan(x + y, lane);
            __syncthreads();
            if (lane == 31)
                s.warp[warp] = upto;
            __syncthreads();
            u64 total = 0;
            before = upto - x - y;
            for (int i = 0; i < WARPS; i++) {
                if (i < warp)
                    before += s.warp[i];
                total += s.warp[i];
            }
            return total;
        };
        const int keep = by_k ? min(top_k, n) : n, p0 = 2 * tid;
        u64 w[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            w[i] = p0 + i < keep ? weigh(Key<TL>::value((uint32_t)(s.few.sorted[p0 + i] >> 32))) : 0;
        u64 before;
        const u64 all = scan(w[0], w[1], before);
        if (by_p && want == 0)
            want = top_p > 0.0f ? min(max((u64)ceil((double)top_p * (double)all), (u64)1), all) : (u64)1;
        int stay = 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const bool in = p0 + i < keep && (!by_p || before + (i ? w[0] : 0) < want) &&
                            ((uint32_t)(s.few.sorted[min(p0 + i, MOST - 1)] >> 32) >= least || p0 + i == 0);
            stay += __syncthreads_count(in);
        }
        const u64 line = s.few.sorted[stay - 1]; // (the first one always stays)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            w[i] = 0;
            if (p0 + i < n && ((u64)s.few.key[p0 + i] << 32 | (0xffffffffu - (uint32_t)(p0 + i))) >= line)
                w[i] = weigh(Key<TL>::value(s.few.key[p0 + i]));
        }
        const u64 total = scan(w[0], w[1], before);
        const double at = u > 0.0f ? floor((double)u * (double)total) : 0.0;
        const u64 target = at >= (double)total ? total - 1 : min((u64)at, total - 1);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (target >= before && target < before + w[i]) {
                a.idx[row] = s.few.id[p0 + i];
                if (a.prob)
                    a.prob[row] = (float)((double)w[i] / (double)total);
            }
            before += w[i];
        }
    };
    // Candidates with keys of `lo` and more to the first CTA, if they are few, and
    // the draw there.  (Their number in this CTA is `mine`, with the warps' in s.warp.)
    auto few = [&](uint32_t lo, u64 all, u64 before, u64 want) {
        if (all > MOST)
            return false;
        int at = (int)before;
        for (int w = 0; w < warp; w++)
            at += (int)s.warp[w];
        // (no histogram has been made yet where they go)
        uint32_t *keys = cl.map_shared_rank(s.few.key, 0);
        int *ids = cl.map_shared_rank(s.few.id, 0);
        for (int i = i0 + lane * VEC; i - lane * VEC < i1; i += 32 * VEC) {
            uint32_t key[VEC], n = 0;
            if (i < i1) {
                const Vec v = *reinterpret_cast<const Vec *>(buf + i);
#pragma unroll
                for (int k = 0; k < VEC; k++)
                    n += (key[k] = Key<TL>::of(v.v[k])) >= lo;
            }
            const uint32_t any = __ballot_sync(0xffffffffu, n > 0);
            if (any) {
                const uint32_t upto = warp_scan(n, lane);
                int to = at + (int)(upto - n);
                if (n > 0)
#pragma unroll
                    for (int k = 0; k < VEC; k++)
                        if (key[k] >= lo) {
                            keys[to] = key[k];
                            ids[to++] = j0 + i + k - first;
                        }
                at += (int)__shfl_sync(0xffffffffu, upto, 31);
            }
        }
        cl.sync();
        if (rank == 0)
            draw_few((int)all, want);
        return true;
    };

    // The place of tie number m (from 1) at the key `cut`.
    auto locate = [&](u64 m) {
        uint32_t n = 0;
        each([&](TL v, int) { n += Key<TL>::of(v) == cut; });
        u64 before;
        const u64 mine = block_sum(n);
        exchange(1, [&](int) { return mine; });
        sum_of(0, before);
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
                            mask |= (uint32_t)(Key<TL>::of(buf[i + k]) == cut) << k;
                    const u64 upto = warp_scan((uint32_t)__popc(mask), lane);
                    if (upto >= rest && upto - __popc(mask) < rest) {
                        for (u64 t = rest - (upto - __popc(mask)); t > 1; t--)
                            mask &= mask - 1;
                        for (int c = 0; c < CL; c++)
                            *cl.map_shared_rank(&s.tie, c) = (uint32_t)(j0 + i + __ffs(mask) - 1);
                    }
                    const u64 here = __shfl_sync(0xffffffffu, upto, 31);
                    if (here >= rest)
                        break;
                    rest -= here;
                }
            }
        }
        cl.sync();
        return (int)s.tie;
    };

    // The key at which the tokens that stay, in the order of falling logits,
    // reach a count (top-k) or weight (top-p; 0: a share p of theirs): `cut` and
    // `last` move there.
    auto search = [&](bool by_weight, u64 want, float p) {
        uint32_t hi = top, lo = cut;
        u64 above = 0;
        bool first_level = true;
        while (true) {
            const int shift = max(0, 32 - __clz(hi - lo) - DIGIT);
            u64 *hist = s.hist[level & 1];
            level++;
            for (int i = tid; i < BINS; i += THREADS)
                hist[i] = 0;
            __syncthreads();
            each([&](TL v, int i) {
                const uint32_t key = Key<TL>::of(v);
                if (key - lo <= hi - lo && stays(key, i))
                    atomicAdd(hist + ((hi - key) >> shift), by_weight ? weigh(to_float(v)) : (u64)1);
            });
            cl.sync();
            u64 bin[BINS / THREADS], sum = 0;
#pragma unroll
            for (int i = 0; i < BINS / THREADS; i++) {
                bin[i] = 0;
                for (int c = 0; c < CL; c++)
                    bin[i] += cl.map_shared_rank(hist, c)[tid * (BINS / THREADS) + i];
                sum += bin[i];
            }
            const u64 in_warp = warp_scan(sum, lane);
            if (lane == 31)
                s.warp[warp] = in_warp;
            __syncthreads();
            u64 upto = in_warp, total = 0;
            for (int i = 0; i < WARPS; i++) {
                if (i < warp)
                    upto += s.warp[i];
                total += s.warp[i];
            }
            if (first_level) {
                first_level = false;
                if (want == 0) // (the first one always stays)
                    want = p > 0.0f ? min(max((u64)ceil((double)p * (double)total), (u64)1), total) : (u64)1;
                if (want > total)
                    return; // all stay
            }
            u64 at = above + upto - sum;
#pragma unroll
            for (int i = 0; i < BINS / THREADS; i++) {
                if (at < want && want <= at + bin[i]) {
                    s.found[0] = tid * (BINS / THREADS) + i;
                    s.found[1] = at;
                    s.found[2] = bin[i];
                }
                at += bin[i];
            }
            __syncthreads();
            const uint32_t b = (uint32_t)s.found[0];
            above = s.found[1];
            const u64 in_bin = s.found[2];
            hi -= b << shift;
            if (shift == 0) { // one key: how many of its ties stay
                const u64 each_one = by_weight ? weigh(Key<TL>::value(hi)) : (u64)1;
                const u64 need = (want - above + each_one - 1) / each_one;
                if (hi != cut) // (at the same key, those that stayed so far do)
                    last = INT_MAX;
                cut = hi;
                if (need * each_one < in_bin)
                    last = locate(need);
                return;
            }
            lo = max(lo, hi - min(hi, (1u << shift) - 1));
        }
    };

    if (greedy) {
        cut = top;
        last = locate(1);
    } else if (by_k) {
        cut = max(low, bound);
        uint32_t n = 0;
        each([&](TL v, int) { n += Key<TL>::of(v) >= cut; });
        const u64 mine = block_sum(n);
        exchange(1, [&](int) { return mine; });
        u64 before;
        const u64 all = sum_of(0, before);
        if (few(cut, all, before, 0))
            return;
        search(false, (u64)top_k, 0.0f);
        if (by_p)
            search(true, 0, top_p);
    } else if (by_p) {
        // the weights, and those within a few octaves of the largest, with their counts
        uint32_t line[LEVELS];
        u64 sum[LEVELS + 1] = {};
        uint32_t n[LEVELS] = {};
#pragma unroll
        for (int i = 0; i < LEVELS; i++)
            line[i] = max(low, Key<TL>::at_least(M - OCTAVES[i] * 0.69314718f * fminf(temp, 1e30f)));
        each([&](TL v, int) {
            const uint32_t key = Key<TL>::of(v);
            if (key >= low) {
                const u64 w = weigh(to_float(v));
                sum[LEVELS] += w;
#pragma unroll
                for (int i = 0; i < LEVELS; i++)
                    if (key >= line[i]) {
                        sum[i] += w;
                        n[i]++;
                    }
            }
        });
        u64 mine[2 * LEVELS + 1];
#pragma unroll
        for (int i = 0; i < LEVELS; i++)
            mine[LEVELS + 1 + i] = block_sum(n[i]);
#pragma unroll
        for (int i = LEVELS; i >= 0; i--)
            mine[i] = block_sum(sum[i]);
        exchange(2 * LEVELS + 1, [&](int i) {
            u64 v = 0;
#pragma unroll
            for (int k = 0; k < 2 * LEVELS + 1; k++)
                v = i == k ? mine[k] : v;
            return v;
        });
        u64 before;
        const u64 all = sum_of(LEVELS, before);
        const u64 want = top_p > 0.0f ? min(max((u64)ceil((double)top_p * (double)all), (u64)1), all) : (u64)1;
        for (int i = 0; i < LEVELS; i++) {
            if (sum_of(i, before) >= want) {
                cut = line[i];
                const u64 cands = sum_of(LEVELS + 1 + i, before);
                uint32_t count = n[0];
#pragma unroll
                for (int k = 1; k < LEVELS; k++)
                    count = i == k ? n[k] : count;
                block_sum(count);
                if (few(cut, cands, before, want))
                    return;
                break;
            }
        }
        search(true, want, top_p);
    }
    if (least > cut)
        cut = least, last = INT_MAX;

    // The draw.
    u64 mine = 0, before;
    if (greedy)
        each([&](TL v, int i) { mine += stays(Key<TL>::of(v), i); });
    else
        each([&](TL v, int i) {
            if (stays(Key<TL>::of(v), i))
                mine += weigh(to_float(v));
        });
    const u64 here = block_sum(mine);
    exchange(1, [&](int) { return here; });
    const u64 total = sum_of(0, before);
    const double at = u > 0.0f ? floor((double)u * (double)total) : 0.0;
    const u64 target = at >= (double)total ? total - 1 : min((u64)at, total - 1); // of the whole numbers 0 .. total - 1
    if (target >= before && target < before + here) {
        u64 rest = target - before;
        int w = 0;
        while (rest >= s.warp[w])
            rest -= s.warp[w++];
        if (warp == w) {
            for (int i = i0 + lane * VEC; i - lane * VEC < i1; i += 32 * VEC) {
                u64 x[VEC], sum = 0;
#pragma unroll
                for (int k = 0; k < VEC; k++) {
                    x[k] = 0;
                    if (i < i1 && stays(Key<TL>::of(buf[i + k]), i + k))
                        x[k] = greedy ? (u64)1 : weigh(to_float(buf[i + k]));
                    sum += x[k];
                }
                const u64 upto = warp_scan(sum, lane);
                if (rest < upto && rest >= upto - sum) {
                    u64 r = rest - (upto - sum);
                    int k = 0;
                    u64 mine_k = 0;
#pragma unroll
                    for (int q = 0; q < VEC; q++) {
                        if (k == q && r >= x[q]) {
                            r -= x[q];
                            k = q + 1;
                        } else if (k == q) {
                            mine_k = x[q];
                        }
                    }
                    a.idx[row] = j0 + i + k - first;
                    if (a.prob)
                        a.prob[row] = (float)((double)mine_k / (double)total);
                }
                const u64 all = __shfl_sync(0xffffffffu, upto, 31);
                if (rest < all)
                    break;
                rest -= all;
            }
        }
    }
}

template <typename TL> luce_status run_sample(SampleArgs a, int R, cudaStream_t stream)
{
    static luce_host::SmemLimit limit;
    constexpr int VEC = 16 / sizeof(TL), UNIT = VEC * WARPS;
    const auto kern = k_sample<TL>;
    // as many CTAs to a row as fill the GPU twice, 2048 logits to a CTA at
    // least, more where shared memory asks for them
    int cl = 1;
    auto slice_of = [&](int n) { return (int)(((a.V + VEC - 1 + n - 1) / n + UNIT - 1) / UNIT * UNIT); };
    while (cl < CL_PORTABLE && ((int64_t)R * cl < 2 * luce_host::sm_count() && (int64_t)a.V > 2048 * cl))
        cl *= 2;
    while (cl < CL_PORTABLE && (size_t)slice_of(cl) * sizeof(TL) > 88 * 1024)
        cl *= 2;
    a.slice = slice_of(cl);
    const size_t smem = (size_t)a.slice * sizeof(TL);
    if (smem + sizeof(Shared) > 48 * 1024 && limit.raise(kern, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    luce_host::make_config(cfg, attr, dim3((unsigned)cl, (unsigned)R), dim3(THREADS), smem, stream);
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)cl;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    cfg.numAttrs++;
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
