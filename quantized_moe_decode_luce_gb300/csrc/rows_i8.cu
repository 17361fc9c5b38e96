// rows_i8.cu -- rows to int8 codes with one scale per row: of the row itself,
// of its RMS norm, or of the RMS norm of the residual sum (luce_quantize_i8,
// luce_rmsnorm_i8, luce_add_rmsnorm_i8), with their C-ABI entry points.
//
// Mathematics.  The codes of a normed row, x_i r gamma_i with one r per row,
// are those of p_i = x_i gamma_i: a positive factor common to a row moves its
// maximum and its values alike.  So q_i = round(p_i / (max|p| / 127)) needs no
// sum, and r = 1 / sqrt(mean x^2 + eps) enters the scale alone.
#include <climits>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>

#include "common.cuh"

namespace {

using namespace luce;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename TX> __device__ __forceinline__ TX from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// The larger of m and |v|; a NaN stays.
__device__ __forceinline__ float max_abs(float m, float v)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

// The same of two 16-bit values at once (as m, v's bits without their signs).
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t v, __nv_bfloat16)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(v & 0x7fff7fffu));
    return r;
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t v, __half)
{
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(v & 0x7fff7fffu));
    return r;
}

// Sum of squares and largest |p| of a row over its threads: `lanes` of a warp, or the whole block.
template <bool NORM> __device__ __forceinline__ void row_totals(float &ss, float &m, int lanes)
{
    __shared__ float s_ss[32];
    __shared__ uint32_t s_m[32];
    uint32_t mb = __float_as_uint(m); // ordered like the values, which are not negative; a NaN lies above infinity
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o < lanes) {
            if (NORM)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (lanes < 32)
                mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        }
    }
    if (lanes >= 32)
        mb = __reduce_max_sync(0xffffffffu, mb);
    if (lanes > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
            if (NORM)
                s_ss[warp] = ss;
            s_m[warp] = mb;
        }
        __syncthreads();
        if (NORM)
            ss = warp_sum(lane < warps ? s_ss[lane] : 0.0f);
        mb = __reduce_max_sync(0xffffffffu, lane < warps ? s_m[lane] : 0u);
    }
    m = __uint_as_float(mb);
}

__device__ __forceinline__ int code_of(float p, float d)
{
    return (int)fminf(fmaxf(roundf(__fdiv_rn(p, d)), -127.0f), 127.0f);
}

// Codes of V values, four to a word.  round(fl(p / d)) is the whole number
// nearest p rinv wherever that is not within 1e-4 of half way between two
// (|p / d| <= 127.0001, and rinv = fl(1 / d) moves it by less than 2e-5), which
// four operations per value find: the sum with 1.5 2^23 rounds to a whole
// number and leaves it in the low bits.  Chunks with a value near half way (or
// a d whose reciprocal overflows: the distance is then a NaN) divide.  Division
// throughout took 54.9 us for 8191 x 4096 bf16 rows with a residual, this 42.3.
template <int V> __device__ __forceinline__ void codes_of(const float (&p)[V], float d, float rinv, uint32_t (&w)[V / 4])
{
    constexpr float M = 12582912.0f;
    uint32_t u[V];
    bool near_half = false;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const float r = fmaf(p[i], rinv, M);
        u[i] = __float_as_uint(r);
        near_half |= !(fabsf(fmaf(p[i], rinv, -__fsub_rn(r, M))) <= 0.4999f);
    }
    if (near_half) {
#pragma unroll
        for (int i = 0; i < V; i++)
            u[i] = (uint32_t)code_of(p[i], d);
    }
#pragma unroll
    for (int i = 0; i < V; i += 4)
        w[i / 4] = __byte_perm(__byte_perm(u[i], u[i + 1], 0x0040), __byte_perm(u[i + 2], u[i + 3], 0x0040), 0x5410);
}

// Squares below the normal range keep 2^-150 of error each, and so does their
// mean: nothing to a mean (with eps) of TINY or more, but too much below it,
// where r itself leaves the range of fp32.  Such a row's scale is left at
// infinity for k_tiny_rows, which follows where eps is below TINY.
constexpr float TINY = 0x1p-120f;

// (a row of zeros has scale zero whatever r is: 1 / 0 when eps is zero too)
__device__ __forceinline__ float scale_of(float d, float ss, int H, float eps, bool norm, bool finite)
{
    const float r2 = __fadd_rn(__fdiv_rn(ss, (float)H), eps), r = __fdiv_rn(1.0f, __fsqrt_rn(r2));
    return !finite ? NAN : norm && d > 0.0f ? (r2 < TINY ? INFINITY : __fmul_rn(d, r)) : d;
}

// ---------------------------------------------------------------------------
// A row in registers: NCH chunks of 16 bytes of x per thread, read once (with
// the residual beside them), codes written once.  Many fp32 rows, and rows with
// a residual, are bound by HBM (add + norm 8191 x 4096 fp32: 63.1 us, a plain copy
// of the bytes 64.5); many 16-bit rows without one by instruction issue, the
// rounding and its half-way test going value by value (quantize 8191 x 4096 bf16
// 20.7 us, the bytes alone 14.9; normed 35.9).  The 32 values of a thread spread what
// every thread does once (the totals, three divisions) thin: with 16 those rows
// took 33 us instead of 24, and with their largest value found two at a time
// 21.  For few rows it is latency: one chunk a thread, all loads at once, one barrier.
//
// blockDim.x threads to a row: 8, 16 or 32 lanes of a warp (blockDim.y rows to
// the block, no barrier), or the block.
//
// ALIGNED: every row starts 16-byte aligned in every array.  Otherwise chunk j
// holds the elements j V - a .. j V - a + V - 1 of the row, a the row's offset
// in x from a 16-byte boundary (the residual and the sum share it: checked by
// the host), the first and last chunk element by element; the codes, whose
// rows lie at other offsets, go through shared memory and leave in 16-byte
// stores (8191 x 4099 fp32 rows: 36.8 us, aligned ones of 4096 27.5; stores of
// 4 or 8 bytes took longer).
template <typename TX, int NCH, bool ALIGNED, bool NORM>
__global__ void __launch_bounds__(1024)
    k_rows_i8(const TX *x, const TX *res, TX *xsum, const float *__restrict__ gamma, float eps, int T, int H, int8_t *q,
              float *scale)
{
    constexpr int V = 16 / sizeof(TX);
    extern __shared__ __align__(16) uint32_t codes[]; // [rows of the block][pitch] (unaligned rows)
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * blockDim.y + threadIdx.y, lanes = blockDim.x;
    const bool live_row = t < T;
    const size_t row = (size_t)(live_row ? t : 0) * H;
    const int n = live_row ? H : 0;
    const int a = ALIGNED ? 0 : (int)((reinterpret_cast<uintptr_t>(x + row) & 15) / sizeof(TX));
    const bool gamma16 = (reinterpret_cast<uintptr_t>(gamma) & 15) == 0;
    const bool in_place = !ALIGNED && (xsum == x || xsum == res) && xsum != nullptr;
    union Chunk {
        uint4 w;
        TX e[V];
    };
    Chunk cx[NCH], cr[NCH];
    auto first = [&](int c) { return (int)(threadIdx.x + c * lanes) * V - a; }; // element of the thread's chunk c
    auto is_whole = [&](int e0) { return ALIGNED ? e0 < n : e0 >= 0 && e0 + V <= n; };
    auto load_edge = [&](Chunk &c, const TX *p, int e0) { // those of them that lie in the row, if not all do
        if (e0 >= n)
            return;
        // whole where the neighbouring row fills it (and nothing is stored to it
        // meanwhile), its other elements set to zero
        if (!in_place && (long long)row + e0 >= 0 && row + e0 + V <= (size_t)T * H) {
            c.w = *reinterpret_cast<const uint4 *>(p + e0);
#pragma unroll
            for (int i = 0; i < V; i++)
                if (e0 + i < 0 || e0 + i >= n)
                    c.e[i] = from_f32<TX>(0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (e0 + i >= 0 && e0 + i < n)
                    c.e[i] = p[e0 + i];
        }
    };
    auto load = [&](Chunk &c, const TX *p, int e0) { // elements e0 .. e0 + V - 1 of the row
        if (is_whole(e0)) {
            c.w = *reinterpret_cast<const uint4 *>(p + e0);
        } else {
            c.w = make_uint4(0, 0, 0, 0);
            if (!ALIGNED && !NORM)
                load_edge(c, p, e0);
        }
    };
#pragma unroll
    for (int c = 0; c < NCH; c++)
        load(cx[c], x + row, first(c));
    if (NORM && res) {
#pragma unroll
        for (int c = 0; c < NCH; c++)
            load(cr[c], res + row, first(c));
    }
    if (!ALIGNED && NORM) {
        // the two threads of a row that hold its edges, apart from the others (3282 x 7374
        // fp32 rows with a residual: 60.2 us, chunk by chunk as above 68.4; luce_quantize_i8
        // of 8191 x 4099 fp32: 39.6 and 36.8)
        bool edge = false;
#pragma unroll
        for (int c = 0; c < NCH; c++)
            edge |= !is_whole(first(c)) && first(c) < n;
        if (edge) {
#pragma unroll
            for (int c = 0; c < NCH; c++) {
                if (is_whole(first(c)))
                    continue;
                load_edge(cx[c], x + row, first(c));
                if (res)
                    load_edge(cr[c], res + row, first(c));
            }
        }
    }
    // gamma of a chunk (one for elements behind the row's ends, which are zero)
    auto gammas = [&](int e0, bool whole, float (&g)[V]) {
        if (ALIGNED) {
            if (whole) {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(gamma + e0 + i));
                    g[i] = w.x, g[i + 1] = w.y, g[i + 2] = w.z, g[i + 3] = w.w;
                }
            }
        } else if (whole && gamma16 && e0 + V + 4 <= n) {
            // the 16-byte pieces of gamma around the chunk, moved down by the row's e0 mod 4 (8191 x
            // 4099 bf16 rows with a residual: 65.0 us, with loads of single elements 71.2)
            const int s = e0 & 3;
            float h[V + 4];
#pragma unroll
            for (int i = 0; i < V + 4; i += 4) {
                const float4 w = __ldg(reinterpret_cast<const float4 *>(gamma + (e0 - s) + i));
                h[i] = w.x, h[i + 1] = w.y, h[i + 2] = w.z, h[i + 3] = w.w;
            }
#pragma unroll
            for (int i = 0; i < V + 2; i++)
                h[i] = s & 1 ? h[i + 1] : h[i];
#pragma unroll
            for (int i = 0; i < V; i++)
                g[i] = s & 2 ? h[i + 2] : h[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                g[i] = whole || (e0 + i >= 0 && e0 + i < n) ? __ldg(gamma + e0 + i) : 1.0f;
        }
    };
    auto scaled = [&](const Chunk &c, int e0, bool whole, float (&p)[V]) {
        float g[V] = {};
        if constexpr (NORM)
            gammas(e0, whole, g);
#pragma unroll
        for (int i = 0; i < V; i++)
            p[i] = NORM ? __fmul_rn(to_f32(c.e[i]), g[i]) : to_f32(c.e[i]);
    };
    // few values a thread: gamma is requested beside them
    constexpr bool EARLY = NORM && NCH * V <= 16;
    float p[NORM ? NCH : 1][V] = {};
    if constexpr (EARLY) {
#pragma unroll
        for (int c = 0; c < NCH; c++) {
            const int e0 = first(c);
            gammas(e0, is_whole(e0), p[c]);
        }
    }
    float ss = 0.0f, m = 0.0f;
    uint32_t mm = 0;
#pragma unroll
    for (int c = 0; c < NCH; c++) {
        const int e0 = first(c);
        const bool whole = is_whole(e0);
        if (res) {
#pragma unroll
            for (int i = 0; i < V; i++)
                cx[c].e[i] = from_f32<TX>(__fadd_rn(to_f32(cx[c].e[i]), to_f32(cr[c].e[i])));
        }
        if (xsum) {
            if (whole) {
                *reinterpret_cast<uint4 *>(xsum + row + e0) = cx[c].w;
            } else if (!ALIGNED) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    if (e0 + i >= 0 && e0 + i < n)
                        xsum[row + e0 + i] = cx[c].e[i];
            }
        }
        float pc[V];
        if constexpr (EARLY) {
#pragma unroll
            for (int i = 0; i < V; i++)
                pc[i] = __fmul_rn(to_f32(cx[c].e[i]), p[c][i]);
        } else {
            scaled(cx[c], e0, whole, pc);
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (NORM) {
                const float v = to_f32(cx[c].e[i]);
                ss = fmaf(v, v, ss);
                p[NORM ? c : 0][i] = pc[i];
            }
            if (!ALIGNED || NORM || V == 4)
                m = max_abs(m, pc[i]);
        }
        if constexpr (ALIGNED && !NORM && V == 8) {
            mm = max_abs2(mm, cx[c].w.x, TX());
            mm = max_abs2(mm, cx[c].w.y, TX());
            mm = max_abs2(mm, cx[c].w.z, TX());
            mm = max_abs2(mm, cx[c].w.w, TX());
        }
    }
    if constexpr (ALIGNED && !NORM && V == 8) {
        const TX *h = reinterpret_cast<const TX *>(&mm);
        m = max_abs(to_f32(h[0]), to_f32(h[1]));
    }
    row_totals<NORM>(ss, m, lanes);
    const bool finite = m < INFINITY;
    const float d = __fdiv_rn(m, 127.0f);
    const bool live = finite && d > 0.0f;
    const float rinv = __fdiv_rn(1.0f, d);
    if (threadIdx.x == 0 && live_row)
        scale[t] = scale_of(d, ss, H, eps, NORM, finite);
    int8_t *qr = q + row;
    const int pitch = (H + 32) / 16 * 4; // words
    uint32_t *buf = codes + threadIdx.y * pitch;
#pragma unroll
    for (int c = 0; c < NCH; c++) {
        const int e0 = first(c);
        const bool whole = is_whole(e0);
        uint32_t w[V / 4] = {};
        if (live) {
            if constexpr (NORM) {
                codes_of<V>(p[c], d, rinv, w);
            } else {
                float pc[V];
                scaled(cx[c], e0, whole, pc);
                codes_of<V>(pc, d, rinv, w);
            }
        }
        if (e0 < n) {
            if (ALIGNED) {
                if constexpr (V == 4)
                    *reinterpret_cast<uint32_t *>(qr + e0) = w[0];
                else
                    *reinterpret_cast<uint2 *>(qr + e0) = make_uint2(w[0], w[V / 4 - 1]);
            } else {
#pragma unroll
                for (int i = 0; i < V / 4; i++)
                    buf[(e0 + a) / 4 + i] = w[i]; // (byte e + a of the buffer is element e)
            }
        }
    }
    if (!ALIGNED) {
        if (lanes <= 32)
            __syncwarp();
        else
            __syncthreads();
        // 16-byte pieces of the row at 16-byte boundaries of q: piece i starts at element 16 i - b
        const int b = (int)(reinterpret_cast<uintptr_t>(qr) & 15);
        for (int i = threadIdx.x; 16 * i < b + n; i += lanes) {
            const int e = 16 * i - b, s = e + a; // first element, its byte in the buffer
            if (e >= 0 && e + 16 <= n) {
                const uint32_t *src = buf + (s >> 2);
                uint32_t w[5];
#pragma unroll
                for (int k = 0; k < 5; k++)
                    w[k] = src[k]; // (the last one may lie behind the row, within the pitch)
                const uint32_t sh = 8 * (s & 3);
                *reinterpret_cast<uint4 *>(qr + e) =
                    make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                               __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
            } else {
                const int8_t *bytes = reinterpret_cast<const int8_t *>(buf);
                for (int k = max(e, 0); k < min(e + 16, n); k++)
                    qr[k] = bytes[k + a];
            }
        }
    }
}

// Any row: one block per row, two passes over it (rows longer than the
// registers of a block hold, or a residual at another offset than x).
constexpr int THREADS = 512;

template <typename TX>
__global__ void __launch_bounds__(THREADS)
    k_rows_i8_any(const TX *x, const TX *res, TX *xsum, const float *gamma, float eps, int T, int H, int8_t *q,
                  float *scale)
{
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const size_t row = (size_t)t * H;
    auto value = [&](int i) {
        const float v = to_f32(x[row + i]);
        return res ? from_f32<TX>(__fadd_rn(v, to_f32(res[row + i]))) : x[row + i];
    };
    float ss = 0.0f, m = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < H; i += THREADS) {
        const float v = to_f32(value(i));
        ss = fmaf(v, v, ss);
        m = max_abs(m, gamma ? __fmul_rn(v, gamma[i]) : v);
    }
    row_totals<true>(ss, m, THREADS);
    const bool finite = m < INFINITY;
    const float d = __fdiv_rn(m, 127.0f);
    const bool live = finite && d > 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < H; i += THREADS) {
        const TX s = value(i);
        const float v = to_f32(s);
        if (xsum)
            xsum[row + i] = s;
        q[row + i] = live ? (int8_t)code_of(gamma ? __fmul_rn(v, gamma[i]) : v, d) : (int8_t)0;
    }
    if (threadIdx.x == 0)
        scale[t] = scale_of(d, ss, H, eps, gamma != nullptr, finite);
}

// The scales of normed rows that the kernels above left at infinity, a warp to
// a row: squares in 64 bits, whose range holds those of all fp32 numbers.  Rare:
// one look at every scale is what it costs a call with such a small eps.
constexpr int TINY_WARPS = 8;

template <typename TX>
__global__ void __launch_bounds__(TINY_WARPS * 32)
    k_tiny_rows(const TX *x, const TX *res, const TX *xsum, const float *gamma, float eps, int T, int H, float *scale)
{
    pdl_wait();
    pdl_trigger();
    const int64_t t = (int64_t)blockIdx.x * TINY_WARPS + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= T || scale[t] != INFINITY)
        return;
    const size_t row = (size_t)t * H;
    double ss = 0.0;
    float m = 0.0f;
    for (int i = lane; i < H; i += 32) {
        const float v = xsum  ? to_f32(xsum[row + i])
                        : res ? to_f32(from_f32<TX>(__fadd_rn(to_f32(x[row + i]), to_f32(res[row + i]))))
                              : to_f32(x[row + i]);
        ss += (double)v * (double)v;
        m = fmaxf(m, fabsf(__fmul_rn(v, gamma[i])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    m = warp_max(m);
    if (lane == 0)
        scale[t] = (float)((double)__fdiv_rn(m, 127.0f) / sqrt(ss / H + (double)eps));
}

constexpr int H_MAX = 65536;

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

template <typename TX, int NCH>
luce_status launch_rows(const TX *x, const TX *res, TX *xsum, const float *gamma, float eps, int T, int H, int8_t *q,
                        float *scale, int threads, bool aligned_rows, cudaStream_t stream)
{
    const int rows = threads <= 32 ? 256 / threads : 1;
    const dim3 grid((unsigned)(((int64_t)T + rows - 1) / rows)), block((unsigned)threads, (unsigned)rows);
    const size_t smem = aligned_rows ? 0 : (size_t)rows * ((H + 32) / 16 * 16);
    auto run = [&](auto kern) {
        return luce_host::launch(kern, grid, block, smem, stream, x, res, xsum, gamma, eps, T, H, q, scale);
    };
    if (gamma)
        return aligned_rows ? run(k_rows_i8<TX, NCH, true, true>) : run(k_rows_i8<TX, NCH, false, true>);
    return aligned_rows ? run(k_rows_i8<TX, NCH, true, false>) : run(k_rows_i8<TX, NCH, false, false>);
}

// Chunks of a thread (of V values each) for T rows of `chunks` chunks.  One
// chunk makes the shortest way through a row, but holds many threads, whose
// totals and divisions many rows then pay for; more chunks leave room for more
// rows on an SM.  Every choice timed for seven widths and 200 to 8191 rows, in
// us (one, two, four chunks; eight for fp32):
//   quantize bf16  512 x 1024: 2.1 2.4 3.3        1024 x 14336: -  18.3 14.1
//                  512 x 4099: 5.8 4.9 5.5        2048 x 6319: 31.3 16.4 14.2
//   quantize fp32  512 x 1024: 2.2 2.3 2.5 3.1    2048 x 8192:  -  20.0 19.3 16.6
//   norm bf16     4000 x 4096: 22.9 23.6 24.5     2048 x 6319: 55.4 33.2 29.6
//   norm fp32      512 x 1024: 3.7 3.8 4.1 6.6    2048 x 4096: 21.9 21.3 18.1 23.7
int chunks_of_a_thread(int V, bool norm, bool aligned_rows, int T, int chunks)
{
    const int64_t work = (int64_t)T * chunks, K = 1024;
    if (chunks <= 32)
        return 1; // a row to a warp, or less
    if (norm && V == 8) {
        if (aligned_rows)
            return chunks <= 1024 ? 1 : 4;
        return work <= 110 * K ? 1 : chunks <= 600 || work <= 200 * K ? 2 : 4;
    }
    if (norm)
        return work <= 250 * K ? 1 : 4;
    if (work <= (aligned_rows ? 280 : 110) * K)
        return 1;
    if (V == 8)
        return (aligned_rows ? (work > 450 * K && chunks >= 512) || chunks > 1024 : work > 330 * K) ? 4 : 2;
    return (aligned_rows ? work > 2000 * K || (work > 600 * K && chunks >= 2048) : work > 500 * K) ? 8 : 2;
}

// Whether five chunks of a thread pay where four would do.  The blocks of both
// have 64 registers a thread (unaligned bf16 rows 56), 1024 threads to an SM:
// five chunks do where the rows then take fewer rounds of blocks.  Aligned bf16 rows spill with five: never
// when normed, else only where a second block fits an SM for it.  us with four
// and five: quantize bf16 4096 x 4099 17.2 16.2, 8191 x 5120 26.4 27.1, 4096 x
// 20480 71.7 58.4; fp16 8191 x 5120 26.2 24.0, 4096 x 20480 73.5 50.9; norm
// bf16 1024 x 6319 13.0 13.9, 8191 x 6319 66.7 63.1, 8191 x 10240 69.8 95.7;
// fp16 8191 x 10240 64.3 59.7, 4096 x 15360 52.9 56.7, 4096 x 20480 91.4 66.2.
template <typename TX> bool five_chunks(bool norm, bool aligned_rows, int T, int chunks)
{
    constexpr bool BF16 = std::is_same_v<TX, __nv_bfloat16>;
    const int resident = BF16 && !norm && !aligned_rows ? 65536 / 56 : 1024;                 // threads of an SM
    auto blocks = [&](int k) { return resident / (((chunks + k - 1) / k + 31) / 32 * 32); }; // of an SM
    if (chunks > 4 * 1024)
        return true; // (four would not do)
    if (BF16 && aligned_rows && (norm || blocks(4) > 1))
        return false;
    auto rounds = [&](int k) {
        const int64_t at_once = (int64_t)luce_host::sm_count() * blocks(k);
        return (T + at_once - 1) / at_once;
    };
    return rounds(5) < rounds(4);
}

template <typename TX>
luce_status launch_tiny_rows(const TX *x, const TX *res, const TX *xsum, const float *gamma, float eps, int T, int H,
                             float *scale, cudaStream_t stream)
{
    const dim3 grid((unsigned)(((int64_t)T + TINY_WARPS - 1) / TINY_WARPS));
    return luce_host::launch(k_tiny_rows<TX>, grid, dim3(TINY_WARPS * 32), 0, stream, x, res, xsum, gamma, eps, T, H, scale);
}

template <typename TX>
luce_status run_rows(const void *vx, const void *vres, void *vsum, const float *gamma, float eps, int T, int H,
                     int8_t *q, float *scale, void *vstream)
{
    using luce_host::aligned;
    constexpr int V = 16 / sizeof(TX);
    const TX *x = (const TX *)vx, *res = (const TX *)vres;
    TX *xsum = (TX *)vsum;
    cudaStream_t stream = luce_host::as_stream(vstream);
    const bool al = H % V == 0 && aligned(x, 16) && (!res || aligned(res, 16)) && (!xsum || aligned(xsum, 16)) &&
                    (!gamma || aligned(gamma, 16)) && aligned(q, V);
    auto off = [](const void *p) { return reinterpret_cast<uintptr_t>(p) & 15; };
    const bool one_offset = (!res || off(res) == off(x)) && (!xsum || off(xsum) == off(x));
    const int chunks = al ? H / V : (H + V - 1) / V + 1; // 16-byte pieces of a row
    int nch = chunks_of_a_thread(V, gamma != nullptr, al, T, chunks);
    while (nch < 32 / V && chunks > 1024 * nch)
        nch *= 2;
    // warps are whole: the next number of chunks where it leaves no more of them to go through in all
    auto in_all = [&](int k) { return ((chunks + k - 1) / k + 31) / 32 * k; };
    if (V == 8 && nch == 4 && !res && in_all(5) <= in_all(4) && five_chunks<TX>(gamma != nullptr, al, T, chunks))
        nch = 5;
    if (V == 4 && nch == 4 && chunks <= 256 && in_all(2) < in_all(4)) // (3577 x 758 fp32, normed: 10.5 us, with four 12.1)
        nch = 2;
    if (!one_offset || chunks > 1024 * nch)
        return luce_host::launch(k_rows_i8_any<TX>, dim3((unsigned)T), dim3(THREADS), 0, stream, x, res, xsum, gamma,
                                 eps, T, H, q, scale);
    const int need = (chunks + nch - 1) / nch;
    int threads = need > 32 ? (need + 31) & ~31 : 8;
    while (threads < need)
        threads *= 2;
    switch (nch) {
    case 1:
        return launch_rows<TX, 1>(x, res, xsum, gamma, eps, T, H, q, scale, threads, al, stream);
    case 2:
        return launch_rows<TX, 2>(x, res, xsum, gamma, eps, T, H, q, scale, threads, al, stream);
    case 4:
        return launch_rows<TX, 4>(x, res, xsum, gamma, eps, T, H, q, scale, threads, al, stream);
    case 5:
        if constexpr (V == 8)
            return launch_rows<TX, 5>(x, res, xsum, gamma, eps, T, H, q, scale, threads, al, stream);
        [[fallthrough]];
    default:
        return launch_rows<TX, 32 / V>(x, res, xsum, gamma, eps, T, H, q, scale, threads, al, stream);
    }
}

// the three entry points: gamma is NULL for the plain rows, res and xsum for those without a residual
luce_status rows_i8(const void *x, const void *res, void *xsum, luce_dtype dtype, const float *gamma, float eps, int T,
                    int H, int8_t *q, float *scale, void *stream)
{
    using luce_host::aligned;
    if (T < 0 || H < 1 || H > H_MAX || (dtype != LUCE_F32 && dtype != LUCE_BF16 && dtype != LUCE_F16) ||
        !(eps >= 0.0f) || !std::isfinite(eps))
        return LUCE_ERR_INVALID_ARG;
    if (T == 0)
        return LUCE_OK;
    const size_t es = dtype == LUCE_F32 ? 4 : 2, nx = (size_t)T * H * es, nq = (size_t)T * H, ns = (size_t)T * 4;
    if (!x || !q || !scale || !aligned(x, es) || !aligned(scale, 4) || (gamma && !aligned(gamma, 4)) ||
        (res && !aligned(res, es)) || (xsum && !aligned(xsum, es)))
        return LUCE_ERR_INVALID_ARG;
    if (xsum && ((xsum != x && overlap(xsum, nx, x, nx)) || (xsum != res && overlap(xsum, nx, res, nx)) ||
                 overlap(xsum, nx, q, nq) || overlap(xsum, nx, scale, ns)))
        return LUCE_ERR_INVALID_ARG;
    const size_t ng = (size_t)H * 4;
    if (overlap(q, nq, x, nx) || overlap(scale, ns, x, nx) || overlap(q, nq, scale, ns) ||
        (res && (overlap(q, nq, res, nx) || overlap(scale, ns, res, nx))) ||
        (gamma && (overlap(q, nq, gamma, ng) || overlap(scale, ns, gamma, ng) ||
                   (xsum && overlap(xsum, nx, gamma, ng)))))
        return LUCE_ERR_INVALID_ARG;
    auto run = [&](auto element) {
        using TX = decltype(element);
        const luce_status st = run_rows<TX>(x, res, xsum, gamma, eps, T, H, q, scale, stream);
        if (st != LUCE_OK || !gamma || eps >= TINY)
            return st;
        return launch_tiny_rows<TX>((const TX *)x, (const TX *)res, (const TX *)xsum, gamma, eps, T, H, scale,
                                    luce_host::as_stream(stream));
    };
    switch (dtype) {
    case LUCE_F32:
        return run(float());
    case LUCE_BF16:
        return run(__nv_bfloat16());
    case LUCE_F16:
        return run(__half());
    }
    return LUCE_ERR_INVALID_ARG;
}

} // namespace

extern "C" luce_status luce_quantize_i8(const void *x, luce_dtype dtype, int T, int H, int8_t *q, float *scale,
                                        void *stream)
{
    return rows_i8(x, nullptr, nullptr, dtype, nullptr, 0.0f, T, H, q, scale, stream);
}

extern "C" luce_status luce_rmsnorm_i8(const void *x, luce_dtype dtype, const float *gamma, float eps, int T, int H,
                                       int8_t *q, float *scale, void *stream)
{
    if (!gamma && T > 0)
        return LUCE_ERR_INVALID_ARG;
    return rows_i8(x, nullptr, nullptr, dtype, gamma, eps, T, H, q, scale, stream);
}

extern "C" luce_status luce_add_rmsnorm_i8(const void *x, const void *residual, void *x_sum, luce_dtype dtype,
                                           const float *gamma, float eps, int T, int H, int8_t *q, float *scale,
                                           void *stream)
{
    if ((!gamma || !residual) && T > 0)
        return LUCE_ERR_INVALID_ARG;
    return rows_i8(x, residual, x_sum, dtype, gamma, eps, T, H, q, scale, stream);
}
