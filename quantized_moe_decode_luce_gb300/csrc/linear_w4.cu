// linear_w4.cu -- products with 4-bit weights that have a scale, and
// optionally a zero point, per group of 32, 64 or 128 values of a row
// (luce_linear_w4), with its C-ABI entry point.
//
//   out[t][n] = (sum_g s[n][g] * S[t][n][g]) (* x_scale[t]) (+ bias[n]),
//   S[t][n][g] = sum_{k in g} x[t][k] (q[n][k] - z[n][g])   (z = 8 without zero points)
//
// Codes are small whole numbers, exact in fp16 and bf16, so a group's sum runs
// on the tensor cores without rounding an operand: fp16 and int8 activations
// go in as fp16, bf16 ones as bf16, and fp32 ones as three bf16 numbers (8
// bits of the mantissa each), three columns that are added at the end.  The
// products are exact, their sums are fp32, and a group's scale multiplies its
// fp32 sum.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda_bf16.h>

#include "common.cuh"

namespace {

using namespace luce;

constexpr int CHUNK = 128;             // values of a row that its packed codes keep together
constexpr int CHUNK_BYTES = CHUNK / 2;
constexpr int K_MAX = 65536;

struct W4Args {
    const void *x;
    luce_dtype x_dtype;
    int parts; // columns of a token: three for fp32, else one
    int64_t ldx;
    const float *xs;
    const uint8_t *wq;
    const void *ws;
    bool ws_bf16;
    const uint8_t *zeros;
    const float *bias;
    int T, N, K, G; // G: groups of a row
    void *out;
    luce_dtype out_dtype;
    int64_t ldo;
};

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ float scale_of(uint32_t bits16, bool bf)
{
    return bf ? __uint_as_float(bits16 << 16) : half_bits_to_float(bits16);
}

__device__ __forceinline__ void store_as(void *out, luce_dtype t, int64_t i, float v)
{
    if (t == LUCE_F32)
        reinterpret_cast<float *>(out)[i] = v;
    else if (t == LUCE_BF16)
        reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
    else
        reinterpret_cast<__half *>(out)[i] = __float2half_rn(v);
}

// Eight codes of a word -> their differences with the zero point, four pairs
// in the order of the values (value i of a word has its bits 4 (i / 2) + 16 (i
// % 2) .. + 3).  A code placed under the exponent of 1024 (fp16) or 128 (bf16)
// is 1024 + q or 128 + q; z2 holds 1024 + z or 128 + z twice.  Bits 4 to 7 of
// an fp16 are the code times 16: one exact multiply-add undoes both.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b, __half)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b, __nv_bfloat16)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma2_f16(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// What a group's zero point contributes to the conversion of its codes.
template <typename E> struct Zero;
template <> struct Zero<__half> {
    uint32_t lo, hi; // 1024 + z; -(64 + z)
    __device__ __forceinline__ explicit Zero(uint32_t z)
    {
        lo = (0x6400u + z) * 0x10001u;
        hi = (0xD400u + 16u * z) * 0x10001u; // 64 .. 79 have steps of 1/16
    }
};
template <> struct Zero<__nv_bfloat16> {
    uint32_t lo;
    __device__ __forceinline__ explicit Zero(uint32_t z) { lo = (0x4300u + z) * 0x10001u; }
};

__device__ __forceinline__ void codes8(uint32_t w, const Zero<__half> &z, uint32_t (&h)[4])
{
    const uint32_t w8 = w >> 8;
    h[0] = sub2(and_or(w, 0x000f000fu, 0x64006400u), z.lo, __half());
    h[1] = fma2_f16(and_or(w, 0x00f000f0u, 0x64006400u), 0x2C002C00u, z.hi);
    h[2] = sub2(and_or(w8, 0x000f000fu, 0x64006400u), z.lo, __half());
    h[3] = fma2_f16(and_or(w8, 0x00f000f0u, 0x64006400u), 0x2C002C00u, z.hi);
}
__device__ __forceinline__ void codes8(uint32_t w, const Zero<__nv_bfloat16> &z, uint32_t (&h)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i++)
        h[i] = sub2(and_or(w >> (4 * i), 0x000f000fu, 0x43004300u), z.lo, __nv_bfloat16());
}

// ---------------------------------------------------------------------------
// Eight consecutive activations of a token as one or three operand octets.
__device__ __forceinline__ uint32_t pair_of(__half a, __half b)
{
    return (uint32_t)__half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
}
__device__ __forceinline__ void octets(const int8_t *p, uint4 (&o)[1])
{
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; i++) { // code + 128 under the exponent of 1024, less 1152: exact
        const uint32_t u = (i < 2 ? v.x : v.y) ^ 0x80808080u;
        h[i] = sub2(__byte_perm(u, 0x64646464u, (i & 1) ? 0x4342 : 0x4140), 0x64806480u, __half());
    }
    o[0] = make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ void octets(const __half *p, uint4 (&o)[1]) { o[0] = *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void octets(const __nv_bfloat16 *p, uint4 (&o)[1]) { o[0] = *reinterpret_cast<const uint4 *>(p); }
// An fp32 number is the sum of its top, middle and low eight mantissa bits,
// each a bf16 number (cut off, not rounded: the first cannot overflow, and
// the rests are exact).  NaN and infinities have no rest.
__device__ __forceinline__ void octets(const float *p, uint4 (&o)[3])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w[3][8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t bits = __float_as_uint(v[i]);
        const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
        const float r1 = finite ? __fsub_rn(v[i], __uint_as_float(bits & 0xffff0000u)) : 0.0f;
        const uint32_t m = __float_as_uint(r1) & 0xffff0000u;
        w[0][i] = finite || !(bits & 0x007fffffu) ? bits >> 16 : 0x7fffu;
        w[1][i] = m >> 16;
        w[2][i] = __float_as_uint(__fsub_rn(r1, __uint_as_float(m))) >> 16;
    }
#pragma unroll
    for (int j = 0; j < 3; j++)
        o[j] = make_uint4(w[j][0] | w[j][1] << 16, w[j][2] | w[j][3] << 16, w[j][4] | w[j][5] << 16, w[j][6] | w[j][7] << 16);
}

// Activations k .. k + 7 of token t, as operands of type E (fp16 from fp16 and
// int8, bf16 from bf16 and fp32): one octet, or three.
template <typename E> __device__ __forceinline__ void load_octets(const W4Args &a, int t, int k, uint4 (&o)[3])
{
    const int64_t at = t * a.ldx + k;
    uint4 one[1];
    if constexpr (std::is_same<E, __half>::value) {
        if (a.x_dtype == LUCE_I8)
            octets(reinterpret_cast<const int8_t *>(a.x) + at, one);
        else
            octets(reinterpret_cast<const __half *>(a.x) + at, one);
    } else {
        if (a.x_dtype == LUCE_F32) {
            octets(reinterpret_cast<const float *>(a.x) + at, o);
            return;
        }
        octets(reinterpret_cast<const __nv_bfloat16 *>(a.x) + at, one);
    }
    o[0] = one[0];
}

// ---------------------------------------------------------------------------
// Few columns: a stream of the weights through mma.sync (16 rows x 16 values
// times 16 values x 8 columns).
//
// What bounds it is the weights' way from HBM, and for small matrices the
// latency of getting there.  A tile is 16 rows; the wk warps of a row group
// split its chunks among them (every wk-th), so that a tile's rows come as one
// run of memory, and add their sums through shared memory.  The packed order
// lets a lane's 16 bytes of a chunk be its operands of eight MMAs: of word j
// the values 32 j + 8 (lane % 4) .. + 7, whose activations are 16 bytes too,
// with every group of 32 values in two MMAs.  A warp keeps U chunks' codes in
// registers and requests a chunk of a later tile as soon as it has used one.
// The activations stay in shared memory for all tiles of the CTA, converted
// once, rows 64 bytes off a multiple of 128 so that reads meet no conflict.
constexpr int S_WARPS = 8;
constexpr int ROWS = 16;
constexpr int U = 4;

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// GPC groups of a row in a chunk: their scales (16 bits each) and zero points
// (8 bits each), those beyond the row's G as zero.
template <int GPC> struct Groups {
    uint32_t s[(GPC + 1) / 2], z;
};
template <int GPC, bool ZEROS>
__device__ __forceinline__ void load_groups(Groups<GPC> &g, const W4Args &a, int row, int g0, bool whole)
{
    const uint16_t *s = reinterpret_cast<const uint16_t *>(a.ws) + (int64_t)row * a.G + g0;
    const uint8_t *z = a.zeros + (int64_t)row * a.G + g0;
    if constexpr (GPC == 1) {
        g.s[0] = __ldg(s);
        if (ZEROS)
            g.z = __ldg(z);
    } else {
        if (whole) { // (every row's groups are whole chunks, aligned)
            if constexpr (GPC == 2) {
                g.s[0] = __ldg(reinterpret_cast<const uint32_t *>(s));
                if (ZEROS)
                    g.z = __ldg(reinterpret_cast<const uint16_t *>(z));
            } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(s));
                g.s[0] = v.x, g.s[1] = v.y;
                if (ZEROS)
                    g.z = __ldg(reinterpret_cast<const uint32_t *>(z));
            }
        } else {
            g.z = 0;
#pragma unroll
            for (int i = 0; i < GPC; i++) {
                const uint32_t v = g0 + i < a.G ? __ldg(s + i) : 0u;
                if (i % 2 == 0)
                    g.s[i / 2] = v;
                else
                    g.s[i / 2] |= v << 16;
                if (ZEROS && g0 + i < a.G)
                    g.z |= (uint32_t)__ldg(z + i) << (8 * i);
            }
        }
    }
}

template <typename E, int NT, int GPC, bool ZEROS>
__global__ void __launch_bounds__(S_WARPS * 32, NT <= 2 ? 2 : 1)
    k_linear_w4_stream(const W4Args a, int wk, int tokens, int pitch, int steps, bool whole)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float4 part[2][S_WARPS][NT][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (int)blockIdx.y * tokens, nt = min(a.T - t0, tokens), P = a.parts, cols = nt * P;
    const int chunks = (a.K + CHUNK - 1) / CHUNK, row_bytes = chunks * CHUNK_BYTES;
    const int groups = S_WARPS / wk, kw = warp % wk, per = (chunks + wk - 1) / wk; // row groups of the CTA; chunks of a warp and tile
    const int quad = lane & 3, r8 = lane >> 2;
    const int rows_step = groups * ROWS; // rows of the CTA at a step
    const int my_row = (warp / wk) * ROWS + r8;

    pdl_wait(); // (weights too may be the previous kernel's: luce_quantize_w4 writes them)
    pdl_trigger();

    struct Slot {
        uint4 w[2];
        Groups<GPC> g[2];
    } slot[U];
    auto load = [&](Slot &s, int step, int j) {
        const int c = kw + j * wk;
        if (step < steps && c < chunks) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int row = (int)min((int64_t)step * rows_step + my_row + 8 * h, (int64_t)a.N - 1);
                s.w[h] = ldg_stream(a.wq + (int64_t)row * row_bytes + c * CHUNK_BYTES + 16 * quad);
                load_groups<GPC, ZEROS>(s.g[h], a, row, c * GPC, whole);
            }
        }
    };
    int ls = blockIdx.x, lj = 0; // the chunk to request next
    auto request = [&](Slot &s) {
        load(s, ls, lj);
        if (++lj == per)
            lj = 0, ls += gridDim.x;
    };
#pragma unroll
    for (int u = 0; u < U; u++)
        request(slot[u]);

    // activations into shared memory, zero from K to the chunk's end
    const int units = chunks * (CHUNK / 8);
    for (int i = threadIdx.x; i < nt * units; i += S_WARPS * 32) {
        const int t = i / units, k = (i % units) * 8;
        uint4 o[3] = {};
        if (k < a.K)
            load_octets<E>(a, t0 + t, k, o);
#pragma unroll
        for (int p = 0; p < 3; p++)
            if (p < P)
                *reinterpret_cast<uint4 *>(smem + (size_t)(t * P + p) * pitch + 2 * k) = o[p];
    }
    __syncthreads();

    const uint8_t *xcol[NT]; // (columns beyond the last repeat it; their sums are not stored)
#pragma unroll
    for (int n = 0; n < NT; n++)
        xcol[n] = smem + (size_t)min(8 * n + r8, cols - 1) * pitch + 16 * quad;

    float acc[NT][4] = {};
    int us = blockIdx.x, uj = 0, buf = 0;
    auto use = [&](const Slot &s) {
        const int c = kw + uj * wk;
        if (c >= chunks)
            return;
        constexpr int JG = 4 / GPC; // words of a group
#pragma unroll
        for (int gi = 0; gi < GPC; gi++) {
            float sum[NT][4] = {};
            const Zero<E> z0(ZEROS ? (s.g[0].z >> (8 * gi)) & 15u : 8u), z1(ZEROS ? (s.g[1].z >> (8 * gi)) & 15u : 8u);
#pragma unroll
            for (int j = gi * JG; j < (gi + 1) * JG; j++) {
                uint32_t h0[4], h1[4];
                codes8(j == 0 ? s.w[0].x : j == 1 ? s.w[0].y : j == 2 ? s.w[0].z : s.w[0].w, z0, h0);
                codes8(j == 0 ? s.w[1].x : j == 1 ? s.w[1].y : j == 2 ? s.w[1].z : s.w[1].w, z1, h1);
                const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(xcol[n] + c * (2 * CHUNK) + j * 64);
                    mma(sum[n], a0, b.x, b.y, E());
                    mma(sum[n], a1, b.z, b.w, E());
                }
            }
            const float s0 = scale_of((s.g[0].s[gi / 2] >> (16 * (gi & 1))) & 0xffffu, a.ws_bf16);
            const float s1 = scale_of((s.g[1].s[gi / 2] >> (16 * (gi & 1))) & 0xffffu, a.ws_bf16);
#pragma unroll
            for (int n = 0; n < NT; n++) {
                acc[n][0] = fmaf(s0, sum[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, sum[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, sum[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, sum[n][3], acc[n][3]);
            }
        }
    };
    auto finish = [&]() { // the rows of a step: the warps' sums joined and stored
#pragma unroll
        for (int n = 0; n < NT; n++) {
            part[buf][warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        }
        __syncthreads();
        // (the next step writes the other half of part, and cannot come back to this one before its own barrier)
        for (int i = threadIdx.x; i < rows_step * nt; i += S_WARPS * 32) {
            const int t = i / rows_step, r = i % rows_step, g = r / ROWS, rr = r % ROWS;
            const int64_t n = (int64_t)us * rows_step + r;
            if (n >= a.N)
                continue;
            float v = 0.0f;
            for (int p = P - 1; p >= 0; p--) {
                const int c = t * P + p;
                float sum = 0.0f;
                for (int w = 0; w < wk; w++)
                    sum += reinterpret_cast<const float *>(&part[buf][g * wk + w][c / 8][(rr & 7) * 4 + (c % 8) / 2])[(rr >> 3) * 2 + (c & 1)];
                v += sum;
            }
            if (a.xs)
                v = __fmul_rn(v, a.xs[t0 + t]);
            if (a.bias)
                v = __fadd_rn(v, a.bias[n]);
            store_as(a.out, a.out_dtype, (t0 + t) * a.ldo + n, v);
        }
        buf ^= 1;
    };
    while (us < steps) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (us < steps) {
                use(slot[u]);
                request(slot[u]);
                if (++uj == per) {
                    finish();
                    uj = 0, us += gridDim.x;
                }
            }
        }
    }
}

constexpr size_t S_SMEM = 190 * 1024; // (32 KB of `part` beside it)

template <typename E, int NT, int GPC, bool ZEROS> luce_status launch_stream(const W4Args &a, int tokens, cudaStream_t stream)
{
    static luce_host::SmemLimit limit;
    const auto kern = k_linear_w4_stream<E, NT, GPC, ZEROS>;
    const int chunks = (a.K + CHUNK - 1) / CHUNK, pitch = chunks * 2 * CHUNK + 64;
    int wk = 1;
    while (wk < S_WARPS && wk < chunks)
        wk *= 2;
    const int rows = S_WARPS / wk * ROWS, steps = (a.N + rows - 1) / rows, blocks = (a.T + tokens - 1) / tokens;
    const size_t smem = (size_t)std::min(tokens, a.T) * a.parts * pitch;
    const bool whole = a.G % GPC == 0 && luce_host::aligned(a.ws, 2 * GPC) && (!ZEROS || luce_host::aligned(a.zeros, GPC));
    if (smem + 8192 * NT > 48 * 1024 && limit.raise(kern, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const int per_sm = (int)std::max<size_t>(1, std::min<size_t>(2, 220 * 1024 / (smem + 8192 * NT + 1024)));
    const int grid = std::min(steps, per_sm * luce_host::sm_count());
    const luce_status st = luce_host::launch(kern, dim3((unsigned)grid, (unsigned)blocks), dim3(S_WARPS * 32), smem, stream,
                                             a, wk, tokens, pitch, steps, whole);
    if (st != LUCE_OK)
        limit.forget();
    return st;
}

template <typename E, int GPC, bool ZEROS> luce_status run_w4(const W4Args &a, cudaStream_t stream)
{
    const int chunks = (a.K + CHUNK - 1) / CHUNK;
    const size_t column = (size_t)chunks * 2 * CHUNK + 64;
    const int room = (int)std::min<size_t>(32, S_SMEM / column), most = room / a.parts; // columns that fit; tokens
    if (most < 1)
        return LUCE_ERR_UNSUPPORTED;
    const int tokens = std::min(a.T, most), nt = (tokens * a.parts + 7) / 8;
    switch (nt) {
    case 1:
        return launch_stream<E, 1, GPC, ZEROS>(a, tokens, stream);
    case 2:
        return launch_stream<E, 2, GPC, ZEROS>(a, tokens, stream);
    default:
        return launch_stream<E, 4, GPC, ZEROS>(a, tokens, stream);
    }
}

template <typename E> luce_status run_type(const W4Args &a, int group, cudaStream_t stream)
{
    if (a.zeros)
        return group == 32 ? run_w4<E, 4, true>(a, stream) : group == 64 ? run_w4<E, 2, true>(a, stream) : run_w4<E, 1, true>(a, stream);
    return group == 32 ? run_w4<E, 4, false>(a, stream) : group == 64 ? run_w4<E, 2, false>(a, stream) : run_w4<E, 1, false>(a, stream);
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

} // namespace

extern "C" luce_status luce_linear_w4(const void *x, luce_dtype x_dtype, int64_t ld_x, const float *x_scale, const uint8_t *wq,
                                      const void *w_scale, luce_dtype scale_dtype, const uint8_t *zeros, int group,
                                      const float *bias, int T, int N, int K, void *out, luce_dtype out_dtype,
                                      int64_t ld_out, void *stream)
{
    using luce_host::aligned;
    constexpr int LIM = 1 << 24;
    if (T < 0 || T >= LIM || N < 1 || N >= LIM || K < 16 || K > K_MAX || K % 16 != 0 ||
        (group != 32 && group != 64 && group != 128) || (scale_dtype != LUCE_F16 && scale_dtype != LUCE_BF16) ||
        (out_dtype != LUCE_F32 && out_dtype != LUCE_BF16 && out_dtype != LUCE_F16) ||
        (x_dtype != LUCE_F32 && x_dtype != LUCE_BF16 && x_dtype != LUCE_F16 && x_dtype != LUCE_I8) || ld_x < K ||
        ld_out < N || ld_x > ((int64_t)1 << 33) || ld_out > ((int64_t)1 << 33))
        return LUCE_ERR_INVALID_ARG;
    if (T == 0)
        return LUCE_OK;
    const size_t ex = x_dtype == LUCE_F32 ? 4 : x_dtype == LUCE_I8 ? 1 : 2, eo = out_dtype == LUCE_F32 ? 4 : 2;
    if (!x || !wq || !w_scale || !out || !aligned(x, 16) || !aligned(wq, 16) || !aligned(w_scale, 2) || !aligned(out, eo) ||
        (bias && !aligned(bias, 4)) || (x_scale && !aligned(x_scale, 4)) || (x_dtype == LUCE_I8) != (x_scale != nullptr) ||
        (T > 1 && ld_x * ex % 16 != 0))
        return LUCE_ERR_INVALID_ARG;
    const int G = (K + group - 1) / group;
    const size_t no = ((size_t)(T - 1) * ld_out + N) * eo;
    if (overlap(out, no, x, ((size_t)(T - 1) * ld_x + K) * ex) ||
        overlap(out, no, wq, (size_t)N * ((K + CHUNK - 1) / CHUNK) * CHUNK_BYTES) || overlap(out, no, w_scale, (size_t)N * G * 2) ||
        (zeros && overlap(out, no, zeros, (size_t)N * G)) || (bias && overlap(out, no, bias, (size_t)N * 4)) ||
        (x_scale && overlap(out, no, x_scale, (size_t)T * 4)))
        return LUCE_ERR_INVALID_ARG;
    const W4Args a{x, x_dtype, x_dtype == LUCE_F32 ? 3 : 1, ld_x, x_scale, wq, w_scale, scale_dtype == LUCE_BF16, zeros, bias, T, N, K, G, out, out_dtype, ld_out};
    cudaStream_t st = luce_host::as_stream(stream);
    return x_dtype == LUCE_F32 || x_dtype == LUCE_BF16 ? run_type<__nv_bfloat16>(a, group, st) : run_type<__half>(a, group, st);
}
