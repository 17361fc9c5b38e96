// linear_w4.cu -- products with 4-bit weights that have a scale, and
// optionally a zero point, per group of 32, 64 or 128 values of a row
// (luce_linear_w4), with its C-ABI entry point.
//
//   out[t][n] = (sum_g s[n][g] * S[t][n][g]) (* x_scale[t]) (+ bias[n]),
//   S[t][n][g] = sum_{k in g} x[t][k] (q[n][k] - z[n][g])   (z = 8 without zero points)
//
// Operands.  The activations go in as fp16, a chunk of 128 of them (a row's packed
// codes are kept in such chunks) brought to one size by a power of two that
// multiplies the chunk's sums again in fp32:
//   whole numbers   int8 codes as they are; others as two columns of twelve bits
//     each, the second 2^-12 of the first.  What they leave is at most 2^-23 of
//     the chunk's largest value (2^-135 where all are below 2^-112), and a group's
//     sums (below 2^24) are exact: the tensor cores cut off what they add.
//   fp16 numbers    bf16 and fp16 values for 16-bit outputs, where two columns a
//     token would not fit one MMA: exact, but for values so far below the
//     chunk's largest that they end in fp16's subnormal steps (off by at most
//     2^-39 of it).
// With whole numbers a code becomes an operand by a mask alone: its four bits at the
// low end of an fp16 are the subnormal number q 2^-24, and four places higher
// 16 q 2^-24.  The factors 2^24 and 16 are put back in fp32 and in the
// activations, and the zero point is taken off a group's sum.  With fp16 numbers
// that would lose digits (the sums are aligned to the largest exponent, and
// subnormal ones are up to ten bits below theirs), so the codes become normal
// numbers, less their zero points: four instructions more for eight of them.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "w4.cuh"

namespace {

using namespace luce;
using namespace w4;

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// ---------------------------------------------------------------------------
// Activations as operands.  Sixteen lanes take a chunk of a token, eight
// values each.
__device__ __forceinline__ void load8(const W4Args &a, int t, int k, float (&v)[8])
{
    const int64_t at = t * a.ldx + k;
    if (a.x_dtype == LUCE_F32) {
        const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.x) + at);
        const float4 b = p[0], c = p[1];
        v[0] = b.x, v[1] = b.y, v[2] = b.z, v[3] = b.w, v[4] = c.x, v[5] = c.y, v[6] = c.z, v[7] = c.w;
    } else {
        const uint4 b = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(a.x) + at);
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
        if (a.x_dtype == LUCE_BF16) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = half_bits_to_float(w[i / 2] >> (16 * (i & 1)));
        }
    }
}

// Activations k .. k + 7 of token t (zero unless live) -> operands of one or two
// columns, the factors of the chunk's sums, and the sum of the group's values
// (GPC groups to a chunk, 16 / GPC lanes each) in the units of those sums, times
// eight.  As whole numbers values 2, 3, 6 and 7 of eight meet codes that count
// sixteenfold.  A NaN or an infinity stays one, and so do the sums of its group.
template <int GPC>
__device__ __forceinline__ void operands(const W4Args &a, int t, int k, bool live, uint4 (&o)[2], float (&factor)[2], float (&sum)[2])
{
    if (a.x_dtype == LUCE_I8) {
        const uint2 b = live ? *reinterpret_cast<const uint2 *>(reinterpret_cast<const int8_t *>(a.x) + t * a.ldx + k) : make_uint2(0, 0);
        int n = __dp4a((int)b.x, 0x01010101, __dp4a((int)b.y, 0x01010101, 0));
#pragma unroll
        for (int d = 1; d < 16 / GPC; d *= 2)
            n += __shfl_xor_sync(0xffffffffu, n, d);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) { // code + 128 under the exponent of 1024, less 1152: exact
            const uint32_t u = __byte_perm((i < 2 ? b.x : b.y) ^ 0x80808080u, 0x64646464u, i & 1 ? 0x4342 : 0x4140);
            const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __half2half2(__ushort_as_half(0x6480)));
            const __half2 s = i & 1 ? __hmul2(h, __half2half2(__ushort_as_half(0x2c00))) : h; // 2^-4
            w[i] = *reinterpret_cast<const uint32_t *>(&s);
        }
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        factor[0] = 16777216.0f / UNIT;
        sum[0] = (float)n * (8.0f / UNIT);
        return;
    }
    float v[8] = {};
    if (live)
        load8(a, t, k, v);
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++)
        most = fmaxf(most, fabsf(v[i]));
#pragma unroll
    for (int d = 1; d < 16; d *= 2)
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const uint32_t e = max(__float_as_uint(most) >> 23, a.whole ? 15u : 29u); // 2^(e - 127) <= most < 2^(e - 126)
    const float up = __uint_as_float(((a.whole ? 264u : 268u) - e) << 23);    // to below 2^11, or 2^15
    factor[0] = __uint_as_float((a.whole ? e : e - 28u) << 23);               // 2^24 / (up UNIT), 1 / (up UNIT)
    factor[1] = __uint_as_float((e - 12u) << 23);
    uint32_t w[2][4];
    sum[0] = sum[1] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float k16 = a.whole && (i & 2) ? 0.0625f : 1.0f, k1 = a.whole && (i & 2) ? 16.0f : 1.0f;
        const float x0 = v[i] * up, x1 = v[i + 1] * up;
        const float p0 = a.whole ? rintf(x0) : x0, p1 = a.whole ? rintf(x1) : x1;
        const __half2 h = __floats2half2_rn(p0 * k16, p1 * k16), r = __floats2half2_rn(rintf((x0 - p0) * 4096.0f) * k16, rintf((x1 - p1) * 4096.0f) * k16);
        const float2 f = __half22float2(h), g = __half22float2(r);
        w[0][i / 2] = *reinterpret_cast<const uint32_t *>(&h);
        w[1][i / 2] = *reinterpret_cast<const uint32_t *>(&r);
        sum[0] = fmaf(f.x + f.y, k1, sum[0]);
        sum[1] = fmaf(g.x + g.y, k1, sum[1]);
    }
#pragma unroll
    for (int p = 0; p < 2; p++) {
        if (p < a.parts) {
#pragma unroll
            for (int d = 1; d < 16 / GPC; d *= 2)
                sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], d);
            sum[p] *= factor[p] * (8.0f / 16777216.0f);
        }
        o[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
}

// ---------------------------------------------------------------------------
// Few columns: a stream of the weights through mma.sync (16 rows x 16 values
// times 16 values x 8 columns).
//
// What bounds it is the weights' way from HBM (one int8 token of 129280 x 4096 in
// groups of 128: 52.1 us, 5.2 TB/s), for small matrices the latency of getting
// there (2048 x 2048: 3.8 us), and close behind both the instructions: a chunk of
// 16 rows takes a warp 8 MMAs, 4 reads of activations and 40 instructions for its
// codes (72 for normal numbers), and twice the MMAs and reads for more than eight
// columns (five fp32 tokens, groups of 64 with zero points: 97 us).
// So everything else is done once for a unit of U chunks: a warp keeps a unit's
// codes in registers, requests each chunk of its next one as soon as it has used
// its place, and the wk warps of a row group take every wk-th unit of a row and
// join their sums through shared memory.
// The packed order lets a lane's 16 bytes of a chunk be its operands of eight
// MMAs: of word j the values 32 j + 8 (lane % 4) .. + 7, whose activations are
// 16 bytes too, with every group of 32 values in two MMAs.  The activations stay
// in shared memory for all tiles of the CTA, rows 64 bytes off a multiple of 128
// so that reads meet no conflict; one large CTA to an SM, as each prepares them
// for itself.
constexpr int S_WARPS = 24; // warps of a CTA at most
constexpr int S_COLS = 16;  // columns at most
constexpr int ROWS = 16;
constexpr int PART = 20; // floats between the columns of a warp's sums: no bank is met twice

__device__ __forceinline__ void mma(float (&d)[4], bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if (first)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Masked codes (of a word's four pairs) less their zero point, as normal fp16
// numbers, exact: under the exponent of 1024 a code is 1024 + q, or 1024 + 16 q.
__device__ __forceinline__ void normal(uint32_t (&h)[4], uint32_t zero)
{
    const uint32_t zl = (0x6400u + zero) * 0x10001u, zh = (0xD400u + 16u * zero) * 0x10001u; // 1024 + z, -(64 + z)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(h[i] | 0x64006400u), "r"(zl));
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[i + 1]) : "r"(h[i + 1] | 0x64006400u), "r"(0x2C002C00u), "r"(zh)); // a sixteenth
    }
}

// GPC groups of a row in a chunk: their scales (16 bits each) and zero points
// (8 bits each), those beyond the row's G as zero.
template <int GPC> struct Groups {
    uint32_t s[(GPC + 1) / 2], z;
};
// EVEN: every row's groups are whole chunks, aligned.  (A choice at run time would
// cost a wait for the loads at its end: 129280 x 4096 in groups of 64 75 us.)
template <int GPC, bool ZEROS, bool EVEN>
__device__ __forceinline__ void load_groups(Groups<GPC> &g, const W4Args &a, int64_t at, int g0)
{ // (group g0 of a row, at `at` among all rows' groups)
    const uint16_t *s = reinterpret_cast<const uint16_t *>(a.ws) + at;
    const uint8_t *z = a.zeros + at;
    if constexpr (GPC == 1) {
        g.s[0] = __ldg(s);
        if (ZEROS)
            g.z = __ldg(z);
    } else {
        if constexpr (EVEN) {
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

// Warps of a CTA at most: those whose registers need no spilling.
template <int NT, int GPC, bool ZEROS, int U> constexpr int S_MOST = NT == 1 && (U == 2 || (GPC == 1 && !ZEROS)) ? S_WARPS : 16;

// WHOLE: activations as whole numbers, codes as they are.
template <int NT, int GPC, bool ZEROS, int U, bool WHOLE, bool EVEN>
__global__ void __launch_bounds__(S_MOST<NT, GPC, ZEROS, U> * 32)
    k_linear_w4_stream(const W4Args a, int wk, int groups, int pitch, int steps)
{
    constexpr int COLS = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = groups * wk;
    const int P = a.parts, nt = a.T, cols = nt * P;
    const int chunks = (a.K + CHUNK - 1) / CHUNK, row_bytes = chunks * CHUNK_BYTES;
    const int units = (chunks + U - 1) / U, per = (units + wk - 1) / wk; // of a row; of a warp and tile
    const int group = warp / wk, kw = warp % wk;                         // row group of the CTA, place in it
    const int quad = lane & 3, r8 = lane >> 2;
    const int rows_step = groups * ROWS; // rows of the CTA at a step (warps beyond them prepare activations only)
    // behind the activations: per group and column the factor and the sum of
    // its activations; then the warps' sums, twice
    float2 *info = reinterpret_cast<float2 *>(smem + (size_t)cols * pitch);
    float *part = reinterpret_cast<float *>(info + chunks * GPC * COLS);

    pdl_wait(); // (weights too may be the previous kernel's: luce_quantize_w4 writes them)
    pdl_trigger();

    uint4 w[U][2];
    Groups<GPC> g[U][2];
    // the unit to request next: its step and place among the tile's, and where
    // this lane's codes and groups of it are in two rows (those beyond the last repeat it)
    int ls = warp < warps ? blockIdx.x : steps, lj = 0, lc;
    const uint8_t *lw[2];
    int64_t lg[2];
    auto aim = [&]() {
        lc = ls < steps ? (kw + lj * wk) * U : chunks;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t row = min(ls * rows_step + group * ROWS + r8 + 8 * h, a.N - 1); // (below 2^24 + 2^16)
            lw[h] = a.wq + row * row_bytes + lc * CHUNK_BYTES + 16 * quad;
            lg[h] = row * a.G + lc * GPC;
        }
        if (++lj == per)
            lj = 0, ls += gridDim.x;
    };
    auto request = [&](int u) {
        if (lc + u < chunks)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                w[u][h] = ldg_stream(lw[h] + u * CHUNK_BYTES);
                load_groups<GPC, ZEROS, EVEN>(g[u][h], a, lg[h] + u * GPC, (lc + u) * GPC);
            }
    };
    aim();
#pragma unroll
    for (int u = 0; u < U; u++)
        request(u);

    // activations into shared memory, zero from K to the chunk's end
    const int half = threadIdx.x >> 4, l16 = threadIdx.x & 15;
    for (int i0 = 0; i0 < nt * chunks; i0 += blockDim.x / 16) {
        const int i = i0 + half, t = i / chunks, c = i % chunks, k = c * CHUNK + 8 * l16;
        const bool live = i < nt * chunks && k < a.K;
        uint4 o[2];
        float f[2], sum[2];
        operands<GPC>(a, t, k, live, o, f, sum);
        if (i < nt * chunks) {
#pragma unroll
            for (int p = 0; p < 2; p++)
                if (p < P) {
                    *reinterpret_cast<uint4 *>(smem + (size_t)(t * P + p) * pitch + 2 * k) = o[p];
                    if (l16 % (16 / GPC) == 0)
                        info[(c * GPC + l16 / (16 / GPC)) * COLS + t * P + p] = make_float2(f[p], sum[p]);
                }
        }
    }
    __syncthreads();
    if (warp >= warps)
        return;

    const uint8_t *xcol[NT]; // (columns beyond the last repeat it; their sums are not stored)
#pragma unroll
    for (int n = 0; n < NT; n++)
        xcol[n] = smem + (size_t)min(8 * n + r8, cols - 1) * pitch + 16 * quad;
    const float2 *const my_info = info + 2 * quad;

    float acc[NT][4] = {};
    int buf = 0;
    for (int step = blockIdx.x; step < steps; step += gridDim.x) {
        for (int j = 0; j < per; j++) {
            const int c0 = (kw + j * wk) * U;
            aim();
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (c0 + u < chunks) {
                    constexpr int JG = 4 / GPC; // words of a group
                    float sc[2][GPC];
                    if (a.ws_bf16) {
#pragma unroll
                        for (int i = 0; i < 2 * GPC; i++) {
                            const uint32_t v = g[u][i & 1].s[i >> 2];
                            sc[i & 1][i >> 1] = __uint_as_float(i & 2 ? v & 0xffff0000u : v << 16);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2 * GPC; i++)
                            sc[i & 1][i >> 1] = half_bits_to_float(g[u][i & 1].s[i >> 2] >> (i & 2 ? 16 : 0));
                    }
#pragma unroll
                    for (int gi = 0; gi < GPC; gi++) {
                        float sum[NT][4];
                        const uint32_t zero0 = ZEROS ? (g[u][0].z >> (8 * gi)) & 15u : 8u, zero1 = ZEROS ? (g[u][1].z >> (8 * gi)) & 15u : 8u;
                        // (eight times the activations' sums are known: the zero point counts in eighths)
                        const float z0 = ZEROS ? (float)zero0 * -0.125f : -1.0f, z1 = ZEROS ? (float)zero1 * -0.125f : -1.0f;
#pragma unroll
                        for (int q = gi * JG; q < (gi + 1) * JG; q++) {
                            const uint32_t w0 = q == 0 ? w[u][0].x : q == 1 ? w[u][0].y : q == 2 ? w[u][0].z : w[u][0].w;
                            const uint32_t w1 = q == 0 ? w[u][1].x : q == 1 ? w[u][1].y : q == 2 ? w[u][1].z : w[u][1].w;
                            uint32_t h0[4] = {w0 & LO, w0 & HI, (w0 >> 8) & LO, (w0 >> 8) & HI};
                            uint32_t h1[4] = {w1 & LO, w1 & HI, (w1 >> 8) & LO, (w1 >> 8) & HI};
                            if constexpr (!WHOLE) {
                                normal(h0, zero0);
                                normal(h1, zero1);
                            }
#pragma unroll
                            for (int n = 0; n < NT; n++) {
                                const uint4 b = *reinterpret_cast<const uint4 *>(xcol[n] + c0 * (2 * CHUNK) + u * (2 * CHUNK) + q * 64);
                                mma(sum[n], q == gi * JG, h0[0], h1[0], h0[1], h1[1], b.x, b.y);
                                mma(sum[n], false, h0[2], h1[2], h0[3], h1[3], b.z, b.w);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            const float4 f = *reinterpret_cast<const float4 *>(my_info + ((c0 + u) * GPC + gi) * COLS + 8 * n);
                            if constexpr (WHOLE) {
                                acc[n][0] = fmaf(sc[0][gi], fmaf(sum[n][0], f.x, z0 * f.y), acc[n][0]);
                                acc[n][1] = fmaf(sc[0][gi], fmaf(sum[n][1], f.z, z0 * f.w), acc[n][1]);
                                acc[n][2] = fmaf(sc[1][gi], fmaf(sum[n][2], f.x, z1 * f.y), acc[n][2]);
                                acc[n][3] = fmaf(sc[1][gi], fmaf(sum[n][3], f.z, z1 * f.w), acc[n][3]);
                            } else {
                                // (the factor first: its product with a scale may leave fp32's range, 2^26 times it cannot)
                                acc[n][0] = fmaf(sc[0][gi], sum[n][0] * f.x, acc[n][0]);
                                acc[n][1] = fmaf(sc[0][gi], sum[n][1] * f.z, acc[n][1]);
                                acc[n][2] = fmaf(sc[1][gi], sum[n][2] * f.x, acc[n][2]);
                                acc[n][3] = fmaf(sc[1][gi], sum[n][3] * f.z, acc[n][3]);
                            }
                        }
                    }
                }
                request(u);
            }
        }
        // the warps' sums joined and stored
        float *const mine = part + (buf * warps + warp) * (COLS * PART);
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float *p = mine + (8 * n + 2 * quad) * PART + r8;
            p[0] = acc[n][0], p[PART] = acc[n][1], p[8] = acc[n][2], p[PART + 8] = acc[n][3];
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        }
        if (wk == 1)
            __syncwarp();
        else
            named_barrier(1 + group, wk * 32);
        // (the next step writes the other half of part, and cannot come back to this one before its own barrier)
        for (int i = kw * 32 + lane; i < ROWS * nt; i += wk * 32) {
            const int t = i / ROWS, r = i % ROWS, n = step * rows_step + group * ROWS + r;
            if (n >= a.N)
                continue;
            float v = 0.0f;
            for (int p = P - 1; p >= 0; p--) {
                const float *q = mine - kw * (COLS * PART) + (t * P + p) * PART + r;
                float sum = 0.0f;
                for (int k = 0; k < wk; k++)
                    sum += q[k * (COLS * PART)];
                v += sum;
            }
            v *= UNIT;
            if (a.xs)
                v = __fmul_rn(v, a.xs[t]);
            if (a.bias)
                v = __fadd_rn(v, a.bias[n]);
            store_as(a.out, a.out_dtype, t * a.ldo + n, v);
        }
        buf ^= 1;
    }
}

constexpr size_t S_SMEM = 225 * 1024;

// Shared memory of the stream for a column's activations.
int s_pitch(int K) { return (K + CHUNK - 1) / CHUNK * 2 * CHUNK + 64; }
size_t s_smem(const W4Args &a, int cols, int gpc, int warps)
{
    const size_t chunks = (a.K + CHUNK - 1) / CHUNK, padded = (cols + 7) / 8 * 8;
    return (size_t)cols * s_pitch(a.K) + chunks * gpc * padded * 8 + 2 * warps * padded * PART * 4;
}

template <int NT, int GPC, bool ZEROS, int U, bool WHOLE, bool EVEN> luce_status launch_stream(const W4Args &a, cudaStream_t stream)
{
    static luce_host::SmemLimit limit;
    const auto kern = k_linear_w4_stream<NT, GPC, ZEROS, U, WHOLE, EVEN>;
    const int chunks = (a.K + CHUNK - 1) / CHUNK;
    // wk warps along a row, and as many row groups to a CTA as SMs ask for, within its warps: those
    // with the fewest units one after another; a step's joining counts as a quarter of a unit (of two
    // chunks a half: 129280 x 4096 takes 2.6 us a unit of four and 0.6 us a step)
    const int tiles = (a.N + ROWS - 1) / ROWS, sms = luce_host::sm_count(), units = (chunks + U - 1) / U;
    int wk = 1, groups = 1;
    int64_t best = INT64_MAX;
    for (int w = 1; w <= S_MOST<NT, GPC, ZEROS, U>; w++) {
        const int n = std::min(S_MOST<NT, GPC, ZEROS, U> / w, (tiles + sms - 1) / sms);
        const int64_t turns = ((tiles + n - 1) / n + sms - 1) / sms, cost = turns * (U * ((units + w - 1) / w) + 1);
        if (cost < best)
            best = cost, wk = w, groups = n;
    }
    const int rows = groups * ROWS, steps = (a.N + rows - 1) / rows;
    const size_t smem = s_smem(a, a.T * a.parts, GPC, wk * groups);
    const int warps = std::max(wk * groups, std::min(S_MOST<NT, GPC, ZEROS, U>, (a.T * chunks + 1) / 2)); // two chunks a warp to prepare
    if (smem > 48 * 1024 && limit.raise(kern, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const luce_status st = luce_host::launch(kern, dim3((unsigned)std::min(steps, sms)), dim3(warps * 32), smem, stream, a, wk, groups,
                                             s_pitch(a.K), steps);
    if (st != LUCE_OK)
        limit.forget();
    return st;
}

// Whether the stream serves a call.  Each of its CTAs prepares the activations
// for itself, 0.02 us a token and chunk (int8 half of that); the tensor cores
// are later to start, and read the codes of large matrices more slowly, most of
// all where they have activations to convert.  In tokens times chunks, with the
// stages of codes that an SM takes:
//   fp32      170 + 9 stages   (8192 x 8192, 5 tokens 23.4 us, tensor cores 25.0; 4096 x 4096, 8 tokens 12.2 and 10.7)
//   int8      290 + 12 stages  (8192 x 8192, 8 tokens 19.4 us and 21.6; 4096 x 4096, 12 tokens 11.2 and 10.5)
//   16 bits   140 + 4 stages   (4096 x 4096, 4 tokens 8.4 us and 9.4; 8192 x 8192, 4 tokens 17.5 and 16.4)
// and for more than four tokens of 16 bits, whose codes take the stream twice the
// instructions, 166 + 2 stages, but 260 at most (4096 x 4096, 5 tokens 9.0 us and
// 9.5, 8 tokens 10.8 and 9.6; 129280 x 4096, 8 tokens 67.4 and 68.2, 12 tokens
// 82.3 and 69.5).
bool stream_serves(const W4Args &a, int gpc)
{
    const int64_t chunks = (a.K + CHUNK - 1) / CHUNK, cols = (int64_t)a.T * a.parts;
    if (cols > S_COLS || s_smem(a, (int)cols, gpc, cols > 8 ? 16 : S_WARPS) > S_SMEM)
        return false;
    const int64_t stages = (int64_t)a.N * chunks / (128 * luce_host::sm_count()), work = a.T * chunks;
    return work <= (a.x_dtype == LUCE_F32 ? 170 + 9 * stages : a.x_dtype == LUCE_I8 ? 290 + 12 * stages : a.whole ? 140 + 4 * stages : std::min<int64_t>(166 + 2 * stages, 260));
}

template <int GPC, bool ZEROS> luce_status run_stream(const W4Args &a, cudaStream_t stream)
{
    // units of two chunks where there are not enough of four for all SMs
    const bool few = (int64_t)a.N * ((a.K + CHUNK - 1) / CHUNK) < (int64_t)1 << 19;
    auto run = [&](auto nt, auto whole) {
        constexpr int NT = decltype(nt)::value;
        constexpr bool WHOLE = decltype(whole)::value;
        const bool even = a.G % GPC == 0 && luce_host::aligned(a.ws, 2 * GPC) && (!ZEROS || luce_host::aligned(a.zeros, GPC));
        if (GPC > 1 && !even)
            return launch_stream<NT, GPC, ZEROS, 2, WHOLE, GPC == 1>(a, stream);
        return few ? launch_stream<NT, GPC, ZEROS, 2, WHOLE, true>(a, stream) : launch_stream<NT, GPC, ZEROS, 4, WHOLE, true>(a, stream);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (a.T * a.parts <= 8)
        return a.whole ? run(One(), std::true_type()) : run(One(), std::false_type());
    return a.whole ? run(Two(), std::true_type()) : run(Two(), std::false_type());
}

luce_status run_groups(const W4Args &a, int group, cudaStream_t stream)
{
    if (a.zeros)
        return group == 32 ? run_stream<4, true>(a, stream) : group == 64 ? run_stream<2, true>(a, stream) : run_stream<1, true>(a, stream);
    return group == 32 ? run_stream<4, false>(a, stream) : group == 64 ? run_stream<2, false>(a, stream) : run_stream<1, false>(a, stream);
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
    const bool whole = x_dtype == LUCE_I8 || x_dtype == LUCE_F32 || out_dtype == LUCE_F32 || 2 * T <= 8;
    const W4Args a{x, x_dtype, whole, whole && x_dtype != LUCE_I8 ? 2 : 1, ld_x, x_scale, wq, w_scale, scale_dtype == LUCE_BF16, zeros, bias, T, N, K, G, out, out_dtype, ld_out};
    cudaStream_t st = luce_host::as_stream(stream);
    return stream_serves(a, CHUNK / group) ? run_groups(a, group, st) : tc_product(a, group, st);
}
