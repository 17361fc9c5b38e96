// rows_w4.cu -- matrices to 4-bit codes in the order of luce_linear_w4
// (luce_quantize_w4, luce_pack_w4), with their C-ABI entry points.
//
// A half-warp takes a chunk of 128 values of a row, a thread eight of them:
// thread 4 j + t the values 32 j + 8 t .. + 7, which are word 4 t + j of the
// chunk.  A group of 32, 64 or 128 values is 4, 8 or 16 threads, which join
// their extremes by shuffles.  Made once for a matrix; bound by instructions, a
// group's extremes and divisions for eight values a thread (4096 x 4096 bf16
// 29.8 us, floor 6.2; packing 9.8, floor 3.7).  Four chunks to a thread at once,
// whose waits overlap but which need 125 registers, took 51.8.
#include <climits>

#include <cuda_bf16.h>

#include "common.cuh"

namespace {

using namespace luce;

constexpr int CHUNK = 128, CHUNK_BYTES = 64, K_MAX = 65536;
constexpr int THREADS = 256;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// A scale in its stored type, kept finite (a group's largest value may need more than fp16 holds).
__device__ __forceinline__ uint16_t scale_bits(float d, bool bf)
{
    if (bf) {
        const uint16_t b = __bfloat16_as_ushort(__float2bfloat16_rn(d));
        return b == 0x7f80u ? 0x7f7fu : b;
    }
    const uint16_t b = __half_as_ushort(__float2half_rn(d));
    return b == 0x7c00u ? 0x7bffu : b;
}
__device__ __forceinline__ float scale_value(uint16_t b, bool bf)
{
    return bf ? __uint_as_float((uint32_t)b << 16) : half_bits_to_float(b);
}

// Value i of a word has its bits 4 (i / 2) + 16 (i % 2) .. + 3.
__device__ __forceinline__ uint32_t place(uint32_t code, int i) { return code << (4 * (i >> 1) + 16 * (i & 1)); }

// A chunk's row and place in it (64-bit division only for matrices that need it).
__device__ __forceinline__ int row_of(int64_t c, int chunks, int &at)
{
    const int64_t row = c >> 32 ? c / chunks : (uint32_t)c / (uint32_t)chunks;
    at = (int)(c - row * chunks);
    return (int)row;
}

// WIDE: eight values of a row in one or two loads (w 16-byte aligned).
template <typename TW, bool WIDE>
__global__ void __launch_bounds__(THREADS)
    k_quantize_w4(const TW *w, int N, int K, int chunks, int group, uint32_t *wq, uint16_t *scale, bool bf, uint8_t *zeros)
{
    pdl_wait();
    pdl_trigger();
    const int64_t c = ((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 4; // chunk of the matrix
    const bool live = c < (int64_t)N * chunks;
    int at = 0;
    const int row = live ? row_of(c, chunks, at) : 0, i0 = threadIdx.x & 15;
    const int k = live ? at * CHUNK + 8 * i0 : K; // first value of this thread (K is a multiple of 16)
    struct __align__(16) Eight { TW v[8]; };
    Eight x = {};
    if (k < K) {
        const TW *p = w + (int64_t)row * K + k;
        if constexpr (WIDE) {
            x = *reinterpret_cast<const Eight *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                x.v[i] = p[i];
        }
    }
    float v[8], lo = 0.0f, hi = 0.0f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        v[i] = to_float(x.v[i]);
        odd |= !isfinite(v[i]);
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
    for (int o = 1; o < group / 8; o *= 2) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        odd |= __shfl_xor_sync(0xffffffffu, (int)odd, o) != 0;
    }
    uint16_t s = scale_bits(zeros ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f), bf);
    const float d = scale_value(s, bf);
    const bool flat = odd || d == 0.0f;
    if (odd)
        s = 0x7fffu; // NaN in either type
    const float z = !zeros ? 8.0f : flat ? 0.0f : fminf(roundf(__fdiv_rn(-lo, d)), 15.0f);
    // round(fl(v / d)) is the whole number nearest v rinv wherever that is not within 1e-4 of half way between
    // two (up to 64 rinv = fl(1 / d) moves it by less than 2e-5): the sum with
    // 1.5 2^23 leaves it in the low bits.  Threads with a value near half way, or a larger one (of a d that its type
    // keeps from being what it should, or whose reciprocal overflows), divide.
    // (8192 x 4144 fp16 in groups of 32: 57 us, with divisions and narrow loads 68.)
    const float rinv = __frcp_rn(d);
    constexpr float MAGIC = 12582912.0f;
    int n[8];
    bool near_half = false;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float r = fmaf(v[i], rinv, MAGIC), whole = __fsub_rn(r, MAGIC);
        n[i] = __float_as_int(r) - 0x4B400000;
        near_half |= !(fabsf(fmaf(v[i], rinv, -whole)) <= 0.4999f && fabsf(whole) <= 64.0f);
    }
    if (flat) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            n[i] = 0;
    } else if (near_half) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            n[i] = (int)fminf(fmaxf(roundf(__fdiv_rn(v[i], d)), -64.0f), 64.0f);
    }
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
        word |= place((uint32_t)min(max(n[i] + (int)z, zeros ? 0 : 1), 15), i);
    if (!live)
        return;
    wq[c * (CHUNK / 8) + 4 * (i0 & 3) + (i0 >> 2)] = word;
    if (k < K && k % group == 0) {
        const int64_t g = (int64_t)row * ((K + group - 1) / group) + k / group;
        scale[g] = s;
        if (zeros)
            zeros[g] = (uint8_t)z;
    }
}

template <bool WIDE> // (codes 8-byte aligned)
__global__ void __launch_bounds__(THREADS) k_pack_w4(const uint8_t *codes, int N, int K, int chunks, uint32_t *wq)
{
    pdl_wait();
    pdl_trigger();
    const int64_t c = ((int64_t)blockIdx.x * THREADS + threadIdx.x) >> 4;
    if (c >= (int64_t)N * chunks)
        return;
    int at;
    const int row = row_of(c, chunks, at), i0 = threadIdx.x & 15, k = at * CHUNK + 8 * i0;
    struct __align__(8) Eight { uint8_t v[8]; };
    Eight x = {};
    if (k < K) {
        const uint8_t *p = codes + (int64_t)row * K + k;
        if constexpr (WIDE) {
            x = *reinterpret_cast<const Eight *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                x.v[i] = p[i];
        }
    }
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
        word |= place(x.v[i] & 15u, i);
    wq[c * (CHUNK / 8) + 4 * (i0 & 3) + (i0 >> 2)] = word;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

// (N and K within luce_linear_w4's limits: at most 2^24 * 2^9 chunks, 2^29 blocks)
unsigned blocks_of(int N, int chunks) { return (unsigned)(((int64_t)N * chunks * 16 + THREADS - 1) / THREADS); }

} // namespace

extern "C" luce_status luce_quantize_w4(const void *w, luce_dtype dtype, int N, int K, int group, uint8_t *wq, void *w_scale,
                                        luce_dtype scale_dtype, uint8_t *zeros, void *stream)
{
    using luce_host::aligned;
    if (N < 0 || N >= (1 << 24) || K < 16 || K > K_MAX || K % 16 != 0 || (group != 32 && group != 64 && group != 128) ||
        (dtype != LUCE_F32 && dtype != LUCE_BF16 && dtype != LUCE_F16) ||
        (scale_dtype != LUCE_F16 && scale_dtype != LUCE_BF16))
        return LUCE_ERR_INVALID_ARG;
    if (N == 0)
        return LUCE_OK;
    const size_t es = dtype == LUCE_F32 ? 4 : 2;
    if (!w || !wq || !w_scale || !aligned(w, es) || !aligned(wq, 16) || !aligned(w_scale, 2))
        return LUCE_ERR_INVALID_ARG;
    const int chunks = (K + CHUNK - 1) / CHUNK, G = (K + group - 1) / group;
    const size_t nw = (size_t)N * K * es, nq = (size_t)N * chunks * CHUNK_BYTES, ns = (size_t)N * G * 2, nz = (size_t)N * G;
    if (overlap(w, nw, wq, nq) || overlap(w, nw, w_scale, ns) || overlap(wq, nq, w_scale, ns) ||
        (zeros && (overlap(zeros, nz, w, nw) || overlap(zeros, nz, wq, nq) || overlap(zeros, nz, w_scale, ns))))
        return LUCE_ERR_INVALID_ARG;
    auto run = [&](auto element) {
        using TW = decltype(element);
        return luce_host::launch(aligned(w, 16) ? k_quantize_w4<TW, true> : k_quantize_w4<TW, false>, dim3(blocks_of(N, chunks)), dim3(THREADS), 0, luce_host::as_stream(stream),
                                 (const TW *)w, N, K, chunks, group, (uint32_t *)wq, (uint16_t *)w_scale,
                                 scale_dtype == LUCE_BF16, zeros);
    };
    return dtype == LUCE_F32 ? run(float()) : dtype == LUCE_BF16 ? run(__nv_bfloat16()) : run(__half());
}

extern "C" luce_status luce_pack_w4(const uint8_t *codes, int N, int K, uint8_t *wq, void *stream)
{
    if (N < 0 || N >= (1 << 24) || K < 16 || K > K_MAX || K % 16 != 0)
        return LUCE_ERR_INVALID_ARG;
    if (N == 0)
        return LUCE_OK;
    const int chunks = (K + CHUNK - 1) / CHUNK;
    if (!codes || !wq || !luce_host::aligned(wq, 16) ||
        overlap(codes, (size_t)N * K, wq, (size_t)N * chunks * CHUNK_BYTES))
        return LUCE_ERR_INVALID_ARG;
    return luce_host::launch(luce_host::aligned(codes, 8) ? k_pack_w4<true> : k_pack_w4<false>, dim3(blocks_of(N, chunks)), dim3(THREADS), 0, luce_host::as_stream(stream), codes, N,
                             K, chunks, (uint32_t *)wq);
}
