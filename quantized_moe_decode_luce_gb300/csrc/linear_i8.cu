// linear_i8.cu -- the dense int8 product with scales per token and per output
// channel (luce_linear_i8), with its C-ABI entry point.
//
//   out[t][n] = isum[t][n] * (x_scale[t] * w_scale[n]) (+ bias[n]),
//   isum[t][n] = sum_k xq[t][k] wq[n][k], an exact int32 sum
//   (K <= 65,536: |isum| <= 2^16 2^14 = 2^30).
#include <climits>
#include <cmath>

#include <cuda_bf16.h>

#include "common.cuh"

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

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

template <typename TO>
luce_status run_linear(const int8_t *xq, const float *xs, const int8_t *wq, const float *ws, const float *bias, int T,
                       int N, int K, TO *out, int64_t ldo, cudaStream_t stream)
{
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
