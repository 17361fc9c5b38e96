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

constexpr int THREADS = 256;

// One CTA per row, two passes over it: the row's sum of squares and its
// largest |p|, then the codes.
template <typename TX>
__global__ void __launch_bounds__(THREADS)
    k_rows_i8(const TX *x, const TX *res, TX *xsum, const float *gamma, float eps, int T, int H, int8_t *q,
              float *scale)
{
    __shared__ float s_ss[THREADS / 32];
    __shared__ uint32_t s_m[THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        const size_t row = (size_t)t * H;
        float ss = 0.0f;
        uint32_t m = 0;
        for (int i = threadIdx.x; i < H; i += THREADS) {
            float v = to_f32(x[row + i]);
            if (res)
                v = to_f32(from_f32<TX>(__fadd_rn(v, to_f32(res[row + i]))));
            const float p = gamma ? __fmul_rn(v, gamma[i]) : v;
            ss = fmaf(v, v, ss);
            m = max(m, __float_as_uint(p) & 0x7fffffffu); // |p| as ordered bits: a NaN lies above infinity
        }
        ss = warp_sum(ss);
        m = __reduce_max_sync(0xffffffffu, m);
        __syncthreads(); // (the previous row's totals have been read)
        if (lane == 0) {
            s_ss[warp] = ss;
            s_m[warp] = m;
        }
        __syncthreads();
        ss = 0.0f;
        m = 0;
        for (int w = 0; w < THREADS / 32; w++) {
            ss += s_ss[w];
            m = max(m, s_m[w]);
        }
        const bool finite = m < 0x7f800000u;
        const float d = __fdiv_rn(__uint_as_float(m), 127.0f);
        for (int i = threadIdx.x; i < H; i += THREADS) {
            float v = to_f32(x[row + i]);
            if (res) {
                const TX s = from_f32<TX>(__fadd_rn(v, to_f32(res[row + i])));
                v = to_f32(s);
                if (xsum)
                    xsum[row + i] = s;
            }
            const float p = gamma ? __fmul_rn(v, gamma[i]) : v;
            const float c = fminf(fmaxf(roundf(__fdiv_rn(p, d)), -127.0f), 127.0f);
            q[row + i] = finite && d > 0.0f ? (int8_t)c : (int8_t)0;
        }
        if (threadIdx.x == 0) {
            float sc = d;
            if (gamma)
                sc = __fmul_rn(d, __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)H), eps))));
            scale[t] = finite ? sc : NAN;
        }
    }
}

constexpr int H_MAX = 65536;

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

template <typename TX>
luce_status run_rows(const void *x, const void *res, void *xsum, const float *gamma, float eps, int T, int H,
                     int8_t *q, float *scale, void *stream)
{
    const unsigned grid = (unsigned)T;
    return luce_host::launch(k_rows_i8<TX>, dim3(grid), dim3(THREADS), 0, luce_host::as_stream(stream),
                             (const TX *)x, (const TX *)res, (TX *)xsum, gamma, eps, T, H, q, scale);
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
    switch (dtype) {
    case LUCE_F32:
        return run_rows<float>(x, res, xsum, gamma, eps, T, H, q, scale, stream);
    case LUCE_BF16:
        return run_rows<__nv_bfloat16>(x, res, xsum, gamma, eps, T, H, q, scale, stream);
    case LUCE_F16:
        return run_rows<__half>(x, res, xsum, gamma, eps, T, H, q, scale, stream);
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
