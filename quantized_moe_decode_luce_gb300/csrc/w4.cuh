// w4.cuh -- what the kernels of luce_linear_w4 share: its arguments, the order
// of packed codes, and the loads of activations, scales and zero points.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace w4 {

using namespace luce;

constexpr int CHUNK = 128;             // values of a row that its packed codes keep together
constexpr int CHUNK_BYTES = CHUNK / 2;
constexpr int K_MAX = 65536;
constexpr float UNIT = 16384.0f; // sums are kept 2^-14 of their size, so that no chunk's factor leaves fp32's range
constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u; // the codes of a word: two as they are, two sixteenfold

struct W4Args {
    const void *x;
    luce_dtype x_dtype;
    bool whole;  // activations as whole numbers
    int parts;   // columns of a token
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

__device__ __forceinline__ void store_as(void *out, luce_dtype t, int64_t i, float v)
{
    if (t == LUCE_F32)
        reinterpret_cast<float *>(out)[i] = v;
    else if (t == LUCE_BF16)
        reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
    else
        reinterpret_cast<__half *>(out)[i] = __float2half_rn(v);
}

// The product on the tensor cores (linear_w4_tc.cu).
luce_status tc_product(const W4Args &a, int group, cudaStream_t stream);

} // namespace w4
