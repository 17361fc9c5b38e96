// logits_process.cu -- penalties for repeated tokens, biases and grammar masks
// on a batch of logits (luce_logits_process), with its C-ABI entry point.
//
// One CTA per stretch of a row's vocabulary.  It counts the row's history
// tokens that fall in its stretch in shared memory (whole numbers, so the
// order of the atomics does not show), and applies everything to the logits
// of the stretch in one pass.
#include <algorithm>
#include <climits>
#include <cmath>

#include <cuda_bf16.h>

#include "common.cuh"

LUCE_DEFINE_FAULT_WORD(luce_internal_fault_logits)

namespace {

using namespace luce;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

struct LogitsArgs {
    const void *logits;
    int64_t V, ldl;
    const int32_t *hist;
    int64_t ldh;
    const int32_t *hist_len, *prompt_len;
    const float *rep, *freq, *pres;
    const int32_t *bias_ids;
    const float *bias_vals;
    int nbias;
    const uint32_t *mask;
    int nmasks;
    int64_t ldm;
    const int32_t *mask_rows;
    float *out;
    int64_t ldo;
};

constexpr int THREADS = 256;
constexpr int PER = 16;              // logits per thread
constexpr int CHUNK = THREADS * PER; // logits of one CTA

template <typename TL> __global__ void __launch_bounds__(THREADS) k_logits_process(const LogitsArgs a)
{
    __shared__ uint32_t cnt[CHUNK];
    pdl_wait();
    pdl_trigger();
    const int r = blockIdx.y;
    const int64_t c0 = (int64_t)blockIdx.x * CHUNK;
    const int nc = (int)min((int64_t)CHUNK, a.V - c0);
    const TL *lr = static_cast<const TL *>(a.logits) + (size_t)r * a.ldl + c0;
    float l[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int v = threadIdx.x + i * THREADS;
        l[i] = v < nc ? to_f32(lr[v]) : 0.0f;
    }
    bool bad = false;
    if (a.hist) {
        for (int i = threadIdx.x; i < CHUNK; i += THREADS)
            cnt[i] = 0;
        __syncthreads();
        // a word holds twice the count of generated tokens, its low bit the prompt's
        const int64_t len = min((int64_t)max(a.hist_len[r], 0), a.ldh);
        const int64_t plen = a.prompt_len ? a.prompt_len[r] : 0;
        const int32_t *h = a.hist + (size_t)r * a.ldh;
        for (int64_t i = threadIdx.x; i < len; i += THREADS) {
            const int32_t id = h[i];
            bad |= id >= a.V;
            const int64_t at = id - c0;
            if (id >= 0 && at >= 0 && at < nc) {
                if (i < plen)
                    atomicOr(&cnt[at], 1u);
                else
                    atomicAdd(&cnt[at], 2u);
            }
        }
        __syncthreads();
        const float rep = a.rep ? a.rep[r] : 1.0f, freq = a.freq ? a.freq[r] : 0.0f, pres = a.pres ? a.pres[r] : 0.0f;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const uint32_t c = cnt[threadIdx.x + i * THREADS];
            if (c) {
                l[i] = l[i] > 0.0f ? __fdiv_rn(l[i], rep) : __fmul_rn(l[i], rep);
                if (c >> 1)
                    l[i] = __fsub_rn(l[i], __fadd_rn(__fmul_rn((float)(c >> 1), freq), pres));
            }
        }
    }
    if (a.nbias) {
        __syncthreads();
        for (int i = threadIdx.x; i < CHUNK; i += THREADS)
            cnt[i] = 0;
        __syncthreads();
        const int32_t *ids = a.bias_ids + (size_t)r * a.nbias;
        for (int j = threadIdx.x; j < a.nbias; j += THREADS) {
            const int32_t id = ids[j];
            bad |= id >= a.V;
            const int64_t at = id - c0;
            if (id >= 0 && at >= 0 && at < nc)
                atomicMax(&cnt[at], (uint32_t)j + 1u); // the last entry of an id
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const uint32_t j = cnt[threadIdx.x + i * THREADS];
            if (j)
                l[i] = __fadd_rn(l[i], a.bias_vals[(size_t)r * a.nbias + j - 1]);
        }
    }
    const uint32_t *mr = nullptr;
    if (a.mask) {
        const int m = a.mask_rows ? a.mask_rows[r] : r;
        if (m >= a.nmasks)
            bad = true;
        else if (m >= 0)
            mr = a.mask + (size_t)m * a.ldm;
    }
    float *o = a.out + (size_t)r * a.ldo + c0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int v = threadIdx.x + i * THREADS;
        if (v < nc) {
            const int64_t g = c0 + v;
            o[v] = mr && !((mr[g >> 5] >> (g & 31)) & 1u) ? -INFINITY : l[i];
        }
    }
    if (bad && blockIdx.x == 0)
        atomicOr(&g_fault_word, LUCE_FAULT_BAD_ID);
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p < q + nb && q < p + na;
}

} // namespace

extern "C" luce_status luce_logits_process(const void *logits, luce_dtype dtype, int R, int64_t V, int64_t ld_logits,
                                           const int32_t *hist, int64_t ld_hist, const int32_t *hist_len,
                                           const int32_t *prompt_len, const float *repetition, const float *frequency,
                                           const float *presence, const int32_t *bias_ids, const float *bias_vals,
                                           int n_bias, const uint32_t *mask, int n_masks, int64_t ld_mask,
                                           const int32_t *mask_rows, float *out, int64_t ld_out, void *stream)
{
    using luce_host::aligned;
    constexpr int64_t LIM = (int64_t)1 << 30;
    if (R < 0 || R > 65535 || V < 1 || V >= ((int64_t)1 << 31) || ld_logits < V || ld_out < V ||
        ld_logits > 8 * LIM || ld_out > 8 * LIM || (dtype != LUCE_F32 && dtype != LUCE_BF16 && dtype != LUCE_F16))
        return LUCE_ERR_INVALID_ARG;
    if (n_bias < 0 || n_bias >= LIM || (hist && (ld_hist < 0 || ld_hist >= LIM)) || (mask && ld_mask < (V + 31) / 32) ||
        (mask && (n_masks < 1 || ld_mask > 8 * LIM || (!mask_rows && n_masks < R))))
        return LUCE_ERR_INVALID_ARG;
    if ((hist == nullptr) != (hist_len == nullptr) || (!hist && prompt_len) || (!mask && mask_rows))
        return LUCE_ERR_INVALID_ARG;
    if (R == 0)
        return LUCE_OK;
    const size_t es = dtype == LUCE_F32 ? 4 : 2;
    if (!logits || !out || !aligned(logits, es) || !aligned(out, 4) || (n_bias && (!bias_ids || !bias_vals)))
        return LUCE_ERR_INVALID_ARG;
    const size_t no = ((size_t)(R - 1) * ld_out + V) * 4, nl = ((size_t)(R - 1) * ld_logits + V) * es;
    const bool in_place = out == logits && dtype == LUCE_F32 && ld_out == ld_logits;
    const struct {
        const void *p;
        size_t n;
    } in[] = {{hist, hist ? (size_t)R * ld_hist * 4 : 0}, {hist_len, (size_t)R * 4}, {prompt_len, (size_t)R * 4},
              {repetition, (size_t)R * 4}, {frequency, (size_t)R * 4}, {presence, (size_t)R * 4},
              {n_bias ? bias_ids : nullptr, (size_t)R * n_bias * 4}, {n_bias ? bias_vals : nullptr, (size_t)R * n_bias * 4},
              {mask, mask ? (size_t)n_masks * ld_mask * 4 : 0}, {mask_rows, (size_t)R * 4}};
    for (const auto &i : in)
        if (i.p && (!aligned(i.p, 4) || overlap(out, no, i.p, i.n)))
            return LUCE_ERR_INVALID_ARG;
    if (!in_place && overlap(out, no, logits, nl))
        return LUCE_ERR_INVALID_ARG;
    const LogitsArgs a{logits, V, ld_logits, hist, ld_hist, hist_len, prompt_len, repetition, frequency, presence,
                       bias_ids, bias_vals, n_bias, mask, n_masks, ld_mask, mask_rows, out, ld_out};
    const dim3 grid((unsigned)((V + CHUNK - 1) / CHUNK), (unsigned)R);
    cudaStream_t st = luce_host::as_stream(stream);
    switch (dtype) {
    case LUCE_F32:
        return luce_host::launch(k_logits_process<float>, grid, dim3(THREADS), 0, st, a);
    case LUCE_BF16:
        return luce_host::launch(k_logits_process<__nv_bfloat16>, grid, dim3(THREADS), 0, st, a);
    case LUCE_F16:
        return luce_host::launch(k_logits_process<__half>, grid, dim3(THREADS), 0, st, a);
    }
    return LUCE_ERR_INVALID_ARG;
}
