// logits_process.cu -- penalties for repeated tokens, biases and grammar masks
// on a batch of logits (luce_logits_process), with its C-ABI entry point.
//
// One CTA per stretch of a row's vocabulary.  It counts the row's history
// tokens that fall in its stretch in shared memory (whole numbers, so the
// order of the atomics does not show), then applies everything to the logits
// of the stretch in one pass, the biases behind it.
//
// What bounds it: the logits' way in and out of HBM for large batches; for a
// few rows the latency of launch, history and logits one behind the other.
// Every CTA of a row reads the whole history (from L2), so stretches are as
// long as shared memory allows with two CTAs to an SM, whose phases overlap;
// and short where rows are few, to have all SMs at work.
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

constexpr int THREADS = 512;
constexpr int NB = 4; // vectors of logits of a thread in flight

// What a slot of shared memory holds for its token: twice the number of
// generated occurrences, the low bit set if the token is among the prompt's.
// Sixteen bits are enough while a row has at most 32,767 tokens.
template <bool S16> struct Slots {
    uint32_t *w;
    __device__ __forceinline__ uint32_t get(int at) const
    {
        return S16 ? reinterpret_cast<const uint16_t *>(w)[at] : w[at];
    }
    __device__ __forceinline__ void put(int at, uint32_t v) const
    {
        if (S16)
            reinterpret_cast<uint16_t *>(w)[at] = (uint16_t)v;
        else
            w[at] = v;
    }
    __device__ __forceinline__ void add(int at, uint32_t v) const
    {
        if (S16)
            atomicAdd(w + (at >> 1), v << (16 * (at & 1))); // (no carry: at most 65,535)
        else
            atomicAdd(w + at, v);
    }
    __device__ __forceinline__ void set_low(int at) const
    {
        if (S16)
            atomicOr(w + (at >> 1), 1u << (16 * (at & 1)));
        else
            atomicOr(w + at, 1u);
    }
    __device__ __forceinline__ void raise(int at, uint32_t v) const // the larger of the slot and v
    {
        if (!S16) {
            atomicMax(w + at, v);
            return;
        }
        uint32_t *p = w + (at >> 1), old = *p;
        const int sh = 16 * (at & 1);
        while (((old >> sh) & 0xffffu) < v) {
            const uint32_t seen = atomicCAS(p, old, (old & ~(0xffffu << sh)) | v << sh);
            if (seen == old)
                break;
            old = seen;
        }
    }
    // four slots from `at` (a multiple of four)
    __device__ __forceinline__ uint4 get4(int at) const
    {
        if (!S16)
            return *reinterpret_cast<const uint4 *>(w + at);
        const uint2 v = *reinterpret_cast<const uint2 *>(w + (at >> 1));
        return make_uint4(v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16);
    }
};

__device__ __forceinline__ float penalized(float l, uint32_t c, float rep, float freq, float pres)
{
    l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
    if (c >> 1)
        l = __fsub_rn(l, __fadd_rn(__fmul_rn((float)(c >> 1), freq), pres));
    return l;
}

// VEC logits a step and thread: 4 where every row starts aligned, else 1.
template <typename TL, int VEC, bool S16>
__global__ void __launch_bounds__(THREADS) k_logits_process(const LogitsArgs a, int stretch)
{
    extern __shared__ __align__(16) uint32_t slot_words[];
    const Slots<S16> slots{slot_words};
    const int r = blockIdx.y, tid = threadIdx.x;
    const int64_t c0 = (int64_t)blockIdx.x * stretch;
    const int nc = (int)min((int64_t)stretch, a.V - c0);
    struct alignas(VEC * sizeof(TL)) In {
        TL e[VEC];
    };
    struct alignas(VEC * 4) Out {
        float e[VEC];
    };
    // slots to zero (they do not depend on the previous kernel)
    if (a.hist) {
        const int words = S16 ? (nc + 1) / 2 : nc;
        for (int i = tid; 4 * i < words; i += THREADS)
            reinterpret_cast<uint4 *>(slot_words)[i] = make_uint4(0, 0, 0, 0);
    }
    pdl_wait();
    pdl_trigger();
    const TL *lr = static_cast<const TL *>(a.logits) + (size_t)r * a.ldl + c0;
    float *o = a.out + (size_t)r * a.ldo + c0;
    In in[NB];
    auto load = [&](int v0) {
#pragma unroll
        for (int i = 0; i < NB; i++) {
            const int v = v0 + (tid + i * THREADS) * VEC;
            if (v + VEC <= nc) {
                in[i] = *reinterpret_cast<const In *>(lr + v);
            } else if (VEC > 1) {
#pragma unroll
                for (int e = 0; e < VEC; e++)
                    if (v + e < nc)
                        in[i].e[e] = lr[v + e];
            }
        }
    };
    load(0);
    const uint32_t *mr = nullptr;
    bool bad = false;
    if (a.mask) {
        const int m = a.mask_rows ? a.mask_rows[r] : r;
        if (m >= a.nmasks)
            bad = true;
        else if (m >= 0)
            mr = a.mask + (size_t)m * a.ldm + (c0 >> 5); // (c0 is a multiple of 32)
    }
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    if (a.hist) {
        __syncthreads();
        const int len = (int)min((int64_t)max(a.hist_len[r], 0), a.ldh);
        const int plen = a.prompt_len ? a.prompt_len[r] : 0;
        rep = a.rep ? a.rep[r] : 1.0f;
        freq = a.freq ? a.freq[r] : 0.0f;
        pres = a.pres ? a.pres[r] : 0.0f;
        const int32_t *h = a.hist + (size_t)r * a.ldh;
        const bool first = blockIdx.x == 0;
        auto count = [&](int32_t id, int i) {
            const uint32_t at = (uint32_t)(id - (int32_t)c0);
            if (id >= 0 && at < (uint32_t)nc) {
                if (i < plen)
                    slots.set_low((int)at);
                else
                    slots.add((int)at, 2u);
            }
            if (first)
                bad |= id >= a.V;
        };
        const int head = (int)(((16 - (reinterpret_cast<uintptr_t>(h) & 15)) & 15) / 4); // tokens before a 16-byte boundary
        if (tid < min(head, len))
            count(h[tid], tid);
        const int quads = len > head ? (len - head) >> 2 : 0;
        const int4 *h4 = reinterpret_cast<const int4 *>(h + head);
        constexpr int HB = 4; // loads in flight
        for (int q0 = 0; q0 < quads; q0 += HB * THREADS) {
            int4 t[HB];
#pragma unroll
            for (int i = 0; i < HB; i++) {
                const int q = q0 + i * THREADS + tid;
                t[i] = q < quads ? h4[q] : make_int4(-1, -1, -1, -1);
            }
#pragma unroll
            for (int i = 0; i < HB; i++) {
                const int at = head + 4 * (q0 + i * THREADS + tid);
                count(t[i].x, at);
                count(t[i].y, at + 1);
                count(t[i].z, at + 2);
                count(t[i].w, at + 3);
            }
        }
        const int tail = head + 4 * quads + tid;
        if (tail < len && tid < 4)
            count(h[tail], tail);
        __syncthreads();
    }
    for (int v0 = 0; v0 < nc; v0 += NB * THREADS * VEC) {
        if (v0 > 0)
            load(v0);
#pragma unroll
        for (int i = 0; i < NB; i++) {
            const int v = v0 + (tid + i * THREADS) * VEC;
            if (v >= nc)
                break;
            Out w;
#pragma unroll
            for (int e = 0; e < VEC; e++)
                w.e[e] = to_f32(in[i].e[e]);
            if (a.hist) {
                if constexpr (VEC == 4) {
                    const uint4 c = slots.get4(v);
                    if (c.x | c.y | c.z | c.w) {
                        const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int e = 0; e < VEC; e++)
                            if (cs[e])
                                w.e[e] = penalized(w.e[e], cs[e], rep, freq, pres);
                    }
                } else {
                    const uint32_t c = slots.get(v);
                    if (c)
                        w.e[0] = penalized(w.e[0], c, rep, freq, pres);
                }
            }
            if (mr) {
                const uint32_t bits = mr[v >> 5] >> (v & 31);
#pragma unroll
                for (int e = 0; e < VEC; e++)
                    if (!((bits >> e) & 1u))
                        w.e[e] = -INFINITY;
            }
            if (v + VEC <= nc) {
                *reinterpret_cast<Out *>(o + v) = w;
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e++)
                    if (v + e < nc)
                        o[v + e] = w.e[e];
            }
        }
    }
    if (a.nbias) {
        // the slots now find each id's last entry, which adds its bias to the
        // value stored above unless the token is masked
        const int32_t *ids = a.bias_ids + (size_t)r * a.nbias;
        const float *vals = a.bias_vals + (size_t)r * a.nbias;
        auto each = [&](auto &&f) {
            for (int j = tid; j < a.nbias; j += THREADS) {
                const int32_t id = ids[j];
                const uint32_t at = (uint32_t)(id - (int32_t)c0);
                if (id >= 0 && at < (uint32_t)nc)
                    f((int)at, j);
                bad |= id >= a.V;
            }
            __syncthreads();
        };
        __syncthreads();
        each([&](int at, int) { slots.put(at, 0); });
        each([&](int at, int j) { slots.raise(at, (uint32_t)j + 1u); });
        each([&](int at, int j) {
            if (slots.get(at) == (uint32_t)j + 1u && !(mr && !((mr[at >> 5] >> (at & 31)) & 1u)))
                o[at] = __fadd_rn(o[at], vals[j]);
        });
    }
    if (bad && blockIdx.x == 0)
        atomicOr(&g_fault_word, LUCE_FAULT_BAD_ID);
}

template <typename TL, int VEC, bool S16>
luce_status launch_logits(const LogitsArgs &a, int R, int stretch, cudaStream_t stream)
{
    static luce_host::SmemLimit limit;
    auto kern = k_logits_process<TL, VEC, S16>;
    const size_t smem = a.hist || a.nbias ? ((size_t)stretch * (S16 ? 2 : 4) + 15) / 16 * 16 : 0;
    if (smem > 48 * 1024 && limit.raise(kern, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const luce_status st = luce_host::launch(kern, dim3((unsigned)((a.V + stretch - 1) / stretch), (unsigned)R),
                                             dim3(THREADS), smem, stream, a, stretch);
    if (st != LUCE_OK)
        limit.forget();
    return st;
}

template <typename TL> luce_status run_logits(const LogitsArgs &a, int R, cudaStream_t stream)
{
    const bool s16 = a.ldh <= 32767 && a.nbias <= 65534; // counts, and the biases' places, fit sixteen bits
    // as few stretches as shared memory allows with two CTAs to an SM, more
    // while that leaves SMs idle, 512 tokens at least, of one length
    const int64_t most = (size_t)100 * 1024 / (s16 ? 2 : 4);
    const int64_t fill = std::max<int64_t>(1, 2 * luce_host::sm_count() / R);
    const int64_t n = std::max((a.V + most - 1) / most, std::min(fill, (a.V + 511) / 512));
    const int stretch = (int)(((a.V + n - 1) / n + 31) & ~(int64_t)31);
    const bool vec = luce_host::aligned(a.logits, 4 * sizeof(TL)) && luce_host::aligned(a.out, 16) &&
                     (R == 1 || (a.ldl % 4 == 0 && a.ldo % 4 == 0));
    if (vec)
        return s16 ? launch_logits<TL, 4, true>(a, R, stretch, stream) : launch_logits<TL, 4, false>(a, R, stretch, stream);
    return s16 ? launch_logits<TL, 1, true>(a, R, stretch, stream) : launch_logits<TL, 1, false>(a, R, stretch, stream);
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
    cudaStream_t st = luce_host::as_stream(stream);
    switch (dtype) {
    case LUCE_F32:
        return run_logits<float>(a, R, st);
    case LUCE_BF16:
        return run_logits<__nv_bfloat16>(a, R, st);
    case LUCE_F16:
        return run_logits<__half>(a, R, st);
    }
    return LUCE_ERR_INVALID_ARG;
}
