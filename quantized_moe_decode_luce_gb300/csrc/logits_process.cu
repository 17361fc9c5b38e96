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
#include <type_traits>

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
// steps of four logits in flight for each thread, and as many requested behind
// them (256 bf16 rows of 129280 with 4096 history tokens: 44.5 us, with two 46.5;
// eight 16-bit logits to a step, whose stores then need a swap between lanes, 46.7)
constexpr int NB = 3;
constexpr int HB = 4; // history loads of a thread in flight (four tokens each)

// What a slot of shared memory holds for its token: twice the number of
// generated occurrences, the low bit set if the token is among the prompt's
// (the two never touch each other's bits, so their order does not matter).
// Sixteen bits hold 32,767 occurrences: enough for rows of up to SHORT tokens,
// whose last token is kept apart when all of them were generated.
constexpr int SHORT = 32768;
template <bool S16> struct Slots {
    uint32_t base;   // shared address
    uint32_t *words; // the same
    __device__ __forceinline__ uint32_t get(int at) const
    {
        uint32_t v;
        if (S16) {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(base + 2 * at));
            v = h;
        } else {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(base + 4 * at));
        }
        return v;
    }
    __device__ __forceinline__ void put(int at, uint32_t v) const
    {
        if (S16)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(base + 2 * at), "h"((uint16_t)v) : "memory");
        else
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + 4 * at), "r"(v) : "memory");
    }
    // one more generated (no carry between sixteen-bit slots: at most 65,535), or among the prompt's; if `live`
    template <bool PROMPT> __device__ __forceinline__ void count(int at, bool live) const
    {
        const uint32_t addr = base + (S16 ? (2 * at) & ~3 : 4 * at);
        const uint32_t v = (PROMPT ? 1u : 2u) << (S16 ? 16 * (at & 1) : 0);
        if (PROMPT)
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p red.shared.or.b32 [%0], %1;\n\t}" ::"r"(addr),
                         "r"(v), "r"((uint32_t)live)
                         : "memory");
        else
            asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p red.shared.add.u32 [%0], %1;\n\t}" ::"r"(addr),
                         "r"(v), "r"((uint32_t)live)
                         : "memory");
    }
    __device__ __forceinline__ void raise(int at, uint32_t v) const // the larger of the slot and v
    {
        if (!S16) {
            atomicMax(words + at, v);
            return;
        }
        uint32_t *p = words + (at >> 1), old = *p;
        const int sh = 16 * (at & 1);
        while (((old >> sh) & 0xffffu) < v) {
            const uint32_t seen = atomicCAS(p, old, (old & ~(0xffffu << sh)) | v << sh);
            if (seen == old)
                break;
            old = seen;
        }
    }
    // the slots of N tokens from `at` (a multiple of N), as words
    template <int N> static constexpr int WORDS = S16 && N > 1 ? N / 2 : N;
    template <int N> __device__ __forceinline__ void get_words(int at, uint32_t (&x)[WORDS<N>]) const
    {
        if constexpr (N == 1)
            x[0] = get(at);
        else if constexpr (S16)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(base + 2 * at));
        else
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(base + 4 * at));
    }
    template <int N> static __device__ __forceinline__ void unpack(const uint32_t (&x)[WORDS<N>], uint32_t (&c)[N])
    {
#pragma unroll
        for (int i = 0; i < N; i++)
            c[i] = !S16 || N == 1 ? x[i] : i & 1 ? x[i / 2] >> 16 : x[i / 2] & 0xffffu;
    }
};

// Logits from LOW to below HIGH, over a penalty from 2^-40 to 2^40, go through
// Markstein's division below without any result that over- or underflows.
constexpr uint32_t LOW = 0x20000000u; // 2^-63
constexpr int HIGH = 0x60000000;      // 2^65

// The penalties of N tokens whose slots hold c, without a branch in the common
// case.  l / rep, correctly rounded, comes from rinv = fl(1 / rep) by Markstein's
// sequence: a product, its exact remainder and one correction (6000 penalties
// over all 2^23 significands of a logit gave no other quotient).  Where one of
// the logits is +0, or positive and below `low` or not below HIGH, all N divide
// (low is LOW, or above all floats where rep is out of range).
template <bool S16, int N>
__device__ __forceinline__ void penalize(float (&w)[N], const uint32_t (&c)[N], float rep, float rinv, uint32_t low,
                                         float freq, float pres)
{
    float p[N];
    uint32_t lowest = ~0u; // of the bits: negative values lie above all positive ones,
    int highest = 0;       // and, signed, below
#pragma unroll
    for (int e = 0; e < N; e++) {
        const float l = w[e], q = __fmul_rn(l, rinv);
        const float s = fmaf(fmaf(-q, rep, l), rinv, q);
        p[e] = l > 0.0f ? s : __fmul_rn(l, rep);
        lowest = min(lowest, __float_as_uint(l));
        highest = max(highest, __float_as_int(l));
    }
    if (lowest < low || highest >= HIGH) {
#pragma unroll
        for (int e = 0; e < N; e++)
            p[e] = w[e] > 0.0f ? __fdiv_rn(w[e], rep) : __fmul_rn(w[e], rep);
    }
#pragma unroll
    for (int e = 0; e < N; e++) {
        const uint32_t k = c[e] >> 1;
        // (at most SHORT: exact in the low bits of 2^23)
        const float f = S16 ? __fsub_rn(__uint_as_float(0x4b000000u | k), 8388608.0f) : (float)k;
        const float g = __fsub_rn(p[e], __fadd_rn(__fmul_rn(f, freq), pres));
        w[e] = k ? g : c[e] ? p[e] : w[e];
    }
}

// N logits as they lie in memory, in whole words.
template <typename TL, int N> struct Raw {
    static constexpr int W = N * sizeof(TL) / 4;
    uint32_t w[W ? W : 1];
    __device__ __forceinline__ void load(const TL *p)
    {
        if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            w[0] = x.x, w[1] = x.y;
        } else if constexpr (W == 1)
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        else
            w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
    __device__ __forceinline__ void values(float (&v)[N]) const
    {
#pragma unroll
        for (int i = 0; i < N; i++) {
            if constexpr (sizeof(TL) == 4)
                v[i] = __uint_as_float(w[i]);
            else if constexpr (std::is_same_v<TL, __half>)
                v[i] = __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> 16 * (i & 1))));
            else
                v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
};

// VEC logits a step and thread: four, or one.  A row may start `sh`
// elements behind a boundary of VEC elements (the same for logits and out:
// checked by the host), so a stretch is gone through in steps that start at
// boundaries, u = v + sh; the tokens before the first whole step and behind the
// last go one to a thread.
template <typename TL, int VEC, bool S16>
__global__ void __launch_bounds__(THREADS, 2) k_logits_process(const LogitsArgs a, int stretch, int mask_at, int bias_at)
{
    extern __shared__ __align__(16) uint32_t slot_words[];
    const Slots<S16> slots{smem_addr(slot_words), slot_words}; // (slot u is that of token c0 + u - sh)
    const Slots<S16> places{smem_addr(slot_words + bias_at), slot_words + bias_at}; // a token's last bias entry, from one on; if bias_at > 0
    const int r = blockIdx.y, tid = threadIdx.x;
    const int64_t c0 = (int64_t)blockIdx.x * stretch;
    const int nc = (int)min((int64_t)stretch, a.V - c0);
    float *o = a.out + (size_t)r * a.ldo + c0;
    const int sh = VEC == 1 ? 0 : (int)((reinterpret_cast<uintptr_t>(o) >> 2) & (VEC - 1));
    // slots to zero (they do not depend on the previous kernel)
    const int words = S16 ? (nc + sh + 1) / 2 : nc + sh;
    if (a.hist)
        for (int i = tid; 4 * i < words; i += THREADS)
            reinterpret_cast<uint4 *>(slot_words)[i] = make_uint4(0, 0, 0, 0);
    if (bias_at)
        for (int i = tid; 4 * i < words; i += THREADS)
            reinterpret_cast<uint4 *>(places.words)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_trigger();
    const TL *lr = static_cast<const TL *>(a.logits) + (size_t)r * a.ldl + c0;
    const uint32_t *mr = nullptr;
    bool bad = false;
    if (a.mask || a.mask_rows) {
        const int m = a.mask_rows ? a.mask_rows[r] : r;
        if (m >= a.nmasks)
            bad = true;
        else if (m >= 0)
            mr = a.mask + (size_t)m * a.ldm + (c0 >> 5); // (c0 is a multiple of 32)
    }
    // the mask's words behind the slots, one word of padding before them
    uint32_t *mw = slot_words + mask_at;
    if (mr)
        for (int i = tid; i < (nc + 31) >> 5; i += THREADS)
            mw[1 + i] = mr[i];
    // a batch: the logits of NB steps
    struct Batch {
        Raw<TL, VEC> in[NB];
    };
    auto load = [&](Batch &b, int u0) {
#pragma unroll
        for (int i = 0; i < NB; i++) {
            const int v = u0 + (tid + i * THREADS) * VEC - sh;
            if (v >= 0 && v + VEC <= nc)
                b.in[i].load(lr + v);
        }
    };
    Batch cur;
    load(cur, 0);
    int edge = -1; // the thread's token outside the whole steps
    if (VEC > 1 && tid < 2 * VEC) {
        const int head = min((VEC - sh) & (VEC - 1), nc), tail = max((nc + sh) / VEC * VEC - sh, head);
        edge = tid < VEC ? (tid < head ? tid : -1) : tail + tid - VEC < nc ? tail + tid - VEC : -1;
    }
    const float edge_value = edge >= 0 ? to_f32(lr[edge]) : 0.0f;
    uint32_t low = LOW;
    float rep = 1.0f, rinv = 1.0f, freq = 0.0f, pres = 0.0f;
    int apart = -VEC; // slot of the generated token that no slot counts, if any
    const int32_t *ids = a.bias_ids + (size_t)r * a.nbias;
    const float *vals = a.bias_vals + (size_t)r * a.nbias;
    const int32_t bias_id = tid < a.nbias ? ids[tid] : -1; // (the first of a thread's)
    const float bias_val = tid < a.nbias ? vals[tid] : 0.0f;
    // f(u, j) for the bias entries j whose token lies in the stretch
    auto biases = [&](auto &&f) {
        for (int j = tid; j < a.nbias; j += THREADS) {
            const int32_t id = j == tid ? bias_id : ids[j];
            const uint32_t at = (uint32_t)id - (uint32_t)c0;
            if (at < (uint32_t)nc)
                f((int)at, j);
            bad |= id >= a.V;
        }
    };
    auto find_places = [&] {
        if (bias_at)
            biases([&](int at, int j) { places.raise(at + sh, (uint32_t)j + 1u); });
    };
    if (a.hist) {
        const int32_t *h = a.hist + (size_t)r * a.ldh;
        // tokens before a 16-byte boundary, quads from there, and a rest; the first
        // quads are requested before the length is known (they lie within ld_hist)
        const int head = (int)((4 - ((reinterpret_cast<uintptr_t>(h) >> 2) & 3)) & 3);
        const int4 *h4 = reinterpret_cast<const int4 *>(h + head);
        const int all_quads = a.ldh > head ? (int)((a.ldh - head) >> 2) : 0;
        int4 t[HB];
        auto request = [&](int q0, int quads) {
#pragma unroll
            for (int i = 0; i < HB; i++) {
                const int q = q0 + i * THREADS + tid;
                t[i] = q < quads ? h4[q] : make_int4(-1, -1, -1, -1);
            }
        };
        request(0, all_quads);
        int len = (int)min((int64_t)max(a.hist_len[r], 0), a.ldh);
        const int plen = a.prompt_len ? a.prompt_len[r] : 0;
        rep = a.rep ? a.rep[r] : 1.0f;
        freq = a.freq ? a.freq[r] : 0.0f;
        pres = a.pres ? a.pres[r] : 0.0f;
        rinv = __fdiv_rn(1.0f, rep);
        low = rep >= 0x1p-40f && rep <= 0x1p40f ? LOW : ~0u;
        const uint32_t lo = (uint32_t)c0;
        int32_t top = -1; // the largest id seen
        if (S16 && len == SHORT && plen <= 0) {
            top = h[--len];
            const uint32_t at = (uint32_t)top - lo;
            apart = at < (uint32_t)nc ? (int)at + sh : -VEC;
        }
        // (c0 + nc <= V < 2^31, so that one unsigned comparison also leaves out negative ids)
        auto prompt = [&](int32_t id) {
            top = max(top, id);
            const uint32_t at = (uint32_t)id - lo;
            slots.template count<true>((int)at + sh, at < (uint32_t)nc);
        };
        auto made = [&](int32_t id) {
            top = max(top, id);
            const uint32_t at = (uint32_t)id - lo;
            slots.template count<false>((int)at + sh, at < (uint32_t)nc);
        };
        auto one = [&](int32_t id, int i) {
            if (i >= len)
                return;
            if (i < plen)
                prompt(id);
            else
                made(id);
        };
        __syncthreads();
        find_places();
        if (tid < min(head, len))
            one(h[tid], tid);
        const int quads = len > head ? (len - head) >> 2 : 0;
        for (int q0 = 0; q0 < quads;) {
#pragma unroll
            for (int i = 0; i < HB; i++) {
                const int q = q0 + i * THREADS + tid, at = head + 4 * q;
                if (q >= quads)
                    break;
                const int32_t id[4] = {t[i].x, t[i].y, t[i].z, t[i].w};
                if (at + 4 <= plen) {
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        prompt(id[k]);
                } else if (at >= plen) {
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        made(id[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        one(id[k], at + k);
                }
            }
            q0 += HB * THREADS;
            if (q0 < quads)
                request(q0, quads);
        }
        const int rest = head + 4 * quads + tid;
        if (tid < 4 && rest < len && len > head)
            one(h[rest], rest);
        bad |= top >= a.V;
    } else if (bias_at) {
        __syncthreads();
        find_places();
    }
    __syncthreads();
    // the N logits of slots u ..
    auto finish = [&](auto &w, int u) {
        constexpr int N = sizeof(w) / sizeof(float);
        if (a.hist) {
            uint32_t x[Slots<S16>::template WORDS<N>], any = 0;
            slots.template get_words<N>(u, x);
#pragma unroll
            for (uint32_t word : x)
                any |= word;
            const bool has_apart = S16 && (uint32_t)(apart - u) < (uint32_t)N;
            if (any || has_apart) {
                uint32_t c[N];
                slots.template unpack<N>(x, c);
                if (has_apart) {
#pragma unroll
                    for (int e = 0; e < N; e++)
                        c[e] += u + e == apart ? 2u : 0u;
                }
                penalize<S16, N>(w, c, rep, rinv, low, freq, pres);
            }
        }
        if (bias_at) {
            uint32_t x[Slots<S16>::template WORDS<N>], any = 0;
            places.template get_words<N>(u, x);
#pragma unroll
            for (uint32_t word : x)
                any |= word;
            if (any) {
                uint32_t j[N];
                places.template unpack<N>(x, j);
#pragma unroll
                for (int e = 0; e < N; e++)
                    if (j[e])
                        w[e] = __fadd_rn(w[e], vals[j[e] - 1]);
            }
        }
        if (mr) {
            const int v = u - sh, at = (v >> 5) + 1;
            const uint32_t bits = N == 1 ? mw[at] >> (v & 31) : __funnelshift_r(mw[at], mw[at + 1], v & 31);
#pragma unroll
            for (int e = 0; e < N; e++)
                if (!((bits >> e) & 1u))
                    w[e] = -INFINITY;
        }
    };
    for (int u0 = 0; u0 < nc + sh; u0 += NB * THREADS * VEC) {
        Batch next;
        load(next, u0 + NB * THREADS * VEC);
#pragma unroll
        for (int i = 0; i < NB; i++) {
            const int u = u0 + (tid + i * THREADS) * VEC, v = u - sh;
            if (v < 0 || v + VEC > nc)
                continue;
            float w[VEC];
            cur.in[i].values(w);
            finish(w, u);
            if constexpr (VEC == 1)
                o[v] = w[0];
            else
                *reinterpret_cast<float4 *>(o + v) = make_float4(w[0], w[1], w[2], w[3]);
        }
        cur = next;
    }
    if (edge >= 0) {
        float w[1] = {edge_value};
        finish(w, edge + sh);
        o[edge] = w[0];
    }
    if (a.nbias && !bias_at) {
        // no room for the places: the slots now find each id's last entry, which
        // adds its bias to the value stored above unless the token is masked
        __syncthreads();
        biases([&](int at, int) { slots.put(at, 0); });
        __syncthreads();
        biases([&](int at, int j) { slots.raise(at, (uint32_t)j + 1u); });
        __syncthreads();
        biases([&](int at, int j) {
            if (slots.get(at) == (uint32_t)j + 1u && (!mr || ((mw[1 + (at >> 5)] >> (at & 31)) & 1u)))
                o[at] = __fadd_rn(o[at], j == tid ? bias_val : vals[j]);
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
    const size_t table = ((size_t)(stretch + 2 * VEC) * (S16 ? 2 : 4) + 15) / 16 * 16;
    const size_t masks = a.mask ? ((size_t)stretch / 32 + 3) * 4 : 0;
    // slots; the biases' places beside them while two CTAs still fit an SM; the mask's words
    const bool beside = a.nbias && 2 * table + masks <= 110 * 1024;
    const size_t bias_at = beside ? table : 0, mask_at = bias_at + (a.hist || a.nbias ? table : 0);
    const size_t smem = mask_at + masks;
    if (smem > 48 * 1024 && limit.raise(kern, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        return LUCE_ERR_CUDA;
    }
    const luce_status st = luce_host::launch(kern, dim3((unsigned)((a.V + stretch - 1) / stretch), (unsigned)R),
                                             dim3(THREADS), smem, stream, a, stretch, (int)(mask_at / 4),
                                             (int)(bias_at / 4));
    if (st != LUCE_OK)
        limit.forget();
    return st;
}

template <typename TL> luce_status run_logits(const LogitsArgs &a, int R, cudaStream_t stream)
{
    const bool s16 = a.ldh <= SHORT && a.nbias <= 65534; // counts, and the biases' places, fit sixteen bits
    // as few stretches as shared memory allows with two CTAs to an SM, more
    // while that leaves SMs idle, 1024 tokens at least, of one length
    const int64_t most = (size_t)100 * 1024 / (s16 ? 2 : 4);
    const int64_t fill = std::max<int64_t>(1, 2 * luce_host::sm_count() / R);
    const int64_t n = std::max((a.V + most - 1) / most, std::min(fill, (a.V + 1023) / 1024));
    const int stretch = (int)(((a.V + n - 1) / n + 31) & ~(int64_t)31);
    // four logits at a step where a row of logits and of out lie at the same place between boundaries of four
    constexpr int VEC = 4;
    auto place = [](const void *p, size_t es) { return (int64_t)(reinterpret_cast<uintptr_t>(p) / es); };
    if ((place(a.logits, sizeof(TL)) - place(a.out, 4)) % VEC == 0 && (R == 1 || (a.ldl - a.ldo) % VEC == 0))
        return s16 ? launch_logits<TL, VEC, true>(a, R, stretch, stream) : launch_logits<TL, VEC, false>(a, R, stretch, stream);
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
    if ((hist == nullptr) != (hist_len == nullptr) || (!hist && prompt_len) || (!mask && mask_rows && n_masks != 0))
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
