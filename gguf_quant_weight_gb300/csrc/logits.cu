// Rules on a batch of logits: penalties for repeated tokens, biases, and a
// grammar's mask, in one pass over the logits.
//
// For a token that comes c times in its row's history
//   x = (x > 0 ? x / repeat : x * repeat) - (c * frequency + presence),
// then its biases are added and what the mask leaves out becomes -inf.
//
// A block takes one slice of one row.  It counts the history's tokens that
// fall into its slice with integer atomics in shared memory (their order does
// not matter), marks the biased ones, and then passes over its logits once,
// which every thread has had on their way meanwhile.  A biased token's list
// entries are added in the list's order, so the result does not depend on
// timing either (an entry alone for its token, the usual case, is added without
// going through the list).  The logits' bytes bound it; each block reads the row's whole
// history, from L2 after the first.
// Measured on GB300: 256 x 131072 f32 in and out, histories of 1..2048, in 50 us
// (5.4 of the 6.7 TB/s of a copy; without histories 40 us: a block's stores wait
// for its row's, and six blocks to an SM do not quite cover it; four take 57 us,
// although six leave f32's 16 tokens a thread 40 registers, 60 bytes too few),
// 37 x 128259 from bf16 with every rule in 10 us, one row of 32003 in 2.4 us.
#include "serving.cuh"

namespace gg {

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;       // of the history, read by a thread at once

template <int DT> struct El;
template <> struct El<GGUF_DT_F32> { using T = float; };
template <> struct El<GGUF_DT_F16> { using T = __half; };
template <> struct El<GGUF_DT_BF16> { using T = __nv_bfloat16; };
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// E: tokens a thread (a slice is kThreads * E).  Groups of tokens start at
// 16-byte boundaries of the row's inputs.
template <int DT, int ODT, int E>
__global__ void __launch_bounds__(kThreads, E == 32 ? 4 : 6) logits_adjust_kernel(const LogitsParams p) {
    using X = typename El<DT>::T;
    using Y = typename El<ODT>::T;
    constexpr int SLICE = kThreads * E;
    constexpr int G = 16 / (int)sizeof(X) < E ? 16 / (int)sizeof(X) : E;      // tokens of a group
    struct alignas(G * sizeof(X)) In { X v[G]; };
    __shared__ int s_count[SLICE];
    __shared__ uint32_t s_biased[SLICE / 32];    // in the list
    __shared__ uint32_t s_again[SLICE / 32];     // more than once
    __shared__ uint16_t s_entry[SLICE];          // where, of one that is there once
    const int r = blockIdx.y, tid = threadIdx.x;
    const X* x = static_cast<const X*>(p.x) + r * p.ld;
    Y* y = static_cast<Y*>(p.y) + r * p.ldo;
    const int m = (int)(r * p.ld & (G - 1));
    const int first = blockIdx.x * SLICE - m;                      // token of s_count[0]
    const int vocab = (int)p.vocab;
    if (p.r.hist)
        for (int i = tid; i < SLICE; i += kThreads) s_count[i] = 0;
    if (p.r.bias_ids && tid < SLICE / 32) s_biased[tid] = s_again[tid] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    // everything that depends on nothing, on its way at once: the row's numbers,
    // then the thread's groups tid, tid + kThreads, ...
    int h0 = 0, h1 = 0, b0 = 0, nb = 0;
    float repeat = 1.f, frequency = 0.f, presence = 0.f;
    if (p.r.hist) h0 = p.r.hist_start[r], h1 = p.r.hist_start[r + 1];
    if (p.r.bias_ids) b0 = p.r.bias_start[r], nb = p.r.bias_start[r + 1] - b0;
    if (p.r.repeat) repeat = p.r.repeat[r];
    if (p.r.frequency) frequency = p.r.frequency[r];
    if (p.r.presence) presence = p.r.presence[r];
    const uint32_t* allow = p.r.allow ? p.r.allow + r * p.r.allow_stride : nullptr;
    In in[E / G];
#pragma unroll
    for (int k = 0; k < E / G; ++k) {
        const int v0 = first + (tid + k * kThreads) * G;
        if (v0 >= 0 && v0 + G <= vocab) in[k] = *reinterpret_cast<const In*>(x + v0);
    }
    // a group's bits of the mask: from one word, or the end of one and the start of the next
    uint32_t bits[E / G];
    if (allow) {
#pragma unroll
        for (int k = 0; k < E / G; ++k) {
            const int v0 = first + (tid + k * kThreads) * G, w = v0 < 0 ? 0 : v0 >> 5;
            if (v0 >= vocab) continue;
            const int sh = v0 - 32 * w;
            const uint32_t lo = allow[w], hi = sh + G > 32 && 32 * (w + 1) < vocab ? allow[w + 1] : 0u;
            bits[k] = sh < 0 ? lo << -sh : __funnelshift_r(lo, hi, sh);
        }
    }
    int b_id = tid < nb ? p.r.bias_ids[b0 + tid] : -1;
    // An id counts where its distance from the slice's first token, modulo 2^32, is
    // inside the slice; what is counted there before the row's first token or past
    // its last is never looked at, so ids outside the vocabulary need no test.
    for (int i0 = h0 + tid; i0 < h1; i0 += kAtOnce * kThreads) {
        unsigned at[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            at[j] = i0 + j * kThreads < h1 ? (unsigned)p.r.hist[i0 + j * kThreads] - (unsigned)first : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (at[j] < SLICE) atomicAdd(&s_count[at[j]], 1);
    }
    for (int i = tid; i < nb; i += kThreads) {
        if (i != tid) b_id = p.r.bias_ids[b0 + i];
        const unsigned at = (unsigned)b_id - (unsigned)first;
        if (at < SLICE) {
            const uint32_t bit = 1u << (at & 31);
            if ((atomicOr(&s_biased[at >> 5], bit) & bit) || i > 0xffff) atomicOr(&s_again[at >> 5], bit);
            s_entry[at] = (uint16_t)i;
        }
    }
    __syncthreads();
    // x / repeat as a product with 1 / repeat, which is within two units of it (for any
    // repeat from 2^-126 to 2^126): a
    // division at every token's place in the unrolled code costs more than the rest
    // of the pass, in instructions to fetch
    const float inv = 1.f / repeat;
    auto penalised = [&](float v, int c) {
        return c ? v * (v > 0.f ? inv : repeat) - fmaf((float)c, frequency, presence) : v;
    };
    const bool out_wide = ((r * p.ldo - m) & (G - 1)) == 0;        // groups are aligned in the outputs too
#pragma unroll
    for (int k = 0; k < E / G; ++k) {
        const int at = (tid + k * kThreads) * G;
        const int v0 = first + at;
        if (v0 >= vocab) break;
        const bool whole = v0 >= 0 && v0 + G <= vocab;
        float f[G];
        if (whole) {
#pragma unroll
            for (int i = 0; i < G; ++i) f[i] = to_f(in[k].v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i) f[i] = v0 + i >= 0 && v0 + i < vocab ? to_f(x[v0 + i]) : 0.f;
        }
        if (p.r.hist) {
#pragma unroll
            for (int i = 0; i < G; i += 4) {
                const int4 c = *reinterpret_cast<const int4*>(s_count + at + i);
                if ((c.x | c.y | c.z | c.w) == 0) continue;
                f[i] = penalised(f[i], c.x);
                f[i + 1] = penalised(f[i + 1], c.y);
                f[i + 2] = penalised(f[i + 2], c.z);
                f[i + 3] = penalised(f[i + 3], c.w);
            }
        }
        if (nb > 0) {
            const int sh = at & 31;                                                // a group lies in one word
            const uint32_t again = s_again[at >> 5] >> sh & ((1u << G) - 1), once = s_biased[at >> 5] >> sh & ~again;
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (once >> i & 1) f[i] += p.r.bias[b0 + s_entry[at + i]];
            if (again) {
#pragma unroll 8
                for (int j = 0; j < nb; ++j) {
                    const unsigned i = (unsigned)p.r.bias_ids[b0 + j] - (unsigned)v0;
                    const float b = p.r.bias[b0 + j];
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        if ((unsigned)g == i && (again >> g & 1)) f[g] += b;
                }
            }
        }
        if (allow) {
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (!(bits[k] >> i & 1)) f[i] = -INFINITY;
        }
        if (whole && out_wide) {
            constexpr int N = 16 / (int)sizeof(Y) < G ? 16 / (int)sizeof(Y) : G;
            struct alignas(N * sizeof(Y)) Out { Y v[N]; };
#pragma unroll
            for (int i = 0; i < G; i += N) {
                Out o;
#pragma unroll
                for (int j = 0; j < N; ++j) put(&o.v[j], f[i + j]);
                *reinterpret_cast<Out*>(y + v0 + i) = o;
            }
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (v0 + i >= 0 && v0 + i < vocab) put(&y[v0 + i], f[i]);
        }
    }
}

template <int DT, int ODT>
cudaError_t launch(const LogitsParams& p, int num_sms, int pdl, cudaStream_t s) {
    // 64 bytes of a row a thread, so 4096 or 8192 tokens a block: fewer blocks read
    // the row's history; 1024 where that leaves SMs idle.  Where rows
    // begin inside a group, the groups start up to seven tokens before them.
    constexpr int E = DT == GGUF_DT_F32 ? 16 : 32;
    constexpr int G = DT == GGUF_DT_F32 ? 4 : 8;
    const int64_t span = p.vocab + (p.ld % G && p.rows > 1 ? G - 1 : 0);
    const bool small = ceil_div(span, kThreads * E) * p.rows < num_sms;
    const dim3 grid((unsigned)ceil_div(span, kThreads * (small ? 4 : E)), (unsigned)p.rows);
    return small ? launch_pdl(logits_adjust_kernel<DT, ODT, 4>, grid, dim3(kThreads), 0, s, pdl, p)
                 : launch_pdl(logits_adjust_kernel<DT, ODT, E>, grid, dim3(kThreads), 0, s, pdl, p);
}

template <int DT>
cudaError_t launch(const LogitsParams& p, int num_sms, int pdl, cudaStream_t s) {
    if (p.odt == GGUF_DT_F32) return launch<DT, GGUF_DT_F32>(p, num_sms, pdl, s);
    return p.odt == GGUF_DT_F16 ? launch<DT, GGUF_DT_F16>(p, num_sms, pdl, s) : launch<DT, GGUF_DT_BF16>(p, num_sms, pdl, s);
}

}  // namespace

cudaError_t logits_adjust_launch(const LogitsParams& p, int num_sms, int pdl, cudaStream_t s) {
    if (p.dt == GGUF_DT_F32) return launch<GGUF_DT_F32>(p, num_sms, pdl, s);
    return p.dt == GGUF_DT_F16 ? launch<GGUF_DT_F16>(p, num_sms, pdl, s) : launch<GGUF_DT_BF16>(p, num_sms, pdl, s);
}

}  // namespace gg
