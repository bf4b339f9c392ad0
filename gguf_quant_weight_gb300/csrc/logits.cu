// Rules on a batch of logits: penalties for repeated tokens, biases, and a
// grammar's mask, in one pass over the logits.
//
// For a token that comes c times in its row's history
//   x = (x > 0 ? x / repeat : x * repeat) - (c * frequency + presence),
// then its biases are added and what the mask leaves out becomes -inf.
//
// A block takes one slice of one row.  It counts the history's tokens that
// fall into its slice with integer atomics in shared memory (their order does
// not matter), marks the biased ones, and then passes over its logits once.
// A biased token's list entries are added in the list's order, so the result
// does not depend on timing either.  The logits' bytes bound it; each block
// reads the row's whole history, from L2 after the first.
#include "serving.cuh"

namespace gg {

namespace {

constexpr int kThreads = 256;
constexpr int kSlice = 4096;   // tokens a block

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

template <int DT, int ODT>
__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(const LogitsParams p) {
    using X = typename El<DT>::T;
    using Y = typename El<ODT>::T;
    __shared__ int s_count[kSlice + 4];
    __shared__ uint32_t s_biased[kSlice / 32 + 1];
    const int r = blockIdx.y, tid = threadIdx.x;
    const X* x = static_cast<const X*>(p.x) + r * p.ld;
    Y* y = static_cast<Y*>(p.y) + r * p.ldo;
    // groups of four tokens start at 16-byte boundaries of the row's inputs
    const int m = (int)(r * p.ld & 3);
    const int64_t first = (int64_t)blockIdx.x * kSlice - m;       // token of s_count[0]
    const int64_t vocab = p.vocab;
    for (int i = tid; i < kSlice + 4; i += kThreads) s_count[i] = 0;
    for (int i = tid; i < kSlice / 32 + 1; i += kThreads) s_biased[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    if (p.r.hist) {
        const int e = p.r.hist_start[r + 1];
        for (int i = p.r.hist_start[r] + tid; i < e; i += kThreads) {
            const int id = p.r.hist[i];
            const int64_t at = id - first;
            if (id >= 0 && id < vocab && at >= 0 && at < kSlice) atomicAdd(&s_count[at], 1);
        }
    }
    int b0 = 0, b1 = 0;
    if (p.r.bias_ids) {
        b0 = p.r.bias_start[r];
        b1 = p.r.bias_start[r + 1];
        for (int i = b0 + tid; i < b1; i += kThreads) {
            const int id = p.r.bias_ids[i];
            const int64_t at = id - first;
            if (id >= 0 && id < vocab && at >= 0 && at < kSlice) atomicOr(&s_biased[at >> 5], 1u << (at & 31));
        }
    }
    __syncthreads();
    const float repeat = p.r.repeat ? p.r.repeat[r] : 1.f;
    const float frequency = p.r.frequency ? p.r.frequency[r] : 0.f;
    const float presence = p.r.presence ? p.r.presence[r] : 0.f;
    const uint32_t* allow = p.r.allow ? p.r.allow + r * p.r.allow_stride : nullptr;
    const bool out4 = ((r * p.ldo - m) & 3) == 0;                  // groups are aligned in the outputs too
    for (int g = tid; g < kSlice / 4; g += kThreads) {
        const int64_t v0 = first + 4 * g;
        if (v0 >= vocab) break;
        const bool whole = v0 >= 0 && v0 + 4 <= vocab;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (whole) {
            struct alignas(4 * sizeof(X)) Pack { X v[4]; };
            const Pack k = *reinterpret_cast<const Pack*>(x + v0);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = to_f(k.v[i]);
        } else {
            for (int i = 0; i < 4; ++i)
                if (v0 + i >= 0 && v0 + i < vocab) f[i] = to_f(x[v0 + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t v = v0 + i;
            if (v < 0 || v >= vocab) continue;
            const int c = s_count[4 * g + i];
            if (c) f[i] = (f[i] > 0.f ? f[i] / repeat : f[i] * repeat) - fmaf((float)c, frequency, presence);
            if (s_biased[(4 * g + i) >> 5] >> ((4 * g + i) & 31) & 1)
                for (int j = b0; j < b1; ++j)
                    if (p.r.bias_ids[j] == v) f[i] += p.r.bias[j];
            if (allow && !(allow[v >> 5] >> (v & 31) & 1)) f[i] = -INFINITY;
        }
        if (whole && out4) {
            struct alignas(4 * sizeof(Y)) Pack { Y v[4]; };
            Pack k;
#pragma unroll
            for (int i = 0; i < 4; ++i) put(&k.v[i], f[i]);
            *reinterpret_cast<Pack*>(y + v0) = k;
        } else {
            for (int i = 0; i < 4; ++i)
                if (v0 + i >= 0 && v0 + i < vocab) put(&y[v0 + i], f[i]);
        }
    }
}

template <int DT>
cudaError_t launch(const LogitsParams& p, int pdl, cudaStream_t s) {
    // a row's groups may start up to three tokens before it
    const dim3 grid((unsigned)ceil_div(p.vocab + 3, kSlice), (unsigned)p.rows);
    switch (p.odt) {
        case GGUF_DT_F32: return launch_pdl(logits_adjust_kernel<DT, GGUF_DT_F32>, grid, dim3(kThreads), 0, s, pdl, p);
        case GGUF_DT_F16: return launch_pdl(logits_adjust_kernel<DT, GGUF_DT_F16>, grid, dim3(kThreads), 0, s, pdl, p);
        default: return launch_pdl(logits_adjust_kernel<DT, GGUF_DT_BF16>, grid, dim3(kThreads), 0, s, pdl, p);
    }
}

}  // namespace

cudaError_t logits_adjust_launch(const LogitsParams& p, int num_sms, int pdl, cudaStream_t s) {
    (void)num_sms;
    if (p.dt == GGUF_DT_F32) return launch<GGUF_DT_F32>(p, pdl, s);
    return p.dt == GGUF_DT_F16 ? launch<GGUF_DT_F16>(p, pdl, s) : launch<GGUF_DT_BF16>(p, pdl, s);
}

}  // namespace gg
