// Rotary positions on the new tokens' queries and keys, and the keys and
// values appended to the paged cache, in one kernel.
//
// A pair (a, b) of a head turns by the angle p * freqs[i]:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos).
// The angle matters modulo one turn only, and p * freqs[i] reaches 10^5 and
// more, where an f32 product has lost the digits that cos and sin depend on:
// the product of a 24-bit and a 32-bit number fits a double, so the turns
// p * freqs[i] / 2 pi are taken in double, their whole part dropped, and the
// rest goes to sincospif in f32.  That is rot/2 angles to a token, shared by
// all its heads through shared memory.
//
// The bytes bound it: every value of q, k and v is read once and written once.
#include "serving.cuh"

namespace gg {

namespace {

constexpr int kThreads = 256;

template <class T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// V consecutive values through accesses of up to 16 bytes.
template <int V, class T>
__device__ __forceinline__ void load_v(const T* p, float (&f)[V]) {
    constexpr int B = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;  // bytes an access
    constexpr int N = B / (int)sizeof(T);
    struct alignas(B) Pack { T v[N]; };
#pragma unroll
    for (int j = 0; j < V / N; ++j) {
        const Pack k = reinterpret_cast<const Pack*>(p)[j];
#pragma unroll
        for (int i = 0; i < N; ++i) f[j * N + i] = to_f(k.v[i]);
    }
}
template <int V, class T>
__device__ __forceinline__ void store_v(T* p, const float (&f)[V]) {
    struct alignas(V * sizeof(T)) Pack { T v[V]; };
    Pack k;
#pragma unroll
    for (int i = 0; i < V; ++i) k.v[i] = from_f<T>(f[i]);
    *reinterpret_cast<Pack*>(p) = k;
}

// X: input type, C: cache type, V: values a thread moves at a time.  Block
// (x, y) takes token x and the y-th of gridDim.y shares of its values.
template <class X, class C, int V, bool NEOX>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
    __shared__ int s_seq;
    __shared__ float s_cos[64], s_sin[64];
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) s_seq = -1;
    __syncthreads();
    pdl_wait();
    for (int i = tid; i < p.b.n_seq; i += kThreads)
        if (p.b.q_start[i] <= t && t < p.b.q_start[i + 1]) s_seq = i;
    __syncthreads();
    pdl_launch_dependents();
    const int seq = s_seq;
    if (seq < 0) return;                          // past the last sequence
    const int pos = p.b.kv_len[seq] - p.b.q_start[seq + 1] + t;
    int64_t slot = -1;                            // element offset of the token in the cache, -1: not stored
    if (pos >= 0) {
        const int64_t col = pos >> p.c.page_shift;
        const int page = col < p.b.pages_stride ? p.b.pages[seq * p.b.pages_stride + col] : -1;
        if ((unsigned)page < (unsigned)p.c.n_pages)
            slot = page * p.c.page_stride + (pos & ((1 << p.c.page_shift) - 1)) * p.c.token_stride;
        else if (tid == 0)
            report(p.status, GGUF_ERR_INVALID_ARG);
    }
    const int half = p.rot >> 1;
    if (tid < half) {
        const int at = p.positions ? p.positions[t] : pos;
        const double turns = (double)at * (double)p.freqs[tid] * 0.15915494309189533577;  // 1 / (2 pi)
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        s_cos[tid] = cs * p.rope_scale;
        s_sin[tid] = sn * p.rope_scale;
    }
    __syncthreads();

    // a head's work: with halves, rot / 2V units that turn two vectors and the
    // rest that copy one; with neighbours, one vector each
    const int D = p.c.dim, HK = p.heads + p.c.kv_heads;
    const int turn = NEOX ? half / V : p.rot / V;
    const int units = turn + (D - p.rot) / V;
    const int n_qk = HK * units, n = n_qk + p.c.kv_heads * (D / V);
    C* kc = static_cast<C*>(p.c.k);
    C* vc = static_cast<C*>(p.c.v);
    for (int u = blockIdx.y * kThreads + tid; u < n; u += gridDim.y * kThreads) {
        if (u >= n_qk) {                          // a value: converted and stored
            const int w = u - n_qk, h = w / (D / V), d = (w - h * (D / V)) * V;
            if (slot < 0) continue;
            float f[V];
            load_v<V>(static_cast<const X*>(p.v) + t * p.ldv + h * D + d, f);
            store_v<V>(vc + slot + h * p.c.head_stride + d, f);
            continue;
        }
        const int h = u / units, w = u - h * units;
        const X* src;
        C* dst;
        if (h < p.heads) {
            src = static_cast<const X*>(p.q) + t * p.ldq + h * D;
            dst = static_cast<C*>(p.q_out) + t * p.ldqo + h * D;
        } else {
            if (slot < 0) continue;
            src = static_cast<const X*>(p.k) + t * p.ldk + (h - p.heads) * D;
            dst = kc + slot + (h - p.heads) * p.c.head_stride;
        }
        float a[V];
        if (w >= turn) {
            const int d = p.rot + (w - turn) * V;
            load_v<V>(src + d, a);
            store_v<V>(dst + d, a);
        } else if (NEOX) {
            const int d = w * V;
            float b[V], y[V], z[V];
            load_v<V>(src + d, a);
            load_v<V>(src + half + d, b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float cs = s_cos[d + i], sn = s_sin[d + i];
                y[i] = a[i] * cs - b[i] * sn;
                z[i] = a[i] * sn + b[i] * cs;
            }
            store_v<V>(dst + d, y);
            store_v<V>(dst + half + d, z);
        } else {
            const int d = w * V;
            float y[V];
            load_v<V>(src + d, a);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float cs = s_cos[d / 2 + i], sn = s_sin[d / 2 + i];
                y[2 * i] = a[2 * i] * cs - a[2 * i + 1] * sn;
                y[2 * i + 1] = a[2 * i] * sn + a[2 * i + 1] * cs;
            }
            store_v<V>(dst + d, y);
        }
    }
}

template <class X, class C, int V, bool NEOX>
cudaError_t launch(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    const int64_t per_token = (int64_t)(p.heads + 2 * p.c.kv_heads) * p.c.dim / V;
    // enough blocks to occupy the SMs when there are few tokens
    const int64_t share = std::max<int64_t>(1, std::min(ceil_div(per_token, kThreads), ceil_div(2 * num_sms, p.b.n_tokens)));
    return launch_pdl(kv_append_kernel<X, C, V, NEOX>, dim3(p.b.n_tokens, (unsigned)share), dim3(kThreads), 0, s, pdl, p);
}

template <class X, class C>
cudaError_t launch_v(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    // the widest vectors whose edges the rotated part's own edges meet
    const bool neox = p.style == GGUF_ROPE_NEOX && p.rot;
    const int edge = neox ? p.rot / 2 : p.rot;
    if (edge % 8 == 0) return neox ? launch<X, C, 8, true>(p, num_sms, pdl, s) : launch<X, C, 8, false>(p, num_sms, pdl, s);
    if (edge % 4 == 0) return neox ? launch<X, C, 4, true>(p, num_sms, pdl, s) : launch<X, C, 4, false>(p, num_sms, pdl, s);
    return neox ? launch<X, C, 1, true>(p, num_sms, pdl, s) : launch<X, C, 2, false>(p, num_sms, pdl, s);
}

template <class X>
cudaError_t launch_c(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    return p.c.bf16 ? launch_v<X, __nv_bfloat16>(p, num_sms, pdl, s) : launch_v<X, __half>(p, num_sms, pdl, s);
}

}  // namespace

cudaError_t kv_append_launch(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    if (p.xdt == GGUF_DT_F32) return launch_c<float>(p, num_sms, pdl, s);
    return p.xdt == GGUF_DT_F16 ? launch_c<__half>(p, num_sms, pdl, s) : launch_c<__nv_bfloat16>(p, num_sms, pdl, s);
}

}  // namespace gg
