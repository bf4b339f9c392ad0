// Rotary positions on the new tokens' queries and keys, and the keys and
// values appended to the paged cache, in one kernel.
//
// A pair (a, b) of a head turns by the angle p * freqs[i]:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos).
// The angle matters modulo one turn only, and p * freqs[i] reaches 10^5 and
// more, where an f32 product has lost the digits that cos and sin depend on:
// the turns p * freqs[i] / 2 pi are taken in double (a position of 31 bits
// leaves 22 and more after the point), their whole part dropped, and the rest
// goes to sincospif in f32.  That is rot/2 angles to a token, shared by
// all its heads through shared memory.
//
// The bytes bound it: every value of q, k and v is read once and written once.
// Measured on GB300 (32 + 2 x 8 heads of 128): 7.6k tokens from f32 rows in 44 us,
// 6.2 of the 6.7 TB/s that a copy reaches; one token in 2.5 us, of which the
// launch is most.  Blocks of 128 threads with two vectors ahead: with 256 threads
// the prompts take 45.5 us, with three vectors ahead 49 us (fewer blocks fit).
#include "serving.cuh"

namespace gg {

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 2;        // of a thread's vectors (pairs of them), on their way at once

template <class T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// V consecutive values as they lie, through accesses of up to 16 bytes.
template <int V, class T>
struct Raw {
    static constexpr int B = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;  // bytes an access
    static constexpr int N = B / (int)sizeof(T);
    struct alignas(B) Pack { T v[N]; };
    Pack p[V / N];
    __device__ __forceinline__ void load(const T* from) {
#pragma unroll
        for (int j = 0; j < V / N; ++j) p[j] = reinterpret_cast<const Pack*>(from)[j];
    }
    __device__ __forceinline__ float operator[](int i) const { return to_f(p[i / N].v[i % N]); }
};
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
//
// What takes time with few tokens is the chain of dependent reads (sequence,
// page, then the angles), so it is kept short -- every thread reads one
// sequence's numbers, and the one whose token it is goes on -- and each
// thread's first values are on their way meanwhile: where they lie does not
// depend on it.
template <class X, class C, int V, bool NEOX>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
    __shared__ int s_found, s_disorder, s_pos;
    __shared__ int64_t s_slot;                    // element offset of the token in the cache, -1: not stored
    __shared__ float s_cos[64], s_sin[64];
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) s_found = s_disorder = 0;

    // a head's work: with halves, rot / 2V units that turn two vectors and the
    // rest that copy one; with neighbours, one vector each
    const int half = p.rot >> 1;
    const int D = p.c.dim, HK = p.heads + p.c.kv_heads;
    const int turn = NEOX ? half / V : p.rot / V;
    const int units = turn + (D - p.rot) / V;
    const int n_qk = HK * units, n = n_qk + p.c.kv_heads * (D / V);
    const int step = gridDim.y * kThreads;
    struct Unit {
        const X* src;
        int h, d;              // head (queries, keys, values one after the other), first value
        bool two;              // turns the vectors at d and half + d
        Raw<V, X> a, b;
    };
    auto find = [&](int u, Unit& w) {
        w.two = false;
        if (u >= n_qk) {
            const int v = u - n_qk, h = v / (D / V);
            w.h = HK + h;
            w.d = (v - h * (D / V)) * V;
            w.src = static_cast<const X*>(p.v) + t * p.ldv + h * D;
        } else {
            w.h = u / units;
            const int x = u - w.h * units;
            w.d = x < turn ? x * V : p.rot + (x - turn) * V;
            w.two = NEOX && x < turn;
            w.src = w.h < p.heads ? static_cast<const X*>(p.q) + t * p.ldq + w.h * D
                                  : static_cast<const X*>(p.k) + t * p.ldk + (w.h - p.heads) * D;
        }
        w.a.load(w.src + w.d);
        if (w.two) w.b.load(w.src + half + w.d);
    };
    __syncthreads();
    pdl_wait();
    int u0 = blockIdx.y * kThreads + tid;
    Unit ws[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        if (u0 + j * step < n) find(u0 + j * step, ws[j]);           // of a row past the last sequence in vain
    const int64_t room = p.b.pages_stride << p.c.page_shift;
    for (int i = tid; i < p.b.n_seq; i += kThreads) {
        const int from = p.b.q_start[i], to = p.b.q_start[i + 1], len = p.b.kv_len[i];
        const bool off = from < 0 || to < from || to > p.b.n_tokens || to - from > p.b.max_q || len > room || len > p.b.max_kv;
        if (to < from) s_disorder = 1;          // a token may be in two sequences: none is touched
        if (off) {
            if (t == 0 && blockIdx.y == 0) report(p.status, GGUF_ERR_INVALID_ARG);
        } else if (from <= t && t < to) {
            const int pos = (int)max((int64_t)INT32_MIN, (int64_t)len - to + t);
            s_pos = pos;
            s_found = 1;
            int64_t slot = -1;
            if (pos >= 0) {
                const int64_t col = pos >> p.c.page_shift;
                const int page = p.b.pages[i * p.b.pages_stride + col];
                if ((unsigned)page < (unsigned)p.c.n_pages)
                    slot = page * p.c.page_stride + (pos & ((1 << p.c.page_shift) - 1)) * p.c.token_stride;
                else
                    report(p.status, GGUF_ERR_INVALID_ARG);
            }
            s_slot = slot;
        }
    }
    __syncthreads();
    pdl_launch_dependents();
    if (!s_found || s_disorder) return;
    if (tid < half) {
        const int at = p.positions ? p.positions[t] : s_pos;
        const double turns = (double)at * (double)p.freqs[tid] * 0.15915494309189533577;  // 1 / (2 pi)
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        s_cos[tid] = cs * p.rope_scale;
        s_sin[tid] = sn * p.rope_scale;
    }
    __syncthreads();
    const int64_t slot = s_slot;
    auto write = [&](const Unit& w) {
        if (w.h < p.heads || slot >= 0) {
            C* dst = w.h < p.heads ? static_cast<C*>(p.q_out) + t * p.ldqo + w.h * D
                   : w.h < HK      ? static_cast<C*>(p.c.k) + slot + (w.h - p.heads) * p.c.head_stride
                                   : static_cast<C*>(p.c.v) + slot + (w.h - HK) * p.c.head_stride;
            if (w.h >= HK || w.d >= p.rot) {
                float y[V];
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = w.a[i];
                store_v<V>(dst + w.d, y);
            } else if (NEOX) {
                float y[V], z[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float cs = s_cos[w.d + i], sn = s_sin[w.d + i];
                    y[i] = w.a[i] * cs - w.b[i] * sn;
                    z[i] = w.a[i] * sn + w.b[i] * cs;
                }
                store_v<V>(dst + w.d, y);
                store_v<V>(dst + half + w.d, z);
            } else {
                float y[V];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float cs = s_cos[w.d / 2 + i], sn = s_sin[w.d / 2 + i];
                    y[2 * i] = w.a[2 * i] * cs - w.a[2 * i + 1] * sn;
                    y[2 * i + 1] = w.a[2 * i] * sn + w.a[2 * i + 1] * cs;
                }
                store_v<V>(dst + w.d, y);
            }
        }
    };
    while (true) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (u0 + j * step < n) write(ws[j]);
        u0 += kAhead * step;
        if (u0 >= n) break;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (u0 + j * step < n) find(u0 + j * step, ws[j]);
    }
}

template <class X, class C, int V, bool NEOX>
cudaError_t launch(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    const int64_t per_token = (int64_t)(p.heads + 2 * p.c.kv_heads) * p.c.dim / V;
    // enough blocks to occupy the SMs when there are few tokens
    const int64_t share = std::max<int64_t>(1, std::min(ceil_div(per_token, kThreads), ceil_div(4 * num_sms, p.b.n_tokens)));
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
