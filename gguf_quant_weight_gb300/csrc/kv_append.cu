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

// Where a block's token belongs, found by all of its threads together.
struct Place {
    int found, disorder, pos;
    int64_t slot;                                 // element offset of the token in the cache, -1: not stored
};

__device__ __forceinline__ void search(const AppendParams& p, int t, Place& at) {
    const int64_t room = p.b.pages_stride << p.c.page_shift;
    for (int i = threadIdx.x; i < p.b.n_seq; i += kThreads) {
        const int from = p.b.q_start[i], to = p.b.q_start[i + 1], len = p.b.kv_len[i];
        const bool off = from < 0 || to < from || to > p.b.n_tokens || to - from > p.b.max_q || len > room || len > p.b.max_kv;
        if (to < from) at.disorder = 1;          // a token may be in two sequences: none is touched
        if (off) {
            if (t == 0 && blockIdx.y == 0) report(p.status, GGUF_ERR_INVALID_ARG);
        } else if (from <= t && t < to) {
            const int pos = (int)max((int64_t)INT32_MIN, (int64_t)len - to + t);
            at.pos = pos;
            at.found = 1;
            int64_t slot = -1;
            if (pos >= 0) {
                const int64_t col = pos >> p.c.page_shift;
                const int page = p.b.pages[i * p.b.pages_stride + col];
                if ((unsigned)page < (unsigned)p.c.n_pages)
                    slot = page * p.c.page_stride + (pos & ((1 << p.c.page_shift) - 1)) * p.c.token_stride;
                else
                    report(p.status, GGUF_ERR_INVALID_ARG);
            }
            at.slot = slot;
        }
    }
}

__device__ __forceinline__ void angle(const AppendParams& p, int t, int pos, int i, float& cos, float& sin) {
    const int at = p.positions ? p.positions[t] : pos;
    const double turns = (double)at * (double)p.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
    float sn, cs;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
    cos = cs * p.rope_scale;
    sin = sn * p.rope_scale;
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
    __shared__ Place at;
    __shared__ float s_cos[64], s_sin[64];
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) at.found = at.disorder = 0;

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
    search(p, t, at);
    __syncthreads();
    pdl_launch_dependents();
    if (!at.found || at.disorder) return;
    if (tid < half) angle(p, t, at.pos, tid, s_cos[tid], s_sin[tid]);
    __syncthreads();
    const int64_t slot = at.slot;
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

// The same for positions below 2^24, which are floats, and angles below 2^22 turns, without doubles (of which an SM does two a
// cycle): the frequency in turns in two floats, and what the product's rounding leaves by a second product.  Off by 2^-46 of
// the turns and by two roundings of a part below one half, 2^-24 of a turn.  (48 mixed sequences: 10.1 us with doubles, 9.5
// so; 9,600 tokens 55.1 and 52.5.)
__device__ __forceinline__ void near_angle(const AppendParams& p, int t, int pos, int i, float& cos, float& sin) {
    const int at = p.positions ? p.positions[t] : pos;
    constexpr float kHigh = 0.15915494f, kLow = 6.4206383e-9f;      // 1 / (2 pi)
    const float f = p.freqs[i], high = __fmul_rn(f, kHigh), low = __fmaf_rn(f, kHigh, -high) + f * kLow;
    const float a = (float)at, turns = __fmul_rn(a, high), rest = __fmaf_rn(a, high, -turns) + a * low;
    if (!(fabsf(a) < 0x1p24f && fabsf(turns) < 0x1p22f)) return angle(p, t, pos, i, cos, sin);
    float sn, cs;
    sincospif(2.f * ((turns - rintf(turns)) + rest), &sn, &cs);
    cos = cs * p.rope_scale;
    sin = sn * p.rope_scale;
}

// V consecutive floats of shared memory (V * 4 bytes aligned, up to 16)
template <int V>
__device__ __forceinline__ void read_v(const float* p, float (&f)[V]) {
    constexpr int N = V < 4 ? V : 4;
    struct alignas(4 * N) Pack { float v[N]; };
#pragma unroll
    for (int i = 0; i < V; i += N) {
        const Pack k = *reinterpret_cast<const Pack*>(p + i);
#pragma unroll
        for (int j = 0; j < N; ++j) f[i + j] = k.v[j];
    }
}

// The same with the heads of q and k normed on the way:
//   x -> x / sqrt(mean(x^2) + eps) * weight, then turned.
// A head is held by a group of `lanes` lanes (a power of two, its last ones
// idle where the head's units are fewer), so that the sum of squares takes a
// few shuffles and each value is still read once; a lane takes U units of the
// head, more than one only where the rotated part's edges keep vectors below
// four values.  Values are copied by the same groups.
// Bytes bound it, and next to them the arithmetic of norm and turn, some 60 % of
// the issue slots.  One head of a lane is on its way while blocks enough are on the
// SM: with two (and 16 more registers, so fewer blocks) 9,600 tokens of 40 heads in f32 take
// 60.5 us and not 53.0 (5.5 TB/s), in bf16 68.7 and not 52.5, and 48 mixed sequences 8.9 and not
// 9.7; with 8 bytes a lane in bf16 54.8, and 66.8 where pairs are neighbours.
template <class X, class C, int V, bool NEOX>
__global__ void __launch_bounds__(kThreads) kv_append_norm_kernel(const AppendParams p, int lanes) {
    constexpr int U = V >= 4 ? 1 : V == 2 ? 2 : 4;
    __shared__ Place at;
    __shared__ __align__(16) float s_cos[64], s_sin[64], s_wq[128], s_wk[128];
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) at.found = at.disorder = 0;
    const int half = p.rot >> 1;
    const int D = p.c.dim, HK = p.heads + p.c.kv_heads, n = HK + p.c.kv_heads;
    const int turn = NEOX ? half / V : p.rot / V;
    const int units = turn + (D - p.rot) / V;
    const int groups = kThreads / lanes, step = gridDim.y * groups, me = tid & (lanes - 1);
    struct Head {
        Raw<V, X> a[U], b[NEOX ? U : 1];
    };
    // unit u of a head starts at value `first` and, in a turned pair of halves, at half + first
    auto first = [&](int u) { return u < turn ? u * V : p.rot + (u - turn) * V; };
    auto fetch = [&](int h, Head& w) {
        const X* src = h < p.heads ? static_cast<const X*>(p.q) + t * p.ldq + h * D
                       : h < HK    ? static_cast<const X*>(p.k) + t * p.ldk + (h - p.heads) * D
                                   : static_cast<const X*>(p.v) + t * p.ldv + (h - HK) * D;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = me + i * lanes;
            if (u >= units) continue;
            w.a[i].load(src + first(u));
            if (NEOX && u < turn) w.b[i].load(src + half + first(u));
        }
    };
    __syncthreads();
    pdl_wait();
    int h0 = blockIdx.y * groups + tid / lanes;
    Head w{};                        // what a lane has no unit for stays 0, so a head's sum can take all lanes
    if (h0 < n) fetch(h0, w);
    if (tid < D) {
        if (p.q_norm) s_wq[tid] = p.q_norm[tid];
        if (p.k_norm) s_wk[tid] = p.k_norm[tid];
    }
    search(p, t, at);
    __syncthreads();
    pdl_launch_dependents();
    if (!at.found || at.disorder) return;
    if (tid < half) near_angle(p, t, at.pos, tid, s_cos[tid], s_sin[tid]);
    __syncthreads();
    const int64_t slot = at.slot;
    // a lane's units are the same of every head, and so are their angles
    constexpr int P = NEOX ? V : V / 2;           // pairs of a unit
    float cs[U][P], sn[U][P];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = me + i * lanes;
        if (u < turn) read_v<P>(s_cos + u * P, cs[i]), read_v<P>(s_sin + u * P, sn[i]);
    }
    const float per_value = 1.f / (float)D;
    // the whole warp comes here for as many heads as any of its groups has
    auto write = [&](int h) {
        float a[U][V], b[U][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                a[i][k] = w.a[i][k];
                sum = fmaf(a[i][k], a[i][k], sum);
                if (NEOX) {
                    b[i][k] = w.b[NEOX ? i : 0][k];
                    sum = fmaf(b[i][k], b[i][k], sum);
                }
            }
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (h >= n || !(h < p.heads || slot >= 0)) return;
        const float* weight = h < p.heads ? (p.q_norm ? s_wq : nullptr) : h < HK && p.k_norm ? s_wk : nullptr;
        const float inv = rsqrtf(fmaf(sum, per_value, p.eps));       // to two units in the last place
        C* dst = h < p.heads ? static_cast<C*>(p.q_out) + t * p.ldqo + h * D
                 : h < HK    ? static_cast<C*>(p.c.k) + slot + (h - p.heads) * p.c.head_stride
                             : static_cast<C*>(p.c.v) + slot + (h - HK) * p.c.head_stride;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = me + i * lanes;
            if (u >= units) continue;
            const int d = first(u);
            if (weight) {
                float f[V];
                read_v<V>(weight + d, f);
#pragma unroll
                for (int k = 0; k < V; ++k) a[i][k] *= inv * f[k];
                if (NEOX && u < turn) {
                    read_v<V>(weight + half + d, f);
#pragma unroll
                    for (int k = 0; k < V; ++k) b[i][k] *= inv * f[k];
                }
            }
            if (h < HK && u < turn) {
                if (NEOX) {
                    float y[V], z[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        y[k] = a[i][k] * cs[i][k % P] - b[i][k] * sn[i][k % P];
                        z[k] = a[i][k] * sn[i][k % P] + b[i][k] * cs[i][k % P];
                    }
                    store_v<V>(dst + d, y);
                    store_v<V>(dst + half + d, z);
                } else {
                    float y[V];
#pragma unroll
                    for (int k = 0; k < V / 2; ++k) {
                        y[2 * k] = a[i][2 * k] * cs[i][k] - a[i][2 * k + 1] * sn[i][k];
                        y[2 * k + 1] = a[i][2 * k] * sn[i][k] + a[i][2 * k + 1] * cs[i][k];
                    }
                    store_v<V>(dst + d, y);
                }
            } else {
                store_v<V>(dst + d, a[i]);
                if (NEOX && u < turn) store_v<V>(dst + half + d, b[i]);
            }
        }
    };
    // a warp's groups hold neighbouring heads, so the first of them says when it is done
    for (int w0 = h0 - (tid & 31) / lanes; w0 < n; w0 += step, h0 += step) {
        write(h0);
        if (h0 + step < n) fetch(h0 + step, w);
    }
}

template <class X, class C, int V, bool NEOX>
cudaError_t launch_norm(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    const int half = p.rot / 2, units = (NEOX ? half / V : p.rot / V) + (p.c.dim - p.rot) / V;
    int lanes = 1;
    while (lanes < 32 && lanes < units) lanes *= 2;
    const int64_t heads = p.heads + 2 * p.c.kv_heads;
    const int64_t share = std::max<int64_t>(1, std::min(ceil_div(heads, kThreads / lanes), ceil_div(4 * num_sms, p.b.n_tokens)));
    return launch_pdl(kv_append_norm_kernel<X, C, V, NEOX>, dim3(p.b.n_tokens, (unsigned)share), dim3(kThreads), 0, s, pdl, p, lanes);
}

template <class X, class C, int V, bool NEOX>
cudaError_t launch(const AppendParams& p, int num_sms, int pdl, cudaStream_t s) {
    if (p.q_norm || p.k_norm) return launch_norm<X, C, V, NEOX>(p, num_sms, pdl, s);
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
