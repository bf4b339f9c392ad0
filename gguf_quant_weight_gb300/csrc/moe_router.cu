// The router of a mixture of experts: scores, the best top_k of them, their
// weights, in one kernel.
//   z[t][e] = x[t] . W[e];   p = softmax(z[t]) or sigmoid(z[t]);
//   the top_k experts of the largest p (+ bias), the lower index first among
//   equals;  weights p of those, divided by their sum if asked, times scale.
//
// Which experts a token takes is decided to twice f32's digits.  The products are summed in
// f32, whose error is at most n 2^-24 |x| |W[e]| (n additions deep, norms by
// Cauchy and Schwarz).  Where two
// neighbours in the order lie closer than that allows, the scores of the experts
// that could be among the first top_k are computed again with compensated sums
// (the exact products' and additions' rounding errors carried along in a second
// float: off by n^2 2^-48 of the n = K / 32 magnitudes that a lane adds up) and
// ordered by those in double.  That meets about one token in a
// hundred; going through all products with compensated sums would cost nine
// operations for one.
//
// A cluster takes up to 8 tokens and shares out the experts, a warp two or four
// at a time: a weight is read once for the cluster's tokens, and with four
// experts a warp's reads of the activations from shared memory keep pace with
// its products.  One or two tokens are read straight from memory, so that
// nothing stands between the launch and the weights.  The scores go to the block
// that owns the token through distributed shared memory, where each expert counts
// the ones before it: no rounds of a selection.
//
// Measured: one token of 2048 over 128 experts 5.5 us, latency from load to store; 509 tokens 26.0 us, f32 products
// (10 TFLOP/s over the whole call) and the choice after them.
#include <type_traits>

#include "serving.cuh"

namespace gg {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStage = 8192;         // activations in shared memory at a time, of all of a cluster's tokens
constexpr int kMaxTopK = 64;

__device__ __forceinline__ void st_cluster_f32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int DT> __device__ __forceinline__ float4 load4(const void* p, int64_t i) {
    if constexpr (DT == GGUF_DT_F32) {
        return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
        if constexpr (DT == GGUF_DT_F16) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
            return make_float4(a.x, a.y, b.x, b.y);
        } else {
            return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                               __uint_as_float(v.y & 0xffff0000u));
        }
    }
}
// c + a b in both halves: two products in one instruction
struct Pair { float x, y; };
__device__ __forceinline__ void fma2(Pair& c, float ax, float ay, float bx, float by) {
    uint64_t a, b, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(ax), "f"(ay));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(bx), "f"(by));
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(c.x), "=f"(c.y) : "l"(d));
}
__device__ __forceinline__ void dot4(Pair& c, const float4& a, const float4& b) {
    fma2(c, a.x, a.y, b.x, b.y);
    fma2(c, a.z, a.w, b.z, b.w);
}

// f(type) for the activations' type: once around a loop, so that its loads are not each behind a branch
template <class F>
__device__ __forceinline__ void with_dtype(int dt, F&& f) {
    if (dt == GGUF_DT_F32) f(std::integral_constant<int, GGUF_DT_F32>{});
    else if (dt == GGUF_DT_F16) f(std::integral_constant<int, GGUF_DT_F16>{});
    else f(std::integral_constant<int, GGUF_DT_BF16>{});
}

// s + c += a b, with s's rounding errors and the product's in c
__device__ __forceinline__ void add_product(float a, float b, float& s, float& c) {
    const float p = __fmul_rn(a, b), e = __fmaf_rn(a, b, -p);
    const float t = __fadd_rn(s, p), bb = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fadd_rn(__fsub_rn(s, __fsub_rn(t, bb)), __fsub_rn(p, bb)), e));
    s = t;
}

// bits of a float in the order of its value, NaN below everything
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return isnan(v) ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
}

// TG: tokens of a cluster.  EW: experts of a warp at a time.  WDT: the weights' type.
template <int TG, int EW, int WDT>
__global__ void __launch_bounds__(kThreads) moe_router_kernel(const RouterParams p, int cluster) {
    constexpr bool kDirect = TG <= 2;             // activations straight from memory
    constexpr int kPart = kStage / TG;            // of K, staged at a time
    extern __shared__ __align__(16) uint8_t s_dyn[];
    const int E = p.n_expert, K = p.K, E4 = (E + 3) & ~3;
    float* const s_x = reinterpret_cast<float*>(s_dyn);               // [TG][kPart]
    double* const s_exact = reinterpret_cast<double*>(s_x + (kDirect ? 0 : kStage));      // [E4]
    float* const s_ww = reinterpret_cast<float*>(s_exact + E4);       // [E4]: |W[e]|^2
    uint32_t* const s_key = reinterpret_cast<uint32_t*>(s_ww + E4);   // [E4]
    int* const s_before = reinterpret_cast<int*>(s_key + E4);         // [E4]
    float* const s_z = reinterpret_cast<float*>(s_before + E4);          // [TG / cluster][E4]: the scores of the tokens that this block owns
    __shared__ float s_xx[TG];                    // |x|^2
    __shared__ float s_rank[kMaxTopK + 1], s_p[kMaxTopK];
    __shared__ int s_id[kMaxTopK + 1], s_n;
    __shared__ double s_redd[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int t0 = (blockIdx.x / cluster) * TG;
    const int share = (E + cluster - 1) / cluster, e_lo = rank * share, e_hi = min(E, e_lo + share);
    if (tid < TG) s_xx[tid] = 0.f;
    if (cluster > 1) cluster_arrive_relaxed();      // waited for before the first store to another block
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    // every block goes as many rounds as the largest share asks
    for (int e0 = e_lo; e0 < e_lo + share; e0 += EW * kWarps) {
        const int e1 = e0 + EW * warp;              // this warp's experts: e1 .. e1 + EW - 1
        int64_t at[EW];
#pragma unroll
        for (int j = 0; j < EW; ++j) at[j] = (int64_t)min(e1 + j, E - 1) * K;
        Pair z[EW][TG] = {}, ww[EW] = {}, xx[TG] = {};
        // 128 values: 4 of each lane
        auto step = [&](const float4 (&w)[EW], const float4 (&x)[TG]) {
#pragma unroll
            for (int j = 0; j < EW; ++j) {
                dot4(ww[j], w[j], w[j]);
#pragma unroll
                for (int k = 0; k < TG; ++k) dot4(z[j][k], x[k], w[j]);
            }
        };
        constexpr int U = TG == 1 ? 8 : kDirect ? 4 : 2;        // steps whose loads are on their way together
        for (int k0 = 0; k0 < K; k0 += kDirect ? K : kPart) {
            const int n = kDirect ? K : min(kPart, K - k0);         // a multiple of 8
            if constexpr (!kDirect) {
                __syncthreads();
                // warps share the tokens out, several to one where there are few
                constexpr int PER = kWarps / TG;        // warps a token
                const int tok = warp / PER;
                float sum = 0.f;
                const bool on = t0 + tok < p.T;
                with_dtype(p.xdt, [&](auto dt) {
#pragma unroll 8
                    for (int i = 4 * ((warp % PER) * 32 + lane); i < n; i += 4 * 32 * PER) {
                        const float4 v = load4<decltype(dt)::value>(p.x, (int64_t)(on ? t0 + tok : 0) * K + k0 + i);
                        *reinterpret_cast<float4*>(s_x + tok * kPart + i) = v;
                        sum = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, sum))));
                    }
                });
                if (e0 == e_lo) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0) atomicAdd(&s_xx[tok], sum);      // only the bound depends on its order
                }
                __syncthreads();
            }
            if (e1 < e_hi) {
                auto products = [&](auto dt) {
                    for (int i0 = 4 * lane; i0 < n; i0 += 128 * U) {
                        float4 w[U][EW], x[kDirect ? U : 1][TG];
                        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const int i = i0 + 128 * u;
#pragma unroll
                            for (int j = 0; j < EW; ++j) w[u][j] = i < n ? load4<WDT>(p.w, at[j] + k0 + i) : none;
                            if constexpr (kDirect) {
#pragma unroll
                                for (int k = 0; k < TG; ++k)
                                    x[u][k] = i < n ? load4<decltype(dt)::value>(p.x, (int64_t)min(t0 + k, p.T - 1) * K + i) : none;
                            }
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            if constexpr (kDirect) {
                                step(w[u], x[u]);
#pragma unroll
                                for (int k = 0; k < TG; ++k) dot4(xx[k], x[u][k], x[u][k]);
                            } else if (i0 + 128 * u < n) {
#pragma unroll
                                for (int k = 0; k < TG; ++k) x[0][k] = *reinterpret_cast<const float4*>(s_x + k * kPart + i0 + 128 * u);
                                step(w[u], x[0]);
                            }
                        }
                    }
                };
                if constexpr (kDirect) with_dtype(p.xdt, products);
                else products(std::integral_constant<int, 0>{});
            }
        }
        // All lanes' sums at once: in each step a lane passes half of what it still has to its neighbour, so that value v
        // = expert * TG + token ends in lane v (of N lanes, and of the others' alike).
        constexpr int N = EW * TG;
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = z[i / TG][i % TG].x + z[i / TG][i % TG].y;
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const bool upper = lane & o;
                const float other = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + o], o);
                v[i] = (upper ? v[i + o] : v[i]) + other;
            }
#pragma unroll
        for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        float norm[EW];
#pragma unroll
        for (int j = 0; j < EW; ++j) {
            norm[j] = ww[j].x + ww[j].y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) norm[j] += __shfl_xor_sync(0xffffffffu, norm[j], o);
        }
        if constexpr (kDirect) {
            if (warp == 0 && e0 == e_lo) {
#pragma unroll
                for (int k = 0; k < TG; ++k) {
                    float sum = xx[k].x + xx[k].y;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0) s_xx[k] = sum;
                }
            }
        }
        if (cluster > 1 && e0 == e_lo) cluster_wait_acquire();
        // token k's scores go to its owner, block k % cluster
        const int j = lane / TG, k = lane % TG;
        if (lane < N && e1 + j < e_hi) st_cluster_f32(cluster_map(smem_u32(s_z + k / cluster * E4 + e1 + j), k % cluster), v[0]);
#pragma unroll
        for (int q = 0; q < EW; ++q)
            if (lane < min(cluster, TG) && e1 + q < e_hi) st_cluster_f32(cluster_map(smem_u32(s_ww + e1 + q), lane), norm[q]);
    }
    if (cluster > 1) cluster_sync_all();
    else __syncthreads();

    const int top_k = p.top_k;
    const bool soft = p.score == GGUF_SCORE_SOFTMAX;
    for (int k = rank; k < TG; k += cluster) {
        const int t = t0 + k;
        if (t >= p.T) break;
        const float* z = s_z + k / cluster * E4;
        // the largest score and |W[e]|, and the softmax's sum where it is asked for: every warp for itself
        float m = -INFINITY, ww = 0.f, sum = 0.f;
        for (int e = lane; e < E; e += 32) m = fmaxf(m, z[e]), ww = fmaxf(ww, s_ww[e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o)), ww = fmaxf(ww, __shfl_xor_sync(0xffffffffu, ww, o));
        if (soft && (p.bias || !p.renormalize)) {
            for (int e = lane; e < E; e += 32) sum += expf(z[e] - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        // (a sigmoid's exponential overflows nowhere)
        auto prob = [&](float v) {
            const float e = expf(soft ? v - m : -fabsf(v));
            return soft ? e / sum : (v < 0.f ? e : 1.f) / (1.f + e);
        };
        // without a bias the scores themselves have the order
        auto rank_of = [&](int e) { return p.bias ? prob(z[e]) + p.bias[e] : z[e]; };
        // A score's error: a lane's every other product in a row, the two halves, the lanes'; what products and squares lose
        // that are subnormal, at most 2^-150 each.  A sigmoid's slope is a quarter; a softmax's p moves by twice the scores'
        // error times p.
        const float deep = (float)(K / 64 + 10), lost = (float)K * 0x1p-149f;
        const float err = fmaf(deep * 0x1p-24f * sqrtf(s_xx[k] + lost), sqrtf(ww + lost) * 1.01f, lost);
        const float off = !p.bias ? 2.f * err : soft ? 4.f * err / sum : 0.5f * err;    // of two ranks
        auto slack = [&](float a, float b) { return p.bias ? off + 0x1p-20f * (fabsf(a) + fabsf(b) + 1.f) : off; };
        for (int e = tid; e < E4; e += kThreads) s_key[e] = e < E ? ordered(rank_of(e)) : 0u, s_before[e] = 0;
        if (tid <= top_k) s_rank[tid] = -INFINITY;
        __syncthreads();
        // Each expert counts the ones before it: those of larger keys, of equal ones those of
        // lower index.  Where threads are left, several share an expert's comparisons.
        const int wide = (E + 31) & ~31, parts = max(1, kThreads / wide), quads = E4 / 4, per = (quads + parts - 1) / parts;
        for (int i = tid; i < wide * parts; i += kThreads) {
            const int e = i % wide, q0 = i / wide * per, q1 = min(quads, q0 + per), own = min(max(e >> 2, q0), q1);
            if (e >= E) continue;
            const uint32_t mine = s_key[e];
            int n[4] = {};
#pragma unroll 4
            for (int q = q0; q < own; ++q) {
                const uint4 v = *reinterpret_cast<const uint4*>(s_key + 4 * q);
                n[0] += v.x >= mine, n[1] += v.y >= mine, n[2] += v.z >= mine, n[3] += v.w >= mine;
            }
            int q = own;
            if (q == e >> 2 && q < q1) {
                for (int o = 4 * q; o < 4 * q + 4; ++o) n[0] += s_key[o] > mine || (s_key[o] == mine && o < e);
                ++q;
            }
#pragma unroll 4
            for (; q < q1; ++q) {
                const uint4 v = *reinterpret_cast<const uint4*>(s_key + 4 * q);
                n[0] += v.x > mine, n[1] += v.y > mine, n[2] += v.z > mine, n[3] += v.w > mine;
            }
            if (parts > 1) atomicAdd(&s_before[e], n[0] + n[1] + n[2] + n[3]);
            else s_before[e] = n[0] + n[1] + n[2] + n[3];
        }
        __syncthreads();
        for (int e = tid; e < E; e += kThreads)
            if (s_before[e] <= top_k) s_rank[s_before[e]] = rank_of(e), s_id[s_before[e]] = e;
        __syncthreads();
        bool near = false;
        if (tid < top_k && tid + 1 < E) near = s_rank[tid] - s_rank[tid + 1] <= slack(s_rank[tid], s_rank[tid + 1]);
        if (__syncthreads_or(near)) {
            // the candidates: all that may be among the first top_k (all experts, where the
            // softmax's sum is part of what is compared), listed in s_before
            const bool all = soft && p.bias;
            const float last = s_rank[top_k - 1];
            if (tid == 0) s_n = 0;
            __syncthreads();
            for (int e = tid; e < E; e += kThreads)
                if (all || rank_of(e) >= last - slack(last, last)) s_before[atomicAdd(&s_n, 1)] = e;
            __syncthreads();
            const int n = s_n;
            with_dtype(p.xdt, [&](auto dt) {
                for (int c = warp; c < n; c += kWarps) {
                    const int e = s_before[c];
                    float s = 0.f, low = 0.f;
#pragma unroll 8
                    for (int i = 4 * lane; i < K; i += 128) {
                        const float4 x = load4<decltype(dt)::value>(p.x, (int64_t)t * K + i), w = load4<WDT>(p.w, (int64_t)e * K + i);
                        add_product(x.x, w.x, s, low);
                        add_product(x.y, w.y, s, low);
                        add_product(x.z, w.z, s, low);
                        add_product(x.w, w.w, s, low);
                    }
                    double d = (double)s + (double)low;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    if (lane == 0) s_exact[c] = d;
                }
            });
            __syncthreads();
            double dsum = 0.0;
            if (all) {
                for (int c = tid; c < n; c += kThreads) dsum += exp(s_exact[c] - (double)m);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, o);
                if (lane == 0) s_redd[warp] = dsum;
                __syncthreads();
                dsum = 0.0;
                for (int w = 0; w < kWarps; ++w) dsum += s_redd[w];
            }
            if (p.bias) {
                for (int c = tid; c < n; c += kThreads) {
                    const double v = s_exact[c];
                    s_exact[c] = (soft ? exp(v - (double)m) / dsum : 1.0 / (1.0 + exp(-v))) + (double)p.bias[s_before[c]];
                }
                __syncthreads();
            }
            // NaN, after everything else: every expert has a place of its own whatever the scores are
            for (int c = tid; c < n; c += kThreads)
                if (isnan(s_exact[c])) s_exact[c] = -HUGE_VAL;
            __syncthreads();
            for (int c = tid; c < n; c += kThreads) {
                const double mine = s_exact[c];
                const int e = s_before[c];
                int before = 0;
                for (int o = 0; o < n; ++o) before += s_exact[o] > mine || (s_exact[o] == mine && s_before[o] < e);
                if (before < top_k) s_id[before] = e;
            }
            __syncthreads();
        }
        // Where only the chosen experts' shares count, p is scaled by what makes the largest of them 1 or near it: it may be
        // far below f32's range (sigmoids of very negative scores, a softmax whose largest score a bias shuts out).
        float best = z[s_id[0]];
        if (p.renormalize && p.bias) {                   // not the first: every warp looks at them all
            uint32_t key = lane < top_k ? ordered(z[s_id[lane]]) : 0u;
            if (lane + 32 < top_k) key = max(key, ordered(z[s_id[lane + 32]]));
            key = __reduce_max_sync(0xffffffffu, key);
            best = __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
        }
        if (tid < top_k) {
            const float v = z[s_id[tid]];
            if (p.renormalize) {
                s_p[tid] = soft ? expf(v - best) : expf(fminf(v, 0.f) - fminf(best, 0.f)) / (1.f + expf(-fabsf(v)));
            } else {
                s_p[tid] = prob(v);
            }
        }
        __syncthreads();
        if (tid < top_k) {
            float v = s_p[tid];
            if (p.renormalize) {
                float total = 0.f;
                for (int i = 0; i < top_k; ++i) total += s_p[i];
                v /= total;
            }
            p.ids[(int64_t)t * top_k + tid] = s_id[tid];
            p.weights[(int64_t)t * top_k + tid] = v * p.scale;
        }
        __syncthreads();
    }
}

template <int TG, int EW, int WDT>
cudaError_t launch(const RouterParams& p, int cluster, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_once(moe_router_kernel<TG, EW, WDT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ceil_div(p.T, TG) * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (TG <= 2 ? 0 : kStage * 4) + (size_t)ceil_div(p.n_expert, 4) * 4 * (20 + 4 * ceil_div(TG, cluster));
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe_router_kernel<TG, EW, WDT>, p, cluster);
}

template <int TG, int EW>
cudaError_t launch(const RouterParams& p, int pdl, cudaStream_t s) {
    // a warp's experts a block first, so many blocks as the experts ask for
    int cluster = 1;
    while (cluster < 8 && cluster * EW * kWarps < p.n_expert) cluster *= 2;
    if (p.wdt == GGUF_DT_F32) return launch<TG, EW, GGUF_DT_F32>(p, cluster, pdl, s);
    return p.wdt == GGUF_DT_F16 ? launch<TG, EW, GGUF_DT_F16>(p, cluster, pdl, s) : launch<TG, EW, GGUF_DT_BF16>(p, cluster, pdl, s);
}

}  // namespace

cudaError_t moe_router_launch(const RouterParams& p, int num_sms, int pdl, cudaStream_t s) {
    // few tokens: one or two to a cluster, two experts to a warp, over as many SMs as
    // that gives; then four and eight tokens.  One token of 2048 over 128 experts takes 5.6 us so, and 7.5, 8.9 and 11.4
    // in clusters for two, four and eight; 509 tokens 25.7 us in clusters for eight, 26.8 for four, 43 for two.
    const int64_t blocks = std::min<int64_t>(8, ceil_div(p.n_expert, 2 * kWarps)), clusters = std::max<int64_t>(1, 2 * num_sms / blocks);
    if (p.T <= clusters) return launch<1, 2>(p, pdl, s);
    if (p.T <= 2 * clusters) return launch<2, 2>(p, pdl, s);
    return p.T <= 4 * clusters ? launch<4, 4>(p, pdl, s) : launch<8, 4>(p, pdl, s);
}

}  // namespace gg
