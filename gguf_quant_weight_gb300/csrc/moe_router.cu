// The router of a mixture of experts: scores, the best top_k of them, their
// weights, in one kernel.
//   z[t][e] = x[t] . W[e];   p = softmax(z[t]) or sigmoid(z[t]);
//   the top_k experts of the largest p (+ bias), the lower index first among
//   equals;  weights p of those, divided by their sum if asked, times scale.
//
// Which experts a token takes is decided exactly.  The products are summed in
// f32, whose error is at most n 2^-24 |x| |W[e]| (n additions deep, norms by
// Cauchy and Schwarz).  Where two neighbours in the order lie closer than that
// allows, the scores of the experts that could be among the first top_k are
// computed again with compensated sums (the exact products' and additions'
// rounding errors carried along, as good as twice the digits) and ordered by
// those in double.  That meets about one token in sixty; going through all products with
// compensated sums would cost nine operations for one.
//
// A cluster takes up to 8 tokens and shares out the experts, a warp two at a
// time: a weight is read once for the cluster's tokens.  The scores go
// to the block that owns the token through distributed shared memory, where each expert
// counts the ones before it -- E comparisons a thread and no rounds of a
// selection.
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
__device__ __forceinline__ float4 load4(const void* p, int dt, int64_t i) {
    return dt == GGUF_DT_F32 ? load4<GGUF_DT_F32>(p, i) : dt == GGUF_DT_F16 ? load4<GGUF_DT_F16>(p, i) : load4<GGUF_DT_BF16>(p, i);
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

// TG: tokens of a cluster.  WDT: the weights' type.
template <int TG, int WDT>
__global__ void __launch_bounds__(kThreads) moe_router_kernel(const RouterParams p, int cluster) {
    constexpr int kPart = kStage / TG;            // of K
    extern __shared__ __align__(16) uint8_t s_dyn[];
    const int E = p.n_expert, K = p.K;
    float* const s_x = reinterpret_cast<float*>(s_dyn);               // [TG][kPart]
    double* const s_exact = reinterpret_cast<double*>(s_x + kStage);  // [E]
    float* const s_ww = reinterpret_cast<float*>(s_exact + E);        // [E]: |W[e]|^2
    uint32_t* const s_key = reinterpret_cast<uint32_t*>(s_ww + E);    // [E]
    float* const s_z = reinterpret_cast<float*>(s_key + E);           // [TG / cluster][E]: the scores of the tokens that this block owns
    __shared__ float s_xx[TG];                    // |x|^2
    __shared__ float s_rank[kMaxTopK + 1], s_p[kMaxTopK];
    __shared__ int s_id[kMaxTopK + 1];
    __shared__ int s_near;
    __shared__ float s_red[kWarps];
    __shared__ double s_redd[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int t0 = (blockIdx.x / cluster) * TG;
    const int share = (E + cluster - 1) / cluster, e_lo = rank * share, e_hi = min(E, e_lo + share);
    if (tid < TG) s_xx[tid] = 0.f;
    if (cluster > 1) cluster_arrive_relaxed();      // waited for before the first store to another block
    pdl_wait();
    pdl_launch_dependents();

    // every block goes as many rounds as the largest share asks
    for (int e0 = e_lo; e0 < e_lo + share; e0 += 2 * kWarps) {
        const int ea = e0 + 2 * warp, eb = ea + 1;
        const bool on_a = ea < e_hi, on_b = eb < e_hi;
        const int64_t wa = (int64_t)(on_a ? ea : 0) * K, wb = (int64_t)(on_b ? eb : 0) * K;
        float za[TG] = {}, zb[TG] = {}, wwa = 0.f, wwb = 0.f;
        for (int k0 = 0; k0 < K; k0 += kPart) {
            const int n = min(kPart, K - k0);       // a multiple of 8
            __syncthreads();
            // warps share the tokens out, several to one where there are few
            constexpr int PER = kWarps / TG;        // warps a token
            const int tok = warp / PER;
            float xx = 0.f;
            for (int i = 4 * ((warp % PER) * 32 + lane); i < n; i += 4 * 32 * PER) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t0 + tok < p.T) v = load4(p.x, p.xdt, (int64_t)(t0 + tok) * K + k0 + i);
                *reinterpret_cast<float4*>(s_x + tok * kPart + i) = v;
                xx = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, xx))));
            }
            if (e0 == e_lo) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) xx += __shfl_xor_sync(0xffffffffu, xx, o);
                if (lane == 0) atomicAdd(&s_xx[tok], xx);       // only the bound depends on its order
            }
            __syncthreads();
            if (on_a) {
#pragma unroll 4
                for (int i = 4 * lane; i < n; i += 128) {
                    const float4 a = load4<WDT>(p.w, wa + k0 + i), b = load4<WDT>(p.w, wb + k0 + i);
                    wwa = fmaf(a.x, a.x, fmaf(a.y, a.y, fmaf(a.z, a.z, fmaf(a.w, a.w, wwa))));
                    wwb = fmaf(b.x, b.x, fmaf(b.y, b.y, fmaf(b.z, b.z, fmaf(b.w, b.w, wwb))));
#pragma unroll
                    for (int k = 0; k < TG; ++k) {
                        const float4 x = *reinterpret_cast<const float4*>(s_x + k * kPart + i);
                        za[k] = fmaf(x.x, a.x, fmaf(x.y, a.y, fmaf(x.z, a.z, fmaf(x.w, a.w, za[k]))));
                        zb[k] = fmaf(x.x, b.x, fmaf(x.y, b.y, fmaf(x.z, b.z, fmaf(x.w, b.w, zb[k]))));
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            wwa += __shfl_xor_sync(0xffffffffu, wwa, o), wwb += __shfl_xor_sync(0xffffffffu, wwb, o);
#pragma unroll
            for (int k = 0; k < TG; ++k)
                za[k] += __shfl_xor_sync(0xffffffffu, za[k], o), zb[k] += __shfl_xor_sync(0xffffffffu, zb[k], o);
        }
        if (cluster > 1 && e0 == e_lo) cluster_wait_acquire();
        // lane 2k (2k + 1) sends token k's score of the first (second) expert to the token's owner, block k % cluster
#pragma unroll
        for (int k = 0; k < TG; ++k) {
            if (lane == 2 * k && on_a) st_cluster_f32(cluster_map(smem_u32(s_z + k / cluster * E + ea), k % cluster), za[k]);
            if (lane == 2 * k + 1 && on_b) st_cluster_f32(cluster_map(smem_u32(s_z + k / cluster * E + eb), k % cluster), zb[k]);
        }
        for (int r = 0; r < min(cluster, TG); ++r) {
            if (lane == 2 * r && on_a) st_cluster_f32(cluster_map(smem_u32(&s_ww[ea]), r), wwa);
            if (lane == 2 * r + 1 && on_b) st_cluster_f32(cluster_map(smem_u32(&s_ww[eb]), r), wwb);
        }
    }
    if (cluster > 1) cluster_sync_all();
    else __syncthreads();

    const int top_k = p.top_k;
    for (int k = rank; k < TG; k += cluster) {
        const int t = t0 + k;
        if (t >= p.T) break;
        const float* z = s_z + k / cluster * E;
        // max and, for the softmax, sum; the largest |W[e]|
        auto block_max = [&](float v) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            __syncthreads();
            if (lane == 0) s_red[warp] = v;
            __syncthreads();
            v = s_red[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v = fmaxf(v, s_red[w]);
            return v;
        };
        float m = -INFINITY, ww = 0.f, sum = 0.f;
        for (int e = tid; e < E; e += kThreads) m = fmaxf(m, z[e]), ww = fmaxf(ww, s_ww[e]);
        m = block_max(m);
        ww = block_max(ww);
        const bool soft = p.score == GGUF_SCORE_SOFTMAX;
        if (soft) {
            for (int e = tid; e < E; e += kThreads) sum += expf(z[e] - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            __syncthreads();
            if (lane == 0) s_red[warp] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_red[w];
        }
        auto prob = [&](float v) { return soft ? expf(v - m) / sum : 1.f / (1.f + expf(-v)); };
        // without a bias the scores themselves have the order
        auto rank_of = [&](int e) { return p.bias ? prob(z[e]) + p.bias[e] : z[e]; };
        // a rank's error: the sums' (K / 32 + 5 additions deep and a few for the products),
        // which a probability does not more than double, and that of expf and the addition
        const float err = ((float)(K / 32 + 12) * 0x1p-24f) * sqrtf(s_xx[k]) * sqrtf(ww) * 1.001f;
        if (tid == 0) s_near = 0;
        for (int e = tid; e < E; e += kThreads) s_key[e] = ordered(rank_of(e));
        if (tid <= top_k) s_rank[tid] = -INFINITY;
        __syncthreads();
        for (int e = tid; e < E; e += kThreads) {
            const uint32_t mine = s_key[e];
            int before = 0;
            for (int o = 0; o < E; ++o) before += s_key[o] > mine || (s_key[o] == mine && o < e);
            if (before <= top_k) s_rank[before] = rank_of(e), s_id[before] = e;
        }
        __syncthreads();
        if (tid < top_k && tid + 1 < E) {
            const float a = s_rank[tid], b = s_rank[tid + 1];
            const float slack = p.bias ? 4.f * err + 0x1p-20f * (fabsf(a) + fabsf(b) + 1.f) : 2.f * err;
            if (a - b <= slack) s_near = 1;
        }
        __syncthreads();
        if (s_near) {
            // the candidates: all that may be among the first top_k (all experts, where the
            // softmax's sum is part of what is compared)
            const bool all = soft && p.bias;
            const float last = s_rank[top_k - 1];
            const float slack = p.bias ? 4.f * err + 0x1p-20f * (2.f * fabsf(last) + 1.f) : 2.f * err;
            auto candidate = [&](int e) { return all || rank_of(e) >= last - slack; };
            for (int e = warp; e < E; e += kWarps) {
                if (!candidate(e)) continue;
                float s = 0.f, c = 0.f;
                for (int i = 4 * lane; i < K; i += 128) {
                    const float4 x = load4(p.x, p.xdt, (int64_t)t * K + i), w = load4<WDT>(p.w, (int64_t)e * K + i);
                    add_product(x.x, w.x, s, c);
                    add_product(x.y, w.y, s, c);
                    add_product(x.z, w.z, s, c);
                    add_product(x.w, w.w, s, c);
                }
                double d = (double)s + (double)c;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                if (lane == 0) s_exact[e] = d;
            }
            __syncthreads();
            double dsum = 0.0;
            if (all) {
                for (int e = tid; e < E; e += kThreads) dsum += exp(s_exact[e] - (double)m);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, o);
                if (lane == 0) s_redd[warp] = dsum;
                __syncthreads();
                dsum = 0.0;
                for (int w = 0; w < kWarps; ++w) dsum += s_redd[w];
            }
            if (p.bias) {
                for (int e = tid; e < E; e += kThreads)
                    if (candidate(e)) {
                        const double v = s_exact[e];
                        s_exact[e] = (soft ? exp(v - (double)m) / dsum : 1.0 / (1.0 + exp(-v))) + (double)p.bias[e];
                    }
                __syncthreads();
            }
            for (int e = tid; e < E; e += kThreads) {
                if (!candidate(e)) continue;
                int before = 0;
                for (int o = 0; o < E; ++o)
                    if (candidate(o)) before += s_exact[o] > s_exact[e] || (s_exact[o] == s_exact[e] && o < e);
                if (before < top_k) s_id[before] = e;
            }
            __syncthreads();
        }
        if (tid < top_k) s_p[tid] = prob(z[s_id[tid]]);
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

template <int TG, int WDT>
cudaError_t launch(const RouterParams& p, int cluster, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_once(moe_router_kernel<TG, WDT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ceil_div(p.T, TG) * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kStage * 4 + (size_t)p.n_expert * (16 + 4 * ceil_div(TG, cluster));
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe_router_kernel<TG, WDT>, p, cluster);
}

template <int TG>
cudaError_t launch(const RouterParams& p, int cluster, int pdl, cudaStream_t s) {
    if (p.wdt == GGUF_DT_F32) return launch<TG, GGUF_DT_F32>(p, cluster, pdl, s);
    return p.wdt == GGUF_DT_F16 ? launch<TG, GGUF_DT_F16>(p, cluster, pdl, s) : launch<TG, GGUF_DT_BF16>(p, cluster, pdl, s);
}

}  // namespace

cudaError_t moe_router_launch(const RouterParams& p, int num_sms, int pdl, cudaStream_t s) {
    // a warp's two experts a block first, then as many tokens a cluster as keep the SMs busy
    int cluster = 1;
    while (cluster < 8 && cluster * 2 * kWarps < p.n_expert) cluster *= 2;
    const int64_t clusters = std::max(1, num_sms / cluster);
    if (p.T <= clusters) return launch<1>(p, cluster, pdl, s);
    if (p.T <= 2 * clusters) return launch<2>(p, cluster, pdl, s);
    return p.T <= 4 * clusters ? launch<4>(p, cluster, pdl, s) : launch<8>(p, cluster, pdl, s);
}

}  // namespace gg
