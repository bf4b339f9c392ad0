// Attention of new tokens over a paged key/value cache.
//
//   out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),  s_j = scale * q . K_j,
// with m the running maximum of the scores seen so far: when it grows, what
// has been summed is multiplied by exp(old m - new m), so one pass over the
// keys is enough.
#include "attn.cuh"
#include "tc_gemm.cuh"

namespace gg {

namespace {

constexpr int kWarps = 8;

template <class T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// One warp to a (token, head): the lanes hold the head's values, d = lane + 32 i.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) attn_rows_kernel(const AttnParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(row / p.heads), h = (int)(row % p.heads);
    if (t >= p.b.n_tokens) return;
    int seq = -1;
    for (int i = lane; i < p.b.n_seq; i += 32)
        if (p.b.q_start[i] <= t && t < p.b.q_start[i + 1]) seq = i;
    seq = __reduce_max_sync(0xffffffffu, seq);
    if (seq < 0) return;
    const int len = p.b.kv_len[seq], pos = len - p.b.q_start[seq + 1] + t;
    int hi = p.causal ? min(len, pos + 1) : len;
    const int lo = p.window ? (int)max((int64_t)0, pos - p.window + 1) : 0;
    if (hi > p.b.pages_stride << p.c.page_shift) {
        hi = (int)(p.b.pages_stride << p.c.page_shift);
        if (lane == 0) report(p.status, GGUF_ERR_INVALID_ARG);
    }
    const int D = p.c.dim;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
    const T* qr = static_cast<const T*>(p.q) + t * p.ldq + h * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = lane + 32 * i < D ? to_f(qr[lane + 32 * i]) * p.scale : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int j = lo; j < hi; ++j) {
        const int page = p.b.pages[seq * p.b.pages_stride + (j >> p.c.page_shift)];
        if ((unsigned)page >= (unsigned)p.c.n_pages) {
            if (lane == 0) report(p.status, GGUF_ERR_INVALID_ARG);
            break;
        }
        const int64_t at = page * p.c.page_stride + (h / p.group) * p.c.head_stride +
                           (j & ((1 << p.c.page_shift) - 1)) * p.c.token_stride;
        const T* k = static_cast<const T*>(p.c.k) + at;
        const T* v = static_cast<const T*>(p.c.v) + at;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < D) s += q[i] * to_f(k[lane + 32 * i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float top = fmaxf(m, s);
        const float old = m == -INFINITY ? 0.f : __expf(m - top), w = top == -INFINITY ? 0.f : __expf(s - top);
        l = l * old + w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < D) o[i] = o[i] * old + w * to_f(v[lane + 32 * i]);
        m = top;
    }
    T* out = static_cast<T*>(p.out) + t * p.ldo + h * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < D) out[lane + 32 * i] = from_f<T>(l > 0.f ? o[i] / l : 0.f);
    if (p.lse && lane == 0) p.lse[(int64_t)t * p.heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

// One warp to a row: joins the splits' partial sums, in their order.
template <class T>
__global__ void __launch_bounds__(32 * kWarps) attn_join_kernel(const AttnParams p, const Partials part) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)p.b.n_tokens * p.heads, row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(row / p.heads), h = (int)(row % p.heads), D = p.c.dim;
    if (row >= rows || t < p.b.q_start[0] || t >= p.b.q_start[p.b.n_seq]) return;
    float top = -INFINITY, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = lane; i < part.splits; i += 32) top = fmaxf(top, part.ml[i * rows + row].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    for (int i = 0; i < part.splits; ++i) {
        const float2 ml = part.ml[i * rows + row];
        if (ml.x == -INFINITY) continue;
        const float f = exp2_fast(ml.x - top);
        sum += f * ml.y;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < D) o[k] += f * part.o[(i * rows + row) * D + lane + 32 * k];
    }
    T* out = static_cast<T*>(p.out) + t * p.ldo + h * D;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < D) out[lane + 32 * k] = from_f<T>(sum > 0.f ? o[k] / sum : (sum == 0.f ? 0.f : sum));
    if (p.lse && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
}

AttnPlan make_plan(const AttnParams& p, int num_sms) {
    AttnPlan a{};
    const int64_t rows = (int64_t)p.b.max_q * p.group;
    a.few = rows <= 64;
    a.tiles = (int)ceil_div(rows, 16);
    // keys in units of one chunk to each warp of a block
    int64_t span = p.b.max_kv;
    if (p.window && p.causal) span = std::min<int64_t>(span, p.window + p.b.max_q);
    const int64_t units = std::max<int64_t>(1, ceil_div(span, 64)), pairs = (int64_t)p.b.n_seq * p.c.kv_heads * a.tiles;
    // two blocks to an SM; sequences of different lengths in shares of about a thousand keys
    int64_t want = std::max(ceil_div(2 * num_sms, pairs), std::min<int64_t>(16, ceil_div(units, 16)));
    want = std::min(want, units);
    a.cluster = 1;
    while (a.cluster < 16 && a.cluster < want) a.cluster *= 2;
    a.splits = (int)ceil_div(want, a.cluster);
    return a;
}

}  // namespace

int make_kv_map(CUtensorMap* map, const void* base, const CacheParams& c, int rows) {
    const uint64_t dims[4] = {(uint64_t)c.dim, uint64_t(1) << c.page_shift, (uint64_t)c.kv_heads, (uint64_t)c.n_pages};
    const uint64_t strides[3] = {(uint64_t)c.token_stride * 2, (uint64_t)c.head_stride * 2, (uint64_t)c.page_stride * 2};
    const uint32_t box[4] = {64, (uint32_t)rows, 1, 1};
    return make_tmap(map, base, c.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t paged_attn_workspace_bytes(const AttnParams& p, int num_sms) {
    const AttnPlan a = make_plan(p, num_sms);
    if (!a.few || a.splits <= 1) return 0;
    return (size_t)a.splits * p.b.n_tokens * p.heads * (p.c.dim * 4 + 8);
}

int paged_attn_launch(const AttnParams& p, void* workspace, int num_sms, int pdl, cudaStream_t s) {
    const AttnPlan a = make_plan(p, num_sms);
    if (a.few) {
        const int64_t rows = (int64_t)p.b.n_tokens * p.heads;
        Partials part{static_cast<float*>(workspace), nullptr, a.splits};
        part.ml = reinterpret_cast<float2*>(part.o + (int64_t)a.splits * rows * p.c.dim);
        const int st = attn_few_launch(p, a, part, pdl, s);
        if (st != GGUF_OK || a.splits == 1) return st;
        const dim3 grid((unsigned)ceil_div(rows, kWarps));
        const cudaError_t e = p.c.bf16 ? launch_pdl(attn_join_kernel<__nv_bfloat16>, grid, dim3(32 * kWarps), 0, s, pdl, p, part)
                                       : launch_pdl(attn_join_kernel<__half>, grid, dim3(32 * kWarps), 0, s, pdl, p, part);
        return e == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
    }
    const dim3 grid((unsigned)ceil_div((int64_t)p.b.n_tokens * p.heads, kWarps));
    const cudaError_t e = p.c.bf16 ? launch_pdl(attn_rows_kernel<__nv_bfloat16>, grid, dim3(32 * kWarps), 0, s, pdl, p)
                                   : launch_pdl(attn_rows_kernel<__half>, grid, dim3(32 * kWarps), 0, s, pdl, p);
    return e == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

}  // namespace gg
