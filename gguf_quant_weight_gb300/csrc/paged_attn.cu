// Attention of new tokens over a paged key/value cache: the form a call takes,
// its tensor maps, and the joining of split keys.
//
//   out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),  s_j = scale * q . K_j.
// With m the running maximum of the scores seen so far, multiplying what has
// been summed by exp(old m - new m) when it grows makes one pass over the keys
// enough, and partial results over disjoint keys join in the same way.
#include "attn.cuh"
#include "tc_gemm.cuh"

namespace gg {

namespace {

constexpr int kWarps = 8;
constexpr int kAtOnce = 8;

template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

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
    for (int i0 = 0; i0 < part.splits; i0 += kAtOnce) {        // so many splits' loads in flight
        float2 ml[kAtOnce];
        float v[kAtOnce][4];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            ml[j] = make_float2(-INFINITY, 0.f);
            if (i0 + j >= part.splits) continue;
            ml[j] = part.ml[(i0 + j) * rows + row];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[j][k] = lane + 32 * k < D ? part.o[((i0 + j) * rows + row) * D + lane + 32 * k] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (ml[j].y == 0.f) continue;                      // saw nothing (the maximum does not tell: it may pass over NaN)
            const float f = exp2_fast(ml[j].x - top);
            sum += f * ml[j].y;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] += f * v[j][k];
        }
    }
    T* out = static_cast<T*>(p.out) + t * p.ldo + h * D;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < D) out[lane + 32 * k] = from_f<T>(sum > 0.f ? o[k] / sum : (sum == 0.f ? 0.f : sum));
    if (p.lse && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
}

// Rows of a sequence up to which the few-rows form takes it.  Measured with 8 key
// heads of 128 (few rows / many rows, us): 16 rows over 500, 4000, 30000 keys 7.2 /
// 10.0, 11.8 / 15.4, 45 / 33; 32 rows 8.2 / 10.1, 21.8 / 15.9, 65 / 34.  Single
// tokens (4 rows) of 64 sequences 105 / 221, over 131071 keys 52 / 56.  The rule
// looks at rows alone, and is the wrong side for 16 rows over the longest histories.
constexpr int kFewRows = 16;
// Chunks of 16 keys from which a call deals its keys out to all warps and joins in
// a second kernel.  Clusters / dealt out, us: 16 sequences of 2000 keys (16128
// chunks) 26.8 / 32.3, 32 of 50..1000 20.2 / 23.4, 36 of 400 16.1 / 23.3, 2 of
// 16000 (16016) 39.2 / 35.0; dealt out, 64 of 100..8000 take 105 (up to 256512
// chunks), and 156 in clusters.  Few long sequences would change sides earlier.
constexpr int64_t kLineChunks = 16384;

// The form and the split of a call, from its sizes alone.
AttnPlan make_plan(const AttnParams& p, int num_sms) {
    AttnPlan a{};
    const int64_t rows = (int64_t)p.b.max_q * p.group;
    int64_t span = p.b.max_kv;                        // keys that a row tile may see
    if (p.window && p.causal) span = std::min<int64_t>(span, p.window + p.b.max_q);
    const int64_t chunks = std::max<int64_t>(1, ceil_div(span, 16));
    a.cluster = a.splits = 1;
    if (rows <= kFewRows) {
        a.few = rows <= 8 ? 8 : 16;
        const int64_t pairs = (int64_t)p.b.n_seq * p.c.kv_heads;
        if (pairs * chunks > kLineChunks) {
            a.blocks = 2 * num_sms;
        } else {
            // as many blocks as two to an SM can be at once, with a chunk to each warp
            const int64_t most = 2 * num_sms / pairs;
            while (a.cluster < 16 && 2 * a.cluster <= most && 4 * a.cluster < chunks) a.cluster *= 2;
        }
    } else {
        a.tiles = (int)ceil_div(p.b.max_q, many_tiles(p) * (128 / p.group));
        // the keys are split where the tiles alone leave SMs idle
        const int64_t units = std::max<int64_t>(1, ceil_div(span, 128)), pairs = (int64_t)p.b.n_seq * p.c.kv_heads * a.tiles;
        a.splits = (int)std::min(units, std::max<int64_t>(1, (3 - many_tiles(p)) * num_sms / pairs));
        // among several sequences some may have few rows
        a.mixed = p.b.n_seq > 1 && a.splits == 1 && p.group <= kFewRows;
        if (a.mixed) {
            a.few = 16;
            // About four thousand keys a block.  As the rule has it / 1 / 2 / 4 / 8 blocks,
            // us: 24 sequences of 1..500 tokens over 100..8000 keys 132 / 137 / 132 / 142 /
            // 133, over up to 1000 keys 50 / 50 / 52 / 54 / 61, 64 of 1..20 tokens over
            // 100..8000 keys 169 / 168 / 168 / 174 / 205; only 16 of 1..100 tokens over
            // 12000..16000 keys are served worse: 404 / 327 / 340 / 415 / 416.
            while (a.cluster < 8 && 256 * a.cluster < chunks) a.cluster *= 2;
        }
    }
    return a;
}

}  // namespace

int make_kv_map(CUtensorMap* map, const void* base, const CacheParams& c, int rows, int blocks) {
    const uint64_t dims[5] = {(uint64_t)(blocks > 1 ? 64 : c.dim), uint64_t(1) << c.page_shift, (uint64_t)blocks,
                              (uint64_t)c.kv_heads, (uint64_t)c.n_pages};
    const uint64_t strides[4] = {(uint64_t)c.token_stride * 2, 128, (uint64_t)c.head_stride * 2, (uint64_t)c.page_stride * 2};
    const uint32_t box[5] = {64, (uint32_t)rows, (uint32_t)blocks, 1, 1};
    return make_tmap(map, base, c.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

int make_q_map(CUtensorMap* map, const AttnParams& p, int heads, int tokens) {
    const uint64_t dims[3] = {(uint64_t)p.c.dim, (uint64_t)p.heads, (uint64_t)p.b.n_tokens};
    const uint64_t strides[2] = {(uint64_t)p.c.dim * 2, (uint64_t)p.ldq * 2};
    const uint32_t box[3] = {64, (uint32_t)heads, (uint32_t)tokens};
    return make_tmap(map, p.q, p.c.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t paged_attn_workspace_bytes(const AttnParams& p, int num_sms) {
    const AttnPlan a = make_plan(p, num_sms);
    if (a.blocks) return attn_line_bytes(p, a);
    return a.splits > 1 ? (size_t)a.splits * p.b.n_tokens * p.heads * (p.c.dim * 4 + 8) : 0;
}

int paged_attn_launch(const AttnParams& call, void* workspace, int num_sms, int pdl, cudaStream_t s) {
    AttnParams p = call;
    const AttnPlan a = make_plan(p, num_sms);
    if (a.tiles > 65535) return GGUF_ERR_UNSUPPORTED;   // a grid's limit
    p.few_rows = a.mixed ? kFewRows : a.few ? INT32_MAX : 0;
    if (a.few && !a.mixed) return attn_few_launch(p, a, workspace, pdl, s);
    const int64_t rows = (int64_t)p.b.n_tokens * p.heads;
    Partials part{static_cast<float*>(workspace), nullptr, a.splits};
    part.ml = reinterpret_cast<float2*>(part.o + (int64_t)a.splits * rows * p.c.dim);
    int st = GGUF_OK;
    if (a.mixed) st = attn_few_launch(p, a, workspace, pdl, s);
    if (st == GGUF_OK) st = attn_many_launch(p, a, part, pdl, s);
    if (st != GGUF_OK || a.splits == 1) return st;
    const dim3 grid((unsigned)ceil_div(rows, kWarps));
    const cudaError_t e = p.c.bf16 ? launch_pdl(attn_join_kernel<__nv_bfloat16>, grid, dim3(32 * kWarps), 0, s, pdl, p, part)
                                   : launch_pdl(attn_join_kernel<__half>, grid, dim3(32 * kWarps), 0, s, pdl, p, part);
    return e == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

}  // namespace gg
