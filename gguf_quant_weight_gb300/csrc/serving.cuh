// Parameters and host entry points of the serving kernels (kv_append.cu,
// paged_attn.cu, logits.cu, moe_router.cu, moe_ffn.cu, sample.cu); the C entry points and their checks are in
// serving.cu.
#pragma once
#include <atomic>

#include "common.cuh"

namespace gg {

// The batch's device arrays, as every kernel reads them.
struct BatchParams {
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* pages;
    int64_t pages_stride;
    int n_seq, n_tokens;
    int max_q, max_kv;
};

struct CacheParams {
    void* k;
    void* v;
    int64_t page_stride, head_stride, token_stride;  // elements
    int n_pages, kv_heads, dim;
    int page_shift;                                  // log2(page_size)
    int bf16;                                        // else f16
};

struct AppendParams {
    BatchParams b;
    CacheParams c;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv, ldqo;
    void* q_out;
    const float* freqs;
    const int32_t* positions;
    float rope_scale;
    int rot, style;
    int xdt, heads;          // heads = 0: no q
    const float *q_norm, *k_norm;    // the heads' norms [dim], null: none
    float eps;
    int* status;
};

struct AttnParams {
    BatchParams b;
    CacheParams c;
    const void* q;
    int64_t ldq;
    void* out;
    int64_t ldo;
    float* lse;
    int heads, group;        // group = heads / kv_heads
    float scale;
    int causal;
    int64_t window;          // 0: none
    int few_rows;            // sequences of up to so many rows (tokens x group) take the few-rows form
    int* status;
};

struct LogitsParams {
    const void* x;
    void* y;
    int64_t ld, ldo;
    int64_t vocab;
    int rows, dt, odt;
    gguf_logit_rules r;
};

struct RouterParams {
    const void* x;
    const void* w;
    const float* bias;
    int32_t* ids;
    float* weights;
    int T, K, n_expert, top_k;
    int xdt, wdt, score, renormalize;
    float scale;
};

constexpr int kMoeFfnRows = 512, kMoeFfnExperts = 1024;      // routed rows and experts at most

struct MoeFfnParams {
    const uint8_t *gate, *up, *down;
    int64_t gate_rb, up_rb, down_rb;     // bytes of a row
    int gate_type, up_type, down_type, act;
    int n_expert, T, top_k;
    int64_t K, F;
    const void* x;
    int xdt, ydt;
    const int32_t* ids;
    const float* weights;
    const void* residual;
    void* y;
    int* status;
    // set by the launch.  In the workspace: hidden values [T * top_k][F], then as
    // the down kernel's columns, the columns' scales, and what up makes of the ids
    float* h;
    uint8_t* columns;
    float* column_scales;
    uint8_t* routes;
    int x_parts, h_parts;                // columns that a row of x and of h takes
    int up_tiles, up_wp, up_stages, up_slot, up_resident;
    int down_stages, splits;
};

struct SampleParams {
    const void* x;
    int64_t ld;
    int rows, vocab, dt;
    gguf_sampler s;
    const float* u;
    int32_t* token;
    float* logprob;
};

cudaError_t kv_append_launch(const AppendParams& p, int num_sms, int pdl, cudaStream_t stream);
size_t paged_attn_workspace_bytes(const AttnParams& p, int num_sms);
int paged_attn_launch(const AttnParams& p, void* workspace, int num_sms, int pdl, cudaStream_t stream);
cudaError_t logits_adjust_launch(const LogitsParams& p, int num_sms, int pdl, cudaStream_t stream);
cudaError_t moe_router_launch(const RouterParams& p, int num_sms, int pdl, cudaStream_t stream);
size_t moe_ffn_workspace_bytes(int64_t F, int64_t T, int64_t top_k);
int moe_ffn_launch(MoeFfnParams p, void* workspace, int num_sms, int pdl, cudaStream_t stream);
cudaError_t sample_launch(const SampleParams& p, int num_sms, int pdl, cudaStream_t stream);

// Sets a kernel's attribute on each device once: `done` is the kernel's own
// set of devices that have it.
template <class F>
cudaError_t set_once(F* kernel, cudaFuncAttribute what, int value, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, what, value);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launches kernel<<<grid, block, smem, stream>>>(args...), as a programmatic
// dependent of the kernel before it on the stream where pdl is set (the kernel
// then calls pdl_wait() before it reads anything that kernel may have written).
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int pdl,
                       const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace gg
