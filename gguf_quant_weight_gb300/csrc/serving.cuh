// Parameters and host entry points of the serving kernels (kv_append.cu,
// paged_attn.cu, logits.cu); the C entry points and their checks are in
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

cudaError_t kv_append_launch(const AppendParams& p, int num_sms, int pdl, cudaStream_t stream);
size_t paged_attn_workspace_bytes(const AttnParams& p, int num_sms);
int paged_attn_launch(const AttnParams& p, void* workspace, int num_sms, int pdl, cudaStream_t stream);
cudaError_t logits_adjust_launch(const LogitsParams& p, int num_sms, int pdl, cudaStream_t stream);

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
