// C entry points of the serving operators: argument checks (all of them before
// anything is launched) and dispatch.
#include <cmath>
#include <cstdlib>

#include "gemm.cuh"
#include "serving.cuh"

using namespace gg;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool valid_dtype(int d) { return d == GGUF_DT_F32 || d == GGUF_DT_F16 || d == GGUF_DT_BF16; }

bool pdl_on() {
    static const bool on = [] {
        const char* e = getenv("GGUF_MM_PDL");
        return !(e && e[0] == '0');
    }();
    return on;
}

constexpr int64_t kMaxTokens = int64_t(1) << 24;

int check_cache(const gguf_kv_cache* c, CacheParams* o) {
    if (!c || !c->k || !c->v) return GGUF_ERR_INVALID_ARG;
    if (c->n_pages <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0) return GGUF_ERR_INVALID_ARG;
    if (c->page_stride <= 0 || c->head_stride <= 0 || c->token_stride <= 0) return GGUF_ERR_INVALID_ARG;
    if (c->dtype != GGUF_DT_F16 && c->dtype != GGUF_DT_BF16) return GGUF_ERR_UNSUPPORTED;
    if (c->head_dim > 128 || c->head_dim % 16) return GGUF_ERR_UNSUPPORTED;
    int shift = 4;
    while (shift < 9 && (1 << shift) != c->page_size) ++shift;
    if (shift == 9) return GGUF_ERR_UNSUPPORTED;
    if (c->n_pages > (int64_t(1) << 30) || c->kv_heads > 1024) return GGUF_ERR_UNSUPPORTED;
    const int64_t lim = int64_t(1) << 38;  // a tensor map's strides are below 2^40 bytes
    if (c->page_stride > lim || c->head_stride > lim || c->token_stride > lim) return GGUF_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride % 8 || c->head_stride % 8 || c->token_stride % 8)
        return GGUF_ERR_MISALIGNED;
    *o = CacheParams{c->k, c->v, c->page_stride, c->head_stride, c->token_stride, (int)c->n_pages, c->kv_heads,
                     c->head_dim, shift, c->dtype == GGUF_DT_BF16};
    return GGUF_OK;
}

// arrays: whether the device arrays are needed (a workspace query has none).
int check_batch(const gguf_kv_batch* b, const CacheParams& c, bool arrays, BatchParams* o) {
    if (!b || (arrays && (!b->q_start || !b->kv_len || !b->pages))) return GGUF_ERR_INVALID_ARG;
    if (b->n_seq <= 0 || b->n_tokens <= 0 || b->max_q_len <= 0 || b->max_kv_len < 0 || b->pages_stride < 0)
        return GGUF_ERR_INVALID_ARG;
    if (b->n_seq > (1 << 16) - 1 || b->n_tokens > kMaxTokens || b->max_kv_len > (1 << 30) ||
        b->pages_stride > (1 << 30))
        return GGUF_ERR_UNSUPPORTED;
    if (b->max_kv_len > b->pages_stride << c.page_shift) return GGUF_ERR_INVALID_ARG;
    if (!aligned4(b->q_start) || !aligned4(b->kv_len) || !aligned4(b->pages)) return GGUF_ERR_MISALIGNED;
    *o = BatchParams{b->q_start, b->kv_len, b->pages, b->pages_stride, (int)b->n_seq, (int)b->n_tokens,
                     (int)std::min<int64_t>(b->max_q_len, b->n_tokens), (int)b->max_kv_len};
    return GGUF_OK;
}

int check_heads(int64_t heads, const CacheParams& c) {
    if (heads <= 0 || heads % c.kv_heads) return GGUF_ERR_INVALID_ARG;
    return heads / c.kv_heads > 128 || heads > (1 << 14) ? GGUF_ERR_UNSUPPORTED : GGUF_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA; }

}  // namespace

extern "C" {

int gguf_kv_append(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv, int xdt,
                   int64_t heads, const gguf_rope* rope, const gguf_kv_batch* batch, const gguf_kv_cache* cache,
                   void* q_out, int64_t ldqo, gguf_stream_t stream) {
    AppendParams p{};
    if (!k || !v || (q == nullptr) != (q_out == nullptr)) return GGUF_ERR_INVALID_ARG;
    int st = check_cache(cache, &p.c);
    if (st == GGUF_OK) st = check_batch(batch, p.c, true, &p.b);
    if (st == GGUF_OK && q) st = check_heads(heads, p.c);
    if (st != GGUF_OK) return st;
    if (!valid_dtype(xdt)) return GGUF_ERR_UNSUPPORTED;
    const int64_t kv_row = (int64_t)p.c.kv_heads * p.c.dim, q_row = heads * p.c.dim;
    if (ldk < kv_row || ldv < kv_row || (q && (ldq < q_row || ldqo < q_row))) return GGUF_ERR_INVALID_ARG;
    if (rope) {
        if (!rope->freqs || rope->rot_dim < 2 || rope->rot_dim > p.c.dim || rope->rot_dim % 2) return GGUF_ERR_INVALID_ARG;
        if (rope->style != GGUF_ROPE_NORM && rope->style != GGUF_ROPE_NEOX) return GGUF_ERR_INVALID_ARG;
        if (!aligned4(rope->freqs) || !aligned4(rope->positions)) return GGUF_ERR_MISALIGNED;
        p.freqs = rope->freqs;
        p.positions = rope->positions;
        p.rope_scale = rope->scale;
        p.rot = rope->rot_dim;
        p.style = rope->style;
    }
    const int per16 = xdt == GGUF_DT_F32 ? 4 : 8;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || ldk % per16 || ldv % per16 ||
        (q && (ldq % per16 || ldqo % 8)))
        return GGUF_ERR_MISALIGNED;
    // in place a row may only overwrite itself
    if (q && q == q_out && (xdt != cache->dtype || (ldq != ldqo && p.b.n_tokens > 1))) return GGUF_ERR_INVALID_ARG;
    int sms = 0;
    if ((st = current_device_launch_facts(&sms, &p.status)) != GGUF_OK) return st;
    p.q = q;
    p.k = k;
    p.v = v;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.q_out = q_out;
    p.ldqo = ldqo;
    p.xdt = xdt;
    p.heads = q ? (int)heads : 0;
    return cuda_status(kv_append_launch(p, sms, pdl_on(), (cudaStream_t)stream));
}

size_t gguf_paged_attn_workspace_size(const gguf_kv_batch* batch, const gguf_kv_cache* cache, int64_t heads) {
    AttnParams p{};
    if (check_cache(cache, &p.c) != GGUF_OK || check_batch(batch, p.c, false, &p.b) != GGUF_OK ||
        check_heads(heads, p.c) != GGUF_OK)
        return 0;
    p.heads = (int)heads;
    p.group = p.heads / p.c.kv_heads;
    int sms = 152, *status = nullptr;  // sized for the current device (152 SMs when none is current)
    if (current_device_launch_facts(&sms, &status) != GGUF_OK) sms = 152;
    return paged_attn_workspace_bytes(p, sms);
}

int gguf_paged_attn(const void* q, int64_t ldq, int64_t heads, const gguf_kv_batch* batch, const gguf_kv_cache* cache,
                    float scale, int causal, int64_t window, void* out, int64_t ldo, float* lse, void* workspace,
                    size_t ws_bytes, gguf_stream_t stream) {
    AttnParams p{};
    if (!q || !out) return GGUF_ERR_INVALID_ARG;
    int st = check_cache(cache, &p.c);
    if (st == GGUF_OK) st = check_batch(batch, p.c, true, &p.b);
    if (st == GGUF_OK) st = check_heads(heads, p.c);
    if (st != GGUF_OK) return st;
    if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 || (causal != 0 && causal != 1)) return GGUF_ERR_INVALID_ARG;
    if (ldq < heads * p.c.dim || ldo < heads * p.c.dim) return GGUF_ERR_INVALID_ARG;
    if (ldq > (int64_t(1) << 38) || ldo > (int64_t(1) << 38)) return GGUF_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(out) || !aligned4(lse) || ldq % 8 || ldo % 8) return GGUF_ERR_MISALIGNED;
    int sms = 0;
    if ((st = current_device_launch_facts(&sms, &p.status)) != GGUF_OK) return st;
    p.q = q;
    p.ldq = ldq;
    p.out = out;
    p.ldo = ldo;
    p.lse = lse;
    p.heads = (int)heads;
    p.group = p.heads / p.c.kv_heads;
    if ((int64_t)p.b.max_q * p.group > (1 << 30)) return GGUF_ERR_UNSUPPORTED;   // rows are counted in 32 bits
    p.scale = scale;
    p.causal = causal;
    // a window that reaches back past any position hides nothing
    p.window = window > (int64_t(1) << 31) ? 0 : window;
    const size_t need = paged_attn_workspace_bytes(p, sms);
    if (need && (!workspace || ws_bytes < need)) return GGUF_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GGUF_ERR_MISALIGNED;
    return paged_attn_launch(p, workspace, sms, pdl_on(), (cudaStream_t)stream);
}

int gguf_logits_adjust(const void* logits, int dt, int64_t ld, int64_t rows, int64_t vocab,
                       const gguf_logit_rules* rules, void* out, int odt, int64_t ldo, gguf_stream_t stream) {
    if (!logits || !out || !rules || rows <= 0 || vocab <= 0 || ld < vocab || ldo < vocab) return GGUF_ERR_INVALID_ARG;
    if (!valid_dtype(dt) || !valid_dtype(odt)) return GGUF_ERR_UNSUPPORTED;
    if (rows > (1 << 16) - 1 || vocab > (1 << 30)) return GGUF_ERR_UNSUPPORTED;
    LogitsParams p{logits, out, ld, ldo, vocab, (int)rows, dt, odt, *rules};
    gguf_logit_rules& r = p.r;
    if (r.hist && !r.hist_start) return GGUF_ERR_INVALID_ARG;
    if (r.bias_ids && (!r.bias || !r.bias_start)) return GGUF_ERR_INVALID_ARG;
    if (r.allow && r.allow_stride < ceil_div(vocab, 32)) return GGUF_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(out)) return GGUF_ERR_MISALIGNED;
    for (const void* a : {(const void*)r.hist, (const void*)r.hist_start, (const void*)r.repeat, (const void*)r.frequency,
                          (const void*)r.presence, (const void*)r.bias_ids, (const void*)r.bias, (const void*)r.bias_start,
                          (const void*)r.allow})
        if (!aligned4(a)) return GGUF_ERR_MISALIGNED;
    // in place a row may only overwrite itself
    if (logits == out && (dt != odt || (ld != ldo && rows > 1))) return GGUF_ERR_INVALID_ARG;
    // a history without a penalty changes nothing
    if (!r.repeat && !r.frequency && !r.presence) r.hist = nullptr;
    int sms = 0, *status = nullptr;
    const int st = current_device_launch_facts(&sms, &status);
    if (st != GGUF_OK) return st;
    return cuda_status(logits_adjust_launch(p, sms, pdl_on(), (cudaStream_t)stream));
}

}  // extern "C"
