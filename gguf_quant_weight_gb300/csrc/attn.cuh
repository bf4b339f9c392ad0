// Pieces shared by the attention kernels: the rows and keys of a block's work,
// tensor maps of the cache, partial results and their joining.
#pragma once
#include "serving.cuh"
#include "tc.cuh"

namespace gg {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {   // 2 units of 2^-23; exp2(-inf) = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two f32 operations in one instruction, on neighbouring registers.
struct f32x2 { float x, y; };
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {   // NaN where one is
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The query heads of one key head and a sequence's new tokens are the rows of
// one attention problem, token by token: row r is token r / group, head
// r % group of the group.  Rows [r0, r0 + rows) of a sequence, the keys
// [lo, hi) that any of them sees, and each row's own limits:
struct RowSpan {
    int seq, t0, n, len;   // sequence, its first packed row, new tokens, keys
    int lo, hi;
};

// Sequence `seq`'s numbers; false where it has no rows at r0, or indexes out
// of range (reported where tell is set).
__device__ __forceinline__ bool row_span(const AttnParams& p, int seq, int r0, int rows, RowSpan& s, bool tell) {
    const int a = p.b.q_start[seq], e = p.b.q_start[seq + 1], len = p.b.kv_len[seq];
    const int64_t room = p.b.pages_stride << p.c.page_shift;
    s.seq = seq;
    s.t0 = a;
    s.n = e - a;
    s.len = len;
    if (a < 0 || e < a || e > p.b.n_tokens || s.n > p.b.max_q || len > room || len > p.b.max_kv) {
        if (tell) report(p.status, GGUF_ERR_INVALID_ARG);
        return false;
    }
    if (r0 >= s.n * p.group) return false;
    const int first = len - s.n + r0 / p.group;                          // positions of the first and last token
    const int last = len - s.n + min(s.n - 1, (r0 + rows - 1) / p.group);
    s.hi = max(0, p.causal ? min(len, last + 1) : len);
    s.lo = p.window ? (int)min((int64_t)s.hi, max((int64_t)0, first - p.window + 1)) : 0;
    return true;
}

// Whether the few-rows form takes a sequence of n new tokens.
__device__ __forceinline__ bool is_few(const AttnParams& p, int n) { return (int64_t)n * p.group <= p.few_rows; }

// Keys [lo, hi) that the token of this position sees.
__device__ __forceinline__ void row_keys(const AttnParams& p, const RowSpan& s, int pos, int& lo, int& hi) {
    hi = p.causal ? min(s.len, pos + 1) : s.len;
    lo = p.window ? (int)max((int64_t)0, pos - p.window + 1) : 0;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

// One box of the cache, swizzled in 128-byte rows: values d.. of tokens slot..
__device__ __forceinline__ void tma_load_kv(uint32_t smem_dst, const CUtensorMap* map, int d, int slot, int head,
                                            int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::
            "r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(slot), "r"(0), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// Tensor map over K or V: (d, slot, block of 64 values, head, page), box 64 x
// rows x blocks x 1 x 1.  With blocks = 1 the third dimension is nothing, and
// values past head_dim read as zeros; with blocks = head_dim / 64 the box brings
// whole heads, one block of 64 values after the other.
int make_kv_map(CUtensorMap* map, const void* base, const CacheParams& c, int rows, int blocks);
// Tensor map over q: (d, head, token), box 64 x heads x tokens.
int make_q_map(CUtensorMap* map, const AttnParams& p, int heads, int tokens);

// Partial results of a call that splits its keys: for split i, packed row
// (token * heads + head): o[i][row][dim], unnormalised f32 sums at the
// exponents of m[i][row], and l[i][row] (ml holds m and l in pairs).
struct Partials {
    float* o;
    float2* ml;
    int splits;
};

struct AttnPlan {
    int few;        // few rows: at most 8 or 16 of a sequence and key head; 0: all sequences in the many-rows form
    int mixed;      // sequences of few rows in the few-rows form, the others in the many-rows form
    int tiles;      // many rows: tiles of 128 rows, or pairs of these, of a sequence and key head
    int cluster;    // few rows, small calls: blocks of a cluster that split the keys
    int blocks;     // few rows, large calls: blocks among whose warps all keys are dealt out; else 0
    int splits;     // many rows: shares of the keys, joined through the workspace where there are several
};

// Row tiles that a block of the many-rows form takes.
inline int many_tiles(const AttnParams& p) { return p.c.dim > 64 ? 2 : 1; }

size_t attn_line_bytes(const AttnParams& p, const AttnPlan& plan);
int attn_few_launch(const AttnParams& p, const AttnPlan& plan, void* workspace, int pdl, cudaStream_t s);
int attn_many_launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s);

}  // namespace gg
