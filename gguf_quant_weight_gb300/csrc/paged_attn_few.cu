// Attention of few rows over a paged cache: single tokens, and short chunks.
//
// Each key and value is read once for the query heads that share it, and is
// used for at most 16 rows, so the cache's bytes bound this: 512 bytes a key
// and key head at 128 values, against 16 rows x 512 operations that legacy
// tensor instructions do in a tenth of the time the bytes take.  The work is
// therefore arranged around loads in flight:
//   * a warp is a worker of its own: it takes every fourth chunk of 16 keys of
//     its block, which a tensor copy brings into the warp's ring of slots
//     (swizzled, zeros past head_dim), and keeps kStages chunks in flight.  No
//     warp waits for another until the end.
//   * scores S = Q K^T with the queries in registers as the first operand; the
//     accumulator's layout of S is the layout that the weights need as first
//     operand of P V, so they never leave the registers.
//   * the keys of a (sequence, key head) are split over the blocks of a
//     cluster, and where those do not fill the GPU over several clusters.  A
//     block's four partial results are joined in shared memory, a cluster's
//     through distributed shared memory, several clusters' by the joining
//     kernel: always in the same order.
#include "attn.cuh"

namespace gg {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 16;      // keys a warp takes at a time
constexpr int kRows = 16;

template <int DP> struct FewCfg {
    static constexpr int BOX = kChunk * 128;                 // 16 keys x 64 values
    static constexpr int SLOT = 2 * (DP / 64) * BOX;         // K, then V
    static constexpr int STAGES = DP == 128 ? 3 : 6;
    static constexpr int RING = kWarps * STAGES * SLOT;      // 96 KB
    static constexpr int SMEM = RING + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <bool BF16> struct Elem { using T = __half; };
template <> struct Elem<true> { using T = __nv_bfloat16; };
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Block (x, y, z): split x (cluster x / cluster size) of the keys, key head and
// row tile y, sequence z.
template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads)
    attn_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p,
                    const Partials part, int tiles, int cluster) {
    using C = FewCfg<DP>;
    using T = typename Elem<BF16>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kWarps * C::STAGES];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];       // the warps' statistics
    __shared__ float2 s_ml[kRows];                                  // the block's
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t* full = s_full + warp * C::STAGES;
    if (lane == 0) {
        if (warp == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        for (int i = 0; i < C::STAGES; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();

    const int kvh = blockIdx.y / tiles, r0 = (blockIdx.y % tiles) * kRows;
    RowSpan s;
    if (!row_span(p, blockIdx.z, r0, kRows, s)) return;             // the whole cluster alike

    // this block's chunks of 16 keys, in equal shares
    const int c_lo = s.lo / kChunk, c_n = s.hi > s.lo ? (s.hi + kChunk - 1) / kChunk - c_lo : 0;
    const int shares = gridDim.x;
    const int c0 = c_lo + (int)((int64_t)c_n * blockIdx.x / shares), c1 = c_lo + (int)((int64_t)c_n * (blockIdx.x + 1) / shares);
    const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;   // chunks c0 + warp + 4 i
    const int32_t* pages = p.b.pages + s.seq * p.b.pages_stride;
    const int per_page = p.c.page_shift - 4;                         // log2 of the chunks in a page
    const uint32_t slots = smem_u32(ring) + warp * C::STAGES * C::SLOT;

    // lane i holds the page of the warp's chunk 32 j + i
    int page_of = 0;
    auto fetch_pages = [&](int from) {
        const int i = from + lane;
        page_of = -1;
        if (i < mine) {
            page_of = pages[(c0 + warp + kWarps * i) >> per_page];
            if ((unsigned)page_of >= (unsigned)p.c.n_pages) {
                report(p.status, GGUF_ERR_INVALID_ARG);
                page_of = -1;
            }
        }
    };
    // whether chunk i was loaded, kept for its use: bit i % 32
    uint32_t have = 0;
    auto issue = [&](int i) {                                        // whole warp
        if (i >= mine) return;
        if ((i & 31) == 0) fetch_pages(i);
        const int page = __shfl_sync(0xffffffffu, page_of, i & 31);
        const uint32_t bit = 1u << (i & 31);
        have = page >= 0 ? have | bit : have & ~bit;
        if (page < 0 || lane != 0) return;
        const int st = i % C::STAGES;
        const int slot = ((c0 + warp + kWarps * i) & ((1 << per_page) - 1)) * kChunk;
        const uint32_t at = slots + st * C::SLOT;
        mbar_arrive_expect_tx(&full[st], C::SLOT);
#pragma unroll
        for (int h = 0; h < DP / 64; ++h) {
            tma_load_kv(at + h * C::BOX, &tmK, 64 * h, slot, kvh, page, &full[st]);
            tma_load_kv(at + (DP / 64 + h) * C::BOX, &tmV, 64 * h, slot, kvh, page, &full[st]);
        }
    };
#pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) issue(i);

    // the queries as first operand: rows lane / 4 and lane / 4 + 8
    const int D = p.c.dim, steps = D / 16;
    uint32_t q[DP / 16][4];
    int lo[2], hi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r = r0 + lane / 4 + 8 * x, tok = r / p.group;
        const bool is = tok < s.n;
        lo[x] = hi[x] = 0;
        if (is) row_keys(p, s, s.len - s.n + tok, lo[x], hi[x]);
        const T* src = static_cast<const T*>(p.q) + (int64_t)(s.t0 + tok) * p.ldq + (kvh * p.group + r % p.group) * D + lane % 4 * 2;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            q[k][x] = is && k < steps ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
            q[k][2 + x] = is && k < steps ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
        }
    }
    const float c2 = p.scale * kLog2e;
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};          // m: of the scores in units of ln 2

    uint32_t phase = 0;                                              // bit st: the parity that slot st waits for
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        const int st = i % C::STAGES;
        if (have >> (i & 31) & 1) {
            if (!mbar_wait(&full[st], phase >> st & 1, p.status)) {
                ok = false;
                break;
            }
            phase ^= 1u << st;
            const uint32_t kb = slots + st * C::SLOT, vb = kb + DP / 64 * C::BOX;
            const int j0 = (c0 + warp + kWarps * i) * kChunk;
            if (j0 + kChunk > s.hi || j0 < s.lo) {
                // values that no row sees may be anything: 0 x NaN must not reach the sums
                for (int e = lane; e < kChunk * 8 * (DP / 64); e += 32) {
                    const int row = e / 8 % kChunk;
                    if (j0 + row >= s.hi || j0 + row < s.lo)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         vb + e / (8 * kChunk) * C::BOX + row * 128 + e % 8 * 16),
                                     "r"(0)
                                     : "memory");
                }
                fence_proxy_async_smem();                            // before the slot's next copy
                __syncwarp();
            }
            // scores of 16 keys: two tiles of 8
            float sc[2][4] = {};
            const int kr = (lane & 7) + (lane >> 4) * 8, kc = lane >> 3 & 1;     // key, and which 8 values
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                uint32_t b[4];
                ldsm4(kb + k / 4 * C::BOX + kr * 128 + (((k % 4 * 2 + kc) ^ (kr & 7)) << 4), b);
                mma16816<BF16>(sc[0], q[k], b[0], b[1]);
                mma16816<BF16>(sc[1], q[k], b[2], b[3]);
            }
            float top[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float t = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int j = j0 + 8 * n + lane % 4 * 2 + y;
                        float& v = sc[n][2 * x + y];
                        v = j >= lo[x] && j < hi[x] ? v * c2 : -INFINITY;
                        t = fmaxf(t, v);
                    }
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                top[x] = fmaxf(m[x], t);
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float f = top[x] > m[x] ? exp2_fast(m[x] - top[x]) : 1.f;
                    m[x] = top[x];
                    l[x] *= f;
#pragma unroll
                    for (int d = 0; d < DP / 8; ++d) {
                        o[d][2 * x] *= f;
                        o[d][2 * x + 1] *= f;
                    }
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float base = m[x] == -INFINITY ? 0.f : m[x];   // a row that has seen nothing yet
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float a = exp2_fast(sc[n][2 * x] - base), b = exp2_fast(sc[n][2 * x + 1] - base);
                    l[x] += a + b;
                    w[2 * n + x] = pack2<BF16>(a, b);
                }
            }
            const int vr = (lane & 7) + (lane >> 3 & 1) * 8, vc = lane >> 4;
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                uint32_t b[4];
                ldsm4t(vb + d / 4 * C::BOX + vr * 128 + (((d % 4 * 2 + vc) ^ (vr & 7)) << 4), b);
                mma16816<BF16>(o[2 * d], w, b[0], b[1]);
                mma16816<BF16>(o[2 * d + 1], w, b[2], b[3]);
            }
            __syncwarp();
        }
        issue(i + C::STAGES);
    }
    if (!ok) {
        // let the copies in flight land before the ring is used for anything else
        for (int i = 0; i < C::STAGES; ++i) mbar_wait(&full[i], phase >> i & 1, p.status, 1 << 12);
    }

    // join the block's warps: the sums at the largest maximum, in the ring's place
    float* so = reinterpret_cast<float*>(ring);                      // [warp][row][DP], the block's result in warp 0's
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (lane % 4 == 0) {
            s_m[warp][lane / 4 + 8 * x] = m[x];
            s_l[warp][lane / 4 + 8 * x] = l[x];
        }
    }
    __syncthreads();                                                 // every ring is done with
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int row = lane / 4 + 8 * x;
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) top = fmaxf(top, s_m[v][row]);
        const float f = m[x] == -INFINITY ? 0.f : exp2_fast(m[x] - top);
#pragma unroll
        for (int d = 0; d < DP / 8; ++d)
            *reinterpret_cast<float2*>(so + (warp * kRows + row) * DP + 8 * d + lane % 4 * 2) =
                make_float2(o[d][2 * x] * f, o[d][2 * x + 1] * f);
        if (warp == 0 && lane % 4 == 0) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) sum += s_m[v][row] == -INFINITY ? 0.f : s_l[v][row] * exp2_fast(s_m[v][row] - top);
            s_ml[row] = make_float2(top, sum);
        }
    }
    __syncthreads();
    const int rows = min(kRows, s.n * p.group - r0);
    for (int e = threadIdx.x; e < rows * DP; e += kThreads) {
        float v = so[e];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) v += so[x * kRows * DP + e];
        so[e] = v;
    }
    if (cluster > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }

    // join the cluster's blocks: each takes its share of the elements
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int split = blockIdx.x / cluster;
    const uint32_t so_a = smem_u32(so), ml_a = smem_u32(s_ml);
    for (int e = rank * kThreads + threadIdx.x; e < rows * D; e += cluster * kThreads) {
        const int row = e / D, d = e - row * D;
        float top = -INFINITY, sum = 0.f, v = 0.f;
        if (cluster > 1) {
            for (int c = 0; c < cluster; ++c) top = fmaxf(top, ld_cluster_f32(cluster_map(ml_a + 8 * row, c)));
            for (int c = 0; c < cluster; ++c) {
                const uint32_t a = cluster_map(ml_a + 8 * row, c);
                const float mc = ld_cluster_f32(a);
                if (mc == -INFINITY) continue;
                const float f = exp2_fast(mc - top);
                sum += f * ld_cluster_f32(a + 4);
                v += f * ld_cluster_f32(cluster_map(so_a + 4 * (row * DP + d), c));
            }
        } else {
            top = s_ml[row].x;
            sum = s_ml[row].y;
            v = so[row * DP + d];
        }
        const int r = r0 + row, tok = s.t0 + r / p.group, head = kvh * p.group + r % p.group;
        const int64_t at = (int64_t)tok * p.heads + head;
        if (part.splits > 1) {
            part.o[((int64_t)split * p.b.n_tokens * p.heads + at) * D + d] = v;
            if (d == 0) part.ml[(int64_t)split * p.b.n_tokens * p.heads + at] = make_float2(top, sum);
        } else {
            put(static_cast<T*>(p.out) + (int64_t)tok * p.ldo + head * D + d, sum > 0.f ? v / sum : (sum == 0.f ? 0.f : sum));
            if (p.lse && d == 0) p.lse[at] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
        }
    }
    if (cluster > 1) {                                               // nobody leaves while another reads its memory
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        cluster_wait_acquire();
    }
}

template <int DP, bool BF16>
int launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s) {
    CUtensorMap k, v;
    if (make_kv_map(&k, p.c.k, p.c, kChunk) != GGUF_OK || make_kv_map(&v, p.c.v, p.c, kChunk) != GGUF_OK)
        return GGUF_ERR_UNSUPPORTED;
    auto f = attn_few_kernel<DP, BF16>;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<DP>::SMEM) != cudaSuccess ||
        cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return GGUF_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(plan.cluster * plan.splits, p.c.kv_heads * plan.tiles, p.b.n_seq);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = FewCfg<DP>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = plan.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, k, v, p, part, plan.tiles, plan.cluster) == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

}  // namespace

int attn_few_launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s) {
    if (p.c.dim > 64) return p.c.bf16 ? launch<128, true>(p, plan, part, pdl, s) : launch<128, false>(p, plan, part, pdl, s);
    return p.c.bf16 ? launch<64, true>(p, plan, part, pdl, s) : launch<64, false>(p, plan, part, pdl, s);
}

}  // namespace gg
