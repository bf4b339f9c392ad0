// Attention of many rows over a paged cache: prompts and chunks, on the fifth
// generation's tensor cores.
//
// A block takes two tiles of up to 128 rows of a (sequence, key head) -- the
// query heads of the group, token by token -- through their keys, 128 at a
// time.  Per tile of keys
//   S = Q K^T   both operands from shared memory, 128 x 128 sums in TMEM
//   P = exp2(c S - c m), c = scale log2 e: one thread to a row, which holds the
//               128 scores in registers, so a row's maximum and sum take no
//               exchange; the weights, in 16 bits, replace the scores in TMEM
//   O += P V    P from TMEM, V from shared memory as it lies in the cache
//               (its rows are the keys: an MN-major operand), sums in TMEM.
// While one tile's threads take exponentials, the tensor cores work on the
// other's products.  The running maximum is only raised when a row's scores
// pass it by 2^8: below that the weights and sums stay far from overflow and
// equally precise, and O keeps its scale; so O is rescaled a few times in all.
//
// Warps 0-3 and 4-7: the two tiles' rows; warp 8 issues copies, warp 9 products.
// What bounds it: 4 x 128 x 128 x D operations a tile pair and key tile on the
// tensor cores, and 2 x 128 x 128 exponentials.
#include "attn.cuh"

namespace gg {

namespace {

constexpr int kThreads = 320;
constexpr int kKeys = 128;          // keys of a tile
constexpr float kRaise = 8.f;       // log2 of how far scores may pass the maximum in use

template <int DP> struct ManyCfg {
    static constexpr int HALF = 128 * 128;                 // bytes of 128 rows x 64 values
    static constexpr int TILE = DP / 64 * HALF;            // 128 rows x DP values
    static constexpr int STAGES = DP == 128 ? 5 : 8;
    static constexpr int SMEM = (2 + STAGES) * TILE + 1024;
};

template <bool BF16> struct Elem { using T = __half; };
template <> struct Elem<true> { using T = __nv_bfloat16; };

__device__ __forceinline__ void tma_load_q(uint32_t smem_dst, const CUtensorMap* map, int d, int head, int token,
                                           uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
}

struct Geometry {
    int rows;        // rows of a tile: whole tokens, at most 128
    int box;         // tokens of a cache box
};

// Block (x, y, z): key head x / splits, split x % splits of the keys; the y-th
// pair of tiles from the end (the longest first); sequence z.
template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const AttnParams p, const Partials part, const Geometry geo) {
    using C = ManyCfg<DP>;
    using T = typename Elem<BF16>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[C::STAGES], s_empty[C::STAGES], s_q, s_score[2], s_weight[2][2], s_sum[2];
    __shared__ uint32_t s_tmem;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sq = smem_u32(base), ring = sq + 2 * C::TILE;

    pdl_wait();
    pdl_launch_dependents();
    const int kvh = blockIdx.x / part.splits, split = blockIdx.x % part.splits;
    const int r0 = (gridDim.y - 1 - blockIdx.y) * 2 * geo.rows;
    RowSpan s;
    if (!row_span(p, blockIdx.z, r0, 2 * geo.rows, s, threadIdx.x == 0)) return;

    // this split's tiles of keys, and how many of them each tile of rows needs
    const int k_lo = s.lo / kKeys, k_n = s.hi > s.lo ? (s.hi + kKeys - 1) / kKeys - k_lo : 0;
    const int k0 = k_lo + (int)((int64_t)k_n * split / part.splits), k1 = k_lo + (int)((int64_t)k_n * (split + 1) / part.splits);
    int tiles[2];
    tiles[0] = k1 - k0;
    tiles[1] = r0 + geo.rows < s.n * p.group ? k1 - k0 : 0;
    if (p.causal && tiles[1]) {
        const int hi = min(s.len, s.len - s.n + (r0 + geo.rows) / p.group);    // the first tile's last token sees up to here
        tiles[0] = max(0, min(k1, (hi + kKeys - 1) / kKeys) - k0);
    }
    const int n = max(tiles[0], tiles[1]);

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 1);
        }
        mbar_init(&s_q, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_score[i], 1);
            mbar_init(&s_weight[i][0], 4);
            mbar_init(&s_weight[i][1], 4);
            mbar_init(&s_sum[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);            // S of the two tiles at 0 and 128, O at 256 and 384

    if (warp == 8) {
        // ---- copies: Q, then K and V of each tile of keys through the ring
        const int32_t* pages = p.b.pages + s.seq * p.b.pages_stride;
        const int nbox = kKeys / geo.box;    // boxes of a tile: a page each, or half of one
        if (lane == 0 && n > 0) {
            const int per = geo.rows / p.group, heads = tiles[1] ? 2 : 1;
            mbar_arrive_expect_tx(&s_q, heads * (DP / 64) * geo.rows * 128);
            for (int t = 0; t < heads; ++t)
                for (int h = 0; h < DP / 64; ++h)
                    tma_load_q(sq + t * C::TILE + h * C::HALF, &tmQ, 64 * h, kvh * p.group,
                               s.t0 + r0 / p.group + t * per, &s_q);
        }
        int done = 0;                        // stages whose copies were started
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            const int j0 = (k0 + i) * kKeys + lane * geo.box;     // lane's first key
            int page = -1;
            if (lane < nbox && j0 < s.hi && j0 + geo.box > s.lo) {
                page = pages[j0 >> p.c.page_shift];
                if ((unsigned)page >= (unsigned)p.c.n_pages) {
                    report(p.status, GGUF_ERR_INVALID_ARG);
                    page = -1;
                }
            }
            const int count = __popc(__ballot_sync(0xffffffffu, page >= 0));
            for (int kv = 0; kv < 2; ++kv, ++done) {
                const int st = done % C::STAGES;
                ok = mbar_wait(&s_empty[st], (done / C::STAGES & 1) ^ 1, p.status);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&s_full[st], count * (DP / 64) * geo.box * 128);
                __syncwarp();
                if (page >= 0)
                    for (int h = 0; h < DP / 64; ++h)
                        tma_load_kv(ring + st * C::TILE + h * C::HALF + lane * geo.box * 128, kv ? &tmV : &tmK, 64 * h,
                                    j0 & ((1 << p.c.page_shift) - 1), kvh, page, &s_full[st]);
            }
        }
        // nothing of this block is in flight when it ends, also after a wait that ran out
        if (lane == 0) {
            if (n > 0) mbar_wait(&s_q, 0, p.status);
            for (int d = max(0, done - C::STAGES); d < done; ++d)
                mbar_wait(&s_full[d % C::STAGES], d / C::STAGES & 1, p.status);
        }
    } else if (warp == 9) {
        // ---- products.  The warp's own instructions are what the tensor cores
        // wait for between products: it goes through them together, descriptors
        // advance by additions, and nothing is divided.
        if (n > 0) {
            const int steps = p.c.dim / 16;
            const uint32_t id_s = idesc_f16(128, 128, BF16), id_o = idesc_f16(128, p.c.dim, BF16) | kIdescBMajorMn;
            constexpr uint32_t kHi = (1024 >> 4) | 1u << 14 | 2u << 29;          // both layouts' upper words are the same
            const uint32_t q_lo = sq >> 4 | 1u << 16, k_lo = ring >> 4 | 1u << 16, v_lo = ring >> 4 | (C::HALF >> 4) << 16;
            bool ok = mbar_wait(&s_q, 0, p.status);
            auto scores = [&](int t, int st) {
                const uint32_t a = q_lo + t * (C::TILE >> 4), b = k_lo + st * (C::TILE >> 4), d = tmem + 128 * t;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < steps) {
                        const uint32_t at = (k / 4 * C::HALF + k % 4 * 32) >> 4;
                        umma_f16_warp(d, a + at, b + at, kHi, id_s, k != 0);
                    }
                umma_commit_warp(&s_score[t]);
            };
            // in halves of 64 keys, as their weights come
            auto sums = [&](int t, int st, uint32_t parity, bool first) {
                const uint32_t b = v_lo + st * (C::TILE >> 4), a = tmem + 128 * t, d = tmem + 256 + 128 * t;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ok = mbar_wait(&s_weight[t][h], parity, p.status);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int k = 4 * h; k < 4 * h + 4; ++k)
                        umma_f16_ts_warp(d, a + 8 * k, b + k * (2048 >> 4), kHi, id_o, k != 0 || !first);
                }
                umma_commit_warp(&s_sum[t]);
            };
            int st = 0;                          // the ring's next stage, and its parity
            uint32_t turn = 0;
            auto next = [&]() {
                const int now = st;
                ok = ok && mbar_wait(&s_full[now], turn, p.status);
                if (++st == C::STAGES) {
                    st = 0;
                    turn ^= 1;
                }
                return now;
            };
            const int k_st = next();
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (tiles[t] > 0) scores(t, k_st);
                umma_commit_warp(&s_empty[k_st]);
            }
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const int v_st = next(), k_next = i + 1 < n ? next() : 0;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (i < tiles[t] && ok) sums(t, v_st, i & 1, i == 0);
                    if (i + 1 < tiles[t] && ok) scores(t, k_next);
                }
                umma_commit_warp(&s_empty[v_st]);
                if (i + 1 < n) umma_commit_warp(&s_empty[k_next]);
            }
        }
        __syncwarp();
    } else {
        // ---- rows: thread `at` of four warps has row at of the tile
        const int t = warp >> 2, at = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + 128 * t + lanes, to = tmem + 256 + 128 * t + lanes;
        const int r = r0 + t * geo.rows + at, tok = r / p.group;
        const bool is = at < geo.rows && tok < s.n;
        int lo = 0, hi = INT32_MAX;         // a row that is none: any scores, never stored
        if (is) row_keys(p, s, s.len - s.n + tok, lo, hi);
        const float c2 = p.scale * kLog2e;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        const int mine = tiles[t];
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            const int j0 = (k0 + i) * kKeys;
            ok = mbar_wait(&s_score[t], i & 1, p.status);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t v[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, v + 32 * c);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 8; ++c) tmem_ld_regs(v + 16 * c);
            if (__any_sync(0xffffffffu, j0 < lo || j0 + kKeys > hi)) {
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (j0 + j < lo || j0 + j >= hi) v[j] = 0xff800000u;      // -inf
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 128; j += 2)
                top[j >> 1 & 3] = max3(top[j >> 1 & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            const bool raise = mx > m && (m == -INFINITY || (mx - m) * c2 > kRaise);
            if (__any_sync(0xffffffffu, raise)) {
                const float f = raise ? exp2_fast((m - mx) * c2) : 1.f;
                if (raise) m = mx;
                l *= f;
                if (i > 0) {
                    ok = mbar_wait(&s_sum[t], (i - 1) & 1, p.status);
                    tc_fence_after();
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t w[16];
                        tmem_ld16(to + 16 * c, w);
                        tmem_ld_wait();
                        tmem_ld_regs(w);
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
                        tmem_st16(to + 16 * c, w);
                    }
                    tmem_st_wait();
                }
            }
            // values that no row of the block sees may be anything: 0 x NaN must
            // not reach the sums.  The products of the first tile of rows come first.
            if ((j0 < s.lo || j0 + kKeys > s.hi) && (t == 0 || i >= tiles[0])) {
                const int d = 2 * i + 1;
                ok = mbar_wait(&s_full[d % C::STAGES], d / C::STAGES & 1, p.status);
                if (j0 + at < s.lo || j0 + at >= s.hi)
                    for (int e = 0; e < DP / 8; ++e)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + d % C::STAGES * C::TILE + e / 8 * C::HALF + at * 128 + e % 8 * 16),
                                     "r"(0)
                                     : "memory");
                fence_proxy_async_smem();
            }
            const float mb = m == -INFINITY ? 0.f : -m * c2;
            const f32x2 cc = {c2, c2}, bb = {mb, mb};
            f32x2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int j = 64 * c; j < 64 * c + 64; j += 2) {
                    const f32x2 x = fma2({__uint_as_float(v[j]), __uint_as_float(v[j + 1])}, cc, bb);
                    const f32x2 w = {exp2_fast(x.x), exp2_fast(x.y)};
                    sum[j >> 1 & 1] = add2(sum[j >> 1 & 1], w);
                    v[j / 2] = pack2<BF16>(w.x, w.y);
                }
                tmem_st32(ts + 32 * c, v + 32 * c);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_weight[t][c]);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        if (mine > 0) ok = ok && mbar_wait(&s_sum[t], (mine - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const int D = p.c.dim, head = kvh * p.group + r % p.group;
        const int64_t row = (int64_t)(s.t0 + tok) * p.heads + head;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        T* out = static_cast<T*>(p.out) + (int64_t)(s.t0 + tok) * p.ldo + head * D;
        float* po = part.o + ((int64_t)split * p.b.n_tokens * p.heads + row) * D;
        for (int c = 0; c < DP / 16; ++c) {
            uint32_t w[16];
            if (mine > 0 && ok) {
                tmem_ld16(to + 16 * c, w);
                tmem_ld_wait();
                tmem_ld_regs(w);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = 0u;
            }
            if (!is || 16 * c >= D) continue;
            if (part.splits > 1) {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<uint4*>(po + 16 * c + j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
            } else {
                uint32_t h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    h[j] = l == 0.f ? 0u : pack2<BF16>(__uint_as_float(w[2 * j]) * inv, __uint_as_float(w[2 * j + 1]) * inv);
                *reinterpret_cast<uint4*>(out + 16 * c) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(out + 16 * c + 8) = make_uint4(h[4], h[5], h[6], h[7]);
            }
        }
        if (is && part.splits > 1)
            part.ml[(int64_t)split * p.b.n_tokens * p.heads + row] = make_float2(l == 0.f ? -INFINITY : m * c2, l);
        else if (is && p.lse)
            p.lse[row] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int DP, bool BF16>
int launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s) {
    Geometry geo;
    const int tokens = 128 / p.group;
    geo.rows = tokens * p.group;
    geo.box = std::min(kKeys, 1 << p.c.page_shift);
    CUtensorMap q, k, v;
    if (make_q_map(&q, p, p.group, tokens) != GGUF_OK || make_kv_map(&k, p.c.k, p.c, geo.box) != GGUF_OK ||
        make_kv_map(&v, p.c.v, p.c, geo.box) != GGUF_OK)
        return GGUF_ERR_UNSUPPORTED;
    auto f = attn_many_kernel<DP, BF16>;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, ManyCfg<DP>::SMEM) != cudaSuccess)
        return GGUF_ERR_CUDA;
    const dim3 grid(p.c.kv_heads * plan.splits, plan.tiles, p.b.n_seq);
    return launch_pdl(f, grid, dim3(kThreads), ManyCfg<DP>::SMEM, s, pdl, q, k, v, p, part, geo) == cudaSuccess
               ? GGUF_OK : GGUF_ERR_CUDA;
}

}  // namespace

int attn_many_launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s) {
    if (p.c.dim > 64) return p.c.bf16 ? launch<128, true>(p, plan, part, pdl, s) : launch<128, false>(p, plan, part, pdl, s);
    return p.c.bf16 ? launch<64, true>(p, plan, part, pdl, s) : launch<64, false>(p, plan, part, pdl, s);
}

}  // namespace gg
