// Attention of many rows over a paged cache: prompts and chunks, on the fifth
// generation's tensor cores.
//
// A block takes two tiles of up to 128 rows of a (sequence, key head) -- the
// query heads of the group, token by token -- through their keys, 128 at a
// time; for heads of up to 64 values one tile, with two blocks to an SM (short
// sequences then leave no half of a block idle: 24 ragged chunks take a tenth
// less; heads of 128 values have no room for two blocks' keys).  Per tile of keys
//   S = Q K^T   both operands from shared memory, 128 x 128 sums in TMEM
//   P = exp2(c S - c m), c = scale log2 e: two threads to a row, 64 scores each
//               in registers; the weights, in 16 bits (as the tensor cores take
//               them: each moves a row by at most its half unit of |V|), replace the
//               scores in TMEM
//   O += P V    P from TMEM, V from shared memory as it lies in the cache
//               (its rows are the keys: an MN-major operand), sums in TMEM.
// While one tile's threads take exponentials, the tensor cores work on the
// other's products.  The running maximum is only raised when a row's scores
// pass it by 2^8: below that the weights and sums stay far from overflow and
// equally precise, and O keeps its scale; so O is rescaled a few times in all.
//
// Eight warps to a tile of rows, then one that issues copies and one for products.
// A block that is done takes over one that has not begun (its index comes from
// the launch's own queue), so its copies and products of the next tiles start
// while the last rows are written; blocks stand in the order of their work, the
// longest first.
//
// What bounds it: a tile's chain of scores (512 cycles of the tensor cores at 128
// values), its rows' threads (about 1300, of them 900 for the weights) and sums
// (512), two of which run side by side; so the tensor cores, which the products
// of a pair of tiles take 2048 cycles, work 70 % of the time.  Measured on GB300:
// 8111-token prompt, 32 heads on 8 of 128, bf16, 333 us in a burst of calls, 1618
// TFLOP/s, and 357 us, 1510, after a second of them, when the power limit lowers the
// clock (a plain bf16 product reaches 1931 and 1740); heads of 64 values have half
// the products for the same weights, and reach 660 to 930.  Short items (a window
// of 1000 keys: 10 tiles) spend a quarter of their time on the first tile and on
// writing their rows.  The row threads' 96 registers, all that 18 to 20 warps leave
// them, are 20 bytes short at 128 values and 52 to 68 at 64.
//
// A row's two warps meet at barriers of their own: where any row raises its maximum,
// after they have rescaled the sums (the products add to all columns of O once the
// first half's weights are there), and where an item begins and ends.  A bounded
// wait that has run out in one of them is made known at these, so that both leave.
// The meetings cost a tenth of the window's 64 us and 1 % of the prompt.
#include "attn.cuh"

namespace gg {

namespace {

constexpr int kKeys = 128;          // keys of a tile
constexpr float kRaise = 8.f;       // log2 of how far scores may pass the maximum in use
// log2 of what the weights of an f16 call are lifted by, with kRaise at most to 2^15: an
// f16 loses digits below 2^-14 and is 0 below 2^-25, and 10^5 keys of such weights are a
// visible part of a row.  Sums of weights and of values carry it alike.
constexpr float kLift = 7.f;

template <int DP, int TILES> struct ManyCfg {
    static constexpr int HALF = 128 * 128;                 // bytes of 128 rows x 64 values
    static constexpr int TILE = DP / 64 * HALF;            // 128 rows x DP values
    static constexpr int STAGES = TILES == 2 ? 4 : 5;
    static constexpr int SMEM = (TILES + STAGES) * TILE;   // 192 KB for two tiles of 128 values, 96 KB for one of 64
    static constexpr int COPIES = 8 * TILES, PRODUCTS = COPIES + 1;           // warps
    static constexpr int THREADS = 32 * (PRODUCTS + 1);
    static constexpr int COLUMNS = 256 * TILES;            // of TMEM: scores of the tiles, then sums, 128 each
};

// LIFT: log2 of the weights' factor; DROP: what takes it out of a sum.
template <bool BF16> struct Elem { using T = __half; static constexpr float LIFT = kLift, DROP = 1.f / 128.f; };
template <> struct Elem<true> { using T = __nv_bfloat16; static constexpr float LIFT = 0.f, DROP = 1.f; };

__device__ __forceinline__ void tma_load_q(uint32_t smem_dst, const CUtensorMap* map, int d, int head, int token,
                                           uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void store32(void* to, const uint32_t* v) {   // 32 bytes, aligned to as many
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Whether x holds for any thread of two warps that share barrier `id`.
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return any != 0;
}

struct Geometry {
    int rows;        // rows of a tile: whole tokens, at most 128
    int box;         // tokens of a cache box
    int beside;      // the few-rows kernel was launched just before
};

// A pair of row tiles and its share of the keys, from a block's index (x, y, z):
// key head x / splits, split x % splits of the keys; the y-th pair from the
// end; sequence z.
struct Item {
    RowSpan s;
    int kvh, split, r0;
    int k0;             // first tile of keys
    int tiles[2], n;    // tiles of keys that each tile of rows needs, and the larger number
    int more;           // 1: an item with rows, 0: one without, -1: the end
};

template <int TILES>
__device__ __forceinline__ bool find_item(const AttnParams& p, int splits, const Geometry& geo, uint3 at, Item& w, bool tell) {
    w.kvh = at.x / splits;
    w.split = at.x - w.kvh * splits;
    w.r0 = (gridDim.y - 1 - at.y) * TILES * geo.rows;
    w.n = w.tiles[0] = w.tiles[1] = 0;
    if (!row_span(p, at.z, w.r0, TILES * geo.rows, w.s, tell) || is_few(p, w.s.n)) return false;
    const RowSpan& s = w.s;
    const int lo = s.lo / kKeys, all = s.hi > s.lo ? (s.hi + kKeys - 1) / kKeys - lo : 0;
    w.k0 = lo;
    int k1 = lo + all;
    if (splits > 1) {
        w.k0 = lo + (int)((int64_t)all * w.split / splits);
        k1 = lo + (int)((int64_t)all * (w.split + 1) / splits);
    }
    w.tiles[0] = k1 - w.k0;
    if (TILES == 2 && w.r0 + geo.rows < s.n * p.group) {
        w.tiles[1] = w.tiles[0];
        if (p.causal) {          // the first tile's last token sees up to here
            const int hi = min(s.len, s.len - s.n + (w.r0 + geo.rows) / p.group);
            w.tiles[0] = max(0, min(k1, (hi + kKeys - 1) / kKeys) - w.k0);
        }
    }
    w.n = max(w.tiles[0], w.tiles[1]);
    return true;
}

// Asks for the index of a block that has not begun, which then never does: 16
// bytes arrive at `to` and on the barrier.
__device__ __forceinline__ void take_block(uint4* to, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(to)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool taken_block(const uint4* from, uint3& at) {
    uint32_t got, x, y, z;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
        "ld.shared.b128 h, [%4];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, _}, h;\n\t}"
        : "=r"(got), "=r"(x), "=r"(y), "=r"(z)
        : "r"(smem_u32(from))
        : "memory");
    at = make_uint3(x, y, z);
    return got != 0;
}

// A row's weight of 0 for a key that only others of its tile see, times a value that
// is not finite, has spoilt sums of the row.  Half of the row's columns, from c0 and
// every other 16, again: those in which a key of [a, b) outside [lo, hi) holds such
// a value, from the keys of [a, b) inside.  (Cold, so its own function.)
struct Redo {
    int a, b, lo, hi;
    int kvh, c0;
    const int32_t* pages;
    const void* q;      // the row's query
    float c2, base;     // weight = exp2(c2 s + base)
    float factor;       // of a sum in what is stored: as f32 at `part`, else in 16 bits at `out`
    float* part;
    void* out;
};
template <bool BF16>
__device__ __noinline__ void redo_row(const AttnParams& p, const Redo& r) {
    using T = typename Elem<BF16>::T;
    auto row_of = [&](const void* cache, int j) -> const T* {
        const int page = r.pages[j >> p.c.page_shift];
        if ((unsigned)page >= (unsigned)p.c.n_pages) return nullptr;
        return static_cast<const T*>(cache) + page * p.c.page_stride + r.kvh * p.c.head_stride +
               (j & ((1 << p.c.page_shift) - 1)) * p.c.token_stride;
    };
    for (int c = r.c0; c < p.c.dim; c += 32) {
        uint32_t spoilt = 0;
        for (int j = r.a; j < r.b; ++j) {
            if (j == max(r.a, r.lo)) j = max(j, min(r.b, r.hi));         // past the keys that the row sees
            const T* v = j < r.b ? row_of(p.c.v, j) : nullptr;
            for (int d = 0; v && d < 16; ++d)
                if (!isfinite((float)v[c + d])) spoilt |= 1u << d;
        }
        if (!spoilt) continue;
        float sum[16] = {};
        for (int j = max(r.a, r.lo); j < min(r.b, r.hi); ++j) {
            const T *k = row_of(p.c.k, j), *v = row_of(p.c.v, j), *q = static_cast<const T*>(r.q);
            if (!k) continue;
            float s = 0.f;
            for (int d = 0; d < p.c.dim; ++d) s = fmaf((float)q[d], (float)k[d], s);
            const float w = exp2_fast(fmaf(s, r.c2, r.base));
#pragma unroll
            for (int d = 0; d < 16; ++d) sum[d] = fmaf(w, (float)v[c + d], sum[d]);
        }
#pragma unroll
        for (int d = 0; d < 16; ++d) {
            if (!(spoilt >> d & 1)) continue;
            if (r.part) r.part[c + d] = sum[d] * r.factor;
            else static_cast<T*>(r.out)[c + d] = T(sum[d] * r.factor);
        }
    }
}

template <int DP, bool BF16, int TILES>
__global__ void __launch_bounds__(ManyCfg<DP, TILES>::THREADS, 3 - TILES)
    attn_many_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnParams p, const Partials part,
                     const Geometry geo) {
    using C = ManyCfg<DP, TILES>;
    using T = typename Elem<BF16>::T;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // copies of K and V; Q; scores, weights (halves) and sums of a tile; the next block's index
    __shared__ __align__(8) uint64_t s_full[C::STAGES], s_empty[C::STAGES], s_q[2], s_qfree[2], s_score[2], s_weight[2][2],
        s_sum[2], s_next, s_item[2], s_read[2];
    __shared__ uint4 s_answer;
    __shared__ Item s_work[2];
    __shared__ float s_pair[2][2][128];          // two threads of a row
    __shared__ uint32_t s_tmem;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t sq = smem_u32(smem_raw), ring = sq + TILES * C::TILE;

    if (sq & 1023) {            // the swizzle's unit; the alignment asked for gives it
        if (threadIdx.x == 0) report(p.status, GGUF_ERR_CUDA);
        return;
    }
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_q[i], 1);
            mbar_init(&s_qfree[i], 1);
            mbar_init(&s_score[i], 1);
            mbar_init(&s_weight[i][0], 4);
            mbar_init(&s_weight[i][1], 4);
            mbar_init(&s_sum[i], 1);
            mbar_init(&s_item[i], 1);
            mbar_init(&s_read[i], C::COPIES + 1);                               // warps that read it
        }
        mbar_init(&s_next, 1);
        fence_mbar_init();
    }
    if (warp == C::PRODUCTS) tmem_alloc(&s_tmem, C::COLUMNS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // S of tile t at column 128 t, O at 128 (TILES + t).  (All 512 columns begin at 0.)
    const uint32_t tmem = TILES == 2 ? 0 : __shfl_sync(0xffffffffu, s_tmem, 0);
    // Beside the few-rows kernel of the same call, which has waited for what came
    // before, this one waits at its end, so that what comes after waits for both.
    if (!geo.beside) pdl_wait();
    pdl_launch_dependents();

    bool ok = true;
    // the k-th item of this block, as the copying warp found it
    auto next_item = [&](int k) -> const Item& {
        ok = mbar_wait(&s_item[k & 1], k >> 1 & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        return s_work[k & 1];
    };
    auto item_done = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_read[k & 1]);
    };

    if (warp == C::COPIES) {
        // ---- copies: Q, then K and V of each tile of keys through the ring
        const int nbox = kKeys / geo.box;    // boxes of a tile: a page each, or half of one
        int st = 0, quse[2] = {0, 0};        // the ring's next stage; copies of Q so far
        uint32_t turn = 1, loaded = 0;       // the parity of an empty stage; bit st: the stage was ever loaded
        uint3 at = blockIdx;
        Item w;
        for (int k = 0;; ++k) {
            if (k > 0) {
                ok = ok && mbar_wait(&s_next, k - 1 & 1, p.status);
                ok = __all_sync(0xffffffffu, ok);
                w.more = ok && taken_block(&s_answer, at) ? 0 : -1;
                fence_proxy_async_smem();
                __syncwarp();
            } else {
                w.more = 0;
            }
            if (w.more == 0) {
                if (lane == 0) take_block(&s_answer, &s_next);
                w.more = find_item<TILES>(p, part.splits, geo, at, w, lane == 0) ? 1 : 0;
            }
            if (k >= 2) ok = ok && mbar_wait(&s_read[k & 1], (k >> 1) - 1 & 1, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                s_work[k & 1] = w;
                mbar_arrive(&s_item[k & 1]);
            }
            if (w.more < 0) break;
            if (w.more == 0) continue;
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                if (w.tiles[t] == 0) continue;
                if (quse[t] > 0) ok = ok && mbar_wait(&s_qfree[t], quse[t] - 1 & 1, p.status);
                ++quse[t];
                if (lane == 0 && ok) {
                    mbar_arrive_expect_tx(&s_q[t], (DP / 64) * geo.rows * 128);
                    for (int h = 0; h < DP / 64; ++h)
                        tma_load_q(sq + t * C::TILE + h * C::HALF, &tmQ, 64 * h, w.kvh * p.group,
                                   w.s.t0 + (w.r0 + t * geo.rows) / p.group, &s_q[t]);
                }
            }
            const int32_t* pages = p.b.pages + w.s.seq * p.b.pages_stride;
            ok = __all_sync(0xffffffffu, ok);
            for (int i = 0; i < w.n && ok; ++i) {
                const int j0 = (w.k0 + i) * kKeys + lane * geo.box;   // lane's first key
                int page = -1;
                if (lane < nbox && j0 < w.s.hi && j0 + geo.box > w.s.lo) {
                    page = pages[j0 >> p.c.page_shift];
                    if ((unsigned)page >= (unsigned)p.c.n_pages) {
                        report(p.status, GGUF_ERR_INVALID_ARG);
                        page = -1;
                    }
                }
                const int count = __popc(__ballot_sync(0xffffffffu, page >= 0));
                for (int kv = 0; kv < 2; ++kv) {
                    ok = mbar_wait(&s_empty[st], turn, p.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&s_full[st], count * (DP / 64) * geo.box * 128);
                    __syncwarp();
                    if (page >= 0)
                        for (int h = 0; h < DP / 64; ++h)
                            tma_load_kv(ring + st * C::TILE + h * C::HALF + lane * geo.box * 128, kv ? &tmV : &tmK, 64 * h,
                                        j0 & ((1 << p.c.page_shift) - 1), w.kvh, page, &s_full[st]);
                    loaded |= 1u << st;
                    if (++st == C::STAGES) {
                        st = 0;
                        turn ^= 1;
                    }
                }
            }
            if (!ok) break;
        }
        // nothing of this block is in flight when it ends, also after a wait that
        // ran out: the last copy of every stage and of Q (the answer has been read)
        if (lane == 0) {
            for (int i = 0; i < C::STAGES; ++i)
                if (loaded >> i & 1) mbar_wait(&s_full[i], i < st ? turn ^ 1 : turn, p.status);
            for (int t = 0; t < 2; ++t)
                if (quse[t] > 0) mbar_wait(&s_q[t], quse[t] - 1 & 1, p.status);
            if (!ok) mbar_wait(&s_next, 0, p.status), mbar_wait(&s_next, 1, p.status);
        }
    } else if (warp == C::PRODUCTS) {
        // ---- products.  The warp's own instructions are what the tensor cores
        // wait for between products: it goes through them together, descriptors
        // advance by additions, and nothing is divided.
        const int steps = p.c.dim / 16;
        const uint32_t id_s = idesc_f16(128, 128, BF16), id_o = idesc_f16(128, p.c.dim, BF16) | kIdescBMajorMn;
        // Q and K are K-major.  V's rows in the cache are its keys, the products' K: as B it is
        // MN-major, eight keys to an atom of 1024 bytes, the next 64 values (the leading byte
        // offset) a HALF further.  The upper words (atoms 1024 apart, 128-byte swizzle) agree.
        constexpr uint32_t kHi = (1024 >> 4) | 1u << 14 | 2u << 29;
        const uint32_t q_lo = sq >> 4 | 1u << 16, k_lo = ring >> 4 | 1u << 16, v_lo = ring >> 4 | (C::HALF >> 4) << 16;
        int st = 0;                          // the ring's next stage, and its parity
        uint32_t turn = 0, quse = 0, weights = 0;   // bit t: parity of the next Q, and of the next weights
        // once a wait has run out there are no more: what follows is worthless, but ends
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.status));
        };
        auto scores = [&](int t, int from, bool last) {
            // (a shuffle's result is known to be the same in all lanes)
            const uint32_t b = __shfl_sync(0xffffffffu, k_lo + from * (C::TILE >> 4), 0);
            const uint32_t a = q_lo + t * (C::TILE >> 4), d = tmem + 128 * t;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
                if (k < steps) {
                    const uint32_t off = (k / 4 * C::HALF + k % 4 * 32) >> 4;
                    umma_f16_warp(d, a + off, b + off, kHi, id_s, k != 0);
                }
            umma_commit_warp(&s_score[t]);
            if (last) umma_commit_warp(&s_qfree[t]);
        };
        // in halves of 64 keys, as their weights come
        auto sums = [&](int t, int from, bool first) {
            const uint32_t b = __shfl_sync(0xffffffffu, v_lo + from * (C::TILE >> 4), 0);
            const uint32_t a = tmem + 128 * t, d = tmem + 128 * (TILES + t);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                wait(&s_weight[t][h], weights >> t & 1);
                tc_fence_after();
#pragma unroll
                for (int k = 4 * h; k < 4 * h + 4; ++k)
                    umma_f16_ts_warp(d, a + 8 * k, b + k * (2048 >> 4), kHi, id_o, k != 0 || !first);
            }
            weights ^= 1u << t;
            umma_commit_warp(&s_sum[t]);
        };
        auto next = [&]() {
            const int now = st;
            wait(&s_full[now], turn);
            if (++st == C::STAGES) {
                st = 0;
                turn ^= 1;
            }
            return now;
        };
        for (int k = 0;; ++k) {
            const Item& w = next_item(k);
            if (!ok) break;
            const int more = __shfl_sync(0xffffffffu, w.more, 0), n = __shfl_sync(0xffffffffu, w.n, 0);
            const int tiles[2] = {__shfl_sync(0xffffffffu, w.tiles[0], 0), __shfl_sync(0xffffffffu, w.tiles[1], 0)};
            item_done(k);
            if (more < 0) break;
            if (more == 0 || n == 0) continue;
            const int first = next();
#pragma unroll
            for (int t = 0; t < TILES; ++t)
                if (tiles[t] > 0) {
                    wait(&s_q[t], quse >> t & 1);
                    quse ^= 1u << t;
                    tc_fence_after();
                    scores(t, first, tiles[t] == 1);
                }
            umma_commit_warp(&s_empty[first]);
            int v_st = next();
            // every wait stands behind products enough to cover it
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const bool more_keys = i + 1 < n;
                int k_st = 0, v_next = 0;
                if (i < tiles[0]) sums(0, v_st, i == 0);
                if (more_keys) k_st = next();
                if (i + 1 < tiles[0]) scores(0, k_st, i + 2 == tiles[0]);
                if (TILES == 2 && i < tiles[1]) sums(1, v_st, i == 0);
                umma_commit_warp(&s_empty[v_st]);
                if (more_keys) v_next = next();
                if (TILES == 2 && i + 1 < tiles[1]) scores(1, k_st, i + 2 == tiles[1]);
                if (more_keys) umma_commit_warp(&s_empty[k_st]);
                v_st = v_next;
            }
            if (!ok) break;
        }
    } else {
        // ---- rows: two threads to a row, in warps of the same TMEM lanes; thread
        // (in, half) has the row's scores 64 half .. 64 half + 63
        const int t = warp >> 3, half = warp >> 2 & 1, in = 32 * (warp & 3) + lane, pair = 1 + t * 4 + (warp & 3);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + 128 * t + lanes, to = tmem + 128 * (TILES + t) + lanes;
        const float c2 = p.scale * kLog2e;
        int stage0 = 1;             // the ring's stage of the item's first V, and its parity
        uint32_t turn0 = 0;
        uint32_t par = 0;           // parity of the tile's next scores, weights and sums
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.status)) != 0;
        };
        // Two warps that share a barrier never leave each other there: one whose wait
        // has run out goes on to the meetings that the other has before it learns of
        // it, and both leave from the same one.
        // The row's two threads' values, to both; false where a warp gives up.
        auto exchange = [&](float x, bool good, float& other) {
            s_pair[t][half][in] = x;
            const bool both = !pair_any(pair, !good);
            other = s_pair[t][half ^ 1][in];
            return both;
        };
        for (int k = 0;; ++k) {
            const Item& w = next_item(k);
            ok = !pair_any(pair, !ok);      // (also: what was exchanged before has been read)
            if (!ok || w.more < 0) break;
            if (w.more == 0) {
                item_done(k);
                continue;
            }
            int lo = 0, hi = INT32_MAX;     // a row that is none: any scores, never stored
            {
                const int tok = (w.r0 + t * geo.rows + in) / p.group;
                if (in < geo.rows && tok < w.s.n) row_keys(p, w.s, w.s.len - w.s.n + tok, lo, hi);
            }
            // the keys that all the warp's rows see need no mask (a warp without rows
            // still has its part in clearing V's edge)
            const int all_lo = max(w.s.lo, __reduce_max_sync(0xffffffffu, lo));
            const int all_hi = min(w.s.hi, __reduce_min_sync(0xffffffffu, hi));
            float m = -INFINITY, l = 0.f;
            const int mine = w.tiles[t], k0 = w.k0;
            int v_st = stage0;              // the ring's stage of this tile of V
            uint32_t v_turn = turn0;
#pragma unroll 1
            for (int i = 0; i < mine; ++i) {
                const int j0 = (k0 + i) * kKeys;
                // without the scores: the two meetings up to the exchange, then away
                auto give_up = [&]() {
                    float none;
                    pair_any(pair, true);
                    exchange(0.f, false, none);
                    ok = false;
                };
                if (!wait(&s_score[t], par)) {
                    give_up();
                    break;
                }
                tc_fence_after();
                uint32_t v[64];
                tmem_ld32(ts + 64 * half, v);
                tmem_ld32(ts + 64 * half + 32, v + 32);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 64; c += 16) tmem_ld_regs(v + c);
                if (j0 < all_lo || j0 + kKeys > all_hi) {
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        // keys [from, to) of the 32 are seen
                        const int j1 = j0 + 64 * half + c, from = max(0, min(32, lo - j1)), end = max(0, min(32, hi - j1));
                        const uint32_t seen = (end == 32 ? 0xffffffffu : (1u << end) - 1) & ~(from == 32 ? 0xffffffffu : (1u << from) - 1);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(seen >> j & 1)) v[c + j] = 0xff800000u;         // -inf
                    }
                    // values that no row of the item sees may be anything: 0 x NaN must
                    // not reach the sums.  The products of the first tile of rows come
                    // first, and those of 64 keys wait for the warps that clear them here.
                    if ((j0 < w.s.lo || j0 + kKeys > w.s.hi) && (t == 0 || i >= w.tiles[0])) {
                        if (!wait(&s_full[v_st], v_turn)) {
                            give_up();
                            break;
                        }
                        const int row = 64 * half + (in >> 1);
                        if (j0 + row < w.s.lo || j0 + row >= w.s.hi)
#pragma unroll 1
                            for (int e = in & 1; e < DP / 8; e += 2)
                                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 ring + v_st * C::TILE + e / 8 * C::HALF + row * 128 + e % 8 * 16),
                                             "r"(0)
                                             : "memory");
                        fence_proxy_async_smem();
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 64; j += 2)
                    top[j >> 1 & 3] = max3_nan(top[j >> 1 & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                float mx = max3_nan(max3_nan(top[0], top[1], top[2]), top[3], top[3]);
                // Whether any row of the two warps has to raise its maximum (or a warp gives
                // up): mostly none has.  (Past this barrier both threads have their scores, and
                // weights may replace them; and what was exchanged before has been read, since
                // products that needed both threads' weights came between.)
                if (pair_any(pair, !(mx <= m) && !((mx - m) * c2 <= kRaise))) {
                    float other;
                    ok = exchange(mx, true, other);
                    if (!ok) break;
                    mx = max3_nan(mx, other, other);
                    const bool raise = !(mx <= m) && !((mx - m) * c2 <= kRaise);
                    const float f = raise ? exp2_fast((m - mx) * c2) : 1.f;
                    if (raise) m = mx < INFINITY ? mx : NAN;     // the row has no finite sum: all of it is NaN
                    l *= f;
                    if (i > 0) {
                        const bool good = wait(&s_sum[t], par ^ 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 16 * half; good && c < DP; c += 32) {
                            uint32_t y[16];
                            tmem_ld16(to + c, y);
                            tmem_ld_wait();
                            tmem_ld_regs(y);
#pragma unroll
                            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                            tmem_st16(to + c, y);
                        }
                        tmem_st_wait();
                        // The products of a tile's first 64 keys wait for the first half's
                        // weights alone and add to every column of O, so neither warp may
                        // deliver weights before both have rescaled their columns.
                        tc_fence_before();
                        ok = !pair_any(pair, !good);
                        if (!ok) break;
                    }
                }
                const float mb = m == -INFINITY ? 0.f : fmaf(-m, c2, Elem<BF16>::LIFT);
                const f32x2 cc = {c2, c2}, bb = {mb, mb};
                f32x2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    const f32x2 u = fma2({__uint_as_float(v[j]), __uint_as_float(v[j + 1])}, cc, bb);
                    const f32x2 e = {exp2_fast(u.x), exp2_fast(u.y)};
                    sum[j >> 1 & 1] = add2(sum[j >> 1 & 1], e);
                    v[j / 2] = pack2<BF16>(e.x, e.y);
                }
                tmem_st32(ts + 32 * half, v);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_weight[t][half]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                par ^= 1;
                if ((v_st += 2) >= C::STAGES) {
                    v_st -= C::STAGES;
                    v_turn ^= 1;
                }
            }
            // the next item's first V
            stage0 += 2 * w.n;
            turn0 ^= stage0 / C::STAGES & 1;
            stage0 %= C::STAGES;
            if (!ok) break;
            float other;
            ok = exchange(l, w.tiles[t] == 0 || wait(&s_sum[t], par ^ 1), other);
            if (!ok) break;
            l += other;
            tc_fence_after();
            // (again, rather than in registers through the loop)
            const int r = w.r0 + t * geo.rows + in, tok = r / p.group;
            const bool is = in < geo.rows && tok < w.s.n;
            const int D = p.c.dim, head = w.kvh * p.group + r % p.group;
            const int64_t row = (int64_t)(w.s.t0 + tok) * p.heads + head;
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            // 32 bytes of its row at a time from each thread: whole sectors
            T* out = static_cast<T*>(p.out) + (int64_t)(w.s.t0 + tok) * p.ldo + head * D;
            float* po = part.o + ((int64_t)w.split * p.b.n_tokens * p.heads + row) * D;
            const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)p.ldo * 2) & 31) == 0;
            float zero = 0.f;        // NaN where a sum is not finite
#pragma unroll 1
            for (int c = 16 * half; c < D; c += 32) {
                uint32_t y[16];
                if (w.tiles[t] > 0) {
                    tmem_ld16(to + c, y);
                    tmem_ld_wait();
                    tmem_ld_regs(y);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = 0u;
                }
                if (!is) continue;
#pragma unroll
                for (int j = 0; j < 16; ++j) zero = fmaf(__uint_as_float(y[j]), 0.f, zero);
                if (part.splits > 1) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (!BF16) y[j] = __float_as_uint(__uint_as_float(y[j]) * Elem<BF16>::DROP);
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<uint4*>(po + c + j) = make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = l == 0.f ? 0u : pack2<BF16>(__uint_as_float(y[2 * j]) * inv, __uint_as_float(y[2 * j + 1]) * inv);
                if (wide) {
                    store32(out + c, y);
                } else {
                    *reinterpret_cast<uint4*>(out + c) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
            if (zero != 0.f && l < INFINITY) {
                Redo r;
                r.a = max(w.s.lo, w.k0 * kKeys);
                r.b = min(w.s.hi, (w.k0 + w.tiles[t]) * kKeys);
                row_keys(p, w.s, w.s.len - w.s.n + tok, r.lo, r.hi);
                r.kvh = w.kvh;
                r.c0 = 16 * half;
                r.pages = p.b.pages + w.s.seq * p.b.pages_stride;
                r.q = static_cast<const T*>(p.q) + (int64_t)(w.s.t0 + tok) * p.ldq + head * D;
                r.c2 = c2;
                r.base = m == -INFINITY ? 0.f : fmaf(-m, c2, Elem<BF16>::LIFT);
                r.factor = part.splits > 1 ? Elem<BF16>::DROP : inv;
                r.part = part.splits > 1 ? po : nullptr;
                r.out = out;
                redo_row<BF16>(p, r);
            }
            __syncwarp();
            if (!is || half != 0) {
            } else if (part.splits > 1)
                part.ml[(int64_t)w.split * p.b.n_tokens * p.heads + row] = make_float2(l == 0.f ? -INFINITY : m * c2, l * Elem<BF16>::DROP);
            else if (p.lse)
                p.lse[row] = l == 0.f ? -INFINITY : m * p.scale + logf(l * Elem<BF16>::DROP);
            tc_fence_before();
            item_done(k);
        }
    }
    if (geo.beside) pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::PRODUCTS) tmem_dealloc(tmem, C::COLUMNS);
}

template <int DP, bool BF16, int TILES>
int launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s) {
    using C = ManyCfg<DP, TILES>;
    Geometry geo;
    const int tokens = 128 / p.group;
    geo.rows = tokens * p.group;
    geo.box = std::min(kKeys, 1 << p.c.page_shift);
    geo.beside = plan.mixed;
    CUtensorMap q, k, v;
    if (make_q_map(&q, p, p.group, tokens) != GGUF_OK || make_kv_map(&k, p.c.k, p.c, geo.box, 1) != GGUF_OK ||
        make_kv_map(&v, p.c.v, p.c, geo.box, 1) != GGUF_OK)
        return GGUF_ERR_UNSUPPORTED;
    auto f = attn_many_kernel<DP, BF16, TILES>;
    static std::atomic<uint64_t> ready{0};
    if (set_once(f, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM, ready) != cudaSuccess) return GGUF_ERR_CUDA;
    const dim3 grid(p.c.kv_heads * plan.splits, plan.tiles, p.b.n_seq);
    return launch_pdl(f, grid, dim3(C::THREADS), C::SMEM, s, pdl, q, k, v, p, part, geo) == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

}  // namespace

int attn_many_launch(const AttnParams& p, const AttnPlan& plan, const Partials& part, int pdl, cudaStream_t s) {
    if (many_tiles(p) == 2) return p.c.bf16 ? launch<128, true, 2>(p, plan, part, pdl, s) : launch<128, false, 2>(p, plan, part, pdl, s);
    return p.c.bf16 ? launch<64, true, 1>(p, plan, part, pdl, s) : launch<64, false, 1>(p, plan, part, pdl, s);
}

}  // namespace gg
