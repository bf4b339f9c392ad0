// Attention of few rows over a paged cache: single tokens, and chunks of up to
// 16 rows (tokens x query heads of a key head).
//
// Each key and value is read once for the query heads that share it, so the
// cache's bytes bound this: 512 bytes a key and key head at 128 values, against
// 16 rows x 512 operations, a tenth of the time even on the legacy tensor
// instructions, whose operands can stay in registers.  The work is therefore
// arranged around loads in flight:
//   * a warp is a worker of its own: tensor copies bring chunks of 16 keys into
//     its ring of slots (swizzled, zeros past head_dim), STAGES of them ahead.
//     No warp waits for another until the end.
//   * scores and weights stay in registers, the weights rounded to 16 bits: an
//     accumulator of S has the layout that they need as first operand of P V (or, for up to 8 rows and
//     with the products turned around, a transpose of 8 x 8 away from it).
//   * small calls split the keys of a (sequence, key head) over the blocks of a
//     cluster; the warps' results are joined in shared memory, the blocks'
//     through distributed shared memory, in one launch.
//   * large calls deal out the batch's keys in equal shares to all the warps
//     that the GPU holds, across sequences, so that a warp's copies never
//     pause and the sequences' lengths do not matter.  A second kernel joins
//     what was cut.
// Partial results are always joined in the same order.  One has seen nothing
// where its sum of weights is 0; its maximum does not tell, since maxima pass
// over NaN: scores of NaN alone leave -inf there, and NaN in the sums.
//
// Measured on GB300, 32 heads on 8 of 128, bf16: one token over 1021 keys 6.2 us;
// 64 tokens over 100..8000 keys, 570 MB, 105 us (5.4 of the 6.7 TB/s of a copy;
// the copies alone take 87 us, joining about 5); one token over 131071 keys of 4
// heads, 268 MB, 52 us.  Two blocks of four warps with three chunks ahead each
// take 105 us of the batch; three blocks with two ahead 124, one with six 135.
#include "attn.cuh"

namespace gg {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 16;      // keys a warp takes at a time
constexpr int kRows = 16;
constexpr int kCluster = 16;    // blocks of a cluster, at most

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
// Element (i, j) of an 8 x 8 matrix of 16-bit values to (j, i); lane: row lane / 4, two values.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// A wait that a warp's lanes give up together, if at all: what follows is for whole warps.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// The workspace of a call in equal shares: sums and statistics in places of
// `rows` rows, two to a worker, and where each sequence begins in the line.
struct LineSpace {
    float* o;
    float2* ml;
    int64_t* begin;
    int rows;
};
LineSpace line_space(const AttnParams& p, const AttnPlan& plan, void* base) {
    LineSpace ws;
    ws.rows = (int)std::min<int64_t>(plan.few, (int64_t)p.b.max_q * p.group);
    const int64_t places = 2 * (int64_t)plan.blocks * kWarps * ws.rows;
    ws.o = static_cast<float*>(base);
    ws.ml = reinterpret_cast<float2*>(ws.o + places * p.c.dim);
    ws.begin = reinterpret_cast<int64_t*>(ws.ml + places);
    return ws;
}

// LIFT: what a weight, at most 1, is multiplied by as operand of P V.  An f16 would
// lose digits below 2^-14 and be 0 below 2^-25, and 10^5 such keys beside a dominant
// one are a visible part of a row; lifted they keep their digits down to 2^-29 and
// vanish below 2^-40.
template <bool BF16> struct Elem { using T = __half; static constexpr float LIFT = 32768.f; };
template <> struct Elem<true> { using T = __nv_bfloat16; static constexpr float LIFT = 1.f; };
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Values of the 16 keys from j0 that no row sees may be anything, and 0 x NaN
// must not reach the sums.
template <int DP>
__device__ __forceinline__ void clear_unseen(const RowSpan& s, uint32_t vb, int j0, int lane) {
    using C = FewCfg<DP>;
    if (j0 >= s.lo && j0 + kChunk <= s.hi) return;
#pragma unroll 1
    for (int e = lane; e < kChunk * 8 * (DP / 64); e += 32) {
        const int row = e / 8 % kChunk;
        if (j0 + row >= s.hi || j0 + row < s.lo)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + e / (8 * kChunk) * C::BOX + row * 128 +
                                                                         e % 8 * 16),
                         "r"(0)
                         : "memory");
    }
    fence_proxy_async_smem();                                        // before the slot's next copy
    __syncwarp();
}

// Whether any of the 16 keys' values is NaN or infinite.
template <int DP, bool BF16>
__device__ __forceinline__ bool any_not_finite(uint32_t vb, int lane) {
    using C = FewCfg<DP>;
    constexpr uint32_t M = BF16 ? 0x7f807f80u : 0x7c007c00u;
    bool bad = false;
#pragma unroll 1
    for (int e = lane; e < kChunk * 8 * (DP / 64); e += 32) {
        uint32_t v[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(vb + e / (8 * kChunk) * C::BOX + e % (8 * kChunk) * 16)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= __vcmpeq2(v[i] & M, M) != 0;
    }
    return __any_sync(0xffffffffu, bad);
}
// Value d of key j of a chunk's values.
template <int DP, bool BF16>
__device__ __forceinline__ float value_at(uint32_t vb, int j, int d) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];"
                 : "=h"(v)
                 : "r"(vb + d / 64 * FewCfg<DP>::BOX + j * 128 + (((d % 64 / 8) ^ (j & 7)) << 4) + d % 8 * 2)
                 : "memory");
    return BF16 ? __bfloat162float(__ushort_as_bfloat16(v)) : __half2float(__ushort_as_half(v));
}

// One warp's work on 16 rows: the queries as first operand (rows lane / 4 and
// lane / 4 + 8), the sums, and the rows' statistics (m in units of ln 2).
template <int DP, bool BF16>
struct Rows16 {
    using C = FewCfg<DP>;
    using T = typename Elem<BF16>::T;
    static constexpr int ROWS = 16;
    uint32_t q[DP / 16][4];
    float o[DP / 8][4];
    float m[2], l[2];
    int lo[2], hi[2];
    int all_lo, all_hi;          // keys that every row sees

    // Whether some of the rows see a key of the chunk from j0 that others do not.  Then
    // values that are not finite must not meet the others' weights of 0.
    __device__ __forceinline__ bool some_see(const RowSpan& s, int j0) const {
        return max(j0, s.lo) < all_lo || min(j0 + kChunk, s.hi) > all_hi;
    }

    static __device__ __forceinline__ int row(int x, int lane) { return lane / 4 + 8 * x; }
    // Whether this lane speaks for its rows' statistics.
    static __device__ __forceinline__ bool speaks(int lane) { return lane % 4 == 0; }
    // f(row's index x, d, value) for each of the lane's sums.
    template <class F>
    __device__ __forceinline__ void each(int lane, F f) const {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                f(x, 8 * i + lane % 4 * 2, o[i][2 * x]);
                f(x, 8 * i + lane % 4 * 2 + 1, o[i][2 * x + 1]);
            }
    }

    __device__ __forceinline__ void begin(const AttnParams& p, const RowSpan& s, int kvh, int lane) {
        const int D = p.c.dim, steps = D / 16;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = row(x, lane), tok = r / p.group;
            const bool is = tok < s.n;
            lo[x] = 0;
            hi[x] = INT32_MAX;           // a row that is none: zeros as queries, never stored
            if (is) row_keys(p, s, s.len - s.n + tok, lo[x], hi[x]);
            const T* src = static_cast<const T*>(p.q) + (int64_t)(s.t0 + tok) * p.ldq + (kvh * p.group + r % p.group) * D +
                           lane % 4 * 2;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                q[k][x] = is && k < steps ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
                q[k][2 + x] = is && k < steps ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
            }
            m[x] = -INFINITY;
            l[x] = 0.f;
        }
        all_lo = max(s.lo, __reduce_max_sync(0xffffffffu, max(lo[0], lo[1])));
        all_hi = min(s.hi, __reduce_min_sync(0xffffffffu, min(hi[0], hi[1])));
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    }

    // The 16 keys from j0 in the ring's slot at kb (K, then V).
    __device__ __forceinline__ void take(const RowSpan& s, uint32_t kb, int j0, float c2, int lane) {
        const uint32_t vb = kb + DP / 64 * C::BOX;
        const bool edge = j0 < all_lo || j0 + kChunk > all_hi;
        if (edge) clear_unseen<DP>(s, vb, j0, lane);
        float sc[2][4] = {};                                         // scores: two tiles of 8 keys
        const int kr = (lane & 7) + (lane >> 4) * 8, kc = lane >> 3 & 1;         // key, and which 8 values
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
                    v = edge && (j < lo[x] || j >= hi[x]) ? -INFINITY : v * c2;
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
            const float base = m[x] == -INFINITY ? 0.f : m[x];       // a row that has seen nothing yet
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float &a = sc[n][2 * x], &b = sc[n][2 * x + 1];
                a = exp2_fast(a - base), b = exp2_fast(b - base);
                l[x] += a + b;
                w[2 * n + x] = pack2<BF16>(a * Elem<BF16>::LIFT, b * Elem<BF16>::LIFT);
            }
        }
        if (edge && some_see(s, j0) && any_not_finite<DP, BF16>(vb, lane)) {
            // each row adds the keys that it sees, key by key
#pragma unroll 1
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int j = 8 * n + 2 * c + y;
                            const float f = __shfl_sync(0xffffffffu, sc[n][2 * x + y], (lane & ~3) | c) * Elem<BF16>::LIFT;
                            if (j0 + j < lo[x] || j0 + j >= hi[x]) continue;
#pragma unroll
                            for (int d = 0; d < DP / 8; ++d)
#pragma unroll
                                for (int z = 0; z < 2; ++z)
                                    o[d][2 * x + z] += f * value_at<DP, BF16>(vb, j, 8 * d + lane % 4 * 2 + z);
                        }
            return;
        }
        const int vr = (lane & 7) + (lane >> 3 & 1) * 8, vc = lane >> 4;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            uint32_t b[4];
            ldsm4t(vb + d / 4 * C::BOX + vr * 128 + (((d % 4 * 2 + vc) ^ (vr & 7)) << 4), b);
            mma16816<BF16>(o[2 * d], w, b[0], b[1]);
            mma16816<BF16>(o[2 * d + 1], w, b[2], b[3]);
        }
    }

    // The lanes' shares of the rows' sums of weights, together; the sums as they are without the lift.
    __device__ __forceinline__ void end() {
        if (!BF16)
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= 1.f / Elem<BF16>::LIFT;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        }
    }
};

// The same on up to 8 rows, the products turned around: S^T = K Q^T has the 16
// keys as rows and the 8 queries as columns, O^T = V^T P^T the values' places as
// rows, so that no half of a 16-row product is spent on rows that are not there.
// The weights pass from accumulator to second operand by transposing two 8 x 8
// matrices.  Lane: queries lane % 4 * 2 + x.
template <int DP, bool BF16>
struct Rows8 {
    using C = FewCfg<DP>;
    using T = typename Elem<BF16>::T;
    static constexpr int ROWS = 8;
    uint32_t q[DP / 16][2];
    float o[DP / 16][4];
    float m[2], l[2];
    int lo[2], hi[2];
    int all_lo, all_hi;

    __device__ __forceinline__ bool some_see(const RowSpan& s, int j0) const {
        return max(j0, s.lo) < all_lo || min(j0 + kChunk, s.hi) > all_hi;
    }

    static __device__ __forceinline__ int row(int x, int lane) { return lane % 4 * 2 + x; }
    static __device__ __forceinline__ bool speaks(int lane) { return lane < 4; }
    template <class F>
    __device__ __forceinline__ void each(int lane, F f) const {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                f(x, 16 * i + lane / 4, o[i][x]);
                f(x, 16 * i + lane / 4 + 8, o[i][2 + x]);
            }
    }

    __device__ __forceinline__ void begin(const AttnParams& p, const RowSpan& s, int kvh, int lane) {
        const int D = p.c.dim, steps = D / 16;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int tok = row(x, lane) / p.group;
            lo[x] = 0;
            hi[x] = INT32_MAX;
            if (tok < s.n) row_keys(p, s, s.len - s.n + tok, lo[x], hi[x]);
            m[x] = -INFINITY;
            l[x] = 0.f;
        }
        all_lo = max(s.lo, __reduce_max_sync(0xffffffffu, max(lo[0], lo[1])));
        all_hi = min(s.hi, __reduce_min_sync(0xffffffffu, min(hi[0], hi[1])));
        // as second operand: query lane / 4, values lane % 4 * 2 and 8 further
        const int r = lane / 4, tok = r / p.group;
        const bool is = tok < s.n;
        const T* src = static_cast<const T*>(p.q) + (int64_t)(s.t0 + tok) * p.ldq + (kvh * p.group + r % p.group) * D +
                       lane % 4 * 2;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[k][h] = is && k < steps ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 * h) : 0u;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    }

    __device__ __forceinline__ void take(const RowSpan& s, uint32_t kb, int j0, float c2, int lane) {
        const uint32_t vb = kb + DP / 64 * C::BOX;
        const bool edge = j0 < all_lo || j0 + kChunk > all_hi;
        if (edge) clear_unseen<DP>(s, vb, j0, lane);
        float sc[2][4] = {};                                         // two sums, to halve the chain
        const int kr = (lane & 7) + (lane >> 3 & 1) * 8, kc = lane >> 4;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            uint32_t a[4];
            ldsm4(kb + k / 4 * C::BOX + kr * 128 + (((k % 4 * 2 + kc) ^ (kr & 7)) << 4), a);
            mma16816<BF16>(sc[k & 1], a, q[k][0], q[k][1]);
        }
        float e[4], top[2];                                          // [2 y + x]: key lane / 4 + 8 y
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = j0 + lane / 4 + 8 * y;
                const float v = sc[0][2 * y + x] + sc[1][2 * y + x];
                e[2 * y + x] = edge && (j < lo[x] || j >= hi[x]) ? -INFINITY : v * c2;
            }
            float t = fmaxf(e[x], e[2 + x]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            top[x] = fmaxf(m[x], t);
        }
        if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float f = top[x] > m[x] ? exp2_fast(m[x] - top[x]) : 1.f;
                m[x] = top[x];
                l[x] *= f;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    o[i][x] *= f;
                    o[i][2 + x] *= f;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float base = m[x] == -INFINITY ? 0.f : m[x];
            e[x] = exp2_fast(e[x] - base);
            e[2 + x] = exp2_fast(e[2 + x] - base);
            l[x] += e[x] + e[2 + x];
        }
        constexpr float up = Elem<BF16>::LIFT;
        if (edge && some_see(s, j0) && any_not_finite<DP, BF16>(vb, lane)) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int j = 8 * y + c;
                        const float f = __shfl_sync(0xffffffffu, e[2 * y + x], 4 * c + lane % 4) * up;
                        if (j0 + j < lo[x] || j0 + j >= hi[x]) continue;
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                            for (int z = 0; z < 2; ++z)
                                o[i][2 * z + x] += f * value_at<DP, BF16>(vb, j, 16 * i + lane / 4 + 8 * z);
                    }
            return;
        }
        const uint32_t w0 = transpose8(pack2<BF16>(e[0] * up, e[1] * up)), w1 = transpose8(pack2<BF16>(e[2] * up, e[3] * up));
        const int vr = (lane & 7) + (lane >> 4) * 8, vc = lane >> 3 & 1;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            uint32_t a[4];
            ldsm4t(vb + i / 4 * C::BOX + vr * 128 + (((i % 4 * 2 + vc) ^ (vr & 7)) << 4), a);
            mma16816<BF16>(o[i], a, w0, w1);
        }
    }

    __device__ __forceinline__ void end() {
        if (!BF16)
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= 1.f / Elem<BF16>::LIFT;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
    }
};

// Whether one copy brings 16 whole keys: the fewer copies, the nearer to the
// memory's rate they come.  (A head that ends inside 64 values takes two, so
// that what is past it reads as zeros.)
__host__ __device__ inline bool whole_heads(const AttnParams& p) { return p.c.dim % 64 == 0; }

template <int DP>
__device__ __forceinline__ void load_chunk(uint32_t at, const CUtensorMap* tmK, const CUtensorMap* tmV, bool whole, int slot,
                                           int kvh, int page, uint64_t* bar) {
    using C = FewCfg<DP>;
    mbar_arrive_expect_tx(bar, C::SLOT);
    tma_load_kv(at, tmK, 0, slot, kvh, page, bar);
    tma_load_kv(at + DP / 64 * C::BOX, tmV, 0, slot, kvh, page, bar);
    if (DP == 128 && !whole) {
        tma_load_kv(at + C::BOX, tmK, 64, slot, kvh, page, bar);
        tma_load_kv(at + 3 * C::BOX, tmV, 64, slot, kvh, page, bar);
    }
}

// ------------------------------------------------------------------ keys split over a cluster

// Block (x, y, z): the x-th block of the cluster, key head y, sequence z.
template <int DP, bool BF16, class W>
__global__ void __launch_bounds__(kThreads)
    attn_few_cluster_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const AttnParams p, int stages) {
    using C = FewCfg<DP>;
    using T = typename Elem<BF16>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kWarps * C::STAGES];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];       // the warps' statistics
    __shared__ float2 s_ml[kRows];                                  // the block's
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cluster = gridDim.x;
    uint64_t* full = s_full + warp * C::STAGES;
    if (lane == 0) {
        if (warp == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();

    const int kvh = blockIdx.y;
    RowSpan s;
    // the whole cluster alike
    if (!row_span(p, blockIdx.z, 0, W::ROWS, s, threadIdx.x == 0) || !is_few(p, s.n)) return;

    // this block's chunks of 16 keys, in equal shares; the warps take them in turn
    const int c_lo = s.lo / kChunk, c_n = s.hi > s.lo ? (s.hi + kChunk - 1) / kChunk - c_lo : 0;
    const int c0 = c_lo + (int)((int64_t)c_n * blockIdx.x / cluster), c1 = c_lo + (int)((int64_t)c_n * (blockIdx.x + 1) / cluster);
    const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;   // chunks c0 + warp + 4 i
    const int32_t* pages = p.b.pages + s.seq * p.b.pages_stride;
    const int per_page = p.c.page_shift - 4;                         // log2 of the chunks in a page
    const uint32_t slots = smem_u32(ring) + warp * stages * C::SLOT;

    int page_of = 0;          // lane i: the page of the warp's chunk 32 j + i
    uint32_t have = 0;        // bit i % 32: chunk i was loaded
    int st_get = 0;
    auto issue = [&](int i) {
        if (i >= mine) return;
        const int to = st_get;
        st_get = to + 1 == stages ? 0 : to + 1;
        if ((i & 31) == 0) {
            page_of = -1;
            if (i + lane < mine) {
                page_of = pages[(c0 + warp + kWarps * (i + lane)) >> per_page];
                if ((unsigned)page_of >= (unsigned)p.c.n_pages) {
                    report(p.status, GGUF_ERR_INVALID_ARG);
                    page_of = -1;
                }
            }
        }
        const int page = __shfl_sync(0xffffffffu, page_of, i & 31);
        const uint32_t bit = 1u << (i & 31);
        have = page >= 0 ? have | bit : have & ~bit;
        if (page < 0 || lane != 0) return;
        load_chunk<DP>(slots + to * C::SLOT, &tmK, &tmV, whole_heads(p), ((c0 + warp + kWarps * i) & ((1 << per_page) - 1)) * kChunk, kvh,
                       page, &full[to]);
    };
#pragma unroll 1
    for (int i = 0; i < stages; ++i) issue(i);

    W w;
    w.begin(p, s, kvh, lane);
    const float c2 = p.scale * kLog2e;
    uint32_t phase = 0;                                              // bit st: the parity that slot st waits for
    bool ok = true;
    int st = 0;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        if (have >> (i & 31) & 1) {
            if (!wait_warp(&full[st], phase >> st & 1, p.status)) {
                ok = false;
                break;
            }
            phase ^= 1u << st;
            w.take(s, slots + st * C::SLOT, (c0 + warp + kWarps * i) * kChunk, c2, lane);
            __syncwarp();
        }
        st = st + 1 == stages ? 0 : st + 1;
        issue(i + stages);
    }
    if (!ok) {
        // let the copies in flight land before the ring is used for anything else
        for (int i = 0; i < stages; ++i) mbar_wait(&full[i], phase >> i & 1, p.status, 1 << 12);
    }

    // join the block's warps: the sums at the largest maximum, in the ring's place
    constexpr int LD = DP + 4;
    float* so = reinterpret_cast<float*>(ring);                      // [warp][row][LD], the block's result in warp 0's
    w.end();
#pragma unroll
    for (int x = 0; x < 2; ++x)
        if (W::speaks(lane)) {
            s_m[warp][W::row(x, lane)] = w.m[x];
            s_l[warp][W::row(x, lane)] = w.l[x];
        }
    __syncthreads();                                                 // every ring is done with
    float f[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int row = W::row(x, lane);
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) top = fmaxf(top, s_m[v][row]);
        f[x] = w.l[x] == 0.f ? 0.f : exp2_fast(w.m[x] - top);
        if (warp == 0 && W::speaks(lane)) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) sum += s_l[v][row] == 0.f ? 0.f : s_l[v][row] * exp2_fast(s_m[v][row] - top);
            s_ml[row] = make_float2(top, sum);
        }
    }
    w.each(lane, [&](int x, int d, float v) { so[(warp * W::ROWS + W::row(x, lane)) * LD + d] = v * f[x]; });
    __syncthreads();
    const int rows = s.n * p.group;
    for (int e = threadIdx.x; e < rows * LD; e += kThreads) {
        float v = so[e];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) v += so[x * W::ROWS * LD + e];
        so[e] = v;
    }
    if (cluster > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }

    // join the cluster's blocks: each takes its share of the elements
    const int D = p.c.dim;
    const uint32_t so_a = smem_u32(so), ml_a = smem_u32(s_ml);
    for (int e = blockIdx.x * kThreads + threadIdx.x; e < rows * D; e += cluster * kThreads) {
        const int row = e / D, d = e - row * D;
        float top = -INFINITY, sum = 0.f, v = 0.f;
        if (cluster > 1) {
            float mc[kCluster], lc[kCluster], vc[kCluster];          // every block's, all loads in flight at once
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                mc[c] = -INFINITY;
                lc[c] = vc[c] = 0.f;
                if (c >= cluster) continue;
                const uint32_t a = cluster_map(ml_a + 8 * row, c);
                mc[c] = ld_cluster_f32(a);
                lc[c] = ld_cluster_f32(a + 4);
                vc[c] = ld_cluster_f32(cluster_map(so_a + 4 * (row * LD + d), c));
            }
#pragma unroll
            for (int c = 0; c < kCluster; ++c) top = fmaxf(top, mc[c]);
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                const float f = lc[c] == 0.f ? 0.f : exp2_fast(mc[c] - top);
                sum += f * lc[c];
                v += f * vc[c];
            }
        } else {
            top = s_ml[row].x;
            sum = s_ml[row].y;
            v = so[row * LD + d];
        }
        const int tok = s.t0 + row / p.group, head = kvh * p.group + row % p.group;
        put(static_cast<T*>(p.out) + (int64_t)tok * p.ldo + head * D + d, sum > 0.f ? v / sum : (sum == 0.f ? 0.f : sum));
        if (p.lse && d == 0) p.lse[(int64_t)tok * p.heads + head] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
    }
    if (cluster > 1) {                                               // nobody leaves while another reads its memory
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        cluster_wait_acquire();
    }
}

// ------------------------------------------------------------------ keys in equal shares to every warp
//
// All chunks of the batch stand in one line: sequence by sequence, key head by key
// head.  Of `total` chunks worker w of W, as many as there are warps or chunks,
// takes [total w / W, total (w + 1) / W), whatever sequences they belong to.  An
// item (a sequence's key head) whose chunks one worker has alone is written at
// once; of the others each worker leaves its sums in the workspace -- in place
// 2 w where its share begins inside the item, 2 w + 1 where the item begins in
// its share -- and the joining kernel adds them in the line's order.

__device__ __forceinline__ int64_t share_begin(int64_t total, int w, int workers) { return total * w / workers; }
// The worker that has chunk x.
__device__ __forceinline__ int share_of(int64_t total, int64_t x, int workers) {
    return (int)(((x + 1) * workers + total - 1) / total) - 1;
}

// Chunks of a sequence; one that sees no key has one, empty.
__device__ __forceinline__ int seq_chunks(const RowSpan& s) {
    return s.hi > s.lo ? (s.hi + kChunk - 1) / kChunk - s.lo / kChunk : 1;
}
// Chunks that it takes of the line, with all key heads.
template <int ROWS>
__device__ __forceinline__ int64_t line_chunks(const AttnParams& p, int seq) {
    RowSpan s;
    return row_span(p, seq, 0, ROWS, s, false) ? (int64_t)seq_chunks(s) * p.c.kv_heads : 0;
}

// A place in the line.
struct Cursor {
    RowSpan s;
    int kvh;
    int c, n;          // chunk of the item, and how many it has
};

// The first item of a sequence with rows from `seq` on (past the end: none is asked for).
template <int ROWS>
__device__ __forceinline__ void settle(const AttnParams& p, Cursor& k, int seq) {
    for (; seq < p.b.n_seq; ++seq)
        if (row_span(p, seq, 0, ROWS, k.s, false)) {
            k.n = seq_chunks(k.s);
            k.kvh = k.c = 0;
            return;
        }
}
template <int ROWS>
__device__ __forceinline__ void next_item(const AttnParams& p, Cursor& k) {
    k.c = 0;
    if (++k.kvh == p.c.kv_heads) settle<ROWS>(p, k, k.s.seq + 1);
}

template <int DP, bool BF16, class W>
__global__ void __launch_bounds__(kThreads)
    attn_few_line_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p,
                         const LineSpace ws) {
    using C = FewCfg<DP>;
    using T = typename Elem<BF16>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kWarps * C::STAGES];
    __shared__ int64_t s_sum[kWarps], s_at[kWarps];
    __shared__ int s_seq[kWarps];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = blockIdx.x * kWarps + warp;
    uint64_t* full = s_full + warp * C::STAGES;
    if (lane == 0) {
        if (warp == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        for (int i = 0; i < C::STAGES; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        s_seq[warp] = p.b.n_seq;
    }
    pdl_wait();
    pdl_launch_dependents();

    // the line's length, then the sequence in which each warp's share begins: one
    // reading of the batch's arrays where a block's threads cover the sequences
    int64_t total = 0, before = 0, own = 0;
    int workers = 0;
    auto scan = [&](int b0) {
        const int b = b0 + threadIdx.x;
        own = b < p.b.n_seq ? line_chunks<W::ROWS>(p, b) : 0;
        int64_t sum = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t v = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += v;
        }
        if (lane == 31) s_sum[warp] = sum;
        __syncthreads();
        before = total + sum - own;
        for (int v = 0; v < kWarps; ++v) {
            if (v < warp) before += s_sum[v];
            total += s_sum[v];
        }
        __syncthreads();
    };
    auto find = [&](int b0, int64_t length) {
        const int b = b0 + threadIdx.x;
        workers = (int)min((int64_t)(gridDim.x * kWarps), length);
        for (int v = 0; v < kWarps && blockIdx.x * kWarps + v < workers; ++v) {
            const int64_t x = share_begin(length, blockIdx.x * kWarps + v, workers);
            if (own && before <= x && x < before + own) {
                s_seq[v] = b;
                s_at[v] = x - before;
            }
        }
        if (blockIdx.x == 0 && b < p.b.n_seq) {
            ws.begin[b] = before;
            RowSpan s;
            row_span(p, b, 0, W::ROWS, s, true);                     // reports what is out of range
        }
    };
    for (int b0 = 0; b0 < p.b.n_seq; b0 += kThreads) scan(b0);
    if (p.b.n_seq <= kThreads) {
        find(0, total);
    } else {
        const int64_t length = total;
        total = 0;
        for (int b0 = 0; b0 < p.b.n_seq; b0 += kThreads) {
            scan(b0);
            find(b0, length);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) ws.begin[p.b.n_seq] = total;
    if (me >= workers) return;
    const int64_t x0 = share_begin(total, me, workers);
    int left = (int)(share_begin(total, me + 1, workers) - x0);       // chunks of this warp's share, at least one

    // two places in the line: what is consumed, and what is loaded, STAGES chunks on
    Cursor use;
    settle<W::ROWS>(p, use, s_seq[warp]);
    use.kvh = (int)(s_at[warp] / use.n);
    use.c = (int)(s_at[warp] - (int64_t)use.kvh * use.n);
    Cursor get = use;
    int to_get = left;
    const int per_page = p.c.page_shift - 4;
    const uint32_t slots = smem_u32(ring) + warp * C::STAGES * C::SLOT;
    int page_of = -1, page_from = -1;                                // lane i: the page of the item's chunk page_from + i
    uint32_t have = 0;
    int st_get = 0;
    auto issue = [&]() {
        if (to_get == 0) return;
        const int first = get.s.lo / kChunk;
        if (page_from < 0 || get.c >= page_from + 32) {
            page_from = get.c;
            page_of = -1;
            const int c = get.c + lane;
            if (c < get.n && get.s.hi > get.s.lo) {
                page_of = p.b.pages[get.s.seq * p.b.pages_stride + ((first + c) >> per_page)];
                if ((unsigned)page_of >= (unsigned)p.c.n_pages) {
                    report(p.status, GGUF_ERR_INVALID_ARG);
                    page_of = -1;
                }
            }
        }
        const int page = __shfl_sync(0xffffffffu, page_of, get.c - page_from);
        have = page >= 0 ? have | 1u << st_get : have & ~(1u << st_get);
        if (page >= 0 && lane == 0)
            load_chunk<DP>(slots + st_get * C::SLOT, &tmK, &tmV, whole_heads(p), ((first + get.c) & ((1 << per_page) - 1)) * kChunk, get.kvh,
                           page, &full[st_get]);
        st_get = st_get + 1 == C::STAGES ? 0 : st_get + 1;
        if (--to_get && ++get.c == get.n) {
            next_item<W::ROWS>(p, get);
            page_from = -1;
        }
    };
#pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) issue();

    const float c2 = p.scale * kLog2e;
    const int D = p.c.dim;
    uint32_t phase = 0;
    int st = 0;
    bool inside = use.c > 0;                                         // the share begins inside an item
    W w;
    w.begin(p, use.s, use.kvh, lane);
#pragma unroll 1
    while (left > 0) {
        if (have >> st & 1) {
            if (!wait_warp(&full[st], phase >> st & 1, p.status)) break;
            phase ^= 1u << st;
            w.take(use.s, slots + st * C::SLOT, (use.s.lo / kChunk + use.c) * kChunk, c2, lane);
            __syncwarp();
        }
        st = st + 1 == C::STAGES ? 0 : st + 1;
        issue();
        --left;
        ++use.c;
        if (use.c < use.n && left > 0) continue;
        // the item's end, or the share's
        w.end();
        const bool whole = !inside && use.c == use.n;
        const int64_t place = 2 * me + (inside ? 0 : 1);
        int64_t to[2];                                               // where the lane's rows go, -1: nowhere
        float inv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int row = W::row(x, lane), tok = use.s.t0 + row / p.group, head = use.kvh * p.group + row % p.group;
            to[x] = -1;
            inv[x] = w.l[x] > 0.f ? 1.f / w.l[x] : (w.l[x] == 0.f ? 0.f : w.l[x]);
            if (row >= use.s.n * p.group) continue;
            to[x] = whole ? (int64_t)tok * p.ldo + head * D : (place * ws.rows + row) * D;
            if (!W::speaks(lane)) continue;
            if (!whole) ws.ml[place * ws.rows + row] = make_float2(w.m[x], w.l[x]);
            else if (p.lse) p.lse[(int64_t)tok * p.heads + head] = w.l[x] == 0.f ? -INFINITY : w.m[x] * kLn2 + logf(w.l[x]);
        }
        if (whole) w.each(lane, [&](int x, int d, float v) { if (to[x] >= 0 && d < D) put(static_cast<T*>(p.out) + to[x] + d, v * inv[x]); });
        else w.each(lane, [&](int x, int d, float v) { if (to[x] >= 0 && d < D) ws.o[to[x] + d] = v; });
        if (left > 0) {
            next_item<W::ROWS>(p, use);
            inside = false;
            w.begin(p, use.s, use.kvh, lane);
        }
    }
    if (left > 0)        // a wait ran out: let the copies in flight land
        for (int i = 0; i < C::STAGES; ++i) mbar_wait(&full[i], phase >> i & 1, p.status, 1 << 12);
}

// Joins the items that several workers had: block (x, y, z) key head x of sequence
// y, of it row z / parts and the z % parts-th `db` values.  Each thread adds four
// values over every per-th worker; then the sums are added in pairs.
constexpr int kJoin = 512;
template <bool BF16>
__global__ void __launch_bounds__(kJoin) attn_line_join_kernel(const AttnParams p, const LineSpace ws, int workers /* warps of the grid */,
                                                               int db, int ROWS) {
    using T = typename Elem<BF16>::T;
    __shared__ float4 s_v[kJoin];
    __shared__ float2 s_ml[kJoin];
    // what the batch's arrays say stands since before the kernel this one follows
    const int kvh = blockIdx.x, seq = blockIdx.y, D = p.c.dim, parts = D / db, row = blockIdx.z / parts;
    RowSpan s;
    const bool is = row_span(p, seq, 0, ROWS, s, false) && row < s.n * p.group;
    pdl_wait();
    pdl_launch_dependents();
    if (!is) return;
    const int n = seq_chunks(s);
    const int64_t x = ws.begin[seq] + (int64_t)n * kvh;
    const int64_t total = ws.begin[p.b.n_seq];
    workers = (int)min((int64_t)workers, total);
    const int w0 = share_of(total, x, workers), w1 = share_of(total, x + n - 1, workers);
    if (w0 == w1) return;                                            // one worker had it and wrote it
    const int work = db / 4, per = blockDim.x / work, g = threadIdx.x / work;
    const int d = blockIdx.z % parts * db + (threadIdx.x - g * work) * 4;
    float top = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, float4 o) {
        if (ml.y == 0.f) return;
        const float t = fmaxf(top, ml.x), a = exp2_fast(top - t), b = exp2_fast(ml.x - t);
        top = t;
        sum = sum * a + ml.y * b;
        v = make_float4(v.x * a + o.x * b, v.y * a + o.y * b, v.z * a + o.z * b, v.w * a + o.w * b);
    };
    if (g < per) {
        for (int w = w0 + g; w <= w1; w += 4 * per) {
            float2 ml[4];
            float4 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                if (w + i * per > w1) continue;
                const int64_t at = (2 * (int64_t)(w + i * per) + (w + i * per == w0)) * ws.rows + row;
                ml[i] = ws.ml[at];
                o[i] = *reinterpret_cast<const float4*>(ws.o + at * D + d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) add(ml[i], o[i]);
        }
    }
    for (int h = per; h > 1;) {                                      // pairs (g, g + ceil(h / 2))
        const int to = (h + 1) / 2;
        if (g >= to && g < h) {
            s_v[threadIdx.x] = v;
            s_ml[threadIdx.x] = make_float2(top, sum);
        }
        __syncthreads();
        if (g + to < h) add(s_ml[threadIdx.x + to * work], s_v[threadIdx.x + to * work]);
        h = to;
    }
    if (g != 0) return;
    const int tok = s.t0 + row / p.group, head = kvh * p.group + row % p.group;
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    T* out = static_cast<T*>(p.out) + (int64_t)tok * p.ldo + head * D + d;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
    if (p.lse && d == 0) p.lse[(int64_t)tok * p.heads + head] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
}

template <int DP, bool BF16, class W>
int launch_line(const AttnParams& p, const AttnPlan& plan, void* workspace, int pdl, cudaStream_t s) {
    CUtensorMap k, v;
    if (make_kv_map(&k, p.c.k, p.c, kChunk, whole_heads(p) ? DP / 64 : 1) != GGUF_OK || make_kv_map(&v, p.c.v, p.c, kChunk, whole_heads(p) ? DP / 64 : 1) != GGUF_OK)
        return GGUF_ERR_UNSUPPORTED;
    const LineSpace ws = line_space(p, plan, workspace);
    auto f = attn_few_line_kernel<DP, BF16, W>;
    static std::atomic<uint64_t> ready{0};
    if (set_once(f, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<DP>::SMEM, ready) != cudaSuccess ||
        launch_pdl(f, dim3(plan.blocks), dim3(kThreads), FewCfg<DP>::SMEM, s, pdl, k, v, p, ws) != cudaSuccess)
        return GGUF_ERR_CUDA;
    // a block to a row of an item, with threads for four shares each; where few
    // items are cut into a great many, a block to 16 values of a row
    const int64_t cuts = plan.blocks * kWarps / ((int64_t)p.b.n_seq * p.c.kv_heads) + 1;
    const int db = cuts >= 64 ? 16 : p.c.dim;
    int per = 1;
    while (per < 16 && per * 4 < cuts) per *= 2;
    const int threads = cuts >= 64 ? kJoin : (int)ceil_div(db / 4 * per, 32) * 32;
    return launch_pdl(attn_line_join_kernel<BF16>, dim3(p.c.kv_heads, p.b.n_seq, ws.rows * (p.c.dim / db)),
                      dim3(threads), 0, s, pdl, p, ws, plan.blocks * kWarps, db, W::ROWS) == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

template <int DP, bool BF16, class W>
int launch_cluster(const AttnParams& p, const AttnPlan& plan, int pdl, cudaStream_t s) {
    CUtensorMap k, v;
    if (make_kv_map(&k, p.c.k, p.c, kChunk, whole_heads(p) ? DP / 64 : 1) != GGUF_OK || make_kv_map(&v, p.c.v, p.c, kChunk, whole_heads(p) ? DP / 64 : 1) != GGUF_OK)
        return GGUF_ERR_UNSUPPORTED;
    auto f = attn_few_cluster_kernel<DP, BF16, W>;
    static std::atomic<uint64_t> ready{0}, wide{0};
    if (set_once(f, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<DP>::SMEM, ready) != cudaSuccess ||
        set_once(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, wide) != cudaSuccess)
        return GGUF_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    // no more slots to a warp than chunks: blocks of short sequences are small, and
    // more of them are on the GPU at once
    using C = FewCfg<DP>;
    const int64_t chunks = ceil_div(ceil_div(p.b.max_kv, kChunk) + 1, plan.cluster * kWarps);
    const int stages = (int)std::min<int64_t>(C::STAGES, std::max<int64_t>(1, chunks));
    cfg.gridDim = dim3(plan.cluster, p.c.kv_heads, p.b.n_seq);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = std::max(kWarps * stages * C::SLOT, kWarps * W::ROWS * (DP + 4) * 4) + 1024;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = plan.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, k, v, p, stages) == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

}  // namespace

size_t attn_line_bytes(const AttnParams& p, const AttnPlan& plan) {
    const LineSpace ws = line_space(p, plan, nullptr);
    return (size_t)reinterpret_cast<uintptr_t>(ws.begin + p.b.n_seq + 1);
}

template <int DP, bool BF16>
static int run(const AttnParams& p, const AttnPlan& plan, void* workspace, int pdl, cudaStream_t s) {
    if (plan.few == 8)
        return plan.blocks ? launch_line<DP, BF16, Rows8<DP, BF16>>(p, plan, workspace, pdl, s)
                           : launch_cluster<DP, BF16, Rows8<DP, BF16>>(p, plan, pdl, s);
    return plan.blocks ? launch_line<DP, BF16, Rows16<DP, BF16>>(p, plan, workspace, pdl, s)
                       : launch_cluster<DP, BF16, Rows16<DP, BF16>>(p, plan, pdl, s);
}

int attn_few_launch(const AttnParams& p, const AttnPlan& plan, void* workspace, int pdl, cudaStream_t s) {
    if (p.c.dim > 64) return p.c.bf16 ? run<128, true>(p, plan, workspace, pdl, s) : run<128, false>(p, plan, workspace, pdl, s);
    return p.c.bf16 ? run<64, true>(p, plan, workspace, pdl, s) : run<64, false>(p, plan, workspace, pdl, s);
}

}  // namespace gg
