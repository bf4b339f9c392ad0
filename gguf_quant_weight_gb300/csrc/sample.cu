// Draws a token from each row of logits, from given random numbers, after
// temperature, top-k, top-p and min-p, in one kernel.
//
// All three filters keep a run of the tokens in falling order (of equal logits
// the lower index first), so together they keep the tokens before or at some (logit K,
// index I); the token drawn is the first in the vocabulary's order whose
// running sum of kept weights passes u times their sum.  Nothing is sorted.
//
// Which token that is must not hang on rounding: among 10^5 kept tokens a sum
// that is off by 10^-7 meets the wrong one once in a hundred rows.  So a
// weight 2^-z, z = (max - x) / temperature * log2 e, is taken to about 1e-9 of
// itself, without a bias (z in two floats; a table of 2^-(j + 1/2)/32 and four terms of the
// series for the rest, as in Tang's table-driven exponential, ACM TOMS 1989) and
// becomes an integer of 46 bits.  Sums of integers do not depend on their order:
// the result is the same however the row is cut, and atomics add them up.
//
// A cluster of up to 8 blocks takes a row, a warp a run of its tokens.  The first
// pass reads the logits for their maximum.  The second, out of L2, counts them by
// their distance from it, in sixteenths of z: there top-k's last token is in a bin
// that is known, and a bin's weights are known to 2.2 %, so that top-p's last
// token lies before a bin that is known too.  The third lists the tokens up to
// that bin (or min-p's bound) in shared memory; what follows looks at those
// alone.  Where a run ends is found by histograms: of z again, with the exact
// weights, then of ranges of the logits' bits, until the bin in which it ends has at most kCap
// tokens, which are compared with each other.  Where that many tokens are all
// that the filters can leave (the usual top-k or top-p), the first block draws
// from them and the other passes are saved.  Lists that would overflow (flat
// distributions) and rows without a filter are read from L2 again instead.
//
// Measured: one row of 128259 with every filter 12.8 us, the latency of three passes and their meetings; 256 rows
// of 131072 f32 with top-p 210 us (0.6 TB/s of logits), bound by the passes' instructions, 56 % of the issue slots.
#include <type_traits>

#include "serving.cuh"

namespace gg {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2 * kThreads, kCap = 256;
constexpr int kList = 896;                       // tokens of a warp's list at most, a multiple of 128
constexpr uint32_t kNone = 0x007fffffu;          // -inf's place in the order: every token above it is kept

// 0.995 * 2^32 * 2^-(j + 1/2) / 32, j = 0 .. 31: all weights are too small by one factor, which changes
// nothing, and stay below 2^32 with the series' up to 1.09 %.  Running products in double.
struct Table {
    uint32_t v[32];
    constexpr Table() : v() {
        double t = 0.995 * 0x1p32 * 0.98922801319397548;     // 2^(-1/64)
        for (int j = 0; j < 32; ++j, t *= 0.97857206208770009) v[j] = (uint32_t)(t + 0.5);   // 2^(-1/32)
    }
};
__device__ constexpr Table kTable;

template <int DT> struct El;
template <> struct El<GGUF_DT_F32> { using T = float; };
template <> struct El<GGUF_DT_F16> { using T = __half; };
template <> struct El<GGUF_DT_BF16> { using T = __nv_bfloat16; };
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// A float's bits in the order of its value (-0 as 0), and back.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

__device__ __forceinline__ uint2 ld_cluster2(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_cluster(uint32_t a, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// the larger of the two, NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Shared {
    float value[kWarps * kList];                         // the warps' lists: logits, and where in the warp's run
    uint16_t offset[kWarps * kList];
    uint32_t table[32 * 32];                             // kTable, a copy for each lane's bank
    alignas(8) uint32_t count[kBins], low[kBins], high[kBins];      // of a histogram: tokens, and their weights' sums
    uint32_t cand_key[kCap], cand_idx[kCap], n_cand;
    u64 cand_w[kCap], kept_w[kCap], cand_order[kCap];
    uint32_t cand_pos[kCap], cand_low[kCap], cand_high[kCap];
    u64 warp_sum[kWarps];
    uint32_t warp_count[kWarps];
    float warp_f[kWarps];
    // from each block of the cluster
    uint32_t peer_max[8], peer_bad[8], peer_lo[8], peer_hi[8], peer_listed[8];
    u64 peer_sum[3][8], peer_tail[8];
    // what one thread found, for all
    uint32_t bin, base_count, bin_count, all_count;
    u64 base_sum, all_sum;
    uint32_t K, I, lo, hi, bad, listed;
};

// f times W, exactly, rounded down or up; f in [0, 1)
__device__ __forceinline__ u64 share_of(float f, u64 W, bool up) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max(1, (int)(bits >> 23));
    const uint32_t mant = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);       // f = mant * 2^(e - 150)
    const u64 lo = W * mant, hi = __umul64hi(W, (u64)mant);
    const int sh = 150 - e;                                                         // 24 .. 149
    u64 v, rest;
    if (sh < 64) v = hi << (64 - sh) | lo >> sh, rest = lo << (64 - sh);
    else if (sh == 64) v = hi, rest = lo;
    else if (sh < 128) v = hi >> (sh - 64), rest = lo | hi << (128 - sh);
    else v = 0, rest = lo | hi;
    return v + (up && rest ? 1 : 0);
}


// seg: tokens of a warp, a multiple of 128; warp w of a row's cluster has those
// from index first + w * seg on.
template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int cluster, int seg) {
    using X = typename El<DT>::T;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    Shared& s = *reinterpret_cast<Shared*>(s_dyn);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int r = blockIdx.x / cluster;
    const X* x = static_cast<const X*>(p.x) + r * p.ld;
    const int first = -(int)((r * p.ld) & 3) + (rank * kWarps + warp) * seg;        // groups of four start at 8- or 16-byte boundaries
    const int V = p.vocab;
    if (cluster > 1) cluster_arrive_relaxed();       // waited for before the first access to another block
    for (int i = tid; i < 32 * 32; i += kThreads) s.table[i] = kTable.v[i >> 5];
    for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.low[i] = s.high[i] = 0;
    if (tid == 0) s.n_cand = 0, s.bad = 0, s.hi = 0, s.lo = 0xffffffffu, s.listed = 0;
    pdl_wait();
    pdl_launch_dependents();
    const float T = p.s.temperature ? p.s.temperature[r] : 1.f;
    int k = p.s.top_k ? p.s.top_k[r] : 0;
    float top_p = p.s.top_p ? p.s.top_p[r] : 1.f, min_p = p.s.min_p ? p.s.min_p[r] : 0.f;
    const float u = p.u[r];
    const bool greedy = T == 0.f;
    if (greedy) k = 1, top_p = 1.f, min_p = 0.f;
    const bool use_k = k > 0 && k < V, use_p = top_p < 1.f, use_m = min_p > 0.f;
    // log2 e / temperature in two floats (no doubles here: an SM does two of them a cycle)
    constexpr float kLog2eHigh = 1.44269502f, kLog2eLow = 1.92596299e-8f;
    const float quotient = greedy ? 0.f : kLog2eHigh / T;
    const bool two = T < INFINITY && quotient < 1e37f && !greedy;
    const float ch = fminf(quotient, 1e37f), cl = two ? (fmaf(-ch, T, kLog2eHigh) + kLog2eLow) / T : 0.f;

    // four tokens at `i` of the warp's run, -inf where the row has none
    struct alignas(4 * sizeof(X)) In { X v[4]; };
    auto load = [&](int i, float (&f)[4]) {
        const int v0 = first + i + 4 * lane;
        if (v0 >= 0 && v0 + 4 <= V) {
            const In in = *reinterpret_cast<const In*>(x + v0);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = to_f(in.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = v0 + j >= 0 && v0 + j < V ? to_f(x[v0 + j]) : -INFINITY;
        }
    };
    constexpr int kAhead = 4;                        // of those, on their way at once
    auto each_four = [&](auto&& f) {
        for (int i = 0; i < seg; i += 128 * kAhead) {
            float v[kAhead][4];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i + 128 * j < seg) load(i + 128 * j, v[j]);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (i + 128 * j < seg) f(v[j], i + 128 * j);
        }
    };

    // the maximum
    float top = -INFINITY;
    each_four([&](float (&f)[4], int) { top = max_nan(top, max_nan(max_nan(f[0], f[1]), max_nan(f[2], f[3]))); });
    const bool bad = !(T >= 0.f) || !(top < INFINITY);       // or NaN
    const uint32_t warp_key = __reduce_max_sync(0xffffffffu, bad ? kNone : key_of(top));
    __syncthreads();                                 // s.bad, s.hi are 0
    if (lane == 0) atomicMax(&s.hi, warp_key);
    if (bad) s.bad = 1;
    __syncthreads();
    uint32_t max_key = s.hi, any_bad = s.bad;
    if (cluster > 1) {
        cluster_wait_acquire();
        if (tid < cluster) {
            st_cluster(cluster_map(smem_u32(&s.peer_max[rank]), tid), max_key);
            st_cluster(cluster_map(smem_u32(&s.peer_bad[rank]), tid), any_bad);
        }
        cluster_sync_all();
        for (int b = 0; b < cluster; ++b) max_key = max(max_key, s.peer_max[b]), any_bad |= s.peer_bad[b];
    }
    if (any_bad || max_key <= kNone) {
        if (rank == 0 && tid == 0) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = NAN;
        }
        return;
    }
    const float m = float_of(max_key);
    const float bin_scale = 16.f * (greedy ? 1.4426950f : fminf(ch, 1e36f));
    float fine_scale = bin_scale;                    // of the histograms: all bins for what is listed
    const int less = V > (1 << 18) ? 32 - __clz(V - 1) - 18 : 0;         // V weights below 2^46 stay below 2^64
    const float last_grid = 393216.f + 46.f - max(less, 1);               // at most 63 bits are shifted off

    auto weight = [&](float v) -> u64 {
        const float dh = m - v, bb = dh - m, dl = (m - (dh - bb)) - (v + bb);          // m - v = dh + dl exactly
        const float grid = __fmaf_rn(dh, ch, 393216.f);  // 1.5 * 2^18: its last bit stands for 1 / 32
        if (!(grid < last_grid)) return 0;
        const float f = __fmaf_rn(dl, ch, __fmaf_rn(dh, cl, __fmaf_rn(dh, ch, -__fsub_rn(grid, 393216.f))));
        const float e = f * fmaf(f, fmaf(f, fmaf(f, 0.0096181291f, -0.055504109f), 0.24022651f), -0.69314718f);    // 2^-f - 1
        const uint32_t bits = __float_as_uint(grid), t = s.table[(bits & 31u) * 32 + lane];
        const float t28 = __uint_as_float(((t >> 8) & 0x7fffffu) | 0x4d000000u);       // t is 2^32 times the table's number: 2^28 ..
        const uint32_t d = __float_as_uint(fmaf(t28, e, 12582912.f)) - 0x4b400000u;    // .. times e, to the nearest integer
        return ((u64)(t + (d << 4)) << 32) >> (18u + ((bits >> 5) & 63u) + less);
    };
    auto bin_of = [&](float v) { return min(kBins - 1, (int)((m - v) * fine_scale)); };
    auto sync = [&] {
        if (cluster > 1) cluster_sync_all();
        else __syncthreads();
    };

    // counters 2 tid and 2 tid + 1 of all blocks, their loads on their way together
    auto pair_of_all = [&](uint32_t* counters, uint32_t (&sum)[2]) {
        uint2 v[8];
        if (cluster == 1) v[0] = *reinterpret_cast<const uint2*>(counters + 2 * tid);
#pragma unroll
        for (int b = 0; b < 8; ++b)
            if (cluster > 1 && b < cluster) v[b] = ld_cluster2(cluster_map(smem_u32(counters + 2 * tid), b));
        sum[0] = v[0].x, sum[1] = v[0].y;
#pragma unroll
        for (int b = 1; b < 8; ++b)
            if (b < cluster) sum[0] += v[b].x, sum[1] += v[b].y;
    };

    // The bounds: a token with (m - x) * bin_scale at `limit` or more is not kept.
    float limit = INFINITY;
    const bool tame = ch >= 1e-30f;                  // temperatures below 1e30, at which a distance that f32 has gives no weight
    const bool by_share = use_p && !use_k && top_p < 0.9999f && tame;
    if (greedy) {
        limit = 1e-37f;
    } else if (use_k || by_share) {
        each_four([&](float (&f)[4], int) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float b = (m - f[j]) * bin_scale;
                if (b < (float)(kBins - 1)) atomicAdd(&s.count[(int)b], 1u);
            }
        });
        sync();
        uint32_t n[2];
        pair_of_all(s.count, n);
        // the weights in the middle of the bins stand for their tokens'
        const float w0 = (float)n[0] * ex2(-(float)(2 * tid) * 0.0625f - 0.03125f), w1 = (float)n[1] * ex2(-(float)(2 * tid + 1) * 0.0625f - 0.03125f);
        uint32_t upto = n[0] + n[1];
        float mass = w0 + w1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            const float w = __shfl_up_sync(0xffffffffu, mass, o);
            if (lane >= o) upto += v, mass += w;
        }
        if (lane == 31) s.warp_count[warp] = upto, s.warp_f[warp] = mass;
        if (tid == 0) s.bin = kBins;
        __syncthreads();
        float all = 0.f;
        for (int v = 0; v < kWarps; ++v) {
            if (v < warp) upto += s.warp_count[v], mass += s.warp_f[v];
            all += s.warp_f[v];
        }
        if (use_k) {
            const uint32_t before = upto - n[0] - n[1];
            if (before < (uint32_t)k && upto >= (uint32_t)k) s.bin = 2 * tid + (before + n[0] < (uint32_t)k ? 1 : 0);
        } else {
            // Weights stand for themselves to a factor 2^(1/32) either way.  So where tokens have the share r, the bins up to
            // theirs have at most r q / (r q + 1 - r), q = 2^(1/16) = 1.04427.  1.0444 covers the rounding of a token's place in
            // the bins and the rest's (1e-5 and 4e-6 of the ratio of the two parts), 4e-6 that of these sums, some 25 operations deep.
            const float share = fmaxf(top_p, 0.f), heavy = 1.0444f * share, goal = heavy / (heavy + 1.f - share) * 1.000004f * all, before = mass - w0 - w1;
            if (before < goal && mass >= goal) s.bin = 2 * tid + (before + w0 < goal ? 1 : 0);
        }
        __syncthreads();
        if (s.bin < kBins - 1) limit = (float)(s.bin + 1);
    }
    if (use_m && !(use_p && (use_k || !tame))) limit = fminf(limit, 16.f * (0.01f - __log2f(fminf(min_p, 1.f))) + 1.f);

    // the tokens above the bounds, listed by warp in the row's order; the others' weights, for top-p
    bool listed = limit < INFINITY;
    float above = -INFINITY;                         // what is below is not kept
    int chunks = seg >> 7;                           // of 128 tokens
    float* const list = s.value + warp * kList;
    uint16_t* const offs = s.offset + warp * kList;
    u64 tail = 0;
    if (listed) {
        __syncthreads();                             // the warps' sums have been read
        const bool want_tail = use_p && !use_k;
        int n = 0;
        // The others' weights, which are at most 2^-below: an integer's sum is the same however the row is cut.  Each goes into
        // two, the first in units of 2^-(21 + below), the second in units 2^20 smaller with what rounding to the first has left.
        // So a weight is off by 2^-(42 + below) beside its own f32 rounding, and those of a whole vocabulary of 2^22 by
        // 2^-20 of a weight at the border.
        uint32_t rest = 0;
        int fine = 0;
        const int below = min((int)(limit * 0.0625f), 80);
        const float unit = __uint_as_float((uint32_t)(127 + 21 + below) << 23), unit2 = unit * 0x1p20f, farthest = 300.f / ch;
        // the same bound for the logits themselves, a little below
        above = fmaxf(m - limit / bin_scale - 1e-6f * (fabsf(m) + limit / bin_scale), -3.402823466e38f);
        each_four([&](float (&f)[4], int i) {
            bool in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                in[j] = f[j] >= above;
                if (want_tail) {
                    const float dh = fmaxf(f[j] - m, -farthest);     // where the weight is 0, and dh * cl still a number
                    const float w = in[j] ? 0.f : ex2(fmaf(dh, ch, dh * cl)), whole = fmaf(w, unit, 8388608.f);
                    rest += __float_as_uint(whole) - 0x4b000000u;
                    // 2^20 (2^23 - whole), exact, and 1.5 * 2^23 for the next one's integer
                    const float less_whole = fmaf(whole, -0x1p20f, 0x1p43f + 12582912.f);
                    fine += (int)(__float_as_uint(fmaf(w, unit2, less_whole)) - 0x4b400000u);
                }
            }
            if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) return;
            unsigned on[4];
            const unsigned lt = (1u << lane) - 1;
            int at = n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                on[j] = __ballot_sync(0xffffffffu, in[j]);
                at += __popc(on[j] & lt);
                n += __popc(on[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j]) {
                    if (at < kList) list[at] = f[j], offs[at] = (uint16_t)(i + 4 * lane + j);
                    ++at;
                }
        });
        if (n <= kList) {
            chunks = (n + 127) >> 7;
            for (int i = n + lane; i < 128 * chunks; i += 32) list[i] = -INFINITY, offs[i] = 0;
        }
        // below 2^32 in a lane: at most 1028 tokens of 2^21 and a half; of all tokens below 2^64, 2^22 of 2^41
        u64 sum = ((u64)rest << 20) + (u64)(int64_t)fine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s.warp_sum[warp] = sum, atomicAdd(&s.listed, n <= kList ? (uint32_t)n : 1u << 24);
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kWarps; ++w) s.warp_sum[0] += s.warp_sum[w];
            if (cluster == 1) s.peer_listed[0] = s.listed, s.peer_tail[0] = s.warp_sum[0];
        }
        __syncthreads();
    }
    // tokens above or at (K, I)
    uint32_t K = kNone, I = 0;                           // I: one past the last index kept of K's
    auto kept = [&](uint32_t key, int i) { return key > K || (key == K && (uint32_t)i < I); };
    auto four = [&](int i, float (&v)[4], int (&at)[4]) {
        if (listed) {
            const float4 a = *reinterpret_cast<const float4*>(list + i + 4 * lane);
            const ushort4 o = *reinterpret_cast<const ushort4*>(offs + i + 4 * lane);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            at[0] = first + o.x, at[1] = first + o.y, at[2] = first + o.z, at[3] = first + o.w;
        } else {
            load(i, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = v[j] >= above ? v[j] : -INFINITY, at[j] = first + i + 4 * lane + j;
        }
    };
    auto each = [&](auto&& f) {
        if (listed) {
            for (int i = 0; i < 128 * chunks; i += 128) {
                float v[4];
                int at[4];
                four(i, v, at);
#pragma unroll
                for (int j = 0; j < 4; ++j) f(v[j], at[j]);
            }
        } else {
            each_four([&](float (&v)[4], int i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) f(v[j] >= above ? v[j] : -INFINITY, first + i + 4 * lane + j);
            });
        }
    };
    auto add_weight = [&](int b, u64 w) {
        const uint32_t lo = (uint32_t)w, old = atomicAdd(&s.low[b], lo);
        const uint32_t up = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
        if (up) atomicAdd(&s.high[b], up);
    };
    // the first bin at which the count (the sum) reaches the goal, from the histograms of all blocks;
    // goal_of(all_count, all_sum).  Leaves s.bin = kBins where it never does.
    auto border = [&](bool by_sum, auto&& goal_of) {
        sync();
        uint32_t c[2];
        u64 w[2] = {0, 0};
        pair_of_all(s.count, c);
        if (by_sum) {
            const uint32_t* const low = s.low + 2 * tid;
            uint2 v[8];
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (b < cluster) v[b] = cluster > 1 ? ld_cluster2(cluster_map(smem_u32(low), b)) : *reinterpret_cast<const uint2*>(low);
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (b < cluster) w[0] += v[b].x, w[1] += v[b].y;
            uint32_t hi[2];
            pair_of_all(s.high, hi);
            w[0] += (u64)hi[0] << 32, w[1] += (u64)hi[1] << 32;
        }
        uint32_t ci = c[0] + c[1];
        u64 wi = w[0] + w[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t cv = __shfl_up_sync(0xffffffffu, ci, o);
            const u64 wv = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o) ci += cv, wi += wv;
        }
        if (lane == 31) s.warp_count[warp] = ci, s.warp_sum[warp] = wi;
        if (tid == 0) s.bin = kBins;
        __syncthreads();
        uint32_t call = 0;
        u64 wall = 0;
        for (int v = 0; v < kWarps; ++v) {
            if (v == warp) ci += call, wi += wall;
            call += s.warp_count[v], wall += s.warp_sum[v];
        }
        const u64 goal = goal_of(call, wall);
        uint32_t cb = ci - c[0] - c[1];
        u64 wb = wi - w[0] - w[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const u64 before = by_sum ? wb : cb, upto = by_sum ? wb + w[j] : cb + c[j];
            if (before < goal && upto >= goal) s.bin = 2 * tid + j, s.base_count = cb, s.base_sum = wb, s.bin_count = c[j];
            cb += c[j], wb += w[j];
        }
        if (tid == 0) s.all_count = call, s.all_sum = wall;
        __syncthreads();
        return goal;
    };
    // the tokens for which `in` holds, at most kCap, into the first block's list
    auto gather = [&](auto&& in) {
        const uint32_t counter = cluster_map(smem_u32(&s.n_cand), 0), keys = cluster_map(smem_u32(s.cand_key), 0),
                       idxs = cluster_map(smem_u32(s.cand_idx), 0);
        each([&](float v, int i) {
            const uint32_t key = key_of(v);
            if (key > kNone && in(v, key, i)) {
                const uint32_t to = add_cluster(counter, 1);
                if (to < kCap) {
                    st_cluster(keys + 4 * to, key);
                    st_cluster(idxs + 4 * to, (uint32_t)i);
                }
            }
        });
        sync();
    };
    // A sum over the n candidates j for each candidate, f(j, candidate, count, sum): several threads share one's, as many as
    // there are, and add their parts up in cand_pos, cand_low and cand_high.
    auto over_candidates = [&](int n, auto&& f) {
        int wide = 32;
        while (wide < n) wide *= 2;
        const int i = tid & (wide - 1), parts = kThreads / wide, per = (n + parts - 1) / parts, j0 = tid / wide * per, j1 = min(n, j0 + per);
        if (tid < n) s.cand_pos[tid] = s.cand_low[tid] = s.cand_high[tid] = 0;
        __syncthreads();
        if (i < n && j0 < j1) {
            uint32_t count = 0;
            u64 sum = 0;
#pragma unroll 4
            for (int j = j0; j < j1; ++j) f(j, i, count, sum);
            atomicAdd(&s.cand_pos[i], count);
            const uint32_t lo = (uint32_t)sum, old = atomicAdd(&s.cand_low[i], lo);
            atomicAdd(&s.cand_high[i], (uint32_t)(sum >> 32) + (old + lo < old ? 1u : 0u));
        }
        __syncthreads();
    };
    // in the first block: this thread's candidate's place in the order and the sum of weights up to it
    auto place = [&](int n, bool with_sum, uint32_t& key, uint32_t& idx, u64& w, int& pos, u64& upto) {
        key = 0, idx = 0, w = 0, pos = 0, upto = 0;
        if (tid < n) {
            key = s.cand_key[tid], idx = s.cand_idx[tid];
            s.cand_order[tid] = (u64)key << 32 | (uint32_t)~idx;        // the larger comes first
            s.cand_w[tid] = w = with_sum ? weight(float_of(key)) : 0;
        }
        over_candidates(n, [&](int j, int i, uint32_t& count, u64& sum) {
            const u64 o = s.cand_order[j], mine = s.cand_order[i];
            count += o > mine;
            sum += o >= mine ? s.cand_w[j] : 0;
        });
        if (tid < n) pos = (int)s.cand_pos[tid], upto = (u64)s.cand_high[tid] << 32 | s.cand_low[tid];
    };
    const u64 least = !use_m ? 0 : min_p < 1.f ? share_of(min_p, weight(m), true) : weight(m);     // min-p's, of a weight
    // the share of W that top-p keeps, the place in W that u asks for
    auto goal_of_p = [&](u64 W) { return max((u64)1, share_of(fmaxf(top_p, 0.f), W, true)); };
    auto target_of = [&](u64 W) { return u < 1.f ? share_of(u > 0.f ? u : 0.f, W, false) : u >= 1.f ? W - 1 : (u64)0; };
    // logprob to f32's rounding: near 0 from what the others have, else from the logit (an unlikely token's integer has few bits)
    auto emit = [&](int i, u64 w, u64 W, float v) {
        p.token[r] = i;
        if (!p.logprob) return;
        const float all = (float)W;
        p.logprob[r] = 2 * w > W ? log1pf(-((float)(W - w) / all)) : -((m - v) / T) - logf(all / (float)weight(m));
    };
    int round = 0;
    // the first index, in the vocabulary's order, at which the sum of f(value, index) passes goal_of(the whole sum)
    auto locate = [&](auto&& f, auto&& goal_of, auto&& found) {
        u64 sum = 0;
        each([&](float v, int i) { sum += f(v, i); });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();
        if (lane == 0) s.warp_sum[warp] = sum;
        __syncthreads();
        u64 all = 0, before = 0;
        for (int v = 0; v < kWarps; ++v) {
            if (v == warp) before = all;
            all += s.warp_sum[v];
        }
        u64* slot = s.peer_sum[round++];
        if (cluster > 1) {
            if (tid < cluster) st_cluster(cluster_map(smem_u32(&slot[rank]), tid), all);
        } else if (tid == 0) {
            slot[0] = all;
        }
        sync();
        u64 W = 0;
        for (int c = 0; c < cluster; ++c) {
            if (c == rank) before += W;
            W += slot[c];
        }
        const u64 goal = goal_of(W);
        if (!(goal >= before && goal - before < sum)) return;       // another warp's
        for (int i = 0; i < 128 * chunks; i += 128) {
            float v[4];
            int at[4];
            four(i, v, at);
            const u64 w[4] = {f(v[0], at[0]), f(v[1], at[1]), f(v[2], at[2]), f(v[3], at[3])};
            u64 upto = w[0] + w[1] + w[2] + w[3];
            const u64 own = upto;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += t;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + upto > goal);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    u64 b = before + upto - own;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (b <= goal && b + w[j] > goal) found(at[j], w[j], W, v[j]);
                        b += w[j];
                    }
                }
                return;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    };
    // From the candidates, which are all that may be kept: the filters and the draw.  limit: top-k, where it is still to be
    // applied; S: the sum that top-p takes its share of, or 0 for that of the top-k and `rest`.
    auto finish = [&](uint32_t limit, u64 S, u64 rest) {
        const int n = (int)s.n_cand;
        uint32_t key, idx;
        u64 w, upto;
        int pos;
        place(n, true, key, idx, w, pos, upto);
        bool keep = tid < n && (uint32_t)pos < limit;
        if (top_p < 1.f) {
            if (S == 0) {
                // the sum up to the last of the top-k
                const uint32_t last = min(limit, (uint32_t)n) - 1;
                if (tid < n && (uint32_t)pos == last) s.all_sum = upto;
                __syncthreads();
                S = s.all_sum + rest;
            }
            const u64 goal = goal_of_p(S);
            keep = keep && upto - w < goal;
        }
        keep = keep && w >= least;
        const u64 own = keep ? w : 0;
        u64 W = own;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
        if (tid < n) s.kept_w[tid] = own;
        if (lane == 0) s.warp_sum[warp] = W;
        // the sums in the vocabulary's order
        over_candidates(n, [&](int j, int i, uint32_t&, u64& sum) { sum += s.cand_idx[j] <= s.cand_idx[i] ? s.kept_w[j] : 0; });
        W = 0;
        for (int v = 0; v < kWarps; ++v) W += s.warp_sum[v];
        if (keep) {
            const u64 c = (u64)s.cand_high[tid] << 32 | s.cand_low[tid], t = target_of(W);
            if (c > t && c - w <= t) emit((int)idx, w, W, float_of(key));
        }
    };

    // Finds where the run ends that reaches the goal and puts (K, I) there; true where finish() has done the rest.
    auto select = [&](bool by_sum, auto&& goal_of, uint32_t limit, u64 rest) -> bool {
        each([&](float v, int i) {
            const uint32_t key = key_of(v);
            if (key > kNone && kept(key, i)) {
                const int b = bin_of(v);
                atomicAdd(&s.count[b], 1u);
                if (by_sum) add_weight(b, weight(v));
            }
        });
        u64 goal = border(by_sum, goal_of);
        const int b0 = (int)s.bin;
        if (b0 == kBins) return false;                   // the goal is past the row: all are kept
        const u64 all_sum = by_sum ? s.all_sum + rest : 0;
        if (s.base_count + s.bin_count <= kCap) {
            gather([&](float v, uint32_t key, int i) { return kept(key, i) && bin_of(v) <= b0; });
            if (rank == 0) finish(limit, all_sum, 0);
            return true;
        }
        uint32_t lo = 0, hi = 0xffffffffu;
        bool one_key = false, by_bin = true;
        u64 base_sum = s.base_sum;
        uint32_t base_count = s.base_count, n = s.bin_count;
        if (n > kCap) {
            // the bin's lowest and highest logit
            by_bin = false;
            if (tid == 0) s.lo = 0xffffffffu, s.hi = 0;
            __syncthreads();
            uint32_t a = 0xffffffffu, z = 0;
            each([&](float v, int i) {
                const uint32_t key = key_of(v);
                if (key > kNone && kept(key, i) && bin_of(v) == b0) a = min(a, key), z = max(z, key);
            });
            a = __reduce_min_sync(0xffffffffu, a), z = __reduce_max_sync(0xffffffffu, z);
            if (lane == 0) atomicMin(&s.lo, a), atomicMax(&s.hi, z);
            __syncthreads();
            if (cluster > 1) {
                if (tid < cluster) {
                    st_cluster(cluster_map(smem_u32(&s.peer_lo[rank]), tid), s.lo);
                    st_cluster(cluster_map(smem_u32(&s.peer_hi[rank]), tid), s.hi);
                }
            } else if (tid == 0) {
                s.peer_lo[0] = s.lo, s.peer_hi[0] = s.hi;
            }
            sync();
            lo = 0xffffffffu, hi = 0;
            for (int c = 0; c < cluster; ++c) lo = min(lo, s.peer_lo[c]), hi = max(hi, s.peer_hi[c]);
            // a round leaves at most a 2^10th of the span
            for (int step = 0; step < 4 && n > kCap && !one_key; ++step) {
                const uint32_t span = hi - lo;
                const int shift = max(0, 32 - __clz(span) - 10);         // at most kBins bins
                for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.low[i] = s.high[i] = 0;
                __syncthreads();
                each([&](float v, int i) {
                    const uint32_t key = key_of(v);
                    if (key >= lo && key <= hi && kept(key, i)) {
                        const int b = (int)((hi - key) >> shift);
                        atomicAdd(&s.count[b], 1u);
                        if (by_sum) add_weight(b, weight(v));
                    }
                });
                border(by_sum, [&](uint32_t, u64) { return goal - (by_sum ? base_sum : (u64)base_count); });
                const uint32_t b = s.bin;
                base_sum += s.base_sum, base_count += s.base_count, n = s.bin_count;
                hi -= b << shift;
                lo = max(lo, hi - ((1u << shift) - 1));
                one_key = shift == 0;
                sync();                                  // every block has read the histograms
            }
        }
        if (n <= kCap) {
            gather([&](float v, uint32_t key, int i) {
                return kept(key, i) && (by_bin ? bin_of(v) == b0 : key >= lo && key <= hi);
            });
            if (rank == 0) {
                uint32_t key, idx;
                u64 w, upto;
                int pos;
                place((int)n, by_sum, key, idx, w, pos, upto);
                const bool last = by_sum ? base_sum + upto >= goal && base_sum + upto - w < goal : base_count + pos + 1 == goal;
                if (tid < (int)n && last)
                    for (int c = 0; c < cluster; ++c) {
                        st_cluster(cluster_map(smem_u32(&s.K), c), key);
                        st_cluster(cluster_map(smem_u32(&s.I), c), idx + 1);
                    }
                if (tid == 0) s.n_cand = 0;
            }
        } else {
            // equal logits: so many of them, the lowest indices first
            const u64 w = by_sum ? weight(float_of(lo)) : 1;
            const u64 many = (goal - (by_sum ? base_sum : (u64)base_count) + w - 1) / w;
            locate([&](float v, int i) -> u64 { const uint32_t key = key_of(v); return key == lo && kept(key, i) ? 1 : 0; },
                   [&](u64) { return many - 1; },
                   [&](int i, u64, u64, float) {
                       for (int c = 0; c < cluster; ++c) {
                           st_cluster(cluster_map(smem_u32(&s.K), c), lo);
                           st_cluster(cluster_map(smem_u32(&s.I), c), (uint32_t)i + 1);
                       }
                   });
        }
        sync();
        K = s.K, I = s.I;
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.low[i] = s.high[i] = 0;
        __syncthreads();
        return false;
    };

    if (listed) {
        if (cluster > 1) {
            if (tid < cluster) {
                st_cluster(cluster_map(smem_u32(&s.peer_listed[rank]), tid), s.listed);
                st_cluster(cluster_map(smem_u32(&s.peer_tail[rank]), tid), s.warp_sum[0]);
            }
            sync();
        }
        uint32_t n = 0;
        u64 others = 0;
        for (int b = 0; b < cluster; ++b) n += s.peer_listed[b], others += s.peer_tail[b];
        // in weight()'s unit, 2^-46 / kTable's factor
        const u64 part = __umul64hi(others, (u64)(0.995 * 0.98922801319397548 * 0x1p64));
        const int down = min((int)(limit * 0.0625f), 80) + less - 5;
        tail = down >= 0 ? down < 64 ? part >> down : 0 : part << -down;
        if (n <= kCap) {
            gather([&](float, uint32_t, int) { return true; });
            if (rank == 0) finish(use_k ? (uint32_t)k : 0xffffffffu, 0, use_k ? 0 : tail);
            return;
        }
        // a list that is too long leaves the same tokens and the same rest to passes over the row
        if (n >= 1u << 24) listed = false, chunks = seg >> 7;
        else if (limit < (float)kBins) fine_scale = bin_scale * ((float)(kBins - 1) / limit);
    } else if (use_k || by_share) {
        sync();                                              // every block has read the counts
    }
    if (use_k || by_share) {
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
        __syncthreads();
    }
    if (use_k) {
        if (select(false, [&](uint32_t, u64) { return (u64)k; }, (uint32_t)k, 0)) return;
    }
    if (use_p) {
        if (use_k && K == kNone) {       // top-k left all: its counts are cleared once every block has read them
            sync();
            for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
            __syncthreads();
        }
        const u64 rest = use_k ? 0 : tail;
        if (select(true, [&](uint32_t, u64 all) { return goal_of_p(all + rest); }, 0xffffffffu, rest)) return;
    }
    locate([&](float v, int i) -> u64 {
        if (!kept(key_of(v), i)) return 0;
        const u64 w = weight(v);
        return w >= least ? w : 0;
    }, target_of, emit);
}

template <int DT>
cudaError_t launch(const SampleParams& p, int num_sms, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_once(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared), done);
    if (e != cudaSuccess) return e;
    // up to 2175 tokens a warp, of which its list holds two fifths; more blocks
    // to a row where there are few rows.  Always as many blocks as there may be: 37 rows of 32003 take 31.5 us and not 26.1,
    // 256 of 131072 242 and not 215; only what the lists ask for: 47 us, and one row of 128259 16.4 and not 13.0.  152064
    // tokens, 2385 a warp with four blocks: 64 rows take 129 us so and 84 with eight, 256 rows 229 and 250.
    const int64_t span = p.vocab + 3;
    int cluster = 1;
    while (cluster < 8 && (span > cluster * (int64_t)(kWarps * 2175) || (p.rows * cluster * 2 <= num_sms && span > cluster * 2048))) cluster *= 2;
    const int64_t seg = ceil_div(span, (int64_t)cluster * kWarps * 128) * 128;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<DT>, p, cluster, (int)seg);
}

}  // namespace

cudaError_t sample_launch(const SampleParams& p, int num_sms, int pdl, cudaStream_t s) {
    if (p.dt == GGUF_DT_F32) return launch<GGUF_DT_F32>(p, num_sms, pdl, s);
    return p.dt == GGUF_DT_F16 ? launch<GGUF_DT_F16>(p, num_sms, pdl, s) : launch<GGUF_DT_BF16>(p, num_sms, pdl, s);
}

}  // namespace gg
