// Draws a token from each row of logits, from given random numbers, after
// temperature, top-k, top-p and min-p, in one kernel that reads the logits once.
//
// All three filters keep a run of the tokens in falling order (of equal logits
// the lower index first), so together they keep the tokens before or at some (logit K,
// index I); the token drawn is the first in the vocabulary's order whose
// running sum of kept weights passes u times their sum.  Nothing is sorted.
//
// Which token that is must not hang on rounding: among 10^5 kept tokens a sum
// that is off by 10^-7 meets the wrong one once in a hundred rows.  So a
// weight 2^-z, z = (max - x) / temperature * log2 e, is taken to about 1e-10 of
// itself (z in two floats; a table of 2^-(j + 1/2)/256 and three terms of the
// series for the rest, as in Tang's table-driven exponential, ACM TOMS 1989) and
// becomes an integer of 46 bits.  Sums of integers do not depend on their order:
// the result is the same however the row is cut, and atomics add them up.
//
// A cluster of up to 8 blocks holds a row in its shared memory.  Where a
// filter's run ends is found by histograms: of z in sixteenths at first, then of
// ranges of the logits' bits, until the bin in which it ends has at most kCap
// tokens, which are compared with each other.  Where that many tokens are all
// that the filters can leave (the usual top-k or top-p), the first block draws
// from them and the other passes are saved.
#include <type_traits>

#include "serving.cuh"

namespace gg {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2 * kThreads, kCap = 256;
constexpr int kMaxSlice = 51200;                 // logits of a block: 200 KB
constexpr uint32_t kNone = 0x007fffffu;          // -inf's place in the order: every token above it is kept

// 2^46 * 2^-(j + 1/2) / 256, j = 0 .. 255; that all weights are 2^(-1/512) too small changes nothing.
// Running products in double: off by at most 256 * 2^-53.
struct Table {
    u64 v[256];
    constexpr Table() : v() {
        double t = 0x1p46 * 0.99864711289097017;         // 2^(-1/512)
        for (int j = 0; j < 256; ++j, t *= 0.99729605608547013) v[j] = (u64)(t + 0.5);   // 2^(-1/256)
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

// A float's bits in the order of its value, and back.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

__device__ __forceinline__ uint32_t ld_cluster(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
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

struct Shared {
    u64 table[256];
    uint32_t count[kBins], low[kBins], high[kBins];      // of a histogram: tokens, and their weights' sums
    uint32_t cand_key[kCap], cand_idx[kCap], n_cand;
    u64 cand_w[kCap], kept_w[kCap];
    u64 warp_sum[kWarps];
    uint32_t warp_count[kWarps];
    // from each block of the cluster
    uint32_t peer_max[8], peer_bad[8], peer_lo[8], peer_hi[8];
    u64 peer_sum[3][8];
    // what one thread found, for all
    uint32_t bin, base_count, bin_count, all_count;
    u64 base_sum, all_sum;
    uint32_t K, I, lo, hi, bad;
};

// logp of w of W, to f32's rounding also where it is near 0
__device__ __forceinline__ float log_share(u64 w, u64 W) {
    const float all = (float)W;
    return 2 * w > W ? log1pf(-((float)(W - w) / all)) : logf((float)w / all);
}

// seg: logits of a warp, a multiple of 128; block `rank` of a row's cluster holds
// 16 seg of them, from index first + rank * 16 seg on.
template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int cluster, int seg) {
    using X = typename El<DT>::T;
    extern __shared__ __align__(16) float s_x[];
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int r = blockIdx.x / cluster;
    const X* x = static_cast<const X*>(p.x) + r * p.ld;
    const int first = -(int)((r * p.ld) & 3) + rank * kWarps * seg;        // groups of four start at 8- or 16-byte boundaries
    const int V = p.vocab;
    if (cluster > 1) cluster_arrive_relaxed();       // waited for before the first access to another block
    if (tid < 256) s.table[tid] = kTable.v[tid];
    for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.low[i] = s.high[i] = 0;
    if (tid == 0) s.n_cand = 0, s.bad = 0, s.hi = 0, s.lo = 0xffffffffu;
    pdl_wait();
    pdl_launch_dependents();
    const float T = p.s.temperature ? p.s.temperature[r] : 1.f;
    int k = p.s.top_k ? p.s.top_k[r] : 0;
    float top_p = p.s.top_p ? p.s.top_p[r] : 1.f, min_p = p.s.min_p ? p.s.min_p[r] : 0.f;
    const float u = p.u[r];

    // the row, and its maximum
    float top = -INFINITY;
    bool bad = !(T >= 0.f);
    float* mine = s_x + warp * seg + 4 * lane;
    const int at0 = first + warp * seg + 4 * lane;
    struct alignas(4 * sizeof(X)) In { X v[4]; };
#pragma unroll 8
    for (int i = 0; i < seg; i += 128) {
        const int v0 = at0 + i;
        float f[4];
        if (v0 >= 0 && v0 + 4 <= V) {
            const In in = *reinterpret_cast<const In*>(x + v0);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = to_f(in.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = v0 + j >= 0 && v0 + j < V ? to_f(x[v0 + j]) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] += 0.f;                                 // -0 and 0 are equals
            bad |= !(f[j] < INFINITY);
            top = fmaxf(top, f[j]);
        }
        *reinterpret_cast<float4*>(mine + i) = make_float4(f[0], f[1], f[2], f[3]);
    }
    __syncthreads();
    {
        const uint32_t m = __reduce_max_sync(0xffffffffu, key_of(top));
        if (lane == 0) atomicMax(&s.hi, m);
        if (bad) s.bad = 1;
    }
    __syncthreads();
    if (cluster > 1) {
        cluster_wait_acquire();
        if (tid < cluster) {
            st_cluster(cluster_map(smem_u32(&s.peer_max[rank]), tid), s.hi);
            st_cluster(cluster_map(smem_u32(&s.peer_bad[rank]), tid), s.bad);
        }
        cluster_sync_all();
    } else {
        if (tid == 0) s.peer_max[0] = s.hi, s.peer_bad[0] = s.bad;
        __syncthreads();
    }
    uint32_t max_key = 0, any_bad = 0;
    for (int c = 0; c < cluster; ++c) max_key = max(max_key, s.peer_max[c]), any_bad |= s.peer_bad[c];
    if (any_bad || max_key <= kNone) {
        if (rank == 0 && tid == 0) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = NAN;
        }
        return;
    }
    const float m = float_of(max_key);
    const bool greedy = T == 0.f;
    if (greedy) k = 1, top_p = 1.f, min_p = 0.f;
    const double per = greedy ? 0.0 : 1.4426950408889634074 / (double)T;     // log2 e / temperature
    const float ch = per < 1e38 ? (float)per : 1e38f, cl = per < 1e38 ? (float)(per - (double)ch) : 0.f;
    const float bin_scale = 16.f * (greedy ? 1.4426950f : ch);
    const int less = V > (1 << 18) ? 1 : 0;              // V weights below 2^46 stay below 2^64

    auto weight = [&](float v) -> u64 {
        const float dh = m - v, bb = dh - m, dl = (m - (dh - bb)) - (v + bb);          // m - v = dh + dl exactly
        // not contracted: zl is what zh's own rounding left
        const float zh = __fmul_rn(dh, ch), zl = __fadd_rn(__fmaf_rn(dh, ch, -zh), __fmaf_rn(dh, cl, __fmul_rn(dl, ch)));
        if (!(zh < 62.f)) return 0;
        const float grid = __fadd_rn(zh, 49152.f);       // 1.5 * 2^15: its last bit stands for 1 / 256
        const float f = __fadd_rn(__fsub_rn(zh, __fsub_rn(grid, 49152.f)), zl);
        const float g = f * -0.69314718f;
        const float e = fmaf(g * g, fmaf(g, 0.16666667f, 0.5f), g);                    // 2^-f - 1
        const uint32_t bits = __float_as_uint(grid);
        const u64 t = s.table[bits & 255u];
        const float t31 = __uint_as_float(((uint32_t)(t >> 22) & 0x7fffffu) | 0x4e800000u);   // the same as 2^31 ..
        const int d = (int)(__float_as_uint(fmaf(t31, e, 12582912.f)) - 0x4b400000u);  // .. times e, to the nearest integer
        return (u64)((long long)t + (long long)d * 32768) >> (((bits >> 8) & 63u) + less);
    };
    auto bin_of = [&](float v) { return min(kBins - 1, (int)((m - v) * bin_scale)); };
    // tokens above or at (K, I)
    uint32_t K = kNone, I = 0;                           // I: one past the last index kept of K's
    auto kept = [&](uint32_t key, int i) { return key > K || (key == K && (uint32_t)i < I); };
    auto each = [&](auto&& f) {
        for (int i = 0; i < seg; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(mine + i);
            f(v.x, at0 + i), f(v.y, at0 + i + 1), f(v.z, at0 + i + 2), f(v.w, at0 + i + 3);
        }
    };
    auto add_weight = [&](int b, u64 w) {
        const uint32_t lo = (uint32_t)w, old = atomicAdd(&s.low[b], lo);
        const uint32_t up = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
        if (up) atomicAdd(&s.high[b], up);
    };
    auto sync = [&] {
        if (cluster > 1) cluster_sync_all();
        else __syncthreads();
    };
    // the first bin at which the count (the sum) reaches the goal, from the histograms of all blocks;
    // goal_of(all_count, all_sum).  Leaves s.bin = kBins where it never does.
    auto border = [&](bool by_sum, auto&& goal_of) {
        sync();
        uint32_t c[2] = {0, 0};
        u64 w[2] = {0, 0};
        for (int b = 0; b < cluster; ++b) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = 2 * tid + j;
                if (cluster > 1) {
                    c[j] += ld_cluster(cluster_map(smem_u32(&s.count[at]), b));
                    if (by_sum) w[j] += (u64)ld_cluster(cluster_map(smem_u32(&s.low[at]), b)) + ((u64)ld_cluster(cluster_map(smem_u32(&s.high[at]), b)) << 32);
                } else {
                    c[j] += s.count[at];
                    if (by_sum) w[j] += (u64)s.low[at] + ((u64)s.high[at] << 32);
                }
            }
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
    // in the first block: this thread's candidate's place in the order and the sum of weights up to it
    auto place = [&](int n, bool with_sum, uint32_t& key, uint32_t& idx, u64& w, int& pos, u64& upto) {
        key = 0, idx = 0, w = 0, pos = 0, upto = 0;
        if (tid < n) {
            key = s.cand_key[tid], idx = s.cand_idx[tid];
            if (with_sum) s.cand_w[tid] = w = weight(float_of(key));
        }
        __syncthreads();
        if (tid < n) {
            for (int j = 0; j < n; ++j) {
                const uint32_t kj = s.cand_key[j], ij = s.cand_idx[j];
                const bool before = kj > key || (kj == key && ij < idx);
                pos += before;
                if (with_sum) upto += before || j == tid ? s.cand_w[j] : 0;
            }
        }
    };
    // min-p as a key: x >= max + T ln(min_p), decided in double
    uint32_t min_key = 0;
    if (min_p > 0.f && T < INFINITY) {                   // at infinity all are equally likely
        const double least = (double)m + (double)T * log((double)fminf(min_p, 1.f));
        float f = (float)least;
        if ((double)f < least) f = nextafterf(f, INFINITY);
        min_key = key_of(f + 0.f);
    }
    const double uu = u > 0.f ? (double)u : 0.0;
    auto target_of = [&](u64 W) { return u >= 1.f ? W - 1 : min(W - 1, (u64)(uu * (double)W)); };
    auto emit = [&](int i, u64 w, u64 W) {
        p.token[r] = i;
        if (p.logprob) p.logprob[r] = log_share(w, W);
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
        for (int i = 0; i < seg; i += 128) {
            const float4 v = *reinterpret_cast<const float4*>(mine + i);
            const u64 w[4] = {f(v.x, at0 + i), f(v.y, at0 + i + 1), f(v.z, at0 + i + 2), f(v.w, at0 + i + 3)};
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
                    int j = 0;
                    while (b + w[j] <= goal) b += w[j++];
                    found(at0 + i + j, w[j], W);
                }
                return;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    };
    // From the candidates, which are all that may be kept: the filters and the draw.  limit: top-k, where it is still to be
    // applied; S: the sum that top-p takes its share of, or 0 for that of the top-k.
    auto finish = [&](uint32_t limit, u64 S) {
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
                S = s.all_sum;
            }
            const u64 goal = max((u64)1, (u64)ceil((double)fmaxf(top_p, 0.f) * (double)S));
            keep = keep && upto - w < goal;
        }
        keep = keep && key >= min_key;
        if (tid < n) s.kept_w[tid] = keep ? w : 0;
        __syncthreads();
        if (keep) {
            u64 c = 0, W = 0;
            for (int j = 0; j < n; ++j) {
                const u64 wj = s.kept_w[j];
                W += wj;
                if (s.cand_idx[j] <= idx) c += wj;
            }
            const u64 t = target_of(W);
            if (c > t && c - w <= t) emit((int)idx, w, W);
        }
    };

    // Finds where the run ends that reaches the goal and puts (K, I) there; true where finish() has done the rest.
    auto select = [&](bool by_sum, auto&& goal_of, uint32_t limit) -> bool {
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
        const u64 all_sum = by_sum ? s.all_sum : 0;
        if (s.base_count + s.bin_count <= kCap) {
            gather([&](float v, uint32_t key, int i) { return kept(key, i) && bin_of(v) <= b0; });
            if (rank == 0) finish(limit, all_sum);
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
                   [&](int i, u64, u64) {
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

    bool histograms_used = false;
    if (k > 0 && k < V) {
        if (select(false, [&](uint32_t, u64) { return (u64)k; }, (uint32_t)k)) return;
        histograms_used = K == kNone;
    }
    if (top_p < 1.f) {
        if (histograms_used) {       // top-k left all: its counts are cleared once every block has read them
            sync();
            for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
            __syncthreads();
        }
        if (select(true, [&](uint32_t, u64 all) { return max((u64)1, (u64)ceil((double)fmaxf(top_p, 0.f) * (double)all)); }, 0xffffffffu)) return;
    }
    if (min_key > K) K = min_key - 1, I = 0;             // everything at min_key and above, and nothing else
    locate([&](float v, int i) -> u64 { return kept(key_of(v), i) ? weight(v) : 0; }, target_of, emit);
}

template <int DT>
cudaError_t launch(const SampleParams& p, int num_sms, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_once(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 4, done);
    if (e != cudaSuccess) return e;
    // blocks of 64 KB, so that two to an SM overlap their loads with their passes;
    // more to a row where there are few rows
    const int64_t span = p.vocab + 3;
    int cluster = 1;
    while (cluster < 8 && (span > cluster * (int64_t)(16384) || (p.rows * cluster < num_sms && span > cluster * 2048))) cluster *= 2;
    const int64_t seg = ceil_div(span, (int64_t)cluster * kWarps * 128) * 128;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)seg * kWarps * sizeof(float);
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
