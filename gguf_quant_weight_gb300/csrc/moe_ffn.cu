// A few tokens through their experts' gated feed-forward, on the GGUF blocks:
//   y[t] = residual[t] + sum_s w[t][s] * Down_e( act(Gate_e x[t]) * Up_e x[t] ),  e = ids[t][s],
// in two kernels: gate, up and the activation; down, the weighted sum and the
// residual.  Unlike the decode GEMV, activations are not rounded to int8: what
// a routed row gives is accurate to f32's rounding (f32 and f16 outputs) or to
// f16's (bf16 outputs).
//
// The weights' bytes bound it, so an expert's blocks are read once for all of
// the batch's rows that it has: the tensor cores' m16n8k16 takes 16 weight rows
// as A and up to 8 columns of activations as B.  A's values are the blocks'
// integers, exact in f16: codes times their sub-block scale where the product
// is (Q2_K .. Q5_K: at most 31 * 63), summed over a block before its d is
// applied, codes alone otherwise (Q6_K, the 32-value types), summed over a
// scale's values.  B's columns are the activations scaled by a power of two per
// 256 of them; an f32 value takes two columns, its f16 rounding and what that
// left, so 22 bits of it.  Which values of a sub-block a lane holds is free as long
// as A and B agree: lane t of four has bytes 4t .. 4t+3 of each 16, and of
// those the even and the odd ones make its two pairs, which is how masks of
// 0x00ff00ff find them in a word of codes.
//
// Mins: sum_j m_j * (sum of sub-block j's activations) is one more product, of
// the mins (exact in f16) with the sums in two f16 parts.
#include <type_traits>

#include "formats.cuh"
#include "serving.cuh"

namespace gg {

namespace {

constexpr int kChunk = 256;                       // values of K a warp takes at a time
constexpr int kTiles = 2;                         // of 8 columns, at a time
constexpr int kColStride = 2 * kChunk + 64;       // bytes of a column in shared memory: 8 lanes' 16 bytes from 2 columns meet no bank twice
constexpr int kTileBytes = 8 * kColStride + 8 * 64 + 8 * 4;   // columns, their sums' parts, their scales
constexpr int kUpWarps = 8, kDownWarps = 24;      // kDownWarps: at most
constexpr size_t kDownSmem = 221184;              // beside the routes

// ---------------------------------------------------------------- the experts' rows

// What each block makes of the ids: the experts with rows, and the rows
// (entries token * top_k + slot) of each.  The order of an expert's rows is
// whatever the atomics give; a row's result does not depend on its column.
struct Routes {
    int n_active;
    int start[kMoeFfnExperts + 1];     // first of expert e's rows in list
    int cursor[kMoeFfnExperts];
    uint16_t active[kMoeFfnRows];   // experts with rows, in order
    uint16_t list[kMoeFfnRows];
};

__device__ void make_routes(Routes& r, const int32_t* ids, int entries, int n_expert, int tid, int threads) {
    for (int e = tid; e < n_expert; e += threads) r.cursor[e] = 0;
    __syncthreads();
    for (int i = tid; i < entries; i += threads) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)n_expert) atomicAdd(&r.cursor[e], 1);
    }
    __syncthreads();
    if (tid < 32) {
        int rows = 0, act = 0;
        for (int b = 0; b < n_expert; b += 32) {
            const int e = b + tid, c = e < n_expert ? r.cursor[e] : 0;
            int sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (tid >= o) sum += v;
            }
            const unsigned on = __ballot_sync(0xffffffffu, c > 0);
            if (e < n_expert) r.start[e] = r.cursor[e] = rows + sum - c;
            if (c > 0) r.active[act + __popc(on & ((1u << tid) - 1))] = (uint16_t)e;
            rows += __shfl_sync(0xffffffffu, sum, 31);
            act += __popc(on);
        }
        if (tid == 0) r.n_active = act, r.start[n_expert] = rows;
    }
    __syncthreads();
    for (int i = tid; i < entries; i += threads) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)n_expert) r.list[atomicAdd(&r.cursor[e], 1)] = (uint16_t)i;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- B: the activations

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

// Four consecutive activations as f32.
__device__ __forceinline__ void load4(const void* p, int dt, int64_t i, float (&f)[4]) {
    if (dt == GGUF_DT_F32) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        if (dt == GGUF_DT_F16) {
            const float2 a = unpack2(v.x), b = unpack2(v.y);
            f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
        } else {
            f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
            f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
        }
    }
}

// One row's values [base, base + 32 * nsub) into column `col` of the warp's
// tiles (and, with two parts, the column after it).  The whole warp calls it.
__device__ __forceinline__ void stage_row(uint8_t* tiles, int col, int parts, const void* x, int dt, int64_t base, int nsub,
                                          int lane) {
    const int j = lane >> 2, t = lane & 3;
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    if (j < nsub) {
        load4(x, dt, base + 32 * j + 4 * t, a);
        load4(x, dt, base + 32 * j + 16 + 4 * t, b);
    }
    // the largest finite magnitude goes to [2^9, 2^10): products and their sums stay
    // far inside f32, and what f16 rounds off is relative to it
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float u = fabsf(a[i]), v = fabsf(b[i]);
        big = fmaxf(big, fmaxf(u < INFINITY ? u : 0.f, v < INFINITY ? v : 0.f));
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));   // of magnitudes, whose bits are in their order
    // powers of two by their bits, both of them normal numbers
    const int ex = max((int)(top >> 23), 10);
    const float scale = __uint_as_float((uint32_t)(263 - ex) << 23), back = __uint_as_float((uint32_t)(ex - 9) << 23);
    float sa = 0.f, sb = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] *= scale, b[i] *= scale;
        sa += a[i], sb += b[i];
    }
    uint8_t* tile = tiles + (col >> 3) * kTileBytes;
    const int c = col & 7;
    uint4 hi;
    hi.x = pack2(a[0], a[2]), hi.y = pack2(a[1], a[3]), hi.z = pack2(b[0], b[2]), hi.w = pack2(b[1], b[3]);
    *reinterpret_cast<uint4*>(tile + c * kColStride + j * 64 + t * 16) = hi;
    sa += __shfl_xor_sync(0xffffffffu, sa, 1), sb += __shfl_xor_sync(0xffffffffu, sb, 1);
    sa += __shfl_xor_sync(0xffffffffu, sa, 2), sb += __shfl_xor_sync(0xffffffffu, sb, 2);
    __half* sums = reinterpret_cast<__half*>(tile + 8 * kColStride + c * 64);    // [hi 16][lo 16]
    float* scales = reinterpret_cast<float*>(tile + 8 * kColStride + 8 * 64);
    if (t == 0) {
        const uint32_t h = pack2(sa, sb);
        const float2 f = unpack2(h);
        *reinterpret_cast<uint32_t*>(sums + 2 * j) = h;
        *reinterpret_cast<uint32_t*>(sums + 16 + 2 * j) = pack2(sa - f.x, sb - f.y);
    }
    if (lane == 0) scales[c] = back;
    if (parts == 2) {
        // a multiple of two columns to a tile: the next column is in the same one
        float2 f = unpack2(hi.x);
        uint4 lo;
        lo.x = pack2(a[0] - f.x, a[2] - f.y);
        f = unpack2(hi.y), lo.y = pack2(a[1] - f.x, a[3] - f.y);
        f = unpack2(hi.z), lo.z = pack2(b[0] - f.x, b[2] - f.y);
        f = unpack2(hi.w), lo.w = pack2(b[1] - f.x, b[3] - f.y);
        *reinterpret_cast<uint4*>(tile + (c + 1) * kColStride + j * 64 + t * 16) = lo;
        if (t == 0) {       // the first column has the whole sums
            *reinterpret_cast<uint32_t*>(sums + 32 + 2 * j) = 0u;
            *reinterpret_cast<uint32_t*>(sums + 48 + 2 * j) = 0u;
        }
        if (lane == 0) scales[c + 1] = back;
    }
}

// ---------------------------------------------------------------- A: the blocks

__device__ __forceinline__ uint32_t ld32(const uint8_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); }
__device__ __forceinline__ uint32_t ld16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint16_t*>(p)); }
// a word at a 2-byte boundary
__device__ __forceinline__ uint32_t ld32h(const uint8_t* p) { return ld16(p) | ld16(p + 2) << 16; }

__host__ __device__ constexpr bool int_scaled(int qt) {
    return qt == GGUF_Q2_K || qt == GGUF_Q3_K || qt == GGUF_Q4_K || qt == GGUF_Q5_K;
}
__host__ __device__ constexpr bool has_min(int qt) {
    return qt == GGUF_Q2_K || qt == GGUF_Q4_K || qt == GGUF_Q5_K || b32_has_min(qt);
}
// what is subtracted from a code
__host__ __device__ constexpr int zero_point(int qt) {
    return qt == GGUF_Q6_K ? 32 : qt == GGUF_Q3_K ? 4 : qt == GGUF_Q8_0 ? 128 : block32(qt) ? b32_zero_point(qt) : 0;
}

// 256 values of one weight row as lane t of four holds them.  load(): row, the
// row's first byte; c, the chunk; nsub, how many of its 32-value groups exist
// (fewer than 8 at the end of a row of 32-value blocks).
template <int QT> struct Raw;

template <> struct Raw<GGUF_Q4_K> {
    uint32_t w[4][2];
    uint4 head;         // d, dmin, scales
    __device__ __forceinline__ void load(const uint8_t* row, int64_t c, int, int t) {
        const uint8_t* b = row + c * 144;
        head = __ldg(reinterpret_cast<const uint4*>(b));
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p][0] = ld32(b + 16 + 32 * p + 4 * t), w[p][1] = ld32(b + 32 + 32 * p + 4 * t);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const { return (w[j >> 1][half] >> (4 * (j & 1))) & 0x0f0f0f0fu; }
};
template <> struct Raw<GGUF_Q5_K> {
    uint32_t w[4][2], h[2];
    uint4 head;
    __device__ __forceinline__ void load(const uint8_t* row, int64_t c, int, int t) {
        const uint8_t* b = row + c * 176;
        head = __ldg(reinterpret_cast<const uint4*>(b));
        h[0] = ld32(b + 16 + 4 * t), h[1] = ld32(b + 32 + 4 * t);
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p][0] = ld32(b + 48 + 32 * p + 4 * t), w[p][1] = ld32(b + 64 + 32 * p + 4 * t);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const {
        const uint32_t high = j < 4 ? h[half] << (4 - j) : h[half] >> (j - 4);
        return ((w[j >> 1][half] >> (4 * (j & 1))) & 0x0f0f0f0fu) | (high & 0x10101010u);
    }
};
template <> struct Raw<GGUF_Q6_K> {
    uint32_t ql[4][2], qh[2][2], sc[4], d;
    __device__ __forceinline__ void load(const uint8_t* row, int64_t c, int, int t) {
        const uint8_t* b = row + c * 210;
#pragma unroll
        for (int p = 0; p < 4; ++p) ql[p][0] = ld32h(b + 32 * p + 4 * t), ql[p][1] = ld32h(b + 32 * p + 16 + 4 * t);
#pragma unroll
        for (int p = 0; p < 2; ++p) qh[p][0] = ld32h(b + 128 + 32 * p + 4 * t), qh[p][1] = ld32h(b + 144 + 32 * p + 4 * t);
#pragma unroll
        for (int p = 0; p < 4; ++p) sc[p] = ld32h(b + 192 + 4 * p);
        d = ld16(b + 208);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const {
        const int h = j >> 2, g = j & 3;
        const uint32_t low = (ql[2 * h + (g & 1)][half] >> (4 * (g >> 1))) & 0x0f0f0f0fu;
        const uint32_t high = g < 2 ? qh[h][half] << (4 - 2 * g) : qh[h][half] >> (2 * g - 4);
        return low | (high & 0x30303030u);
    }
};
template <> struct Raw<GGUF_Q2_K> {
    uint32_t w[2][2], sc[4], dm;
    __device__ __forceinline__ void load(const uint8_t* row, int64_t c, int, int t) {
        const uint8_t* b = row + c * 84;
#pragma unroll
        for (int p = 0; p < 4; ++p) sc[p] = ld32(b + 4 * p);
#pragma unroll
        for (int p = 0; p < 2; ++p) w[p][0] = ld32(b + 16 + 32 * p + 4 * t), w[p][1] = ld32(b + 32 + 32 * p + 4 * t);
        dm = ld32(b + 80);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const { return (w[j >> 2][half] >> (2 * (j & 3))) & 0x03030303u; }
};
template <> struct Raw<GGUF_Q3_K> {
    uint32_t w[2][2], h[2], sc[3], d;
    __device__ __forceinline__ void load(const uint8_t* row, int64_t c, int, int t) {
        const uint8_t* b = row + c * 110;
        h[0] = ld32h(b + 4 * t), h[1] = ld32h(b + 16 + 4 * t);
#pragma unroll
        for (int p = 0; p < 2; ++p) w[p][0] = ld32h(b + 32 + 32 * p + 4 * t), w[p][1] = ld32h(b + 48 + 32 * p + 4 * t);
#pragma unroll
        for (int p = 0; p < 3; ++p) sc[p] = ld32h(b + 96 + 4 * p);
        d = ld16(b + 108);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const {
        const uint32_t high = j < 2 ? h[half] << (2 - j) : h[half] >> (j - 2);
        return ((w[j >> 2][half] >> (2 * (j & 3))) & 0x03030303u) | (high & 0x04040404u);
    }
    // its sixteen scales of six bits, less 32, as four words of signed bytes (i = 4 p + byte)
    __device__ __forceinline__ uint32_t scales(int p) const {
        const uint32_t low = (sc[p & 1] >> (4 * (p >> 1))) & 0x0f0f0f0fu, high = (sc[2] >> (2 * p)) & 0x03030303u;
        return low | high << 4;
    }
};
// the 32-value types: a block to a 32-value group
template <int QT> struct Raw {
    static constexpr int BB = block_bytes(QT), WORDS = QT == GGUF_Q8_0 ? 2 : 1;
    uint32_t w[8][WORDS], qh[b32_has_qh(QT) ? 8 : 1], d[8];      // d: d and, where there is one, m above it
    __device__ __forceinline__ void load(const uint8_t* row, int64_t c, int nsub, int t) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint8_t* b = row + (c * 8 + min(j, nsub - 1)) * BB;
            if constexpr (QT == GGUF_Q8_0) {
                w[j][0] = ld32h(b + 2 + 4 * t), w[j][1] = ld32h(b + 18 + 4 * t);
            } else if constexpr (BB % 4 == 0) {
                w[j][0] = ld32(b + b32_qs_offset(QT) + 4 * t);
                if constexpr (b32_has_qh(QT)) qh[j] = ld32(b + b32_qs_offset(QT) - 4);
            } else {
                w[j][0] = ld32h(b + b32_qs_offset(QT) + 4 * t);
                if constexpr (b32_has_qh(QT)) qh[j] = ld32h(b + b32_qs_offset(QT) - 4);
            }
            d[j] = b32_has_min(QT) ? ld32(b) : ld16(b);
        }
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int t) const {
        if constexpr (QT == GGUF_Q8_0) {
            return w[j][half] ^ 0x80808080u;
        } else {
            uint32_t c = (w[j][0] >> (4 * half)) & 0x0f0f0f0fu;
            if constexpr (b32_has_qh(QT)) {
                // bits 16 half + 4 t .. + 3, one to a byte: bit i times 2^7i lands on bit 8i, and no other product does
                const uint32_t four = (qh[j] >> (16 * half + 4 * t)) & 15u;
                c |= ((four * 0x00204081u) & 0x01010101u) << 4;
            }
            return c;
        }
    }
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
// byte i of a word twice over, as the f16 numbers 1024 + byte
__device__ __forceinline__ __half2 byte_h2(uint32_t w, int i) { return as_h2(__byte_perm(w, 0x64646464u, 0x4040 | i | i << 8)); }
__device__ __forceinline__ float f16_low(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v & 0xffffu))); }
__device__ __forceinline__ float f16_high(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v >> 16))); }

// The 6-bit scales (lo, hi of four) and mins of Q4_K / Q5_K as words of bytes.
__device__ __forceinline__ void six_bits(const uint4& head, uint32_t (&sc)[2], uint32_t (&mn)[2]) {
    sc[0] = head.y & 0x3f3f3f3fu;
    mn[0] = head.z & 0x3f3f3f3fu;
    sc[1] = (head.w & 0x0f0f0f0fu) | ((head.y >> 2) & 0x30303030u);
    mn[1] = ((head.w >> 4) & 0x0f0f0f0fu) | ((head.z >> 2) & 0x30303030u);
}

// acc[tile] += (16 weight rows x 256 values) * (the tile's columns).  r[0], r[1]:
// the rows lane / 4 and lane / 4 + 8.
template <int QT>
__device__ __forceinline__ void multiply(const Raw<QT> (&r)[2], const uint8_t* tiles, int n_tiles, int nsub, int lane,
                                         float (&acc)[kTiles][4]) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* col = tiles + g * kColStride + t * 16;
    constexpr int Z = 1024 + zero_point(QT);
    float total[kTiles][4] = {};
    uint32_t sc[2][4], mn[2][4];        // by row: scales and mins as bytes
    float d[2], dmin[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        d[i] = 1.f, dmin[i] = 1.f;
        if constexpr (QT == GGUF_Q4_K || QT == GGUF_Q5_K) {
            uint32_t s[2], m[2];
            six_bits(r[i].head, s, m);
            sc[i][0] = s[0], sc[i][1] = s[1], mn[i][0] = m[0], mn[i][1] = m[1];
            d[i] = f16_low(r[i].head.x), dmin[i] = f16_high(r[i].head.x);
        } else if constexpr (QT == GGUF_Q2_K) {
#pragma unroll
            for (int p = 0; p < 4; ++p) sc[i][p] = r[i].sc[p] & 0x0f0f0f0fu, mn[i][p] = (r[i].sc[p] >> 4) & 0x0f0f0f0fu;
            d[i] = f16_low(r[i].dm), dmin[i] = f16_high(r[i].dm);
        } else if constexpr (QT == GGUF_Q3_K) {
#pragma unroll
            for (int p = 0; p < 4; ++p) sc[i][p] = r[i].scales(p);
            d[i] = f16_low(r[i].d);
        } else if constexpr (QT == GGUF_Q6_K) {
            d[i] = f16_low(r[i].d);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (block32(QT) && j >= nsub) break;
        uint4 b[kTiles];
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
            if (n < n_tiles) b[n] = *reinterpret_cast<const uint4*>(col + n * kTileBytes + j * 64);
        float part[kTiles][4] = {};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t c = r[i].codes(j, half, t);
                const __half2 even = as_h2((c & 0x00ff00ffu) | 0x64006400u), odd = as_h2(((c >> 8) & 0x00ff00ffu) | 0x64006400u);
                if constexpr (int_scaled(QT)) {
                    // (1024 + code) * scale - (1024 + zero point) * scale, one exact operation
                    constexpr bool wide = QT == GGUF_Q4_K || QT == GGUF_Q5_K;
                    const int s = wide ? j : 2 * j + half;
                    constexpr int bias = QT == GGUF_Q3_K ? 1024 + 32 : 1024;
                    const __half2 scale = __hsub2(byte_h2(sc[i][s >> 2], s & 3), __float2half2_rn((float)bias));
                    // (1024 + 4) * scale leaves f16's exact integers for the 6-bit scales of Q3_K: its codes lose their 4 first
                    if constexpr (QT == GGUF_Q3_K) {
                        a[i] = as_u32(__hmul2(__hsub2(even, __float2half2_rn((float)Z)), scale));
                        a[i + 2] = as_u32(__hmul2(__hsub2(odd, __float2half2_rn((float)Z)), scale));
                    } else {
                        const __half2 less = __hmul2(scale, __float2half2_rn(-1024.f));
                        a[i] = as_u32(__hfma2(even, scale, less));
                        a[i + 2] = as_u32(__hfma2(odd, scale, less));
                    }
                } else {
                    a[i] = as_u32(__hsub2(even, __float2half2_rn((float)Z)));
                    a[i + 2] = as_u32(__hsub2(odd, __float2half2_rn((float)Z)));
                }
            }
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                if (n >= n_tiles) continue;
                const uint32_t b0 = half ? b[n].z : b[n].x, b1 = half ? b[n].w : b[n].y;
                if constexpr (int_scaled(QT)) {
                    mma(total[n], a, b0, b1);
                } else if constexpr (QT == GGUF_Q6_K) {
                    float one[4] = {};
                    mma(one, a, b0, b1);
                    const int s = 2 * j + half;
                    const float s0 = (float)(int8_t)(r[0].sc[s >> 2] >> (8 * (s & 3))), s1 = (float)(int8_t)(r[1].sc[s >> 2] >> (8 * (s & 3)));
                    total[n][0] = fmaf(one[0], s0, total[n][0]);
                    total[n][1] = fmaf(one[1], s0, total[n][1]);
                    total[n][2] = fmaf(one[2], s1, total[n][2]);
                    total[n][3] = fmaf(one[3], s1, total[n][3]);
                } else {
                    mma(part[n], a, b0, b1);
                }
            }
        }
        if constexpr (block32(QT)) {
            const float d0 = f16_low(r[0].d[j]), d1 = f16_low(r[1].d[j]);
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                total[n][0] = fmaf(part[n][0], d0, total[n][0]);
                total[n][1] = fmaf(part[n][1], d0, total[n][1]);
                total[n][2] = fmaf(part[n][2], d1, total[n][2]);
                total[n][3] = fmaf(part[n][3], d1, total[n][3]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
        if (n >= n_tiles) continue;
        const uint8_t* tile = tiles + n * kTileBytes;
        const float2 back = *reinterpret_cast<const float2*>(tile + 8 * kColStride + 8 * 64 + 8 * t);
        if constexpr (has_min(QT)) {
            // sums 2t, 2t + 1 of the first eight 16-value groups, then of the others
            float low[4] = {};
            const uint8_t* sums = tile + 8 * kColStride + g * 64 + 4 * t;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t a[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (QT == GGUF_Q2_K) {
                        const uint32_t two = ((t < 2 ? mn[i][2 * k] : mn[i][2 * k + 1]) >> (16 * (t & 1))) & 0xffffu;
                        a[i] = as_u32(__hsub2(as_h2((two & 0xffu) | (two & 0xff00u) << 8 | 0x64006400u), __float2half2_rn(1024.f)));
                    } else if constexpr (block32(QT)) {
                        // group 4k + t's m: no register is indexed by a lane
                        const uint32_t m = t < 2 ? (t ? r[i].d[4 * k + 1] : r[i].d[4 * k]) : (t == 2 ? r[i].d[4 * k + 2] : r[i].d[4 * k + 3]);
                        const bool in = 4 * k + t < nsub;
                        a[i] = in ? __byte_perm(m, 0u, 0x3232) : 0u;
                    } else {
                        const uint32_t m = (mn[i][k] >> (8 * t)) & 0xffu;
                        a[i] = as_u32(__hsub2(as_h2(m * 0x00010001u | 0x64006400u), __float2half2_rn(1024.f)));
                    }
                    a[i + 2] = a[i];        // with the sums' first part and their second
                }
                mma(low, a, *reinterpret_cast<const uint32_t*>(sums + 16 * k), *reinterpret_cast<const uint32_t*>(sums + 32 + 16 * k));
            }
            const float sign = block32(QT) ? 1.f : -1.f;    // Q4_1, Q5_1 add their m
            total[n][0] = fmaf(sign * dmin[0], low[0], d[0] * total[n][0]);
            total[n][1] = fmaf(sign * dmin[0], low[1], d[0] * total[n][1]);
            total[n][2] = fmaf(sign * dmin[1], low[2], d[1] * total[n][2]);
            total[n][3] = fmaf(sign * dmin[1], low[3], d[1] * total[n][3]);
            acc[n][0] = fmaf(total[n][0], back.x, acc[n][0]);
            acc[n][1] = fmaf(total[n][1], back.y, acc[n][1]);
            acc[n][2] = fmaf(total[n][2], back.x, acc[n][2]);
            acc[n][3] = fmaf(total[n][3], back.y, acc[n][3]);
        } else {
            acc[n][0] = fmaf(d[0] * total[n][0], back.x, acc[n][0]);
            acc[n][1] = fmaf(d[0] * total[n][1], back.y, acc[n][1]);
            acc[n][2] = fmaf(d[1] * total[n][2], back.x, acc[n][2]);
            acc[n][3] = fmaf(d[1] * total[n][3], back.y, acc[n][3]);
        }
    }
}

// The rows at and after `n` of a matrix's last 16 stand for its last row (their results are dropped).
template <int QT>
__device__ __forceinline__ void load_rows(Raw<QT> (&r)[2], const uint8_t* w, int64_t row0, int64_t n, int64_t rb, int64_t c, int nsub,
                                          int lane) {
    const int g = lane >> 2, t = lane & 3;
    r[0].load(w + min(row0 + g, n - 1) * rb, c, nsub, t);
    r[1].load(w + min(row0 + g + 8, n - 1) * rb, c, nsub, t);
}

// f(QT) for a type known at run time only
template <class F>
__device__ __forceinline__ void with_type(int qt, F&& f) {
    switch (qt) {
        case GGUF_Q4_0: f(std::integral_constant<int, GGUF_Q4_0>{}); break;
        case GGUF_Q4_1: f(std::integral_constant<int, GGUF_Q4_1>{}); break;
        case GGUF_Q5_0: f(std::integral_constant<int, GGUF_Q5_0>{}); break;
        case GGUF_Q5_1: f(std::integral_constant<int, GGUF_Q5_1>{}); break;
        case GGUF_Q8_0: f(std::integral_constant<int, GGUF_Q8_0>{}); break;
        case GGUF_Q2_K: f(std::integral_constant<int, GGUF_Q2_K>{}); break;
        case GGUF_Q3_K: f(std::integral_constant<int, GGUF_Q3_K>{}); break;
        case GGUF_Q4_K: f(std::integral_constant<int, GGUF_Q4_K>{}); break;
        case GGUF_Q5_K: f(std::integral_constant<int, GGUF_Q5_K>{}); break;
        default: f(std::integral_constant<int, GGUF_Q6_K>{}); break;
    }
}

__device__ __forceinline__ float activate(float a, int act) {
    if (act == GGUF_ACT_SILU) return a / (1.f + expf(-a));
    // tanh form: 0.79788... = sqrt(2 / pi)
    return 0.5f * a * (1.f + tanhf(0.79788456080286536f * (a + 0.044715f * a * a * a)));
}

// ---------------------------------------------------------------- gate, up, activation

// Block (x, y): rows 16 x .. of gate and up, of the y-th expert that has rows.
// Its warps take the chunks of K in turn; their sums meet in shared memory.
// QT: both matrices' type, or -1 where they differ.
template <int QT>
__global__ void __launch_bounds__(32 * kUpWarps, QT < 0 ? 2 : 3) moe_ffn_up_kernel(const MoeFfnParams p) {
    extern __shared__ __align__(16) uint8_t s_tiles[];      // a warp's tiles, then its sums
    __shared__ Routes s_routes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    make_routes(s_routes, p.ids, p.T * p.top_k, p.n_expert, tid, 32 * kUpWarps);
    if ((int)blockIdx.y >= s_routes.n_active) return;
    const int e = s_routes.active[blockIdx.y], first = s_routes.start[e], rows = s_routes.start[e + 1] - first;
    const int64_t row0 = 16 * (int64_t)blockIdx.x;
    const uint8_t* gate = p.gate + e * p.F * p.gate_rb;
    const uint8_t* up = p.up + e * p.F * p.up_rb;
    const int parts = p.x_parts, chunks = (int)ceil_div(p.K, kChunk);
    const int at_once = 8 * p.tiles / parts;                // rows
    uint8_t* tiles = s_tiles + warp * p.tiles * kTileBytes;
    float* sums = reinterpret_cast<float*>(s_tiles);        // [warp][matrix][16 rows][16 columns]
    for (int r0 = 0; r0 < rows; r0 += at_once) {
        const int n = min(at_once, rows - r0), n_tiles = (n * parts + 7) >> 3;
        float a[2][kTiles][4] = {};
        for (int c = warp; c < chunks; c += kUpWarps) {
            const int nsub = (int)min((int64_t)8, (p.K - (int64_t)c * kChunk) / 32);
            auto stage = [&] {
                __syncwarp();
                for (int i = 0; i < n; ++i) {
                    const int token = s_routes.list[first + r0 + i] / p.top_k;
                    stage_row(tiles, i * parts, parts, p.x, p.xdt, token * p.K + (int64_t)c * kChunk, nsub, lane);
                }
                __syncwarp();
            };
            if constexpr (QT >= 0) {
                Raw<QT> rg[2], ru[2];
                load_rows<QT>(rg, gate, row0, p.F, p.gate_rb, c, nsub, lane);
                load_rows<QT>(ru, up, row0, p.F, p.up_rb, c, nsub, lane);
                stage();
                multiply<QT>(rg, tiles, n_tiles, nsub, lane, a[0]);
                multiply<QT>(ru, tiles, n_tiles, nsub, lane, a[1]);
            } else {
                stage();
                with_type(p.gate_type, [&](auto q) {
                    Raw<decltype(q)::value> r[2];
                    load_rows<decltype(q)::value>(r, gate, row0, p.F, p.gate_rb, c, nsub, lane);
                    multiply<decltype(q)::value>(r, tiles, n_tiles, nsub, lane, a[0]);
                });
                with_type(p.up_type, [&](auto q) {
                    Raw<decltype(q)::value> r[2];
                    load_rows<decltype(q)::value>(r, up, row0, p.F, p.up_rb, c, nsub, lane);
                    multiply<decltype(q)::value>(r, tiles, n_tiles, nsub, lane, a[1]);
                });
            }
        }
        __syncthreads();            // the tiles are read
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < kTiles; ++k) {
                if (k >= n_tiles) continue;
                float* to = sums + ((warp * 2 + m) * 16) * 16 + k * 8 + 2 * t;
                *reinterpret_cast<float2*>(to + g * 16) = make_float2(a[m][k][0], a[m][k][1]);
                *reinterpret_cast<float2*>(to + (g + 8) * 16) = make_float2(a[m][k][2], a[m][k][3]);
            }
        __syncthreads();
        for (int i = tid; i < n * 16; i += 32 * kUpWarps) {
            const int r = i & 15, k = i >> 4;
            if (row0 + r >= p.F) continue;
            float v[2] = {0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kUpWarps; ++w)
                for (int q = 0; q < parts; ++q) {
                    const float* from = sums + (w * 2 * 16 + r) * 16 + k * parts + q;
                    v[0] += from[0];
                    v[1] += from[16 * 16];
                }
            p.h[(int64_t)s_routes.list[first + r0 + k] * p.F + row0 + r] = activate(v[0], p.act) * v[1];
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- down, weights, residual

// Block x: rows 16 x .. of down, every expert's.  `splits` warps share an
// expert's chunks of F; each routed row's sums of each of them have their own
// place in shared memory and are added up in one order.
template <int QT>
__global__ void __launch_bounds__(32 * kDownWarps, 1) moe_ffn_down_kernel(const MoeFfnParams p) {
    extern __shared__ __align__(16) uint8_t s_dyn[];        // warps' tiles, then the rows' sums [split][entry][16]
    __shared__ Routes s_routes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int entries = p.T * p.top_k, parts = p.h_parts, splits = p.splits;
    float* sums = reinterpret_cast<float*>(s_dyn + p.down_warps * p.tiles * kTileBytes);
    uint8_t* tiles = s_dyn + warp * p.tiles * kTileBytes;
    pdl_wait();
    make_routes(s_routes, p.ids, entries, p.n_expert, tid, 32 * p.down_warps);
    const int64_t row0 = 16 * (int64_t)blockIdx.x;
    const int chunks = (int)ceil_div(p.F, kChunk), at_once = 8 * p.tiles / parts;
    const int items = s_routes.n_active * splits;
    for (int item = warp; item < items; item += p.down_warps) {
        const int e = s_routes.active[item / splits], split = item % splits;
        const int first = s_routes.start[e], rows = s_routes.start[e + 1] - first;
        const uint8_t* down = p.down + e * p.K * p.down_rb;
        for (int r0 = 0; r0 < rows; r0 += at_once) {
            const int n = min(at_once, rows - r0), n_tiles = (n * parts + 7) >> 3;
            float a[kTiles][4] = {};
            for (int c = split; c < chunks; c += splits) {
                const int nsub = (int)min((int64_t)8, (p.F - (int64_t)c * kChunk) / 32);
                Raw<QT> r[2];
                load_rows<QT>(r, down, row0, p.K, p.down_rb, c, nsub, lane);
                __syncwarp();
                for (int i = 0; i < n; ++i)
                    stage_row(tiles, i * parts, parts, p.h, GGUF_DT_F32,
                              (int64_t)s_routes.list[first + r0 + i] * p.F + (int64_t)c * kChunk, nsub, lane);
                __syncwarp();
                multiply<QT>(r, tiles, n_tiles, nsub, lane, a);
            }
            const int g = lane >> 2, t = lane & 3;
#pragma unroll
            for (int k = 0; k < kTiles; ++k) {
                if (k >= n_tiles) continue;
                // columns 2t, 2t + 1: the two parts of one row, or two rows
                const int col = 8 * k + 2 * t;
                if (parts == 2) {
                    if (col / 2 < n) {
                        float* to = sums + ((int64_t)split * entries + s_routes.list[first + r0 + col / 2]) * 16;
                        to[g] = a[k][0] + a[k][1];
                        to[g + 8] = a[k][2] + a[k][3];
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (col + q < n) {
                            float* to = sums + ((int64_t)split * entries + s_routes.list[first + r0 + col + q]) * 16;
                            to[g] = a[k][q];
                            to[g + 8] = a[k][q + 2];
                        }
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * 16; i += 32 * p.down_warps) {
        const int r = i & 15, t = i >> 4;
        if (row0 + r >= p.K) continue;
        const int64_t o = t * p.K + row0 + r;
        float v = p.residual ? load_act(p.residual, p.ydt, o) : 0.f;
        for (int s = 0; s < p.top_k; ++s) {
            const int at = t * p.top_k + s;
            if ((unsigned)p.ids[at] >= (unsigned)p.n_expert) continue;
            float row = 0.f;
            for (int q = 0; q < splits; ++q) row += sums[((int64_t)q * entries + at) * 16 + r];
            v = fmaf(p.weights[at], row, v);
        }
        store_out(p.y, p.ydt, o, v);
    }
}

template <int QT>
int launch_up(const MoeFfnParams& p, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    // a warp's tiles, or the warps' sums
    const size_t smem = std::max<size_t>((size_t)kUpWarps * p.tiles * kTileBytes, kUpWarps * 2 * 256 * sizeof(float));
    if (set_once(moe_ffn_up_kernel<QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kUpWarps * kTiles * kTileBytes, done) != cudaSuccess)
        return GGUF_ERR_CUDA;
    const dim3 grid((unsigned)ceil_div(p.F, 16), (unsigned)std::min(p.T * p.top_k, p.n_expert));
    return launch_pdl(moe_ffn_up_kernel<QT>, grid, dim3(32 * kUpWarps), smem, s, pdl, p) == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

template <int QT>
int launch_down(const MoeFfnParams& p, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    if (set_once(moe_ffn_down_kernel<QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDownSmem, done) != cudaSuccess)
        return GGUF_ERR_CUDA;
    const size_t smem = (size_t)p.down_warps * p.tiles * kTileBytes + (size_t)p.splits * p.T * p.top_k * 16 * sizeof(float);
    const cudaError_t e = launch_pdl(moe_ffn_down_kernel<QT>, dim3((unsigned)ceil_div(p.K, 16)), dim3(32 * p.down_warps), smem, s, pdl, p);
    return e == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA;
}

int dispatch_up(int qt, const MoeFfnParams& p, int pdl, cudaStream_t s) {
    switch (qt) {
        case GGUF_Q4_0: return launch_up<GGUF_Q4_0>(p, pdl, s);
        case GGUF_Q4_1: return launch_up<GGUF_Q4_1>(p, pdl, s);
        case GGUF_Q5_0: return launch_up<GGUF_Q5_0>(p, pdl, s);
        case GGUF_Q5_1: return launch_up<GGUF_Q5_1>(p, pdl, s);
        case GGUF_Q8_0: return launch_up<GGUF_Q8_0>(p, pdl, s);
        case GGUF_Q2_K: return launch_up<GGUF_Q2_K>(p, pdl, s);
        case GGUF_Q3_K: return launch_up<GGUF_Q3_K>(p, pdl, s);
        case GGUF_Q4_K: return launch_up<GGUF_Q4_K>(p, pdl, s);
        case GGUF_Q5_K: return launch_up<GGUF_Q5_K>(p, pdl, s);
        case GGUF_Q6_K: return launch_up<GGUF_Q6_K>(p, pdl, s);
        default: return launch_up<-1>(p, pdl, s);
    }
}

int dispatch_down(int qt, const MoeFfnParams& p, int pdl, cudaStream_t s) {
    switch (qt) {
        case GGUF_Q4_0: return launch_down<GGUF_Q4_0>(p, pdl, s);
        case GGUF_Q4_1: return launch_down<GGUF_Q4_1>(p, pdl, s);
        case GGUF_Q5_0: return launch_down<GGUF_Q5_0>(p, pdl, s);
        case GGUF_Q5_1: return launch_down<GGUF_Q5_1>(p, pdl, s);
        case GGUF_Q8_0: return launch_down<GGUF_Q8_0>(p, pdl, s);
        case GGUF_Q2_K: return launch_down<GGUF_Q2_K>(p, pdl, s);
        case GGUF_Q3_K: return launch_down<GGUF_Q3_K>(p, pdl, s);
        case GGUF_Q4_K: return launch_down<GGUF_Q4_K>(p, pdl, s);
        case GGUF_Q5_K: return launch_down<GGUF_Q5_K>(p, pdl, s);
        default: return launch_down<GGUF_Q6_K>(p, pdl, s);
    }
}

}  // namespace

int moe_ffn_launch(MoeFfnParams p, int pdl, cudaStream_t s) {
    p.x_parts = p.xdt == GGUF_DT_F32 ? 2 : 1;           // the 16-bit types' values are f16 numbers, scaled
    // the hidden values' rounding to f16 is below what a bf16 output rounds, and would not be below an f16 output's
    p.h_parts = p.ydt == GGUF_DT_BF16 ? 1 : 2;
    p.tiles = p.T * p.x_parts <= 8 ? 1 : kTiles;
    int st = dispatch_up(p.gate_type == p.up_type ? p.gate_type : -1, p, pdl, s);
    if (st != GGUF_OK) return st;
    p.tiles = p.T * p.h_parts <= 8 ? 1 : kTiles;
    p.down_warps = p.tiles == 1 ? kDownWarps : 16;
    // with few experts, several warps share one's chunks, as far as there is room for their sums
    const int64_t entries = p.T * p.top_k, experts = std::min<int64_t>(entries, p.n_expert);
    const int64_t room = (kDownSmem - (size_t)p.down_warps * p.tiles * kTileBytes) / (entries * 16 * sizeof(float));
    p.splits = (int)std::max<int64_t>(1, std::min({p.down_warps / experts, ceil_div(p.F, kChunk), room}));
    return dispatch_down(p.down_type, p, pdl, s);
}

}  // namespace gg
