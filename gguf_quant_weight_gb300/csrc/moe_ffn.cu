// A few tokens through their experts' gated feed-forward, on the GGUF blocks:
//   y[t] = residual[t] + sum_s w[t][s] * Down_e( act(Gate_e x[t]) * Up_e x[t] ),  e = ids[t][s],
// in three kernels: gate, up and the activation; the hidden values made ready
// for the tensor cores; down, the weighted sum and the residual.  Unlike the
// decode GEMV, activations are not rounded to int8: what a routed row gives is
// accurate to f32's rounding (f32 and f16 outputs) or to f16's (bf16 outputs).
//
// The weights' bytes bound it, and next to them the instructions that take
// blocks apart, so an expert's blocks are read and taken apart once for all of
// the batch's rows that it has: the tensor cores' m16n8k16 takes 16 weight rows
// as A and up to 8 columns of activations as B.  A's values are the blocks'
// codes.  A code without an offset needs no conversion: an integer's bits are
// the f16 number 2^-24 times it (a subnormal, which the tensor cores take), so a shift and a mask give
// two of them.  Codes
// with a zero point become 1024 + code by a byte permutation, less 1024 + zero
// point.  The products of a sub-block are summed by the tensor cores, and its
// scale is applied in f32.  B's columns are the activations scaled by a power of two
// per 256 of them; an f32 value takes two columns, its f16 rounding and what
// that left, so 22 bits of it.  Which values of a sub-block a lane holds is free as
// long as A and B agree: lane t of four has bytes 4t .. 4t+3 of each 16, and of
// those the even and the odd ones make its two pairs, which is how masks find
// them in a word of codes.
//
// Mins: sum_j m_j * (sum of sub-block j's activations) is one more product, of
// the mins (exact in f16) with the sums in two f16 parts.
//
// Each warp streams its own pieces of the weights, 16 rows x 256 values, through a
// ring of asynchronous copies that runs on across the experts and row tiles of its
// block, one block to an SM.  A row's piece is copied from the 16-byte boundary
// before it on; the rows lie an odd multiple of 16 bytes apart, so that the eight
// rows that a load of the warp meets fall into different banks.  Where pieces start at such a
// boundary (Q4_K, Q5_K) the lanes copy 16 bytes each; where they do not, which
// costs the lanes the arithmetic of every row's offset, one bulk copy moves a row.
// (A bulk copy of some 150 bytes holds its engine for about 19 cycles: with those
// 64 tokens through Q4_K experts take 167 us and not 123.  Before the codes were moved up
// in their subnormals, lanes' own copies made three tokens' Q6_K projection of 14336 take 127 us and not 101.)
//
// Measured: one token through 8 of 128 experts of 2048 x 768 (Q4_K, Q6_K) 20.7 us, the three kernels' latency; 64 tokens
// (Q4_K) 123 us, 2.4 TB/s, with three of five issue slots used, most by the integer instructions that take blocks
// apart; three tokens through 2 of 8 experts of 4096 x 14336 213 us, 3.0 TB/s.
#include <type_traits>

#include "formats.cuh"
#include "serving.cuh"

namespace gg {

namespace {

constexpr int kChunk = 256;                       // values of K a warp takes at a time
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kColStride = 2 * kChunk + 64;       // bytes of a column: f16 values, then the sums of its 16-value groups in two f16
                                                  // parts; 8 lanes' 16 bytes from 2 columns meet no bank twice
constexpr int kTileBytes = 8 * kColStride;
constexpr int kTiles = 2;                         // of 8 columns, at most
constexpr int kMaxStages = 4;                     // pieces of a warp on their way
constexpr size_t kSmem = 232448 - 2048;           // of a block, beside its static part

// ---------------------------------------------------------------- the experts' rows

// A group is some rows of one expert, as many as one pass over its weights takes.
struct Group {
    int16_t expert, n;
    int16_t first;                  // of its rows (entries token * top_k + slot) in Routes::list
    int16_t wide;                   // of up: groups of two tiles before it
};

// The rows by expert and, within one, in the order of the entries; the groups for
// up's passes and for down's.  Every block of up makes them for itself from the
// ids (an expert's groups may be different blocks' work, so all have to agree),
// and the first leaves them in the workspace for down.
struct Routes {
    Group* up;                      // [entries]
    Group* down;                    // [entries]
    uint16_t* list;                 // [entries]
    __host__ __device__ static size_t bytes(int entries) { return (size_t)ceil_div(18 * (int64_t)entries, 16) * 16; }
    __device__ Routes(uint8_t* at, int entries)
        : up(reinterpret_cast<Group*>(at)), down(up + entries), list(reinterpret_cast<uint16_t*>(down + entries)) {}
};
// What make_routes works in: a bit for each expert and entry, [entries / 32][n_expert], and the experts' first rows.
__host__ __device__ inline size_t routes_scratch(int entries, int n_expert) { return (size_t)(ceil_div(entries, 32) + 1) * n_expert * 4; }

// Returns the groups of up (low half) and of down.
__device__ int make_routes(const Routes& r, uint32_t* scratch, const int32_t* ids, int entries, int n_expert, int up_rows, int down_rows,
                           int tid) {
    __shared__ int s_warp[kWarps];
    const int lane = tid & 31, warp = tid >> 5, words = (entries + 31) >> 5;
    if (entries <= 32) {
        // one warp's work, the experts in the order in which they come
        if (warp == 0) {
            const int id = lane < entries ? ids[lane] : -1;
            const bool in = (unsigned)id < (unsigned)n_expert;
            const unsigned same = __match_any_sync(0xffffffffu, in ? id : -1 - lane), before = same & ((1u << lane) - 1);
            const int rows = in && !before ? __popc(same) : 0, ups = (rows + up_rows - 1) / up_rows, downs = (rows + down_rows - 1) / down_rows;
            const int mine = rows | ups << 10 | downs << 20;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const int at = upto - mine, first = at & 1023;
            for (int k = 0; k < ups; ++k)
                r.up[(at >> 10 & 1023) + k] = Group{(int16_t)id, (int16_t)min(up_rows, rows - k * up_rows), (int16_t)(first + k * up_rows), 0};
            for (int k = 0; k < downs; ++k)
                r.down[(at >> 20) + k] = Group{(int16_t)id, (int16_t)min(down_rows, rows - k * down_rows), (int16_t)(first + k * down_rows), 0};
            const int start = __shfl_sync(0xffffffffu, first, __ffs(same) - 1);
            if (in) r.list[start + __popc(before)] = (uint16_t)lane;
            if (lane == 31) s_warp[0] = (upto >> 10 & 1023) | (upto >> 20) << 16;
        }
        __syncthreads();
        return s_warp[0];
    }
    uint32_t* const first = scratch + words * n_expert;
    const int id = tid < entries ? ids[tid] : -1;           // at most kThreads entries
    for (int i = tid; i < words * n_expert; i += kThreads) scratch[i] = 0;
    __syncthreads();
    const bool in = (unsigned)id < (unsigned)n_expert;
    if (in) atomicOr(&scratch[warp * n_expert + id], 1u << lane);
    __syncthreads();
    int done = 0;                                           // rows, groups of up, groups of down: 10 bits each
    for (int b = 0; b < n_expert; b += kThreads) {
        const int e = b + tid;
        int rows = 0;
        if (e < n_expert)
            for (int w = 0; w < words; ++w) rows += __popc(scratch[w * n_expert + e]);
        const int ups = (rows + up_rows - 1) / up_rows, downs = (rows + down_rows - 1) / down_rows;
        const int mine = rows | ups << 10 | downs << 20;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = upto;
        __syncthreads();
        int before = done + upto - mine;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_warp[w];
            done += s_warp[w];
        }
        if (rows) {
            const int at = before & 1023;
            first[e] = at;
            for (int k = 0; k < ups; ++k)
                r.up[(before >> 10 & 1023) + k] = Group{(int16_t)e, (int16_t)min(up_rows, rows - k * up_rows), (int16_t)(at + k * up_rows), 0};
            for (int k = 0; k < downs; ++k)
                r.down[(before >> 20) + k] = Group{(int16_t)e, (int16_t)min(down_rows, rows - k * down_rows), (int16_t)(at + k * down_rows), 0};
        }
    }
    __syncthreads();
    if (in) {
        int at = first[id] + __popc(scratch[warp * n_expert + id] & ((1u << lane) - 1));
        for (int w = 0; w < warp; ++w) at += __popc(scratch[w * n_expert + id]);
        r.list[at] = (uint16_t)tid;
    }
    fence_proxy_async_smem();                               // the scratch's place is the ring's too
    __syncthreads();
    return (done >> 10 & 1023) | (done >> 20) << 16;
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

// One row's values [base, base + 32 * nsub) of x as a column of kColStride bytes (and,
// with two parts, the column after it).  Returns what the column's products are
// multiplied by.  The whole warp calls it.
__device__ __forceinline__ float make_column(uint8_t* col, int parts, const void* x, int dt, int64_t base, int nsub, int lane) {
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
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] *= scale, b[i] *= scale;
    uint4 hi;
    hi.x = pack2(a[0], a[2]), hi.y = pack2(a[1], a[3]), hi.z = pack2(b[0], b[2]), hi.w = pack2(b[1], b[3]);
    *reinterpret_cast<uint4*>(col + lane * 16) = hi;
    if (parts == 1 && dt == GGUF_DT_F32) {
        // a min meets the values that the codes meet: what f16 rounds off counts for the
        // weights as they are, not for their codes alone, which may be far larger
        const float2 f[4] = {unpack2(hi.x), unpack2(hi.y), unpack2(hi.z), unpack2(hi.w)};
        a[0] = f[0].x, a[2] = f[0].y, a[1] = f[1].x, a[3] = f[1].y;
        b[0] = f[2].x, b[2] = f[2].y, b[1] = f[3].x, b[3] = f[3].y;
    }
    float sa = (a[0] + a[1]) + (a[2] + a[3]), sb = (b[0] + b[1]) + (b[2] + b[3]);
    sa += __shfl_xor_sync(0xffffffffu, sa, 1), sb += __shfl_xor_sync(0xffffffffu, sb, 1);
    sa += __shfl_xor_sync(0xffffffffu, sa, 2), sb += __shfl_xor_sync(0xffffffffu, sb, 2);
    uint32_t* sums = reinterpret_cast<uint32_t*>(col + 2 * kChunk);      // [first parts 16][second parts 16] f16
    if (t == 0) {
        const uint32_t h = pack2(sa, sb);
        const float2 f = unpack2(h);
        sums[j] = h;
        sums[8 + j] = pack2(sa - f.x, sb - f.y);
    }
    if (parts == 2) {
        float2 f = unpack2(hi.x);
        uint4 lo;
        lo.x = pack2(a[0] - f.x, a[2] - f.y);
        f = unpack2(hi.y), lo.y = pack2(a[1] - f.x, a[3] - f.y);
        f = unpack2(hi.z), lo.z = pack2(b[0] - f.x, b[2] - f.y);
        f = unpack2(hi.w), lo.w = pack2(b[1] - f.x, b[3] - f.y);
        *reinterpret_cast<uint4*>(col + kColStride + lane * 16) = lo;
        if (t == 0) sums[kColStride / 4 + j] = sums[kColStride / 4 + 8 + j] = 0u;       // the first column has the whole sums
    }
    return back;
}

// ---------------------------------------------------------------- A: the blocks

// 256 values of a row: their bytes, and how far apart rows lie in shared memory
// (the piece from the 16-byte boundary before it to the one after it, and an odd
// multiple of 16)
__host__ __device__ constexpr int piece_bytes(int qt) { return block32(qt) ? 8 * block_bytes(qt) : block_bytes(qt); }
__host__ __device__ constexpr bool piece_aligned(int qt) { return qt == GGUF_Q4_K || qt == GGUF_Q5_K; }
__host__ __device__ constexpr int piece_stride(int qt) {
    const int slack = piece_aligned(qt) ? 0 : block_bytes(qt) % 4 ? 14 : 12;
    return ((piece_bytes(qt) + slack + 15) / 16 | 1) * 16;
}

__device__ __forceinline__ uint32_t ld32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t ld16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
// a word at a 2-byte boundary
__device__ __forceinline__ uint32_t ld32h(const uint8_t* p) { return ld16(p) | ld16(p + 2) << 16; }

__host__ __device__ constexpr bool has_min(int qt) {
    return qt == GGUF_Q2_K || qt == GGUF_Q4_K || qt == GGUF_Q5_K || b32_has_min(qt);
}
// what is subtracted from a code
__host__ __device__ constexpr int zero_point(int qt) {
    return qt == GGUF_Q6_K ? 32 : qt == GGUF_Q3_K ? 4 : qt == GGUF_Q8_0 ? 128 : block32(qt) ? b32_zero_point(qt) : 0;
}

// Codes without a zero point stand this far up in their bytes (see multiply()).
__host__ __device__ constexpr int code_shift(int qt) {
    return qt == GGUF_Q2_K ? 6 : qt == GGUF_Q4_K || qt == GGUF_Q4_1 ? 4 : qt == GGUF_Q5_K || qt == GGUF_Q5_1 ? 3 : 0;
}

// 256 values of one weight row as lane t of four holds them.  load(): from their
// first byte; nsub, how many of their 32-value groups exist (fewer than 8 at the
// end of a row of 32-value blocks).
template <int QT> struct Raw;

template <> struct Raw<GGUF_Q4_K> {
    uint32_t w[4][2];
    uint4 head;         // d, dmin, scales
    __device__ __forceinline__ void load(const uint8_t* b, int, int t) {
        head = *reinterpret_cast<const uint4*>(b);
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p][0] = ld32(b + 16 + 32 * p + 4 * t), w[p][1] = ld32(b + 32 + 32 * p + 4 * t);
    }
};
template <> struct Raw<GGUF_Q5_K> {
    uint32_t w[4][2], h[2];
    uint4 head;
    __device__ __forceinline__ void load(const uint8_t* b, int, int t) {
        head = *reinterpret_cast<const uint4*>(b);
        h[0] = ld32(b + 16 + 4 * t), h[1] = ld32(b + 32 + 4 * t);
#pragma unroll
        for (int p = 0; p < 4; ++p) w[p][0] = ld32(b + 48 + 32 * p + 4 * t), w[p][1] = ld32(b + 64 + 32 * p + 4 * t);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const {
        return ((j & 1 ? w[j >> 1][half] >> 1 : w[j >> 1][half] << 3) & 0x78787878u) | ((h[half] << (7 - j)) & 0x80808080u);
    }
};
template <> struct Raw<GGUF_Q6_K> {
    uint32_t ql[4][2], qh[2][2], sc[4], d;
    __device__ __forceinline__ void load(const uint8_t* b, int, int t) {
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
    __device__ __forceinline__ void load(const uint8_t* b, int, int t) {
#pragma unroll
        for (int p = 0; p < 4; ++p) sc[p] = ld32(b + 4 * p);
#pragma unroll
        for (int p = 0; p < 2; ++p) w[p][0] = ld32(b + 16 + 32 * p + 4 * t), w[p][1] = ld32(b + 32 + 32 * p + 4 * t);
        dm = ld32(b + 80);
    }
    __device__ __forceinline__ uint32_t codes(int j, int half, int) const { return (w[j >> 2][half] << (6 - 2 * (j & 3))) & 0xc0c0c0c0u; }
};
template <> struct Raw<GGUF_Q3_K> {
    uint32_t w[2][2], h[2], sc[3], d;
    __device__ __forceinline__ void load(const uint8_t* b, int, int t) {
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
    __device__ __forceinline__ void load(const uint8_t* row, int nsub, int t) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint8_t* b = row + min(j, nsub - 1) * BB;
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
            constexpr int up = code_shift(QT);
            uint32_t c = (up >= 4 * half ? w[j][0] << (up - 4 * half) : w[j][0] >> (4 * half - up)) & (0x0f0f0f0fu << up);
            if constexpr (b32_has_qh(QT)) {
                // bits 16 half + 4 t .. + 3, one to a byte: bit i times 2^7i lands on bit 8i, and no other product does
                const uint32_t four = (qh[j] >> (16 * half + 4 * t)) & 15u;
                c |= ((four * 0x00204081u) & 0x01010101u) << (4 + up);
            }
            return c;
        }
    }
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same, onto zeros
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ float f16_low(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v & 0xffffu))); }
__device__ __forceinline__ float f16_high(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v >> 16))); }
// byte i of a word as a float, less `less`: the mantissa's last bits of 2^23
__device__ __forceinline__ float byte_f(uint32_t w, int i, float less = 0.f) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 | i)) - (8388608.f + less);
}

// The 6-bit scales (lo, hi of four) and mins of Q4_K / Q5_K as words of bytes.
__device__ __forceinline__ void six_bits(const uint4& head, uint32_t (&sc)[4], uint32_t (&mn)[4]) {
    sc[0] = head.y & 0x3f3f3f3fu;
    mn[0] = head.z & 0x3f3f3f3fu;
    sc[1] = (head.w & 0x0f0f0f0fu) | ((head.y >> 2) & 0x30303030u);
    mn[1] = ((head.w >> 4) & 0x0f0f0f0fu) | ((head.z >> 2) & 0x30303030u);
}

// acc[tile] += (16 weight rows x 256 values) * (the tile's columns).  r[0], r[1]:
// the rows lane / 4 and lane / 4 + 8.  B gives column lane / 4's values of 32-value group j
// (values), its sums' parts (sums(tile, k): those of groups 8k + 2t, 2t + 1 of 16), and what columns 2t, 2t + 1 are
// multiplied by (back).
template <int QT, int TILES, class B>
__device__ __forceinline__ void multiply(const Raw<QT> (&r)[2], const B& col, int nsub, int lane, float (&acc)[TILES][4]) {
    const int t = lane & 3;
    // Codes as they are, subnormals, 2^(code_shift - 24) of them.  The tensor cores line products up by their exponents,
    // and a subnormal's is the lowest whatever its leading bits: a sum loses as many of its last bits as there are zeros
    // ahead of a code.  So codes and mins stand as high as shifts that are needed anyway leave them: two-bit codes in the lowest bits
    // gave an error of 1.4e-5 of the output, four bits 3.3e-6.
    constexpr bool plain = zero_point(QT) == 0;
    constexpr float kCode = (float)(1 << (24 - code_shift(QT)));
    constexpr int kMinUp = QT == GGUF_Q2_K ? 6 : 4;
    constexpr bool narrow = QT == GGUF_Q2_K || QT == GGUF_Q3_K || QT == GGUF_Q6_K;      // scales of 16 values
    const __half2 zero = __float2half2_rn(-(float)(1024 + zero_point(QT)));
    float total[TILES][4] = {};
    uint32_t sc[2][4] = {}, mn[2][4] = {};      // by row: scales and mins as bytes
    float d[2], dmin[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        d[i] = 1.f, dmin[i] = 1.f;
        if constexpr (QT == GGUF_Q4_K || QT == GGUF_Q5_K) {
            six_bits(r[i].head, sc[i], mn[i]);
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
#pragma unroll
            for (int p = 0; p < 4; ++p) sc[i][p] = r[i].sc[p] ^ 0x80808080u;
            d[i] = f16_low(r[i].d);
        }
    }
    // scale of 16-value group 2 j + half (of group j, where they have 32 values) of row i
    auto scale = [&](int i, int j, int half) -> float {
        if constexpr (block32(QT)) return f16_low(r[i].d[j]);
        const int s = narrow ? 2 * j + half : j;
        return byte_f(sc[i][s >> 2], s & 3, QT == GGUF_Q6_K ? 128.f : QT == GGUF_Q3_K ? 32.f : 0.f);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (block32(QT) && j >= nsub) break;
        uint4 b[TILES];
#pragma unroll
        for (int n = 0; n < TILES; ++n)
            b[n] = col.values(n, j);
        float part[TILES][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (QT == GGUF_Q4_K) {
                    const uint32_t w = r[i].w[j >> 1][half], m = 0x00f000f0u;
                    a[i] = (j & 1 ? w : w << 4) & m;
                    a[i + 2] = (j & 1 ? w >> 8 : w >> 4) & m;
                } else {
                    const uint32_t c = r[i].codes(j, half, t);
                    if constexpr (plain) {
                        a[i] = __byte_perm(c, 0u, 0x4240);
                        a[i + 2] = __byte_perm(c, 0u, 0x4341);
                    } else {
                        a[i] = as_u32(__hadd2(as_h2(__byte_perm(c, 0x64646464u, 0x4240)), zero));
                        a[i + 2] = as_u32(__hadd2(as_h2(__byte_perm(c, 0x64646464u, 0x4341)), zero));
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < TILES; ++n) {
                if (half == 0) mma0(part[n], a[0], a[1], a[2], a[3], b[n].x, b[n].y);
                else if (narrow) mma0(part[n], a[0], a[1], a[2], a[3], b[n].z, b[n].w);
                else mma(part[n], a[0], a[1], a[2], a[3], b[n].z, b[n].w);
            }
            if (narrow || half == 1) {
                const float s0 = scale(0, j, half), s1 = scale(1, j, half);
#pragma unroll
                for (int n = 0; n < TILES; ++n) {
                    total[n][0] = fmaf(part[n][0], s0, total[n][0]);
                    total[n][1] = fmaf(part[n][1], s0, total[n][1]);
                    total[n][2] = fmaf(part[n][2], s1, total[n][2]);
                    total[n][3] = fmaf(part[n][3], s1, total[n][3]);
                }
            }
        }
    }
    if constexpr (plain) d[0] *= kCode, d[1] *= kCode;
#pragma unroll
    for (int n = 0; n < TILES; ++n) {
        const float2 back = col.back(n);
        if constexpr (has_min(QT)) {
            float low[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t a[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // mins are subnormals too, but those of the 32-value blocks, f16 numbers
                    if constexpr (QT == GGUF_Q2_K) {
                        const uint32_t two = (t < 2 ? mn[i][2 * k] : mn[i][2 * k + 1]) >> (16 * (t & 1));
                        a[i] = (two & 0xffu) << kMinUp | (two & 0xff00u) << (8 + kMinUp);
                    } else if constexpr (block32(QT)) {
                        // group 4k + t's m: no register is indexed by a lane
                        const uint32_t m = t < 2 ? (t ? r[i].d[4 * k + 1] : r[i].d[4 * k]) : (t == 2 ? r[i].d[4 * k + 2] : r[i].d[4 * k + 3]);
                        a[i] = 4 * k + t < nsub ? __byte_perm(m, 0u, 0x3232) : 0u;
                    } else {
                        a[i] = ((mn[i][k] >> (8 * t)) & 0xffu) * (0x00010001u << kMinUp);
                    }
                }
                const uint2 s = col.sums(n, k);         // the same mins with the sums' first part and their second
                if (k == 0) mma0(low, a[0], a[1], a[0], a[1], s.x, s.y);
                else mma(low, a[0], a[1], a[0], a[1], s.x, s.y);
            }
            // Q4_1, Q5_1 add their m
            constexpr float kMin = (float)(1 << (24 - kMinUp));
            const float m0 = block32(QT) ? 1.f : -kMin * dmin[0], m1 = block32(QT) ? 1.f : -kMin * dmin[1];
            acc[n][0] = fmaf(fmaf(m0, low[0], d[0] * total[n][0]), back.x, acc[n][0]);
            acc[n][1] = fmaf(fmaf(m0, low[1], d[0] * total[n][1]), back.y, acc[n][1]);
            acc[n][2] = fmaf(fmaf(m1, low[2], d[1] * total[n][2]), back.x, acc[n][2]);
            acc[n][3] = fmaf(fmaf(m1, low[3], d[1] * total[n][3]), back.y, acc[n][3]);
        } else {
            acc[n][0] = fmaf(d[0] * total[n][0], back.x, acc[n][0]);
            acc[n][1] = fmaf(d[0] * total[n][1], back.y, acc[n][1]);
            acc[n][2] = fmaf(d[1] * total[n][2], back.x, acc[n][2]);
            acc[n][3] = fmaf(d[1] * total[n][3], back.y, acc[n][3]);
        }
    }
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

// ---------------------------------------------------------------- the weights' ring

// A matrix of one expert, as rows of pieces.  The rows at and after n of its last 16 stand for its last row (their results
// are dropped).
struct Matrix {
    const uint8_t* w;
    const uint8_t* end;             // of all experts' bytes: nothing is read past it
    int64_t rb;                     // bytes of a row
    int n;                          // rows
};

// Where this lane's 16-byte units of an aligned piece lie, from the tile's first row on.
template <int QT>
struct Units {
    static constexpr int ROW = piece_stride(QT) / 16, N = piece_aligned(QT) ? (16 * ROW + 31) / 32 : 1;
    uint32_t rel[N];
    __device__ __forceinline__ Units(const Matrix& m, int lane) {
        if constexpr (piece_aligned(QT))
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int u = 32 * i + lane, row = u / ROW;
                rel[i] = (uint32_t)row * (uint32_t)m.rb + 16 * (u - row * ROW);         // 16 rows are below 2^32 bytes
            }
    }
};
// What a piece's barrier counts: the lanes, whose own copies arrive for them, or the one that announces the bulk copies.
// A kernel whose pieces are all aligned has no barriers: each lane waits for its own copies, in order.
__host__ __device__ constexpr int piece_arrivals(int qt) { return piece_aligned(qt) ? 32 : 1; }

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last n groups of this thread's copies have arrived
__device__ __forceinline__ void copies_wait(int n) {
    if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

template <int QT>
__device__ __forceinline__ void fetch_piece(uint8_t* slot, uint64_t* bar, const Matrix& m, const Units<QT>& units, int row0, int c, int lane) {
    if constexpr (piece_aligned(QT)) {
        using U = Units<QT>;
        const bool whole = row0 + 16 <= m.n;
        const uint8_t* const base = m.w + (int64_t)(whole ? row0 : 0) * m.rb + c * piece_bytes(QT);
        const uint32_t to = smem_u32(slot) + 16 * lane;
#pragma unroll
        for (int i = 0; i < U::N; ++i) {
            const int u = 32 * i + lane;
            if (16 * U::ROW % 32 && u >= 16 * U::ROW) break;
            const uint8_t* src = base + units.rel[i];
            if (!whole) src = base + (int64_t)min(row0 + u / U::ROW, m.n - 1) * m.rb + 16 * (u % U::ROW);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * i), "l"(src) : "memory");
        }
        if (bar) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    } else {
        // Lane l copies row l's piece.  The last bytes of all experts may end inside 16: no copy goes past them, and they
        // are moved by hand.
        const uint8_t* src = m.w + (int64_t)min(row0 + (lane & 15), m.n - 1) * m.rb + (int64_t)c * piece_bytes(QT);
        uint8_t* const dst = slot + (lane & 15) * piece_stride(QT);
        const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
        // fewer at the end of a row of 32-value blocks
        const int bytes = off + (int)min((int64_t)piece_bytes(QT), m.rb - (int64_t)c * piece_bytes(QT));
        src -= off;
        int size = (bytes + 15) & ~15;
        if (m.end - src < size) {
            size = (int)(m.end - src) & ~15;
            if (lane < 16)
                for (int i = size; i < bytes; i += 2) *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
        }
        const uint32_t all = __reduce_add_sync(0xffffffffu, lane < 16 ? (uint32_t)size : 0u);
        if (lane == 0) mbar_arrive_expect_tx(bar, all);
        __syncwarp();
        if (lane < 16 && size) bulk_g2s(dst, src, (uint32_t)size, bar);
    }
}

// A warp's ring: where the next piece goes, which is read next, and its turn.
// BARS: whether the pieces have barriers.
template <bool BARS>
struct Ring {
    uint8_t* at;
    uint64_t* bars;
    int* status;
    int slot_bytes, stages, into = 0, from = 0;
    uint32_t parity = 0;
    bool dead = false;              // a wait has been given up: no more copies, no more waits
    __device__ __forceinline__ void init(int arrivals, int lane) {
        if (BARS && lane < stages) mbar_init(bars + lane, arrivals);
        if (BARS) fence_mbar_init();
        __syncwarp();
    }
    __device__ __forceinline__ uint8_t* put(uint64_t*& bar) {
        const int k = into;
        into = into + 1 == stages ? 0 : into + 1;
        bar = BARS ? bars + k : nullptr;
        return at + k * slot_bytes;
    }
    // all lanes together
    __device__ __forceinline__ const uint8_t* get() {
        const int k = from;
        if constexpr (BARS) {
            if (!dead && !__all_sync(0xffffffffu, mbar_wait(bars + k, parity, status))) dead = true;
        } else {
            copies_wait(stages - 1);
            __syncwarp();
        }
        if (++from == stages) from = 0, parity ^= 1;
        return at + k * slot_bytes;
    }
    // what was on its way when a wait was given up does not outlive the block
    __device__ __forceinline__ void close() {
        if (BARS && dead)
            for (int k = 0; k < stages; ++k) mbar_wait(bars + k, (k < from ? parity ^ 1 : parity), status);
    }
};

template <int QT>
__device__ __forceinline__ void read_piece(Raw<QT> (&r)[2], const uint8_t* slot, const Matrix& m, int row0, int c, int nsub, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int off = 0;
        if constexpr (!piece_aligned(QT))
            off = (int)(reinterpret_cast<uintptr_t>(m.w) + (uint32_t)min(row0 + g + 8 * i, m.n - 1) * (uint32_t)m.rb + (uint32_t)c * piece_bytes(QT)) & 15;
        r[i].load(slot + (g + 8 * i) * piece_stride(QT) + off, nsub, t);
    }
}

__device__ __forceinline__ float activate(float a, int act) {
    if (act == GGUF_ACT_SILU) return a / (1.f + expf(-a));
    // tanh form: 0.79788... = sqrt(2 / pi)
    return 0.5f * a * (1.f + tanhf(0.79788456080286536f * (a + 0.044715f * a * a * a)));
}

// ---------------------------------------------------------------- gate, up, activation

// A job is 16 rows of gate and up, for one group; a block takes a run of jobs, so
// that it makes a group's columns once for many of them.  Its warps work in teams of
// 2 wp, each on its own job: of each matrix wp warps take every wp-th chunk of K, and
// their sums meet in shared memory.  Small teams meet seldom for what they do in
// between; larger ones are for calls that have too few jobs.
// QT: both matrices' type, or -1 where they differ.  TILES: of 8 columns that a group may have.
struct ColumnsInShared {
    const uint8_t* at;              // the chunk's tiles, at this lane's column and 16 bytes
    const float* scales;            // the chunk's, at 2t
    int t;
    __device__ __forceinline__ uint4 values(int n, int j) const { return *reinterpret_cast<const uint4*>(at + n * kTileBytes + j * 64); }
    __device__ __forceinline__ uint2 sums(int n, int k) const {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(at + n * kTileBytes + 2 * kChunk - 16 * t);
        return make_uint2(s[4 * k + t], s[8 + 4 * k + t]);
    }
    __device__ __forceinline__ float2 back(int n) const { return *reinterpret_cast<const float2*>(scales + 8 * n); }
};

template <int QT, int TILES>
__global__ void __launch_bounds__(kThreads, 1) moe_ffn_up_kernel(const MoeFfnParams p) {
    extern __shared__ __align__(16) uint8_t s_dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int entries = p.T * p.top_k, chunks = (int)ceil_div(p.K, kChunk), parts = p.x_parts;
    constexpr int tiles = TILES;
    const Routes routes(s_dyn, entries);
    // a group's columns: of all chunks, or, where K is too long, of the one that each warp is at
    const int held = p.up_resident ? chunks : kWarps;
    uint8_t* const columns = s_dyn + Routes::bytes(entries);                                // [held][tile]
    float* const scales = reinterpret_cast<float*>(columns + (size_t)held * tiles * kTileBytes);        // [held][8 * tiles]
    float* const sums = scales + held * 8 * tiles;                                          // [2][warp][16 rows][8 * tiles]
    __shared__ uint64_t s_bars[kWarps * kMaxStages];
    constexpr bool kBars = QT < 0 || !piece_aligned(QT);
    Ring<kBars> ring{reinterpret_cast<uint8_t*>(sums + 2 * kWarps * 128 * tiles) + (size_t)warp * p.up_stages * p.up_slot, s_bars + warp * kMaxStages,
              p.status, p.up_slot, p.up_stages};
    pdl_wait();
    pdl_launch_dependents();        // all blocks of this kernel are running
    const int both = make_routes(routes, reinterpret_cast<uint32_t*>(columns), p.ids, entries, p.n_expert, 8 * tiles / parts, 8 / p.h_parts, tid);
    const int groups = both & 0xffff;
    if (blockIdx.x == 0) {
        const uint4* from = reinterpret_cast<const uint4*>(s_dyn);
        uint4* to = reinterpret_cast<uint4*>(p.routes);
        for (int i = tid; i < (int)(Routes::bytes(entries) / 16); i += kThreads) to[i + 1] = from[i];
        if (tid == 0) to[0] = make_uint4(both >> 16, 0, 0, 0);
    }
    const int K = (int)p.K, F = (int)p.F, per_group = (F + 15) / 16, jobs = per_group * groups;
    // The blocks' shares of the jobs, where a job of two tiles counts 4 and one of one tile 3 (the blocks
    // are taken apart once either way).
    int job0, job1;
    if constexpr (TILES == 1) {
        auto share = [&](unsigned b) { return jobs < 1 << 23 ? (int)((unsigned)jobs * b / gridDim.x) : (int)((int64_t)jobs * b / gridDim.x); };
        job0 = share(blockIdx.x), job1 = share(blockIdx.x + 1);      // at most 152 blocks
    } else {
        __shared__ int s_from[2], s_wide;
        if (tid < 2) s_from[tid] = jobs;
        if (warp == 0) {
            int wide = 0;
            for (int b = 0; b < groups; b += 32) {
                const bool two = b + lane < groups && routes.up[b + lane].n * parts > 8;
                const unsigned on = __ballot_sync(0xffffffffu, two);
                if (b + lane < groups) routes.up[b + lane].wide = (int16_t)(wide + __popc(on & ((1u << lane) - 1)));
                wide += __popc(on);
            }
            if (lane == 0) s_wide = wide;
        }
        __syncthreads();
        const int64_t whole = (int64_t)per_group * (3 * groups + s_wide);
        if (tid < groups) {
            const int cost = routes.up[tid].n * parts > 8 ? 4 : 3;
            const int64_t lo = (int64_t)per_group * (3 * tid + routes.up[tid].wide);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t at = whole * (blockIdx.x + k) / gridDim.x - lo;
                if (at >= 0 && at < (int64_t)per_group * cost) s_from[k] = tid * per_group + (int)at / cost;
            }
        }
        __syncthreads();
        job0 = s_from[0], job1 = s_from[1];
    }
    // this warp's part of a job
    const int wp = p.up_wp, teams = kWarps / (2 * wp), team = warp / (2 * wp), mat = (warp / wp) & 1, c0 = warp % wp;
    const int qt = mat ? p.up_type : p.gate_type;
    ring.init(qt == GGUF_Q4_K || qt == GGUF_Q5_K ? piece_arrivals(GGUF_Q4_K) : piece_arrivals(GGUF_Q6_K), lane);
    Matrix m;
    m.rb = mat ? p.up_rb : p.gate_rb;
    m.n = F;
    m.end = (mat ? p.up : p.gate) + p.n_expert * p.F * m.rb;
    auto matrix_of = [&](int group) { return (mat ? p.up : p.gate) + routes.up[group].expert * p.F * m.rb; };
    // A group's jobs [begin, end) go to the teams in turn.  The ring's next piece to fetch runs ahead.
    int fgroup = job0 / per_group, fend = min(job1, (fgroup + 1) * per_group), fjob = job0 + team, fc = c0;
    Matrix fm = m;
    const Units<(QT < 0 ? GGUF_Q6_K : QT)> units(m, lane);
    auto settle = [&] {             // to a job that there is
        while (fjob >= fend && fend < job1) fjob = fend + team, ++fgroup, fend = min(job1, fend + per_group);
        if (fjob < fend) fm.w = matrix_of(fgroup);
    };
    settle();
    auto fetch = [&] {
        if (fjob < fend && !ring.dead) {
            const int row0 = (fjob - fgroup * per_group) * 16;
            uint64_t* bar;
            uint8_t* const slot = ring.put(bar);
            if constexpr (QT >= 0) fetch_piece<QT>(slot, bar, fm, units, row0, fc, lane);
            else with_type(qt, [&](auto q) { fetch_piece<decltype(q)::value>(slot, bar, fm, Units<decltype(q)::value>(fm, lane), row0, fc, lane); });
            fc += wp;
            if (fc >= chunks) {
                fc = c0;
                fjob += teams;
                if (fjob >= fend) settle();
            }
        }
        if (!kBars) copies_commit();
    };
    for (int i = 0; i < p.up_stages; ++i) fetch();

    int buffer = 0;
    Group g{};
    auto make = [&](int k, int c, int at) {         // the columns of the group's row k, chunk c
        const int col = k * parts, token = routes.list[g.first + k] / p.top_k;
        const int nsub = min(8, (K - c * kChunk) / 32);
        const float back = make_column(columns + (size_t)(at * tiles * 8 + col) * kColStride, parts, p.x, p.xdt,
                                       token * p.K + c * kChunk, nsub, lane);
        if (lane < parts) scales[at * 8 * tiles + col + lane] = back;
    };
    for (int group = job0 / per_group, begin = job0; begin < job1; ++group) {
      const int end = min(job1, (group + 1) * per_group);
      g = routes.up[group];
      m.w = matrix_of(group);
      if (p.up_resident) {
          if (begin != job0) __syncthreads();       // the columns before are read
          for (int i = warp; i < g.n * chunks; i += kWarps) make(i % g.n, i / g.n, i / g.n);
          __syncthreads();
      }
      const int n_tiles = (g.n * parts + 7) >> 3;
      for (int job = begin + team; job < end; job += teams, buffer ^= 1) {
        const int row0 = (job - group * per_group) * 16;
        float acc[TILES][4] = {};
        for (int c = c0; c < chunks; c += wp) {
            const int at = p.up_resident ? c : warp;
            if (!p.up_resident)
                for (int k = 0; k < g.n; ++k) make(k, c, at);
            __syncwarp();
            const uint8_t* const slot = ring.get();
            const int nsub = min(8, (K - c * kChunk) / 32), t = lane & 3;
            const ColumnsInShared col{columns + (size_t)at * tiles * kTileBytes + (lane >> 2) * kColStride + t * 16, scales + at * 8 * tiles + 2 * t, t};
            auto unit = [&](auto q) {
                constexpr int Q = decltype(q)::value;
                Raw<Q> r[2];
                read_piece<Q>(r, slot, m, row0, c, nsub, lane);
                __syncwarp();       // the piece is read: its place may be filled
                fetch();
                // (an instruction that a predicate turns off still takes its turn)
                if (TILES == 1 || n_tiles == 1) multiply<Q, 1>(r, col, nsub, lane, reinterpret_cast<float(&)[1][4]>(acc));
                else multiply<Q, TILES>(r, col, nsub, lane, acc);
            };
            if constexpr (QT >= 0) unit(std::integral_constant<int, QT>{});
            else with_type(qt, unit);
            if (!p.up_resident) __syncwarp();       // the columns are read
        }
        float* const to = sums + (size_t)(buffer * kWarps + warp) * 128 * tiles;
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            if (k >= n_tiles) continue;
            float* at = to + (lane >> 2) * 8 * tiles + 8 * k + 2 * (lane & 3);
            *reinterpret_cast<float2*>(at) = make_float2(acc[k][0], acc[k][1]);
            *reinterpret_cast<float2*>(at + 64 * tiles) = make_float2(acc[k][2], acc[k][3]);
        }
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(64 * wp) : "memory");
        // the sums of two jobs have places of their own, so the team goes on meanwhile
        for (int i = tid - team * 64 * wp; i < 128 * tiles; i += 64 * wp) {
            const int r = i & 15, k = i >> 4;
            if (k >= g.n || row0 + r >= F) continue;
            float v[2] = {0.f, 0.f};
            const float* from = sums + (size_t)(buffer * kWarps + team * 2 * wp) * 128 * tiles + r * 8 * tiles + k * parts;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                for (int w = 0; w < wp; ++w) {
                    const float* f = from + (size_t)(q * wp + w) * 128 * tiles;
                    v[q] += parts == 2 ? f[0] + f[1] : f[0];
                }
            p.h[(int64_t)routes.list[g.first + k] * p.F + row0 + r] = activate(v[0], p.act) * v[1];
        }
      }
      begin = end;
    }
    ring.close();
}

// ---------------------------------------------------------------- the hidden values as columns

// A warp a column: [entry][chunk][part] of kColStride bytes, and what its products are multiplied by [entry][chunk].
__global__ void __launch_bounds__(256) moe_ffn_columns_kernel(const MoeFfnParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, chunks = (int)ceil_div(p.F, kChunk);
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= p.T * p.top_k * chunks) return;
    const int entry = i / chunks, c = i - entry * chunks;
    const int nsub = min(8, ((int)p.F - c * kChunk) / 32);
    const float back = make_column(p.columns + (int64_t)i * p.h_parts * kColStride, p.h_parts, p.h, GGUF_DT_F32, entry * p.F + c * kChunk, nsub, lane);
    if (lane == 0) p.column_scales[i] = back;
}

// ---------------------------------------------------------------- down, weights, residual

// Block x: rows 16 x .. of down, every group's.  `splits` warps share a group's
// chunks of F; each routed row's sums of each of them have their own place in
// shared memory and are added up in one order.
struct ColumnsInRegisters {
    uint4 v[8];
    uint2 s[2];
    float2 f;
    __device__ __forceinline__ uint4 values(int, int j) const { return v[j]; }
    __device__ __forceinline__ uint2 sums(int, int k) const { return s[k]; }
    __device__ __forceinline__ float2 back(int) const { return f; }
};

template <int QT>
__global__ void __launch_bounds__(kThreads, 1) moe_ffn_down_kernel(const MoeFfnParams p) {
    extern __shared__ __align__(16) uint8_t s_dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int entries = p.T * p.top_k, parts = p.h_parts, splits = p.splits;
    const Routes routes(s_dyn, entries);
    float* const weights = reinterpret_cast<float*>(s_dyn + Routes::bytes(entries));                // [entry]
    float* const sums = weights + (entries + 3) / 4 * 4;                                            // [split][entry][16]
    constexpr int kSlot = 16 * piece_stride(QT);
    __shared__ uint64_t s_bars[kWarps * kMaxStages];
    constexpr bool kBars = !piece_aligned(QT);
    Ring<kBars> ring{reinterpret_cast<uint8_t*>(sums + (size_t)splits * entries * 16) + (size_t)warp * p.down_stages * kSlot, s_bars + warp * kMaxStages,
              p.status, kSlot, p.down_stages};
    ring.init(piece_arrivals(QT), lane);
    // The kernel before this one let it begin when up had ended, so the routes are
    // there (read past L1, as nothing has been waited for here); the columns are waited
    // for once the first weights are on their way.
    for (int i = tid; i < (int)(Routes::bytes(entries) / 16); i += kThreads)
        reinterpret_cast<uint4*>(s_dyn)[i] = __ldcg(reinterpret_cast<const uint4*>(p.routes) + i + 1);
    const int items = __ldcg(reinterpret_cast<const int*>(p.routes)) * splits;
    if (tid < entries) weights[tid] = (unsigned)__ldcg(p.ids + tid) < (unsigned)p.n_expert ? __ldcg(p.weights + tid) : 0.f;
    // an id of no expert adds 0 * 0
    for (int i = tid; i < splits * entries * 4; i += kThreads) reinterpret_cast<float4*>(sums)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    const int row0 = 16 * blockIdx.x, F = (int)p.F, chunks = (F + kChunk - 1) / kChunk;
    Matrix m{nullptr, p.down + p.n_expert * p.K * p.down_rb, p.down_rb, (int)p.K};
    auto matrix_of = [&](int item) { return p.down + routes.down[item / splits].expert * p.K * p.down_rb; };
    int fitem = warp, fc = warp % splits;
    Matrix fm = m;
    const Units<QT> units(m, lane);
    if (fitem < items) fm.w = matrix_of(fitem);
    auto fetch = [&] {
        if (fitem < items && !ring.dead) {
            uint64_t* bar;
            uint8_t* const slot = ring.put(bar);
            fetch_piece<QT>(slot, bar, fm, units, row0, fc, lane);
            fc += splits;
            if (fc >= chunks && (fitem += kWarps) < items) fc = fitem % splits, fm.w = matrix_of(fitem);
        }
        if (!kBars) copies_commit();
    };
    for (int i = 0; i < p.down_stages; ++i) fetch();
    pdl_wait();
    float residual = 0.f;           // of this thread's first output
    if (p.residual && tid < p.T * 16 && row0 + (tid & 15) < p.K)
        residual = load_act(p.residual, p.ydt, (tid >> 4) * p.K + row0 + (tid & 15));
    const int g = lane >> 2, t = lane & 3;
    for (int item = warp; item < items; item += kWarps) {
        const Group group = routes.down[item / splits];
        m.w = matrix_of(item);
        float acc[1][4] = {};
        // this lane's column, and columns 2t, 2t + 1, of the group's rows
        auto entry_of = [&](int col) { return (int64_t)routes.list[group.first + min(col / parts, group.n - 1)]; };
        const int64_t mine = entry_of(g) * chunks, first = entry_of(2 * t) * chunks, second = entry_of(2 * t + 1) * chunks;
        for (int c = item % splits; c < chunks; c += splits) {
            ColumnsInRegisters col;
            const uint8_t* at = p.columns + ((mine + c) * parts + g % parts) * kColStride;
#pragma unroll
            for (int j = 0; j < 8; ++j) col.v[j] = __ldg(reinterpret_cast<const uint4*>(at + j * 64 + t * 16));
            if constexpr (has_min(QT)) {
                const uint32_t* s = reinterpret_cast<const uint32_t*>(at + 2 * kChunk);
                col.s[0] = make_uint2(__ldg(s + t), __ldg(s + 8 + t)), col.s[1] = make_uint2(__ldg(s + 4 + t), __ldg(s + 12 + t));
            }
            col.f = make_float2(__ldg(p.column_scales + first + c), __ldg(p.column_scales + second + c));
            const uint8_t* const slot = ring.get();
            const int nsub = min(8, (F - c * kChunk) / 32);
            Raw<QT> r[2];
            read_piece<QT>(r, slot, m, row0, c, nsub, lane);
            __syncwarp();           // the piece is read: its place may be filled
            fetch();
            multiply<QT, 1>(r, col, nsub, lane, acc);
        }
        // columns 2t, 2t + 1: the two parts of one row, or two rows
        float* const to = sums + (size_t)(item % splits) * entries * 16;
        if (parts == 2) {
            if (t < group.n) {
                float* at = to + routes.list[group.first + t] * 16;
                at[g] = acc[0][0] + acc[0][1];
                at[g + 8] = acc[0][2] + acc[0][3];
            }
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (2 * t + q < group.n) {
                    float* at = to + routes.list[group.first + 2 * t + q] * 16;
                    at[g] = acc[0][q];
                    at[g + 8] = acc[0][q + 2];
                }
        }
    }
    ring.close();
    __syncthreads();
    for (int i = tid; i < p.T * 16; i += kThreads) {
        const int r = i & 15, token = i >> 4;
        if (row0 + r >= p.K) continue;
        const int64_t o = token * p.K + row0 + r;
        float v = i == tid ? residual : p.residual ? load_act(p.residual, p.ydt, o) : 0.f;
        for (int s = 0; s < p.top_k; ++s) {
            const int at = token * p.top_k + s;
            float row = 0.f;
            for (int q = 0; q < splits; ++q) row += sums[((size_t)q * entries + at) * 16 + r];
            v = fmaf(weights[at], row, v);
        }
        store_out(p.y, p.ydt, o, v);
    }
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? GGUF_OK : GGUF_ERR_CUDA; }

template <int QT, int TILES>
int launch_up(const MoeFfnParams& p, int blocks, size_t smem, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    auto* k = moe_ffn_up_kernel<QT, TILES>;
    if (set_once(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem, done) != cudaSuccess) return GGUF_ERR_CUDA;
    return cuda_status(launch_pdl(k, dim3((unsigned)blocks), dim3(kThreads), smem, s, pdl, p));
}
template <int QT>
int launch_up(const MoeFfnParams& p, int blocks, size_t smem, int pdl, cudaStream_t s) {
    return p.up_tiles == 1 ? launch_up<QT, 1>(p, blocks, smem, pdl, s) : launch_up<QT, kTiles>(p, blocks, smem, pdl, s);
}

template <int QT>
int launch_down(const MoeFfnParams& p, size_t smem, int pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    if (set_once(moe_ffn_down_kernel<QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem, done) != cudaSuccess) return GGUF_ERR_CUDA;
    return cuda_status(launch_pdl(moe_ffn_down_kernel<QT>, dim3((unsigned)ceil_div(p.K, 16)), dim3(kThreads), smem, s, pdl, p));
}

int dispatch_up(int qt, const MoeFfnParams& p, int blocks, size_t smem, int pdl, cudaStream_t s) {
    switch (qt) {
#define GG_CASE(Q) case Q: return launch_up<Q>(p, blocks, smem, pdl, s);
        GG_CASE(GGUF_Q4_0) GG_CASE(GGUF_Q4_1) GG_CASE(GGUF_Q5_0) GG_CASE(GGUF_Q5_1) GG_CASE(GGUF_Q8_0)
        GG_CASE(GGUF_Q2_K) GG_CASE(GGUF_Q3_K) GG_CASE(GGUF_Q4_K) GG_CASE(GGUF_Q5_K) GG_CASE(GGUF_Q6_K)
#undef GG_CASE
        default: return launch_up<-1>(p, blocks, smem, pdl, s);
    }
}

int dispatch_down(const MoeFfnParams& p, size_t smem, int pdl, cudaStream_t s) {
    switch (p.down_type) {
#define GG_CASE(Q) case Q: return launch_down<Q>(p, smem, pdl, s);
        GG_CASE(GGUF_Q4_0) GG_CASE(GGUF_Q4_1) GG_CASE(GGUF_Q5_0) GG_CASE(GGUF_Q5_1) GG_CASE(GGUF_Q8_0)
        GG_CASE(GGUF_Q2_K) GG_CASE(GGUF_Q3_K) GG_CASE(GGUF_Q4_K) GG_CASE(GGUF_Q5_K)
#undef GG_CASE
        default: return launch_down<GGUF_Q6_K>(p, smem, pdl, s);
    }
}

int slot_bytes(int qt) {
    switch (qt) {
#define GG_CASE(Q) case Q: return 16 * piece_stride(Q);
        GG_CASE(GGUF_Q4_0) GG_CASE(GGUF_Q4_1) GG_CASE(GGUF_Q5_0) GG_CASE(GGUF_Q5_1) GG_CASE(GGUF_Q8_0)
        GG_CASE(GGUF_Q2_K) GG_CASE(GGUF_Q3_K) GG_CASE(GGUF_Q4_K) GG_CASE(GGUF_Q5_K)
#undef GG_CASE
        default: return 16 * piece_stride(GGUF_Q6_K);
    }
}

// hidden values, their columns, the columns' scales, the routes and how many groups down has
size_t hidden_bytes(int64_t entries, int64_t F) { return (size_t)ceil_div(entries * F * 4, 256) * 256; }
size_t column_bytes(int64_t entries, int64_t F) { return (size_t)(entries * ceil_div(F, kChunk) * 2 * kColStride); }
size_t scale_bytes(int64_t entries, int64_t F) { return (size_t)ceil_div(entries * ceil_div(F, kChunk) * 4, 16) * 16; }

}  // namespace

size_t moe_ffn_workspace_bytes(int64_t F, int64_t T, int64_t top_k) {
    const int64_t entries = T * top_k;
    return hidden_bytes(entries, F) + column_bytes(entries, F) + scale_bytes(entries, F) + 16 + Routes::bytes((int)entries);
}

int moe_ffn_launch(MoeFfnParams p, void* workspace, int num_sms, int pdl, cudaStream_t s) {
    const int entries = p.T * p.top_k;
    p.h = static_cast<float*>(workspace);
    p.columns = static_cast<uint8_t*>(workspace) + hidden_bytes(entries, p.F);
    p.column_scales = reinterpret_cast<float*>(p.columns + column_bytes(entries, p.F));
    p.routes = reinterpret_cast<uint8_t*>(p.column_scales) + scale_bytes(entries, p.F);
    p.x_parts = p.xdt == GGUF_DT_F32 ? 2 : 1;           // the 16-bit types' values are f16 numbers, scaled
    // the hidden values' rounding to f16 is below what a bf16 output rounds, and would not be below an f16 output's (two columns
    // for bf16 as well: 64 tokens through 8 of 128 experts 133 us and not 123, 64 rows of each of 8 experts 150 and not 107; the
    // error against 64 bits is bf16's own, 1.7e-3 by norm, either way)
    p.h_parts = p.ydt == GGUF_DT_BF16 ? 1 : 2;
    const size_t routes = Routes::bytes(entries);

    // up: two tiles of columns where the experts have 48 columns and more each, by the mean, and there is room for two
    // pieces to a warp beside them.  A second tile saves taking the blocks apart again, and leaves half as many jobs to
    // share out, each with more to add up at its end.  2048 x 768 through 8 experts, one tile / two: 16 columns each 37 /
    // 46 us, 32 61 / 65, 64 109 / 108, 64 of Q5_0 and Q5_1 142 / 124; 4 each of 128 experts 123 / 127.
    const int64_t chunks = ceil_div(p.K, kChunk);
    p.up_slot = std::max(slot_bytes(p.gate_type), slot_bytes(p.up_type));
    auto fixed = [&](int64_t held, int tiles) { return routes + (size_t)(held * tiles * (kTileBytes + 32) + 2 * kWarps * 128 * tiles * 4); };
    auto stages = [&](size_t used, size_t slot) { return used > kSmem ? 0 : (int)std::min<size_t>(kMaxStages, (kSmem - used) / (kWarps * slot)); };
    p.up_tiles = entries * p.x_parts >= 48 * std::min(entries, p.n_expert) && stages(fixed(chunks, 2), p.up_slot) >= 2 ? 2 : 1;
    // The columns of all of K stay in shared memory while one piece a warp still fits: making them again for every job costs
    // more than a ring of one piece.  8 tokens through 2 of 8 experts of K x 2048, held / one chunk a warp at a time with two or
    // three pieces: Q6_K, 5120 108 / 173 us, 7168 133 / 225, 8192 155 / 261; Q8_0, 5120 110 / 163, 7168 135 / 213; Q5_K, 7168
    // 99 / 193; Q4_K, 8192 106 / 211.  One token, Q6_K: 38 / 41, 45 / 50, 52 / 57.
    p.up_resident = stages(fixed(chunks, p.up_tiles), p.up_slot) >= 1;
    const size_t up_fixed = fixed(p.up_resident ? chunks : kWarps, p.up_tiles);
    p.up_stages = stages(up_fixed, p.up_slot);
    // what making the routes takes is shared with the columns and the ring
    const size_t up_smem = std::max(up_fixed + (size_t)kWarps * p.up_stages * p.up_slot, routes + routes_scratch(entries, p.n_expert));
    // Few jobs, larger teams: one token's one expert of 2048 x 768 takes 13.3 us with teams of 4 warps, 12.6 with 16;
    // 64 tokens through 8 of 128 experts take 139 us with teams of 16, 123 with 4.
    const int64_t jobs = ceil_div(p.F, 16) * std::min(entries, p.n_expert);
    p.up_wp = jobs <= num_sms ? 8 : jobs <= 2 * num_sms ? 4 : 2;
    while (p.up_wp > chunks) p.up_wp /= 2;
    const int64_t most = ceil_div(p.F, 16) * entries;
    int st = dispatch_up(p.gate_type == p.up_type ? p.gate_type : -1, p, (int)std::min<int64_t>(num_sms, most),
                         up_smem, pdl, s);
    if (st != GGUF_OK) return st;

    const int64_t fchunks = ceil_div(p.F, kChunk);
    st = cuda_status(launch_pdl(moe_ffn_columns_kernel, dim3((unsigned)ceil_div(entries * fchunks, 8)), dim3(256), 0, s, pdl, p));
    if (st != GGUF_OK) return st;

    // down: with few experts, several warps share one's chunks, so that each warp has some three shares to take, as
    // far as there is room for their sums and two pieces to a warp (three tokens through 14336 x 4096: 299 us with one
    // warp to an expert's row tile, 213 so; 64 tokens through 8 of 128 experts: 123 either way; 64 rows of each of 8 experts: 97 with
    // one, 107 so)
    const size_t slot = slot_bytes(p.down_type), one = (size_t)entries * 16 * 4, down_fixed = routes + (entries + 3) / 4 * 16;
    const int64_t room = ((int64_t)kSmem - (int64_t)down_fixed - (int64_t)(kWarps * 2 * slot)) / (int64_t)one;
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({ceil_div(3 * kWarps, std::min(entries, p.n_expert)), fchunks, room}));
    p.down_stages = stages(down_fixed + p.splits * one, slot);
    return dispatch_down(p, down_fixed + p.splits * one + kWarps * p.down_stages * slot, pdl, s);
}

}  // namespace gg
