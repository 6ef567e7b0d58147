// kvq_rope.cu -- rotary positions outside the store: the table of cosines and
// sines that kvq_store reads (kvq_rope_table), and the rotation of rows that
// are not stored, queries before the attention and its outputs after it
// (kvq_rope).
#include <math.h>

#include "kvq_launch.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------- table
// table[p, i] = A cos((first + p) f_i), table[p, h + i] = A sin(...), h = rot / 2.
//
// What matters of an angle is its fraction of a turn, and a fraction of a turn
// times a whole number is exact in integers modulo 2^64: with
// F = round(2^64 frac(f / 2 pi)) the phase of position p is p F mod 2^64, off
// by p 2^-65 turns, less than 2^-34 at every position.  F comes from f's 53 bits
// times 126 bits of 1 / 2 pi, in integers too: of a product of doubles, off by
// 2^-53 of itself, far positions of fast pairs show the error (10^-4 at position
// 10^6 of a million radians each).  A step of rows is an integer addition.  The
// top two bits (after half a quarter is added) are the quadrant, the rest an
// angle within pi / 4 whose sine and cosine are their Taylor series up to x^9
// and x^10 (what is left out is below 2^-28 and 2^-32).
//
// Bound by the stores: 1,048,576 x 64 in 42.5 us is 6.3 TB/s; 8,192 x 64 in 2.4 us
// (with F by doubles 42.0 and 2.3).
constexpr int kTabThreads = 256;
constexpr int kMaxRot = 1024;

struct TableArgs {
    const double *freq;
    int h;
    int64_t first, rows;
    float amplitude;
    float *table;
};

// 2^64 frac(f / 2 pi), rounded, for |f| < 2^55.
__device__ __forceinline__ uint64_t turn_step(double f) {
    constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;  // 2^128 / 2 pi
    const uint64_t bits = uint64_t(__double_as_longlong(f));
    const int e = int(bits >> 52) & 0x7FF;
    const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (e ? 1ull << 52 : 0ull);  // |f| = m 2^(max(e, 1) - 1075)
    const int right = 64 + 1075 - max(e, 1);                                   // of the product with 2^128 / 2 pi
    const uint64_t p0 = m * kLo, up = __umul64hi(m, kLo), mid = m * kHi;
    const uint64_t p1 = up + mid, p2 = __umul64hi(m, kHi) + (p1 < mid ? 1 : 0);
    if (right >= 192 || right < 62) return 0;  // nothing is left of it; out of range
    const int w = right >> 6, r = right & 63;
    const uint64_t a0 = w == 0 ? p0 : w == 1 ? p1 : p2, a1 = w == 0 ? p1 : w == 1 ? p2 : 0;
    const uint64_t below = r ? a0 : w == 1 ? p0 : p1;  // the word that the bit to round by is in
    const uint64_t v = (r ? (a0 >> r) | (a1 << (64 - r)) : a0) + ((below >> ((right - 1) & 63)) & 1);
    return bits >> 63 ? 0 - v : v;
}

__device__ __forceinline__ void turn_sincos(uint64_t phase, float &s, float &c) {
    const uint32_t hi = uint32_t(phase >> 32) + 0x20000000u;
    const int32_t r = int32_t(hi & 0x3FFFFFFFu) - 0x20000000;  // a 2^32nd of a turn each
    const float x = float(r) * 1.4629180792671596e-9f;         // 2 pi / 2^32
    const float y = x * x;
    float a = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);  // 1 / 9!, 1 / 7!
    a = fmaf(y, a, 8.3333333e-3f);
    a = fmaf(y, a, -1.6666667e-1f);
    const float sx = fmaf(x * y, a, x);
    float b = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);  // 1 / 10!, 1 / 8!
    b = fmaf(y, b, -1.3888889e-3f);
    b = fmaf(y, b, 4.1666667e-2f);
    b = fmaf(y, b, -0.5f);
    const float cx = fmaf(y, b, 1.f);
    const bool odd = hi & 0x40000000u;
    s = odd ? cx : sx;
    c = odd ? sx : cx;
    s = __uint_as_float(__float_as_uint(s) ^ (hi & 0x80000000u));
    c = __uint_as_float(__float_as_uint(c) ^ ((hi ^ (hi << 1)) & 0x80000000u));
}

// V columns a thread, the same ones in every row that it writes.
template <int V>
__global__ void __launch_bounds__(kTabThreads) rope_table_kernel(const TableArgs a) {
    __shared__ uint64_t s_step[kMaxRot / 2];  // a column's phase for one position
    __shared__ float s_amp[kMaxRot / 2];
    pdl_wait();
    for (int i = threadIdx.x; i < a.h; i += kTabThreads) {
        const double f = a.freq[i];
        const bool fine = fabs(f) * 0.15915494309189535 < 4503599627370496.0;  // turns; a double has no fraction of more
        s_step[i] = fine ? turn_step(f) : 0;
        s_amp[i] = fine ? a.amplitude : NAN;
    }
    __syncthreads();
    pdl_trigger();
    const int groups = a.h / V;                       // threads a row
    const int per = groups < kTabThreads ? kTabThreads / groups : 1;  // rows a CTA has at a time
    const int r0 = groups < kTabThreads ? threadIdx.x / groups : 0;
    if (r0 >= per) return;
    for (int g = groups < kTabThreads ? threadIdx.x % groups : threadIdx.x; g < groups; g += kTabThreads) {
        uint64_t phase[V], step[V];
        float amp[V];
        int64_t row = int64_t(blockIdx.x) * per + r0;
        const int64_t stride = int64_t(gridDim.x) * per;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            phase[v] = s_step[g * V + v] * uint64_t(a.first + row);
            step[v] = s_step[g * V + v] * uint64_t(stride);
            amp[v] = s_amp[g * V + v];
        }
        float *to = a.table + row * (2 * a.h) + g * V;
        for (; row < a.rows; row += stride, to += stride * (2 * a.h)) {
            float s[V], c[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                turn_sincos(phase[v], s[v], c[v]);
                s[v] *= amp[v], c[v] *= amp[v];
                phase[v] += step[v];
            }
            if constexpr (V == 4) {
                *reinterpret_cast<float4 *>(to) = make_float4(c[0], c[1], c[2], c[3]);
                *reinterpret_cast<float4 *>(to + a.h) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
                to[0] = c[0];
                to[a.h] = s[0];
            }
        }
    }
}

// ---------------------------------------------------------------- rotation
// (u, v) -> (u c - v s, v c + u s), or with the sine's sign turned the way back
// (the transpose).  A pair is neighbours (interleaved) or rot / 2 apart
// (halves).  A row's work is cut into pieces of 16 or 8 bytes: first those that
// are rotated, with halves two at a time, then those that are copied (none where
// the rows are rotated in place).  A thread has the same piece of several heads
// of one token, so it reads its cosines and sines once; the heads' loads are all
// under way before the first is used.
//
// Bound by memory: a value is read once and written once, and some 45
// instructions go to the 32 bytes of a piece.  8,191 tokens of 64 heads, bf16
// rows of 512 (1.08 GB): 159 us = 6.8 TB/s; one token of 16 heads: 1.8 us.
// (A thread's first rows requested after its position instead of before it:
// 161 and 1.9.  Rotated and copied pieces one after the other: 179.)
constexpr int kRopeThreads = 256, kRopeBatch = 4;

struct RopeArgs {
    const uint8_t *x;
    uint8_t *out;
    int64_t x_tok, x_head, out_tok, out_head;  // bytes
    int64_t n;
    int heads, start, rot;  // elements
    int turning, copied;    // a row's pieces that are rotated, those that are copied (value by value: pairs, values)
    int heads_cta, splits;  // heads a CTA has, CTAs a token
    const float *cos_sin;
    int64_t rows;
    const int32_t *pos;
    int32_t *err;
    float sign;
};

// W words.  Not by way of the read-only path: the rows may be rotated in place.
template <int W>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&r)[W]) {
    if constexpr (W == 4) {
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "l"(p)
                     : "memory");
    } else {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p) : "memory");
    }
}
template <int W>
__device__ __forceinline__ void store_words(uint8_t *p, const uint32_t (&r)[W]) {
    if constexpr (W == 4) st_u4(p, make_uint4(r[0], r[1], r[2], r[3]));
    else *reinterpret_cast<uint2 *>(p) = make_uint2(r[0], r[1]);
}

// One element, bf16 or fp32, from / to memory.
template <bool kBf16>
__device__ __forceinline__ float load_one(const uint8_t *p) {
    if constexpr (kBf16) return __uint_as_float(uint32_t(*reinterpret_cast<const volatile uint16_t *>(p)) << 16);
    else return *reinterpret_cast<const volatile float *>(p);
}
template <bool kBf16>
__device__ __forceinline__ void store_one(uint8_t *p, float v) {
    if constexpr (kBf16) *reinterpret_cast<uint16_t *>(p) = uint16_t(pack_bf16x2(v, 0.f));
    else *reinterpret_cast<float *>(p) = v;
}

template <bool kBf16, int W>
__device__ __forceinline__ void unpack(const uint32_t (&w)[W], float (&v)[kBf16 ? 2 * W : W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if constexpr (kBf16) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        } else {
            v[i] = __uint_as_float(w[i]);
        }
    }
}
template <bool kBf16, int W>
__device__ __forceinline__ void pack(const float (&v)[kBf16 ? 2 * W : W], uint32_t (&w)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if constexpr (kBf16) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else w[i] = __float_as_uint(v[i]);
    }
}

// Pieces of W words.
template <bool kBf16, bool kHalf, int W>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    constexpr int kItem = kBf16 ? 2 : 4, E = 4 * W / kItem;
    constexpr int kUse = kHalf ? E : E / 2;  // cosines of a piece
    const int64_t tok = int64_t(blockIdx.x) / a.splits;
    const int h0 = int(int64_t(blockIdx.x) % a.splits) * a.heads_cta, h1 = min(a.heads, h0 + a.heads_cta);
    const int half = a.rot / 2;
    const int pieces = a.turning + a.copied, width = min(pieces, kRopeThreads), lines = kRopeThreads / width;
    const int line = threadIdx.x / width;
    if (line >= lines) return;
    uint32_t u[kRopeBatch][W], w[kHalf ? kRopeBatch : 1][W];
    // a piece's first element
    auto element = [&](int piece) {
        if (piece < a.turning) return a.start + piece * E;
        const int at = (piece - a.turning) * E;
        return at < a.start ? at : at + a.rot;
    };
    auto load = [&](int piece, int h) {
        const uint8_t *from = a.x + tok * a.x_tok + int64_t(element(piece)) * kItem;
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            const int hb = h + b * lines;
            if (hb < h1) {
                load_words<W>(from + hb * a.x_head, u[b]);
                if constexpr (kHalf) {
                    if (piece < a.turning) load_words<W>(from + hb * a.x_head + half * kItem, w[b]);
                }
            }
        }
    };
    int piece = threadIdx.x % width;
    pdl_wait();
    load(piece, h0 + line);  // while the position and its row of the table come
    bool loaded = true;
    const int32_t pos = __ldg(a.pos + tok);
    const bool good = pos >= 0 && pos < a.rows;
    if (!good) {
        if (threadIdx.x == 0 && h0 == 0) raise_err(a.err, KVQ_DEVERR_POS);
        return;
    }
    pdl_trigger();
    for (; piece < pieces; piece += width) {
        const bool turns = piece < a.turning;
        uint8_t *to = a.out + tok * a.out_tok + int64_t(element(piece)) * kItem;
        float c[kUse], s[kUse];
        if (turns) {
            const float *t = a.cos_sin + int64_t(pos) * a.rot + piece * kUse;
            if constexpr (kUse % 2 == 0) {
#pragma unroll
                for (int i = 0; i < kUse; i += 2) {  // halves of a table row need not be 16-byte aligned
                    const float2 cc = __ldg(reinterpret_cast<const float2 *>(t + i));
                    const float2 ss = __ldg(reinterpret_cast<const float2 *>(t + half + i));
                    c[i] = cc.x, c[i + 1] = cc.y;
                    s[i] = ss.x * a.sign, s[i + 1] = ss.y * a.sign;
                }
            } else {
                c[0] = __ldg(t);
                s[0] = __ldg(t + half) * a.sign;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kUse; ++i) c[i] = 1.f, s[i] = 0.f;
        }
        for (int h = h0 + line; h < h1; h += kRopeBatch * lines) {
            if (!loaded) load(piece, h);
            loaded = false;
#pragma unroll
            for (int b = 0; b < kRopeBatch; ++b) {
                const int hb = h + b * lines;
                if (hb >= h1) continue;
                uint8_t *o = to + hb * a.out_head;
                if (!turns) {
                    store_words<W>(o, u[b]);
                    continue;
                }
                float v[E];
                unpack<kBf16, W>(u[b], v);
                if constexpr (kHalf) {
                    float z[E];
                    unpack<kBf16, W>(w[b], z);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float p = __fsub_rn(__fmul_rn(v[i], c[i]), __fmul_rn(z[i], s[i]));
                        z[i] = __fadd_rn(__fmul_rn(z[i], c[i]), __fmul_rn(v[i], s[i]));
                        v[i] = p;
                    }
                    pack<kBf16, W>(z, w[b]);
                    store_words<W>(o + half * kItem, w[b]);
                } else {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        const float p = __fsub_rn(__fmul_rn(v[2 * i], c[i]), __fmul_rn(v[2 * i + 1], s[i]));
                        v[2 * i + 1] = __fadd_rn(__fmul_rn(v[2 * i + 1], c[i]), __fmul_rn(v[2 * i], s[i]));
                        v[2 * i] = p;
                    }
                }
                pack<kBf16, W>(v, u[b]);
                store_words<W>(o, u[b]);
            }
        }
    }
}

// The same, value by value: rows, heads or rotated parts that do not come in
// pieces of 8 bytes.  A thread has one pair or one copied value of a head.
// Bound by its instructions, of which a 64-bit division a value is most: the
// 8,191 x 64 rows of 512 off by one value 635 us, in place (64 values) 72.
template <bool kBf16>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const RopeArgs a, bool halves) {
    constexpr int kItem = kBf16 ? 2 : 4;
    const int64_t tok = int64_t(blockIdx.x) / a.splits;
    const int h0 = int(int64_t(blockIdx.x) % a.splits) * a.heads_cta, h1 = min(a.heads, h0 + a.heads_cta);
    const int half = a.rot / 2;
    pdl_wait();
    const int32_t pos = __ldg(a.pos + tok);
    const bool good = pos >= 0 && pos < a.rows;
    if (!good) {
        if (threadIdx.x == 0 && h0 == 0) raise_err(a.err, KVQ_DEVERR_POS);
        return;
    }
    pdl_trigger();
    const float *t = a.cos_sin + int64_t(pos) * a.rot;
    const int pieces = a.turning + a.copied;
    for (int64_t i = threadIdx.x; i < int64_t(h1 - h0) * pieces; i += kRopeThreads) {
        const int h = h0 + int(i / pieces), k = int(i % pieces);
        const uint8_t *from = a.x + tok * a.x_tok + h * a.x_head;
        uint8_t *to = a.out + tok * a.out_tok + h * a.out_head;
        if (k >= half) {  // copied
            const int el = k - half < a.start ? k - half : k - half + a.rot;
            store_one<kBf16>(to + el * kItem, load_one<kBf16>(from + el * kItem));
            continue;
        }
        const int u = a.start + (halves ? k : 2 * k), v = halves ? u + half : u + 1;
        const float c = __ldg(t + k), s = __ldg(t + half + k) * a.sign;
        const float x = load_one<kBf16>(from + u * kItem), y = load_one<kBf16>(from + v * kItem);
        store_one<kBf16>(to + u * kItem, __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)));
        store_one<kBf16>(to + v * kItem, __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)));
    }
}

// Whether rows of `dim` elements, (n, heads) of them, lie apart: one stride spans the other axis.
bool rows_apart(int64_t n, int64_t heads, int64_t dim, int64_t tok, int64_t head) {
    if (n > 1 && tok < dim) return false;
    if (heads > 1 && head < dim) return false;
    if (n > 1 && heads > 1) {
        const bool by_token = tok >= head;
        const int64_t inner = by_token ? head : tok, outer = by_token ? tok : head;
        if (outer - dim < inner * ((by_token ? heads : n) - 1)) return false;
    }
    return true;
}

// Whether two sets of rows (elements' byte size `item`) certainly share no byte: apart as ranges, or with equal strides
// beside each other in every pitch.
bool sets_apart(const void *xp, const void *op, int64_t n, int64_t heads, int64_t dim, int64_t x_tok, int64_t x_head,
                int64_t o_tok, int64_t o_head, int64_t item) {
    const int64_t x = int64_t(reinterpret_cast<uintptr_t>(xp)), o = int64_t(reinterpret_cast<uintptr_t>(op));
    const int64_t xs = ((n - 1) * x_tok + (heads - 1) * x_head + dim) * item;
    const int64_t os = ((n - 1) * o_tok + (heads - 1) * o_head + dim) * item;
    if (x + xs <= o || o + os <= x) return true;
    if ((n > 1 && x_tok != o_tok) || (heads > 1 && x_head != o_head)) return false;
    const int64_t tok = n > 1 ? x_tok : 0, head = heads > 1 ? x_head : 0;
    const int64_t pitch = (tok && head ? (tok < head ? tok : head) : tok + head) * item;
    if (pitch <= 0 || (tok * item) % pitch || (head * item) % pitch) return false;
    const int64_t off = ((o - x) % pitch + pitch) % pitch;
    return off >= dim * item && off <= pitch - dim * item;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_rope_table(const double *freq, int64_t rot_dim, int64_t first, int64_t rows, float amplitude,
                                     float *table, struct CUstream_st *stream) {
    if (rot_dim < 2 || rot_dim % 2 || rows < 0 || first < 0) return KVQ_ERR_INVALID_ARG;
    if (rot_dim > kMaxRot || rows > 0x7FFFFFFFll || first > 0x7FFFFFFFll - rows) return KVQ_ERR_UNSUPPORTED;
    if (!(amplitude - amplitude == 0.f)) return KVQ_ERR_INVALID_ARG;  // NaN or infinite
    if (!freq || !aligned(freq, 8)) return KVQ_ERR_INVALID_ARG;
    if (rows == 0) return KVQ_OK;
    if (!table || !aligned(table, 16)) return KVQ_ERR_INVALID_ARG;
    TableArgs a = {};
    a.freq = freq;
    a.h = int(rot_dim / 2);
    a.first = first;
    a.rows = rows;
    a.amplitude = amplitude;
    a.table = table;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // four columns a thread, stored as 16 bytes, where columns come in fours
    return with_bool(a.h % 4 == 0, [&](auto Vc) {
        constexpr int V = decltype(Vc)::value ? 4 : 1;
        int64_t cap = 0;
        kvq_status st = resident_grid<rope_table_kernel<V>, kTabThreads>(0, &cap);
        if (st != KVQ_OK) return st;
        const int64_t groups = a.h / V, per = groups < kTabThreads ? kTabThreads / groups : 1;
        const int64_t need = (rows + per - 1) / per;
        return launch_pdl(rope_table_kernel<V>, dim3(unsigned(need < cap ? need : cap)), dim3(kTabThreads), s, a);
    });
}

extern "C" kvq_status kvq_rope(const void *x, kvq_dtype dtype, int64_t n_tokens, int64_t heads, int64_t dim,
                               int64_t x_token_stride, int64_t x_head_stride, int64_t rot_start, int64_t rot_dim,
                               unsigned flags, const float *cos_sin, int64_t cos_sin_rows, const int32_t *pos, void *out,
                               int64_t out_token_stride, int64_t out_head_stride, int32_t *err,
                               struct CUstream_st *stream) {
    if (dtype != KVQ_F32 && dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
    if (flags & ~unsigned(KVQ_ROPE_HALF | KVQ_ROPE_INVERSE)) return KVQ_ERR_INVALID_ARG;
    if (n_tokens < 0 || heads < 1 || dim < 2 || cos_sin_rows < 0) return KVQ_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim % 2 || rot_start < 0 || rot_dim > dim || rot_start > dim - rot_dim) return KVQ_ERR_INVALID_ARG;
    if (rot_dim > kMaxRot || dim > (1 << 16) || heads > (1 << 16) || n_tokens > (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
    if (err && !aligned(err, 4)) return KVQ_ERR_INVALID_ARG;
    if (n_tokens == 0) return KVQ_OK;
    const int64_t item = dtype == KVQ_BF16 ? 2 : 4;
    if (!x || !out || !aligned(x, item) || !aligned(out, item) || !pos || !aligned(pos, 4)) return KVQ_ERR_INVALID_ARG;
    if (cos_sin_rows > 0 && (!cos_sin || !aligned(cos_sin, 8))) return KVQ_ERR_INVALID_ARG;
    if (n_tokens == 1) x_token_stride = out_token_stride = 0;  // the stride of an axis of one element is never used
    if (heads == 1) x_head_stride = out_head_stride = 0;
    const int64_t most = int64_t(1) << 58;  // elements that an axis spans: sums of bytes fit 64 bits
    if (x_token_stride < 0 || x_head_stride < 0 || x_token_stride > most / n_tokens || x_head_stride > most / heads ||
        out_token_stride > most / n_tokens || out_head_stride > most / heads)
        return KVQ_ERR_INVALID_ARG;
    if (!rows_apart(n_tokens, heads, dim, out_token_stride, out_head_stride)) return KVQ_ERR_INVALID_ARG;
    const bool in_place = x == out && x_token_stride == out_token_stride && x_head_stride == out_head_stride;
    if (!in_place && !sets_apart(x, out, n_tokens, heads, dim, x_token_stride, x_head_stride, out_token_stride, out_head_stride, item))
        return KVQ_ERR_INVALID_ARG;

    const bool halves = flags & KVQ_ROPE_HALF;
    RopeArgs a = {};
    a.x = static_cast<const uint8_t *>(x);
    a.out = static_cast<uint8_t *>(out);
    a.x_tok = x_token_stride * item;
    a.x_head = x_head_stride * item;
    a.out_tok = out_token_stride * item;
    a.out_head = out_head_stride * item;
    a.n = n_tokens;
    a.heads = int(heads);
    a.start = int(rot_start);
    a.rot = int(rot_dim);
    a.cos_sin = cos_sin;
    a.rows = cos_sin_rows;
    a.pos = pos;
    a.err = err;
    a.sign = (flags & KVQ_ROPE_INVERSE) ? -1.f : 1.f;
    // 16 or 8 bytes at a time where rows, the rotated part and (with halves) its halves begin and end on such a boundary.
    // Halves of bf16 rows go by 8 (a piece is two places of a row, and twice as many cosines in registers cost more than
    // shorter loads: 8,000 x 64 rows of 128, 64 rotated, 51.6 us by 8, 59.6 by 16; fp32, 8,000 x 30 of 336, 125 and 117).
    auto fits = [&](int64_t bytes) {
        const int64_t E = bytes / item;
        return aligned(x, bytes) && aligned(out, bytes) && x_token_stride % E == 0 && x_head_stride % E == 0 &&
               out_token_stride % E == 0 && out_head_stride % E == 0 && dim % E == 0 && rot_start % E == 0 &&
               rot_dim % (halves ? 2 * E : E) == 0;
    };
    const int words = fits(16) && !(halves && dtype == KVQ_BF16) ? 4 : fits(8) ? 2 : 0;
    const int64_t E = words ? words * 4 / item : 1;
    a.turning = int(words && !halves ? rot_dim / E : rot_dim / 2 / E);
    a.copied = int(in_place ? 0 : (dim - rot_dim) / E);
    // heads that a CTA has at a time, and those it has under way
    const int64_t pieces = int64_t(a.turning) + a.copied;
    const int64_t lines = pieces < kRopeThreads ? kRopeThreads / pieces : 1, step = words ? kRopeBatch * lines : lines;
    // A CTA has a token's heads; fewer where there are too few tokens to fill the machine.
    constexpr int64_t kFill = 608;
    int64_t per = n_tokens >= kFill ? heads : (n_tokens * heads + kFill - 1) / kFill;
    per = (per + lines - 1) / lines * lines;
    if (per > lines && per < step) per = step < heads ? step : heads;
    a.heads_cta = int(per < heads ? per : heads);
    a.splits = int((heads + a.heads_cta - 1) / a.heads_cta);
    const int64_t blocks = n_tokens * a.splits;
    if (blocks > 0x7FFFFFFF) return KVQ_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_bool(dtype == KVQ_BF16, [&](auto Bc) {
        constexpr bool B = decltype(Bc)::value;
        if (!words) return launch_pdl(rope_any_kernel<B>, dim3(unsigned(blocks)), dim3(kRopeThreads), s, a, halves);
        return with_bool(halves, [&](auto Hc) {
            constexpr bool H = decltype(Hc)::value;
            if constexpr (!(B && H)) {
                if (words == 4) return launch_pdl(rope_kernel<B, H, 4>, dim3(unsigned(blocks)), dim3(kRopeThreads), s, a);
            }
            return launch_pdl(rope_kernel<B, H, 2>, dim3(unsigned(blocks)), dim3(kRopeThreads), s, a);
        });
    });
}
