// kvq_attend_rows.cuh -- what the attention and the attention-mass kernels share:
// cached rows decoded to fp16, the powers of two that keep them and the
// queries within it, and the split of blocks over CTAs.
#pragma once

#include <math.h>

#include "kvq_attend.cuh"

namespace kvq {
namespace {

constexpr int kNoToken = 0x7FFFFFFF;  // in the place of a row's power of two: no such token

template <Layout L>
struct Raw {  // 16 codes
    uint32_t w[L == Layout::V41 ? 4 : 2];
};

// Vector e of 16 codes: codes times `mul` (fp16 twice) as fp16 pairs.
template <Layout L>
__device__ __forceinline__ void decode8(const Raw<L> &r, int e, uint32_t mul, uint32_t (&o)[4]) {
    if constexpr (L == Layout::V41) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 t;\n\t"
                "mov.b32 {lo, hi}, %2;\n\t"
                "cvt.rn.f16x2.e4m3x2 t, lo;\n\tmul.rn.f16x2 %0, t, %3;\n\t"
                "cvt.rn.f16x2.e4m3x2 t, hi;\n\tmul.rn.f16x2 %1, t, %3;\n\t}"
                : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
                : "r"(r.w[2 * e + i]), "r"(mul));
    } else {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 t;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b0;\n\tmul.rn.f16x2 %0, t, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b1;\n\tmul.rn.f16x2 %1, t, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b2;\n\tmul.rn.f16x2 %2, t, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b3;\n\tmul.rn.f16x2 %3, t, %5;\n\t}"
            : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
            : "r"(r.w[e]), "r"(mul));
    }
}

// A row's scales.  FP4: code * e4m3 scale is exact in fp16 as it is.  V41: the
// ue8m0 scales of a row span more than fp16 does, so a row is decoded times
// 2^-texp, which brings its largest scale to 2^7 (448 * 2^7 < 65504); the
// softmax warps put 2^texp back into the scores and the weights.  A
// block whose scale is 2^-32 of the row's largest or less vanishes, other
// values are off by at most 2^-40 of the row's largest value; both are below
// what fp32 sums of the row resolve.  A row whose largest scale is below 2^-40 counts as
// if it were 2^-40, which keeps the weights of tiny rows apart from zero.
constexpr int kMinScaleByte = 127 - 40;
// A V41 score is S 2^texp c with S the product of the fp16 operands (up to 2^40), 2^texp (2^-47 to 2^121) the row's and c
// the query row's factor (down to 2^-127 and less).  S 2^texp alone can pass fp32, so 2^kLift of the row's power is c's.
// The weights of the outputs are relative to the running maximum m of score + texp, 2^(x - m); their sum, which has no
// row in it, takes 2^(x - m - texp).  A row of small power beside one of large power has a weight that fp32 cannot hold
// in the first and can have as large a share of the second as any, so what is computed is E = 2^(x - m - texp + kLift):
// the sum takes E (2^94 at most, and 2^-89 at least for the token that is the maximum), the outputs E 2^(texp - kLift).
constexpr int kLift = 32;

// scale 2^(127 - up) 2^lift, within fp32's finite values (a score that is 0 stays 0, whatever its factor).  A query row
// that is not finite, whose scores are infinite or NaN one and all, has the factor NaN, as all scores of -inf would look
// like no token seen.
constexpr uint32_t kUpNotFinite = 268 - 255;
template <Layout L>
__device__ __forceinline__ float score_factor(float scale, uint32_t up) {
    if (up == kUpNotFinite) return NAN;
    const int e = 127 - int(up) + (L == Layout::V41 ? kLift : 0), half = e / 2;  // -127 .. 146
    const float f = scale * __uint_as_float(uint32_t(127 + half) << 23) * __uint_as_float(uint32_t(127 + e - half) << 23);
    return fminf(fmaxf(f, -3.4e38f), 3.4e38f);
}

template <Layout L>
__device__ __forceinline__ int row_texp(const uint4 &v) {
    if constexpr (L == Layout::FP4) return 0;
    // largest byte: even and odd bytes as 16-bit lanes
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        hi = __vmaxu2(hi, (w[b] >> 8) & 0x00FF00FFu);
        lo = __vmaxu2(lo, w[b] & 0x00FF00FFu);
    }
    lo = __vmaxu2(lo, hi);
    return max(max(int(lo >> 16), int(lo & 0xFFFFu)), kMinScaleByte) - 134;
}

// A block's multiplier, fp16 twice.
template <Layout L>
__device__ __forceinline__ uint32_t block_mul(uint32_t byte, int texp) {
    uint32_t r;
    if constexpr (L == Layout::V41) {
        // 2^(byte - 127 - texp): through bf16, which holds every ue8m0 value and NaN
        uint32_t h;
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(h) : "h"(uint16_t(byte)));
        const float f = bf16_lo(h) * __uint_as_float(uint32_t(127 - texp) << 23);
        asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(f));
    } else {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(byte * 0x101u)));
    }
    return r;
}

// This CTA's share [u0, u1) of `total` blocks: as equal as can be, none past the first `total` CTAs.
__device__ __forceinline__ void share(int64_t total, int64_t &u0, int64_t &u1) {
    const int64_t g = min(int64_t(gridDim.x), total), x = blockIdx.x;
    if (x >= g) {
        u0 = u1 = 0;
    } else if (total <= 0xFFFFFFFFll / (kMaxAttendCtas + 1)) {  // short divisions
        u0 = uint32_t(x) * uint32_t(total) / uint32_t(g);
        u1 = uint32_t(x + 1) * uint32_t(total) / uint32_t(g);
    } else {
        u0 = x * total / g;
        u1 = (x + 1) * total / g;
    }
}

}  // namespace
}  // namespace kvq
