// kvq_norm_quant.cu -- RMS norm of x + residual, written as V41 blocks: e4m3
// codes and one ue8m0 scale per 32 values ("[sglang] DeepSeek V4.1 Paged KV
// Cache: V41 and FP4 formats", section 1, the block rule; the fused K norm of
// its store-latency table for the norm).
//
// With z = x + residual, r = 1 / sqrt(mean(z^2) + eps): y = z r weight, and per
// block of 32 the scale byte b = exponent field of max |y| minus 8 and the
// codes e4m3(y 2^(127 - b)).  A value costs 4 to 8 bytes of traffic and some
// ten operations, so a large call is bound by memory and a small one by the
// latency of a row: one load, the sum over the row, one store.
//
// A row is read once: W warps hold it in registers (ITER pieces of 8 values a
// thread, piece i of thread t is t + 32 W i), so the sum of squares, the block
// maxima and the outputs all come from one pass over memory.  A quant block is
// the pieces of four neighbouring lanes, its maximum two shuffles.
//
// One piece a thread makes the shortest row (bf16 with residual, 1 row and 300
// rows: dim 512 with 2 warps 1.7 and 2.1 us, with 1 warp 2.2 and 2.6; dim 2048
// with 8 warps 1.7 and 2.3, with 4 warps 2.3 and 2.6; dim 4096 with 16 warps
// 2.0 and 2.8, with 8 warps 2.4 and 3.3; dim 16384 with 32 warps 3.7 and 6.1,
// with 8 warps 6.3 and 10.8), so up to dim 2048 a row has just the warps that
// its pieces fill (1537 fp32 rows of 1056: 5 warps 3.3 us, 8 warps 4.0).  Large
// batches agree (8192 rows: dim 1024 with 4
// warps 10.1, with 8 warps 12.9; dim 8192 with 16 warps 75 us = 6.3 TB/s, with
// 8 warps 82, with 32 warps 88; dim 16384 with 32 warps 155, with 8 warps
// 195), but for dim 4096, where two pieces a thread keep more bytes in flight
// (39.1 us = 6.0 TB/s against 40.7).
#include "kvq_launch.cuh"

namespace kvq {
namespace {

// Threads a CTA: as many rows of W warps as eight warps hold, or one.
template <int W>
constexpr int kNqThreads = W >= 8 ? 32 * W : 8 / W * W * 32;
constexpr int64_t kNqMaxDim = 16384;

struct NormQuantArgs {
    const uint8_t *x, *res;
    uint8_t *res_out;
    int64_t x_stride, res_stride, res_out_stride;  // bytes
    const float *w;
    float eps;
    int64_t n;
    int dim;
    uint8_t *codes, *scales;
    int64_t codes_stride, scales_stride;
};

// 16 bytes; with kShared of memory that this kernel may write (residual_out may be an input), so not by way of the
// read-only path.
template <bool kShared>
__device__ __forceinline__ uint4 load16(const uint8_t *p) {
    if constexpr (!kShared) return ld_stream_u4(p);
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

template <bool kBf16, bool kShared>
__device__ __forceinline__ void load8(const uint8_t *p, float (&v)[8]) {
    const uint4 u = load16<kShared>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const uint4 u2 = load16<kShared>(p + 16);
        const uint32_t w2[4] = {u2.x, u2.y, u2.z, u2.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(w[i]);
            v[4 + i] = __uint_as_float(w2[i]);
        }
    }
}

// W warps a row, ITER pieces of 8 values a thread.
template <bool kBf16, bool kRes, int W, int ITER>
__global__ void __launch_bounds__(kNqThreads<W>) norm_quant_kernel(const NormQuantArgs a) {
    constexpr int kRows = kNqThreads<W> / 32 / W;
    constexpr int kPieceBytes = kBf16 ? 16 : 32;
    __shared__ float s_sum[kNqThreads<W> / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (warp % W) * 32 + lane;
    const int64_t row = int64_t(blockIdx.x) * kRows + warp / W;
    const bool live = row < a.n;
    const int pieces = a.dim / 8;

    pdl_wait();
    float z[ITER][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int p = t + 32 * W * i;
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] = 0.f;
        if (live && p < pieces) {
            load8<kBf16, kRes>(a.x + row * a.x_stride + int64_t(p) * kPieceBytes, z[i]);
            if constexpr (kRes) {
                float r[8];
                load8<kBf16, kRes>(a.res + row * a.res_stride + int64_t(p) * kPieceBytes, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[i][e] += r[e];
            }
        }
    }
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(z[i][e], z[i][e], sum);
        const int p = t + 32 * W * i;
        if constexpr (kRes) {
            if (live && p < pieces) {
                uint8_t *o = a.res_out + row * a.res_out_stride + int64_t(p) * kPieceBytes;
                if constexpr (kBf16) {
                    st_u4(o, make_uint4(pack_bf16x2(z[i][0], z[i][1]), pack_bf16x2(z[i][2], z[i][3]),
                                        pack_bf16x2(z[i][4], z[i][5]), pack_bf16x2(z[i][6], z[i][7])));
                } else {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(z[i][e]);
                    st_u4(o, make_uint4(w[0], w[1], w[2], w[3]));
                    st_u4(o + 16, make_uint4(w[4], w[5], w[6], w[7]));
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if constexpr (W > 1) {
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) sum += s_sum[warp / W * W + i];
    }
    const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, float(a.dim)), a.eps));
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int p = t + 32 * W * i;
        const bool on = live && p < pieces;
        uint32_t amax = 0;
        if (on) {
            const float4 w0 = __ldg(reinterpret_cast<const float4 *>(a.w) + 2 * p);
            const float4 w1 = __ldg(reinterpret_cast<const float4 *>(a.w) + 2 * p + 1);
            const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[i][e] = __fmul_rn(__fmul_rn(z[i][e], r), w[e]);
                amax = max(amax, abs_bits(z[i][e]));
            }
        }
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        if (on) {
            const uint32_t sb = v41_scale_byte(amax);
            const float mul = v41_multiplier(sb);
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = cvt_e4m3x2(z[i][2 * e] * mul, z[i][2 * e + 1] * mul);
            *reinterpret_cast<uint2 *>(a.codes + row * a.codes_stride + int64_t(p) * 8) =
                make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
            if ((p & 3) == 0) a.scales[row * a.scales_stride + p / 4] = uint8_t(sb);
        }
    }
}

template <bool kBf16, bool kRes, int W, int ITER>
kvq_status launch_nq(const NormQuantArgs &a, cudaStream_t s) {
    constexpr int kRows = kNqThreads<W> / 32 / W;
    const int64_t blocks = (a.n + kRows - 1) / kRows;
    if (blocks > 0x7FFFFFFF) return KVQ_ERR_INVALID_ARG;
    return launch_pdl(norm_quant_kernel<kBf16, kRes, W, ITER>, dim3(unsigned(blocks)), dim3(kNqThreads<W>), s, a);
}

// Whether some of n rows of `width` bytes, `as` apart from `a`, share a byte with some of n such rows `bs` apart from
// `b`; as, bs >= width.
bool rows_overlap(const void *a_ptr, int64_t as, const void *b_ptr, int64_t bs, int64_t width, int64_t n) {
    const int64_t a = int64_t(reinterpret_cast<uintptr_t>(a_ptr)), b = int64_t(reinterpret_cast<uintptr_t>(b_ptr));
    if (a + (n - 1) * as + width <= b || b + (n - 1) * bs + width <= a) return false;
    // Row i of a against the first row of b that ends behind its start.  With one stride only i - j counts, so the first
    // and the last row stand for all.
    for (int64_t i = 0; i < n; i += as == bs && n > 1 ? n - 1 : 1) {
        const int64_t at = a + i * as, j = at < b + width ? 0 : (at - b - width) / bs + 1;
        if (j < n && b + j * bs < at + width) return true;
    }
    return false;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_norm_quant(const void *x, kvq_dtype x_dtype, int64_t n, int64_t dim, int64_t x_row_stride,
                                     const void *residual, int64_t residual_row_stride, void *residual_out,
                                     int64_t residual_out_row_stride, const float *weight, float eps, uint8_t *codes,
                                     int64_t codes_stride, uint8_t *scales, int64_t scales_stride,
                                     struct CUstream_st *stream) {
    if (x_dtype != KVQ_F32 && x_dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
    if (n < 0 || dim <= 0 || dim % kBlock != 0) return KVQ_ERR_INVALID_ARG;
    if (dim > kNqMaxDim) return KVQ_ERR_UNSUPPORTED;
    if (!(eps >= 0.f)) return KVQ_ERR_INVALID_ARG;
    if ((residual == nullptr) != (residual_out == nullptr)) return KVQ_ERR_INVALID_ARG;
    if (n == 0) return KVQ_OK;  // nothing to enqueue; the arrays may be empty
    const int64_t item = x_dtype == KVQ_BF16 ? 2 : 4;
    auto rows_ok = [&](const void *p, int64_t stride) {
        return p && aligned(p, 16) && (n == 1 || (stride >= dim && stride * item % 16 == 0));
    };
    if (!rows_ok(x, x_row_stride)) return KVQ_ERR_INVALID_ARG;
    if (residual && (!rows_ok(residual, residual_row_stride) || !rows_ok(residual_out, residual_out_row_stride)))
        return KVQ_ERR_INVALID_ARG;
    if (residual) {  // residual_out is an input, row for row, or apart from it
        auto clash = [&](const void *in, int64_t stride) {
            if (in == residual_out && (n == 1 || stride == residual_out_row_stride)) return false;
            const int64_t width = dim * item;
            return rows_overlap(residual_out, n == 1 ? width : residual_out_row_stride * item, in,
                                n == 1 ? width : stride * item, width, n);
        };
        if (clash(x, x_row_stride) || clash(residual, residual_row_stride)) return KVQ_ERR_INVALID_ARG;
    }
    if (!weight || !aligned(weight, 16)) return KVQ_ERR_INVALID_ARG;
    if (!codes || !aligned(codes, 8) || (n > 1 && (codes_stride < dim || codes_stride % 8 != 0)))
        return KVQ_ERR_INVALID_ARG;
    if (!scales || (n > 1 && scales_stride < dim / kBlock)) return KVQ_ERR_INVALID_ARG;

    NormQuantArgs a = {};
    a.x = static_cast<const uint8_t *>(x);
    a.res = static_cast<const uint8_t *>(residual);
    a.res_out = static_cast<uint8_t *>(residual_out);
    a.x_stride = x_row_stride * item;
    a.res_stride = residual_row_stride * item;
    a.res_out_stride = residual_out_row_stride * item;
    a.w = weight;
    a.eps = eps;
    a.n = n;
    a.dim = int(dim);
    a.codes = codes;
    a.scales = scales;
    a.codes_stride = codes_stride;
    a.scales_stride = scales_stride;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_bool(x_dtype == KVQ_BF16, [&](auto Bc) {
        return with_bool(residual != nullptr, [&](auto Rc) {
            constexpr bool B = decltype(Bc)::value, R = decltype(Rc)::value;
            switch ((dim + 255) / 256) {
                case 1: return launch_nq<B, R, 1, 1>(a, s);
                case 2: return launch_nq<B, R, 2, 1>(a, s);
                case 3: return launch_nq<B, R, 3, 1>(a, s);
                case 4: return launch_nq<B, R, 4, 1>(a, s);
                case 5: return launch_nq<B, R, 5, 1>(a, s);
                case 6: return launch_nq<B, R, 6, 1>(a, s);
                case 7: return launch_nq<B, R, 7, 1>(a, s);
                case 8: return launch_nq<B, R, 8, 1>(a, s);
                default: break;
            }
            if (dim <= 4096) return n < 2048 ? launch_nq<B, R, 16, 1>(a, s) : launch_nq<B, R, 8, 2>(a, s);
            if (dim <= 8192) return launch_nq<B, R, 16, 2>(a, s);
            return launch_nq<B, R, 32, 2>(a, s);
        });
    });
}
