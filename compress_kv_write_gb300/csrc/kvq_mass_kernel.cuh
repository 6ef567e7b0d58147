// kvq_mass_kernel.cuh -- the weight that attention gives each cached token,
// summed over the query rows that see it.
//
// For a tile of N query rows and the cached rows k[t], block after block of
// 128 tokens:
//   S[t, r] = sum_d k[t, d] q[r, d]                    (tokens x rows)
//   mass[t] = sum_r 2^(scale log2(e) S[t, r] - log2(e) lse_r)
// There is one product and no state between blocks: the softmax's statistics
// come with the call, a token's sum is one thread's (a TMEM lane), and nothing
// is joined but the tiles of a sequence with more than 128 query rows.
//
// The products are tcgen05 with 128 tokens on the wide side and N = 16, 32, 64
// or 128 rows on the narrow one.  Codes and scales come by bulk copies, pages or
// what a block has of them, up to four blocks ahead; a decode warp takes 128
// dims of 32 tokens to registers, frees the block, and writes fp16 into TMEM as
// the product's A operand (nothing goes back to shared memory).  A query tile stays in shared
// memory as long as its blocks last.
//
// The numerics are the attention's: queries times a power of two in fp16 (exact
// down to 2^-28 of a row's largest value), cached rows exact in fp16 (V41:
// relative to a power of two of their own), fp32 sums, here kept short (kMParts,
// kMShift).  What fp32 constants of the exponent leave out is made up for by a
// factor a row.
//
// Rules for N by the rows of a sequence (kvq_mass.cuh), in us, one sequence of
// 100 tokens / 48 of 1,024 to 8,192 in even steps / 152 of 4,096:
//              as 16              32                 64                 128
//   16 heads V41  6.9/26.8/57.4   7.6/27.8/58.4      9.3/30.0/61.3      12.4/37.1/71.6
//            FP4  6.7/21.6/42.2   7.5/22.6/44.9      8.8/24.4/46.9      11.3/28.6/51.9
//   64 heads V41                                     9.5/31.2/62.7      12.9/39.9/75.0
//            FP4                                     9.1/25.2/48.5      11.6/30.0/53.5
//  128 heads V41                            twice:  11.4/53.7/123       13.6/41.3/76.5
//            FP4                                    10.7/43.0/94.3      12.0/31.5/56.0
//
// What bounds it: a block of 128 tokens takes 1.53 to 1.55 us (V41, up to 32
// rows), what its 67.6 KB take from memory; 1.08 to 1.22 us (FP4, up to 64 rows;
// memory alone would be 0.79), where issue slots are 57 to 71 % full and the
// decode warps' work is most of that (without the conversions 0.93); 1.62 us (V41,
// 64 rows), 1.91 (V41) and 1.40 us (FP4) with 128 rows, whose products alone take
// 2,048 clocks, 1.05 us: the queries leave shared memory for one (V41) or two
// blocks, and a block's weights take 2,700 clocks.  A call costs 6 to 15 us
// besides: launch, shares (3,400 clocks), queries, the first block's way through
// all roles (8,000) and the last one's.
#pragma once

#include "kvq_attend_rows.cuh"
#include "kvq_mass.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kMTile = 128;  // cached tokens a block
constexpr int kMChunks = kD / 128;
// Warps: 0-15 decode (four a quarter of the lanes, a chunk of 128 dims each), 16-23 weights (a lane quarter and half of the
// rows each; with all rows of every other block a score buffer was free later: 4 bits, 128 rows, 1.77 instead of 1.44 us a
// block), 24 issues the products, 25 looks up pages and issues the copies.  The decode warps load a tile's queries too: at its
// start they have nothing else to do (four warps for that alone took 13 us for 128 rows, and 8 registers of every thread).
constexpr int kMDeq = 16, kMSoft = 8;
constexpr int kMSoft0 = kMDeq, kMMma = kMSoft0 + kMSoft, kMLoad = kMMma + 1;
constexpr int kMThreads = (kMLoad + 1) * 32;
// What a tile costs beside its blocks (its queries), in blocks, when blocks are shared out.
constexpr int kMTileCost = 2;

// Blocks whose codes and scales shared memory holds.
template <Layout L>
constexpr int kMStageBytes = kMTile * kTokenBytes<L>;
template <Layout L, int N>
constexpr int kMStages = (L == Layout::V41 ? 1 : 2) * (N == 128 ? 1 : 2);
// The tensor cores take a score's 512 products 16 at a time and round the sum so far towards zero each time, so a score falls
// short by more the larger the sums on its way are: as one sum, 0.8 to 1.7 10^-7 of the scores that count.  Up to 32 rows TMEM
// has room for four sums a score, a chunk each (32 rows over 4-bit slots take 4 % longer so, others 1 to 2 %).  Beyond, half of a
// number near the row's largest scores is taken off after a quarter of the dims and half after three quarters, so that the sums
// of scores that count stay near zero (64 rows take 1 to 4 % longer than without, 128 rows up to 2 %).  Measured instead: two sums
// a score, 3 % (64 rows) and 28 % (128 rows, as twice 64) longer for half as much of the error; four steps, 3 to 9 %.
template <int N>
constexpr int kMParts = N <= 32 ? 4 : 1;
template <int N>
constexpr bool kMShift = N > 32;
// Chunks that TMEM holds for the products, beside two blocks' scores; four or more, so that a wait for the one that had
// a slot before is at most one phase off.
template <int N>
constexpr int kMRing = (512 - 2 * kMParts<N> * N) / 64;
// What is taken off is 2 16 a b: 16 columns of an A operand with a factor a of the token's, and of a B operand with b of the
// row's.  V41: a = 2^-texp, in the sum's own unit, where fp16 holds it (other tokens' scores are as they are).
constexpr float kMStep = 32.f;
template <Layout L>
constexpr float kMFactor = L == Layout::V41 ? 1.f : 16.f;
constexpr int kMTexpMin = -15, kMTexpMax = 14;
template <Layout L, int N>
constexpr int kMFactors = !kMShift<N> ? 0 : L == Layout::V41 ? 2 : 1;  // blocks in turn; the same for all
constexpr int kMFactorBytes = kMTile * 32;

template <Layout L, int N>
struct MassShared {
    static constexpr int S = kMStages<L, N>, KR = kMRing<N>;
    uint64_t full[S], empty[S];     // a block's codes are there; are read
    uint64_t ready[KR], scored[KR]; // a chunk is in TMEM; its products are done
    uint64_t sdone[2], sread[2];    // a block's scores are done; are read
    uint64_t tready[4];             // a block's powers of two are there
    uint64_t qready, qfree, cready[4];
    uint64_t drain;
    uint32_t scan[2][kMThreads / 32];
    int b0, b1;                     // this CTA's blocks, counted over all tiles
    int start_tile, start_kb;
    uint32_t tmem;
    int abort;
    uint32_t pieces[S];             // which of a block's copies there are
    int texp[4][kMTile];            // a token's power of two, or kNoToken
    float other[2][kMTile];         // a token's weights of the second half of the rows
    // of a tile's rows, four tiles in turn: factor, -log2(e) lse (less what is taken off a score), what their roundings leave
    // out, tokens seen; the fewest that one of a warp's rows sees
    // (for tokens whose scores are as they are behind those for the others)
    static constexpr int kSets = L == Layout::V41 && kMShift<N> ? 8 : 4;
    alignas(16) float sc[4][N], nl[kSets][N], wf[kSets][N];
    alignas(16) int vis[4][N];
    int words[4][N];                // where a row's mask begins, of a tree; -1: it sees no drafted token
    int least[4][kMDeq];
};

template <Layout L, int N>
constexpr size_t kMassSmem = 1024 + size_t(N) * kD * 2 + size_t(kMStages<L, N>) * kMStageBytes<L> + kMFactors<L, N> * kMFactorBytes +
                             (kMShift<N> ? N * 32 : 0) + sizeof(MassShared<L, N>);
static_assert(kMassSmem<Layout::V41, 16> <= 232448 && kMassSmem<Layout::V41, 32> <= 232448 &&
                  kMassSmem<Layout::V41, 64> <= 232448 && kMassSmem<Layout::V41, 128> <= 232448 &&
                  kMassSmem<Layout::FP4, 16> <= 232448 && kMassSmem<Layout::FP4, 32> <= 232448 &&
                  kMassSmem<Layout::FP4, 64> <= 232448 && kMassSmem<Layout::FP4, 128> <= 232448,
              "227 KB a CTA");

struct MassSeq {
    int len, err;
    int64_t trow, mrow;
};

__device__ __forceinline__ MassSeq mass_seq(const MassArgs &a, int seq) {
    MassSeq s;
    s.trow = a.req ? __ldg(a.req + seq) : seq;
    s.mrow = a.rows ? __ldg(a.rows + seq) : seq;
    s.len = __ldg(a.kv_len + seq);
    s.err = 0;
    if (s.trow < 0 || s.trow >= a.table_rows || s.mrow < 0 || s.mrow >= a.n_rows) s.err = KVQ_DEVERR_STATE;
    else if (s.len < 0 || s.len > a.max_len) s.err = KVQ_DEVERR_LEN;
    if (s.err) s.len = 0;
    return s;
}

// Walks a CTA's blocks in order; tiles of empty sequences have none.
struct MassCursor {
    int tile, kb, left, seq, rt, nb, nth;  // nth: which of this CTA's tiles
    MassSeq s;
    __device__ __forceinline__ MassCursor(const MassArgs &a, int start_tile, int start_kb, int units)
        : tile(start_tile), kb(start_kb), left(units), nth(0) {
        look(a);
    }
    __device__ __forceinline__ void look(const MassArgs &a) {
        seq = int(uint32_t(tile) / uint32_t(a.row_tiles));
        rt = int(uint32_t(tile) % uint32_t(a.row_tiles));
        s = mass_seq(a, seq);
        nb = (s.len + kMTile - 1) / kMTile;
    }
    __device__ __forceinline__ void next(const MassArgs &a) {
        if (--left <= 0) return;
        if (++kb < nb) return;
        next_tile(a);
    }
    __device__ __forceinline__ void next_tile(const MassArgs &a) {  // there is one
        kb = 0;
        ++nth;
        do {
            ++tile;
            look(a);
        } while (nb == 0);
    }
};

// Where a decoded row lies.  A decode thread has, of tokens r + 8 h (r = lane /
// 4, h = 0..3) of its warp's 32, the 32 dims (a quant block) from 32 q (q =
// lane % 4) of its warp's chunk, as vectors v = 0..3 of eight.  In TMEM vector v
// fills the columns 16 v + 4 i + q, i = 0..3, two dims a column: the contraction
// runs over the dims in that order, and this is the byte offset in a query
// tile's shared memory (two 128-byte-swizzled tiles of 32 columns a chunk) of
// word i of piece g = 0..63 (dims 8 g + 2 i, 8 g + 2 i + 1) of row r.
template <int N>
__device__ __forceinline__ uint32_t mass_q_word(int r, int g, int i) {
    const int b = g >> 4, q = (g >> 2) & 3, v = g & 3;
    return uint32_t((2 * b + (v >> 1)) * N * 128 + r * 128 + (((4 * (v & 1) + i) ^ (r & 7)) << 4) + q * 4);
}

// Decode warp w loads its rows of a tile's queries (w, w + 16, ..) and their constants.
template <Layout L, int N>
__device__ __forceinline__ void mass_queries(const MassArgs &a, MassShared<L, N> &sh, uint32_t sq, uint32_t sb, const MassCursor &cur,
                                             int w, int lane, uint32_t &tries) {
    constexpr int kRows = N / kMDeq, kBatch = kRows < 4 ? kRows : 4;  // a warp's rows; those whose loads are in flight
    static_assert(N % kMDeq == 0 && kMDeq % 8 == 0, "a warp's rows are equal modulo 8");
    const int per = a.q_len * a.heads, slot = cur.nth & 3;
    // lane l has the constants of the warp's l-th row
    const int row_l = cur.rt * N + w + lane * kMDeq;
    const bool real = lane < kRows && row_l < per;
    const float lse = real ? __ldg(a.lse + int64_t(cur.seq) * per + row_l) : -INFINITY;
    uint32_t up_l = 254;
    // byte offsets of a lane's words within a row (see mass_q_word); of its second piece, 32 further, 4 N 128 more
    uint32_t word[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) word[i] = sq + mass_q_word<N>(w & 7, lane, i) - (w & 7) * 128;
#pragma unroll 1
    for (int k0 = 0; k0 < kRows; k0 += kBatch) {
        uint32_t v[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = cur.rt * N + w + (k0 + b) * kMDeq, rc = min(row, per - 1);
            const int j = rc / a.heads, head = rc - j * a.heads;
            const uint16_t *from = a.q + (int64_t(cur.seq) * a.q_len + j) * a.q_tok + head * a.q_head;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (row < per) u = ld_stream_u4(from + (lane + 32 * h) * 8);
                v[b][4 * h] = u.x, v[b][4 * h + 1] = u.y, v[b][4 * h + 2] = u.z, v[b][4 * h + 3] = u.w;
            }
        }
        // the last tile's queries are free when its products are done
        if (k0 == 0 && cur.nth > 0) mbar_wait(smem_addr(&sh.qfree), (cur.nth - 1) & 1, tries);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int k = k0 + b;
            // fp16: the row times a power of two that brings its largest magnitude to [2^14, 2^15)
            uint32_t big = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) big = max(big, max((v[b][e] << 16) & 0x7FFF0000u, v[b][e] & 0x7FFF0000u));
            big = __reduce_max_sync(0xFFFFFFFFu, big);
            const uint32_t up = min(268u - (big >> 23), 254u);
            const float f = __uint_as_float(up << 23);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t h;
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(bf16_hi(v[b][e]) * f), "f"(bf16_lo(v[b][e]) * f));
                sts_u32(word[e & 3] + (w + k * kMDeq) * 128 + (e >> 2) * (4 * N * 128), h);
            }
            if (lane == k) up_l = up;
        }
    }
    // a row of no one's, and one that saw nothing (lse = -inf), has no weight
    const bool none = lse == -INFINITY;
    const int j_l = row_l / a.heads;
    const int vis = none ? 0 : max(0, cur.s.len - (a.mask ? a.q_len : a.q_len - 1 - j_l));
    if (lane < kRows) {
        const int r = w + lane * kMDeq;
        sh.words[slot][r] = none || !a.mask ? -1 : (cur.seq * a.q_len + j_l) * a.mask_words;
        // n = -log2(e) l in two parts, l = lse (less what is taken off the scores) and log2(e) in two as well
        auto constants = [&](int set, float l, float l_lo) {
            const float n = -l * kLog2e;
            const float rest = fmaf(-l, kLog2e, -n) - l * 1.9259629e-8f - l_lo * kLog2e;
            sh.nl[set][r] = none ? -INFINITY : n;
            // (up to |lse| = 2^28 within 2^64; beyond, where fp32 no longer tells weights apart, it stays finite and above zero,
            // so that no weight is NaN)
            sh.wf[set][r] = !(fabsf(n) < INFINITY) ? 1.f : ex2_approx(fminf(fmaxf(rest - n * a.c_off, -64.f), 64.f));
        };
        sh.sc[slot][r] = none ? 0.f : score_factor<L>(a.c, up_l);
        float l = lse, l_lo = 0.f;
        if constexpr (kMShift<N>) {
            if constexpr (sh.kSets == 8) constants(4 + slot, lse, 0.f);
            // Half way between lse, near which the scores of a peaked row count, and lse - ln(tokens), where all are of a flat
            // one; in fp16, so that sums of few bits stay sums of few bits.
            uint32_t b16 = 0;
            if (!none && up_l >= 40 && up_l <= 214) {
                const float unit = kMStep * kMFactor<L> * __uint_as_float((254 - up_l) << 23);  // of a score, a unit of b
                const float b = (lse - 0.5f * __logf(float(max(vis, 1)))) / a.scale / unit;
                uint32_t h;
                asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(h) : "f"(fminf(fmaxf(b, -61440.f), 61440.f)));
                float m;
                asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(m) : "r"(h));
                m *= unit;
                const float p = a.scale * m, p_lo = fmaf(a.scale, m, -p);
                if (fabsf(b) < INFINITY && fabsf(p) < 1e30f) {
                    l = lse - p;
                    const float t = l - lse;
                    l_lo = ((lse - (l - t)) - (p + t)) - p_lo;
                    b16 = h ^ 0x80008000u;
                }
            }
            const uint32_t four[4] = {b16, b16, b16, b16}, to = sb + r * 32;
            sts_u4(to, four);
            sts_u4(to + 16, four);
        }
        constants(slot, l, l_lo);
        sh.vis[slot][r] = vis;
    }
    const int least = __reduce_min_sync(0xFFFFFFFFu, real ? vis : 0x7FFFFFFF);
    if (lane == 0) sh.least[slot][w] = least;
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(smem_addr(&sh.qready));
        mbar_arrive(smem_addr(&sh.cready[slot]));
    }
}

template <Layout L, int N>
__global__ void __launch_bounds__(kMThreads, 1) mass_kernel(const __grid_constant__ MassArgs a) {
    using T = LayoutTraits<L>;
    constexpr int S = kMStages<L, N>, KR = kMRing<N>;
    constexpr int G = kMParts<N>;
    constexpr bool kShift = kMShift<N>, kTokens = kShift && L == Layout::V41;  // a factor for each token
    constexpr uint32_t kTmemK = 2 * G * N, kTmemCols = 512;  // scores, then chunks of rows
    static_assert(KR >= 4 && kTmemK + 64 * KR <= kTmemCols, "they fit");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + (-(uintptr_t(smem_addr(smem_raw))) & 1023);
    uint8_t *const sQ = base, *const sStage = sQ + N * kD * 2, *const sA = sStage + S * kMStageBytes<L>;
    uint8_t *const sB = sA + kMFactors<L, N> * kMFactorBytes;
    auto &sh = *reinterpret_cast<MassShared<L, N> *>(sB + (kMShift<N> ? N * 32 : 0));
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), kMDeq);
        }
        for (int i = 0; i < KR; ++i) {
            mbar_init(smem_addr(&sh.ready[i]), 4);
            mbar_init(smem_addr(&sh.scored[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.sdone[i]), 1);
            mbar_init(smem_addr(&sh.sread[i]), kMSoft);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&sh.tready[i]), 4);
            mbar_init(smem_addr(&sh.cready[i]), kMDeq);
        }
        mbar_init(smem_addr(&sh.qready), kMDeq);
        mbar_init(smem_addr(&sh.qfree), 1);
        mbar_init(smem_addr(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMMma) tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
    if constexpr (kShift && !kTokens) {
        static_assert(kMFactor<Layout::FP4> == 16.f, "0x4C00");
        for (int i = tid; i < kMFactorBytes / 4; i += kMThreads) reinterpret_cast<uint32_t *>(sA)[i] = 0x4C004C00u;
        fence_proxy_async();
    }
    pdl_wait();

    // ---- this CTA's share of all tiles' blocks in order, each tile with kMTileCost units before its blocks
    const int tiles = int(a.n_seq * a.row_tiles);
    {
        const int each = (tiles + kMThreads - 1) / kMThreads;
        const int t0 = min(tiles, tid * each), t1 = min(tiles, t0 + each);
        auto blocks_of = [&](int t, bool tell) {
            const MassSeq s = mass_seq(a, int(uint32_t(t) / uint32_t(a.row_tiles)));
            if (tell && s.err) raise_err(a.err, s.err);
            return uint32_t(s.len + kMTile - 1) / kMTile;
        };
        uint32_t units = 0, blocks = 0;
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
            const uint32_t nb = blocks_of(t, blockIdx.x == 0);
            blocks += nb;
            units += nb ? nb + kMTileCost : 0;
        }
        uint32_t iu = units, ib = blocks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, iu, o), w = __shfl_up_sync(0xFFFFFFFFu, ib, o);
            if (lane >= o) iu += v, ib += w;
        }
        if (lane == 31) sh.scan[0][warp] = iu, sh.scan[1][warp] = ib;
        if (tid == 0) sh.b0 = sh.b1 = 0;
        __syncthreads();
        // every warp sums the warps' totals: lane w has those of warp w
        const uint32_t wu = lane < kMThreads / 32 ? sh.scan[0][lane] : 0, wb = lane < kMThreads / 32 ? sh.scan[1][lane] : 0;
        const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, wu), all = __reduce_add_sync(0xFFFFFFFFu, wb);
        const uint32_t at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wu : 0) + iu - units;
        const uint32_t bat = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wb : 0) + ib - blocks;
        int64_t u0, u1;
        share(total, u0, u1);
        if (tid == 0 && u1 > u0 && u1 == total) sh.b1 = int(all);
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const uint32_t u = uint32_t(e ? u1 : u0);
            if (u1 == u0 || u < at || u - at >= units) continue;  // one thread goes on
            uint32_t vs = at, vb = bat;
            int t = t0;
#pragma unroll 1
            for (;; ++t) {
                const uint32_t nb = blocks_of(t, false), w = nb ? nb + kMTileCost : 0;
                if (u - vs < w) break;
                vs += w, vb += nb;
            }
            const uint32_t kb = u - vs > kMTileCost ? u - vs - kMTileCost : 0;
            if (e) {
                sh.b1 = int(vb + kb);
            } else {
                sh.b0 = int(vb + kb);
                sh.start_tile = t;
                sh.start_kb = int(kb);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int units = sh.b1 - sh.b0, start_tile = sh.start_tile, start_kb = sh.start_kb;
    if (units <= 0) {  // the same for every thread
        if (warp == kMMma) tmem_dealloc(sh.tmem, kTmemCols);
        pdl_trigger();
        return;
    }
    uint32_t tries = a.wait_tries;

    if (warp < kMDeq) {
        // ------------------------------------------------------ decode
        const int quarter = warp & 3, chunk = warp >> 2, q = lane & 3, r8 = lane >> 2;
        const uint32_t tlane = kTmemK + ((32 * quarter) << 16);
        const uint32_t code_at = (32 * quarter + r8) * T::kCodeBytes + chunk * (T::kCodeBytes / kMChunks) + q * (T::kCodeBytes / kNBlk);
        const uint32_t scale_at = kMTile * T::kCodeBytes + (32 * quarter + r8) * T::kScaleBytes;
        const int piece_bits = min(7, a.page_bits);
        int slot = 0, kslot = chunk;
        uint32_t parity = 0, kparity = 1;  // of the block; of the chunk that had this one's TMEM slot before
        MassCursor cur(a, start_tile, start_kb, units);
        int known = -1;  // the tile whose queries are loaded
#pragma unroll 1
        for (int i = 0; i < units; ++i, cur.next(a)) {
            if (known != cur.nth) {
                known = cur.nth;
                mass_queries<L, N>(a, sh, smem_addr(sQ), smem_addr(sB), cur, warp, lane, tries);
            }
            mbar_wait(smem_addr(&sh.full[slot]), parity, tries);
            const uint32_t stage = smem_addr(sStage) + slot * kMStageBytes<L>;
            const uint32_t pieces = sh.pieces[slot];
            Raw<L> raw[4][2];  // token, half of the 32 codes
            int texp[4];
            uint32_t mul[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t at = stage + code_at + 8 * h * T::kCodeBytes;
                if constexpr (L == Layout::V41) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 u = lds_u4(at + 16 * j);
                        raw[h][j].w[0] = u.x, raw[h][j].w[1] = u.y, raw[h][j].w[2] = u.z, raw[h][j].w[3] = u.w;
                    }
                } else {
                    const uint4 u = lds_u4(at);
                    raw[h][0].w[0] = u.x, raw[h][0].w[1] = u.y, raw[h][1].w[0] = u.z, raw[h][1].w[1] = u.w;
                }
                const uint4 sc = lds_u4(stage + scale_at + 8 * h * T::kScaleBytes);
                texp[h] = row_texp<L>(sc);
                const uint32_t w = chunk == 0 ? sc.x : chunk == 1 ? sc.y : chunk == 2 ? sc.z : sc.w;
                mul[h] = block_mul<L>((w >> (8 * q)) & 0xFFu, texp[h]);
            }
            __syncwarp();
            // (once the wait for it has given up its copy may be under way: then nothing is copied over it)
            if (lane == 0 && tries) mbar_arrive(smem_addr(&sh.empty[slot]));
            // a slot in TMEM is free when the products over what it held are done
            if (i * kMChunks + chunk >= KR) mbar_wait(smem_addr(&sh.scored[kslot]), kparity, tries);
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 4; h += 2)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t v0[4], v1[4];
                    decode8<L>(raw[h][v >> 1], v & 1, mul[h], v0);
                    decode8<L>(raw[h + 1][v >> 1], v & 1, mul[h + 1], v1);
                    tmem_st_16x128b_x4(tlane + (uint32_t(8 * h) << 16) + kslot * 64 + 16 * v, v0, v1);
                }
            if (chunk == 0 && q == 0) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int t = 32 * quarter + 8 * h + r8;
                    const bool there = cur.kb * kMTile + t < cur.s.len && ((pieces >> (t >> piece_bits)) & 1);
                    sh.texp[i & 3][t] = there ? texp[h] : kNoToken;
                }
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&sh.ready[kslot]));
                if (chunk == 0) mbar_arrive(smem_addr(&sh.tready[i & 3]));
            }
            if (++slot == S) {
                slot = 0;
                parity ^= 1;
            }
            kslot += kMChunks;
            if (kslot >= KR) {
                kslot -= KR;
                kparity ^= 1;
            }
        }
    } else if (warp < kMMma) {
        // ------------------------------------------------------ weights
        // A warp has 32 tokens, a lane each, and half of the rows; the warp with the first half adds the other's sums.
        constexpr int NC = N / 2, NL = NC < 16 ? NC : 16;  // a warp's columns; those of a load
        const int quarter = warp & 3, half = (warp - kMSoft0) >> 2, tok = 32 * quarter + lane, c0 = half * NC;
        const uint32_t tfrom = (uint32_t(32 * quarter) << 16) + c0;
        MassCursor cur(a, start_tile, start_kb, units);
        int known = -1, least = 0;  // the tile whose rows are known to be there; the fewest tokens that one of them sees
#pragma unroll 1
        for (int i = 0; i < units; ++i, cur.next(a)) {
            const int c = cur.nth & 3;
            if (known != cur.nth) {
                known = cur.nth;
                mbar_wait(smem_addr(&sh.cready[c]), (cur.nth >> 2) & 1, tries);
                least = __reduce_min_sync(0xFFFFFFFFu, sh.least[c][lane & (kMDeq - 1)]);
            }
            const int t = cur.kb * kMTile + tok;
            const bool mine = half == 0 && t < cur.s.len;
            float before = 0.f;
            if (a.row_tiles == 1 && a.prev && mine) before = a.prev[cur.s.mrow * a.prev_stride + t];
            mbar_wait(smem_addr(&sh.tready[i & 3]), (i >> 2) & 1, tries);
            const int te = sh.texp[i & 3][tok];
            const bool there = te != kNoToken;
            const int set = !kTokens || (te >= kMTexpMin && te <= kMTexpMax) ? c : 4 + c;
            const float up = L == Layout::V41 && there ? __uint_as_float(uint32_t(127 + te - kLift) << 23) : 1.f;
            const bool masked = (cur.kb + 1) * kMTile > least;
            // whether row r, of the tile, sees this thread's token: it is one of the first `vis`, or drafted and in its mask
            const int drafted = t - (cur.s.len - a.q_len);
            auto sees = [&](int r, int vis) {
                if (t < vis) return true;
                if (!a.mask || drafted < 0 || drafted >= a.q_len) return false;
                const int at = sh.words[c][r];
                return at >= 0 && ((__ldg(a.mask + at + (drafted >> 6)) >> (drafted & 63)) & 1) != 0;
            };
            mbar_wait(smem_addr(&sh.sdone[i & 1]), (i >> 1) & 1, tries);
            tc_fence_after();
            // 2^(exponent) of four rows from r on, and their factors
            auto weigh = [&](float x0, float x1, float x2, float x3, int r, float2 (&p)[2], float4 &wf) {
                const float4 sc = *reinterpret_cast<const float4 *>(&sh.sc[c][r]);
                const float4 nl = *reinterpret_cast<const float4 *>(&sh.nl[set][r]);
                wf = *reinterpret_cast<const float4 *>(&sh.wf[set][r]);
                float2 u0 = make_float2(x0, x1), u1 = make_float2(x2, x3);
                if constexpr (L == Layout::V41) {
                    u0 = fmul2(u0, make_float2(up, up));
                    u1 = fmul2(u1, make_float2(up, up));
                }
                u0 = ffma2(u0, make_float2(sc.x, sc.y), make_float2(nl.x, nl.y));
                u1 = ffma2(u1, make_float2(sc.z, sc.w), make_float2(nl.z, nl.w));
                p[0] = make_float2(ex2_approx(u0.x), ex2_approx(u0.y));
                p[1] = make_float2(ex2_approx(u1.x), ex2_approx(u1.y));
            };
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const uint32_t at = tfrom + (i & 1) * (G * N);
            if (!masked) {
#pragma unroll 1
                for (int j0 = 0; j0 < NC; j0 += NL) {
                    float x[NL];
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        uint32_t y[NL];
                        if constexpr (NL == 16) tmem_ld16(at + g * N + j0, y);
                        else tmem_ld8(at + g * N + j0, y);
#pragma unroll
                        for (int j = 0; j < NL; j += 2) {
                            float2 v = make_float2(__uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                            if (g) v = fadd2(make_float2(x[j], x[j + 1]), v);
                            x[j] = v.x, x[j + 1] = v.y;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NL; j += 4) {
                        float2 p[2];
                        float4 wf;
                        weigh(x[j], x[j + 1], x[j + 2], x[j + 3], c0 + j0 + j, p, wf);
                        sum[0] = ffma2(p[0], make_float2(wf.x, wf.y), sum[0]);
                        sum[1] = ffma2(p[1], make_float2(wf.z, wf.w), sum[1]);
                    }
                }
            } else {
                // A tile's last block or two, in a loop of their own: the roles share the instruction cache (128 rows over
                // 4-bit slots 1.39 us a block, with masks in the other loop 1.61).
#pragma unroll 1
                for (int j0 = 0; j0 < NC; j0 += 4) {
                    float x[4];
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        uint32_t y[4];
                        tmem_ld4(at + g * N + j0, y);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = g ? x[j] + __uint_as_float(y[j]) : __uint_as_float(y[j]);
                    }
                    const int r = c0 + j0;
                    const int4 vis = *reinterpret_cast<const int4 *>(&sh.vis[c][r]);
                    float2 p[2];
                    float4 wf;
                    weigh(x[0], x[1], x[2], x[3], r, p, wf);
                    p[0] = make_float2(sees(r, vis.x) ? p[0].x : 0.f, sees(r + 1, vis.y) ? p[0].y : 0.f);
                    p[1] = make_float2(sees(r + 2, vis.z) ? p[1].x : 0.f, sees(r + 3, vis.w) ? p[1].y : 0.f);
                    sum[0] = ffma2(p[0], make_float2(wf.x, wf.y), sum[0]);
                    sum[1] = ffma2(p[1], make_float2(wf.z, wf.w), sum[1]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.sread[i & 1]));
            const float2 two = fadd2(sum[0], sum[1]);
            float all = two.x + two.y;
            if (half == 1) sh.other[i & 1][tok] = all;
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");  // the quarter's two warps
            if (mine && tries) {
                all = there ? all + sh.other[i & 1][tok] : 0.f;
                if (a.row_tiles == 1) a.mass[cur.s.mrow * a.mass_stride + t] = a.prev ? fmaf(a.decay, before, all) : all;
                else a.part[int64_t(cur.tile) * a.part_stride + t] = all;
            }
        }
    } else if (warp == kMMma) {
        // ------------------------------------------------------ products
        constexpr uint32_t kIdesc = mma_idesc(kMTile, N, false, false), kHi = desc_hi(1024, kSwizzle128);
        const uint32_t qd = desc_lo(smem_addr(sQ), 16);
        constexpr uint32_t kHi32 = desc_hi(256, kSwizzle32);  // of rows of 16 equal columns
        const uint32_t ad = desc_lo(smem_addr(sA), 16), bd = desc_lo(smem_addr(sB), 16);
        static_assert(!kShift || G == 1, "one sum");
        MassCursor cur(a, start_tile, start_kb, units);
        int kslot = 0;
        uint32_t kparity = 0;
        bool fresh = true;
#pragma unroll 1
        for (int i = 0; i < units; ++i) {
            if (fresh) mbar_wait(smem_addr(&sh.qready), cur.nth & 1, tries);
            fresh = cur.kb + 1 == cur.nb;
            // the score buffer is free when the block before the last has been read
            if (i >= 2) mbar_wait(smem_addr(&sh.sread[i & 1]), ((i - 2) >> 1) & 1, tries);
            const uint32_t to = (i & 1) * (G * N), factors = ad + (kTokens ? (i & 1) * (kMFactorBytes >> 4) : 0);
#pragma unroll
            for (int b = 0; b < kMChunks; ++b) {
                mbar_wait(smem_addr(&sh.ready[kslot]), kparity, tries);
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t at = qd + ((2 * b * N * 128) >> 4), from = kTmemK + kslot * 64;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if constexpr (kShift) {
                            if (b == 1 && k == 0) mma_ss(to, factors, kHi32, bd, kHi32, kIdesc, true);
                        }
                        mma_ts(to + b * G / kMChunks * N, from + 8 * k, at + (((k >> 2) * N * 128 + (k & 3) * 32) >> 4), kHi, kIdesc,
                               b % (kMChunks / G) + k > 0);
                        if constexpr (kShift) {
                            if (b == 2 && k == 7) mma_ss(to, factors, kHi32, bd, kHi32, kIdesc, true);
                        }
                    }
                    mma_commit(smem_addr(&sh.scored[kslot]));
                    if (b == kMChunks - 1) {
                        mma_commit(smem_addr(&sh.sdone[i & 1]));
                        if (fresh) mma_commit(smem_addr(&sh.qfree));
                    }
                }
                __syncwarp();
                if constexpr (kTokens) {
                    // The tokens' factors, while the first chunk's products run.  (That this chunk is there tells that the first
                    // three chunks of two blocks ago are done, which took the factors that were in this place.)
                    if (b == 0) {
                        mbar_wait(smem_addr(&sh.tready[i & 3]), (i >> 2) & 1, tries);
#pragma unroll
                        for (int t = lane; t < kMTile; t += 32) {
                            const int te = sh.texp[i & 3][t];
                            const uint32_t f = te >= kMTexpMin && te <= kMTexpMax ? uint32_t(15 - te) * 0x04000400u : 0u;  // 2^-te
                            const uint32_t four[4] = {f, f, f, f}, at = smem_addr(sA) + (i & 1) * kMFactorBytes + t * 32;
                            sts_u4(at, four);
                            sts_u4(at + 16, four);
                        }
                        fence_proxy_async();
                        __syncwarp();
                    }
                }
                if (++kslot == KR) {
                    kslot = 0;
                    kparity ^= 1;
                }
            }
            cur.next(a);
        }
        if (!tries) sh.abort = 1;
        tries = kWaitTries;
        if (elect_one()) mma_commit(smem_addr(&sh.drain));  // nothing may write TMEM once it is freed
        __syncwarp();
        mbar_wait(smem_addr(&sh.drain), 0, tries);
    } else {
        // ------------------------------------------------------ pages and copies
        // Lane l has the piece of piece_rows tokens from token l * piece_rows of the block on: a page, or what the block has of
        // it.  (32 tokens a copy and a barrier: 780 clocks each, all of them this warp's latencies.)
        const int64_t page_bytes = int64_t(kTokenBytes<L>) << a.page_bits, area = int64_t(T::kCodeBytes) << a.page_bits;
        const int in_page = (1 << a.page_bits) - 1;
        const int piece_bits = min(7, a.page_bits), piece_rows = 1 << piece_bits;
        const int at = lane << piece_bits;  // of the block
        MassCursor cur(a, start_tile, start_kb, units);
        int64_t entry = -1;
        auto fetch = [&]() {
            const int t = cur.kb * kMTile + at;
            entry = -1;
            if (at < kMTile && t < cur.s.len) entry = __ldg(a.table + cur.s.trow * a.table_stride + (t >> a.page_bits));
        };
        // Where the queries leave room for one block, the next one is sent for to L2.
        constexpr bool kAhead = S == 1;
        fetch();
        int slot = 0, issued = 0;
        uint32_t parity = 1;
#pragma unroll 1
        for (int i = 0; i < units; ++i) {
            const int64_t page = entry;
            const int t = cur.kb * kMTile + at;
            const bool has = at < kMTile && t < cur.s.len, good = has && page >= 0 && page < a.pool_limit;
            if (i + 1 < units) {  // the next block's pages, while this one's place becomes free
                cur.next(a);
                fetch();
            }
            if (has && !good) raise_err(a.err, KVQ_DEVERR_PAGE);
            const uint32_t pieces = __ballot_sync(0xFFFFFFFFu, good), bar = smem_addr(&sh.full[slot]);
            if (i >= S) mbar_wait(smem_addr(&sh.empty[slot]), parity, tries);
            if (__any_sync(0xFFFFFFFFu, tries == 0)) {  // the warp's decision
                tries = 0;
                break;
            }
            if (lane == 0) {
                sh.pieces[slot] = pieces;
                mbar_arrive_expect(bar, __popc(pieces) * piece_rows * kTokenBytes<L>);
            }
            __syncwarp();
            if (good) {
                const uint32_t to = smem_addr(sStage) + slot * kMStageBytes<L>;
                const uint8_t *from = a.pool + page * page_bytes;
                const int row = t & in_page;
                bulk_load(to + at * T::kCodeBytes, from + int64_t(row) * T::kCodeBytes, piece_rows * T::kCodeBytes, bar);
                bulk_load(to + kMTile * T::kCodeBytes + at * T::kScaleBytes, from + area + int64_t(row) * T::kScaleBytes,
                          piece_rows * T::kScaleBytes, bar);
            }
            if constexpr (kAhead) {
                const int ta = cur.kb * kMTile + at;
                if (i + 1 < units && at < kMTile && ta < cur.s.len && entry >= 0 && entry < a.pool_limit) {
                    const uint8_t *from = a.pool + entry * page_bytes;
                    prefetch_l2_bulk(from + int64_t(ta & in_page) * T::kCodeBytes, piece_rows * T::kCodeBytes);
                    prefetch_l2_bulk(from + area + int64_t(ta & in_page) * T::kScaleBytes, piece_rows * T::kScaleBytes);
                }
            }
            ++issued;
            if (++slot == S) {
                slot = 0;
                parity ^= 1;
            }
        }
        if (!tries) sh.abort = 1;
        // no copy may be under way when the CTA ends: each slot's last one
        tries = kWaitTries;
        for (int k = 0; k < S && k < issued; ++k) {
            const int last = (issued - 1 - k) / S;  // how often the slot was used before
            mbar_wait(smem_addr(&sh.full[k]), last & 1, tries);
        }
        tries = 1;
    }
    if (!tries) sh.abort = 1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) pdl_trigger();
    if (warp == kMMma) tmem_dealloc(sh.tmem, kTmemCols);
    if (sh.abort) {  // a wait gave up: the weights that this CTA worked on are NaN, at once or by way of the join
        if (tid == 0) raise_err(a.err, KVQ_DEVERR_WAIT);
        MassCursor cur(a, start_tile, start_kb, units);
#pragma unroll 1
        for (int i = 0; i < units; ++i, cur.next(a)) {
            const int t = cur.kb * kMTile + tid;
            if (tid >= kMTile || t >= cur.s.len) continue;
            if (a.row_tiles == 1) a.mass[cur.s.mrow * a.mass_stride + t] = NAN;
            else a.part[int64_t(cur.tile) * a.part_stride + t] = NAN;
        }
    }
}

// Adds the tiles of sequences that have several, in order, and what was before.
constexpr int kMJoinThreads = 256;

__global__ void __launch_bounds__(kMJoinThreads) mass_join_kernel(const __grid_constant__ MassArgs a) {
    pdl_wait();
    const int seq = blockIdx.y;
    const MassSeq s = mass_seq(a, seq);
    const float *part = a.part + int64_t(seq) * a.row_tiles * a.part_stride;
    for (int64_t t = int64_t(blockIdx.x) * kMJoinThreads + threadIdx.x; t < s.len; t += int64_t(gridDim.x) * kMJoinThreads) {
        float sum = 0.f;
#pragma unroll 8
        for (int k = 0; k < a.row_tiles; ++k) sum += part[k * a.part_stride + t];
        if (a.prev) sum = fmaf(a.decay, a.prev[s.mrow * a.prev_stride + t], sum);
        a.mass[s.mrow * a.mass_stride + t] = sum;
    }
}

template <Layout L, int N>
kvq_status launch_mass_n(MassArgs a, cudaStream_t s) {
    const int64_t per = int64_t(a.q_len) * a.heads;
    a.row_tiles = int(mass_tiles(per));
    const int64_t tiles = a.n_seq * a.row_tiles;
    int64_t grid = 0;
    kvq_status st = resident_grid<mass_kernel<L, N>, kMThreads>(kMassSmem<L, N>, &grid);
    if (st != KVQ_OK) return st;
    if (grid > kMaxAttendCtas) grid = kMaxAttendCtas;
    const int64_t most = (a.max_len + kMTile - 1) / kMTile;  // blocks of the longest tile there can be
    if (tiles > 0x7FFFFFFF / (most + kMTileCost)) return KVQ_ERR_UNSUPPORTED;  // units fit an int
    if (most <= 1 && tiles < grid) grid = tiles;
    st = launch_pdl_smem(mass_kernel<L, N>, dim3(unsigned(grid)), dim3(kMThreads), kMassSmem<L, N>, s, a);
    if (st != KVQ_OK || a.row_tiles == 1) return st;
    const int64_t wide = (a.max_len + kMJoinThreads - 1) / kMJoinThreads;
    return launch_pdl(mass_join_kernel, dim3(unsigned(wide < 1 ? 1 : wide < 1024 ? wide : 1024), unsigned(a.n_seq)), dim3(kMJoinThreads), s, a);
}

template <Layout L>
kvq_status launch_mass_layout(const MassArgs &a, cudaStream_t s) {
    switch (mass_rows(int64_t(a.q_len) * a.heads)) {
        case 16: return launch_mass_n<L, 16>(a, s);
        case 32: return launch_mass_n<L, 32>(a, s);
        case 64: return launch_mass_n<L, 64>(a, s);
        default: return launch_mass_n<L, 128>(a, s);
    }
}

}  // namespace
}  // namespace kvq
