// kvq_attend_kernel.cuh -- the tensor-core attention kernel and its join.
#pragma once

#include <math.h>

#include "kvq_attend.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTile = 128;          // cached tokens a block
constexpr int kSoftWarps = 4;       // one thread a token of the block
constexpr int kDeqWarps = 8;
constexpr int kAttendThreads = (kSoftWarps + kDeqWarps + 1) * 32;
constexpr int kChunk = 128;         // dims a step of decoding
constexpr int kChunks = kD / kChunk;
constexpr int kSubBytes = kTile * 128;  // 64 dims of a block, 128 B a token
constexpr float kStaleMax = 8.f;    // how far (log2) a score may pass the running maximum before it moves

template <int N>
struct AttendShared {
    uint64_t full[kChunks], oblk[kChunks], kfree[2], sdone, pready, qready, drain;
    int64_t scan[kAttendThreads / 32];
    int64_t u0, u1, total;
    int start_tile, start_kb;
    uint32_t tmem;
    int abort, soft_abort;
    alignas(16) float sc[N], nm[N], m[N], alpha[N], inv[N];
    float red[kSoftWarps][N];
    alignas(16) int vis[N];
    int64_t row[N];
    uint8_t valid[2][kTile];
};

template <int N>
constexpr size_t kAttendSmem = 1024 + size_t(kTile) * kD * 2 + size_t(N) * kD * 2 + size_t(kTile) * N * 2 +
                               sizeof(AttendShared<N>);

// Tiles are N query rows of a sequence (row = query token * heads + head);
// a tile's blocks are the 128-token pieces of what its last query token sees.
struct TileInfo {
    int64_t seq;
    int rt, len, seen, nb;  // cached tokens, tokens the last row sees, blocks (at least one)
    int64_t trow;
    int err;
};

template <int N, bool kSlots>
__device__ __forceinline__ TileInfo tile_info(const AttendArgs &a, int64_t tile) {
    TileInfo t;
    t.seq = uint32_t(tile) / uint32_t(a.row_tiles);
    t.rt = int(uint32_t(tile) % uint32_t(a.row_tiles));
    t.err = 0;
    t.trow = t.seq;
    if constexpr (kSlots) {
        t.len = t.seen = int(a.max_len);
    } else {
        if (a.req) t.trow = __ldg(a.req + t.seq);
        t.len = __ldg(a.kv_len + t.seq);
        if (t.trow < 0 || t.trow >= a.table_rows) {
            t.err = KVQ_DEVERR_STATE;
            t.len = 0;
        } else if (t.len < 0 || t.len > a.max_len) {
            t.err = KVQ_DEVERR_LEN;
            t.len = 0;
        }
        t.seen = t.len;
        if (a.q_len > 1) {
            const int64_t per = int64_t(a.q_len) * a.heads;
            const int64_t last = min(int64_t(t.rt + 1) * N, per) - 1;
            t.seen = max(0, t.len - (a.q_len - 1 - int(last / a.heads)));
        }
    }
    t.nb = max(1, (t.seen + kTile - 1) / kTile);
    return t;
}

// Walks a CTA's blocks in order.
template <int N, bool kSlots>
struct Cursor {
    int64_t tile;
    int kb;
    int64_t left;
    TileInfo t;
    __device__ __forceinline__ Cursor(const AttendArgs &a, const AttendShared<N> &sh)
        : tile(sh.start_tile), kb(sh.start_kb), left(sh.u1 - sh.u0), t(tile_info<N, kSlots>(a, tile)) {}
    __device__ __forceinline__ void next(const AttendArgs &a) {
        --left;
        if (++kb >= t.nb) {
            kb = 0;
            ++tile;
            if (left > 0) t = tile_info<N, kSlots>(a, tile);
        }
    }
};

// Where chunk and word of the decoded rows lie.  A dequant thread holds
// tokens r and r + 8 (r = lane / 4) and, of each chunk of 128 dims, 32 dims
// of each: V41 the 16-dim pieces q and q + 4 (q = lane % 4), FP4 the 32 dims
// from 32q.  It makes four 8-dim vectors ci = 0..3 of them; vector ci of FP4
// is piece ci ^ (q & 2), which lets the eight lanes of a shared-memory phase
// (two tokens, four q) store to eight different banks groups.
//
// In TMEM (the A operand of the scores' product) vector ci of thread q fills
// columns 16 ci + 4 e + q, e = 0..3, two dims a column, so the contraction
// runs over the dims in another order; q_word() puts a query's dims in the
// same order.

template <Layout L>
struct Raw;  // one token's 32 codes of a chunk
template <>
struct Raw<Layout::V41> {
    uint4 p[2];
};
template <>
struct Raw<Layout::FP4> {
    uint4 p[1];
};

template <Layout L>
__device__ __forceinline__ void load_raw(Raw<L> &r, const uint8_t *row, int chunk, int q) {
    constexpr int kChunkBytes = LayoutTraits<L>::kCodeBytes / kChunks;
#pragma unroll
    for (int h = 0; h < int(sizeof(Raw<L>) / 16); ++h)
        r.p[h] = row ? __ldg(reinterpret_cast<const uint4 *>(row + chunk * kChunkBytes + h * 64) + q)
                     : make_uint4(0u, 0u, 0u, 0u);
}

// Vector ci of a token's 32 dims: 8 values as four packed 16-bit pairs.
template <Layout L>
__device__ __forceinline__ void decode8(const Raw<L> &r, int ci, int q, uint32_t scales, uint32_t (&o)[4]) {
    if constexpr (L == Layout::V41) {
        const uint4 &p = r.p[ci >> 1];
        const uint32_t w[2] = {(ci & 1) ? p.z : p.x, (ci & 1) ? p.w : p.y};
        const float s = ue8m0_to_f32((scales >> (8 * (2 * (ci >> 1) + (q >> 1)))) & 0xFFu);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = fmul2(e4m3x2_to_f32x2((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), make_float2(s, s));
            o[i] = pack_bf16x2(f.x, f.y);
        }
    } else {
        const uint4 &p = r.p[0];
        const bool swap = q & 2;
        const uint32_t w = ci == 0 ? (swap ? p.z : p.x) : ci == 1 ? (swap ? p.w : p.y) : ci == 2 ? (swap ? p.x : p.z)
                                                                                              : (swap ? p.y : p.w);
        const uint32_t sb = (scales >> (8 * q)) & 0xFFu;
        uint32_t s2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(uint16_t(sb * 0x101u)));
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 t;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b0;\n\tmul.rn.f16x2 %0, t, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b1;\n\tmul.rn.f16x2 %1, t, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b2;\n\tmul.rn.f16x2 %2, t, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 t, b3;\n\tmul.rn.f16x2 %3, t, %5;\n\t}"
            : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
            : "r"(w), "r"(s2));
    }
}

// Byte offset, in a query tile's shared memory, of word e (dims 8g + 2e,
// 8g + 2e + 1) of piece g = 0..63 of row r.
template <Layout L, int N>
__device__ __forceinline__ uint32_t q_word(int r, int g, int e) {
    const int b = g >> 4, gi = g & 15;
    int ci, q;
    if constexpr (L == Layout::V41) {
        ci = 2 * (gi >> 3) + (gi & 1);
        q = (gi >> 1) & 3;
    } else {
        q = gi >> 2;
        ci = (gi & 3) ^ (q & 2);
    }
    return uint32_t((2 * b + (ci >> 1)) * N * 128 + r * 128 + (((4 * (ci & 1) + e) ^ (r & 7)) << 4) + q * 4);
}

// Swizzled byte offset of 16-byte vector j of row t of the weights' tile
// (rows of N 16-bit values).
template <int N>
__device__ __forceinline__ uint32_t p_vec(int t, int j) {
    constexpr int kVecs = N / 8;
    const int x = N == 64 ? (t & 7) : N == 32 ? ((t >> 1) & 3) : ((t >> 2) & 1);
    return uint32_t(t * N * 2 + ((j ^ (x & (kVecs - 1))) << 4));
}

// Lane-transposing reductions: from N values a thread to the warp's total of
// column col, i = 0 .. max(1, N / 32) - 1, in v[i].
template <int N>
__device__ __forceinline__ int warp_columns_sum(float (&v)[N], int lane) {
    int col = 0;
    int half = N / 2;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (half >= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < half) {
                    const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
                    v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
                }
            if (up) col += half;
            half >>= 1;
        } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
        }
    }
    return col;
}

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Barrier of the four softmax warps; the second form returns whether any of
// their threads brought true.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
        "bar.red.or.pred b, 1, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(p))
        : "memory");
    return r != 0;
}

template <Layout L, int N, bool kSlots>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
    using T = LayoutTraits<L>;
    constexpr bool kBf16 = L == Layout::V41;
    constexpr uint32_t kTmemS = 4 * N, kTmemK = 5 * N;
    constexpr uint32_t kTmemCols = 5 * N + 128 <= 256 ? 256 : 512;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + (-(uintptr_t(smem_addr(smem_raw))) & 1023);
    uint8_t *const sK = base, *const sQ = sK + kTile * kD * 2, *const sP = sQ + N * kD * 2;
    auto &sh = *reinterpret_cast<AttendShared<N> *>(sP + kTile * N * 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_wait();

    // ---- this CTA's share: block units [u0, u1) of the tiles in order
    const int64_t tiles = a.n_seq * a.row_tiles;
    if constexpr (kSlots) {
        if (tid == 0) {
            const int64_t nb = max(int64_t(1), (a.max_len + kTile - 1) / kTile);
            sh.total = tiles * nb;
            const int64_t g = min(int64_t(gridDim.x), sh.total);
            sh.u0 = blockIdx.x < g ? int64_t(blockIdx.x) * sh.total / g : 0;
            sh.u1 = blockIdx.x < g ? int64_t(blockIdx.x + 1) * sh.total / g : 0;
            sh.start_tile = int(sh.u0 / nb);
            sh.start_kb = int(sh.u0 % nb);
        }
    } else {
        const int64_t per = (tiles + kAttendThreads - 1) / kAttendThreads;
        const int64_t t0 = min(tiles, tid * per), t1 = min(tiles, t0 + per);
        int64_t mine = 0;
        for (int64_t t = t0; t < t1; ++t) mine += tile_info<N, kSlots>(a, t).nb;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, (long long)incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        int64_t before = 0, total = 0;
        for (int i = 0; i < kAttendThreads / 32; ++i) {
            if (i < warp) before += sh.scan[i];
            total += sh.scan[i];
        }
        const int64_t g = min(int64_t(gridDim.x), total);
        const int64_t u0 = blockIdx.x < g ? int64_t(blockIdx.x) * total / g : 0;
        const int64_t u1 = blockIdx.x < g ? int64_t(blockIdx.x + 1) * total / g : 0;
        if (tid == 0) {
            sh.u0 = u0;
            sh.u1 = u1;
            sh.total = total;
        }
        int64_t at = before + incl - mine;
        if (u0 >= at && u0 < at + mine)
            for (int64_t t = t0; t < t1; ++t) {
                const int nb = tile_info<N, kSlots>(a, t).nb;
                if (u0 < at + nb) {
                    sh.start_tile = int(t);
                    sh.start_kb = int(u0 - at);
                    break;
                }
                at += nb;
            }
    }
    if (tid == 0) {
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(smem_addr(&sh.full[i]), kDeqWarps);
            mbar_init(smem_addr(&sh.oblk[i]), 1);
        }
        mbar_init(smem_addr(&sh.kfree[0]), 1);
        mbar_init(smem_addr(&sh.kfree[1]), 1);
        mbar_init(smem_addr(&sh.sdone), 1);
        mbar_init(smem_addr(&sh.pready), kSoftWarps);
        mbar_init(smem_addr(&sh.qready), kSoftWarps);
        mbar_init(smem_addr(&sh.drain), 1);
        sh.abort = sh.soft_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const int64_t units = sh.u1 - sh.u0;
    if (units == 0) {  // the same for every thread
        if (tid == 0) a.join[blockIdx.x] = make_int2(-1, 0);
        pdl_trigger();
        return;
    }
    if (warp == kSoftWarps + kDeqWarps) tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp >= kSoftWarps && warp < kSoftWarps + kDeqWarps) {
        // ------------------------------------------------------ decode
        const int w = warp - kSoftWarps, q = lane & 3, r8 = lane >> 2;
        const int tok0 = 32 * (w & 3) + 16 * (w >> 2) + r8;  // and tok0 + 8
        const uint32_t krow = smem_addr(sK) + tok0 * 128;
        const uint32_t kxor = (L == Layout::V41 ? 2 * q : ((q & 1) * 4) ^ (q & 2)) ^ r8;
        const uint32_t tlane = tmem + kTmemK + ((32 * (w & 3) + 16 * (w >> 2)) << 16);
        const int64_t page_bytes = int64_t(kTokenBytes<L>) << a.page_bits;
        const int in_page = (1 << a.page_bits) - 1;

        Cursor<N, kSlots> cur(a, sh);
        int64_t idx[2];   // page or slot, -1: no token
        int in[2];        // row in the page (paged)
        auto fetch = [&]() {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t t = int64_t(cur.kb) * kTile + tok0 + 8 * h;
                idx[h] = -1;
                in[h] = int(t) & in_page;
                if (cur.left > 0 && t < cur.t.seen) {
                    if constexpr (kSlots) {
                        const int64_t at = cur.t.seq * a.slots_stride + t;
                        idx[h] = a.slots64 ? __ldg(static_cast<const int64_t *>(a.slots) + at)
                                           : int64_t(__ldg(static_cast<const int32_t *>(a.slots) + at));
                    } else {
                        idx[h] = __ldg(a.table + cur.t.trow * a.table_stride + (t >> a.page_bits));
                        if (idx[h] < 0) idx[h] = -2;
                    }
                }
            }
        };
        const uint8_t *code[2];
        uint4 sc[2];
        auto resolve = [&]() {  // row pointers and scales of the fetched block
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                code[h] = nullptr;
                sc[h] = make_uint4(0u, 0u, 0u, 0u);
                if (idx[h] >= 0 && idx[h] < a.pool_limit) {
                    const int64_t page = kSlots ? idx[h] >> a.page_bits : idx[h];
                    const int row = kSlots ? int(idx[h]) & in_page : in[h];
                    const uint8_t *p = a.pool + page * page_bytes;
                    code[h] = p + row * T::kCodeBytes;
                    sc[h] = __ldg(reinterpret_cast<const uint4 *>(p + (int64_t(T::kCodeBytes) << a.page_bits) +
                                                                  row * T::kScaleBytes));
                } else if (idx[h] != -1 && q == 0) {
                    raise_err(a.err, kSlots ? KVQ_DEVERR_SLOT : KVQ_DEVERR_PAGE);
                }
            }
        };

        Raw<L> raw[kChunks][2];
        fetch();
        resolve();
#pragma unroll
        for (int b = 0; b < kChunks; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) load_raw<L>(raw[b][h], code[h], b, q);
        bool ok[2] = {code[0] != nullptr, code[1] != nullptr};
        uint4 now[2] = {sc[0], sc[1]};
        cur.next(a);
        fetch();
        for (int64_t i = 0; i < units; ++i) {
            resolve();   // the next block; its indexes came a block ago
            if (cur.left > 0) cur.next(a);
            fetch();
            const uint32_t phase = uint32_t(i) & 1;
            bool live = true;
#pragma unroll
            for (int b = 0; b < kChunks; ++b) {
                // shared memory is free when the last block's product over these dims is done; the TMEM slot
                // when the scores' product two chunks ago is
                if (i > 0) live = live && mbar_wait(smem_addr(&sh.oblk[b]), phase ^ 1);
                if (i > 0 || b >= 2) live = live && mbar_wait(smem_addr(&sh.kfree[b & 1]), b >= 2 ? 0 : 1);
                tc_fence_after();
                if (b == 0 && q == 0) {
                    sh.valid[phase][tok0] = ok[0];
                    sh.valid[phase][tok0 + 8] = ok[1];
                }
                const uint32_t s0 = b == 0 ? now[0].x : b == 1 ? now[0].y : b == 2 ? now[0].z : now[0].w;
                const uint32_t s1 = b == 0 ? now[1].x : b == 1 ? now[1].y : b == 2 ? now[1].z : now[1].w;
#pragma unroll
                for (int ci = 0; ci < 4; ++ci) {
                    uint32_t v0[4], v1[4];
                    decode8<L>(raw[b][0], ci, q, s0, v0);
                    decode8<L>(raw[b][1], ci, q, s1, v1);
                    const int sub = 2 * b + (L == Layout::V41 ? ci >> 1 : 0);
                    const uint32_t at = krow + sub * kSubBytes + (L == Layout::V41 ? 0 : (q >> 1) * kSubBytes) +
                                        ((kxor ^ (L == Layout::V41 ? (ci & 1) : ci)) << 4);
                    sts_u4(at, v0);
                    sts_u4(at + 8 * 128, v1);
                    tmem_st_16x128b_x4(tlane + (b & 1) * 64 + 16 * ci, v0, v1);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) load_raw<L>(raw[b][h], code[h], b, q);
                tc_wait_st();
                tc_fence_before();
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.full[b]));
            }
            if (!live) {
                sh.abort = 1;
                break;
            }
            ok[0] = code[0] != nullptr;
            ok[1] = code[1] != nullptr;
            now[0] = sc[0];
            now[1] = sc[1];
        }
    } else if (warp == kSoftWarps + kDeqWarps) {
        // ------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t kIdescS = mma_idesc(kTile, N, kBf16, false, false);
            constexpr uint32_t kIdescO = mma_idesc(kTile, N, kBf16, true, true);
            constexpr uint64_t kPSwizzle = N == 64 ? kSwizzle128 : N == 32 ? kSwizzle64 : kSwizzle32;
            const uint64_t qd = smem_desc(smem_addr(sQ), 16, 1024, kSwizzle128);
            const uint64_t vd = smem_desc(smem_addr(sK), kSubBytes, 1024, kSwizzle128);
            const uint64_t pd = smem_desc(smem_addr(sP), 16, 16 * N, kPSwizzle);
            int64_t left_tile = 0;
            uint32_t seg = 0;
            int64_t tile = sh.start_tile;
            int kb = sh.start_kb;
            bool live = true;
            for (int64_t i = 0; i < units && live; ++i) {
                const uint32_t phase = uint32_t(i) & 1;
                bool first = false;
                if (left_tile == 0) {  // a new tile: its queries, a fresh accumulator
                    left_tile = tile_info<N, kSlots>(a, tile).nb - kb;
                    ++tile;
                    kb = 0;
                    first = true;
                    live = live && mbar_wait(smem_addr(&sh.qready), seg & 1);
                    ++seg;
                }
                --left_tile;
                for (int b = 0; b < kChunks && live; ++b) {
                    live = live && mbar_wait(smem_addr(&sh.full[b]), phase);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(tmem + kTmemS, tmem + kTmemK + (b & 1) * 64 + 8 * k,
                               qd + ((((2 * b + (k >> 2)) * N * 128) + (k & 3) * 32) >> 4), kIdescS, b + k > 0);
                    mma_commit(smem_addr(&sh.kfree[b & 1]));
                }
                mma_commit(smem_addr(&sh.sdone));
                live = live && mbar_wait(smem_addr(&sh.pready), phase);
                tc_fence_after();
                for (int b = 0; b < kChunks; ++b) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ss(tmem + b * N, vd + ((2 * b * kSubBytes + k * 2048) >> 4), pd + ((k * 32 * N) >> 4),
                               kIdescO, !first || k > 0);
                    mma_commit(smem_addr(&sh.oblk[b]));
                }
            }
            if (!live) {
                sh.abort = 1;
                mma_commit(smem_addr(&sh.drain));   // nothing may write TMEM once it is freed
                mbar_wait(smem_addr(&sh.drain), 0);
            }
        }
    } else {
        // ------------------------------------------------------ softmax, queries, outputs
        const float c = a.scale * kLog2e;
        const int64_t per = int64_t(a.q_len) * a.heads;
        const uint32_t trow = tmem + (uint32_t(warp * 32) << 16);
        Cursor<N, kSlots> cur(a, sh);
        float l[N];
        // A warp that gives up a wait says so before the four warps' next barrier, so that all leave together.
        volatile int &gone = sh.soft_abort;
        bool unset = false, live = true;
        int kb0 = 0;
        for (int64_t i = 0; i < units && live; ++i, cur.next(a)) {
            const uint32_t phase = uint32_t(i) & 1;
            const bool first = i == 0 || cur.kb == 0;
            if (first) {
                // the scores' products of the last tile are done (their result was waited for)
                kb0 = cur.kb;
                if (tid == 0 && cur.kb == 0 && cur.t.rt == 0 && cur.t.err) raise_err(a.err, cur.t.err);
                const int64_t row0 = int64_t(cur.t.rt) * N;
                const uint32_t sq = smem_addr(sQ);
#pragma unroll 4
                for (int r = warp; r < N; r += kSoftWarps) {
                    const int64_t R = row0 + r;
                    uint4 u[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
                    if (R < per) {
                        const uint16_t *p = a.q + (cur.t.seq * a.q_len + R / a.heads) * a.q_tok + (R % a.heads) * a.q_head;
                        u[0] = ld_stream_u4(p + lane * 8);
                        u[1] = ld_stream_u4(p + (lane + 32) * 8);
                    }
                    float back = 1.f;
                    uint32_t v[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
                    if constexpr (!kBf16) {
                        // fp16: the row times a power of two that brings its largest magnitude to [2^14, 2^15)
                        uint32_t big = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) big = max(big, max((v[e] << 16) & 0x7FFF0000u, v[e] & 0x7FFF0000u));
                        big = __reduce_max_sync(0xFFFFFFFFu, big);
                        const uint32_t up = min(268u - (big >> 23), 254u);
                        const float f = __uint_as_float(up << 23);
                        back = ue8m0_to_f32(254u - up);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v[e]) : "f"(bf16_hi(v[e]) * f), "f"(bf16_lo(v[e]) * f));
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sts_u32(sq + q_word<L, N>(r, lane + 32 * (e >> 2), e & 3), v[e]);
                    if (lane == 0) {
                        const int64_t Rc = min(R, per - 1);
                        const int64_t tok = cur.t.seq * a.q_len + Rc / a.heads;
                        sh.sc[r] = c * back;
                        sh.m[r] = -INFINITY;
                        sh.vis[r] = kSlots || R >= per ? cur.t.seen : max(0, cur.t.len - (a.q_len - 1 - int(Rc / a.heads)));
                        sh.row[r] = R < per ? tok * a.out_tok + (Rc % a.heads) * a.out_head : -1;
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.qready));
                soft_sync();
#pragma unroll
                for (int j = 0; j < N; ++j) l[j] = 0.f;
                unset = true;
            }
            // full[0] orders this thread's read of `valid`
            if (!mbar_wait(smem_addr(&sh.full[0]), phase) || !mbar_wait(smem_addr(&sh.sdone), phase)) gone = 1;
            tc_fence_after();
            const int64_t t64 = int64_t(cur.kb) * kTile + tid;
            const bool have = sh.valid[phase][tid];
            const int t_at = have ? int(t64) : 0x7FFFFFFF;
            // whether some of the block is masked for some row (the first row of a tile sees least)
            const bool masked = !__all_sync(0xFFFFFFFFu, have) || (int64_t(cur.kb) + 1) * kTile > sh.vis[0];

            auto scores = [&](int j0, uint32_t (&s)[1][16]) {
                tmem_ld16(trow + kTmemS + j0, s[0]);
                tmem_ld_done(s);
            };
            bool move = unset;
            if (!move) {
                float top = -INFINITY;
#pragma unroll
                for (int j0 = 0; j0 < N; j0 += 16) {
                    uint32_t s[1][16];
                    scores(j0, s);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 x = ffma2(make_float2(__uint_as_float(s[0][j]), __uint_as_float(s[0][j + 1])),
                                               *reinterpret_cast<const float2 *>(&sh.sc[j0 + j]),
                                               *reinterpret_cast<const float2 *>(&sh.nm[j0 + j]));
                        if (masked) {
                            if (t_at < sh.vis[j0 + j]) top = fmaxf(top, x.x);
                            if (t_at < sh.vis[j0 + j + 1]) top = fmaxf(top, x.y);
                        } else {
                            top = fmax3(top, x.x, x.y);
                        }
                    }
                }
                move = soft_any(top > kStaleMax);
            }
            if (move) {
                // the columns' new maxima, and what is summed so far in their terms
                float mine[(N + 31) / 32];
#pragma unroll
                for (int k = 0; k < (N + 31) / 32; ++k) mine[k] = -INFINITY;
#pragma unroll
                for (int j0 = 0; j0 < N; j0 += 16) {
                    uint32_t s[1][16];
                    scores(j0, s);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float x = __uint_as_float(s[0][j]) * sh.sc[j0 + j];
                        if (!(t_at < sh.vis[j0 + j])) x = -INFINITY;
                        x = redux_max(x);
                        if (lane == ((j0 + j) & 31)) mine[(j0 + j) >> 5] = x;
                    }
                }
#pragma unroll
                for (int k = 0; k < (N + 31) / 32; ++k)
                    if (lane + 32 * k < N) sh.red[warp][lane + 32 * k] = mine[k];
                soft_sync();
                bool none = false;
                if (tid < N) {
                    const float m0 = sh.m[tid];
                    const float m1 = fmaxf(fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid])), m0);
                    sh.m[tid] = m1;
                    sh.nm[tid] = m1 == -INFINITY ? 0.f : -m1;
                    sh.alpha[tid] = m1 == -INFINITY ? 1.f : ex2_approx(m0 - m1);
                    none = m1 == -INFINITY;
                }
                unset = soft_any(none);
#pragma unroll
                for (int j = 0; j < N; ++j) l[j] *= sh.alpha[j];
                if (!first) {
#pragma unroll 1
                    for (int b = 0; b < kChunks; ++b)
#pragma unroll
                        for (int j0 = 0; j0 < N; j0 += 16) {
                            uint32_t o[1][16];
                            tmem_ld16(trow + b * N + j0, o[0]);
                            tmem_ld_done(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                o[0][j] = __float_as_uint(__uint_as_float(o[0][j]) * sh.alpha[j0 + j]);
                            tmem_st16(trow + b * N + j0, o[0]);
                        }
                    tc_wait_st();
                }
            }
            if (gone) {   // a barrier lies between any warp's wait and here
                live = false;
                break;
            }
            bool odd = false;   // a score that is not finite, where some rows do not see the token
#pragma unroll
            for (int j0 = 0; j0 < N; j0 += 16) {
                uint32_t s[1][16];
                scores(j0, s);
                float p[16];
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    float2 x = ffma2(make_float2(__uint_as_float(s[0][j]), __uint_as_float(s[0][j + 1])),
                                     *reinterpret_cast<const float2 *>(&sh.sc[j0 + j]),
                                     *reinterpret_cast<const float2 *>(&sh.nm[j0 + j]));
                    if (masked) {
                        odd = odd || !(fabsf(__uint_as_float(s[0][j])) < INFINITY) ||
                              !(fabsf(__uint_as_float(s[0][j + 1])) < INFINITY);
                        if (!(t_at < sh.vis[j0 + j])) x.x = -INFINITY;
                        if (!(t_at < sh.vis[j0 + j + 1])) x.y = -INFINITY;
                    }
                    p[j] = ex2_approx(x.x);
                    p[j + 1] = ex2_approx(x.y);
                    l[j0 + j] += p[j];
                    l[j0 + j + 1] += p[j + 1];
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (kBf16)
                            w[e] = pack_bf16x2(p[8 * v + 2 * e], p[8 * v + 2 * e + 1]);
                        else
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(p[8 * v + 2 * e + 1]), "f"(p[8 * v + 2 * e]));
                    }
                    sts_u4(smem_addr(sP) + p_vec<N>(tid, j0 / 8 + v), w);
                }
            }
            if (masked && odd && have) {
                // a weight of 0 does not silence a NaN: if the token's row itself is not finite, the rows that see
                // it are NaN by their weights already, and the others must meet zeros
                const uint32_t row = smem_addr(sK) + tid * 128;
                bool bad = false;
                for (int v = 0; v < 64; ++v) {
                    const uint4 u = lds_u4(row + (v >> 3) * kSubBytes + (v & 7) * 16);
                    constexpr uint32_t kInf = kBf16 ? 0x7F80u : 0x7C00u;
                    const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
                    for (int e = 0; e < 4; ++e)
                        bad = bad || (ws[e] & kInf) == kInf || ((ws[e] >> 16) & kInf) == kInf;
                }
                if (bad)
                    for (int v = 0; v < 64; ++v) {
                        const uint32_t z[4] = {0u, 0u, 0u, 0u};
                        sts_u4(row + (v >> 3) * kSubBytes + (v & 7) * 16, z);
                    }
            }
            tc_fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.pready));

            const bool last = i + 1 == units || cur.kb + 1 == cur.t.nb;
            if (last) {
                // ---- this CTA's part of the tile is done
                const bool whole = kb0 == 0 && cur.kb + 1 == cur.t.nb;
                const int col = warp_columns_sum<N>(l, lane);
#pragma unroll
                for (int k = 0; k < (N + 31) / 32; ++k)
                    if (N >= 32 || (lane & 1) == 0) sh.red[warp][col + k] = l[k];
                soft_sync();
                float *part = nullptr;
                if (!whole) part = a.part + (2 * int64_t(blockIdx.x) + (kb0 == 0 ? 1 : 0)) * N * kPartRow;
                if (tid < N) {
                    const float sum = (sh.red[0][tid] + sh.red[1][tid]) + (sh.red[2][tid] + sh.red[3][tid]);
                    const float m = sh.m[tid];
                    sh.inv[tid] = whole ? (m == -INFINITY && sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                    const int64_t R = int64_t(cur.t.rt) * N + tid;
                    if (!whole) {
                        part[tid * kPartRow + kD] = m;
                        part[tid * kPartRow + kD + 1] = sum;
                    } else if (a.lse && R < per) {
                        a.lse[cur.t.seq * per + R] = attend_lse(m, sum);
                    }
                }
                if (tid == 0 && (i + 1 == units)) {
                    int2 join = make_int2(-1, 0);
                    if (kb0 == 0 && !whole) {  // later CTAs hold the rest of this tile
                        const int64_t end = sh.u1 + (cur.t.nb - 1 - cur.kb) - 1;   // its last unit
                        const int64_t g = min(int64_t(gridDim.x), int64_t(sh.total));
                        join = make_int2(int(cur.tile), int(((end + 1) * g - 1) / sh.total));
                    }
                    a.join[blockIdx.x] = join;
                }
                soft_sync();
                const bool done = mbar_wait(smem_addr(&sh.oblk[kChunks - 1]), phase);
                if (!done) gone = 1;
                tc_fence_after();
                if (done) {
#pragma unroll 1
                    for (int b = 0; b < kChunks; ++b) {
                        const int d = b * kChunk + tid;
#pragma unroll 1
                        for (int j0 = 0; j0 < N; j0 += 16) {
                            uint32_t o[1][16];
                            tmem_ld16(trow + b * N + j0, o[0]);
                            tmem_ld_done(o);
                            if (!whole) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) part[(j0 + j) * kPartRow + d] = __uint_as_float(o[0][j]);
                            } else if (a.out_bf16) {
                                // neighbouring lanes swap columns, so that a store is two dims of one row
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    const float x = __uint_as_float(o[0][j]) * sh.inv[j0 + j];
                                    const float y = __uint_as_float(o[0][j + 1]) * sh.inv[j0 + j + 1];
                                    const float z = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? x : y, 1);
                                    const int64_t row = sh.row[j0 + j + (lane & 1)];
                                    const uint32_t two = (lane & 1) ? pack_bf16x2(z, y) : pack_bf16x2(x, z);
                                    if (row >= 0)
                                        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + row + (d & ~1)) = two;
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const int64_t row = sh.row[j0 + j];
                                    if (row >= 0) static_cast<float *>(a.out)[row + d] = __uint_as_float(o[0][j]) * sh.inv[j0 + j];
                                }
                            }
                        }
                    }
                }
                tc_fence_before();
                soft_sync();   // the tile's arrays are free for the next one
                live = !gone;
            }
        }
        if (!live) {
            if (lane == 0) raise_err(a.err, KVQ_DEVERR_WAIT);
            sh.abort = 1;
            if (tid == 0) a.join[blockIdx.x] = make_int2(-1, 0);
        }
    }
    __syncwarp();
    if (tid == 0) pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sh.abort) raise_err(a.err, KVQ_DEVERR_WAIT);
    if (warp == kSoftWarps + kDeqWarps) tmem_dealloc(tmem, kTmemCols);
}

// Joins the tiles that CTAs split: CTA (x, y) takes rows 4y .. 4y+3 of the
// tile whose first part CTA x made, one warp a row, and adds the parts in
// order, each weighted by 2^(its maximum - the largest).
template <int N>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendArgs a) {
    pdl_wait();
    const int2 join = a.join[blockIdx.x];
    const int r = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (join.x < 0) return;
    const int64_t per = int64_t(a.q_len) * a.heads;
    const int64_t seq = join.x / a.row_tiles, R = int64_t(join.x % a.row_tiles) * N + r;
    if (R >= per) return;
    const int parts = join.y - int(blockIdx.x) + 1;
    auto at = [&](int i) {
        return a.part + ((i == 0 ? 2 * int64_t(blockIdx.x) + 1 : 2 * (int64_t(blockIdx.x) + i)) * N + r) * kPartRow;
    };
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, at(i)[kD]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float zero = top == -INFINITY ? 0.f : top;
    float acc[16], sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float *p = at(i);
        const float w = ex2_approx(p[kD] - zero);
        sum = fmaf(w, p[kD + 1], sum);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = *reinterpret_cast<const float4 *>(p + 128 * k + 4 * lane);
            acc[4 * k] = fmaf(w, v.x, acc[4 * k]);
            acc[4 * k + 1] = fmaf(w, v.y, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(w, v.z, acc[4 * k + 2]);
            acc[4 * k + 3] = fmaf(w, v.w, acc[4 * k + 3]);
        }
    }
    const float inv = top == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
    const int64_t tok = seq * a.q_len + R / a.heads;
    const int64_t row = tok * a.out_tok + (R % a.heads) * a.out_head + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x = acc[4 * k] * inv, y = acc[4 * k + 1] * inv, z = acc[4 * k + 2] * inv, w = acc[4 * k + 3] * inv;
        if (a.out_bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row + 128 * k) =
                make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row + 128 * k) = make_float4(x, y, z, w);
    }
    if (a.lse && lane == 0) a.lse[seq * per + R] = attend_lse(top, sum);
}

template <Layout L, int N, bool kSlots>
kvq_status launch_attend_n(AttendArgs a, cudaStream_t s) {
    const int64_t per = int64_t(a.q_len) * a.heads;
    a.row_tiles = int((per + N - 1) / N);
    const int64_t tiles = a.n_seq * a.row_tiles;
    if (tiles > 0x7FFFFFFF) return KVQ_ERR_UNSUPPORTED;
    int64_t grid = 0;
    kvq_status st = resident_grid<attend_kernel<L, N, kSlots>, kAttendThreads>(kAttendSmem<N>, &grid);
    if (st != KVQ_OK) return st;
    if (grid > kMaxAttendCtas) grid = kMaxAttendCtas;
    const int64_t most = (a.max_len + kTile - 1) / kTile;   // blocks of the longest tile there can be
    if (most <= 1 && tiles < grid) grid = tiles;
    a.join = reinterpret_cast<int2 *>(a.ws);
    a.part = reinterpret_cast<float *>(a.ws + kMaxAttendCtas * sizeof(int2));
    st = launch_pdl_smem(attend_kernel<L, N, kSlots>, dim3(unsigned(grid)), dim3(kAttendThreads), kAttendSmem<N>, s, a);
    if (st != KVQ_OK || most <= 1) return st;  // a tile of one block is never split
    return launch_pdl(attend_join_kernel<N>, dim3(unsigned(grid), N / 4), dim3(128), s, a);
}

template <Layout L, bool kSlots>
kvq_status launch_attend_layout(const AttendArgs &a, cudaStream_t s) {
    switch (attend_rows(int64_t(a.q_len) * a.heads)) {
        case 16: return launch_attend_n<L, 16, kSlots>(a, s);
        case 32: return launch_attend_n<L, 32, kSlots>(a, s);
        default: return launch_attend_n<L, 64, kSlots>(a, s);
    }
}

}  // namespace
}  // namespace kvq
