// kvq_attend_kernel.cuh -- the tensor-core attention kernel and its join.
//
// For a tile of N query rows q and the cached rows k[t] (512 dims, key and
// value at once), block after block of 64 tokens:
//   S^T[t, r] = sum_d k[t, d] q[r, d]           (tokens x rows)
//   x = scale log2(e) S,  p[t, r] = 2^(x - m_r),  l_r += sum_t p
//   O^T[d, r] += sum_t k[t, d] p[t, r]          (dims x rows)
// and in the end out = O / l, lse = (m + log2 l) ln 2.  Both products have the
// cached rows on the tensor cores' wide side (M = 64 tokens, M = 128 dims) and
// the query rows on the narrow one (N = 16, 32, 64), so few heads waste no
// more than their tile's padding.  m_r lags: a block moves it, and rescales O
// in TMEM, only when a weight would pass 2^kStaleMax, which still fits fp16;
// after a tile's first block that is rare.
//
// A block is decoded once for both products: 16 bits a value into shared
// memory (the A operand of O^T, dims contiguous) and into TMEM (the A operand
// of S^T).  From TMEM the scores' products take 18 to 33 clocks each (N = 16 to
// 64), from shared memory 42 to 49, since the 128 bytes a clock of shared
// memory carry the decoded rows' stores, the outputs' operands and the weights
// already.  Loads touch eight rows at a time (a thread a token: 1.4 times as
// long in all).
//
// The tiles' blocks in order are cut into equal shares, one a CTA (one an SM),
// whatever the lengths: a long sequence is spread over the machine and short
// ones are packed.  Tiles that a cut passes through leave partial sums, which
// attend_join_kernel adds in order, so the result does not depend on timing.
//
// Rules for N by the rows of a sequence (kvq_attend.cuh), in us, one sequence of
// 100 tokens / 48 of 1,024 to 8,192 tokens:
//             V41, as 16    32         64           FP4, as 16    32         64
//   16 heads  10.2 / 38   11.4 / 45  14.1 / 61      10.1 / 37   11.2 / 43  13.9 / 58
//   32 heads              11.5 / 45  14.2 / 61                  11.3 / 43  14.0 / 59
//   64 heads              11.5 / 78  14.4 / 64                  11.4 / 74  14.1 / 61
// (64 heads as twice 32: shorter where there are two blocks in all, longer from
// then on.)
//
// What bounds it: a block of 64 tokens takes 2,150 to 2,180 clocks at N = 16,
// 2,270 (FP4) to 2,400 (V41) at N = 32, 2,810 to 3,060 at N = 64 (152 equal
// sequences, 40 against 200 blocks, at 2,070 MHz: 0.3, 0.6 and 0.9 PFLOP/s, of
// which tensor cores need about 1,240 clocks at N = 16 and 1,850 at N = 64), and
// no unit is full.  The rest is the chain of a block: its outputs free the slots
// that the block after the next is decoded into (wait 100, codes from L2 to
// registers, conversions and stores 500, fences 250), then the scores (600 to
// 1,100), the softmax (1,200 to 1,500) and the outputs (700 to 800); two blocks
// are under way at a time.  A tile costs 3.2, 4.7 and 8.8 us besides (queries,
// first maximum, outputs; 80 blocks a CTA as one tile or as eight), and shares
// count blocks alone: CTAs that hold many short tiles end last.  With blocks of
// 128 tokens 129 x 2,048 slots of 32 heads take 65 instead of 55 us and long
// calls 1 to 4 % longer (a call of two blocks 8.4 instead of 9.8); a ring of
// three blocks at N = 16, a second code buffer in registers, two score buffers
// at N = 64 and one wait for a block's four chunks change nothing or cost up to
// 10 %.
#pragma once

#include <math.h>

#include "kvq_attend.cuh"
#include "kvq_attend_rows.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTile = 64;    // cached tokens a block
constexpr int kChunk = 128;  // dims a step of decoding
constexpr int kChunks = kD / kChunk;
constexpr int kSubBytes = kTile * 128;         // 64 dims of a block, 128 B a token
constexpr int kChunkSmem = 2 * kSubBytes;
// Warps: 0-7 softmax (two a TMEM lane quarter, each half of the columns), 8-23 decode (four a chunk, so that one
// chunk's stores overlap the others' waits), 24 the scores' products, 25 and 26 look up where the rows of coming blocks
// lie, 27 the outputs' products.
constexpr int kSoftWarps = 8, kDeqWarps = 16, kMmaWarp = kSoftWarps + kDeqWarps;
constexpr int kAttendThreads = (kMmaWarp + 4) * 32;
// Registers a thread: the launch gives 896 threads 72 each, and the warpgroups' shares stay within that sum.  With
// these none spills; 88/64/72 costs the 64-row tiles 3 % (spills), 96/72/24 1 to 2 %.
constexpr int kLaunchRegs = 72, kSoftRegs = 104, kDeqRegs = 56;
static_assert(2 * kSoftRegs + 4 * kDeqRegs + kLaunchRegs <= 7 * kLaunchRegs, "a larger sum would wait for ever");
// How large (log2) a weight may become before the running maximum moves: weights stay below fp16's 65504, and a move
// (which rescales the outputs in TMEM) is rare after a tile's first block.
constexpr float kStaleMax = 15.f;
// A moved maximum gives the largest weight 2^headroom, and a weight that is 2^-(25 + headroom) of it or less is fp16's
// zero.  What a long flat tail behind one large weight can lose that way grows with the tokens summed, so the headroom
// does too: of n tokens at most n 2^-(25 + headroom) <= 2^-13 of the largest weight is lost, up to 2^26 tokens.  Less
// headroom means fewer moves (4-bit decode / long / chunk 99.8 / 77.3 / 774 us with none, 103 / 82 / 804 with 4, 113 /
// 91 / 892 with 8, 137 / 112 / 1016 with 12, whatever the length), and a part of up to 64 blocks, as most are, needs none.
constexpr int kTailBlocks = 6, kMaxHeadroom = 14, kFoldBlocks = 64;
// The tensor cores round their sums down, so what is summed in TMEM falls short by more the longer it goes on (2^-17 of
// it after 2,048 blocks, 2^-10 after 16,384, 2 % after 131,072).  Every kFoldOut blocks the outputs so far are added to
// the part's place in the workspace, which rounds to nearest, and the products start afresh.
constexpr int kFoldOut = 256;
static_assert(kFoldOut % kFoldBlocks == 0, "one test finds a block that begins with neither");
__device__ __forceinline__ float headroom(int blocks) {
    return float(min(max(32 - __clz(max(blocks - 1, 0)) - kTailBlocks, 0), kMaxHeadroom));
}

// Decoded chunks: two blocks (a block is four), so that one is decoded while the other is multiplied.
constexpr int kRing = 2 * kChunks;
// Chunks that TMEM holds for the scores' products, beside the outputs (4 N columns) and one or two blocks' scores.
template <int N>
constexpr int kTmemRing = N == 64 ? 3 : N == 32 ? 5 : 6;
template <int N>
constexpr int kScoreBufs = N == 64 ? 1 : 2;
// Barriers that tell which chunks' scores are done, in turn.  A wait tells a phase only from its neighbours: the
// chunk that it waits for is KR = kTmemRing chunks back, the phase after is complete only once this chunk is decoded
// if there are KR barriers or more, and the phase before is known to be if there are kChunks or more (the warp's last
// chunk waited for it).
template <int N>
constexpr int kScored = kTmemRing<N> > kChunks ? kTmemRing<N> : kChunks;
// What a tile costs beside its blocks, in blocks, where shares count it: a tree's rows make many tiles, and those of short
// sequences among long ones would all be one CTA's (8 trees of 63 tokens, 64 heads, two of the 8 sequences shorter than a
// block: 1,396 us without, 386 with; 24 trees of 24, 16 heads: 169 and 78).
template <int N, int kKind>
constexpr int kTileCost = kKind != kByTree ? 0 : N == 64 ? 6 : N == 32 ? 4 : 3;
constexpr int kLookups = 6, kLookupWarps = 2;
constexpr uint32_t kLookupTries = 16;  // a lookup warp's try is a sleep of 64 ns, a barrier's may take a microsecond

template <int N>
struct AttendShared {
    uint64_t full[kRing], oblk[kRing], scored[kScored<N>], sdone[2], sread[2], pready[2], qready, drain[2];
    int64_t scan[kAttendThreads / 32];
    int64_t total, u0, end_block;
    int units, start_tile, start_kb;
    uint32_t tmem;
    int abort, progress;
    alignas(16) float sc[N], nm[N], m[N], alpha[N], inv[N];
    float red[4][N], lsum[4][N];
    union {
        alignas(16) int vis[N];  // tokens that a query row sees; of a tree:
        uint32_t win[N][2];      // which of a block's tokens it sees
    };
    int64_t q[N], row[N];  // a query row's element offsets, -1: none
    // What the lookup warps found for a block's tokens, kLookups blocks in turn.
    uint64_t addr[kLookups];                   // full
    alignas(16) uint4 scale[kLookups][kTile];  // a row's scale bytes
    const uint8_t *code[kLookups][kTile];      // a row's codes
    int texp[kLookups][kTile];                 // a row's power of two, or kNoToken
};

template <int N>
constexpr size_t kAttendSmem = 1024 + size_t(kRing) * kChunkSmem + size_t(N) * kD * 2 + 2 * size_t(kTile) * N * 2 +
                               sizeof(AttendShared<N>);
static_assert(kAttendSmem<16> <= 232448 && kAttendSmem<32> <= 232448 && kAttendSmem<64> <= 232448, "227 KB a CTA");

// Tiles are N query rows of a sequence (row = query token * heads + head);
// a tile's blocks are the 64-token pieces of what its last query token sees.
struct TileInfo {
    int seq, rt, len, seen, nb;  // cached tokens, tokens the last row sees, blocks (at least one)
    int trow, err;
};

template <int N, int kKind>
__device__ __forceinline__ TileInfo tile_info(const AttendArgs &a, int tile) {
    TileInfo t;
    t.seq = int(uint32_t(tile) / uint32_t(a.row_tiles));
    t.rt = int(uint32_t(tile) % uint32_t(a.row_tiles));
    t.err = 0;
    t.trow = t.seq;
    if constexpr (kKind == kBySlots) {
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
        if (kKind == kByPages && a.q_len > 1) {
            const int64_t per = int64_t(a.q_len) * a.heads;
            const int last = int(min(int64_t(t.rt + 1) * N, per) - 1);
            t.seen = max(0, t.len - (a.q_len - 1 - last / a.heads));
        }
    }
    t.nb = max(1, (t.seen + kTile - 1) / kTile);
    return t;
}

// Which of the 64 tokens from t0 on a drafted token sees, of a tree that begins at token `base`: all those before it, and
// of the drafted ones those in its mask.
__device__ __forceinline__ uint64_t tree_window(const uint64_t *mask, int words, int t0, int base) {
    const int off = t0 - base;
    if (off <= -kTile) return ~0ull;
    if (off < 0) return ((1ull << -off) - 1) | (__ldg(mask) << -off);
    const int w = off >> 6, sh = off & 63;
    uint64_t r = w < words ? __ldg(mask + w) >> sh : 0;
    if (sh && w + 1 < words) r |= __ldg(mask + w + 1) << (64 - sh);
    return r;
}

// Walks a CTA's blocks in order.
template <int N, int kKind>
struct Cursor {
    int tile, kb, left;
    TileInfo t;
    __device__ __forceinline__ Cursor(const AttendArgs &a, const AttendShared<N> &sh)
        : tile(sh.start_tile), kb(sh.start_kb), left(sh.units), t(tile_info<N, kKind>(a, tile)) {}
    __device__ __forceinline__ void next(const AttendArgs &a) {
        --left;
        if (++kb >= t.nb) {
            kb = 0;
            ++tile;
            if (left > 0) t = tile_info<N, kKind>(a, tile);
        }
    }
};

// The ring of decoded chunks, walked by every role in the same order.
template <int R>
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++slot == R) {
            slot = 0;
            parity ^= 1;
        }
    }
};

// Where a decoded row lies.  A decode thread holds, of tokens r and r + 8
// (r = lane / 4) of its warp's 16 and of its chunk of 128 dims, the 16 dims
// from 64 s + 16 q (q = lane % 4, s = 0, 1), as two vectors e = 0, 1 of eight:
// a warp's load touches eight rows, where a thread a token would touch 32 (and
// take 1.4 times as long in all).  In shared memory a chunk is two
// 128-byte-swizzled tiles of 64 dims; the eight lanes of a store's phase (two
// tokens, four q) hit different banks.  In TMEM (the A operand of the scores'
// product) a block's 64 rows are the first 16 lanes of each of the four lane
// quarters, and vector e of half s fills the columns 32 s + 16 e + 4 i + q,
// i = 0..3, two dims a column: the contraction runs over the dims in another
// order, and q_word() puts a query's dims in the same one.
//
// p: the thread's first code of the chunk.
template <Layout L>
__device__ __forceinline__ Raw<L> load_raw(const uint8_t *p, int s) {
    Raw<L> r;
    // volatile: a load stays where it is issued
    if constexpr (L == Layout::V41) {
        asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                     : "l"(p + s * 64));
    } else {
        asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p + s * 32));
    }
    return r;
}

// Byte offset, in a query tile's shared memory, of word i (dims 8g + 2i,
// 8g + 2i + 1) of piece g = 0..63 of row r.
template <int N>
__device__ __forceinline__ uint32_t q_word(int r, int g, int i) {
    const int b = g >> 4, s = (g >> 3) & 1, q = (g >> 1) & 3, e = g & 1;
    return uint32_t((2 * b + s) * N * 128 + r * 128 + (((4 * e + i) ^ (r & 7)) << 4) + q * 4);
}

// Swizzled byte offset of 16-byte vector j of row t of the weights' tile
// (rows of N 16-bit values).
template <int N>
__device__ __forceinline__ uint32_t p_vec(int t, int j) {
    const int x = N == 64 ? (t & 7) : N == 32 ? ((t >> 1) & 3) : ((t >> 2) & 1);
    return uint32_t(t * N * 2 + ((j ^ x) << 4));
}

// Over the eight lanes that differ in lane / 4.
__device__ __forceinline__ float rows_max(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float rows_sum(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Barrier of the softmax warps; the second form returns whether any of
// their threads brought true.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The other warps tell that they are done, the softmax warps wait for that.
__device__ __forceinline__ void done_arrive() {
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(kAttendThreads) : "memory");
}
__device__ __forceinline__ void done_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kAttendThreads) : "memory"); }
__device__ __forceinline__ bool soft_any(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
        "bar.red.or.pred b, 1, 256, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(p))
        : "memory");
    return r != 0;
}

template <Layout L, int N, int kKind>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
    using T = LayoutTraits<L>;
    constexpr bool kSlots = kKind == kBySlots, kTree = kKind == kByTree;
    constexpr int kCost = kTileCost<N, kKind>;
    constexpr bool kExp = L == Layout::V41;   // rows carry a power of two
    constexpr int R = kRing;
    constexpr int KR = kTmemRing<N>, kBufs = kScoreBufs<N>;
    // TMEM columns: outputs, scores, chunks of rows
    constexpr uint32_t kTmemS = 4 * N, kTmemK = (4 + kBufs) * N;
    constexpr uint32_t kTmemCols = 512;  // all of them, which begin at column 0
    static_assert(kTmemK + 64 * KR <= kTmemCols, "they fit");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + (-(uintptr_t(smem_addr(smem_raw))) & 1023);
    uint8_t *const sK = base, *const sQ = sK + R * kChunkSmem, *const sP = sQ + N * kD * 2;
    auto &sh = *reinterpret_cast<AttendShared<N> *>(sP + 2 * kTile * N * 2);
    // shuffled, so that the compiler knows it to be the same for a warp's lanes
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;

    // ---- what needs nothing of the grid before
    for (int i = tid; i < kLookups * kTile; i += kAttendThreads) sh.code[0][i] = a.pool;
    if (tid == 0) {
        for (int i = 0; i < kLookups; ++i) mbar_init(smem_addr(&sh.addr[i]), kLookupWarps);
        for (int i = 0; i < R; ++i) {
            mbar_init(smem_addr(&sh.full[i]), kDeqWarps / kChunks);
            mbar_init(smem_addr(&sh.oblk[i]), 1);
        }
        for (int i = 0; i < kScored<N>; ++i) mbar_init(smem_addr(&sh.scored[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.sread[i]), kSoftWarps);
            mbar_init(smem_addr(&sh.sdone[i]), 1);
            mbar_init(smem_addr(&sh.pready[i]), kSoftWarps);
        }
        mbar_init(smem_addr(&sh.qready), kSoftWarps);
        mbar_init(smem_addr(&sh.drain[0]), 1);
        mbar_init(smem_addr(&sh.drain[1]), 1);
        sh.abort = sh.progress = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&sh.tmem), kTmemCols);
    pdl_wait();

    // ---- this CTA's share: blocks [u0, u1) of all tiles' blocks in order
    const int tiles = int(a.n_seq * a.row_tiles);
    if constexpr (kSlots) {
        if (tid == 0) {
            const int64_t nb = max(int64_t(1), (a.max_len + kTile - 1) / kTile);
            const int64_t total = tiles * nb;
            int64_t u0, u1;
            share(total, u0, u1);
            sh.total = total;
            sh.u0 = u0;
            sh.units = int(u1 - u0);
            sh.start_tile = int(u0 / nb);
            sh.start_kb = int(u0 % nb);
        }
    } else {
        const int per = (tiles + kAttendThreads - 1) / kAttendThreads;
        const int t0 = int(min(int64_t(tiles), int64_t(tid) * per)), t1 = int(min(int64_t(tiles), int64_t(t0) + per));
        int64_t mine = 0;
#pragma unroll 1
        for (int t = t0; t < t1; ++t) mine += tile_info<N, kKind>(a, t).nb + kCost;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, (long long)incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        // every warp sums the warps' totals: lane w has that of warp w
        const int64_t of_warp = lane < kAttendThreads / 32 ? sh.scan[lane] : 0;
        int64_t before = lane < warp ? of_warp : 0, total = of_warp;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            before += __shfl_xor_sync(0xFFFFFFFFu, (long long)before, o);
            total += __shfl_xor_sync(0xFFFFFFFFu, (long long)total, o);
        }
        int64_t u0, u1;
        share(total, u0, u1);
        if (tid == 0) {
            sh.total = total;
            sh.u0 = u0;
            sh.units = int(u1 - u0);
        }
        int64_t at = before + incl - mine;
        if constexpr (kCost == 0) {
            if (u0 >= at && u0 < at + mine) {  // one thread
                int t = t0;
#pragma unroll 1
                for (; t + 1 < t1; ++t) {
                    const int nb = tile_info<N, kKind>(a, t).nb;
                    if (u0 < at + nb) break;
                    at += nb;
                }
                sh.start_tile = t;
                sh.start_kb = int(u0 - at);
            }
        } else {
            // The shares are of units of which every tile has kCost before its blocks.  A share that ends among these has
            // no block of the tile, one that begins there has its first.  u0 and `units` count blocks, as without.
            __syncthreads();
            const int64_t blocks = total - int64_t(kCost) * tiles;
            if (tid == 0 && u1 == total) sh.end_block = blocks;
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const int64_t u = e ? u1 : u0;
                if (!(u >= at && u < at + mine)) continue;  // one thread goes on
                int t = t0;
                int64_t vs = at;
#pragma unroll 1
                for (; t + 1 < t1; ++t) {
                    const int nb = tile_info<N, kKind>(a, t).nb + kCost;
                    if (u < vs + nb) break;
                    vs += nb;
                }
                const int kb = int(max(int64_t(0), u - vs - kCost));
                const int64_t block = vs - int64_t(kCost) * t + kb;
                if (e) {
                    sh.end_block = block;
                } else {
                    sh.start_tile = t;
                    sh.start_kb = kb;
                    sh.u0 = block;
                }
            }
            __syncthreads();
            if (tid == 0) sh.units = u1 > u0 ? int(sh.end_block - sh.u0) : 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    const int units = __shfl_sync(0xFFFFFFFFu, sh.units, 0);
    tc_fence_after();
    if (units == 0) {  // the same for every thread
        if (tid == 0) a.join[blockIdx.x] = make_int2(-1, 0);
        if (warp == kMmaWarp) tmem_dealloc(sh.tmem, kTmemCols);
        pdl_trigger();
        return;
    }

    if (warp >= kSoftWarps && warp < kMmaWarp) {
        // ------------------------------------------------------ decode
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDeqRegs));
        const int quarter = warp & 3, chunk = (warp - kSoftWarps) >> 2, q = lane & 3, r8 = lane >> 2;
        const int tok0 = 16 * quarter + r8;  // and tok0 + 8
        const uint32_t krow = smem_addr(sK) + tok0 * 128;
        const uint32_t at0 = krow + (((2 * q) ^ r8) << 4), at1 = krow + (((2 * q + 1) ^ r8) << 4);
        const uint32_t tlane = kTmemK + ((32 * quarter) << 16);
        const uint32_t lane_at = q * (T::kCodeBytes / 32) + chunk * (T::kCodeBytes / kChunks);
        const int scale_at = 4 * chunk + (q >> 1);  // and 2 further for the second half

        // A chunk's codes are loaded a block ahead, from L2, where the lookup warps have sent for them.  (A warp that has
        // given up follows no pointer that may be half written.)
        Raw<L> raw[2][2] = {};  // token, half
        auto load = [&](int k) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int s = 0; s < 2; ++s) raw[h][s] = load_raw<L>(sh.code[k][tok0 + 8 * h] + lane_at, s);
        };
        uint32_t tries = a.wait_tries;
        mbar_wait(smem_addr(&sh.addr[0]), 0, tries);
        if (tries) load(0);
        int slot = chunk, kslot = chunk % KR, k = 0;
        int before = (chunk + kScored<N> - KR) % kScored<N>;  // the barrier of the chunk that had this one's TMEM slot
        uint32_t parity = 0, looked = 0;  // `looked`: the phase of the next block's lookup
        uint32_t bparity = chunk + kScored<N> - KR < kScored<N> ? 1 : 0;
#pragma unroll 1
        for (int i = 0; i < units; ++i) {
            // the next block's entries (of the last block: its own again)
            const int kn = i + 1 == units ? k : k + 1 == kLookups ? 0 : k + 1;
            if (kn == 0 && i > 0) looked ^= 1;
            int texp[2];
            uint32_t m[2][2];  // token, half
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                texp[h] = sh.texp[k][tok0 + 8 * h];
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    m[h][s] = block_mul<L>(reinterpret_cast<const uint8_t *>(&sh.scale[k][tok0 + 8 * h])[scale_at + 2 * s], texp[h]);
            }
            if (!__all_sync(0xFFFFFFFFu, texp[0] != kNoToken && texp[1] != kNoToken)) {
                // a token that is not there has the pool's first row, which may hold anything: its codes are cleared, and
                // so are its multipliers, since 0 times a NaN or an infinity would be a NaN in every output
                asm volatile("");
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        m[h][s] = texp[h] != kNoToken ? m[h][s] : 0u;
#pragma unroll
                        for (int x = 0; x < int(sizeof(Raw<L>) / 4); ++x)
                            raw[h][s].w[x] = texp[h] != kNoToken ? raw[h][s].w[x] : 0u;
                    }
            }
            // a slot in shared memory is free when the product over the dims that it held is done, one in TMEM when
            // the scores over them are
            if (i * kChunks + chunk >= R) mbar_wait(smem_addr(&sh.oblk[slot]), parity ^ 1, tries);
            if (i * kChunks + chunk >= KR) mbar_wait(smem_addr(&sh.scored[before]), bparity, tries);
            tc_fence_after();
            const uint32_t off = slot * kChunkSmem;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t v0[4], v1[4];
                    decode8<L>(raw[0][s], e, m[0][s], v0);
                    decode8<L>(raw[1][s], e, m[1][s], v1);
                    const uint32_t at = (e ? at1 : at0) + off + s * kSubBytes;
                    sts_u4(at, v0);
                    sts_u4(at + 8 * 128, v1);
                    tmem_st_16x128b_x4(tlane + kslot * 64 + 32 * s + 16 * e, v0, v1);
                }
            fence_proxy_async();
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.full[slot]));
            if (i + 1 < units) mbar_wait(smem_addr(&sh.addr[kn]), looked, tries);
            if (tries) load(kn);
            slot += kChunks;
            if (slot >= R) {
                slot -= R;
                parity ^= 1;
            }
            kslot += kChunks % KR;
            if (kslot >= KR) kslot -= KR;
            before += kChunks;
            if (before >= kScored<N>) {
                before -= kScored<N>;
                bparity ^= 1;
            }
            if (warp == kSoftWarps && lane == 0) *const_cast<volatile int *>(&sh.progress) = i + 1;
            k = kn;
        }
        if (!tries) sh.abort = 1;
        done_arrive();
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------------ products
        if (warp == kMmaWarp) {
            // Scores, block after block: over a chunk as soon as it is decoded.  They run beside the softmax and the
            // outputs of the block before.
            constexpr uint32_t kIdesc = mma_idesc(kTile, N, false, false), kHi = desc_hi(1024, kSwizzle128);
            const uint32_t qd = desc_lo(smem_addr(sQ), 16);
            int left_tile = 0, tile = __shfl_sync(0xFFFFFFFFu, sh.start_tile, 0), kb = __shfl_sync(0xFFFFFFFFu, sh.start_kb, 0);
            uint32_t seg = 0;
            int kslot = 0, done = 0;
            uint32_t tries = a.wait_tries;
            Ring<R> ring;
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                if (left_tile == 0) {  // a new tile: its queries
                    left_tile = __shfl_sync(0xFFFFFFFFu, tile_info<N, kKind>(a, tile).nb, 0) - kb;
                    ++tile;
                    kb = 0;
                    mbar_wait(smem_addr(&sh.qready), seg & 1, tries);
                    ++seg;
                }
                --left_tile;
                // the score buffer is free when the softmax warps have read what it held
                if (i >= kBufs) mbar_wait(smem_addr(&sh.sread[(i - kBufs) & 1]), ((i - kBufs) >> 1) & 1, tries);
                const uint32_t to = kTmemS + (kBufs == 2 ? (i & 1) * N : 0);
#pragma unroll
                for (int b = 0; b < kChunks; ++b) {
                    mbar_wait(smem_addr(&sh.full[ring.slot]), ring.parity, tries);
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = qd + ((2 * b * N * 128) >> 4), from = kTmemK + kslot * 64;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_ts(to, from + 8 * k, at + (((k >> 2) * N * 128 + (k & 3) * 32) >> 4), kHi, kIdesc, b + k > 0);
                        mma_commit(smem_addr(&sh.scored[done]));
                        if (b == kChunks - 1) mma_commit(smem_addr(&sh.sdone[i & 1]));
                    }
                    __syncwarp();
                    ring.next();
                    if (++kslot == KR) kslot = 0;
                    if (++done == kScored<N>) done = 0;
                }
            }
            if (!tries) sh.abort = 1;
            tries = kWaitTries;
            if (elect_one()) mma_commit(smem_addr(&sh.drain[0]));  // nothing may write TMEM once it is freed
            mbar_wait(smem_addr(&sh.drain[0]), 0, tries);
        } else if (warp == kMmaWarp + 3) {
            // Outputs, block after block: 128 dims a product of the block's chunk with its weights.
            constexpr uint32_t kIdesc = mma_idesc(kChunk, N, true, true);
            constexpr uint32_t kPSwizzle = N == 64 ? kSwizzle128 : N == 32 ? kSwizzle64 : kSwizzle32;
            constexpr uint32_t kVHi = desc_hi(1024, kSwizzle128), kPHi = desc_hi(16 * N, kPSwizzle);
            const uint32_t vd = desc_lo(smem_addr(sK), kSubBytes), pd = desc_lo(smem_addr(sP), 16);
            int left_tile = 0, tile = __shfl_sync(0xFFFFFFFFu, sh.start_tile, 0), kb = __shfl_sync(0xFFFFFFFFu, sh.start_kb, 0);
            uint32_t tries = a.wait_tries;
            int since = 0;  // blocks of this part so far
            static_assert(R == 2 * kChunks, "a block's slots alternate between two runs");
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                if (left_tile == 0) {  // a new tile
                    since = 0;
                    left_tile = __shfl_sync(0xFFFFFFFFu, tile_info<N, kKind>(a, tile).nb, 0) - kb;
                    ++tile;
                    kb = 0;
                }
                --left_tile;
                const bool first = (since++ & (kFoldOut - 1)) == 0;  // a fresh accumulator
                mbar_wait(smem_addr(&sh.pready[i & 1]), (i >> 1) & 1, tries);
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t v = vd + (((i & 1) * kChunks * kChunkSmem) >> 4), p = pd + (((i & 1) * kTile * N * 2) >> 4);
#pragma unroll
                    for (int b = 0; b < kChunks; ++b) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            mma_ss(b * N, v + ((b * kChunkSmem + k * 2048) >> 4), kVHi, p + ((k * 32 * N) >> 4), kPHi, kIdesc,
                                   !first || k > 0);
                        mma_commit(smem_addr(&sh.oblk[(i & 1) * kChunks + b]));
                    }
                }
                __syncwarp();
            }
            if (!tries) sh.abort = 1;
            tries = kWaitTries;
            if (elect_one()) mma_commit(smem_addr(&sh.drain[1]));
            mbar_wait(smem_addr(&sh.drain[1]), 0, tries);
        } else if (warp <= kMmaWarp + kLookupWarps) {
            // Looks up where a block's rows lie and fetches their scales, up to three blocks ahead of the decode warps.
            // Every 128-byte line of a row is sent for to L2 (8-bit decode 44.2 us; without 46.6, a prefetch every 32
            // bytes 48.0, one bulk prefetch a row 51.9).  Lane l of a warp has a token.
            constexpr int K = kTile / 32 / kLookupWarps;
            const int mine = (warp - kMmaWarp - 1) * 32 * K + lane;  // the first of the lane's tokens
            using Index = std::conditional_t<kSlots, int64_t, int>;
            const uint32_t page_bytes = uint32_t(kTokenBytes<L>) << a.page_bits, in_page = (1u << a.page_bits) - 1;
            const uint32_t scale_at = uint32_t(T::kCodeBytes) << a.page_bits;
            volatile int &progress = sh.progress;
            Cursor<N, kKind> cur(a, sh);
            Index idx[K];
            int t0 = 0, seen = 0;
            uint32_t tries = a.wait_tries * kLookupTries;
            auto fetch = [&]() {
                t0 = cur.kb * kTile + mine;
                seen = cur.left > 0 ? cur.t.seen : 0;
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const int t = t0 + 32 * j;
                    idx[j] = -1;
                    if (t >= seen) continue;
                    if constexpr (kSlots) {
                        const int64_t at = cur.t.seq * a.slots_stride + t;
                        idx[j] = a.slots64 ? __ldg(static_cast<const int64_t *>(a.slots) + at)
                                           : int64_t(__ldg(static_cast<const int32_t *>(a.slots) + at));
                    } else {
                        idx[j] = __ldg(a.table + cur.t.trow * a.table_stride + (t >> a.page_bits));
                    }
                }
            };
            fetch();
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                const uint8_t *row[K];
                uint4 sc[K];
                uint32_t good = 0;
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const int t = t0 + 32 * j;
                    const bool g = t < seen && idx[j] >= 0 && idx[j] < a.pool_limit;
                    if (t < seen && !g && !(kSlots && idx[j] == -1)) raise_err(a.err, kSlots ? KVQ_DEVERR_SLOT : KVQ_DEVERR_PAGE);
                    // a token that is not there has the pool's first row, which always exists
                    const uint32_t page = !g ? 0 : kSlots ? uint32_t(idx[j] >> a.page_bits) : uint32_t(idx[j]);
                    const uint32_t r = !g ? 0 : (kSlots ? uint32_t(idx[j]) : uint32_t(t)) & in_page;
                    const uint8_t *p = a.pool + uint64_t(page) * page_bytes;
                    good |= uint32_t(g) << j;
                    row[j] = p + r * T::kCodeBytes;
                    sc[j] = __ldg(reinterpret_cast<const uint4 *>(p + (scale_at + r * T::kScaleBytes)));
#pragma unroll
                    for (int z = 0; z < T::kCodeBytes; z += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row[j] + z));
                }
                if (i > 0) {  // the next block's indexes, while the scales come
                    cur.next(a);
                    fetch();
                }
                // wait until the entries are free (every reader of block i - kLookups is done); as the other waits, it
                // gives up once and for all
                const int need = i - (kLookups - 1 - (R + kChunks - 1) / kChunks);
                for (uint32_t n = tries; progress < need; --n) {
                    if (n == 0) {
                        tries = 0;
                        break;
                    }
                    __nanosleep(64);
                }
                const int k = i % kLookups;
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    sh.scale[k][mine + 32 * j] = sc[j];
                    sh.code[k][mine + 32 * j] = row[j];
                    sh.texp[k][mine + 32 * j] = (good >> j) & 1 ? row_texp<L>(sc[j]) : kNoToken;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.addr[k]));
                if (i == 0) {  // the first block has gone out first
                    cur.next(a);
                    fetch();
                }
            }
            if (!tries) sh.abort = 1;
        }
        done_arrive();
    } else {
        // ------------------------------------------------------ softmax, queries, outputs
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // A warp has 16 tokens (those of its TMEM lane quarter) and NC columns (query rows) from c0; a thread of it the
        // tokens tok and tok + 8 and of every eight columns two, 8 g + 2 (lane % 4) + {0, 1}.
        constexpr int NC = N / 2, G = NC / 8;
        const int quarter = warp & 3, half = warp >> 2, c0 = half * NC, tok = 16 * quarter + (lane >> 2);
        const int col0 = c0 + 2 * (lane & 3);
        const int t_row = tid & 127;  // lane of the outputs: a dim of 128
        const float c = a.scale * kLog2e;
        const int per = a.q_len * a.heads;
        const uint32_t trow = (uint32_t(quarter * 32) << 16);
        Cursor<N, kKind> cur(a, sh);
        Ring<R> ring;
        float l[G][2], sc[G][2], nm[G][2];
        Ring<R> end;  // the slot of the block's last chunk
        bool unset = false;
        uint32_t tries = a.wait_tries;
        int kb0 = 0;
        float room = 0.f;
        // where a part's sums go that another CTA goes on with or began, or that are too long for TMEM
        auto part_of = [&](int kb0) { return a.part + (2 * int64_t(blockIdx.x) + (kb0 == 0 ? 1 : 0)) * N * kPartRow; };
#pragma unroll 1
        for (int i = 0; i < units; ++i, cur.next(a)) {
            const bool first = i == 0 || cur.kb == 0;
            if (first) {
                // the scores' products of the last tile are done (their result was waited for)
                kb0 = cur.kb;
                if (tid == 0 && cur.kb == 0 && cur.t.rt == 0 && cur.t.err) raise_err(a.err, cur.t.err);
                room = headroom(min(cur.left, cur.t.nb - cur.kb));
                if (tid < N) {
                    const int row = cur.t.rt * N + tid, rc = min(row, per - 1);
                    const int j = rc / a.heads, head = rc - j * a.heads;
                    const int64_t tok = int64_t(cur.t.seq) * a.q_len + j;
                    sh.q[tid] = row < per ? tok * a.q_tok + head * a.q_head : -1;
                    sh.row[tid] = row < per ? tok * a.out_tok + head * a.out_head : -1;
                    if constexpr (!kTree) sh.vis[tid] = kSlots || row >= per ? cur.t.seen : max(0, cur.t.len - (a.q_len - 1 - j));
                    sh.m[tid] = -INFINITY;
                    sh.nm[tid] = 0.f;
                }
                soft_sync();
                const uint32_t sq = smem_addr(sQ);
                constexpr int kBatch = N / kSoftWarps < 4 ? N / kSoftWarps : 4;  // rows whose loads are in flight
#pragma unroll 1
                for (int r0 = warp; r0 < N; r0 += kBatch * kSoftWarps) {
                    uint32_t v[kBatch][8];
#pragma unroll
                    for (int t = 0; t < kBatch; ++t) {
                        const int64_t at = sh.q[r0 + t * kSoftWarps];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint4 u = make_uint4(0u, 0u, 0u, 0u);
                            if (at >= 0) u = ld_stream_u4(a.q + at + (lane + 32 * h) * 8);
                            v[t][4 * h] = u.x, v[t][4 * h + 1] = u.y, v[t][4 * h + 2] = u.z, v[t][4 * h + 3] = u.w;
                        }
                    }
#pragma unroll
                    for (int t = 0; t < kBatch; ++t) {
                        const int r = r0 + t * kSoftWarps;
                        // fp16: the row times a power of two that brings its largest magnitude to [2^14, 2^15)
                        uint32_t big = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) big = max(big, max((v[t][e] << 16) & 0x7FFF0000u, v[t][e] & 0x7FFF0000u));
                        big = __reduce_max_sync(0xFFFFFFFFu, big);
                        const uint32_t up = min(268u - (big >> 23), 254u);
                        const float f = __uint_as_float(up << 23);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            uint32_t h;
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(bf16_hi(v[t][e]) * f), "f"(bf16_lo(v[t][e]) * f));
                            sts_u32(sq + q_word<N>(r, lane + 32 * (e >> 2), e & 3), h);
                        }
                        if (lane == 0) sh.sc[r] = score_factor<L>(c, up);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.qready));
                soft_sync();
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        l[g][e] = nm[g][e] = 0.f;
                        sc[g][e] = sh.sc[col0 + 8 * g + e];
                    }
                unset = true;
            }
            // Weights below 2^-24 of a thread's sum add nothing to it, however many they are, so the sum starts afresh
            // every kFoldBlocks blocks.
            const int since = cur.kb - kb0;  // blocks of this part so far
            if (__builtin_expect((since & (kFoldBlocks - 1)) == 0 && since > 0, 0)) {
                asm volatile("");
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = rows_sum(l[g][e]);
                        if (since > kFoldBlocks) v += sh.lsum[quarter][col0 + 8 * g + e];
                        if (lane < 4) sh.lsum[quarter][col0 + 8 * g + e] = v;
                        l[g][e] = 0.f;
                    }
                if ((since & (kFoldOut - 1)) == 0) {
                    mbar_wait(smem_addr(&sh.oblk[end.slot]), end.parity, tries);
                    tc_fence_after();
#pragma unroll 1
                    for (int b = 2 * half; b < 2 * half + 2; ++b)
#pragma unroll 1
                        for (int j0 = 0; j0 < N; j0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(trow + b * N + j0, o);
                            float *to = part_of(kb0) + j0 * kPartRow + b * kChunk + t_row;
#pragma unroll
                            for (int j = 0; j < 16; ++j, to += kPartRow)
                                *to = since > kFoldOut ? *to + __uint_as_float(o[j]) : __uint_as_float(o[j]);
                        }
                }
            }
            // whether the block holds drafted tokens, and which of them each row sees (a row of no one's: all, so that it
            // has a maximum).  The block before's windows were read before its last barrier.
            const int base = kTree ? cur.t.len - a.q_len : 0;
            const bool of_tree = kTree && (cur.kb + 1) * kTile > base;
            if (of_tree) {
                if (tid < N) {
                    const int row = cur.t.rt * N + tid, j = row / a.heads;
                    const uint64_t w = row < per ? tree_window(a.mask + (int64_t(cur.t.seq) * a.q_len + j) * a.mask_words,
                                                               a.mask_words, cur.kb * kTile, base)
                                                 : ~0ull;
                    sh.win[tid][0] = uint32_t(w);
                    sh.win[tid][1] = uint32_t(w >> 32);
                }
                soft_sync();
            }
            // `full` of the block's first chunk orders this thread's read of texp
            mbar_wait(smem_addr(&sh.full[ring.slot]), ring.parity, tries);
            int t_at[2];
            float up[2] = {1.f, 1.f}, et[2] = {0.f, 0.f}, lift[2] = {0.f, 0.f};
            bool have = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int te = sh.texp[i % kLookups][tok + 8 * h];
                const bool there = te != kNoToken;
                have = have && there;
                t_at[h] = there ? cur.kb * kTile + tok + 8 * h : 0x7FFFFFFF;
                if constexpr (kExp) {
                    et[h] = there ? float(te) : 0.f;
                    up[h] = there ? __uint_as_float(uint32_t(127 + te - kLift) << 23) : 1.f;
                    lift[h] = there ? float(kLift - te) : 0.f;
                }
            }
            // whether some of the block is masked for some row (the first row of a tile sees least)
            const bool masked = !__all_sync(0xFFFFFFFFu, have) || (kTree ? of_tree : int64_t(cur.kb + 1) * kTile > sh.vis[0]);
            mbar_wait(smem_addr(&sh.sdone[i & 1]), (i >> 1) & 1, tries);
            tc_fence_after();
            // x = score in log2 units, plus the row's power of two; -inf where it is masked.  [.][h][e]: token tok + 8 h.
            float x[G][2][2];
            tmem_ld_rows<G>(trow + kTmemS + (kBufs == 2 ? (i & 1) * N : 0) + c0, x);
            tc_fence_before();
            if (lane == 0) mbar_arrive(smem_addr(&sh.sread[i & 1]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float2 u = make_float2(x[g][h][0], x[g][h][1]);
                    const float2 k = make_float2(sc[g][0], sc[g][1]);
                    if constexpr (kExp) u = ffma2(fmul2(u, make_float2(up[h], up[h])), k, make_float2(et[h], et[h]));
                    else u = fmul2(u, k);
                    x[g][h][0] = u.x, x[g][h][1] = u.y;
                }
            }
            bool odd[2] = {false, false};  // a score that is not finite, where some rows do not see the token
            if (masked) {
                asm volatile("");  // a branch, not selects in every block
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // of a tree: the half of the row's window that this warp's 16 tokens lie in
                        const uint32_t win = !kTree ? 0u : of_tree ? sh.win[col0 + 8 * g + e][quarter >> 1] : 0xFFFFFFFFu;
                        const int vis = kTree ? 0 : sh.vis[col0 + 8 * g + e];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            odd[h] = odd[h] || !(fabsf(x[g][h][e]) < INFINITY);
                            const bool sees = kTree ? t_at[h] != 0x7FFFFFFF && ((win >> ((tok + 8 * h) & 31)) & 1) : t_at[h] < vis;
                            if (!sees) x[g][h][e] = -INFINITY;
                        }
                    }
            }
            // The weights 2^(x - maximum), which go to shared memory as fp16; returns the largest exponent.
            float p[G][2][2];
            const uint32_t sp = smem_addr(sP) + (i & 1) * kTile * N * 2 + 4 * (lane & 3);
            auto weights = [&]() {
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 u = fadd2(make_float2(x[g][h][0], x[g][h][1]), make_float2(nm[g][0], nm[g][1]));
                        top = fmax3(top, u.x, u.y);
                        const float2 at = kExp ? fadd2(u, make_float2(lift[h], lift[h])) : u;
                        p[g][h][0] = ex2_approx(at.x), p[g][h][1] = ex2_approx(at.y);
                        float2 o = make_float2(p[g][h][0], p[g][h][1]);
                        if constexpr (kExp) o = fmul2(o, make_float2(up[h], up[h]));
                        uint32_t w;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(o.y), "f"(o.x));
                        sts_u32(sp + p_vec<N>(tok + 8 * h, c0 / 8 + g), w);
                    }
                return top;
            };
            bool move = unset;
            if (!unset) move = soft_any(weights() > kStaleMax);
            if (move) {
                // the columns' new maxima, and what is summed so far in their terms
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float v = rows_max(fmaxf(x[g][0][e], x[g][1][e]));
                        if (lane < 4) sh.red[quarter][col0 + 8 * g + e] = v;
                    }
                soft_sync();
                bool none = false;
                if (tid < N) {
                    const float m0 = sh.m[tid];
                    const float top = fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid]));
                    const float m1 = fmaxf(top - room, m0);
                    none = m1 == -INFINITY;
                    sh.m[tid] = m1;
                    sh.nm[tid] = none ? 0.f : -m1;
                    sh.alpha[tid] = none ? 1.f : ex2_approx(0.5f * (m0 - m1));  // twice, as the whole can pass fp32
                }
                unset = soft_any(none);
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float alpha = sh.alpha[col0 + 8 * g + e];
                        l[g][e] = l[g][e] * alpha * alpha;
                        if (since >= kFoldBlocks && lane < 4) sh.lsum[quarter][col0 + 8 * g + e] *= alpha * alpha;
                        nm[g][e] = sh.nm[col0 + 8 * g + e];
                    }
                if (!first) {
                    // the outputs so far: the last block's must be in (`end` is still its last chunk)
                    mbar_wait(smem_addr(&sh.oblk[end.slot]), end.parity, tries);
                    tc_fence_after();
#pragma unroll 1
                    for (int b = 2 * half; b < 2 * half + 2; ++b)
#pragma unroll 1
                        for (int j0 = 0; j0 < N; j0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(trow + b * N + j0, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sh.alpha[j0 + j] * sh.alpha[j0 + j]);
                            tmem_st16(trow + b * N + j0, o);
                        }
                    tc_wait_st();
                    if (since >= kFoldOut) {
#pragma unroll 1
                        for (int j = 0; j < N; ++j) {
                            float *to = part_of(kb0) + j * kPartRow + 2 * half * kChunk + t_row;
                            to[0] = to[0] * sh.alpha[j] * sh.alpha[j];
                            to[kChunk] = to[kChunk] * sh.alpha[j] * sh.alpha[j];
                        }
                    }
                }
                weights();
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float2 sum = make_float2(l[g][0], l[g][1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) sum = fadd2(sum, make_float2(p[g][h][0], p[g][h][1]));
                l[g][0] = sum.x, l[g][1] = sum.y;
            }
            if (masked && half == 0) {
                // A weight of 0 does not silence a NaN: if a token's row itself is not finite, the rows that see it are
                // NaN by their weights already, and the others must meet zeros.  (Such a row's scores are odd in every
                // column, so each of its four lanes knows; one of them looks.)
                for (int h = 0; h < 2; ++h) {
                    if (!odd[h] || t_at[h] == 0x7FFFFFFF || (lane & 3) != 0) continue;
                    bool bad = false;
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {
                        Ring<R> at = ring;
#pragma unroll 1
                        for (int v = 0; v < 64 && (pass == 0 || bad); ++v) {
                            const uint32_t where = smem_addr(sK) + at.slot * kChunkSmem + ((v >> 3) & 1) * kSubBytes +
                                                   (tok + 8 * h) * 128 + (v & 7) * 16;
                            if (pass == 0) {
                                const uint4 u = lds_u4(where);
                                const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
                                for (int e = 0; e < 4; ++e)
                                    bad = bad || (ws[e] & 0x7C00u) == 0x7C00u || (ws[e] & 0x7C000000u) == 0x7C000000u;
                            } else {
                                const uint32_t z[4] = {0u, 0u, 0u, 0u};
                                sts_u4(where, z);
                            }
                            if ((v & 15) == 15) at.next();
                        }
                    }
                }
            }
            tc_fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.pready[i & 1]));
            // the ring moves on by a block; the last chunk's slot tells when the block's outputs are summed
            for (int b = 0; b < kChunks; ++b) {
                end = ring;
                ring.next();
            }

            if (i + 1 == units || cur.kb + 1 == cur.t.nb) {
                // ---- this CTA's part of the tile is done
                const bool whole = kb0 == 0 && cur.kb + 1 == cur.t.nb;
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = rows_sum(l[g][e]);
                        if (since >= kFoldBlocks) v += sh.lsum[quarter][col0 + 8 * g + e];
                        if (lane < 4) sh.lsum[quarter][col0 + 8 * g + e] = v;
                        l[g][e] = 0.f;  // (without this the chunk takes 787 instead of 740 us)
                    }
                soft_sync();
                float *const part = part_of(kb0);
                if (tid < N) {
                    const float sum = ((sh.lsum[0][tid] + sh.lsum[1][tid]) + (sh.lsum[2][tid] + sh.lsum[3][tid])) *
                                      (kExp ? 1.f / float(int64_t(1) << kLift) : 1.f);
                    const float m = sh.m[tid];
                    sh.inv[tid] = whole ? (m == -INFINITY && sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                    const int row = cur.t.rt * N + tid;
                    if (!whole) {
                        part[tid * kPartRow + kD] = m;
                        part[tid * kPartRow + kD + 1] = sum;
                    } else if (a.lse && row < per) {
                        a.lse[int64_t(cur.t.seq) * per + row] = attend_lse(m, sum);
                    }
                }
                if (tid == 0 && i + 1 == units) {
                    int2 join = make_int2(-1, 0);
                    if (kb0 == 0 && !whole) {  // later CTAs hold the rest of this tile
                        const int64_t end_unit = sh.u0 + units - 1 + (cur.t.nb - 1 - cur.kb) + int64_t(kCost) * (cur.tile + 1);
                        const int64_t g = min(int64_t(gridDim.x), sh.total);
                        join = make_int2(cur.tile, int(((end_unit + 1) * g - 1) / sh.total));
                    }
                    a.join[blockIdx.x] = join;
                }
                soft_sync();
                mbar_wait(smem_addr(&sh.oblk[end.slot]), end.parity, tries);
                tc_fence_after();
                if (__builtin_expect(since >= kFoldOut, 0)) {
#pragma unroll 1
                    for (int b = 2 * half; b < 2 * half + 2; ++b)
#pragma unroll 1
                        for (int j0 = 0; j0 < N; j0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(trow + b * N + j0, o);
                            const float *from = part + j0 * kPartRow + b * kChunk + t_row;
#pragma unroll
                            for (int j = 0; j < 16; ++j, from += kPartRow) o[j] = __float_as_uint(__uint_as_float(o[j]) + *from);
                            tmem_st16(trow + b * N + j0, o);
                        }
                    tc_wait_st();
                }
                if (__all_sync(0xFFFFFFFFu, tries != 0)) {  // for the warp: loads of TMEM and shuffles follow
#pragma unroll 1
                    for (int b = 2 * half; b < 2 * half + 2; ++b) {
                        const int d = b * kChunk + t_row;
#pragma unroll 1
                        for (int j0 = 0; j0 < N; j0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(trow + b * N + j0, o);
                            if (!whole) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) part[(j0 + j) * kPartRow + d] = __uint_as_float(o[j]);
                            } else if (a.out_bf16) {
                                // neighbouring lanes swap columns, so that a store is two dims of one row
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    const float u = __uint_as_float(o[j]) * sh.inv[j0 + j];
                                    const float v = __uint_as_float(o[j + 1]) * sh.inv[j0 + j + 1];
                                    const float z = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? u : v, 1);
                                    const int64_t row = sh.row[j0 + j + (lane & 1)];
                                    const uint32_t two = (lane & 1) ? pack_bf16x2(z, v) : pack_bf16x2(u, z);
                                    if (row >= 0)
                                        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + row + (d & ~1)) = two;
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const int64_t row = sh.row[j0 + j];
                                    if (row >= 0) static_cast<float *>(a.out)[row + d] = __uint_as_float(o[j]) * sh.inv[j0 + j];
                                }
                            }
                        }
                    }
                }
                tc_fence_before();
                soft_sync();  // the tile's arrays are free for the next one
            }
        }
        if (!tries) sh.abort = 1;
        done_sync();
        if (*const_cast<volatile int *>(&sh.abort)) {  // the same for every thread
            // A wait gave up: the rows that this CTA worked on are NaN, at once or by way of the join.
            if (tid == 0) raise_err(a.err, KVQ_DEVERR_WAIT);
            int tile = sh.start_tile, kb = sh.start_kb;
#pragma unroll 1
            for (int left = units; left > 0; ++tile, kb = 0) {
                const TileInfo t = tile_info<N, kKind>(a, tile);
                const int blocks = min(left, t.nb - kb);
                left -= blocks;
                if (blocks < t.nb) {
                    if (tid < N) *reinterpret_cast<float2 *>(part_of(kb) + tid * kPartRow + kD) = make_float2(NAN, NAN);
                    continue;
                }
#pragma unroll 1
                for (int r = warp; r < N && t.rt * N + r < per; r += kSoftWarps) {
                    const int row = t.rt * N + r, j = row / a.heads;
                    const int64_t to = (int64_t(t.seq) * a.q_len + j) * a.out_tok + (row - j * a.heads) * a.out_head;
                    for (int d = lane; d < kD; d += 32) {
                        if (a.out_bf16) static_cast<uint16_t *>(a.out)[to + d] = 0x7FFF;
                        else static_cast<float *>(a.out)[to + d] = NAN;
                    }
                    if (a.lse && lane == 0) a.lse[int64_t(t.seq) * per + row] = NAN;
                }
            }
        }
    }
    __syncwarp();
    if (tid == 0) pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(sh.tmem, kTmemCols);
}

// Joins the tiles that CTAs split.  Every CTA lists the `ctas` shares' split
// tiles, and the warps of the grid go round (tile, query row, quarter of the
// dims): a warp adds the parts of 128 dims in order, each weighted by 2^(its
// maximum - the largest so far), with eight parts' loads in flight.  Of that
// weight the root is applied twice: a V41 part's maximum contains its rows'
// powers of two, and two of them may differ by more than fp32 holds.
constexpr int kJoinThreads = 512, kJoinBatch = 8;

template <int N>
__global__ void __launch_bounds__(kJoinThreads, 2) attend_join_kernel(const __grid_constant__ AttendArgs a, int ctas) {
    __shared__ int3 split[kMaxAttendCtas];  // first CTA, its tile, last CTA
    __shared__ int counts[kJoinThreads / 32];
    static_assert(kMaxAttendCtas <= kJoinThreads, "a thread a share");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    const int2 join = tid < ctas ? a.join[tid] : make_int2(-1, 0);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, join.x >= 0);
    if (lane == 0) counts[warp] = __popc(some);
    __syncthreads();
    int before = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        if (w < warp) before += counts[w];
        n += counts[w];
    }
    if (join.x >= 0) split[before + __popc(some & ((1u << lane) - 1))] = make_int3(tid, join.x, join.y);
    __syncthreads();
    const int per = a.q_len * a.heads;
    const int warps = gridDim.x * (kJoinThreads / 32);
    for (int item = blockIdx.x * (kJoinThreads / 32) + warp; item < n * N * 4; item += warps) {
        const int3 s = split[item / (4 * N)];
        const int r = item / 4 % N, d = item % 4 * 128 + 4 * lane;
        const int seq = s.y / a.row_tiles, row = s.y % a.row_tiles * N + r;
        if (row >= per) continue;
        const int parts = s.z - s.x + 1;
        auto at = [&](int i) {
            return a.part + ((i == 0 ? 2 * int64_t(s.x) + 1 : 2 * (int64_t(s.x) + i)) * N + r) * kPartRow;
        };
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < parts; i0 += kJoinBatch) {
            float2 ml[kJoinBatch];
            float4 v[kJoinBatch];
            float to = top;
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + k < parts) {
                    ml[k] = __ldg(reinterpret_cast<const float2 *>(at(i0 + k) + kD));
                    v[k] = __ldg(reinterpret_cast<const float4 *>(at(i0 + k) + d));
                }
            }
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) to = fmaxf(to, ml[k].x);
            const float zero = to == -INFINITY ? 0.f : to;
            const float keep = ex2_approx(0.5f * (top - zero)), keep2 = keep * keep;   // of nothing: 0
            acc.x *= keep2, acc.y *= keep2, acc.z *= keep2, acc.w *= keep2, sum = sum * keep * keep;
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                const float root = ex2_approx(0.5f * (ml[k].x - zero)), w = root * root;
                sum = fmaf(root, root * ml[k].y, sum);
                acc.x = fmaf(w, v[k].x, acc.x), acc.y = fmaf(w, v[k].y, acc.y);
                acc.z = fmaf(w, v[k].z, acc.z), acc.w = fmaf(w, v[k].w, acc.w);
            }
            top = to;
        }
        const float inv = top == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
        const int j = row / a.heads;
        const int64_t to = (int64_t(seq) * a.q_len + j) * a.out_tok + (row - j * a.heads) * a.out_head + d;
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        if (a.out_bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to) = acc;
        if (a.lse && item % 4 == 0 && lane == 0) a.lse[int64_t(seq) * per + row] = attend_lse(top, sum);
    }
}

template <Layout L, int N, int kKind>
kvq_status launch_attend_n(AttendArgs a, cudaStream_t s) {
    const int64_t per = int64_t(a.q_len) * a.heads;
    a.row_tiles = int((per + N - 1) / N);
    const int64_t tiles = a.n_seq * a.row_tiles;
    int64_t grid = 0;
    kvq_status st = resident_grid<attend_kernel<L, N, kKind>, kAttendThreads>(kAttendSmem<N>, &grid);
    if (st != KVQ_OK) return st;
    if (grid > kMaxAttendCtas) grid = kMaxAttendCtas;
    const int64_t most = (a.max_len + kTile - 1) / kTile;  // blocks of the longest tile there can be
    if (tiles > 0x7FFFFFFF || per > 0x7FFFFFFF || tiles * (most ? most : 1) / grid >= 0x7FFFFFFF / kChunks)
        return KVQ_ERR_UNSUPPORTED;
    if (most <= 1 && tiles < grid) grid = tiles;
    a.join = reinterpret_cast<int2 *>(a.ws);
    a.part = reinterpret_cast<float *>(a.ws + kMaxAttendCtas * sizeof(int2));
    st = launch_pdl_smem(attend_kernel<L, N, kKind>, dim3(unsigned(grid)), dim3(kAttendThreads), kAttendSmem<N>, s, a);
    if (st != KVQ_OK || most <= 1) return st;  // a tile of one block is never split
    return launch_pdl(attend_join_kernel<N>, dim3(unsigned(2 * grid)), dim3(kJoinThreads), s, a, int(grid));
}

template <Layout L, int kKind>
kvq_status launch_attend_layout(const AttendArgs &a, cudaStream_t s) {
    switch (attend_rows(int64_t(a.q_len) * a.heads)) {
        case 16: return launch_attend_n<L, 16, kKind>(a, s);
        case 32: return launch_attend_n<L, 32, kKind>(a, s);
        default: return launch_attend_n<L, 64, kKind>(a, s);
    }
}

}  // namespace
}  // namespace kvq
