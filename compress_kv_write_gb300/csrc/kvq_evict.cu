// kvq_evict.cu -- eviction from the paged cache by accumulated attention
// weight: which tokens of a sequence stay (kvq_evict_select), and their rows
// moved, in order, to pages of their own (kvq_evict_move).
#include "kvq_launch.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------- selection
// Of n tokens the first and last few stay anyway; of those between, the m of
// most weight, among equals the ones that come first.  A weight becomes a
// 32-bit key of the same order, and the m-th largest key is found digit by
// digit from the top (11, 11 and 10 bits): a histogram of the digit over the
// keys that share the digits found so far, and the bin in which the count from
// the top reaches m.  A bin all of whose keys stay ends the search.  Then every
// token's fate is known from its key, but for those equal to the m-th: of these
// the first ones stay.
//
// A sequence is a CTA's, or with many tokens a cluster's: its CTAs have equal
// pieces of it in order, and their warps equal pieces of those.  A thread holds
// 8 or 16 keys in registers (one pass over global memory); what a cluster of
// eight cannot hold that way is in shared memory or read again.  CTAs add their
// filled bins to the first one's and read back what it found.  Places in the
// output come from counts: of the CTAs before, of the warps before, and of the
// lanes before by ballot.
//
// Bound by latency and by the instructions a key takes in one or a few SMs:
// some five a round.  (Keys in shared memory and ballots to add up equal bins,
// which the hardware's counting increments do by themselves, took 60 a round.)
// One sequence of 4,097 tokens 5.9 us, 32 of up to 24,577 10.7, one of 131,072
// 15.4 to 17; by way of shared memory one of 400,000 51, a million 114.
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSelKeys = 52224;  // keys that a CTA can hold in shared memory (204 KB)

struct SelectArgs {
    const float *mass;
    int64_t stride;
    const int32_t *rows;
    int64_t n_rows;
    int64_t width;  // tokens a row of weights has
    const int32_t *kv_len;
    int32_t *kept;
    int64_t kept_stride;
    int keep, first, last;
    int32_t *count;
    int32_t *err;
    int held;  // keys that a CTA holds in shared memory
};

// Larger weight, larger key; zeros are equal, a NaN is above everything.
__device__ __forceinline__ uint32_t mass_key(float m) {
    const uint32_t b = __float_as_uint(m);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    if (b == 0x80000000u) return 0x80000000u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Adds to a 32-bit word at a shared-window address of this CTA, in another CTA of the cluster.
__device__ __forceinline__ void adds_of(uint32_t addr, uint32_t rank, uint32_t v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
// Such a word's value.
__device__ __forceinline__ uint32_t lds_of(uint32_t addr, uint32_t rank) {
    uint32_t at, r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}

struct SelShared {
    uint32_t hist[2][kBins];  // by turns, so that a CTA may be counting while the first one still reads
    uint32_t warp[2][kSelWarps];
    uint32_t gt, eq;          // this CTA's tokens above the m-th key, and equal to it
    uint32_t bin, above, in;  // the bin that was found, the keys above it and in it
};

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// kRegs keys a thread in registers; 0: keys in shared memory, or read again.
template <int kRegs>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectArgs a, int cluster) {
    extern __shared__ uint8_t smem[];
    auto &sh = *reinterpret_cast<SelShared *>(smem);
    uint32_t *const held = reinterpret_cast<uint32_t *>(smem + sizeof(SelShared));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int seq = int(blockIdx.x) / cluster;
    const int rank = cluster > 1 ? int(cluster_rank()) : 0;
    auto sync_all = [&]() {
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    };
    for (int i = tid; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    pdl_wait();
    int64_t n = __ldg(a.kv_len + seq);
    int64_t row = a.rows ? __ldg(a.rows + seq) : seq;
    int bits = 0;
    if (row < 0 || row >= a.n_rows) bits = KVQ_DEVERR_STATE;
    else if (n < 0 || n > a.width) bits = KVQ_DEVERR_LEN;
    if (bits) {
        n = 0;
        row = 0;
        if (tid == 0 && rank == 0) raise_err(a.err, bits);
    }
    int32_t *const out = a.kept + seq * a.kept_stride;
    const bool all = n <= a.keep;
    const int m = a.keep - a.first - a.last;

    // this CTA's piece of the tokens between, and this warp's: a multiple of 32 tokens from w0 on
    const int between = all || m == 0 ? 0 : int(n) - a.first - a.last;
    const int per = (between + cluster - 1) / cluster;
    const int t0 = min(between, rank * per), mine = min(between, t0 + per) - t0;
    const float *const from = a.mass + row * a.stride + a.first + t0;
    const int steps = (mine + kSelThreads - 1) / kSelThreads, w0 = warp * steps * 32;
    const int in_smem = kRegs ? 0 : min(mine, a.held);
    uint32_t keys[kRegs ? kRegs : 1];
    if constexpr (kRegs > 0) {
        float v[kRegs];
#pragma unroll
        for (int j = 0; j < kRegs; ++j) {
            const int i = w0 + j * 32 + lane;
            v[j] = j < steps && i < mine ? __ldg(from + i) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kRegs; ++j) keys[j] = j < steps && w0 + j * 32 + lane < mine ? mass_key(v[j]) : 0u;
    } else {
#pragma unroll 8
        for (int i = tid; i < in_smem; i += kSelThreads) held[i] = mass_key(__ldg(from + i));
    }
    pdl_trigger();

    // what does not depend on the weights: the first and the last, or all, and the entries of no token
    const int count = int(min(n, int64_t(a.keep)));
    for (int k = rank * kSelThreads + tid; k < a.keep; k += cluster * kSelThreads) {
        if (all) out[k] = k < count ? k : -1;
        else if (k < a.first) out[k] = k;
        else if (k >= a.keep - a.last) out[k] = int(n) - (a.keep - k);
    }
    if (rank == 0 && tid == 0) a.count[seq] = count;
    if (between == 0) return;  // the same for the whole cluster
    sync_all();  // bins are clear, keys are there

    // The warp's tokens in order, 32 at a time: f(token, key), key 0 (lower than any weight's) for none.
    auto for_each = [&](auto &&f) {
        if constexpr (kRegs > 0) {
#pragma unroll
            for (int j = 0; j < kRegs; ++j)
                if (j < steps) f(w0 + j * 32 + lane, keys[j]);
        } else {
            constexpr int kBatch = 16;  // loads under way
#pragma unroll 1
            for (int j0 = 0; j0 < steps; j0 += kBatch) {
                uint32_t k[kBatch];
                if (w0 + j0 * 32 >= in_smem) {
                    float v[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) v[b] = __ldg(from + min(w0 + (j0 + b) * 32 + lane, mine - 1));
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) k[b] = w0 + (j0 + b) * 32 + lane < mine ? mass_key(v[b]) : 0u;
                } else {
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int i = w0 + (j0 + b) * 32 + lane;
                        k[b] = i >= mine ? 0u : i < in_smem ? held[i] : mass_key(__ldg(from + i));
                    }
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (j0 + b < steps) f(w0 + (j0 + b) * 32 + lane, k[b]);
            }
        }
    };

    // the m-th largest key, from the top: `prefix` its digits so far, `left` how many of the keys with these digits stay
    uint32_t prefix = 0, left = uint32_t(m);
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, digit = round == 2 ? 1024 : 2048;
        uint32_t *const hist = sh.hist[round & 1];
        const uint32_t same = round == 0 ? 0u : 0xFFFFFFFFu << (round == 1 ? 21 : 10);
        for_each([&](int, uint32_t k) {
            if (k && ((k ^ prefix) & same) == 0) atomicAdd(&hist[(k >> shift) & (digit - 1)], 1u);
        });
        __syncthreads();
        // thread t has bins digit - 1 - 2 t and the one below (from the top)
        const int top = digit - 1 - 2 * tid;
        uint32_t c0 = top > 0 ? hist[top] : 0, c1 = top > 0 ? hist[top - 1] : 0;
        if (cluster > 1) {
            if (rank > 0) {
                if (c0) adds_of(smem_addr(hist + top), 0, c0);
                if (c1) adds_of(smem_addr(hist + top - 1), 0, c1);
            }
            cluster_sync();
            if (rank == 0 && top > 0) c0 = hist[top], c1 = hist[top - 1];
        }
        if (rank == 0) {
            const uint32_t of_warp = __reduce_add_sync(0xFFFFFFFFu, c0 + c1);
            if (lane == 0) sh.warp[0][warp] = of_warp;
            __syncthreads();
            const uint32_t upto = warp_scan(sh.warp[0][lane]);
            const uint32_t here = __shfl_sync(0xFFFFFFFFu, upto, warp), before_warp = here - of_warp;
            if (before_warp < left && here >= left) {  // one warp has the bin
                const uint32_t before = before_warp + warp_scan(c0 + c1) - c0 - c1;
                if (before < left && before + c0 >= left) sh.bin = top, sh.above = before, sh.in = c0;
                else if (before + c0 < left && before + c0 + c1 >= left) sh.bin = top - 1, sh.above = before + c0, sh.in = c1;
            }
        }
        sync_all();
        if (round == 0)  // for the third round; the first CTA's was read until here
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        const uint32_t bin = cluster > 1 ? lds_of(smem_addr(&sh.bin), 0) : sh.bin;
        const uint32_t above = cluster > 1 ? lds_of(smem_addr(&sh.above), 0) : sh.above;
        const uint32_t in = cluster > 1 ? lds_of(smem_addr(&sh.in), 0) : sh.in;
        prefix |= bin << shift;
        left -= above;
        if (in == left) {  // all of them stay: they are above a key of their lowest, less one (no key is that low)
            prefix -= 1;
            left = 0;
            break;
        }
    }

    // counts of what is above and equal, of the warps and of the CTAs before
    uint32_t gt = 0, eq = 0;
    for_each([&](int, uint32_t k) {
        gt += k > prefix;
        eq += k == prefix;
    });
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    __syncthreads();
    if (lane == 0) sh.warp[0][warp] = gt, sh.warp[1][warp] = eq;
    __syncthreads();
    const uint32_t gt_upto = warp_scan(sh.warp[0][lane]), eq_upto = warp_scan(sh.warp[1][lane]);
    uint32_t gt_before = __shfl_sync(0xFFFFFFFFu, gt_upto, warp) - gt, eq_before = __shfl_sync(0xFFFFFFFFu, eq_upto, warp) - eq;
    if (cluster > 1) {
        if (tid == 31) {
            sh.gt = gt_upto;
            sh.eq = eq_upto;
        }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            gt_before += lds_of(smem_addr(&sh.gt), r);
            eq_before += lds_of(smem_addr(&sh.eq), r);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA's memory may still be read
    }
    for_each([&](int i, uint32_t k) {
        const uint32_t g = __ballot_sync(0xFFFFFFFFu, k > prefix), e = __ballot_sync(0xFFFFFFFFu, k == prefix);
        const uint32_t low = (1u << lane) - 1;
        const uint32_t gb = gt_before + __popc(g & low), eb = eq_before + __popc(e & low);
        if (k > prefix || (k == prefix && eb < left)) out[a.first + gb + min(eb, left)] = a.first + t0 + i;
        gt_before += __popc(g);
        eq_before += __popc(e);
    });
    if (cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int kRegs>
kvq_status launch_select(SelectArgs a, int64_t n_seq, int cluster, cudaStream_t s) {
    const int64_t per = (a.width + cluster - 1) / cluster;
    a.held = kRegs ? 0 : int(per < kSelKeys ? per : kSelKeys);
    int64_t cap = 0;
    kvq_status st = resident_grid<evict_select_kernel<kRegs>, kSelThreads>(sizeof(SelShared) + (kRegs ? 0 : kSelKeys * 4), &cap);
    if (st != KVQ_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n_seq * cluster));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = sizeof(SelShared) + size_t(a.held) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel<kRegs>, a, cluster) != cudaSuccess) {
        (void)cudaGetLastError();
        return KVQ_ERR_LAUNCH;
    }
    return KVQ_OK;
}

// ---------------------------------------------------------------- the move
// Row kept[i][k] of sequence i becomes row k of its new pages: codes and scale
// bytes as they are.  A warp has 8 (V41) or 16 (V41_FP4) tokens: as many lanes
// look up where these lie and shall lie, then all rows' loads (8 a lane) are
// under way before the first store.  Bound by memory: rows of 256 or 512 bytes,
// read and written once: 224 MB of V41 rows in 38 us = 5.9 TB/s (with 4 tokens a
// warp 39.8, with more warps an SM 40.0), 2,048 V41_FP4 rows in 3.0 (2.5).
constexpr int kMoveThreads = 256;
template <Layout L>
constexpr int kMoveTok = L == Layout::V41 ? 8 : 16;

struct MoveArgs {
    uint8_t *pool;
    int64_t pages;
    int page_bits;
    const int32_t *table, *to_table;
    int64_t table_rows, table_stride, to_stride;
    int64_t max_len;  // tokens that a row of the table, and of the weights, has
    const int32_t *req;
    const int32_t *kept;
    int64_t kept_stride;
    int keep;
    int64_t groups;  // warps a sequence
    int64_t total;   // groups
    const float *mass;
    int64_t mass_stride;
    const int32_t *rows;
    int64_t n_rows;
    float *mass_out;
    int64_t mass_out_stride;
    int32_t *err;
};

template <Layout L>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a) {
    using T = LayoutTraits<L>;
    constexpr int kTok = kMoveTok<L>;
    constexpr int kLanes = T::kCodeBytes / 16;           // lanes a code row
    constexpr int kAtOnce = 32 / kLanes;                 // rows a load has
    constexpr int kLoads = kTok / kAtOnce;
    constexpr int kScaleLanes = T::kScaleBytes / 16;     // lanes a scale row
    const int lane = threadIdx.x & 31;
    const int64_t group = (int64_t(blockIdx.x) * kMoveThreads + threadIdx.x) >> 5;
    if (group >= a.total) return;
    const int64_t seq = group / a.groups;
    const int k = int(group % a.groups) * kTok + lane;
    pdl_wait();
    const int64_t page_bytes = int64_t(kTokenBytes<L>) << a.page_bits;
    const int in_page = (1 << a.page_bits) - 1;
    int64_t row = seq, mrow = seq;
    if (a.req) row = __ldg(a.req + seq);
    if (a.rows) mrow = __ldg(a.rows + seq);
    int t = -1;
    if (lane < kTok && k < a.keep) t = __ldg(a.kept + seq * a.kept_stride + k);
    int bits = 0;
    if (t != -1 && (row < 0 || row >= a.table_rows || (a.mass && (mrow < 0 || mrow >= a.n_rows)))) bits = KVQ_DEVERR_STATE;
    else if (t != -1 && (t < 0 || t >= a.max_len)) bits = KVQ_DEVERR_SLOT;
    bool go = t != -1 && !bits;
    int64_t from = 0, to = 0;  // pages
    if (go) {
        from = __ldg(a.table + row * a.table_stride + (t >> a.page_bits));
        to = __ldg(a.to_table + seq * a.to_stride + (k >> a.page_bits));
        if (from < 0 || from >= a.pages || to < 0 || to >= a.pages) {
            bits = KVQ_DEVERR_PAGE;
            go = false;
        }
    }
    if (bits) raise_err(a.err, bits);
    if (go && a.mass) a.mass_out[seq * a.mass_out_stride + k] = __ldg(a.mass + mrow * a.mass_stride + t);
    const int r0 = t & in_page, r1 = k & in_page;
    go = go && (from != to || r0 != r1);  // a row that stays where it is
    // byte offsets of the code rows and of the scale rows
    const int64_t c0 = from * page_bytes + int64_t(r0) * T::kCodeBytes, c1 = to * page_bytes + int64_t(r1) * T::kCodeBytes;
    const int64_t area = int64_t(T::kCodeBytes) << a.page_bits;
    const int64_t s0 = from * page_bytes + area + int64_t(r0) * T::kScaleBytes, s1 = to * page_bytes + area + int64_t(r1) * T::kScaleBytes;
    const uint32_t live = __ballot_sync(0xFFFFFFFFu, go);
    uint4 v[kLoads], sc;
    int64_t at[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int j = i * kAtOnce + lane / kLanes;
        const int64_t src = __shfl_sync(0xFFFFFFFFu, (long long)c0, j);
        at[i] = __shfl_sync(0xFFFFFFFFu, (long long)c1, j);
        if ((live >> j) & 1) v[i] = ld_stream_u4(a.pool + src + (lane % kLanes) * 16);
    }
    const int js = lane / kScaleLanes;
    const int64_t ssrc = __shfl_sync(0xFFFFFFFFu, (long long)s0, js & (kTok - 1));
    const int64_t sdst = __shfl_sync(0xFFFFFFFFu, (long long)s1, js & (kTok - 1));
    const bool scales = js < kTok && ((live >> js) & 1);
    if (scales) sc = ld_stream_u4(a.pool + ssrc + (lane % kScaleLanes) * 16);
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int j = i * kAtOnce + lane / kLanes;
        if ((live >> j) & 1) st_u4(a.pool + at[i] + (lane % kLanes) * 16, v[i]);
    }
    if (scales) st_u4(a.pool + sdst + (lane % kScaleLanes) * 16, sc);
}

bool apart(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x + uintptr_t(a_bytes) <= y || y + uintptr_t(b_bytes) <= x;
}

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxSeqs = int64_t(1) << 20;

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_evict_select(const float *mass, int64_t mass_rows, int64_t mass_width, int64_t mass_row_stride,
                                       const int32_t *rows, const int32_t *kv_len, int64_t n_seq, int64_t keep,
                                       int64_t first, int64_t last, int32_t *kept, int64_t kept_stride, int32_t *count,
                                       int32_t *err, struct CUstream_st *stream) {
    if (n_seq < 0 || mass_rows < 0 || mass_width < 0 || keep < 1 || first < 0 || last < 0) return KVQ_ERR_INVALID_ARG;
    if (first > keep || last > keep - first) return KVQ_ERR_INVALID_ARG;
    if (mass_width > kMaxTokens || keep > kMaxTokens || n_seq > kMaxSeqs) return KVQ_ERR_UNSUPPORTED;
    if (mass_rows > 1 && mass_row_stride < mass_width) return KVQ_ERR_INVALID_ARG;
    if (err && !aligned(err, 4)) return KVQ_ERR_INVALID_ARG;
    if (n_seq == 0) return KVQ_OK;
    if (!rows && n_seq > mass_rows) return KVQ_ERR_INVALID_ARG;
    if (mass_rows > 0 && mass_width > 0 && (!mass || !aligned(mass, 4))) return KVQ_ERR_INVALID_ARG;
    if (!kv_len || !aligned(kv_len, 4) || (rows && !aligned(rows, 4))) return KVQ_ERR_INVALID_ARG;
    if (!kept || !aligned(kept, 4) || (n_seq > 1 && kept_stride < keep) || !count || !aligned(count, 4)) return KVQ_ERR_INVALID_ARG;
    SelectArgs a = {};
    a.mass = mass;
    a.stride = mass_row_stride;
    a.rows = rows;
    a.n_rows = mass_rows;
    a.width = mass_width;
    a.kv_len = kv_len;
    a.kept = kept;
    a.kept_stride = kept_stride;
    a.keep = int(keep);
    a.first = int(first);
    a.last = int(last);
    a.count = count;
    a.err = err;
    // As many CTAs a sequence as hold its keys in registers, 8 a thread, or 16 where eight CTAs need them (one sequence of
    // 4,097 tokens 5.9 us with 8, 7.3 with 16; 32 of 24,577 10.7 and 12.8; one of 131,072 15.6 with 16, 19 otherwise).
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t ctas = (mass_width + kSelThreads * 8 - 1) / (kSelThreads * 8);
    const int cluster = ctas <= 1 ? 1 : ctas <= 2 ? 2 : ctas <= 4 ? 4 : kMaxCluster;
    if (ctas <= kMaxCluster) return launch_select<8>(a, n_seq, cluster, s);
    if (ctas <= 2 * kMaxCluster) return launch_select<16>(a, n_seq, cluster, s);
    return launch_select<0>(a, n_seq, cluster, s);
}

extern "C" kvq_status kvq_evict_move(kvq_layout layout, int page_bits, uint8_t *pool, int64_t pool_pages,
                                     const int32_t *page_table, int64_t table_rows, int64_t table_width,
                                     int64_t table_stride, const int32_t *req, const int32_t *new_table,
                                     int64_t new_width, int64_t new_stride, const int32_t *kept, int64_t n_seq,
                                     int64_t keep, int64_t kept_stride, const float *mass, int64_t mass_rows,
                                     int64_t mass_width, int64_t mass_row_stride, const int32_t *rows, float *mass_out,
                                     int64_t mass_out_stride, int32_t *err, struct CUstream_st *stream) {
    kvq_status st = check_pool(layout, page_bits, pool, pool_pages > 0 && pool_pages <= (int64_t(1) << 40) ? pool_pages << page_bits : 0);
    if (st != KVQ_OK) return st;
    if (n_seq < 0 || keep < 1 || table_rows < 0 || table_width < 0 || table_stride < table_width) return KVQ_ERR_INVALID_ARG;
    if (keep > kMaxTokens || n_seq > kMaxSeqs || table_width > (kMaxTokens >> page_bits)) return KVQ_ERR_UNSUPPORTED;
    if (new_width < 0 || (n_seq > 1 && new_stride < new_width) || new_width < ((keep - 1) >> page_bits) + 1) return KVQ_ERR_INVALID_ARG;
    if (err && !aligned(err, 4)) return KVQ_ERR_INVALID_ARG;
    if ((mass == nullptr) != (mass_out == nullptr)) return KVQ_ERR_INVALID_ARG;
    if (!mass && rows) return KVQ_ERR_INVALID_ARG;
    if (n_seq == 0) return KVQ_OK;
    if (!req && n_seq > table_rows) return KVQ_ERR_INVALID_ARG;
    if (table_rows > 0 && table_width > 0 && !page_table) return KVQ_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || (req && !aligned(req, 4)) || !new_table || !aligned(new_table, 4)) return KVQ_ERR_INVALID_ARG;
    if (!kept || !aligned(kept, 4) || (n_seq > 1 && kept_stride < keep)) return KVQ_ERR_INVALID_ARG;
    if (mass) {
        if (mass_rows < 0 || mass_width < 0 || (mass_rows > 1 && mass_row_stride < mass_width)) return KVQ_ERR_INVALID_ARG;
        if (!aligned(mass, 4) || !aligned(mass_out, 4) || (n_seq > 1 && mass_out_stride < keep)) return KVQ_ERR_INVALID_ARG;
        if (rows ? !aligned(rows, 4) : n_seq > mass_rows) return KVQ_ERR_INVALID_ARG;
        const int64_t in = mass_rows > 0 ? ((mass_rows - 1) * mass_row_stride + mass_width) * 4 : 0;
        if (!apart(mass, in, mass_out, ((n_seq - 1) * mass_out_stride + keep) * 4)) return KVQ_ERR_INVALID_ARG;
    }
    MoveArgs a = {};
    a.pool = pool;
    a.pages = pool_pages;
    a.page_bits = page_bits;
    a.table = page_table;
    a.to_table = new_table;
    a.table_rows = table_rows;
    a.table_stride = table_stride;
    a.to_stride = new_stride;
    a.max_len = table_width << page_bits;
    if (mass && mass_width < a.max_len) a.max_len = mass_width;
    a.req = req;
    a.kept = kept;
    a.kept_stride = kept_stride;
    a.keep = int(keep);
    a.mass = mass;
    a.mass_stride = mass_row_stride;
    a.rows = rows;
    a.n_rows = mass_rows;
    a.mass_out = mass_out;
    a.mass_out_stride = mass_out_stride;
    a.err = err;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_layout(layout, [&](auto Lc) {
        constexpr int kTok = kMoveTok<decltype(Lc)::value>;
        a.groups = (keep + kTok - 1) / kTok;
        a.total = a.groups * n_seq;
        const int64_t per = kMoveThreads / 32, blocks = (a.total + per - 1) / per;
        if (blocks > 0x7FFFFFFF) return KVQ_ERR_UNSUPPORTED;
        return launch_pdl(evict_move_kernel<decltype(Lc)::value>, dim3(unsigned(blocks)), dim3(kMoveThreads), s, a);
    });
}
