// kvq_tree.cu -- the masks and positions of trees of drafted tokens, from each
// token's parent (kvq_tree_mask): what kvq_attend_tree and the rotary positions
// of the drafted tokens take.
//
// A token sees itself and its ancestors.  A thread walks up from its token: the
// parents come before their children, so the bits are set from the top down and
// a word is done when the walk leaves it.  Bound by latency: one load of the
// parents into shared memory, and as many steps as the tree is deep.
#include "kvq_launch.cuh"

namespace kvq {
namespace {

constexpr int kTreeThreads = 256;
constexpr int kMaxTree = 1024;

struct TreeArgs {
    const int32_t *parent;
    int64_t stride;
    int q_len, words;
    const int32_t *kv_len;
    unsigned long long *mask;
    int32_t *pos;
    int32_t *err;
};

__global__ void __launch_bounds__(kTreeThreads) tree_mask_kernel(const TreeArgs a) {
    __shared__ int16_t up[kMaxTree];
    const int64_t seq = blockIdx.x;
    pdl_wait();
    bool bad = false;
    for (int j = threadIdx.x; j < a.q_len; j += blockDim.x) {
        const int p = __ldg(a.parent + seq * a.stride + j);
        const bool good = p >= -1 && p < j;
        bad = bad || !good;
        up[j] = int16_t(good ? p : -1);
    }
    pdl_trigger();
    if (bad) raise_err(a.err, KVQ_DEVERR_STATE);
    const int base = a.kv_len ? __ldg(a.kv_len + seq) - a.q_len : 0;
    __syncthreads();
    for (int j = threadIdx.x; j < a.q_len; j += blockDim.x) {
        unsigned long long *const to = a.mask + (seq * a.q_len + j) * a.words;
        int depth = -1, at = j;
        for (int w = a.words - 1; w >= 0; --w) {
            unsigned long long bits = 0;
            for (; at >= w * 64; at = up[at], ++depth) bits |= 1ull << (at & 63);
            to[w] = bits;
        }
        if (a.pos) a.pos[seq * a.q_len + j] = max(0, base + depth);
    }
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_tree_mask(const int32_t *parent, int64_t n_seq, int64_t q_len, int64_t parent_stride,
                                    const int32_t *kv_len, uint64_t *mask, int32_t *pos, int32_t *err,
                                    struct CUstream_st *stream) {
    if (n_seq < 0 || q_len < 1) return KVQ_ERR_INVALID_ARG;
    if (q_len > kMaxTree || n_seq > (int64_t(1) << 24)) return KVQ_ERR_UNSUPPORTED;
    if (err && !aligned(err, 4)) return KVQ_ERR_INVALID_ARG;
    if (n_seq == 0) return KVQ_OK;
    if (!parent || !aligned(parent, 4) || (n_seq > 1 && parent_stride < q_len)) return KVQ_ERR_INVALID_ARG;
    if (!mask || !aligned(mask, 8) || !aligned(kv_len, 4) || !aligned(pos, 4)) return KVQ_ERR_INVALID_ARG;
    TreeArgs a = {};
    a.parent = parent;
    a.stride = parent_stride;
    a.q_len = int(q_len);
    a.words = int((q_len + 63) / 64);
    a.kv_len = kv_len;
    a.mask = reinterpret_cast<unsigned long long *>(mask);
    a.pos = pos;
    a.err = err;
    const int threads = q_len < kTreeThreads ? int((q_len + 31) / 32 * 32) : kTreeThreads;
    return launch_pdl(tree_mask_kernel, dim3(unsigned(n_seq)), dim3(threads), reinterpret_cast<cudaStream_t>(stream), a);
}
