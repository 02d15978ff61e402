// xs_tree.cu -- masks and positions of drafted token trees from the tokens' parents.
//
// Row i of a tree has bit j set iff token j is token i itself or one of those it
// follows; its position is the context's length plus its depth. A block takes a
// sequence, a thread a token, the parents go to shared memory. A thread first walks 16
// levels up from its token, one read a level. On longer branches the tokens then double their
// reach in rounds: a token that knows its next ancestors takes over the bits of the
// one behind them, what that one knows, and the one behind that.
//
// Bound: latency. Few kilobytes move; the chain is q_start, parents, rounds, store. Measured on
// one GB300, replayed: 4 trees of 8 tokens 2.3 us, 256 of 60 to 250 4.0; a chain of 256 4.8 (14.4 by the walk alone; with
// rounds alone 5.2, and the trees 3.0 and 5.0).
#include "xs_internal.h"

namespace xs {

__global__ void tree_mask_kernel(const TreeMaskParams p) {
    extern __shared__ int tree_s[];  // parents, the ancestor behind the known ones, their number [most], then bits [words][most]
    const int seq = (int)blockIdx.x, most = 32 * p.words;
    const int q0 = min(max(p.q_start[seq], 0), p.T), q_len = max(0, min(max(p.q_start[seq + 1], 0), p.T) - q0);
    const int n = min(q_len, most), i = (int)threadIdx.x;
    const int len = p.pos ? max(p.kv_len[seq], 0) : 0;
    int *next_s = tree_s + most, *depth_s = tree_s + 2 * most;
    uint32_t *bits_s = reinterpret_cast<uint32_t *>(tree_s + 3 * most);
    int next = -1, depth = 0;
    if (i < n) {
        next = p.parents[q0 + i];
        if (next < 0 || next >= i) next = -1;  // (so that every walk ends)
        tree_s[i] = next;
        for (int w = 0; w < p.words; ++w) bits_s[w * most + i] = 0u;
        bits_s[(i >> 5) * most + i] = 1u << (i & 31);
    }
    __syncthreads();
    for (; next >= 0 && depth < 16; next = tree_s[next], ++depth) bits_s[(next >> 5) * most + i] |= 1u << (next & 31);
    if (i < n) {
        next_s[i] = next;
        depth_s[i] = depth;
    }
    while (__syncthreads_or(next >= 0)) {  // at most 4 rounds
        const int from = next;
        int further = 0, behind = -1;
        uint32_t bits[kTreeMaxWords] = {};
        if (from >= 0) {
            further = depth_s[from] + 1;
            behind = next_s[from];
#pragma unroll
            for (int w = 0; w < kTreeMaxWords; ++w)
                if (w < p.words) bits[w] = bits_s[w * most + from];
        }
        __syncthreads();
        if (from >= 0) {
            depth_s[i] = depth += further;
            next_s[i] = next = behind;
#pragma unroll
            for (int w = 0; w < kTreeMaxWords; ++w)
                if (w < p.words) bits_s[w * most + i] |= bits[w];
        }
    }
    if (i < n && p.pos) p.pos[q0 + i] = len - q_len + depth;
    int *mask = p.mask + (int64_t)q0 * p.words;
    for (int e = i; e < n * p.words; e += most) {
        const int r = e / p.words;
        mask[e] = (int)bits_s[(e - r * p.words) * most + r];
    }
    for (int r = most + i; r < q_len; r += most) {  // more tokens than bits: they see the context alone
        for (int w = 0; w < p.words; ++w) mask[(int64_t)r * p.words + w] = 0;
        if (p.pos) p.pos[q0 + r] = len - q_len;
    }
}

cudaError_t launch_tree_mask(const TreeMaskParams &p, cudaStream_t stream) {
    const int most = 32 * p.words;
    tree_mask_kernel<<<(unsigned)p.N, most, (size_t)most * (p.words + 3) * sizeof(int), stream>>>(p);
    return cudaGetLastError();
}

}  // namespace xs
