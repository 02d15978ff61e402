// xs_tree.cu -- masks and positions of drafted token trees from the tokens' parents.
//
// Row i of a tree has bit j set iff token j is token i itself or one of those it
// follows; its position is the context's length plus its depth. A block takes a
// sequence: the parents go to shared memory and each thread walks from one token
// to its root, so a walk costs one shared-memory read a level.
//
// Bound: latency. Few kilobytes move; the chain is q_start, parents, walk, store. Measured on one GB300, replayed: 4 trees of
// 8 tokens 2.1 us, 256 of 60 to 250 3.8.
#include "xs_internal.h"

namespace xs {

__global__ void tree_mask_kernel(const TreeMaskParams p) {
    extern __shared__ int tree_s[];  // parents [most], then bits [words][most]
    const int seq = (int)blockIdx.x, most = 32 * p.words;
    const int q0 = min(max(p.q_start[seq], 0), p.T), q_len = max(0, min(max(p.q_start[seq + 1], 0), p.T) - q0);
    const int n = min(q_len, most), i = (int)threadIdx.x;
    const int len = p.pos ? max(p.kv_len[seq], 0) : 0;
    int *bits = tree_s + most;
    int parent = -1;
    if (i < n) {
        parent = p.parents[q0 + i];
        if (parent < 0 || parent >= i) parent = -1;
        tree_s[i] = parent;
        for (int w = 0; w < p.words; ++w) bits[w * most + i] = 0;
        bits[(i >> 5) * most + i] = (int)(1u << (i & 31));
    }
    __syncthreads();
    if (i < n) {
        int depth = 0;
        for (int j = parent; j >= 0; j = tree_s[j]) {  // ends: a parent comes before its child
            bits[(j >> 5) * most + i] |= (int)(1u << (j & 31));
            ++depth;
        }
        if (p.pos) p.pos[q0 + i] = len - q_len + depth;
    }
    __syncthreads();
    int *mask = p.mask + (int64_t)q0 * p.words;
    for (int e = i; e < n * p.words; e += most) {
        const int r = e / p.words;
        mask[e] = bits[(e - r * p.words) * most + r];
    }
    for (int r = most + i; r < q_len; r += most) {  // more tokens than bits: they see the context alone
        for (int w = 0; w < p.words; ++w) mask[(int64_t)r * p.words + w] = 0;
        if (p.pos) p.pos[q0 + r] = len - q_len;
    }
}

cudaError_t launch_tree_mask(const TreeMaskParams &p, cudaStream_t stream) {
    const int most = 32 * p.words;
    tree_mask_kernel<<<(unsigned)p.N, most, (size_t)most * (p.words + 1) * sizeof(int), stream>>>(p);
    return cudaGetLastError();
}

}  // namespace xs
