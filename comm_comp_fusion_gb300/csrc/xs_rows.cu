// xs_rows.cu -- attention of packed rows, one warp a row and query head: over the
// rows of the same sequence (packed prompts), or over a paged cache with a mask of
// bits among the new tokens (drafted trees). Softmax with a running maximum; sums,
// maximum and output in fp32.
#include "xs_internal.h"
#include "xs_ptx.cuh"

namespace xs {

template <int D> __global__ void __launch_bounds__(128) rows_kernel(const RowsParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(w / p.H), h = (int)(w - (int64_t)t * p.H);
    if (t >= p.T) return;
    const CacheRow at = find_sequence(p.q_start, p.N, p.T, t, lane);
    if (at.seq < 0) return;
    const int kh = h / (p.H / p.Hk);
    const uint16_t *q = p.q + t * p.q_stride + h * D + lane * E;
    float qf[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qf[e] = __uint_as_float((uint32_t)q[e] << 16);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    int keys = at.q_len;
    if (p.table) keys = (int)min((int64_t)max(p.kv_len[at.seq], 0), (int64_t)p.max_pages * p.page);
    const int ctx = keys - at.q_len;  // of a paged cache
    for (int j = 0; j < keys; ++j) {
        const uint16_t *k, *v;
        if (p.table) {
            const int b = j - ctx;
            if (b >= 0 && (b >= 32 * p.words || !(p.mask[(int64_t)t * p.words + (b >> 5)] >> (b & 31) & 1))) continue;
            const int id = p.table[(int64_t)at.seq * p.max_pages + j / p.page];
            if (id < 0 || id >= p.n_pages) continue;
            const int64_t row = (((int64_t)id * p.page + j % p.page) * p.Hk + kh) * D + lane * E;
            k = p.k + row;
            v = p.v + row;
        } else {
            if (j > at.i + p.right || (j < at.i - p.left && j >= p.sinks)) continue;
            const int64_t r = t - at.i + j;
            k = p.k + r * p.k_stride + kh * D + lane * E;
            v = p.v + r * p.v_stride + kh * D + lane * E;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(qf[e], __uint_as_float((uint32_t)k[e] << 16), s);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.scale_log2;
        const float top = fmaxf(m, s), a = exp2f(m - top), x = exp2f(s - top);
        m = top;
        l = l * a + x;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(x, __uint_as_float((uint32_t)v[e] << 16), o[e] * a);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        p.out[((int64_t)t * p.H + h) * D + lane * E + e] = (uint16_t)pack_bf16x2(o[e] * inv, 0.f);
}

cudaError_t launch_rows(const RowsParams &p, int D, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)p.T * p.H + 3) / 4);
    if (D == 64) rows_kernel<64><<<grid, 128, 0, stream>>>(p);
    if (D == 96) rows_kernel<96><<<grid, 128, 0, stream>>>(p);
    if (D == 128) rows_kernel<128><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace xs
