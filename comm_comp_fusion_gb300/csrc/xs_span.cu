// xs_span.cu -- attention over a span of keys per token: a sliding window with
// sinks over whole sequences (head-partitioned, xs_attn_window), and a chunk of
// new tokens over a paged cache (xs_attn_paged).
//
// Mathematics. A token at place i sees the key at place j iff
//   j <= i + right  and  (j >= i - left  or  j < sinks),
// and o = sum_j exp(scale q.k_j - m) v_j / sum_j exp(scale q.k_j - m) over the
// keys it sees, m their largest scaled score; a token that sees no key gets
// zeros. m, the sum and o are held in fp32, in base 2.
//
// One warp per (token, head): each lane holds D/32 elements of q and o; the keys
// are walked one at a time with a warp reduction per score.
#include "xs_internal.h"
#include "xs_ptx.cuh"

namespace xs {

template <int D, bool PAGED>
__global__ void __launch_bounds__(128) span_attn_kernel(const SpanParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)p.T * p.H) return;
    // PAGED: row = (token, head); otherwise row ((r B + b) S + s) Hl + hl of the head partition
    int64_t q_off = row * D, o_off = row * D;
    int pos, keys, seq = 0, hk = 0;
    int64_t kv0 = 0, kv_step = 0;  // element offset of key 0 and between keys (not paged)
    if (PAGED) {
        const int t = (int)(row / p.H), h = (int)(row - (int64_t)t * p.H);
        const CacheRow at = find_sequence(p.q_start, p.N, p.T, t, lane);
        if (at.seq < 0) return;
        seq = at.seq;
        keys = min(max(p.kv_len[seq], 0), p.max_pages * p.page);
        pos = keys - at.q_len + at.i;
        hk = h / p.G;
    } else {
        const int hl = (int)(row % p.Hl);
        const int64_t rbs = row / p.Hl;
        pos = (int)(rbs % p.S);
        const int rb = (int)(rbs / p.S);
        keys = p.S;
        kv0 = ((int64_t)rb * p.S * p.Hl + hl) * D;
        kv_step = (int64_t)p.Hl * D;
        if (!p.head_out) {
            const int b = rb % p.B, r = rb / p.B, rd = pos / p.Sl;
            o_off = ((((int64_t)rd * p.B + b) * p.Sl + (pos - rd * p.Sl)) * p.H + r * p.Hl + hl) * D;
        }
    }
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float((uint32_t)p.q[q_off + e * 32 + lane] << 16);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int last = (int)min((int64_t)keys - 1, (int64_t)pos + p.right);
    const int first = max(0, pos - p.left);
    const int n_sink = min(min(p.sinks, first), last + 1);
    for (int x = 0; x < n_sink + max(0, last - first + 1); ++x) {
        const int j = x < n_sink ? x : first + (x - n_sink);
        int64_t off;
        if (PAGED) {
            const int id = p.table[(int64_t)seq * p.max_pages + j / p.page];
            if (id < 0 || id >= p.n_pages) continue;
            off = (((int64_t)id * p.page + j % p.page) * p.Hk + hk) * D;
        } else {
            off = kv0 + j * kv_step;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], __uint_as_float((uint32_t)p.k[off + e * 32 + lane] << 16), s);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = fmaf(w, __uint_as_float((uint32_t)p.v[off + e * 32 + lane] << 16), o[e] * a);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) p.out[o_off + e * 32 + lane] = (uint16_t)pack_bf16x2(o[e] * inv, 0.f);
}

size_t span_workspace_bytes(int D, int num_sms) {
    return (size_t)2 * num_sms * partial_record_bytes(D);
}

cudaError_t launch_span(int D, const SpanParams &p, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const unsigned grid = (unsigned)(((int64_t)p.T * p.H + 3) / 4);
#define XS_SPAN_CASE(d)                                            \
    case d:                                                        \
        if (p.table)                                               \
            span_attn_kernel<d, true><<<grid, 128, 0, stream>>>(p);  \
        else                                                       \
            span_attn_kernel<d, false><<<grid, 128, 0, stream>>>(p); \
        break;
    switch (D) {
        XS_SPAN_CASE(64)
        XS_SPAN_CASE(96)
        XS_SPAN_CASE(128)
        default: return cudaErrorInvalidValue;
    }
#undef XS_SPAN_CASE
    return cudaGetLastError();
}

}  // namespace xs
