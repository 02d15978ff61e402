// xs_append_rope.cu -- turns the queries and keys of new tokens by their rotary
// positions and writes the keys and values into the pages of a paged cache, all
// in one pass over the rows.
//
// Mathematics: that of xs_rope.cu for the turning and of xs_cache.cu for the rows'
// places; a token's position is given, or it is its place in the sequence.
//
// Bound: HBM for many tokens, latency for few. A row of H + 2 Hk heads is read once and
// written once (keys twice where they are kept in a row as well). What a token needs
// besides its row, its sequence, length, page and sines, is a chain of loads of some 2 us:
// a block takes one to eight tokens (more of few heads), a thread eight pairs of some of a
// token's heads, and its first rows are on their way while the chain runs. Measured on one
// GB300, replayed: 8 prompts (19,181 tokens of 32 + 8 + 8 heads, D = 128, keys kept) 83 us, 6.15 TB/s;
// 601 tokens of 24 + 8 + 8 heads, D = 96, 5.6 us; 8 single tokens 3.9 us.
// Bulk copies through a ring of stages in shared memory, with a warp for the chain, were
// no faster for these prompts (82 us) and slower elsewhere: 40 + 40 + 40 heads 208 us against
// 187, 8 + 8 + 8 of D = 64 43 against 25 (19,200 tokens), 600 tokens 8.5 against 5.8.
#include <algorithm>

#include "xs_rope.cuh"

namespace xs {

// Rows of two chunks in flight per thread, so that four blocks fit an SM: the prompts 87 us (before the sines' frequencies
// were kept in registers), with four rows and three blocks 109, with four and four 100, and 97 where a thread's first rows
// wait for the sines.
constexpr int kAppendUnroll = 2;

template <int D, bool HALVES>
__global__ void __launch_bounds__(D == 96 ? 192 : 256, 4) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int U = D / 16, kThreads = D == 96 ? 192 : 256, kRows = kThreads / U, kWarps = kThreads / 32;
    extern __shared__ float2 cs_tab[];  // [token][pair], D / 2 pairs a token
    __shared__ int64_t row_s[kRows];    // the row's first element in the pools; -1: in no page; -2: of no sequence
    __shared__ int place_s[kRows];
    const int t0 = (int)blockIdx.x * p.tile, nt = min(p.tile, p.T - t0);
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int unit = (int)threadIdx.x % U, rr = (int)threadIdx.x / U;
    const int lanes = kRows / p.tile;  // threads of a token and unit: each takes every lanes-th head of q, k and v
    const int t = rr / lanes, h0 = rr - t * lanes;
    const int pairs = min(8, p.n_pairs - unit * 8);  // pairs of this unit that turn
    int c0 = unit * 16, c1 = c0 + 8;                 // its chunks' first elements
    if (HALVES) {
        c0 = p.unit_first[unit];
        c1 = c0 + p.unit_half[unit];
    }
    // heads of q, then k, then v: the rows of this token, from where head 0 would be
    const int64_t tok = t0 + min(t, nt - 1);
    const int hk = p.H, hv = p.H + p.Hk, heads = t < nt ? hv + p.Hk : 0;
    const uint16_t *q = p.q + tok * p.q_stride, *k = p.k + (tok * p.k_stride - hk * D), *v = p.v + (tok * p.v_stride - hv * D);
    uint4 x[kAppendUnroll], y[kAppendUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int g = h + u * lanes;
            if (g < heads) {
                const uint16_t *src = (g < hk ? q : g < hv ? k : v) + g * D;
                x[u] = rope_load(src + c0);
                y[u] = rope_load(src + c1);
            }
        }
    };
    load(h0);  // on their way while the tokens' places and sines are found
    const int pair = (int)threadIdx.x % (D / 2), axis = p.axis[pair];  // whose sines this thread computes
    const uint64_t frac = p.frac[pair];
    {
        // one warp looks up several tokens in a row, which mostly are of one sequence
        const int per = (p.tile + kWarps - 1) / kWarps, end = min((warp + 1) * per, nt);
        CacheRow at{-1, 0, 0};
        int64_t len = 0;
        for (int i = warp * per; i < end; ++i) {
            if (at.seq >= 0 && at.i + 1 < at.q_len) {
                ++at.i;
            } else {
                at = find_sequence(p.q_start, p.N, p.T, t0 + i, lane);
                if (at.seq >= 0) len = min(max((int64_t)p.kv_len[at.seq], (int64_t)0), (int64_t)p.max_pages * p.page);
            }
            int64_t row = -2, place = 0;
            if (at.seq >= 0) {
                row = -1;
                place = len - at.q_len + at.i;
                if (place >= 0) {
                    const int pg = (int)place >> p.page_log2;
                    const int id = p.table[(int64_t)at.seq * p.max_pages + pg];
                    if (id >= 0 && id < p.n_pages) row = ((int64_t)id * p.page + ((int)place & (p.page - 1))) * p.Hk * D;
                }
            }
            if (lane == 0) {
                row_s[i] = row;
                place_s[i] = (int)place;
            }
        }
    }
    __syncthreads();
    static_assert(kThreads % (D / 2) == 0, "a thread's pair");
    if (pair < p.n_pairs)
        for (int i = (int)threadIdx.x / (D / 2); i < nt; i += kThreads / (D / 2)) {
            if (row_s[i] == -2) continue;
            const int pos = p.pos ? p.pos[(int64_t)(t0 + i) * p.n_axes + axis] : place_s[i];
            cs_tab[i * (D / 2) + pair] = rope_sines(pos, frac, false);
        }
    __syncthreads();
    if (t >= nt || row_s[t] == -2) return;
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = cs_tab[t * (D / 2) + unit * 8 + j];
    const int64_t row = row_s[t];
    uint16_t *q_out = p.q_out + tok * p.H * D, *k_out = p.k_out ? p.k_out + (tok * p.Hk - hk) * D : nullptr;
    uint16_t *k_row = row < 0 ? nullptr : p.k_pages + (row - hk * D), *v_row = row < 0 ? nullptr : p.v_pages + (row - hv * D);
    for (int h = h0; h < heads; h += kAppendUnroll * lanes) {
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int g = h + u * lanes;
            if (g >= heads) break;
            rope_unit<HALVES>(x[u], y[u], cs, g < hv ? pairs : 0);
            uint16_t *dst = g < hk ? q_out : g < hv ? k_row : v_row;
            if (dst) {
                *reinterpret_cast<uint4 *>(dst + g * D + c0) = x[u];
                *reinterpret_cast<uint4 *>(dst + g * D + c1) = y[u];
            }
            if (k_out && g >= hk && g < hv) {
                *reinterpret_cast<uint4 *>(k_out + g * D + c0) = x[u];
                *reinterpret_cast<uint4 *>(k_out + g * D + c1) = y[u];
            }
        }
        load(h + kAppendUnroll * lanes);
    }
}

cudaError_t launch_append_rope(AppendRopeParams &p, int D, bool halves, int num_sms, cudaStream_t stream) {
    // Tokens per block: eight share the chain and the sines, or more while the threads of a token and unit would have
    // fewer than four heads each; fewer for short calls, as long as all blocks run at once, four an SM (1200 tokens of 32 +
    // 8 + 8 heads with two a block 7.7 us, with one, in two waves, 9.7; 601 of D = 96 5.6 and 6.9).
    const int rows = (D == 96 ? 192 : 256) / (D / 16), heads = p.H + 2 * p.Hk;
    p.tile = rows;
    while (p.tile > 1 && ((p.tile > 8 && rows / p.tile * 4 < heads) || ((long long)p.T + p.tile / 2 - 1) / (p.tile / 2) <= 4ll * num_sms))
        p.tile >>= 1;
    for (p.page_log2 = 4; 1 << p.page_log2 < p.page;) ++p.page_log2;
    const unsigned grid = (unsigned)((p.T + p.tile - 1) / p.tile);
    const size_t smem = (size_t)p.tile * (D / 2) * sizeof(float2);
#define XS_APPEND_CASE(d)                                                              \
    case d:                                                                            \
        if (halves)                                                                    \
            append_rope_kernel<d, true><<<grid, d == 96 ? 192 : 256, smem, stream>>>(p);  \
        else                                                                           \
            append_rope_kernel<d, false><<<grid, d == 96 ? 192 : 256, smem, stream>>>(p); \
        break;
    switch (D) {
        XS_APPEND_CASE(64)
        XS_APPEND_CASE(96)
        XS_APPEND_CASE(128)
        default: return cudaErrorInvalidValue;
    }
#undef XS_APPEND_CASE
    return cudaGetLastError();
}

}  // namespace xs
