// xs_append_rope.cu -- turns the queries and keys of new tokens by their rotary
// positions and writes the keys and values into the pages of a paged cache, all
// in one pass over the rows.
//
// Mathematics: that of xs_rope.cu for the turning and of xs_cache.cu for the rows'
// places; a token's position is given, or it is its place in the sequence.
//
// Bound: HBM. A row of H + 2 Hk heads is read once and written once (keys
// twice where they are kept in a row as well).
#include <algorithm>

#include "xs_rope.cuh"

namespace xs {

constexpr int kAppendUnroll = 4;

template <int D, bool HALVES>
__global__ void __launch_bounds__(D == 96 ? 192 : 256) append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int U = D / 16, kThreads = D == 96 ? 192 : 256, kRows = kThreads / U, kWarps = kThreads / 32;
    extern __shared__ float2 cs_tab[];  // [token][pair], D / 2 pairs a token
    __shared__ int64_t row_s[kRows];    // the row's first element in the pools; -1: in no page; -2: of no sequence
    __shared__ int place_s[kRows];
    const int t0 = (int)blockIdx.x * p.tile, nt = min(p.tile, p.T - t0);
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
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
                    const int pg = (int)(place / p.page);
                    const int id = p.table[(int64_t)at.seq * p.max_pages + pg];
                    if (id >= 0 && id < p.n_pages) row = ((int64_t)id * p.page + (place - (int64_t)pg * p.page)) * p.Hk * D;
                }
            }
            if (lane == 0) {
                row_s[i] = row;
                place_s[i] = (int)place;
            }
        }
    }
    __syncthreads();
    for (int i = (int)threadIdx.x; i < nt * (D / 2); i += kThreads) {
        const int t = i / (D / 2), j = i - t * (D / 2);
        if (j >= p.n_pairs || row_s[t] == -2) continue;
        const int pos = p.pos ? p.pos[(int64_t)(t0 + t) * p.n_axes + p.axis[j]] : place_s[t];
        cs_tab[i] = rope_sines(pos, p.frac[j], false);
    }
    __syncthreads();
    const int unit = (int)threadIdx.x % U, rr = (int)threadIdx.x / U;
    const int lanes = kRows / p.tile;  // threads of a token and unit: each takes every lanes-th head
    const int t = rr / lanes, h0 = rr - t * lanes;
    if (t >= nt || row_s[t] == -2) return;
    const int pairs = min(8, p.n_pairs - unit * 8);  // pairs of this unit that turn
    int c0 = unit * 16, c1 = c0 + 8;                 // its chunks' first elements
    if (HALVES) {
        c0 = p.unit_first[unit];
        c1 = c0 + p.unit_half[unit];
    }
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = cs_tab[t * (D / 2) + unit * 8 + j];
    const int64_t tok = t0 + t, row = row_s[t];
#pragma unroll 1
    for (int which = 0; which < 3; ++which) {  // q, k, v
        const int nh = which ? p.Hk : p.H, turn = which < 2 ? pairs : 0;
        const uint16_t *src = which == 0 ? p.q + tok * p.q_stride : which == 1 ? p.k + tok * p.k_stride : p.v + tok * p.v_stride;
        uint16_t *dst = which == 0 ? p.q_out + tok * p.H * D : row < 0 ? nullptr : (which == 1 ? p.k_pages : p.v_pages) + row;
        uint16_t *also = which == 1 && p.k_out ? p.k_out + tok * p.Hk * D : nullptr;
        if (!dst && !also) continue;
        for (int h = h0; h < nh; h += kAppendUnroll * lanes) {
            uint4 x[kAppendUnroll], y[kAppendUnroll];
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u)
                if (h + u * lanes < nh) {
                    x[u] = rope_load(src + (h + u * lanes) * D + c0);
                    y[u] = rope_load(src + (h + u * lanes) * D + c1);
                }
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u)
                if (h + u * lanes < nh) {
                    const int at = (h + u * lanes) * D;
                    rope_unit<HALVES>(x[u], y[u], cs, turn);
                    if (dst) {
                        *reinterpret_cast<uint4 *>(dst + at + c0) = x[u];
                        *reinterpret_cast<uint4 *>(dst + at + c1) = y[u];
                    }
                    if (also) {
                        *reinterpret_cast<uint4 *>(also + at + c0) = x[u];
                        *reinterpret_cast<uint4 *>(also + at + c1) = y[u];
                    }
                }
        }
    }
}

cudaError_t launch_append_rope(AppendRopeParams &p, int D, bool halves, int num_sms, cudaStream_t stream) {
    // tokens per block: the rule of launch_rope
    const int rows = (D == 96 ? 192 : 256) / (D / 16), heads = std::max(p.H, p.Hk);
    p.tile = rows;
    while (p.tile > 1 && ((p.tile > 8 && rows / p.tile * kAppendUnroll < heads) ||
                          ((long long)p.T + p.tile - 1) / p.tile < 4ll * num_sms))
        p.tile >>= 1;
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
