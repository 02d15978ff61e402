// xs_rope.cu -- rotary positions with several axes for queries and keys, in
// either partition of the Ulysses layouts, optionally moving them from one
// partition to the other on the way (the pre-attention All-to-All).
//
// Mathematics. A head's first sum(axis_dims) elements are split into axes, and
// an axis into pairs (a, b): neighbours, or elements half an axis apart. A
// token at place p of the pair's axis turns it by the angle p f:
//   a' = a cos(p f) - b sin(p f),  b' = a sin(p f) + b cos(p f);
// the inverse (the transpose, which is also the gradient) turns it by -p f.
//
// Angles. p is an integer, so the angle in turns modulo 1 needs no floating
// range reduction: the frequency in turns, f / 2 pi, is kept as a 64-bit binary
// fraction, and p times it modulo 2^64 is the exact phase of that fraction. The
// error, |p| 2^-64 turns plus f's own 53 bits, stays below fp32's rounding of
// the angle for every 32-bit place. The phase's high 32 bits go through
// sincospif.
//
// Bound: HBM. Every element is read and written once (4 bytes of traffic for 3
// flops). A block turns a few tokens of one batch: it computes their sines and
// cosines once into shared memory, and each thread keeps those of its eight pairs
// of one token in registers while it walks heads of q and then of k, four at a
// time (eight 16-byte loads in flight). Measured on one GB300: B = 2, S = 16384, H = 40,
// D = 128 199 us, 6.75 TB/s (with one unit of a random row per step instead of a
// thread's own token, 251 us); S = 4096, H = 24 to the head partition 26 us with changing inputs,
// 3.9 TB/s (21 replayed on buffers that stay in the L2).
#include <algorithm>

#include "xs_internal.h"
#include "xs_rope.cuh"

namespace xs {

constexpr int kRopeUnroll = 4;

// The rows of one token in a tensor of nh heads: heads in order, `hop` elements
// apart, with a jump of `jump` more after every nhl (head partition: the next rank's
// slice; sequence partition: never).
struct RopeRows {
    int64_t at, jump;
    int hop, left;  // left: heads before the next jump
};
__device__ __forceinline__ RopeRows rope_rows(const RopeParams &p, bool seq, int b, int s, int h, int nh, int nhl) {
    RopeRows r;
    r.hop = p.D;
    if (seq) {
        const int rk = s / p.Sl;
        r.at = ((((int64_t)rk * p.B + b) * p.Sl + (s - rk * p.Sl)) * nh + h) * p.D;
        r.jump = 0;
        r.left = 1 << 30;
    } else {
        const int rk = h / nhl;
        r.at = ((((int64_t)rk * p.B + b) * p.S + s) * nhl + (h - rk * nhl)) * p.D;
        r.jump = ((int64_t)p.B * p.S - 1) * nhl * p.D;
        r.left = nhl - (h - rk * nhl);
    }
    return r;
}
// The row `by` heads on.
__device__ __forceinline__ void rope_advance(RopeRows &r, int by, int nhl) {
    r.at += (int64_t)by * r.hop;
    r.left -= by;
    while (r.left <= 0) {
        r.at += r.jump;
        r.left += nhl;
    }
}

// A thread's unit is two 16-byte chunks of a row, eight pairs: 16 elements in a row
// (neighbouring pairs), or two chunks half an axis apart (HALVES); units past the
// rotated elements are copied.
template <int D, bool HALVES>
__global__ void __launch_bounds__(D == 96 ? 192 : 256) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int U = D / 16, kThreads = D == 96 ? 192 : 256, kRows = kThreads / U;
    extern __shared__ float2 cs_tab[];  // [token][pair], D / 2 pairs a token
    const int tiles = (p.S + p.tile - 1) / p.tile;
    const int b = (int)(blockIdx.x / (unsigned)tiles), s0 = ((int)blockIdx.x - b * tiles) * p.tile;
    const int nt = min(p.tile, p.S - s0);
    const int *pos = p.pos + ((int64_t)b * p.pos_batch + s0) * p.n_axes;
    auto sines = [&](int i) {
        const int t = i / (D / 2), j = i - t * (D / 2);
        if (j >= p.n_pairs) return;
        cs_tab[i] = rope_sines(pos[t * p.n_axes + p.axis[j]], p.frac[j], p.inverse);
    };
    const int n = nt * (D / 2);
    if (p.tile > 8) {  // several a thread: their places are fetched together
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kThreads) sines(i);
    } else {
        for (int i = threadIdx.x; i < n; i += kThreads) sines(i);
    }
    __syncthreads();
    const int unit = (int)threadIdx.x % U, rr = (int)threadIdx.x / U;
    const int lanes = kRows / p.tile;  // threads of a token and unit: each takes every lanes-th head
    const int t = rr / lanes, h0 = rr - t * lanes;
    if (t >= nt) return;
    const int pairs = min(8, p.n_pairs - unit * 8);  // pairs of this unit that turn
    int c0 = unit * 16, c1 = c0 + 8;                 // its chunks' first elements
    if (HALVES) {
        c0 = p.unit_first[unit];
        c1 = c0 + p.unit_half[unit];
    }
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = cs_tab[t * (D / 2) + unit * 8 + j];
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int nh = which ? p.Hk : p.H, nhl = which ? p.Hkl : p.Hl;
        if (h0 >= nh) continue;
        const uint16_t *src = which ? p.k : p.q;
        uint16_t *dst = which ? p.k_out : p.q_out;
        RopeRows in = rope_rows(p, p.seq_in, b, s0 + t, h0, nh, nhl), out = rope_rows(p, p.seq_out, b, s0 + t, h0, nh, nhl);
        for (int h = h0; h < nh; h += kRopeUnroll * lanes) {
            uint4 x[kRopeUnroll], y[kRopeUnroll];
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u)
                if (h + u * lanes < nh) {
                    x[u] = rope_load(src + in.at + c0);
                    y[u] = rope_load(src + in.at + c1);
                    rope_advance(in, lanes, nhl);
                }
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u)
                if (h + u * lanes < nh) {
                    rope_unit<HALVES>(x[u], y[u], cs, pairs);
                    *reinterpret_cast<uint4 *>(dst + out.at + c0) = x[u];
                    *reinterpret_cast<uint4 *>(dst + out.at + c1) = y[u];
                    rope_advance(out, lanes, nhl);
                }
        }
    }
}

cudaError_t launch_rope(RopeParams &p, bool halves, int num_sms, cudaStream_t stream) {
    // Tokens per block: eight share the table's set-up, or more while the threads of a
    // token and unit would have fewer than four heads each; fewer for short calls, so that
    // four blocks are left for every SM (S = 4096: 21 us with 4, 27 with 2; 2 + 1 heads of
    // 111,900 tokens, D = 96: 39 us with 32 tokens a block, 98 with 8).
    const int rows = (p.D == 96 ? 192 : 256) / (p.D / 16), heads = std::max(p.H, p.Hk);
    p.tile = rows;
    while (p.tile > 1 && ((p.tile > 8 && rows / p.tile * kRopeUnroll < heads) ||
                          (long long)p.B * ((p.S + p.tile - 1) / p.tile) < 4ll * num_sms))
        p.tile >>= 1;
    const unsigned grid = (unsigned)((p.S + p.tile - 1) / p.tile) * (unsigned)p.B;
    const size_t smem = (size_t)p.tile * (p.D / 2) * sizeof(float2);
#define XS_ROPE_CASE(d)                                                        \
    case d:                                                                    \
        if (halves)                                                            \
            rope_kernel<d, true><<<grid, d == 96 ? 192 : 256, smem, stream>>>(p);  \
        else                                                                   \
            rope_kernel<d, false><<<grid, d == 96 ? 192 : 256, smem, stream>>>(p); \
        break;
    switch (p.D) {
        XS_ROPE_CASE(64)
        XS_ROPE_CASE(96)
        XS_ROPE_CASE(128)
        XS_ROPE_CASE(256)
        default: return cudaErrorInvalidValue;
    }
#undef XS_ROPE_CASE
    return cudaGetLastError();
}

}  // namespace xs
