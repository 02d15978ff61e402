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
// flops); a block computes its tokens' sines and cosines once into shared
// memory and uses them for every head of q and k.
#include "xs_internal.h"
#include "xs_ptx.cuh"

namespace xs {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;

__device__ __forceinline__ uint32_t rope_div(uint32_t n, uint32_t m, uint32_t s) { return (__umulhi(n, m) + n) >> s; }

__device__ __forceinline__ uint4 rope_load(const uint4 *ptr) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(ptr));
    return v;
}

// Turns the pair (a, b); fp32 throughout, rounded to bf16 once by the caller.
__device__ __forceinline__ void rope_turn(float &a, float &b, float2 cs) {
    const float x = a * cs.x - b * cs.y;
    b = fmaf(a, cs.y, b * cs.x);
    a = x;
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Neighbouring pairs: one word holds a pair.
__device__ __forceinline__ uint32_t turn_word(uint32_t w, float2 cs) {
    float a = lo_f(w), b = hi_f(w);
    rope_turn(a, b, cs);
    return pack_bf16x2(a, b);
}
// Pairs half an axis apart: two words hold two pairs.
__device__ __forceinline__ void turn_words(uint32_t &u, uint32_t &v, float2 c0, float2 c1) {
    float a0 = lo_f(u), a1 = hi_f(u), b0 = lo_f(v), b1 = hi_f(v);
    rope_turn(a0, b0, c0);
    rope_turn(a1, b1, c1);
    u = pack_bf16x2(a0, a1);
    v = pack_bf16x2(b0, b1);
}

// Element offset of (b, s, head h of nh) in the sequence or the head partition.
__device__ __forceinline__ int64_t rope_row(const RopeParams &p, bool seq, int b, int s, int h, int nh, int nhl) {
    if (seq) {
        const int r = (int)rope_div((uint32_t)s, p.mSl, p.sSl);
        return ((((int64_t)r * p.B + b) * p.Sl + (s - r * p.Sl)) * nh + h) * p.D;
    }
    const int r = h / nhl;
    return ((((int64_t)r * p.B + b) * p.S + s) * nhl + (h - r * nhl)) * p.D;
}

// A block turns `tile` tokens of one batch, all heads of q then of k. A unit is
// 16 bytes of a row (neighbouring pairs), or two 16-byte chunks half an axis
// apart (HALVES); chunks past the rotated elements are copied.
template <bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float2 cs_tab[];  // [token][pair]
    const int tiles = (p.S + p.tile - 1) / p.tile;
    const int b = (int)(blockIdx.x / (unsigned)tiles), s0 = ((int)blockIdx.x - b * tiles) * p.tile;
    const int nt = min(p.tile, p.S - s0);
    const int *pos = p.pos + ((int64_t)b * p.pos_batch + s0) * p.n_axes;
    for (int i = threadIdx.x; i < nt * p.n_pairs; i += kRopeThreads) {
        const int t = i / p.n_pairs, j = i - t * p.n_pairs;
        const uint64_t phase = (uint64_t)(int64_t)pos[t * p.n_axes + p.axis[j]] * p.frac[j];
        const int turns = (int)(uint32_t)((phase + 0x80000000ull) >> 32);  // nearest multiple of 2^-32 turns
        float sn, cn;
        sincospif((float)turns * 0x1p-31f, &sn, &cn);
        cs_tab[i] = make_float2(cn, p.inverse ? -sn : sn);
    }
    __syncthreads();
    const uint32_t per_row = (uint32_t)p.units, heads = (uint32_t)(p.H + p.Hk);
    const uint32_t total = (uint32_t)nt * heads * per_row;
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kRopeUnroll * kRopeThreads) {
        uint4 x[kRopeUnroll], y[kRopeUnroll];
        uint16_t *dst[kRopeUnroll];
        int first[kRopeUnroll], half[kRopeUnroll], tok[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const uint32_t i = i0 + u * kRopeThreads;
            if (i >= total) break;
            const uint32_t row = rope_div(i, p.mU, p.sU), unit = i - row * per_row;
            const int t = (int)rope_div(row, p.mH, p.sH);
            int h = (int)(row - (uint32_t)t * heads);
            const bool is_q = h < p.H;
            if (!is_q) h -= p.H;
            const int nh = is_q ? p.H : p.Hk, nhl = is_q ? p.Hl : p.Hkl;
            const uint16_t *src = (is_q ? p.q : p.k) + rope_row(p, p.seq_in, b, s0 + t, h, nh, nhl);
            dst[u] = (is_q ? p.q_out : p.k_out) + rope_row(p, p.seq_out, b, s0 + t, h, nh, nhl);
            tok[u] = t;
            if (HALVES) {
                first[u] = p.unit_first[unit];
                half[u] = p.unit_half[unit];  // elements between the two chunks; 0: a copied chunk
                x[u] = rope_load(reinterpret_cast<const uint4 *>(src + first[u]));
                if (half[u]) y[u] = rope_load(reinterpret_cast<const uint4 *>(src + first[u] + half[u]));
            } else {
                first[u] = (int)unit * 8;
                half[u] = 0;
                x[u] = rope_load(reinterpret_cast<const uint4 *>(src + first[u]));
            }
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const uint32_t i = i0 + u * kRopeThreads;
            if (i >= total) break;
            if (HALVES) {
                if (half[u]) {
                    const uint32_t unit = i - rope_div(i, p.mU, p.sU) * per_row;
                    const float2 *cs = cs_tab + tok[u] * p.n_pairs + unit * 8;  // rotated units come first, 8 pairs each
                    turn_words(x[u].x, y[u].x, cs[0], cs[1]);
                    turn_words(x[u].y, y[u].y, cs[2], cs[3]);
                    turn_words(x[u].z, y[u].z, cs[4], cs[5]);
                    turn_words(x[u].w, y[u].w, cs[6], cs[7]);
                    *reinterpret_cast<uint4 *>(dst[u] + first[u] + half[u]) = y[u];
                }
            } else {
                const int j = first[u] >> 1;  // the chunk's first pair
                const float2 *cs = cs_tab + tok[u] * p.n_pairs + j;
                if (j + 0 < p.n_pairs) x[u].x = turn_word(x[u].x, cs[0]);
                if (j + 1 < p.n_pairs) x[u].y = turn_word(x[u].y, cs[1]);
                if (j + 2 < p.n_pairs) x[u].z = turn_word(x[u].z, cs[2]);
                if (j + 3 < p.n_pairs) x[u].w = turn_word(x[u].w, cs[3]);
            }
            *reinterpret_cast<uint4 *>(dst[u] + first[u]) = x[u];
        }
    }
}

cudaError_t launch_rope(RopeParams &p, bool halves, int num_sms, cudaStream_t stream) {
    // tokens per block: eight share a table when that still leaves several blocks
    // for every SM, fewer for short calls
    p.tile = 8;
    while (p.tile > 1 && (long long)p.B * ((p.S + p.tile - 1) / p.tile) < 4ll * num_sms) p.tile >>= 1;
    fastdiv_magic((uint32_t)p.units, &p.mU, &p.sU);
    fastdiv_magic((uint32_t)(p.H + p.Hk), &p.mH, &p.sH);
    fastdiv_magic((uint32_t)p.Sl, &p.mSl, &p.sSl);
    const unsigned grid = (unsigned)((p.S + p.tile - 1) / p.tile) * (unsigned)p.B;
    const size_t smem = (size_t)p.tile * p.n_pairs * sizeof(float2);
    if (halves)
        rope_kernel<true><<<grid, kRopeThreads, smem, stream>>>(p);
    else
        rope_kernel<false><<<grid, kRopeThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace xs
