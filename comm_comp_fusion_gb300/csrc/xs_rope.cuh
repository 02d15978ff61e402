// xs_rope.cuh -- turning bf16 rows by rotary positions, for the calls that do it
// (xs_rope.cu, xs_append_rope.cu). The mathematics is described in xs_rope.cu.
#pragma once

#include "xs_internal.h"
#include "xs_ptx.cuh"

namespace xs {

// Cosine and sine of the angle at place `pos` of an axis, for a frequency of `frac` 2^-64 turns.
__device__ __forceinline__ float2 rope_sines(int pos, uint64_t frac, bool inverse) {
    const uint64_t phase = (uint64_t)(int64_t)pos * frac;
    const int turns = (int)(uint32_t)((phase + 0x80000000ull) >> 32);  // nearest multiple of 2^-32 turns
    float sn, cn;
    sincospif((float)turns * 0x1p-31f, &sn, &cn);
    return make_float2(cn, inverse ? -sn : sn);
}

__device__ __forceinline__ uint4 rope_load(const uint16_t *ptr) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
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

// Turns a unit, two 16-byte chunks of a row (x, y) with eight pairs, of which the first `pairs` turn.
template <bool HALVES> __device__ __forceinline__ void rope_unit(uint4 &x, uint4 &y, const float2 (&cs)[8], int pairs) {
    if (HALVES) {
        if (pairs > 0) {
            turn_words(x.x, y.x, cs[0], cs[1]);
            turn_words(x.y, y.y, cs[2], cs[3]);
            turn_words(x.z, y.z, cs[4], cs[5]);
            turn_words(x.w, y.w, cs[6], cs[7]);
        }
    } else {
        if (pairs > 0) x.x = turn_word(x.x, cs[0]);
        if (pairs > 1) x.y = turn_word(x.y, cs[1]);
        if (pairs > 2) x.z = turn_word(x.z, cs[2]);
        if (pairs > 3) x.w = turn_word(x.w, cs[3]);
        if (pairs > 4) y.x = turn_word(y.x, cs[4]);
        if (pairs > 5) y.y = turn_word(y.y, cs[5]);
        if (pairs > 6) y.z = turn_word(y.z, cs[6]);
        if (pairs > 7) y.w = turn_word(y.w, cs[7]);
    }
}

}  // namespace xs
