// xs_ops_checks.h -- argument checks and host-side tables that the C ABI of the
// operators around the fused attention shares (xs_ops_api.cpp, xs_serve_api.cpp).
// Each check records the thread's last error and returns a status (0: fine).
#pragma once

#include "../../include/xs.h"

#include <algorithm>
#include <cmath>

#include "xs_internal.h"

namespace xs {

inline bool misaligned16(const void *p) { return ((uintptr_t)p & 15u) != 0; }
inline bool misaligned4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

struct Buffer {
    const void *ptr;
    size_t bytes;
    const char *name;
};

// No buffer of `out` may overlap one of `in` or another of `out`.
inline int check_disjoint(const Buffer *out, int n_out, const Buffer *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (api_overlaps(out[i].ptr, out[i].bytes, in[j].ptr, in[j].bytes))
                return api_fail(XS_ERR_ALIAS, "%s overlaps %s", out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (api_overlaps(out[i].ptr, out[i].bytes, out[j].ptr, out[j].bytes))
                return api_fail(XS_ERR_ALIAS, "%s overlaps %s", out[i].name, out[j].name);
    }
    return 0;
}
inline int check_device(const Buffer *b, int n, int dev) {
    for (int i = 0; i < n; ++i)
        if (b[i].bytes)
            if (const int st = api_device_pointer(b[i].ptr, dev, b[i].name)) return st;
    return 0;
}

// f (radians per unit of place) in turns, modulo 1, as a 64-bit binary fraction
// (two's complement for a negative f). |f| / 2 pi is formed in double-double
// arithmetic (1 / 2 pi in two doubles), so the fraction is as exact as f.
inline uint64_t turns_fraction(double f) {
    const double hi_c = 0.15915494309189535, lo_c = -9.839338337591243e-18;  // 1 / 2 pi
    const double x = std::fabs(f), hi = x * hi_c, lo = std::fma(x, hi_c, -hi) + x * lo_c;
    const double frac = hi - std::floor(hi);  // exact, below 1
    const uint64_t u = (uint64_t)(frac * 0x1p64) + (uint64_t)(int64_t)std::llrint(lo * 0x1p64);  // (exact products)
    return f < 0 ? 0 - u : u;
}

// Fills the pairs' axes and frequencies (and, for pairs half an axis apart, a unit's chunks) of a rotary
// call's parameters.
template <typename P> int rope_table(int n_axes, const int *axis_dims, const double *freqs, bool halves, int D, P *p) {
    if (n_axes < 1 || n_axes > kRopeMaxAxes)
        return api_fail(XS_ERR_SHAPE, "n_axes must be 1 to %d (got %d)", kRopeMaxAxes, n_axes);
    int rot = 0;
    for (int a = 0; a < n_axes; ++a) {
        const int d = axis_dims[a];
        if (d < 2 || d > D || d % 2)
            return api_fail(XS_ERR_SHAPE, "axis_dims[%d]=%d is not an even number from 2 to D", a, d);
        if (halves && d % 16)
            return api_fail(XS_ERR_UNSUPPORTED,
                            "pairs half an axis apart need axis_dims in multiples of 16 (axis_dims[%d]=%d)", a, d);
        if (rot + d > D) return api_fail(XS_ERR_SHAPE, "axis_dims add up to more than D=%d", D);
        for (int j = 0; j < d / 2; ++j) p->axis[rot / 2 + j] = (uint8_t)a;
        for (int u = 0; halves && u < d / 16; ++u) {
            p->unit_first[rot / 16 + u] = (uint8_t)(rot + 8 * u);
            p->unit_half[rot / 16 + u] = (uint8_t)(d / 2);
        }
        rot += d;
    }
    for (int j = 0; j < rot / 2; ++j) {
        if (!std::isfinite(freqs[j]) || std::fabs(freqs[j]) > 1e6)
            return api_fail(XS_ERR_SHAPE, "freqs[%d] is not finite or beyond 1e6", j);
        p->frac[j] = turns_fraction(freqs[j]);
    }
    p->n_axes = n_axes;
    p->n_pairs = rot / 2;
    for (int u = rot / 16; halves && u < D / 16; ++u) {  // copied
        p->unit_first[u] = (uint8_t)(16 * u);
        p->unit_half[u] = 8;
    }
    return 0;
}

inline int span_limits(int left, int right, int sinks, SpanParams *p) {
    if (left < -1 || right < -1) return api_fail(XS_ERR_SHAPE, "left and right must be >= 0, or -1 for no limit");
    if (sinks < 0) return api_fail(XS_ERR_SHAPE, "sinks must be >= 0");
    const int far = 1 << 29;  // past every place
    p->left = left < 0 || left > far ? far : left;
    p->right = right < 0 || right > far ? far : right;
    p->sinks = sinks > far ? far : sinks;
    return 0;
}
inline int check_scale(float scale) {
    if (!std::isfinite(scale) || !(scale > 0.0f)) return api_fail(XS_ERR_SHAPE, "scale must be positive and finite");
    return 0;
}
inline int check_workspace(const void *ws, size_t bytes, const Buffer *others, int n) {
    if (!ws && bytes) return api_fail(XS_ERR_WORKSPACE, "workspace is NULL but workspace_bytes is %zu", bytes);
    if (!ws) return 0;
    if (((uintptr_t)ws & 255u) != 0) return api_fail(XS_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    for (int i = 0; i < n; ++i)
        if (api_overlaps(ws, bytes, others[i].ptr, others[i].bytes))
            return api_fail(XS_ERR_WORKSPACE, "workspace overlaps %s", others[i].name);
    return 0;
}
inline float scale_log2(float scale) { return (float)((double)scale * 1.4426950408889634073599246810019); }

// Shape rules of the paged cache; the sizes of one pool and of the table in bytes.
inline int check_cache(int N, int T, int Hk, int D, int page, int n_pages, int max_pages, size_t *pool, size_t *table) {
    if (N < 0 || T < 0) return api_fail(XS_ERR_SHAPE, "N and T must be >= 0 (got N=%d T=%d)", N, T);
    if (Hk < 1 || n_pages < 1 || max_pages < 1)
        return api_fail(XS_ERR_SHAPE, "Hk, n_pages and max_pages must be >= 1 (got %d, %d, %d)", Hk, n_pages, max_pages);
    if (D != 64 && D != 96 && D != 128)
        return api_fail(XS_ERR_UNSUPPORTED, "the paged cache takes D = 64, 96 or 128 (got D=%d)", D);
    if (page < 16 || page > 1024 || (page & (page - 1)))
        return api_fail(XS_ERR_UNSUPPORTED, "page=%d is not a power of two from 16 to 1024", page);
    if ((long long)max_pages * page > (1ll << 29))
        return api_fail(XS_ERR_SHAPE, "max_pages * page = %lld exceeds 2^29 keys", (long long)max_pages * page);
    const unsigned long long rows = (unsigned long long)n_pages * page;
    if (Hk > (1 << 16) || rows * (unsigned long long)Hk * D * 2 >= (1ull << 40))
        return api_fail(XS_ERR_SHAPE, "a pool of %d pages exceeds 2^40 bytes", n_pages);
    if (T > (1 << 29)) return api_fail(XS_ERR_SHAPE, "T=%d exceeds 2^29 rows", T);
    if (N > (1 << 16)) return api_fail(XS_ERR_SHAPE, "N=%d exceeds 65536 sequences", N);
    *pool = (size_t)rows * Hk * D * 2;
    *table = (size_t)N * max_pages * sizeof(int);
    return 0;
}
// The query heads of the attention over it.
inline int check_heads(int T, int H, int Hk) {
    if (H < 1 || H % Hk) return api_fail(XS_ERR_SHAPE, "H=%d is not a positive multiple of Hk=%d", H, Hk);
    if (H / Hk > 128) return api_fail(XS_ERR_UNSUPPORTED, "H/Hk=%d query heads a key head exceed 128", H / Hk);
    if ((long long)T * H >= (1ll << 31)) return api_fail(XS_ERR_SHAPE, "T * H exceeds 2^31-1 rows");
    return 0;
}

// Rows, tiles and tensor maps of attention over a paged cache (everything but the pointers and the
// span of keys).
inline int span_paged(const void *q, const void *k_pages, const void *v_pages, int N, int T, int H, int Hk, int D, int page,
                      int n_pages, int max_pages, SpanParams *p, SpanMaps *maps) {
    p->N = N;
    p->T = T;
    p->H = H;
    p->Hk = Hk;
    p->G = H / Hk;
    p->page = page;
    p->n_pages = n_pages;
    p->max_pages = max_pages;
    // Few rows: batches of mostly single new tokens. The rows that a sequence and key head
    // have on average decide (the lengths are on the device); a longer sequence among them takes
    // an item for each tile of 16 or 32 rows, each of which walks all its keys. Tiles of 16, 32
    // and 128 rows, us, 8 key heads:
    //   rows  16 x 4000 keys D = 128  16 x 4000 D = 64   16 x 1000 D = 128  4 x 1000 D = 64
    //     8     48.6   49.2   52.9     33.0  34.9  36.0
    //    16     49.7   50.9   53.5     34.2  36.5  36.2   19.2  22.6  20.1   12.9  14.0  12.3
    //    20            52.8   55.7           37.8  36.5         23.5  20.3         14.7  12.4
    //    24            53.9   55.2           38.9  36.4         24.8  20.4         15.3  12.5
    //    32            57.8   55.8           42.5  36.3         27.7  21.0         17.8  12.7
    // and with more parts an item 32 gains more: 3 x 20000, 2 heads, 20 rows, D = 128 21.4 us, 25.7 with
    // tiles of 128. A chunk among single tokens costs: 64 of them over 1000 keys with 400 tokens over 8000
    // (G = 4, so 29 rows) took 244 us in tiles of 32 and 92 in tiles of 128, apart 50 and 52.
    // Trees take tiles of 16 and of 128 rows only, masks of 32 rows a thread costing what they save: 16, 32 and 128, us, 8 key
    // heads, D = 128: 16 rows, 16 x 4000 keys 51.0, -, 54.0 (D = 64 33.2, -, 35.1); 24 rows -, 55.3, 55.0, 4 x 1000 -, 16.8, 14.0;
    // 32 rows -, 58.9, 55.0 and -, 19.5, 14.3.
    const long long rows_avg = ((long long)T * p->G + N - 1) / N;
    p->few = p->G <= 16 && rows_avg <= 16 ? 16 : p->kind == SPAN_PAGED && D > 64 && p->G <= 32 && rows_avg <= 24 ? 32 : 0;
    p->tile_tok = (p->few ? p->few : 128) / p->G;
    p->item_tok = p->few ? p->tile_tok : 2 * p->tile_tok;
    for (p->page_log2 = 4; 1 << p->page_log2 < page;) ++p->page_log2;
    p->g_magic = (65536u + (uint32_t)p->G - 1u) / (uint32_t)p->G;
    p->heads = Hk;
    const uint64_t d = (uint64_t)D * 2;
    const uint64_t q_dims[4] = {(uint64_t)D, (uint64_t)p->G, (uint64_t)Hk, (uint64_t)T};
    const uint64_t q_strides[3] = {d, p->G * d, H * d};
    const uint32_t q_box[4] = {64, (uint32_t)p->G, 1, (uint32_t)p->tile_tok};
    const uint64_t kv_dims[4] = {(uint64_t)D, (uint64_t)Hk, (uint64_t)page, (uint64_t)n_pages};
    const uint64_t kv_strides[3] = {d, Hk * d, page * Hk * d};
    const uint32_t kv_box[4] = {64, 1, (uint32_t)(page < 128 ? page : 128), 1};
    int st = api_tile_map(&maps->q, q, q_dims, q_strides, q_box, "q");
    if (!st) st = api_tile_map(&maps->k, k_pages, kv_dims, kv_strides, kv_box, "k_pages");
    if (!st) st = api_tile_map(&maps->v, v_pages, kv_dims, kv_strides, kv_box, "v_pages");
    return st;
}

}  // namespace xs
