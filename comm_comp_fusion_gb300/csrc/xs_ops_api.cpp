// xs_ops_api.cpp -- the C ABI of the operators around the fused attention:
// rotary positions, windowed attention, the paged cache and attention over it.
// Arguments are checked before any CUDA call, like in xs_api.cpp.
#include "../../include/xs.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "xs_internal.h"

namespace {

using namespace xs;

bool misaligned16(const void *p) { return ((uintptr_t)p & 15u) != 0; }
bool misaligned4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

struct Buffer {
    const void *ptr;
    size_t bytes;
    const char *name;
};

// No buffer of `out` may overlap one of `in` or another of `out`.
int check_disjoint(const Buffer *out, int n_out, const Buffer *in, int n_in) {
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
int check_device(const Buffer *b, int n, int dev) {
    for (int i = 0; i < n; ++i)
        if (b[i].bytes)
            if (const int st = api_device_pointer(b[i].ptr, dev, b[i].name)) return st;
    return 0;
}

// f (radians per unit of place) in turns, modulo 1, as a 64-bit binary fraction
// (two's complement for a negative f). |f| / 2 pi is formed in double-double
// arithmetic (1 / 2 pi in two doubles), so the fraction is as exact as f.
uint64_t turns_fraction(double f) {
    const double hi_c = 0.15915494309189535, lo_c = -9.839338337591243e-18;  // 1 / 2 pi
    const double x = std::fabs(f), hi = x * hi_c, lo = std::fma(x, hi_c, -hi) + x * lo_c;
    const double frac = hi - std::floor(hi);  // exact, below 1
    const uint64_t u = (uint64_t)std::ldexp(frac, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(lo, 64));
    return f < 0 ? 0 - u : u;
}

int span_limits(int left, int right, int sinks, SpanParams *p) {
    if (left < -1 || right < -1) return api_fail(XS_ERR_SHAPE, "left and right must be >= 0, or -1 for no limit");
    if (sinks < 0) return api_fail(XS_ERR_SHAPE, "sinks must be >= 0");
    const int far = 1 << 29;  // past every place
    p->left = left < 0 || left > far ? far : left;
    p->right = right < 0 || right > far ? far : right;
    p->sinks = sinks > far ? far : sinks;
    return 0;
}
int check_scale(float scale) {
    if (!std::isfinite(scale) || !(scale > 0.0f)) return api_fail(XS_ERR_SHAPE, "scale must be positive and finite");
    return 0;
}
int check_workspace(const void *ws, size_t bytes, const Buffer *others, int n) {
    if (!ws && bytes) return api_fail(XS_ERR_WORKSPACE, "workspace is NULL but workspace_bytes is %zu", bytes);
    if (!ws) return 0;
    if (((uintptr_t)ws & 255u) != 0) return api_fail(XS_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    for (int i = 0; i < n; ++i)
        if (api_overlaps(ws, bytes, others[i].ptr, others[i].bytes))
            return api_fail(XS_ERR_WORKSPACE, "workspace overlaps %s", others[i].name);
    return 0;
}
float scale_log2(float scale) { return (float)((double)scale * 1.4426950408889634073599246810019); }

// Most K/V tiles of a query tile pair without a workspace: 2^20 keys, after which a sum in
// tensor memory, whose additions truncate, has lost about half a bf16 step. (With a workspace it is
// taken in stretches.)
constexpr int kStepsWithoutWorkspace = 1 << 13;

// K/V tiles that the two query tiles of pair i of a whole sequence walk.
int pair_steps(const SpanParams &p, int i) {
    const int tok = 256 * i, last = std::min(tok + 255, p.S - 1);
    const int hi = std::min(p.S - 1, last + p.right), lo = std::max(0, tok - p.left) / 128;
    return hi / 128 - lo + 1 + std::min((std::min(p.sinks, hi + 1) + 127) / 128, lo);
}

// Whether to take a CTA for each pair of query tiles, none cut: if that makes the longest
// part at most three steps longer than an even split of all steps (in parts of four and
// more), since pieces, their schedule and merge cost as much, or seven where the split would
// keep half the SMs and more busy with pieces, whose traffic then counts. 30 heads of S =
// 1000, causal, D = 128 (8 steps against 4): 19.2 us whole, 22.7 split; 20 of S = 1500 (12
// against 5) 24.3, 28.3; 4 of S = 1000, D = 64 (8 against 4, 32 parts) 17.2, 15.2; 8 of S =
// 1500 (12 against 4) 24.0, 21.6.
bool whole_pairs(const SpanParams &p, int sms) {
    if ((long long)p.heads * p.n_pairs > sms) return false;
    long long sum = 0;
    int most = 0;
    for (int i = 0; i < p.n_pairs; ++i) {
        const int n = pair_steps(p, i);
        sum += n;
        most = std::max(most, n);
    }
    sum *= p.heads;
    return most <= std::max(sum / sms, 4ll) + (sum >= 2ll * sms ? 7 : 3);
}

// Shape rules of the windowed calls; the size of one tensor in bytes.
int check_window(int B, int S, int H, int D, int P, size_t *bytes) {
    if (const int st = api_shape(B, S, H, D, P, bytes)) return st;
    if (D == 256) return api_fail(XS_ERR_UNSUPPORTED, "windowed attention takes D = 64, 96 or 128 (got D=256)");
    if (S > (1 << 24)) return api_fail(XS_ERR_SHAPE, "S=%d exceeds 2^24", S);
    return 0;
}

int window_call(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D, int P, float scale,
                int left, int right, int sinks, void *ws, size_t ws_bytes, void *stream, bool a2a) {
    if (!q || !k || !v || !out) return api_fail(XS_ERR_NULL, "q, k, v and out must be non-NULL");
    size_t bytes = 0;
    int st = check_window(B, S, H, D, P, &bytes);
    if (st || (st = check_scale(scale))) return st;
    SpanParams p{};
    if ((st = span_limits(left, right, sinks, &p))) return st;
    if (misaligned16(q) || misaligned16(k) || misaligned16(v) || misaligned16(out))
        return api_fail(XS_ERR_ALIGN, "q, k, v and out must be 16-byte aligned");
    const Buffer in[3] = {{q, bytes, "q"}, {k, bytes, "k"}, {v, bytes, "v"}}, o = {out, bytes, "out"};
    if ((st = check_disjoint(&o, 1, in, 3))) return st;
    const Buffer all[4] = {in[0], in[1], in[2], o};
    if ((st = check_workspace(ws, ws_bytes, all, 4))) return st;
    if (bytes == 0) return XS_OK;
    p.S = S;
    p.n_pairs = (S + 255) / 256;
    for (int i = 0; !ws && S > 128 * kStepsWithoutWorkspace && i < p.n_pairs; ++i)
        if (pair_steps(p, i) > kStepsWithoutWorkspace)
            return api_fail(XS_ERR_WORKSPACE, "query tiles that walk over more than 2^20 keys need a workspace");
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(all, 4, dev))) return st;
    if (ws) {
        const size_t need = span_workspace_bytes(D, sms);
        if (ws_bytes < need)
            return api_fail(XS_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes, need);
        if ((st = api_device_pointer(ws, dev, "workspace"))) return st;
    }
    p.out = static_cast<uint16_t *>(out);
    p.T = S;
    p.H = H;
    p.G = 1;
    p.B = B;
    p.P = P;
    p.Hl = H / P;
    p.Sl = S / P;
    p.head_out = a2a ? 0 : 1;
    p.scale_log2 = scale_log2(scale);
    p.tile_tok = 128;
    p.item_tok = 256;
    p.heads = B * H;
    if (ws && !whole_pairs(p, sms)) span_workspace_parts(ws, D, sms, &p);
    SpanMaps maps;
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.Hl, (uint64_t)S, (uint64_t)P * B};
    const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)p.Hl * D * 2, (uint64_t)S * p.Hl * D * 2};
    const uint32_t box[4] = {64, 1, 128, 1};
    if ((st = api_tile_map(&maps.q, q, dims, strides, box, "q")) ||
        (st = api_tile_map(&maps.k, k, dims, strides, box, "k")) ||
        (st = api_tile_map(&maps.v, v, dims, strides, box, "v")))
        return st;
    const cudaError_t e = launch_span(D, maps, p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? (int)XS_OK : api_cuda_error("windowed attention launch", e);
}

// Shape rules of the paged cache; the sizes of one pool and of the table in bytes.
int check_cache(int N, int T, int Hk, int D, int page, int n_pages, int max_pages, size_t *pool, size_t *table) {
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
int check_heads(int T, int H, int Hk) {
    if (H < 1 || H % Hk) return api_fail(XS_ERR_SHAPE, "H=%d is not a positive multiple of Hk=%d", H, Hk);
    if (H / Hk > 128) return api_fail(XS_ERR_UNSUPPORTED, "H/Hk=%d query heads a key head exceed 128", H / Hk);
    if ((long long)T * H >= (1ll << 31)) return api_fail(XS_ERR_SHAPE, "T * H exceeds 2^31-1 rows");
    return 0;
}

}  // namespace

extern "C" {

xs_status xs_rope(const void *q, const void *k, void *q_out, void *k_out, const int32_t *pos, int pos_batches, int B,
                  int S, int H, int Hk, int D, int P, int n_axes, const int *axis_dims, const double *freqs, int flags,
                  void *stream) {
    if (!q || !q_out || !pos || !axis_dims || !freqs)
        return (xs_status)api_fail(XS_ERR_NULL, "q, q_out, pos, axis_dims and freqs must be non-NULL");
    if (Hk < 0) return (xs_status)api_fail(XS_ERR_SHAPE, "Hk must be >= 0 (got %d)", Hk);
    if (Hk > 0 && (!k || !k_out)) return (xs_status)api_fail(XS_ERR_NULL, "k and k_out must be non-NULL unless Hk is 0");
    size_t qb = 0, kb = 0;
    int st = api_shape(B, S, H, D, P, &qb);
    if (!st && Hk > 0) st = api_shape(B, S, Hk, D, P, &kb);
    if (st) return (xs_status)st;
    if (H + Hk > (1 << 16)) return (xs_status)api_fail(XS_ERR_SHAPE, "H + Hk = %d exceeds 65536 heads", H + Hk);
    if (n_axes < 1 || n_axes > kRopeMaxAxes)
        return (xs_status)api_fail(XS_ERR_SHAPE, "n_axes must be 1 to %d (got %d)", kRopeMaxAxes, n_axes);
    if (pos_batches != 1 && pos_batches != B)
        return (xs_status)api_fail(XS_ERR_SHAPE, "pos_batches must be 1 or B (got %d)", pos_batches);
    if (flags & ~(XS_ROPE_HALVES | XS_ROPE_INVERSE | XS_ROPE_IN_SEQ | XS_ROPE_OUT_SEQ))
        return (xs_status)api_fail(XS_ERR_SHAPE, "unknown flags 0x%x", flags);
    const bool halves = flags & XS_ROPE_HALVES;
    RopeParams p;
    memset(&p, 0, sizeof p);
    int rot = 0;
    for (int a = 0; a < n_axes; ++a) {
        const int d = axis_dims[a];
        if (d < 2 || d > D || d % 2)
            return (xs_status)api_fail(XS_ERR_SHAPE, "axis_dims[%d]=%d is not an even number from 2 to D", a, d);
        if (halves && d % 16)
            return (xs_status)api_fail(XS_ERR_UNSUPPORTED,
                                       "pairs half an axis apart need axis_dims in multiples of 16 (axis_dims[%d]=%d)", a, d);
        if (rot + d > D) return (xs_status)api_fail(XS_ERR_SHAPE, "axis_dims add up to more than D=%d", D);
        for (int j = 0; j < d / 2; ++j) p.axis[rot / 2 + j] = (uint8_t)a;
        for (int u = 0; halves && u < d / 16; ++u) {
            p.unit_first[rot / 16 + u] = (uint8_t)(rot + 8 * u);
            p.unit_half[rot / 16 + u] = (uint8_t)(d / 2);
        }
        rot += d;
    }
    for (int j = 0; j < rot / 2; ++j) {
        if (!std::isfinite(freqs[j]) || std::fabs(freqs[j]) > 1e6)
            return (xs_status)api_fail(XS_ERR_SHAPE, "freqs[%d] is not finite or beyond 1e6", j);
        p.frac[j] = turns_fraction(freqs[j]);
    }
    p.n_pairs = rot / 2;
    for (int u = rot / 16; halves && u < D / 16; ++u) {  // copied
        p.unit_first[u] = (uint8_t)(16 * u);
        p.unit_half[u] = 8;
    }
    p.seq_in = flags & XS_ROPE_IN_SEQ;
    p.seq_out = flags & XS_ROPE_OUT_SEQ;
    p.inverse = flags & XS_ROPE_INVERSE;
    if (misaligned16(q) || misaligned16(q_out) || (Hk && (misaligned16(k) || misaligned16(k_out))))
        return (xs_status)api_fail(XS_ERR_ALIGN, "q, k, q_out and k_out must be 16-byte aligned");
    if (misaligned4(pos)) return (xs_status)api_fail(XS_ERR_ALIGN, "pos must be 4-byte aligned");
    const Buffer Q = {q, qb, "q"}, K = {k, kb, "k"}, QO = {q_out, qb, "q_out"}, KO = {k_out, kb, "k_out"};
    const Buffer POS = {pos, (size_t)pos_batches * S * n_axes * 4, "pos"};
    const bool in_place_ok = p.seq_in == p.seq_out || P == 1;
    const Buffer in_q[3] = {in_place_ok && q_out == q ? Buffer{q, 0, "q"} : Q, K, POS};
    const Buffer in_k[4] = {Q, in_place_ok && k_out == k ? Buffer{k, 0, "k"} : K, POS, QO};
    if ((st = check_disjoint(&QO, 1, in_q, Hk ? 3 : 1)) || (!Hk && (st = check_disjoint(&QO, 1, &POS, 1))) ||
        (Hk && (st = check_disjoint(&KO, 1, in_k, 4))))
        return (xs_status)st;
    if (qb == 0) return XS_OK;
    int dev, sms;
    const Buffer all[5] = {Q, QO, K, KO, POS};
    if ((st = api_device(&dev, &sms)) || (st = check_device(all, 5, dev))) return (xs_status)st;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.pos = pos;
    p.pos_batch = pos_batches == 1 ? 0 : S;
    p.B = B;
    p.S = S;
    p.H = H;
    p.Hk = Hk;
    p.Hl = H / P;
    p.Hkl = Hk / P;
    p.Sl = S / P;
    p.D = D;
    p.n_axes = n_axes;
    const cudaError_t e = launch_rope(p, halves, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("rotary launch", e);
}

xs_status xs_attn_window(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D, int P,
                         float scale, int left, int right, int sinks, void *workspace, size_t workspace_bytes,
                         void *stream) {
    return (xs_status)window_call(q, k, v, out, B, S, H, D, P, scale, left, right, sinks, workspace, workspace_bytes,
                                  stream, false);
}

xs_status xs_attn_window_a2a(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D, int P,
                             float scale, int left, int right, int sinks, void *workspace, size_t workspace_bytes,
                             void *stream) {
    return (xs_status)window_call(q, k, v, out, B, S, H, D, P, scale, left, right, sinks, workspace, workspace_bytes,
                                  stream, true);
}

xs_status xs_attn_window_workspace_size(int B, int S, int H, int D, int P, size_t *bytes) {
    if (!bytes) return (xs_status)api_fail(XS_ERR_NULL, "bytes must be non-NULL");
    size_t tb = 0;
    int st = check_window(B, S, H, D, P, &tb);
    if (st) return (xs_status)st;
    *bytes = 0;
    if (tb == 0) return XS_OK;
    int dev, sms;
    if ((st = api_device(&dev, &sms))) return (xs_status)st;
    *bytes = span_workspace_bytes(D, sms);
    return XS_OK;
}

xs_status xs_cache_append(const void *k, const void *v, void *k_pages, void *v_pages, const int32_t *page_table,
                          const int32_t *q_start, const int32_t *kv_len, int N, int T, int Hk, int D, int page,
                          int n_pages, int max_pages, void *stream) {
    if (!k || !v || !k_pages || !v_pages || !page_table || !q_start || !kv_len)
        return (xs_status)api_fail(XS_ERR_NULL, "k, v, k_pages, v_pages, page_table, q_start and kv_len must be non-NULL");
    size_t pool, table;
    int st = check_cache(N, T, Hk, D, page, n_pages, max_pages, &pool, &table);
    if (st) return (xs_status)st;
    if ((long long)T * Hk >= (1ll << 31)) return (xs_status)api_fail(XS_ERR_SHAPE, "T * Hk exceeds 2^31-1 rows");
    if (misaligned16(k) || misaligned16(v) || misaligned16(k_pages) || misaligned16(v_pages))
        return (xs_status)api_fail(XS_ERR_ALIGN, "k, v, k_pages and v_pages must be 16-byte aligned");
    if (misaligned4(page_table) || misaligned4(q_start) || misaligned4(kv_len))
        return (xs_status)api_fail(XS_ERR_ALIGN, "page_table, q_start and kv_len must be 4-byte aligned");
    const size_t rows = (size_t)T * Hk * D * 2;
    const Buffer out[2] = {{k_pages, pool, "k_pages"}, {v_pages, pool, "v_pages"}};
    const Buffer in[5] = {{k, rows, "k"}, {v, rows, "v"}, {page_table, table, "page_table"},
                          {q_start, (size_t)(N + 1) * 4, "q_start"}, {kv_len, (size_t)N * 4, "kv_len"}};
    if ((st = check_disjoint(out, 2, in, 5))) return (xs_status)st;
    if (N == 0 || T == 0) return XS_OK;
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(out, 2, dev)) || (st = check_device(in, 5, dev)))
        return (xs_status)st;
    AppendParams p;
    p.k = static_cast<const uint4 *>(k);
    p.v = static_cast<const uint4 *>(v);
    p.k_pages = static_cast<uint4 *>(k_pages);
    p.v_pages = static_cast<uint4 *>(v_pages);
    p.table = page_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.N = N;
    p.T = T;
    p.chunks = Hk * D / 8;
    p.page = page;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    const cudaError_t e = launch_append(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("cache append launch", e);
}

xs_status xs_attn_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                        const int32_t *q_start, const int32_t *kv_len, void *out, int N, int T, int H, int Hk, int D,
                        int page, int n_pages, int max_pages, float scale, int left, int right, int sinks,
                        void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k_pages || !v_pages || !page_table || !q_start || !kv_len || !out)
        return (xs_status)api_fail(XS_ERR_NULL, "q, k_pages, v_pages, page_table, q_start, kv_len and out must be non-NULL");
    size_t pool, table;
    int st = check_cache(N, T, Hk, D, page, n_pages, max_pages, &pool, &table);
    if (st) return (xs_status)st;
    if ((st = check_heads(T, H, Hk)) || (st = check_scale(scale))) return (xs_status)st;
    SpanParams p{};
    if ((st = span_limits(left, right, sinks, &p))) return (xs_status)st;
    if (misaligned16(q) || misaligned16(k_pages) || misaligned16(v_pages) || misaligned16(out))
        return (xs_status)api_fail(XS_ERR_ALIGN, "q, k_pages, v_pages and out must be 16-byte aligned");
    if (misaligned4(page_table) || misaligned4(q_start) || misaligned4(kv_len))
        return (xs_status)api_fail(XS_ERR_ALIGN, "page_table, q_start and kv_len must be 4-byte aligned");
    const size_t rows = (size_t)T * H * D * 2;
    const Buffer o = {out, rows, "out"};
    const Buffer in[6] = {{q, rows, "q"}, {k_pages, pool, "k_pages"}, {v_pages, pool, "v_pages"},
                          {page_table, table, "page_table"}, {q_start, (size_t)(N + 1) * 4, "q_start"},
                          {kv_len, (size_t)N * 4, "kv_len"}};
    const Buffer all[7] = {o, in[0], in[1], in[2], in[3], in[4], in[5]};
    if ((st = check_disjoint(&o, 1, in, 6)) || (st = check_workspace(workspace, workspace_bytes, all, 7)))
        return (xs_status)st;
    if (N == 0 || T == 0) return XS_OK;
    if (!workspace) return (xs_status)api_fail(XS_ERR_NULL, "workspace must be non-NULL");
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(all, 7, dev))) return (xs_status)st;
    const size_t need = span_workspace_bytes(D, sms);
    if (workspace_bytes < need)
        return (xs_status)api_fail(XS_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed",
                                   workspace_bytes, need);
    if ((st = api_device_pointer(workspace, dev, "workspace"))) return (xs_status)st;
    p.out = static_cast<uint16_t *>(out);
    p.table = page_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.N = N;
    p.T = T;
    p.H = H;
    p.Hk = Hk;
    p.G = H / Hk;
    p.page = page;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.scale_log2 = scale_log2(scale);
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
    const long long rows_avg = ((long long)T * p.G + N - 1) / N;
    p.few = p.G <= 16 && rows_avg <= 16 ? 16 : D > 64 && p.G <= 32 && rows_avg <= 24 ? 32 : 0;
    p.tile_tok = (p.few ? p.few : 128) / p.G;
    p.item_tok = p.few ? p.tile_tok : 2 * p.tile_tok;
    for (p.page_log2 = 4; 1 << p.page_log2 < page;) ++p.page_log2;
    p.g_magic = (65536u + (uint32_t)p.G - 1u) / (uint32_t)p.G;
    p.heads = Hk;
    span_workspace_parts(workspace, D, sms, &p);
    SpanMaps maps;
    const uint64_t d = (uint64_t)D * 2;
    const uint64_t q_dims[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)Hk, (uint64_t)T};
    const uint64_t q_strides[3] = {d, p.G * d, H * d};
    const uint32_t q_box[4] = {64, (uint32_t)p.G, 1, (uint32_t)p.tile_tok};
    const uint64_t kv_dims[4] = {(uint64_t)D, (uint64_t)Hk, (uint64_t)page, (uint64_t)n_pages};
    const uint64_t kv_strides[3] = {d, Hk * d, page * Hk * d};
    const uint32_t kv_box[4] = {64, 1, (uint32_t)(page < 128 ? page : 128), 1};
    if ((st = api_tile_map(&maps.q, q, q_dims, q_strides, q_box, "q")) ||
        (st = api_tile_map(&maps.k, k_pages, kv_dims, kv_strides, kv_box, "k_pages")) ||
        (st = api_tile_map(&maps.v, v_pages, kv_dims, kv_strides, kv_box, "v_pages")))
        return (xs_status)st;
    const cudaError_t e = launch_span(D, maps, p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("paged attention launch", e);
}

xs_status xs_attn_paged_workspace_size(int N, int T, int H, int Hk, int D, size_t *bytes) {
    if (!bytes) return (xs_status)api_fail(XS_ERR_NULL, "bytes must be non-NULL");
    size_t pool, table;
    int st = check_cache(N, T, Hk, D, 16, 1, 1, &pool, &table);
    if (st) return (xs_status)st;
    if ((st = check_heads(T, H, Hk))) return (xs_status)st;
    *bytes = 0;
    if (N == 0 || T == 0) return XS_OK;
    int dev, sms;
    if ((st = api_device(&dev, &sms))) return (xs_status)st;
    *bytes = span_workspace_bytes(D, sms);
    return XS_OK;
}

}  // extern "C"
