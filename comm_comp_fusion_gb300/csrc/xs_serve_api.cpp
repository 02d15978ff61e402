// xs_serve_api.cpp -- the C ABI of the operators of a serving step around the paged
// cache: rotation on the way into the cache, drafted trees, packed prompts.
// Arguments are checked before any CUDA call, like in xs_api.cpp.
#include <cstring>

#include "xs_ops_checks.h"

namespace {

using namespace xs;

constexpr int64_t kMaxStride = 1 << 30;

// Elements from one token's row to the next (0: its heads lie one after the other), and the bytes
// that T rows span.
int check_rows(const char *name, int T, int heads, int D, int64_t *stride, size_t *bytes) {
    const int64_t row = (int64_t)heads * D;
    if (*stride == 0) *stride = row;
    if (*stride < row || *stride > kMaxStride || *stride % 8)
        return api_fail(XS_ERR_SHAPE, "%s_stride=%lld is not a multiple of 8 from %lld to 2^30", name, (long long)*stride,
                        (long long)row);
    *bytes = T && heads ? ((size_t)(T - 1) * (size_t)*stride + (size_t)row) * 2 : 0;
    return 0;
}

// Shape rules of the packed prompts.
int check_packed(int N, int T, int H, int Hk, int D) {
    if (N < 0 || T < 0) return api_fail(XS_ERR_SHAPE, "N and T must be >= 0 (got N=%d T=%d)", N, T);
    if (Hk < 1 || Hk > (1 << 16)) return api_fail(XS_ERR_SHAPE, "Hk must be 1 to 65536 (got %d)", Hk);
    if (D != 64 && D != 96 && D != 128)
        return api_fail(XS_ERR_UNSUPPORTED, "packed attention takes D = 64, 96 or 128 (got D=%d)", D);
    if (T > (1 << 29)) return api_fail(XS_ERR_SHAPE, "T=%d exceeds 2^29 rows", T);
    if (N > (1 << 16)) return api_fail(XS_ERR_SHAPE, "N=%d exceeds 65536 sequences", N);
    return check_heads(T, H, Hk);
}

int check_words(int words) {
    if (words < 1 || words > kTreeMaxWords)
        return api_fail(XS_ERR_SHAPE, "words must be 1 to %d (got %d)", kTreeMaxWords, words);
    return 0;
}

// The workspace's place and size, once the device is known.
int check_workspace_size(const void *ws, size_t bytes, size_t need, int dev) {
    if (bytes < need)
        return api_fail(XS_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", bytes, need);
    return api_device_pointer(ws, dev, "workspace");
}

}  // namespace

extern "C" {

xs_status xs_cache_append_rope(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, void *q_out, void *k_out, void *k_pages, void *v_pages,
                               const int32_t *page_table, const int32_t *q_start, const int32_t *kv_len,
                               const int32_t *pos, int N, int T, int H, int Hk, int D, int page, int n_pages,
                               int max_pages, int n_axes, const int *axis_dims, const double *freqs, int flags,
                               void *stream) {
    const bool work = N && T;
    if (!axis_dims || !freqs || (work && (!k || !v || !k_pages || !v_pages || !page_table || !q_start || !kv_len)))
        return (xs_status)api_fail(XS_ERR_NULL, "k, v, k_pages, v_pages, page_table, q_start, kv_len, axis_dims and freqs "
                                                "must be non-NULL");
    if (H < 0) return (xs_status)api_fail(XS_ERR_SHAPE, "H must be >= 0 (got %d)", H);
    if (work && H > 0 && (!q || !q_out)) return (xs_status)api_fail(XS_ERR_NULL, "q and q_out must be non-NULL unless H is 0");
    size_t pool, table, qb, kb, vb;
    int st = check_cache(N, T, Hk, D, page, n_pages, max_pages, &pool, &table);
    if (st) return (xs_status)st;
    if ((long long)H + Hk > (1 << 16)) return (xs_status)api_fail(XS_ERR_SHAPE, "H + Hk = %lld exceeds 65536 heads", (long long)H + Hk);
    if ((long long)T * std::max(H, Hk) >= (1ll << 31)) return (xs_status)api_fail(XS_ERR_SHAPE, "T * max(H, Hk) exceeds 2^31-1 rows");
    if ((H && (st = check_rows("q", T, H, D, &q_stride, &qb))) || (st = check_rows("k", T, Hk, D, &k_stride, &kb)) ||
        (st = check_rows("v", T, Hk, D, &v_stride, &vb)))
        return (xs_status)st;
    if (flags & ~XS_ROPE_HALVES) return (xs_status)api_fail(XS_ERR_SHAPE, "unknown flags 0x%x", flags);
    AppendRopeParams p;
    memset(&p, 0, sizeof p);
    if ((st = rope_table(n_axes, axis_dims, freqs, (flags & XS_ROPE_HALVES) != 0, D, &p))) return (xs_status)st;
    if (work && !pos && n_axes > 1) return (xs_status)api_fail(XS_ERR_NULL, "pos must be non-NULL with more than one axis");
    if ((H && (misaligned16(q) || misaligned16(q_out))) || misaligned16(k) || misaligned16(v) || misaligned16(k_out) ||
        misaligned16(k_pages) || misaligned16(v_pages))
        return (xs_status)api_fail(XS_ERR_ALIGN, "q, k, v, q_out, k_out, k_pages and v_pages must be 16-byte aligned");
    if (misaligned4(page_table) || misaligned4(q_start) || misaligned4(kv_len) || misaligned4(pos))
        return (xs_status)api_fail(XS_ERR_ALIGN, "page_table, q_start, kv_len and pos must be 4-byte aligned");
    if (!H) q = nullptr, q_out = nullptr, qb = 0;
    const size_t q_rows = (size_t)T * H * D * 2, k_rows = (size_t)T * Hk * D * 2;
    // in place: a row is written by the threads that have read it
    const bool q_same = q_out == q && q_stride == (int64_t)H * D, k_same = k_out == k && k_stride == (int64_t)Hk * D;
    const Buffer Q = {q, qb, "q"}, K = {k, kb, "k"}, V = {v, vb, "v"};
    const Buffer out[4] = {{k_pages, pool, "k_pages"}, {v_pages, pool, "v_pages"}, {q_out, q_rows, "q_out"},
                           {k_out, k_out ? k_rows : 0, "k_out"}};
    const Buffer in[7] = {{page_table, table, "page_table"}, {q_start, (size_t)(N + 1) * 4, "q_start"},
                          {kv_len, (size_t)N * 4, "kv_len"}, {pos, pos ? (size_t)T * n_axes * 4 : 0, "pos"}, V, Q, K};
    Buffer in_q[7], in_k[7];
    for (int i = 0; i < 7; ++i) in_q[i] = in_k[i] = in[i];
    if (q_same) in_q[5].bytes = 0;
    if (k_same) in_k[6].bytes = 0;
    if ((st = check_disjoint(out, 4, in, 5)) || (st = check_disjoint(out, 2, in, 7)) ||
        (st = check_disjoint(out + 2, 1, in_q, 7)) || (st = check_disjoint(out + 3, 1, in_k, 7)))
        return (xs_status)st;
    if (N == 0 || T == 0) return XS_OK;
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(out, 4, dev)) || (st = check_device(in, 7, dev)))
        return (xs_status)st;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.k_pages = static_cast<uint16_t *>(k_pages);
    p.v_pages = static_cast<uint16_t *>(v_pages);
    p.table = page_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.pos = pos;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.N = N;
    p.T = T;
    p.H = H;
    p.Hk = Hk;
    p.page = page;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    const cudaError_t e = launch_append_rope(p, D, (flags & XS_ROPE_HALVES) != 0, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("rotary cache append launch", e);
}

xs_status xs_tree_mask(const int32_t *parents, const int32_t *q_start, const int32_t *kv_len, int32_t *mask, int32_t *pos,
                       int N, int T, int words, void *stream) {
    const bool work = N && T;
    if (work && (!parents || !q_start || !mask))
        return (xs_status)api_fail(XS_ERR_NULL, "parents, q_start and mask must be non-NULL");
    if (work && pos && !kv_len) return (xs_status)api_fail(XS_ERR_NULL, "kv_len must be non-NULL unless pos is NULL");
    if (N < 0 || T < 0) return (xs_status)api_fail(XS_ERR_SHAPE, "N and T must be >= 0 (got N=%d T=%d)", N, T);
    if (N > (1 << 16)) return (xs_status)api_fail(XS_ERR_SHAPE, "N=%d exceeds 65536 sequences", N);
    if (T > (1 << 29)) return (xs_status)api_fail(XS_ERR_SHAPE, "T=%d exceeds 2^29 rows", T);
    int st = check_words(words);
    if (st) return (xs_status)st;
    if (misaligned4(parents) || misaligned4(q_start) || misaligned4(kv_len) || misaligned4(mask) || misaligned4(pos))
        return (xs_status)api_fail(XS_ERR_ALIGN, "parents, q_start, kv_len, mask and pos must be 4-byte aligned");
    const Buffer out[2] = {{mask, (size_t)T * words * 4, "mask"}, {pos, pos ? (size_t)T * 4 : 0, "pos"}};
    const Buffer in[3] = {{parents, (size_t)T * 4, "parents"}, {q_start, (size_t)(N + 1) * 4, "q_start"},
                          {kv_len, pos ? (size_t)N * 4 : 0, "kv_len"}};
    if ((st = check_disjoint(out, 2, in, 3))) return (xs_status)st;
    if (N == 0 || T == 0) return XS_OK;
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(out, 2, dev)) || (st = check_device(in, 3, dev)))
        return (xs_status)st;
    const cudaError_t e = launch_tree_mask(TreeMaskParams{parents, q_start, kv_len, mask, pos, N, T, words},
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("tree mask launch", e);
}

xs_status xs_attn_tree(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                       const int32_t *q_start, const int32_t *kv_len, const int32_t *mask, void *out, int N, int T, int H,
                       int Hk, int D, int page, int n_pages, int max_pages, int words, float scale, void *workspace,
                       size_t workspace_bytes, void *stream) {
    if (N && T && (!q || !k_pages || !v_pages || !page_table || !q_start || !kv_len || !mask || !out))
        return (xs_status)api_fail(XS_ERR_NULL, "q, k_pages, v_pages, page_table, q_start, kv_len, mask and out must be non-NULL");
    size_t pool, table;
    int st = check_cache(N, T, Hk, D, page, n_pages, max_pages, &pool, &table);
    if (st || (st = check_heads(T, H, Hk)) || (st = check_words(words)) || (st = check_scale(scale))) return (xs_status)st;
    if (misaligned16(q) || misaligned16(k_pages) || misaligned16(v_pages) || misaligned16(out))
        return (xs_status)api_fail(XS_ERR_ALIGN, "q, k_pages, v_pages and out must be 16-byte aligned");
    if (misaligned4(page_table) || misaligned4(q_start) || misaligned4(kv_len) || misaligned4(mask))
        return (xs_status)api_fail(XS_ERR_ALIGN, "page_table, q_start, kv_len and mask must be 4-byte aligned");
    const size_t rows = (size_t)T * H * D * 2;
    const Buffer o = {out, rows, "out"};
    const Buffer in[7] = {{q, rows, "q"}, {k_pages, pool, "k_pages"}, {v_pages, pool, "v_pages"},
                          {page_table, table, "page_table"}, {q_start, (size_t)(N + 1) * 4, "q_start"},
                          {kv_len, (size_t)N * 4, "kv_len"}, {mask, (size_t)T * words * 4, "mask"}};
    const Buffer all[8] = {o, in[0], in[1], in[2], in[3], in[4], in[5], in[6]};
    if ((st = check_disjoint(&o, 1, in, 7)) || (st = check_workspace(workspace, workspace_bytes, all, 8)))
        return (xs_status)st;
    if (N == 0 || T == 0) return XS_OK;
    if (!workspace) return (xs_status)api_fail(XS_ERR_NULL, "workspace must be non-NULL");
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(all, 8, dev)) ||
        (st = check_workspace_size(workspace, workspace_bytes, span_workspace_bytes(D, sms), dev)))
        return (xs_status)st;
    SpanParams p{};
    if ((st = span_limits(-1, -1, 0, &p))) return (xs_status)st;
    p.kind = SPAN_TREE;
    p.out = static_cast<uint16_t *>(out);
    p.table = page_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.mask = mask;
    p.words = words;
    p.scale_log2 = scale_log2(scale);
    span_workspace_parts(workspace, D, sms, &p);
    SpanMaps maps;
    if ((st = span_paged(q, k_pages, v_pages, N, T, H, Hk, D, page, n_pages, max_pages, &p, &maps))) return (xs_status)st;
    const cudaError_t e = launch_span(D, maps, p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("tree attention launch", e);
}

xs_status xs_attn_tree_workspace_size(int N, int T, int H, int Hk, int D, size_t *bytes) {
    return xs_attn_paged_workspace_size(N, T, H, Hk, D, bytes);
}

xs_status xs_attn_packed(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                         const int32_t *q_start, void *out, int N, int T, int H, int Hk, int D, float scale, int left,
                         int right, int sinks, void *workspace, size_t workspace_bytes, void *stream) {
    if (N && T && (!q || !k || !v || !q_start || !out))
        return (xs_status)api_fail(XS_ERR_NULL, "q, k, v, q_start and out must be non-NULL");
    int st = check_packed(N, T, H, Hk, D);
    if (st || (st = check_scale(scale))) return (xs_status)st;
    SpanParams p{};
    if ((st = span_limits(left, right, sinks, &p))) return (xs_status)st;
    size_t qb, kb, vb;
    if ((st = check_rows("q", T, H, D, &q_stride, &qb)) || (st = check_rows("k", T, Hk, D, &k_stride, &kb)) ||
        (st = check_rows("v", T, Hk, D, &v_stride, &vb)))
        return (xs_status)st;
    if (misaligned16(q) || misaligned16(k) || misaligned16(v) || misaligned16(out))
        return (xs_status)api_fail(XS_ERR_ALIGN, "q, k, v and out must be 16-byte aligned");
    if (misaligned4(q_start)) return (xs_status)api_fail(XS_ERR_ALIGN, "q_start must be 4-byte aligned");
    const Buffer o = {out, (size_t)T * H * D * 2, "out"};
    const Buffer in[4] = {{q, qb, "q"}, {k, kb, "k"}, {v, vb, "v"}, {q_start, (size_t)(N + 1) * 4, "q_start"}};
    const Buffer all[5] = {o, in[0], in[1], in[2], in[3]};
    if ((st = check_disjoint(&o, 1, in, 4)) || (st = check_workspace(workspace, workspace_bytes, all, 5)))
        return (xs_status)st;
    if (N == 0 || T == 0) return XS_OK;
    if (!workspace) return (xs_status)api_fail(XS_ERR_NULL, "workspace must be non-NULL");
    int dev, sms;
    if ((st = api_device(&dev, &sms)) || (st = check_device(all, 5, dev)) ||
        (st = check_workspace_size(workspace, workspace_bytes, span_workspace_bytes(D, sms), dev)))
        return (xs_status)st;
    p.kind = SPAN_PACKED;
    p.out = static_cast<uint16_t *>(out);
    p.q_start = q_start;
    p.N = N;
    p.T = T;
    p.H = H;
    p.Hk = Hk;
    p.G = H / Hk;
    p.page = 128;  // K/V tiles come in one box
    p.scale_log2 = scale_log2(scale);
    p.tile_tok = 128 / p.G;
    p.item_tok = 2 * p.tile_tok;
    p.g_magic = (65536u + (uint32_t)p.G - 1u) / (uint32_t)p.G;
    p.heads = Hk;
    p.n_pairs = T / p.item_tok + std::min(N, T);  // at most so many items a head
    // A CTA for each item, none cut, where there are no more items than SMs and none is long, whatever the lengths: pieces
    // and their merge cost more than their balance gains. Whole and cut, us: 4 prompts of 17 to 300 tokens, 8 heads, D = 64
    // 11.2, 16.0; one of 500, 32 and 8 heads, D = 128 15.9, 20.1; of 900 20.9, 27.6; of 1000, 24 heads, D = 64 18.4, 20.1;
    // but one of 1000, 8 and 1 heads 21.3, 19.8 and of 1500 26.2, 22.4; of 1500, 16 and 4 heads, D = 64 23.1, 20.9.
    if ((long long)p.heads * p.n_pairs > sms || T > 1024) span_workspace_parts(workspace, D, sms, &p);
    SpanMaps maps;
    const uint64_t d = (uint64_t)D * 2;
    const uint64_t q_dims[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)Hk, (uint64_t)T};
    const uint64_t q_strides[3] = {d, p.G * d, (uint64_t)q_stride * 2};
    const uint32_t q_box[4] = {64, (uint32_t)p.G, 1, (uint32_t)p.tile_tok};
    const uint64_t kv_dims[4] = {(uint64_t)D, (uint64_t)Hk, (uint64_t)T, 1};
    const uint64_t k_strides[3] = {d, (uint64_t)k_stride * 2, (uint64_t)k_stride * 2};  // (the last dimension has one place)
    const uint64_t v_strides[3] = {d, (uint64_t)v_stride * 2, (uint64_t)v_stride * 2};
    const uint32_t kv_box[4] = {64, 1, 128, 1};
    if ((st = api_tile_map(&maps.q, q, q_dims, q_strides, q_box, "q")) ||
        (st = api_tile_map(&maps.k, k, kv_dims, k_strides, kv_box, "k")) ||
        (st = api_tile_map(&maps.v, v, kv_dims, v_strides, kv_box, "v")))
        return (xs_status)st;
    const cudaError_t e = launch_span(D, maps, p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? XS_OK : (xs_status)api_cuda_error("packed attention launch", e);
}

xs_status xs_attn_packed_workspace_size(int N, int T, int H, int Hk, int D, size_t *bytes) {
    if (!bytes) return (xs_status)api_fail(XS_ERR_NULL, "bytes must be non-NULL");
    int st = check_packed(N, T, H, Hk, D);
    if (st) return (xs_status)st;
    *bytes = 0;
    if (N == 0 || T == 0) return XS_OK;
    int dev, sms;
    if ((st = api_device(&dev, &sms))) return (xs_status)st;
    *bytes = span_workspace_bytes(D, sms);
    return XS_OK;
}

}  // extern "C"
