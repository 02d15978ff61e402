// xs_ops_api.cpp -- the C ABI of the operators around the fused attention:
// rotary positions, windowed attention, the paged cache and attention over it.
// Arguments are checked before any CUDA call, like in xs_api.cpp.
#include "../../include/xs.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "xs_internal.h"
#include "xs_ops_checks.h"

namespace {

using namespace xs;

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
    if (B && S && (!q || !k || !v || !out)) return api_fail(XS_ERR_NULL, "q, k, v and out must be non-NULL");
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

}  // namespace

extern "C" {

xs_status xs_rope(const void *q, const void *k, void *q_out, void *k_out, const int32_t *pos, int pos_batches, int B,
                  int S, int H, int Hk, int D, int P, int n_axes, const int *axis_dims, const double *freqs, int flags,
                  void *stream) {
    const bool work = B && S;
    if (!axis_dims || !freqs || (work && (!q || !q_out || !pos)))
        return (xs_status)api_fail(XS_ERR_NULL, "q, q_out, pos, axis_dims and freqs must be non-NULL");
    if (Hk < 0) return (xs_status)api_fail(XS_ERR_SHAPE, "Hk must be >= 0 (got %d)", Hk);
    if (work && Hk > 0 && (!k || !k_out)) return (xs_status)api_fail(XS_ERR_NULL, "k and k_out must be non-NULL unless Hk is 0");
    size_t qb = 0, kb = 0;
    int st = api_shape(B, S, H, D, P, &qb);
    if (!st && Hk > 0) st = api_shape(B, S, Hk, D, P, &kb);
    if (st) return (xs_status)st;
    if (H + Hk > (1 << 16)) return (xs_status)api_fail(XS_ERR_SHAPE, "H + Hk = %d exceeds 65536 heads", H + Hk);
    if (pos_batches != 1 && pos_batches != B)
        return (xs_status)api_fail(XS_ERR_SHAPE, "pos_batches must be 1 or B (got %d)", pos_batches);
    if (flags & ~(XS_ROPE_HALVES | XS_ROPE_INVERSE | XS_ROPE_IN_SEQ | XS_ROPE_OUT_SEQ))
        return (xs_status)api_fail(XS_ERR_SHAPE, "unknown flags 0x%x", flags);
    const bool halves = flags & XS_ROPE_HALVES;
    RopeParams p;
    memset(&p, 0, sizeof p);
    if ((st = rope_table(n_axes, axis_dims, freqs, halves, D, &p))) return (xs_status)st;
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
    if (N && T && (!k || !v || !k_pages || !v_pages || !page_table || !q_start || !kv_len))
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
    if (N && T && (!q || !k_pages || !v_pages || !page_table || !q_start || !kv_len || !out))
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
    p.kind = SPAN_PAGED;
    p.out = static_cast<uint16_t *>(out);
    p.table = page_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.scale_log2 = scale_log2(scale);
    span_workspace_parts(workspace, D, sms, &p);
    SpanMaps maps;
    if ((st = span_paged(q, k_pages, v_pages, N, T, H, Hk, D, page, n_pages, max_pages, &p, &maps))) return (xs_status)st;
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
