// xs_span.cu -- host side of the attention over a span of keys per token
// (xs_span_kernel.cuh): the workspace's parts and the dispatch to the
// per-head-dimension instances.
#include <algorithm>

#include "xs_span_kernel.cuh"

namespace xs {

static size_t span_record_bytes(int D, int num_sms) { return (size_t)3 * num_sms * partial_record_bytes(D); }

size_t span_workspace_bytes(int D, int num_sms) {
    return span_record_bytes(D, num_sms) + (size_t)num_sms * sizeof(SpanPieces);
}

void span_workspace_parts(void *ws, int D, int num_sms, SpanParams *p) {
    p->rec = static_cast<float *>(ws);
    p->pieces = reinterpret_cast<SpanPieces *>(static_cast<char *>(ws) + span_record_bytes(D, num_sms));
}

cudaError_t launch_span(int D, const SpanMaps &maps, const SpanParams &p, int num_sms, cudaStream_t stream) {
    SpanParams q = p;
    // 2^18 keys: what a sum loses by truncation, about 2^-10, stays well below an output's rounding.
    // Where no item can walk over more, the instances without stretches (their code costs short
    // items 1 to 3%: mixed paged batch 82.9 us, 80.4 without).
    constexpr int kStretch = 2048;
    const long long held = p.kind == SPAN_WHOLE ? p.S : p.kind == SPAN_PACKED ? p.T : (long long)p.max_pages * p.page;
    const long long window = (long long)p.left + p.right + p.item_tok + p.sinks + 3 * 128;  // and whole tiles at its ends
    q.stretch = p.rec && std::min(held, window) > 128 * kStretch ? kStretch : 0;
    // The least part of a CTA: one step with few rows (4 sequences of 4 tokens over 1165 to 2941
    // keys, one key head: 15.6 us, 17.1 with two), two for other chunks (5 of 267 to 669
    // tokens over 996 keys: 20.9 us, 24.9 with four), four of whole sequences.
    q.min_steps_log2 = p.few ? 0 : p.kind != SPAN_WHOLE ? 1 : 2;
    // With 0, 2, 3, 4 and 6: 12 prompts of 130 to 4001 tokens 525, 428, 433, 446, 455 us; one of 2048 50.3, 41.5, 42.5,
    // 43.2, 43.7; 9 trees of 7 to 61 tokens over 500 to 8000 63.2, 55.3, 56.7, 56.9, 60.0; 16 prompts of 2048 alike 450, 445,
    // 442, 447, 452.
    q.item_cost = 2;
    // a merge block adds up 32 rows of an item, or with few rows 256 groups of 4 columns
    const int rows = std::min(p.T, p.item_tok) * p.G, tile = p.tile_tok * p.G;
    q.merge_y = p.few ? (rows * (D / 4) + 255) / 256 : rows > tile ? 8 : (rows + 31) / 32;
    const int grid = p.rec ? num_sms : (int)std::min((long long)num_sms, (long long)p.heads * p.n_pairs);
    // Trees of more than an item a key head on average may walk side by side. An instance apart: its schedule costs the
    // others' short calls 1 to 2 us (4 trees of 8 tokens 16.3 us, 17.1).
    if (p.kind == SPAN_TREE && !p.few && p.T > (long long)p.N * p.item_tok) q.kind = SPAN_TREE_LANES;
    if (p.kind >= SPAN_PACKED) {
        if (D == 64) return launch_span_serve_d64(maps, q, grid, stream);
        if (D == 96) return launch_span_serve_d96(maps, q, grid, stream);
        if (D == 128) return launch_span_serve_d128(maps, q, grid, stream);
        return cudaErrorInvalidValue;
    }
    if (D == 64) return launch_span_d64(maps, q, grid, stream);
    if (D == 96) return launch_span_d96(maps, q, grid, stream);
    if (D == 128) return launch_span_d128(maps, q, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace xs
