// xs_internal.h -- declarations shared by the host API (xs_api.cpp) and the
// kernel translation units. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace xs {

// Work decomposition of one attention call. A work item is a pair of
// consecutive 128-row query tiles of one (rank, batch, local head); the second
// tile of the last pair is absent when ceil(S/128) is odd, and the last tile
// is partial when S is not a multiple of 128. A unit is one item and
// one 128-row K/V tile.
//
// Schedule: CTA c first takes whole items c, c + G, ..., c + (n_dp - 1) G
// (G = gridDim.x). The remaining items, the "balanced region" starting at
// sk_item0, hold sk_units units that are dealt out as G contiguous ranges of
// equal length, [c*U/G, (c+1)*U/G); an item whose units fall into several
// ranges is computed in pieces whose partial results meet in the workspace.
struct AttnParams {
    int B, S, H, P, Hl, Sl;
    int ld_rows;  // sequence-partitioned inputs: token rows per TMA box (gcd(Sl, 128))
    int n_qt;     // 128-row query tiles per head  (ceil(S / 128))
    int n_pairs;  // work items per head           (ceil(n_qt / 2))
    int n_kv;     // 128-row K/V tiles per head    (ceil(S / 128))
    int kv_tail;  // keys in the last K/V tile (128 unless S is ragged); later columns are masked
    int n_items;  // P * B * Hl * n_pairs (P * B * Hl * n_qt for single-tile items), or a rank range's share
    int item0 = 0;  // global index of work item 0 (a call over the ranks from rank0 on: rank0 * B * Hl * items per head)
    float scale_log2;  // scale * log2(e): softmax runs in base 2
    uint16_t *out;
    int head_out;          // 1: output head-partitioned like q (attention only); 0: the All-to-All scatter
    int n_dp;              // round-robin waves of whole items
    int sk_item0;          // first item of the balanced region
    uint32_t sk_units;     // units U in the balanced region (0: none), below 2^31
    uint32_t sk_q, sk_r;   // U = sk_q * G + sk_r, so range starts are c*q + (c*r)/G
    float *ws_rec;         // 2 * G partial records (see partial_record_bytes)
    unsigned long long *ws_cnt;  // arrival counters, 4 per tile of each item of the balanced region
    unsigned long long gen;      // this launch's 48-bit generation, stamped into the counters
    unsigned long long *trace;  // traced instances: epilogue records, kTraceWords per (CTA, item, tile, warp)
};

// Epilogue trace record of one output tile and epilogue warp (32 rows):
// clock64 when the tile's O and row sums were ready, before its first store,
// after its last store was issued; %globaltimer when ready; then
// item << 8 | tile << 4 | warp, with bit 3 set for an absent tile.
constexpr int kTraceWords = 5;

// Head dimension 256 runs the single-query-tile kernel (xs_attn1_kernel.cuh):
// its work item is one 128-row query tile instead of a pair.
inline bool single_tile_items(int D) { return D > 128; }
inline int tiles_per_item(int D) { return single_tile_items(D) ? 1 : 2; }

// Bytes of one partial record: unnormalised O of the item's tiles (fp32) plus
// their row max and row sum.
inline size_t partial_record_bytes(int D) {
    return (size_t)tiles_per_item(D) * (128 * (size_t)D * 4 + 2 * 128 * 4);
}

// Chooses the grid and fills the schedule fields of p. With a workspace the
// tail waves are balanced; without one every CTA takes whole items only.
int attn_schedule(AttnParams &p, int num_sms, bool balanced);
// Chunks of the host-buffer pipeline over (slice, head) units; fills bounds[0..n], returns n.
int host_chunk_plan(int units, long long unit_bytes, long long min_bytes, int max_chunks, int *bounds);
// Workspace bytes a balanced call needs (records, then counters), 256-aligned parts.
size_t attn_workspace_bytes(int n_items, int n_kv, int D, int num_sms);

// Most simulated ranks a call with sequence-partitioned inputs accepts: the
// kernel takes two TMA tensor maps per source rank and operand as a parameter.
constexpr int kMaxRanks = 8;
constexpr int kSeqMaps = 2 * kMaxRanks;

// TMA tensor maps of Q, K and V. NM = 1: one map per operand over the
// head-partitioned tensor. NM = kSeqMaps: maps over each source rank's
// sequence-partitioned slice; entry r (r < P) has boxes of ld_rows = gcd(Sl, 128)
// rows, which never straddle two ranks, and entry kMaxRanks + r boxes of 128 rows
// for tiles that lie inside rank r's slice (used only when Sl >= 128).
template <int NM> struct OperandMaps {
    CUtensorMap q[NM], k[NM], v[NM];
};

// The output layout is p.head_out (head-partitioned) or the All-to-All scatter;
// both run the same compiled kernel.
cudaError_t launch_attention(int D, const OperandMaps<1> &maps, const AttnParams &p, int grid,
                             cudaStream_t stream);
// The fused call with epilogue tracing (p.trace set, whole-item schedule).
cudaError_t launch_attention_traced(int D, const OperandMaps<1> &maps, const AttnParams &p, int grid,
                                    cudaStream_t stream);
// Causal attention (query token i sees keys 0..i), whole-item schedule.
cudaError_t launch_causal(int D, const OperandMaps<1> &maps, const AttnParams &p, int grid,
                          cudaStream_t stream);
// Sequence-partitioned inputs (the pre-attention All-to-All done by the loads),
// sequence-partitioned output.
cudaError_t launch_ulysses(int D, const OperandMaps<kSeqMaps> &maps, const AttnParams &p, int grid,
                           cudaStream_t stream);

// Per-head-dimension instances (xs_attn_d64.cu, xs_attn_d96.cu, xs_attn_d128.cu).
#define XS_DECLARE_ATTN_ENTRY(D)                                                                                  \
    cudaError_t launch_attention_d##D(const OperandMaps<1> &maps, const AttnParams &p, int grid,          \
                                      cudaStream_t stream);                                                       \
    cudaError_t launch_ulysses_d##D(const OperandMaps<kSeqMaps> &maps, const AttnParams &p, int grid,             \
                                    cudaStream_t stream);                                                         \
    cudaError_t launch_causal_d##D(const OperandMaps<1> &maps, const AttnParams &p, int grid,             \
                                   cudaStream_t stream);                                                          \
    cudaError_t read_error_word_d##D(unsigned int *value, bool clear);
XS_DECLARE_ATTN_ENTRY(64)
XS_DECLARE_ATTN_ENTRY(96)
XS_DECLARE_ATTN_ENTRY(128)
XS_DECLARE_ATTN_ENTRY(256)
cudaError_t launch_attention_traced_d128(const OperandMaps<1> &maps, const AttnParams &p, int grid,
                                         cudaStream_t stream);
// E4M3 inputs, D = 128 only (xs_attn_f8.cu): f8 = 1 for E4M3 q and k (maps over
// bytes) with bf16 v, f8 = 2 for E4M3 q, k and v.
cudaError_t launch_attention_f8_d128(int f8, const OperandMaps<1> &maps, const AttnParams &p, int grid,
                                     cudaStream_t stream);
cudaError_t read_error_word_f8(unsigned int *value, bool clear);

// Sets the calling thread's xs_last_error() text; returns `status`.
int report_error(int status, const char *message);

// Device-side error word (bit 31: a bounded wait ran out; low bits: which wait).
cudaError_t read_device_error(unsigned int *value, bool clear, cudaStream_t stream);
cudaError_t launch_wait_selftest(unsigned long long limit_ns, cudaStream_t stream);

struct PermParams {
    uint32_t rows;       // B * S * H rows of D elements
    uint32_t cpr;        // 16-byte chunks per row (D / 8)
    uint32_t cpr_log2;   // log2(cpr) when cpr is a power of two
    uint32_t mC, sC;     // magic numbers for division by cpr otherwise
    uint32_t B, S, H, Hl, Sl;
    // magic numbers for division by H, Sl, B, Hl and S (round-up method)
    uint32_t mH, sH, mSl, sSl, mB, sB, mHl, sHl, mS, sS;
};
void fastdiv_magic(uint32_t d, uint32_t *m, uint32_t *s);
// inverse = false: head-partitioned -> sequence-partitioned (post-attention
// All-to-All); inverse = true: the reverse (pre-attention All-to-All).
cudaError_t launch_permute(const void *in, void *out, const PermParams &p, bool inverse, int num_sms,
                           cudaStream_t stream);

// ------------------------------------------------------------ rotary positions
constexpr int kRopeMaxPairs = 128, kRopeMaxUnits = 16, kRopeMaxAxes = 4;
struct RopeParams {
    const uint16_t *q, *k;  // k NULL: none (Hk = 0)
    uint16_t *q_out, *k_out;
    const int *pos;         // [pos batches][S][n_axes]
    int64_t pos_batch;      // S, or 0 when every batch shares the positions
    int B, S, H, Hk, Hl, Hkl, Sl, D;
    int n_axes, n_pairs;
    int tile;               // tokens per block
    bool seq_in, seq_out, inverse;
    uint64_t frac[kRopeMaxPairs];       // frequency in turns, a 64-bit binary fraction
    uint8_t axis[kRopeMaxPairs];
    uint8_t unit_first[kRopeMaxUnits], unit_half[kRopeMaxUnits];  // pairs half an axis apart: a unit's first
                                                                  // chunk, and how far the second is (rope_kernel)
};
cudaError_t launch_rope(RopeParams &p, bool halves, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ paged cache
struct AppendParams {
    const uint4 *k, *v;
    uint4 *k_pages, *v_pages;
    const int *table, *q_start, *kv_len;
    int N, T, chunks;  // chunks: 16-byte chunks of a token's Hk * D elements
    int page, n_pages, max_pages;
};
cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);

// ------------------------------------------------------------ window and paged attention
struct SpanPieces;
struct SpanParams {
    uint16_t *out;
    const int *table, *q_start, *kv_len;  // table NULL: whole sequences, head-partitioned
    int N, T, H, Hk, G;         // whole sequences: T = B * S rows of H heads
    int page, page_log2, n_pages, max_pages;
    int B, S, P, Hl, Sl, head_out;  // whole sequences only
    int left, right, sinks;     // at most 2^29 each
    float scale_log2;
    int few;                    // 0: query tiles of 128 rows; 16 or 32: the few-rows form
    int tile_tok;               // tokens of a query tile: 128 / G, or few / G
    int item_tok;               // tokens of an item: two tiles, or one with few rows
    uint32_t g_magic;           // row / G = row * g_magic >> 16 for rows below 128: ceil(2^16 / G)
    int heads, n_pairs;         // key heads of a sequence; query tile pairs of a head (whole sequences)
    int min_steps_log2;         // fewest steps that a CTA is started for
    int stretch;                // most steps that one sum in tensor memory takes; 0: no item has more (LONG = false)
    int merge_y;                // blocks per item in the merge
    float *rec;                 // workspace: 2 records a CTA (Rec<D>), one more a CTA for the segment at hand of a part in
                                // several, then a SpanPieces a CTA; NULL: whole items, each one segment
    SpanPieces *pieces;
};
// TMA maps: q by query tile, k and v by 128-key tile or page (see xs_ops_api.cpp).
struct SpanMaps {
    CUtensorMap q, k, v;
};
// Workspace bytes, and its parts' places in p.
size_t span_workspace_bytes(int D, int num_sms);
void span_workspace_parts(void *ws, int D, int num_sms, SpanParams *p);
cudaError_t launch_span(int D, const SpanMaps &maps, const SpanParams &p, int num_sms, cudaStream_t stream);
#define XS_DECLARE_SPAN_ENTRY(D)                                                                                \
    cudaError_t launch_span_d##D(const SpanMaps &maps, const SpanParams &p, int grid, cudaStream_t stream);     \
    cudaError_t read_error_word_span_d##D(unsigned int *value, bool clear);
XS_DECLARE_SPAN_ENTRY(64)
XS_DECLARE_SPAN_ENTRY(96)
XS_DECLARE_SPAN_ENTRY(128)

// ------------------------------------------------------------ host helpers of the C ABI (xs_api.cpp)
// Each records the thread's last error and returns a status (0: fine).
int api_fail(int status, const char *fmt, ...);
int api_cuda_error(const char *what, cudaError_t e);
int api_device(int *dev, int *num_sms);
int api_device_pointer(const void *ptr, int dev, const char *name);
int api_tile_map(CUtensorMap *m, const void *ptr, const uint64_t (&dims)[4], const uint64_t (&strides)[3],
                 const uint32_t (&box)[4], const char *name);
int api_shape(int B, int S, int H, int D, int P, size_t *bytes);
bool api_overlaps(const void *a, size_t na, const void *b, size_t nb);

}  // namespace xs

#ifdef __CUDACC__
namespace xs {

// The sequence that packed row t belongs to, its place among the sequence's new
// tokens and their number; seq = -1 for a row of none. Bounds of q_start are
// cut to [0, T], so no table leads outside the packed rows. All 32 lanes of a
// warp call it with the same t: each round narrows N to N / 32 with one load
// per lane.
struct CacheRow {
    int seq, i, q_len;
};
__device__ __forceinline__ CacheRow find_sequence(const int *q_start, int N, int T, int t, int lane) {
    int lo = 0, n = N + 1;  // the last of q_start[lo .. lo + n) that is at most t
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool ok = lane * step < n && q_start[at] <= t;
        const uint32_t votes = __ballot_sync(0xffffffffu, ok);
        const int hit = votes ? 31 - __clz((int)votes) : 0;
        n = min(step, n - hit * step);
        lo += hit * step;
    }
    CacheRow r{-1, 0, 0};
    if (lo >= N) return r;
    const int a = min(max(q_start[lo], 0), T), b = min(max(q_start[lo + 1], 0), T);
    if (t < a || t >= b) return r;
    r.seq = lo;
    r.i = t - a;
    r.q_len = b - a;
    return r;
}

}  // namespace xs
#endif
