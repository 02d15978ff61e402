/*
 * xs.h -- C ABI of the fused attention + post-attention All-to-All library (libxs.so).
 *
 * What the calls compute. Source: "X-Stage: An Overlooked Pipeline Stage for
 * Communication-Computation Overlap in DiT Inference" (arXiv 2607.23264v1).
 *   - Section 4.3: DiT self-attention is full, non-causal softmax attention,
 *       O = softmax(scale * Q K^T) V   per (batch, head),
 *     computed FlashAttention-style: a CTA owns a block of 128 query rows and
 *     walks all K/V tiles (Figure 6); finishing the walk yields one output tile.
 *   - Section 4.3, Figure 5 (d-e): Ulysses sequence parallelism runs attention
 *     head-partitioned and then an All-to-All restores the sequence partition.
 *     The fused design (Figure 7) issues each finished output tile's stores to
 *     its destination at the tile boundary and then starts the next tile.
 *   - Section 5.3: "FA-only" (xs_attn), "A2A-only" (xs_a2a_permute), "Serial"
 *     (xs_attn then xs_a2a_permute) and "Fused" (xs_attn_a2a) are the four
 *     compared implementations.
 *   - Section 4.3, Figure 5 (a-c): before attention a first All-to-All turns
 *     the sequence partition into the head partition (xs_a2a_permute_inverse);
 *     xs_ulysses_attn folds it into the attention kernel's loads.
 *
 * Ranks. P ranks are simulated as P contiguous slices of one allocation on the
 * calling GPU, so the All-to-All is a scatter of rows into slices; nothing
 * crosses a device boundary. Hl = H / P heads per rank, Sl = S / P tokens per rank.
 *
 * Layouts (row-major, elements are bf16 stored as uint16_t, D contiguous):
 *   head-partitioned      [P][B][S][Hl][D]  rank r holds global heads r*Hl .. r*Hl+Hl-1
 *                                            for all S tokens
 *   sequence-partitioned  [P][B][Sl][H][D]  rank r' holds tokens r'*Sl .. r'*Sl+Sl-1
 *                                            for all H heads, heads in ascending order
 *   element (r,b,s,hl,d) of the first is element (r',b,s-r'*Sl,h,d) of the second,
 *   with h = r*Hl + hl and r' = s / Sl. With P = 1 both are plain [B][S][H][D].
 *
 * Common rules for every compute call:
 *   - Pointers are DEVICE pointers on the current CUDA device, 16-byte aligned,
 *     owned and allocated by the caller. The library allocates no device memory;
 *     it keeps only host-side state (per-device attributes).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Calls are asynchronous: they return after the kernel is enqueued.
 *   - Arguments are checked before anything is enqueued. A violation returns a
 *     non-zero xs_status, enqueues nothing and leaves `out` untouched;
 *     xs_last_error() then describes it.
 *   - Shapes: B >= 0, S >= 0 (B == 0 or S == 0 is a valid empty call that
 *     enqueues nothing; its device pointers may be NULL), H >= 1, P >= 1, H % P == 0, S % P == 0, D in {64, 96, 128, 256},
 *     scale positive and finite. Every tensor must stay below 2^40 bytes. S need
 *     not be a multiple of 128: the last query tile is then partial (rows past
 *     S are neither computed into nor stored) and the keys past S in the last
 *     K/V tile are masked out of the softmax.
 *   - `out` must not overlap q, k or v (XS_ERR_ALIAS).
 *   - The GPU must be compute capability 10.3 (sm_103); otherwise
 *     XS_ERR_UNSUPPORTED.
 *   - Inside the kernels every wait is bounded in time. A wait that runs out sets
 *     a device-side error word and the kernel returns; xs_device_status() reports
 *     it as XS_ERR_TIMEOUT. No valid input causes this.
 */
#ifndef XS_H
#define XS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    XS_OK = 0,
    XS_ERR_NULL = 1,        /* a pointer that the call needs is NULL */
    XS_ERR_SHAPE = 2,       /* a shape rule above is violated */
    XS_ERR_ALIGN = 3,       /* a pointer is not 16-byte aligned */
    XS_ERR_UNSUPPORTED = 4, /* D not in {64,96,128,256}, wrong GPU, or a pointer that is not device memory */
    XS_ERR_CUDA = 5,        /* a CUDA runtime or driver call failed (message in xs_last_error) */
    XS_ERR_TIMEOUT = 6,     /* a bounded in-kernel wait ran out (reported by xs_device_status) */
    XS_ERR_ALIAS = 7,       /* out overlaps an input */
    XS_ERR_WORKSPACE = 8    /* workspace too small, misaligned or overlapping */
} xs_status;

/*
 * Fused attention + All-to-All scatter (the paper's "X-Stage-Fused" variant,
 * section 4.3, Figure 7).
 *   q, k, v : head-partitioned [P][B][S][Hl][D] bf16, read only.
 *   out     : sequence-partitioned [P][B][Sl][H][D] bf16, fully overwritten.
 *   scale   : multiplies Q K^T before the softmax (usually 1/sqrt(D)); > 0.
 * Each finished 128-row output tile of head (r, b, hl) is written straight into
 * the slices of the ranks that own its tokens. Bit-identical to
 * xs_a2a_permute(xs_attn(q, k, v)) for the same arguments.
 */
xs_status xs_attn_a2a(const void *q, const void *k, const void *v, void *out, int B, int S, int H,
                      int D, int P, float scale, void *stream);

/*
 * Attention only (the paper's "FA-only" variant, section 5.3).
 *   q, k, v : head-partitioned [P][B][S][Hl][D] bf16.
 *   out     : head-partitioned [P][B][S][Hl][D] bf16 (same layout as q), fully
 *             overwritten. P only defines the layout; P = 1 is plain [B][S][H][D].
 */
xs_status xs_attn(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D,
                  int P, float scale, void *stream);

/*
 * Standalone post-attention All-to-All (the paper's "A2A-only" variant, and the
 * second half of "Serial", section 5.3).
 *   in  : head-partitioned [P][B][S][Hl][D], 16-bit elements (any payload).
 *   out : sequence-partitioned [P][B][Sl][H][D], fully overwritten.
 * A pure copy: out is bit-for-bit a permutation of in. Same shape rules as the
 * attention calls except that scale does not apply. in and out must not overlap.
 */
xs_status xs_a2a_permute(const void *in, void *out, int B, int S, int H, int D, int P, void *stream);

/*
 * Standalone pre-attention All-to-All (Ulysses, section 4.3, Figure 5 (a-c)):
 * the inverse of xs_a2a_permute.
 *   in  : sequence-partitioned [P][B][Sl][H][D], 16-bit elements (any payload).
 *   out : head-partitioned [P][B][S][Hl][D], fully overwritten.
 * A pure copy; xs_a2a_permute(xs_a2a_permute_inverse(x)) == x bit for bit.
 * Shape and pointer rules as for xs_a2a_permute.
 */
xs_status xs_a2a_permute_inverse(const void *in, void *out, int B, int S, int H, int D, int P, void *stream);

/*
 * Both Ulysses All-to-Alls fused into one attention call (section 4.3,
 * Figure 5 (a-e), with the output side of Figure 7): attention over the whole
 * sequence for every head, from and to the sequence partition.
 *   q, k, v : sequence-partitioned [P][B][Sl][H][D] bf16, read only. Each
 *             128-row tile of head h is loaded where the sequence partition
 *             keeps it, from the slices of the ranks that own its tokens (one
 *             TMA tensor map per rank and operand), so no head-partitioned
 *             copy is ever made.
 *   out     : sequence-partitioned [P][B][Sl][H][D] bf16, fully overwritten.
 *   workspace, workspace_bytes : as for xs_attn_a2a_ws (NULL, 0: whole-item
 *             schedule); the size is xs_attn_workspace_size's.
 * Bit-identical to xs_attn_a2a_ws(xs_a2a_permute_inverse(q), ...(k), ...(v))
 * with the same workspace choice. Extra rules: P <= 8 and S/P % 8 == 0
 * (XS_ERR_UNSUPPORTED otherwise).
 */
xs_status xs_ulysses_attn(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D,
                          int P, float scale, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Causal attention, the autoregressive-LLM case the paper contrasts with DiT's
 * full attention (section 4.3): query token i of a head attends to key tokens
 * 0..i of the same sequence only. Same arguments, layouts and rules as
 * xs_attn_a2a (fused scatter, sequence-partitioned out) and xs_attn
 * (head-partitioned out); xs_attn_causal_a2a is bit-identical to
 * xs_a2a_permute(xs_attn_causal(...)). K/V tiles entirely above the diagonal
 * are skipped; work items (pairs of 128-row query tiles) are dealt longest
 * first to balance the CTAs.
 */
xs_status xs_attn_causal_a2a(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D,
                             int P, float scale, void *stream);
xs_status xs_attn_causal(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D,
                         int P, float scale, void *stream);

/*
 * Balanced-schedule variants. Identical results contract and layouts as
 * xs_attn_a2a / xs_attn, plus a caller-owned device workspace that lets the
 * last one to two waves of work be split evenly over all SMs instead of
 * leaving some SMs idle: an output tile pair whose K/V range is split across
 * CTAs is computed in pieces whose partial rows (unnormalised O in fp32, row
 * max, row sum) meet in the workspace and are merged in a fixed order.
 * Small calls run on fewer CTAs so that pieces hold at least 16 K/V tiles,
 * but never on fewer CTAs than work items (or SMs).
 *   workspace       : device memory, 256-byte aligned, at least the size that
 *                     xs_attn_workspace_size reports for these shapes on the
 *                     current device; its contents need no initialisation and
 *                     may be left arbitrary between calls. NULL (with
 *                     workspace_bytes = 0) falls back to the whole-item schedule.
 *   workspace_bytes : its size in bytes.
 * Calls that may run concurrently must not share a workspace. xs_attn_a2a_ws
 * and xs_a2a_permute(xs_attn_ws(...)) are bit-identical for the same
 * arguments on the same device; against the whole-item schedule the split
 * tiles differ only by rounding.
 */
xs_status xs_attn_a2a_ws(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D,
                         int P, float scale, void *workspace, size_t workspace_bytes, void *stream);
xs_status xs_attn_ws(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D, int P,
                     float scale, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes that the *_ws calls need for these shapes on the current
 * device (written to *bytes). Shape rules as for the attention calls. */
xs_status xs_attn_workspace_size(int B, int S, int H, int D, int P, size_t *bytes);

/*
 * The balanced fused call for callers that cannot allocate device memory. The
 * paper has no counterpart to this call; it exists for deployment.
 * Some callers can pass q, k, v and out but cannot allocate a workspace: a
 * plug-in inside a framework that owns all device memory through its own pool,
 * a latency-critical path that cannot afford cudaMalloc's implicit device-wide
 * synchronisation, or a process whose device memory is reserved up front.
 * This call computes what xs_attn_a2a_ws computes (same arguments minus the
 * workspace), using instead a scratch area built into the library: 48 MiB per
 * device that loads the library, held until the process exits. It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *   - Shapes whose balanced schedule needs more than the 48 MiB are rejected
 *     with XS_ERR_WORKSPACE before anything is enqueued
 *     (xs_attn_workspace_size reports the need).
 *   - Every call on a device shares the one scratch area, which keeps the
 *     previous call's contents. Nothing in it needs clearing: partial rows are
 *     written before they are read, and the arrival counters carry a per-launch
 *     generation stamp. Only the kernel of a call that passed every argument
 *     check writes it. Calls that may overlap on the GPU race on the scratch
 *     area and must not be issued.
 *   - The first call on a device looks up the scratch area's device address
 *     with that device current; make that first call before any stream capture.
 */
xs_status xs_attn_a2a_noalloc(const void *q, const void *k, const void *v, void *out, int B, int S, int H,
                              int D, int P, float scale, void *stream);

/*
 * Fused attention + All-to-All scatter with 8-bit queries and keys: an
 * extension, the X-Stage paper evaluates bf16 only. Same operation as
 * xs_attn_a2a_ws / xs_attn_ws, with Q K^T taken from E4M3 inputs.
 *   q8, k8 : head-partitioned [P][B][S][Hl][D] bytes, each one OCP OFP8 E4M3
 *            value (sign, 4 exponent bits with bias 7, 3 mantissa bits; no
 *            infinities; 0x7F and 0xFF are NaN). Read only.
 *   v      : head-partitioned [P][B][S][Hl][D] bf16, read only.
 *   out    : bf16, sequence-partitioned [P][B][Sl][H][D] (xs_attn_a2a_q8) or
 *            head-partitioned like v (xs_attn_q8), fully overwritten.
 *   scale  : multiplies the exact product of the decoded q8 and k8 before the
 *            softmax; per-tensor dequantisation factors of q8 and k8 fold in
 *            here (softmax scale x q factor x k factor). > 0.
 *   workspace, workspace_bytes : as for xs_attn_a2a_ws (the same size;
 *            NULL, 0: whole-item schedule).
 * D = 128 only (XS_ERR_UNSUPPORTED otherwise). Q K^T runs on the 8-bit tensor
 * path with fp32 accumulation; the softmax, P and P V stay as in the bf16
 * calls. xs_attn_a2a_q8 is bit-identical to xs_a2a_permute(xs_attn_q8(...)).
 * XS_ERR_ALIAS when out overlaps the B*S*H*D bytes of q8 or k8 or the bf16 v.
 */
xs_status xs_attn_a2a_q8(const void *q8, const void *k8, const void *v, void *out, int B, int S, int H, int D,
                         int P, float scale, void *workspace, size_t workspace_bytes, void *stream);
xs_status xs_attn_q8(const void *q8, const void *k8, const void *v, void *out, int B, int S, int H, int D, int P,
                     float scale, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same with E4M3 values as well (an extension; the X-Stage paper evaluates
 * bf16 only): q8, k8 and v8 are head-partitioned [P][B][S][Hl][D] E4M3 bytes,
 * out bf16 as for xs_attn_a2a_q8 / xs_attn_q8. Each V tile is widened exactly
 * to f16 on chip, P is rounded to f16 (10 mantissa bits, against bf16's 7 in
 * the other calls) and P V runs as f16 x f16 with fp32 accumulation. A
 * dequantisation factor of v8 multiplies the output; apply it to out (or fold
 * it into the next operation). D = 128 only. xs_attn_a2a_qkv8 is bit-identical
 * to xs_a2a_permute(xs_attn_qkv8(...)). XS_ERR_ALIAS when out overlaps the
 * B*S*H*D bytes of q8, k8 or v8.
 */
xs_status xs_attn_a2a_qkv8(const void *q8, const void *k8, const void *v8, void *out, int B, int S, int H, int D,
                           int P, float scale, void *workspace, size_t workspace_bytes, void *stream);
xs_status xs_attn_qkv8(const void *q8, const void *k8, const void *v8, void *out, int B, int S, int H, int D, int P,
                       float scale, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The fused call (xs_attn_a2a_host) and attention only (xs_attn_host) on inputs
 * and output in HOST memory, for callers whose tensors live on the host. The X-Stage
 * paper has no counterpart; these calls exist for deployment. The copies are pipelined
 * with the compute: the inputs' units, one head of one (rank, batch) slice each, are
 * split in order into up to 16 chunks of at least 8 MiB of inputs each (one chunk
 * for small calls), the first and the last the smallest. Chunk c's rows of q, k, v
 * (whole slices, and the chunk's heads of every row of a partial slice at either
 * end) are copied in on an internal stream, the caller's stream
 * runs the attention kernel over that chunk's work items, and an internal stream
 * copies the chunk's output out while later chunks are copied in and computed. For
 * xs_attn_a2a_host that output is the columns of the chunk's heads in the rows of its
 * batches of the sequence-partitioned output; for xs_attn_host, its part of the
 * head-partitioned one.
 *   q_host, k_host, v_host : head-partitioned [P][B][S][Hl][D] bf16 in host
 *       memory, read only. out_host : host memory for the output (layouts as for
 *       xs_attn_a2a / xs_attn), fully overwritten. Page-locked (pinned) host
 *       memory lets the copies run asynchronously and overlap; pageable memory
 *       works but the copies then serialise. Device or managed memory passed
 *       as a host buffer is rejected with XS_ERR_UNSUPPORTED.
 *   q, k, v, out : device staging buffers of the full sizes, 16-byte aligned,
 *       overwritten by the call (q, k, v hold the inputs afterwards, out the
 *       output). No two buffers, host or device, may overlap (XS_ERR_ALIAS).
 *   workspace, workspace_bytes : as for xs_attn_a2a_ws (NULL, 0: whole-item
 *       schedule); each chunk's launch uses it in turn. A chunk holds only a
 *       share of the work items, so without a workspace most SMs idle.
 * Asynchronous like every call. When the caller's stream reaches the point after
 * the call, out_host holds the result, and later work on that stream is ordered
 * after the copies. The first call on a device creates two streams and 34 events
 * there, kept until the process exits. A per-device lock keeps concurrent calls'
 * enqueue sequences apart. The result equals that of xs_attn_a2a_ws / xs_attn_ws
 * with the same workspace up to the rounding of split tiles (the chunks split
 * differently). Without a workspace it is bit-identical to xs_attn_a2a / xs_attn.
 */
xs_status xs_attn_a2a_host(const void *q_host, const void *k_host, const void *v_host, void *out_host, void *q,
                           void *k, void *v, void *out, int B, int S, int H, int D, int P, float scale,
                           void *workspace, size_t workspace_bytes, void *stream);
xs_status xs_attn_host(const void *q_host, const void *k_host, const void *v_host, void *out_host, void *q, void *k,
                       void *v, void *out, int B, int S, int H, int D, int P, float scale, void *workspace,
                       size_t workspace_bytes, void *stream);

/*
 * The fused call (xs_attn_a2a, whole-item schedule) with its epilogue traced:
 * the per-tile record the paper's section 5.2.3 uses to measure each output
 * tile's sender-visible store span, and the section 4.3 audit its Q-loop gap.
 * Results are bit-identical to xs_attn_a2a; the records cost a few clock reads
 * and one 40-byte store per tile and epilogue warp. D = 128 only
 * (XS_ERR_UNSUPPORTED otherwise).
 *   trace, trace_bytes : device buffer of at least the size xs_attn_trace_layout
 *       reports, 16-byte aligned; zeroed and then filled by the call. Layout:
 *       [ctas][items_per_cta][tile 0..1][epilogue warp 0..3] records of five
 *       uint64: clock64 when the tile's O and row sums were ready, clock64 just
 *       before its first global store, clock64 after its last store was issued,
 *       %globaltimer (ns) when ready, and item << 8 | tile << 4 | warp (bit 3
 *       set when the tile is absent: ceil(S/128) odd). Records of a CTA that ran out
 *       of items stay zero. clock64 values compare only within one CTA. After
 *       the records come 20 uint64 per CTA; the first four are the CTA's
 *       %globaltimer at kernel entry, after set-up (barriers, tensor memory),
 *       when its first Q load was issued, and when it finished. Last come
 *       [2 items][2 tiles][64 K/V steps][4] uint64 for CTA 0's first two items:
 *       clock64 when the softmax's first warp saw the step's scores ready,
 *       when it handed P over, when the MMA issuer saw P complete, and after
 *       it issued that P V.
 */
xs_status xs_attn_a2a_trace(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D,
                            int P, float scale, void *trace, size_t trace_bytes, void *stream);

/* Grid size, items per CTA and trace bytes of xs_attn_a2a_trace for these
 * shapes on the current device. */
xs_status xs_attn_trace_layout(int B, int S, int H, int D, int P, int *ctas, int *items_per_cta, size_t *bytes);

/*
 * The operators around the fused attention. The X-Stage paper has no
 * counterpart to them: a video DiT turns q and k by rotary positions before
 * attention, long sequences attend through a window, and an autoregressive
 * model keeps its keys and values in a paged cache. The common rules above hold
 * unless a call says otherwise. None of these calls synchronises, allocates or
 * keeps anything between calls, so each can be captured into a CUDA graph and
 * replayed (make one call of each kind, of the same sizes, on a device before the
 * first capture: it loads the kernels); calls or replays that may run at the same time must not
 * share a workspace or write the same memory.
 */

/*
 * Rotary positions with one to four axes (time, height and width of a video
 * token, or the place in a text) for queries and keys.
 *   q, q_out : [..][H][D] bf16; k, k_out: the same with Hk heads (Hk = 0: no keys,
 *            k and k_out are ignored). Head-partitioned [P][B][S][H/P][D], or
 *            sequence-partitioned [P][B][S/P][H][D] where the flags say so;
 *            with XS_ROPE_IN_SEQ and not XS_ROPE_OUT_SEQ the call is also the
 *            pre-attention All-to-All (xs_a2a_permute_inverse) of its input.
 *   pos    : device, [pos_batches][S][n_axes] int32, token s's place on each axis
 *            (any 32-bit value). pos_batches = B, or 1 for positions that all
 *            batches share.
 *   axis_dims, freqs : HOST arrays, read before the call returns. Axis a turns
 *            axis_dims[a] elements of each head, axes in order from element 0;
 *            elements past their sum are copied unchanged. freqs holds
 *            sum(axis_dims) / 2 frequencies in radians per unit of place, one per
 *            pair in order (commonly theta^(-2 i / axis_dims[a]) for the axis's
 *            pair i); |freqs| <= 1e6.
 *   flags  : XS_ROPE_HALVES: an axis's pair i is its elements i and
 *            i + axis_dims[a] / 2 (otherwise 2i and 2i + 1). XS_ROPE_INVERSE: turn
 *            by the negative angle, which undoes the call and is also its
 *            gradient (d q_out -> d q).
 * The pair (x, y) at place p becomes (x cos pf - y sin pf, x sin pf + y cos pf),
 * in fp32, rounded to bf16 once. Angles are reduced exactly, so far places are
 * as accurate as near ones.
 * q_out may be q and k_out may be k when the layouts in and out are the same (or
 * P = 1); any other overlap is XS_ERR_ALIAS. Extra rules: axis_dims even, in
 * multiples of 16 with XS_ROPE_HALVES (XS_ERR_UNSUPPORTED otherwise), their sum at
 * most D; Hk % P == 0; H + Hk <= 65536; pos 4-byte aligned.
 */
enum { XS_ROPE_HALVES = 1, XS_ROPE_INVERSE = 2, XS_ROPE_IN_SEQ = 4, XS_ROPE_OUT_SEQ = 8 };
xs_status xs_rope(const void *q, const void *k, void *q_out, void *k_out, const int32_t *pos, int pos_batches, int B,
                  int S, int H, int Hk, int D, int P, int n_axes, const int *axis_dims, const double *freqs, int flags,
                  void *stream);

/*
 * Attention through a sliding window with sinks, over whole sequences. Token i
 * of a head sees key token j of the same sequence iff
 *     j <= i + right   and   (j >= i - left  or  j < sinks):
 * the `left` tokens before it, itself, the `right` tokens after it, and, within
 * the same right end, the first `sinks` tokens of the sequence. -1 for left or
 * right sets no limit on that side: (left -1, right 0) is causal attention,
 * (left w, right w) a two-sided window, (left w, right 0) a causal window.
 *   q, k, v, out, scale : as for xs_attn (xs_attn_window, head-partitioned out)
 *            and xs_attn_a2a (xs_attn_window_a2a, All-to-All scatter); the second
 *            is bit-identical to xs_a2a_permute of the first. K/V tiles that no
 *            token of a query tile sees are skipped.
 *   workspace, workspace_bytes : device memory, 256-byte aligned, of at least
 *            xs_attn_window_workspace_size bytes; it needs no initialisation. With
 *            it the work is split evenly over the SMs, pieces of a query tile
 *            meeting in the workspace. NULL (with 0): whole query tiles only, and
 *            XS_ERR_WORKSPACE where those walk over more than 2^20 keys: sums in
 *            tensor memory truncate, and longer ones are added up in a workspace.
 * k and v must be finite: a key that a token does not see has no weight, but 0
 * times an infinity or NaN next to keys that it sees is NaN.
 * A row of q that is not finite gives an output row of no particular values, and
 * changes no other.
 * Rounding: scores, row maxima, sums and outputs are held in fp32; the softmax's weights
 * are rounded to bf16 (by at most 2^-8 each) before their product with v, the output once
 * at the end. Outputs differ from exact ones by 0.0021 to 0.0024 of their norm, 0.0017
 * being the output's own rounding.
 * left, right >= -1, sinks >= 0, S <= 2^24. D = 64, 96 or 128 (XS_ERR_UNSUPPORTED otherwise).
 */
xs_status xs_attn_window(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D, int P,
                         float scale, int left, int right, int sinks, void *workspace, size_t workspace_bytes,
                         void *stream);
xs_status xs_attn_window_a2a(const void *q, const void *k, const void *v, void *out, int B, int S, int H, int D, int P,
                             float scale, int left, int right, int sinks, void *workspace, size_t workspace_bytes,
                             void *stream);
xs_status xs_attn_window_workspace_size(int B, int S, int H, int D, int P, size_t *bytes);

/*
 * A paged key/value cache. A pool holds n_pages pages of `page` tokens each:
 *   k_pages, v_pages : [n_pages][page][Hk][D] bf16.
 * Each of N sequences has a row of the page table, and new tokens of all
 * sequences are packed one after the other:
 *   page_table : device [N][max_pages] int32; key j of sequence n is row j % page
 *            of page page_table[n][j / page]. Entries that no key of the
 *            sequence needs are not looked at and may hold anything.
 *   q_start : device [N + 1] int32, ascending from 0: sequence n's new tokens are the
 *            packed rows q_start[n] .. q_start[n + 1] - 1 (none if equal). Rows from
 *            q_start[N] up to T belong to no sequence.
 *   kv_len : device [N] int32, keys of each sequence, its new tokens included:
 *            new token i stands at place kv_len[n] - (q_start[n + 1] - q_start[n]) + i.
 *            A length of more than max_pages * page keys counts as that many, a
 *            negative one as none, here and in the two calls below.
 * All three are read by the kernels, so a captured call follows them when they
 * change between replays. They are not checked on the host. What they name
 * outside the pool, the table or the packed rows is never accessed: keys in
 * pages outside 0 .. n_pages - 1 are undefined in attention and are not written by
 * the append. With a kv_len past the table's end the new tokens stand at the
 * table's last places, are written there and attend from there.
 * page: a power of two from 16 to 1024; max_pages * page <= 2^29; N <= 65536;
 * T <= 2^29; D = 64, 96 or 128. N == 0 or T == 0 is an empty call, here and in the calls
 * below: it enqueues nothing, and its device pointers may be NULL.
 *
 * xs_cache_append writes the new tokens' keys and values,
 *   k, v : [T][Hk][D] bf16,
 * into their pages. Everything else in the pools stays as it is. Two tokens must
 * not land in one row (pages shared by two sequences are only for reading).
 */
xs_status xs_cache_append(const void *k, const void *v, void *k_pages, void *v_pages, const int32_t *page_table,
                          const int32_t *q_start, const int32_t *kv_len, int N, int T, int Hk, int D, int page,
                          int n_pages, int max_pages, void *stream);

/*
 * Attention of the new tokens over the cache (which holds their own keys too: append
 * first). The token at place i sees the keys 0 .. kv_len[n] - 1 of its sequence
 * under the rule of xs_attn_window; (-1, 0, 0) is causal attention over the
 * whole cache, for a chunk of a prompt or for single new tokens.
 *   q, out : [T][H][D] bf16; query head h reads key head h / (H / Hk). Rows of no
 *            sequence are left as they are in out. A token that sees no key
 *            (kv_len shorter than the new tokens) gets zeros.
 *   workspace, workspace_bytes : required (unless the call is empty), as for
 *            xs_attn_window, of xs_attn_paged_workspace_size bytes.
 * K and V of a sequence's own kv_len tokens must be finite; what lies behind them
 * in the last page, and in pages the window has passed, may hold anything. Rows of
 * q that are not finite, and rounding: as for xs_attn_window.
 * H % Hk == 0 and H / Hk <= 128.
 * Speed: the kernel's form is chosen on the host, from T * H / (N * Hk), the query rows
 * that a sequence and key head have on average: at most 16 (with D > 64, 24) mean single
 * tokens and tiles of few rows. A long chunk in such a call takes an item for each such
 * tile, and is faster in a call of its own (255 single tokens over 1000 keys with a chunk of
 * 256 over 8000, H = 64, Hk = 8: 616 us in one call, 246 in two). Single tokens in a call of
 * mostly chunks take tiles of 128 rows, which costs them 3 to 13%. Rows of no sequence
 * count in T too.
 */
xs_status xs_attn_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                        const int32_t *q_start, const int32_t *kv_len, void *out, int N, int T, int H, int Hk, int D,
                        int page, int n_pages, int max_pages, float scale, int left, int right, int sinks,
                        void *workspace, size_t workspace_bytes, void *stream);
xs_status xs_attn_paged_workspace_size(int N, int T, int H, int Hk, int D, size_t *bytes);

/*
 * The append with rotary positions on the way: of the new tokens, q is turned into
 * q_out, k is turned and written into its pages, v is written into its pages, in one
 * pass. It equals xs_rope of q and k followed by xs_cache_append, to the bit.
 *   q, k, v : rows of T tokens with H, Hk and Hk heads of D elements; a token's heads
 *            lie one after the other, and one token's row begins q_stride (k_stride,
 *            v_stride) elements behind the one before, so that q, k and v may be
 *            columns of one [T][(H + 2 Hk) D] projection. 0: H * D (Hk * D), rows
 *            without a gap. A stride is a multiple of 8, at least a row, at most 2^30.
 *   q_out  : [T][H][D] bf16. H = 0: no queries, q and q_out are ignored.
 *   k_out  : [T][Hk][D] bf16, the turned keys once more in packed rows (for
 *            xs_attn_packed); NULL: not wanted.
 *   pos    : device, [T][n_axes] int32, a token's place on each axis (any 32-bit
 *            value), as the trees of xs_tree_mask need; NULL, with one axis: its
 *            place in its sequence, kv_len[n] - new tokens + i.
 *   axis_dims, freqs, flags : as for xs_rope; of the flags XS_ROPE_HALVES alone.
 * Rows of no sequence are left as they are in q_out and k_out. A token whose place
 * lies before its sequence or whose page outside the pool is turned in q_out and k_out
 * and written into no page. q_out may be q, and k_out k, when their rows have no
 * gap; any other overlap of an output with another buffer is XS_ERR_ALIAS.
 * Extra rules: H + Hk <= 65536, T * max(H, Hk) < 2^31.
 */
xs_status xs_cache_append_rope(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, void *q_out, void *k_out, void *k_pages, void *v_pages,
                               const int32_t *page_table, const int32_t *q_start, const int32_t *kv_len,
                               const int32_t *pos, int N, int T, int H, int Hk, int D, int page, int n_pages,
                               int max_pages, int n_axes, const int *axis_dims, const double *freqs, int flags,
                               void *stream);

/*
 * Drafted token trees. The new tokens of a sequence may be a tree: each follows
 * the sequence's last token or another new token before it in the rows. All of them
 * are appended to the cache, one place each in the rows' order, and verified by one
 * attention call in which a token sees the context and the tokens that it follows.
 *
 * xs_tree_mask makes a tree's masks and positions from its tokens' parents, once for
 * all layers of a step:
 *   parents : device [T] int32, the parent's place among the sequence's new tokens;
 *            -1, or anything else that is not an earlier token of the sequence: the
 *            token follows the context.
 *   mask   : device [T][words] int32, overwritten: bit j % 32 of word j / 32 of row i
 *            is set iff j = i or token i follows token j, directly or not.
 *   pos    : device [T] int32, overwritten: the context's length (kv_len[n] - new
 *            tokens) plus the token's depth, 0 for those that follow the context; NULL:
 *            not wanted, and kv_len is not read (and may be NULL). This call knows no page
 *            table, so a kv_len past the table's end is not cut here: the positions are
 *            those of the length given, while the keys stand at the table's last places.
 *   q_start, kv_len, N, T : as below xs_cache_append.
 *   words  : 1 to 8. The first 32 * words new tokens of a sequence form its tree. Rows
 *            behind those get an empty mask and the context's length as position.
 * Rows of no sequence are left as they are.
 */
xs_status xs_tree_mask(const int32_t *parents, const int32_t *q_start, const int32_t *kv_len, int32_t *mask, int32_t *pos,
                       int N, int T, int words, void *stream);

/*
 * Attention of the new tokens over the cache (which holds their own keys too) under
 * masks of bits. With c = kv_len[n] - new tokens, token i of sequence n sees the keys
 * 0 .. c - 1, and key c + j iff bit j % 32 of word j / 32 of its row of mask is set;
 * bits of places at or past kv_len[n] are not looked at, and keys from c + 32 * words
 * on are not seen. The masks may be any, those of xs_tree_mask or not.
 *   mask   : device [T][words] int32, words 1 to 8.
 *   everything else: as for xs_attn_paged, without limits to the left. Keys and
 *            values of the new tokens must be finite, seen or not.
 *   workspace, workspace_bytes : as there, of xs_attn_tree_workspace_size bytes.
 * Speed: the form is chosen as there, but few rows mean at most 16 for every D. With
 * more, an item is 2 * floor(128 / (H / Hk)) tokens of a tree. Where all trees of a
 * call take equally many items, two to four, neighbouring SMs share what they read of K and V (16
 * trees of 64 tokens over 4000 to 16384 keys, H = 64, Hk = 8: 225 us, 246 each by itself); one tree
 * of another number among them ends that for the call.
 */
xs_status xs_attn_tree(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                       const int32_t *q_start, const int32_t *kv_len, const int32_t *mask, void *out, int N, int T, int H,
                       int Hk, int D, int page, int n_pages, int max_pages, int words, float scale, void *workspace,
                       size_t workspace_bytes, void *stream);
xs_status xs_attn_tree_workspace_size(int N, int T, int H, int Hk, int D, size_t *bytes);

/*
 * Attention over whole prompts of different lengths, packed one after the other.
 * Sequence n is the rows q_start[n] .. q_start[n + 1] - 1 of q, k, v and out, and its
 * token i sees its token j under the rule of xs_attn_window; (-1, 0, 0) is causal,
 * (-1, -1, 0) sees everything.
 *   q, k, v : rows of T tokens with H, Hk and Hk heads of D elements and the strides of
 *            xs_cache_append_rope; query head h reads key head h / (H / Hk).
 *   out    : [T][H][D] bf16. Rows of no sequence are left as they are.
 *   q_start, N, T : as below xs_cache_append; read by the kernels, so a captured call
 *            follows it when it changes between replays.
 *   workspace, workspace_bytes : required (unless the call is empty), as for
 *            xs_attn_window, of xs_attn_packed_workspace_size bytes.
 * k and v of a sequence's rows must be finite; rows of no sequence may hold anything,
 * and what one sequence holds touches no other. Rows of q that are not finite, and
 * rounding: as for xs_attn_window. H % Hk == 0 and H / Hk <= 128; N <= 65536;
 * T <= 2^29, T * H < 2^31; D = 64, 96 or 128.
 */
xs_status xs_attn_packed(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                         const int32_t *q_start, void *out, int N, int T, int H, int Hk, int D, float scale, int left,
                         int right, int sinks, void *workspace, size_t workspace_bytes, void *stream);
xs_status xs_attn_packed_workspace_size(int N, int T, int H, int Hk, int D, size_t *bytes);

/* Human-readable description of the last non-OK status returned on this host
 * thread (empty string if none). The pointer stays valid until the next call
 * on this thread. */
const char *xs_last_error(void);

/*
 * Synchronises `stream` and reads the device-side error word that the kernels
 * set when a bounded wait runs out. Returns XS_OK, XS_ERR_TIMEOUT (the word is
 * then cleared if `clear` != 0) or XS_ERR_CUDA if the synchronisation failed.
 */
xs_status xs_device_status(void *stream, int clear);

/*
 * Self-test of the bounded-wait path: launches one small kernel that waits on a
 * barrier nothing will ever complete, with a limit of `timeout_us` microseconds
 * (1 .. 2,000,000), then returns. The call synchronises `stream` and returns
 * XS_ERR_TIMEOUT when the wait ran out as designed (XS_OK would mean it did not),
 * leaving the device error word cleared afterwards.
 */
xs_status xs_selftest_wait_timeout(unsigned int timeout_us, void *stream);

/* Library version, major*10000 + minor*100 + patch. */
int xs_version(void);

#ifdef __cplusplus
}
#endif

#endif /* XS_H */
