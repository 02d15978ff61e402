// xs_span_schedule.cuh -- how the steps of a span attention call (items x K/V tiles) are
// shared out over the CTAs, and each CTA's walk through its part. Lengths are read on
// the device; one warp finds a part (span_schedule) and describes its stretches
// (span_next). See xs_span_kernel.cuh for what the steps are. Nothing here is tied to
// the tensor cores: the warp votes and shuffles apart this is plain arithmetic, which
// runs on the host as well.
#pragma once

#include <climits>

#include "xs_internal.h"

namespace xs {

// One CTA's share, found by span_schedule: first `rounds` whole items (blockIdx.x,
// blockIdx.x + ctas, ... in the items' order), then `rem` steps of the shared rest
// from (seq, head, pair, j) on.
struct SpanSched {
    long long shared, rem;  // steps shared out, of the call and of this CTA
    long long q;            // shared / ctas, and the remainder
    uint32_t r;
    int ctas;
    int rounds;
    int seq, head, pair, j;
    int cost;   // what an item counts for besides its steps
    int lanes;  // trees: CTAs that walk the same keys side by side (span_tree_lanes)
};
static_assert(sizeof(SpanSched) <= 64, "its place in shared memory");

constexpr int kSpanMaxChunks = 2048;  // groups of 32 sequences (or query tile pairs) in shared memory, 16 bytes each

// An item's K/V tiles by step y: hi, hi - 1, ... (nw of them, the window's), then
// ns - 1, ..., 0 (those of the sinks that lie before it).
struct SpanItem {
    int ntok;  // tokens of the item's tiles
    int tok0;  // first of them among the sequence's new tokens
    int pos0;  // its place
    int hi, nw, ns;
    int n;     // steps
    int s0, e1;  // pair: tile 0 takes part from step s0 on, tile 1 up to e1 and from nw on
    bool dual;
};

__device__ __forceinline__ SpanItem span_item(const SpanParams &p, int q_len, int keys, int pair) {
    SpanItem it;
    it.tok0 = pair * p.item_tok;
    it.ntok = min(p.item_tok, q_len - it.tok0);
    it.pos0 = keys - q_len + it.tok0;
    it.dual = it.ntok <= p.tile_tok;
    const int hi = min(keys - 1, it.pos0 + it.ntok - 1 + p.right);
    const int lo = max(0, it.pos0 - p.left) >> 7;
    it.s0 = it.ns = it.hi = 0;
    it.n = it.nw = it.e1 = 1;  // no key at all: one step, fully masked
    if (hi >= 0) {
        it.hi = hi >> 7;
        it.nw = it.hi - lo + 1;
        const int sink_tiles = (min(p.sinks, hi + 1) + 127) >> 7;
        it.ns = min(sink_tiles, lo);
        it.n = it.nw + it.ns;
        const int hi0 = max(0, min(keys - 1, it.pos0 + p.tile_tok - 1 + p.right)) >> 7;
        const int lo1 = max(0, it.pos0 + p.tile_tok - p.left) >> 7;
        it.s0 = it.hi - min(it.hi, max(hi0, lo));
        it.e1 = sink_tiles > lo ? it.nw : it.hi - min(lo1, it.hi) + 1;
    }
    return it;
}

// New tokens and keys of a sequence, cut to what the packed rows and the table hold.
// (KIND: a SpanKind.)
template <int KIND>
__device__ __forceinline__ void span_lengths(const SpanParams &p, int seq, int &q0, int &q_len, int &keys) {
    if (!KIND) {
        q0 = 0;
        q_len = keys = p.S;
        return;
    }
    q0 = min(max(p.q_start[seq], 0), p.T);
    q_len = max(0, min(max(p.q_start[seq + 1], 0), p.T) - q0);
    if (KIND == SPAN_PACKED) {
        keys = q_len;
        return;
    }
    keys = min(max(p.kv_len[seq], 0), p.max_pages * p.page);
}

__device__ __forceinline__ int span_pairs(const SpanParams &p, int q_len) {
    const int t2 = p.item_tok;
    return q_len <= t2 ? (q_len > 0) : (q_len + t2 - 1) / t2;
}

template <typename T> __device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
// Packed prompts and trees come in any lengths. What an item of theirs counts for, when the work
// is shared out, is its K/V steps and p.item_cost more for the change to it (12 prompts of 130 to
// 4001 tokens: CTAs with short prompts ran for 600 us where the others took 410). Not with fewer
// items than CTAs: a CTA's first item costs them all the same (span_schedule).
template <int KIND> __device__ __forceinline__ constexpr bool span_weighs() { return KIND >= SPAN_PACKED; }
// Packed prompts without a workspace: whole items are shared out, each a unit.
template <int KIND> __device__ __forceinline__ bool span_by_items(const SpanParams &p) { return KIND == SPAN_PACKED && !p.rec; }
// The items of a tree's key head walk the same keys. Where all trees have as many items a key head, two to four, that many
// neighbouring CTAs, the lanes, take the steps of one item each side by side and find in the L2 what the first of them has
// read: lane r shares the items r of all heads out over the CTAs r, r + lanes, ... 16 trees over 4000 to 16384 keys, 8 heads
// a key head, D = 128, so 32 tokens an item, us with lanes and without: 64 tokens 225, 246; 70 316, 340; 96 322, 354; 100
// 418, 446; 128 420, 471; but 40 tokens, whose second item holds 8, 236, 233, and 70 tokens of 4 heads a key head, D = 64,
// 185, 176. DRAM reads for 671 MB of K and V: 64 tokens 697 MB, 1317 without; 70 tokens, whose third item of 6 tokens soon
// runs ahead of the others, 1236.
__device__ __forceinline__ int span_tree_lanes(const SpanParams &p, int lane) {
    if (p.N > 1024) return 1;
    int lo = INT_MAX, hi = 0;
#pragma unroll 1
    for (int g = lane; g < p.N; g += 32) {
        int q0, q_len, keys;
        span_lengths<SPAN_TREE>(p, g, q0, q_len, keys);
        const int n = span_pairs(p, q_len);
        if (n > 0) {
            lo = min(lo, n);
            hi = max(hi, n);
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    return lo == hi && hi >= 2 && hi <= 4 && hi <= (int)gridDim.x ? hi : 1;
}
// Lanes of a call, a CTA's place among its lane's, and its lane.
template <int KIND> __device__ __forceinline__ int span_lanes(const SpanSched &s) { return KIND == SPAN_TREE_LANES ? s.lanes : 1; }
template <int KIND> __device__ __forceinline__ int span_cta(const SpanSched &s) {
    return KIND == SPAN_TREE_LANES && s.lanes > 1 ? (int)blockIdx.x / s.lanes : (int)blockIdx.x;
}
// The units of an item of n steps.
template <int KIND> __device__ __forceinline__ int span_units(const SpanParams &p, int n, int cost) {
    return span_by_items<KIND>(p) ? 1 : n + cost;
}

// Steps of the 32 groups of chunk ch, group ch * 32 + lane in each lane. A group
// is a sequence (all its heads and query rows) or, for whole sequences, which
// are all alike, a query tile pair of one head. `cost`: what an item counts for besides its steps.
template <int KIND>
__device__ __forceinline__ long long span_group_steps(const SpanParams &p, int ch, int lane, int cost) {
    const int g = ch * 32 + lane;
    if (!KIND) return g < p.n_pairs ? (long long)span_item(p, p.S, p.S, g).n : 0ll;
    int q0 = 0, q_len = 0, keys = 0;
    if (g < p.N) span_lengths<KIND>(p, g, q0, q_len, keys);
    const int pairs = span_pairs(p, q_len);
    long long u = pairs == 1 ? (long long)span_units<KIND>(p, span_item(p, q_len, keys, 0).n, cost) * p.heads : 0ll;
    uint32_t todo = __ballot_sync(0xffffffffu, pairs > 1);  // these the whole warp sums up, one after the other
#pragma unroll 1
    while (todo) {
        const int src = __ffs((int)todo) - 1;
        todo &= todo - 1;
        const int ql = __shfl_sync(0xffffffffu, q_len, src), kl = __shfl_sync(0xffffffffu, keys, src);
        const int np = span_pairs(p, ql);
        long long s = 0;
#pragma unroll 1
        for (int i = lane; i < np; i += 32) s += span_units<KIND>(p, span_item(p, ql, kl, i).n, cost);
        s = warp_sum(s);
        if (lane == src) u = s * p.heads;
    }
    return u;
}

// Items of the 32 groups of chunk ch.
template <int KIND> __device__ __forceinline__ long long span_group_items(const SpanParams &p, int ch, int lane) {
    int q0, q_len = 0, keys;
    const int g = ch * 32 + lane;
    if (g < p.N) span_lengths<KIND>(p, g, q0, q_len, keys);
    return (long long)span_pairs(p, q_len) * p.heads;
}

// First step of CTA c's part of the shared steps: floor(c * shared / ctas), with the
// quotient and remainder of shared / ctas (T is 32 bits wide unless they are not).
template <typename T> __device__ __forceinline__ T span_first(T q, uint32_t r, int ctas, int c) {
    return (T)c * q + (T)((uint32_t)c * r / (uint32_t)ctas);
}

// In a run of 32 values (one per lane, in order) that start at step `base`, the
// lane that holds step u, and the step its value starts at; base moves past the
// run. -1: behind the run.
template <typename T> __device__ __forceinline__ int span_locate(T v, T u, T &base, T &at, int lane) {
    T incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + incl > u);
    const int l = past ? __ffs((int)past) - 1 : -1;
    at = base + __shfl_sync(0xffffffffu, incl - v, l < 0 ? 0 : l);
    base += __shfl_sync(0xffffffffu, incl, 31);
    return l;
}

// (The loops of the schedule stay rolled: they run once, and their code is fetched cold.)

// Steps of chunk ch and `cost` for each of its items, from what span_chunk_sums has left.
// (A lane's share of them.)
template <int KIND>
__device__ __forceinline__ long long span_chunk_sum(const long long *sums, int chunks, int ch, int cost, int lanes) {
    if (!span_weighs<KIND>()) return sums[ch];
    const long long sum = sums[ch] + cost * sums[chunks + ch];
    return KIND == SPAN_TREE_LANES && lanes > 1 ? sum / lanes : sum;
}

// Where this CTA's part of the shared steps begins, by one warp. The shared steps
// are the call's from step `before` on. `sum`: the steps of one head (whole
// sequences). `mine`: the steps of this lane's group in the only chunk, when there
// is one; otherwise the chunks' sums are in `sums`.
template <typename T, int KIND>
__device__ __forceinline__ void span_find(const SpanParams &p, SpanSched &s, T before, long long sum, long long mine,
                                          int chunks, const long long *sums, int lane) {
    const int c = span_cta<KIND>(s), cost = span_weighs<KIND>() ? s.cost : 0, lanes = span_lanes<KIND>(s);
    const T total = (T)s.shared, q = total / (T)s.ctas;
    const uint32_t r = (uint32_t)(total - q * (T)s.ctas);
    s.q = (long long)q;
    s.r = r;
    const T u0 = span_first<T>(q, r, s.ctas, c);
    s.rem = (long long)(span_first<T>(q, r, s.ctas, c + 1) - u0);
    if (s.rem == 0) return;
    T u = before + u0, base = 0, at = 0;
    if (!KIND) {
        s.head = (int)(u / (T)sum);
        u -= (T)s.head * (T)sum;
    }
    int l = -1, ch = 0;
    if (chunks > 1) {
#pragma unroll 1
        for (; l < 0 && ch < chunks; ch += 32)
            l = span_locate<T>(ch + lane < chunks ? (T)span_chunk_sum<KIND>(sums, chunks, ch + lane, cost, lanes) : (T)0, u, base, at, lane);
        ch = ch - 32 + l;  // the chunk that holds step u, starting at step `at`
        base = at;
        mine = span_group_steps<KIND>(p, ch, lane, cost);
        if (lanes > 1) mine /= lanes;
    }
    l = span_locate<T>((T)mine, u, base, at, lane);
    u -= at;
    if (!KIND) {
        s.pair = ch * 32 + l;
        s.j = (int)u;
        return;
    }
    s.seq = ch * 32 + l;
    int q0, q_len, keys;
    span_lengths<KIND>(p, s.seq, q0, q_len, keys);
    const int np = span_pairs(p, q_len);
    if (np == 1 || lanes > 1) {
        if (lanes > 1) s.pair = (int)blockIdx.x - c * lanes;
        const T n = (T)span_units<KIND>(p, span_item(p, q_len, keys, 0).n, cost);
        s.head = (int)(u / n);
        s.j = (int)(u - (T)s.head * n);
        return;
    }
    T per_head = 0;
#pragma unroll 1
    for (int i = lane; i < np; i += 32) per_head += (T)span_units<KIND>(p, span_item(p, q_len, keys, i).n, cost);
    per_head = warp_sum(per_head);
    s.head = (int)(u / per_head);
    u -= (T)s.head * per_head;
    base = 0;
    l = -1;
    int i = 0;
#pragma unroll 1
    for (; l < 0 && i < np; i += 32)
        l = span_locate<T>(i + lane < np ? (T)span_units<KIND>(p, span_item(p, q_len, keys, i + lane).n, cost) : (T)0, u, base, at, lane);
    s.pair = i - 32 + l;
    s.j = (int)(u - at);
}

// Whole items dealt out round by round first, and the steps they hold (whole
// sequences). None unless the items are of about one length (their mean at least
// 4/5 of the longest: a CTA's rounds then end about when the others' do) and
// there are two for each CTA. S = 4096, H = 48, D = 128, windows to the left: mean 0.62 of the
// longest, 182 us in rounds and 164 without; 0.75 154 and 144; 0.81 131 and 128; 0.88 106 and
// 122; 0.94 83 and 89. All full rounds are dealt out, however little is left: sharing the
// last of them too costs 2 to 20% (two-sided window of 512, S = 4096: 60.7 us, 64.9 with 23 heads,
// 0.42 items a CTA left; 57.3, 62.2 with 22; 52.3, 56.4 with 20; 104.1, 107.8 with 48, 5
// rounds). Of many rounds of long items it gains 1%: S = 16384, H = 24, 10 rounds of up to 35
// steps and 0.1 items left 501 us, 496 shared; S = 8192, 5 rounds of up to 18, 0.05 left
// 160.1, 158.6; 0.26 164.3, 163.1; 0.47 168.7, 173.5; but 2 rounds 75.1, 82.2. `sum`: the
// steps of one head.
__device__ __forceinline__ int span_rounds(const SpanParams &p, int grid, long long sum, int lane, long long &steps) {
    steps = 0;
    const long long items = (long long)p.heads * p.n_pairs;
    int most = max(span_item(p, p.S, p.S, p.n_pairs >> 1).n, span_item(p, p.S, p.S, p.n_pairs - 1).n);
    most = max(most, span_item(p, p.S, p.S, 0).n);
    if (items < 2ll * grid || 5 * sum < 4ll * p.n_pairs * most) return 0;
    int rounds = (int)(items / grid);
    const int rest = (int)(items - (long long)rounds * grid);
    if (rest && rounds >= 5 && most >= 16 && 5 * rest < 2 * grid) --rounds;
    const long long first = (long long)rounds * grid, head = first / p.n_pairs;  // the first shared item
    const int pairs = (int)(first - head * p.n_pairs);
#pragma unroll 1
    for (int i = lane; i < pairs; i += 32) steps += span_item(p, p.S, p.S, i).n;
    steps = warp_sum(steps) + head * sum;
    return rounds;
}

// Sums of the steps of 32 groups each, when there are more, and behind them of their items where
// those count; by all threads, and followed by a barrier.
template <int KIND> __device__ __forceinline__ void span_chunk_sums(const SpanParams &p, int chunks, long long *sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int ch = warp; ch < chunks; ch += (int)(blockDim.x >> 5)) {
        const long long s = warp_sum(span_group_steps<KIND>(p, ch, lane, 0));
        if (lane == 0) sums[ch] = s;
        if (span_weighs<KIND>()) {
            const long long i = warp_sum(span_group_items<KIND>(p, ch, lane));
            if (lane == 0) sums[chunks + ch] = i;
        }
    }
}

// The call's steps, how many CTAs share them and where this CTA's part starts; by one warp.
template <int KIND>
__device__ __forceinline__ SpanSched span_schedule(const SpanParams &p, int chunks, const long long *sums, int lane) {
    long long mine = 0, sum = 0, items = 0;
    if (chunks > 1) {
#pragma unroll 1
        for (int ch = lane; ch < chunks; ch += 32) {
            sum += sums[ch];
            if (span_weighs<KIND>()) items += sums[chunks + ch];
        }
    } else {
        sum = mine = span_group_steps<KIND>(p, 0, lane, 0);
        if (span_weighs<KIND>()) items = span_group_items<KIND>(p, 0, lane);
    }
    sum = warp_sum(sum);
    int cost = 0;
    if (span_weighs<KIND>()) {
        const long long all = warp_sum(items);
        if (all > (long long)gridDim.x && !span_by_items<KIND>(p)) {
            cost = p.item_cost;
            sum += cost * all;
            mine += cost * items;
        }
    }
    SpanSched s;
    int grid = (int)gridDim.x;
    s.cost = cost;
    if (KIND == SPAN_TREE_LANES) {
        s.lanes = span_tree_lanes(p, lane);
        if (s.lanes > 1) {  // a lane's: a key head's items are alike
            sum /= s.lanes;
            mine /= s.lanes;
            grid /= s.lanes;
        }
    }
    const long long total = KIND ? sum : sum * p.heads;  // whole sequences: `sum` is one head's
    // parts of a few steps or more, or a CTA for each key head of the sequences
    const long long least = KIND ? min(total, (long long)p.N * p.heads) : 0ll;
    s.ctas = (int)max(1ll, min((long long)grid, max(total >> (span_by_items<KIND>(p) ? 0 : p.min_steps_log2), least)));
    s.rem = s.q = 0;
    s.r = 0;
    s.rounds = s.seq = s.head = s.pair = s.j = 0;
    long long before = 0;
    if (!KIND && s.ctas == (int)gridDim.x) s.rounds = span_rounds(p, s.ctas, sum, lane, before);
    s.shared = total - before;
    // Every CTA that shares them has a step: a part without one between two pieces of an item would
    // have written no record for the merge.
    if (s.shared > 0 && s.shared < s.ctas) s.ctas = (int)s.shared;
    if (span_cta<KIND>(s) < s.ctas && s.shared > 0) {
        if (total < (1ll << 31))
            span_find<uint32_t, KIND>(p, s, (uint32_t)before, sum, mine, chunks, sums, lane);
        else
            span_find<unsigned long long, KIND>(p, s, (unsigned long long)before, sum, mine, chunks, sums, lane);
    }
    return s;
}

// The CTA whose part holds shared step u.
__device__ __forceinline__ int span_cta_of(const SpanSched &s, long long u) {
    return (int)(((u + 1) * s.ctas - 1) / s.shared);
}

// The walk through a CTA's share, one stretch (segment) of an item at a time.
struct SpanWalk {
    int rounds;      // whole items left
    long long rem;   // shared steps left
    int seq, head, pair, j;
    int q0, q_len, keys;
    bool first;      // no shared segment yet
};
// What a CTA has of an item, its part, is one segment, or several of p.stretch steps: O of a
// segment is one sum in tensor memory, whose additions truncate (values of 1: 0.4% are missing
// after 2^20 keys, 2.3% after 2^22; in two chains 1.2% after 2^22, 5% after 2^24). Segments
// of a part are added up in a workspace record (the epilogue).
enum : int {
    SPAN_PIECE = 1,  // the part is not the whole item
    SPAN_ADD = 2,    // not the part's first segment
    SPAN_MORE = 4,   // not its last: the steps behind it
    SPAN_REST = 3    // are flags >> SPAN_REST
};
// What the roles need to know of a segment (96 bytes: with 100, mixed paged batch 80.7 us instead of 80.3).
struct SpanSeg {
    int n;            // steps; 0: no segment, the roles are done
    int j0;           // the item's step that it starts with
    int dual, flags;
    int hi, nw, ns, s0, e1;
    int seq, head;
    int q0, tok0, ntok;  // the sequence's first packed row; the item's first token, their number
    int pos0, keys;      // the first token's place; the sequence's keys
    int slot;            // the part's workspace record
    int fix;             // rows of the first V tile that hold keys, where the rest has to be cleared; -1: nothing to do
    int lo, last;        // first key of the window, last key that any token sees
    // a row of tile t misses a key of the K/V tile at c0 iff c0 > all_hi[t], or
    // c0 < all_lo[t] and the tile's keys are not all sinks
    int all_hi[2], all_lo[2];
};
static_assert(sizeof(SpanSeg) == 96, "segment ring");
__device__ __forceinline__ int span_tile(const volatile SpanSeg &g, int y) {
    const int nw = g.nw;
    return y < nw ? g.hi - y : g.ns - 1 - (y - nw);
}
// Moves the walk `by` items on in the items' order (whole sequences).
__device__ __forceinline__ void span_skip(const SpanParams &p, SpanWalk &w, int by) {
    const int at = w.pair + by, heads = at / p.n_pairs;
    w.head += heads;
    w.pair = at - heads * p.n_pairs;
}
// The walk's start in the shared steps.
template <int KIND>
__device__ __forceinline__ void span_walk_shared(const SpanParams &p, const SpanSched &s, SpanWalk &w) {
    w.rem = s.rem;
    w.seq = s.seq;
    w.head = s.head;
    w.pair = s.pair;
    w.j = s.j;
    if (w.rem > 0) span_lengths<KIND>(p, w.seq, w.q0, w.q_len, w.keys);
}
template <int KIND>
__device__ __forceinline__ void span_walk_init(const SpanParams &p, const SpanSched &s, SpanWalk &w) {
    w.first = true;
    w.rounds = 0;
    if (KIND) {
        span_walk_shared<KIND>(p, s, w);
        return;
    }
    if (p.rec) {
        w.rounds = s.rounds;
    } else {  // no workspace: whole items only
        const long long items = (long long)p.heads * p.n_pairs;
        w.rounds = (int)((items - blockIdx.x + gridDim.x - 1) / gridDim.x);
    }
    if (w.rounds == 0) {
        span_walk_shared<KIND>(p, s, w);
        return;
    }
    w.rem = 0;
    w.seq = w.head = w.pair = w.j = 0;
    span_lengths<KIND>(p, 0, w.q0, w.q_len, w.keys);
    span_skip(p, w, (int)blockIdx.x);
}
// The walk's next shared item.
template <int KIND> __device__ __forceinline__ void span_next_item(const SpanParams &p, const SpanSched &s, SpanWalk &w) {
    w.j = 0;
    const bool lanes = span_lanes<KIND>(s) > 1;  // the item of the next head
    if (lanes || ++w.pair * p.item_tok >= w.q_len) {
        if (!lanes) w.pair = 0;
        if (++w.head == p.heads) {
            w.head = 0;
            w.q_len = KIND ? 0 : w.q_len;  // the next sequence is looked up when it is needed
        }
    }
}
// The next part, as one segment; no steps and no flags if there is none.
template <int KIND>
__device__ __forceinline__ bool span_next(const SpanParams &p, const SpanSched &sched, SpanWalk &w, SpanSeg &g) {
    g.n = g.flags = 0;  // (no segment, unless one is described below)
    if ((KIND || w.rounds == 0) && w.rem <= 0) return false;
    if (KIND)
        while (w.q_len == 0) {
            if (++w.seq >= p.N) return false;
            span_lengths<KIND>(p, w.seq, w.q0, w.q_len, w.keys);
        }
    const SpanItem it = span_item(p, w.q_len, w.keys, w.pair);
    const int w_keys = w.keys;
    g.dual = it.dual;
    g.hi = it.hi;
    g.nw = it.nw;
    g.ns = it.ns;
    g.s0 = it.s0;
    g.e1 = it.e1;
    g.seq = w.seq;
    g.head = w.head;
    g.q0 = w.q0;
    g.tok0 = it.tok0;
    g.ntok = it.ntok;
    g.pos0 = it.pos0;
    g.keys = w.keys;
    g.lo = max(0, it.pos0 - p.left);
    g.last = min(w.keys - 1, it.pos0 + it.ntok - 1 + p.right);
    g.slot = 2 * (int)blockIdx.x + (w.first ? 0 : 1);
    if (!KIND && w.rounds > 0) {
        g.j0 = 0;
        g.n = it.n;
        if (--w.rounds > 0)
            span_skip(p, w, (int)gridDim.x);
        else if (p.rec)
            span_walk_shared<KIND>(p, sched, w);
    } else if (span_by_items<KIND>(p)) {
        g.j0 = 0;
        g.n = it.n;
        --w.rem;
        span_next_item<KIND>(p, sched, w);
    } else {
        // The item's steps lie behind `lead` units, which stand for the change to it.
        const int lead = span_weighs<KIND>() ? sched.cost : 0;
        if (span_weighs<KIND>()) {
            const int skip = max(lead - w.j, 0);
            if (w.rem <= skip) return false;  // the part ends before them
            w.rem -= skip;
            w.j += skip;
        }
        w.first = false;
        g.j0 = w.j - lead;
        g.n = (int)min((long long)(it.n + lead - w.j), w.rem);
        w.rem -= g.n;
        w.j += g.n;
        if (w.j == it.n + lead) span_next_item<KIND>(p, sched, w);
    }
    g.flags = g.n < it.n ? SPAN_PIECE : 0;
    for (int t = 0; t < 2; ++t) {
        if (kIsTree<KIND>) {  // every token sees all keys before the sequence's new tokens
            g.all_hi[t] = it.pos0 - it.tok0 - 128;
            g.all_lo[t] = INT_MIN;
            continue;
        }
        const int tt = it.dual ? 0 : t * p.tile_tok, toks = min(it.ntok - tt, p.tile_tok);
        g.all_hi[t] = min(it.pos0 + tt + p.right, w_keys - 1) - 127;
        g.all_lo[t] = it.pos0 + tt + toks - 1 - p.left;
    }
    // rows behind the last key, in a box that holds keys (boxes without are zeros)
    const int box = KIND ? min(p.page, 128) : 128;
    g.fix = KIND && g.j0 == 0 && it.hi == w_keys >> 7 && (w_keys & (box - 1)) ? w_keys & 127 : -1;
    return true;
}

// Cuts what follows the first `stretch` steps off a part.
__device__ __forceinline__ void span_cut(SpanSeg &g, int stretch) {
    const int rest = max(g.n - stretch, 0);
    g.n -= rest;
    if (rest) g.flags |= SPAN_MORE | rest << SPAN_REST;
}
// The segment d that follows segment o in its part.
__device__ __forceinline__ void span_continue(volatile SpanSeg &d, const volatile SpanSeg &o, int stretch) {
#pragma unroll 1
    for (int i = 0; i < (int)(sizeof(SpanSeg) / sizeof(int)); ++i)
        reinterpret_cast<volatile int *>(&d)[i] = reinterpret_cast<const volatile int *>(&o)[i];
    const int rest = o.flags >> SPAN_REST;
    d.j0 = o.j0 + o.n;
    d.n = min(rest, stretch);
    d.fix = -1;
    d.flags = (o.flags & SPAN_PIECE) | SPAN_ADD | (rest > stretch ? SPAN_MORE | (rest - stretch) << SPAN_REST : 0);
}

// Written by each CTA for span_merge_kernel: the item whose first piece is the
// CTA's last part (pieces 0: none).
struct SpanPieces {
    int pieces, slot, seq, head, tok0, ntok, q0;
    int lanes;  // trees: the pieces' CTAs are so far apart
};
// Of a part that is an item's first piece: its pieces lie in this CTA and the next ones.
template <int KIND = SPAN_WHOLE>
__device__ __forceinline__ SpanPieces span_pieces_of(const SpanSched &s, const SpanSeg &g) {
    const int left = g.nw + g.ns - g.n, c = span_cta<KIND>(s);
    const long long end = span_first<unsigned long long>(s.q, s.r, s.ctas, c + 1) + left;  // behind the item's last step
    return SpanPieces{span_cta_of(s, end - 1) - c + 1, g.slot, g.seq, g.head, g.tok0, g.ntok, g.q0, KIND == SPAN_TREE_LANES ? s.lanes : 0};
}

}  // namespace xs
