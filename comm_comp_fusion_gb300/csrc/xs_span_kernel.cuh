// xs_span_kernel.cuh -- attention over a span of keys per token on the tensor
// cores: a sliding window with sinks over whole sequences of equal lengths
// (xs_attn_window), or packed ones (xs_attn_packed), chunks of new tokens over a paged
// cache (xs_attn_paged), drafted trees over it (xs_attn_tree). KIND, a SpanKind, says which.
//
// Mathematics. The token at place i sees the key at place j iff
//   j <= i + right  and  (j >= i - left  or  j < sinks),
// (a tree's token: iff j lies before the sequence's new tokens, or its mask has the bit of j),
// and o = sum_j p_j v_j / sum_j p_j, p_j = 2^(s_j scale log2(e) - m) over the keys
// it sees; a token that sees none gets zeros. S = Q K^T and P V run on tcgen05
// with fp32 accumulators in tensor memory; row maxima, sums and O stay in fp32;
// P is rounded to bf16 for the product with V, the type that the tensor cores take with a
// bf16 V: at most 2^-8 of each weight. The sums use the unrounded p. Against 64 bits the
// results are off by 0.0021 to 0.0024 of their norm, of which the output's own rounding makes 0.0017.
//
// Rows. A query tile is 128 rows: 128 tokens of one head, or, with G query heads
// per key head, floor(128 / G) tokens x G heads, so that the heads of a group
// share the K/V tiles they read. An item is one key head of one sequence and
// two query tiles; it walks the 128-key tiles that any of its tokens sees, from
// the window's last down to its first (with a causal mask every row then meets
// a key of its own at once, which is what the running maximum wants), then the
// sinks'. Keys outside a row's own span are masked in the tiles where some row
// has any.
//   * Two tiles (pair): each K/V tile is used by both, one tile's softmax running
//     under the other's MMAs. A K/V tile that only one of them sees (at the
//     window's ends) costs the other nothing. Where a pair follows a pair, its first S
//     is issued with the last step before it (12 packed prompts 631 us, 536 with it and
//     the elected issuer; two-sided window S = 4096 64.0, 61.7).
//   * One tile (dual; the last rows of a chunk): the even and the odd K/V tiles
//     form two chains with an O of their own each, which the epilogue adds up. A
//     chain's step is a long dependent sequence (MMA, softmax, MMA), so two of
//     them are what keeps K/V streaming.
//   * Few rows (FEW = 16 or 32; single new tokens): dual with the products
//     turned round, S^T = K Q^T and O^T = V^T P^T, so that the 128 rows of an MMA
//     are keys (or columns of V) and the query rows are its N. A softmax thread
//     then holds one key's scores of all rows: 16 exponentials a step where the
//     other form spends 128 on rows that mostly do not exist (16 single tokens of 8
//     heads a key head over 4000 keys, D = 128: 48.3 us against 52.9, D = 64 32.9
//     against 35.9; four over 1000 keys, 14 rows, 12.7 against 13.9; both sides of
//     the choice at xs_attn_paged in xs_ops_api.cpp).
//
// Schedule. The steps (items x K/V tiles) of the whole call form one sequence,
// ordered by sequence, head and query rows, and each CTA takes an equal,
// contiguous part. Of whole sequences with several items of about one length for
// each CTA, whole items are dealt out round by round first, and only what is left is
// shared out in steps: the CTAs then work on neighbouring query rows of a few
// heads at a time, whose K/V stay in L2 (S = 16384, H = 24, a window of 4096: 2.85
// GB of DRAM reads without the rounds, for 0.3 GB of inputs). Lengths are read on
// the device: every CTA sums the steps per sequence and finds its part by itself
// (span_schedule), so the call can be captured and replayed with other lengths.
// An item that a part's border cuts is computed in pieces; each piece writes its
// unnormalised O, row maxima and sums to the workspace, and span_merge_kernel
// adds them up in piece order (no atomics: the result is the same every time).
// Packed prompts and trees: an item counts for two steps more than it has, short packed
// calls take whole items, and alike trees walk side by side (xs_span_schedule.cuh).
//
// Long items (LONG). The tensor cores' additions to O truncate: with values of 1, one sum over
// 2^18 keys still rounds to 1, after 2^20 0.4% are missing, after 2^22 2.3%. Where a
// sequence can hold more than 2^18 keys, what a CTA has of an item is therefore taken in
// segments of 2048 tiles, each with a sum, maxima and row sums of its own. A segment's O goes
// to the CTA's third record and is added to its part's record, in fp32 and rounded to
// nearest, by the thread that has the row (or, with few rows, the column). These are instances
// apart: their code costs short items 1 to 3% (mixed paged batch 82.9 us instead of 80.4).
// They also keep every wait far below its limit, however long the sequence.
//
// Bounds. Single new tokens: HBM (32 sequences of 16000 keys, 8 key heads, D = 128, pages
// of 32 tokens and more: 305 us, 6.9 TB/s; D = 64 and 96 reach 5.4; pages of 16 tokens
// 5.9, their boxes' issue being the limit). Long chunks and windows: the chain S -
// softmax - P V of a step, 2600 to 2850 cycles for two tiles at D = 128 (chunks of 2048
// over 16K keys, 32 heads: 630 us at best, 1.70 PFLOP/s, and 742 in a stream of calls, at the
// power limit; one packed prompt of 16384, 40 and 8 heads, causal: 1560, 1.76 PFLOP/s, and
// 1693). Items of few steps (a two-sided window of 512: 10; packed prompts of 4000 tokens, 4
// heads a key head: 16 on average): what lies between two items, about 5400 cycles of masked
// steps and cold code (a line of instructions not met lately takes some 120), and steps that
// few rows need whole. Short calls: about 8 us of set-up, first loads and first steps, whose
// instructions are fetched cold.
//
// Roles of the 512 threads:
//   warp 0      TMA producer: Q tiles, then K and V tiles into a 128 KB ring. Pages
//               shorter than a tile take one box each, issued by as many lanes (by
//               one lane in turn: 431 us instead of 371 for 32 long single tokens);
//               page numbers are fetched three tiles ahead. Pages that no token
//               sees are not read (their box lies outside the pool: zeros).
//   warp 1      MMA issuer
//   warp 2      tensor-memory allocator, then the schedule: it walks the CTA's part
//               and describes each stretch of an item (SpanSeg) in a ring in shared
//               memory, ahead of the other roles
//   warp 3      (paged, packed) zeroes the V rows behind the last key, which no one has
//               written or which are another sequence's: a weight of 0 times NaN would still be NaN
//   warps 4-11  softmax, one warpgroup per tile or chain, one thread per row
//   warps 12-15 epilogue
#pragma once

#include "xs_attn_kernel.cuh"
#include "xs_span_schedule.cuh"

namespace xs {

// One lane of the warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// 32 lanes x 32-bit, 16 consecutive columns per thread, to tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// The same value to 32 columns.
__device__ __forceinline__ void tmem_fill32(uint32_t taddr, uint32_t v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(taddr),
        "r"(v)
        : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint32_t x) {
    asm volatile("{\n\t.reg .b16 h, z;\n\tmov.b32 {h, z}, %1;\n\tst.shared.b16 [%0], h;\n\t}" ::"r"(a), "r"(x) : "memory");
}

// Bounded waits in few instructions, a retry in a loop: there are some forty of them, and
// what the kernel spends between two items is to a good part the fetch of code. With
// each wait's retries unrolled it held 300 KB of it instead of 175: two-sided window S =
// 4096 78 us instead of 67, S = 16384 545 instead of 497, four short single tokens 14.7
// instead of 12.8.
__device__ __forceinline__ bool span_bwait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, uint32_t site) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    int i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (++i & 63) continue;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 0x80000000u | (1u << site);  // the kernel's end passes it on
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool span_warp_bwait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, uint32_t site) {
    const bool ok = span_bwait(bar, parity, abort_flag, site);
    return __all_sync(0xffffffffu, ok);
}

constexpr int kSegs = 6;  // segments in the ring
// mbarriers; per query tile (chain) 2 of each of the first eight, per ring slot 2, per segment 2.
enum : int {
    SPQ_FULL = 0, SPQ_EMPTY = 2, SPS_FULL = 4, SPP_FULL = 6, SPO_FINAL = 8, SPO_FREE = 10, SPL_FULL = 12, SPL_EMPTY = 14,
    SP_DRAIN = 16, SPFIX_ASK = 17, SPFIX_DONE = 18,  // the issuer asks warp 3 to clear a V tile's end, and its answer
    SPCHAIN = 19,                                    // few rows: the four softmax warps of a chain meet
    SPKV_FULL = 21, SPKV_EMPTY = 31, SPSEG_FULL = 41, SPSEG_EMPTY = 41 + kSegs, SP_BARS = 41 + 2 * kSegs
};
enum SpanSite : uint32_t { kSiteFix = 13, kSiteSeg = 14 };

// FEW: query rows of a tile in the few-rows form; 0: tiles of 128 rows.
template <int D, int KIND, int FEW> struct SpanCfg {
    // Registers a thread of warps 0-3, of the softmax warps and of the epilogue's. One split for
    // both calls with 128-row tiles costs 2-3% of one of them (56 / 176 / 104: two-sided window
    // S = 4096 65.1 us, mixed paged batch 83.0; 48 / 184 / 96: 66.3 and 80.6); few rows have few scores.
    static constexpr int kRegsOther = FEW ? 80 : KIND ? 48 : 56;
    static constexpr int kRegsSoftmax = FEW ? 160 : KIND ? 184 : 176;
    static constexpr int kRegsEpilogue = FEW ? 112 : KIND ? 96 : 104;
    static_assert(kRegsOther + 2 * kRegsSoftmax + kRegsEpilogue == 4 * 128, "the registers the block is launched with");
    static constexpr int kNDB = Cfg<D>::kNDB;
    static constexpr uint32_t kBlk = Cfg<D>::kBlk, kTile = Cfg<D>::kTile;
    // K/V ring of 128 KB, in 16 KB (D = 64) or 32 KB slots. More in flight, where few
    // rows leave the room, was slower: 32 single tokens over 16000 keys of 8 heads, D =
    // 128, 320 us with 4 slots, 328 with 5, 339 with 6.
    static constexpr int kSlots = D == 64 ? 8 : 4;
    static constexpr uint32_t kOffKV = 0;
    // Q: two tiles of the item, or with few rows two items' tiles
    static constexpr uint32_t kQBlk = FEW ? FEW * 128u : kBlk, kQTile = kNDB * kQBlk;
    static constexpr uint32_t kOffQ = kOffKV + kSlots * kTile;
    static constexpr uint32_t kStageWarp = Cfg<D>::kStageWarp;
    static constexpr uint32_t kOffStage = kOffQ + 2 * kQTile;  // output rows; few rows: P of the two chains
    static constexpr uint32_t kPTile = 2u * FEW * 128u;        // P: [64-key block][row][64 keys]
    // few rows at D = 64: V^T is read as 128 rows, the last 64 from the next slot or,
    // behind the ring, from here (they end in rows of O^T that nothing reads)
    static constexpr uint32_t kBehind = FEW ? 2 * kPTile : 4 * kStageWarp;
    static constexpr uint32_t kPad = 2 * kQTile + kBehind < kBlk ? kBlk - 2 * kQTile - kBehind : 0;
    static constexpr uint32_t kOffRed = kOffStage + kBehind + kPad;    // few rows: float [chain][4 warps + m, exponent, alpha][FEW]
    static constexpr uint32_t kOffBar = kOffRed + (FEW ? 2u * 8u * FEW * 4u : 0u);
    static constexpr uint32_t kOffL = kOffBar + 8 * ((SP_BARS + 1) & ~1);  // float [tile][l, m][128]
    static constexpr uint32_t kOffMisc = kOffL + 2 * 2 * 128 * 4;          // tmem base, abort flag, chain flags
    static constexpr uint32_t kOffSeg = kOffMisc + 16;                     // the ring of segments, then a SpanSched
    static constexpr uint32_t kSmemAlloc = kOffSeg + (uint32_t)sizeof(SpanSeg) * kSegs + 64 + 1024;
    __host__ __device__ static constexpr uint32_t colS(int t) { return (FEW ? (uint32_t)FEW : 128u) * (uint32_t)t; }
    __host__ __device__ static constexpr uint32_t colO(int t) {
        return FEW ? (uint32_t)FEW * (uint32_t)(2 + t) : 256u + (uint32_t)D * (uint32_t)t;
    }
    static constexpr uint32_t kTmemCols = FEW ? 4 * FEW : 512;
    static_assert(kSmemAlloc <= 232448, "shared memory budget");
    static_assert(kSlots <= SPKV_EMPTY - SPKV_FULL, "barriers of the ring");
    static_assert(kSlots * kTile >= 16u * kSpanMaxChunks, "the schedule's sums");
    static_assert((kOffSeg + sizeof(SpanSeg) * kSegs) % 8 == 0, "the SpanSched's place");
    static_assert(kOffQ % 1024 == 0 && kOffStage % 1024 == 0, "swizzled tiles");
};

constexpr float kSpanRise = 16384.0f;  // see the softmax
constexpr int kMidSteps = 4;           // see the issuer

// row / G of a query tile's row
template <int KIND> __device__ __forceinline__ int span_row_tok(const SpanParams &p, int row) {
    return KIND ? (int)((uint32_t)row * p.g_magic >> 16) : row;
}

// Element offset of the output row of token `tok` (of the sequence's new tokens,
// packed rows from q0) and query head g of the group.
template <int D, int KIND>
__device__ __forceinline__ int64_t span_out_offset(const SpanParams &p, int head, int64_t q0, int tok, int g) {
    if (KIND) return ((q0 + tok) * p.H + (int64_t)head * p.G + g) * D;
    const int hl = head % p.Hl, rb = head / p.Hl;
    if (p.head_out) return (((int64_t)rb * p.S + tok) * p.Hl + hl) * D;
    const int b = rb % p.B, r = rb / p.B;
    const int rd = tok / p.Sl;
    return ((((int64_t)rd * p.B + b) * p.Sl + (tok - rd * p.Sl)) * p.H + r * p.Hl + hl) * D;
}

// Bits of the 32 columns from col0 (relative to the tile) that a row sees: columns
// a .. b, and those below s up to b.
__device__ __forceinline__ uint32_t span_mask_word(int a, int b, int s, int col0) {
    a -= col0;
    b -= col0;
    s -= col0;
    const uint32_t le = b < 0 ? 0u : b >= 31 ? ~0u : (2u << b) - 1u;
    const uint32_t ge = a <= 0 ? ~0u : a > 31 ? 0u : ~0u << a;
    const uint32_t lt = s <= 0 ? 0u : s > 31 ? ~0u : (1u << s) - 1u;
    return le & (ge | lt);
}

// Word w of a tree token's mask, for places counted from the sequence's first new token: those before it
// are seen, those behind the mask are not.
__device__ __forceinline__ uint32_t span_tree_word(const int *mask, int words, int w) {
    return w < 0 ? ~0u : w < words ? (uint32_t)mask[w] : 0u;
}
// Few rows: the rows of the item (bits) that see the key at place `key`.
template <int FEW> __device__ __forceinline__ uint32_t span_tree_rows(const SpanParams &p, const volatile SpanSeg &g, int key) {
    const int at = key - (g.pos0 - g.tok0), ntok = g.ntok;
    if (key >= g.keys) return 0u;
    if (at < 0) return ~0u;
    if (at >= 32 * p.words) return 0u;
    const int *mask = p.mask + ((int64_t)g.q0 + g.tok0) * p.words + (at >> 5);
    const uint32_t group = p.G < 32 ? (1u << p.G) - 1u : ~0u;
    uint32_t rows = 0;
#pragma unroll 4
    for (int i = 0; i < ntok; ++i)
        if (((uint32_t)mask[(int64_t)i * p.words] >> (at & 31)) & 1u) rows |= group << (i * p.G);
    return rows;
}

template <int D, int KIND, int FEW, bool LONG>
__global__ void __launch_bounds__(512, 1)
    span_attn_kernel(const __grid_constant__ SpanMaps tm, const __grid_constant__ SpanParams p) {
    using C = SpanCfg<D, KIND, FEW>;
    using R = Rec<D>;
    constexpr bool kPages = KIND == SPAN_PAGED || kIsTree<KIND>;  // K and V lie in pages
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - raw);
    const uint32_t sQ = base + C::kOffQ, sKV = base + C::kOffKV, sStage = base + C::kOffStage;
    const uint32_t sBar = base + C::kOffBar;
    float *row_ml = reinterpret_cast<float *>(sm + C::kOffL);
    uint32_t *misc = reinterpret_cast<uint32_t *>(sm + C::kOffMisc);
    volatile uint32_t *abort_flag = misc + 1;
    volatile SpanSeg *segs = reinterpret_cast<volatile SpanSeg *>(sm + C::kOffSeg);
#define BAR(i) (sBar + 8u * (uint32_t)(i))
#define SEG_FULL(i) BAR(SPSEG_FULL + (i))
#define SEG_EMPTY(i) BAR(SPSEG_EMPTY + (i))
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(BAR(SPQ_FULL + t), 1);
            mbar_init(BAR(SPQ_EMPTY + t), 1);
            mbar_init(BAR(SPS_FULL + t), 1);
            mbar_init(BAR(SPP_FULL + t), 4);
            mbar_init(BAR(SPO_FINAL + t), 1);
            mbar_init(BAR(SPO_FREE + t), 4);
            mbar_init(BAR(SPL_FULL + t), 4);
            mbar_init(BAR(SPL_EMPTY + t), 4);
            mbar_init(BAR(SPCHAIN + t), 4);
        }
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(BAR(SPKV_FULL + s), 1);
            mbar_init(BAR(SPKV_EMPTY + s), 1);
        }
        mbar_init(BAR(SP_DRAIN), 1);
        mbar_init(BAR(SPFIX_ASK), 1);
        mbar_init(BAR(SPFIX_DONE), 1);
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(SEG_FULL(s), 1);
            mbar_init(SEG_EMPTY(s), KIND ? 15 : 14);  // producer, issuer, (V clearing,) 8 softmax warps, 4 epilogue warps
        }
        misc[1] = 0u;
        fence_mbar_init();
        prefetch_tmap(&tm.q);
        prefetch_tmap(&tm.k);
        prefetch_tmap(&tm.v);
    }
    if (warp == 2) {
        tmem_alloc(smem_u32(misc), C::kTmemCols);
        tmem_relinquish();
    }
    const int chunks = ((KIND ? p.N : p.n_pairs) + 31) / 32;
    long long *sums = reinterpret_cast<long long *>(sm + C::kOffKV);  // the ring is not in use yet
    SpanSched *sched = reinterpret_cast<SpanSched *>(sm + C::kOffSeg + (uint32_t)sizeof(SpanSeg) * kSegs);
    if (KIND || p.rec) {
        if (chunks > 1) {
            span_chunk_sums<KIND>(p, chunks, sums);
            __syncthreads();
        }
        if (warp == 3) {  // here, not by warp 2 in its role: with 48 registers it takes twice as long
            const SpanSched s = span_schedule<KIND>(p, chunks, sums, lane);
            if (lane == 0) *sched = s;
        }
        if (chunks > 1) fence_proxy_async_smem();  // before TMA writes there
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const int wg = warp >> 2;
    if (KIND || p.rec) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // span_merge_kernel may be set up
    // The roles walk the ring of segments alike.
    uint32_t seg_it = 0;
#define SEG (segs[seg_it % kSegs])
#define SEG_WAIT(wait) wait(SEG_FULL(seg_it % kSegs), (seg_it / kSegs) & 1u, abort_flag, kSiteSeg)
#define SEG_DONE()  /* after the warp's last look at the segment */      \
    do {                                                                \
        if (warp != 1) __syncwarp();                                    \
        if (warp == 1 || lane == 0) mbar_arrive(SEG_EMPTY(seg_it % kSegs));          \
        ++seg_it;                                                       \
    } while (0)

    if (wg == 0) {
        setmaxnreg_dec<C::kRegsOther>();
        if (warp == 2) {
            // ---------------------------------------------------------- schedule
            SpanPieces pieces{};
            SpanWalk w;
            span_walk_init<KIND>(p, *sched, w);
            for (bool more = true; more;) {
                SpanSeg g;
                more = span_next<KIND>(p, *sched, w, g);
                if (more && g.flags && g.j0 == 0) pieces = span_pieces_of<KIND>(*sched, g);  // its first piece: this CTA's last part
                if (LONG) span_cut(g, p.stretch);
                bool ok = span_warp_bwait(SEG_EMPTY(seg_it % kSegs), ((seg_it / kSegs) & 1u) ^ 1u, abort_flag, kSiteSeg);
                if (!ok) break;
                if (lane == 0) {
                    volatile SpanSeg &d = SEG;
                    d.n = g.n;
                    d.j0 = g.j0;
                    d.dual = g.dual;
                    d.flags = g.flags;
                    d.hi = g.hi;
                    d.nw = g.nw;
                    d.ns = g.ns;
                    d.s0 = g.s0;
                    d.e1 = g.e1;
                    d.seq = g.seq;
                    d.head = g.head;
                    d.q0 = g.q0;
                    d.tok0 = g.tok0;
                    d.ntok = g.ntok;
                    d.pos0 = g.pos0;
                    d.keys = g.keys;
                    d.slot = g.slot;
                    d.fix = g.fix;
                    d.lo = g.lo;
                    d.last = g.last;
                    for (int t = 0; t < 2; ++t) {
                        d.all_hi[t] = g.all_hi[t];
                        d.all_lo[t] = g.all_lo[t];
                    }
                    mbar_arrive(SEG_FULL(seg_it % kSegs));
                }
                if (LONG) __syncwarp();
                ++seg_it;
#pragma unroll 1
                while (LONG && segs[(seg_it - 1) % kSegs].flags & SPAN_MORE) {  // the segments behind it
                    ok = span_warp_bwait(SEG_EMPTY(seg_it % kSegs), ((seg_it / kSegs) & 1u) ^ 1u, abort_flag, kSiteSeg);
                    if (!ok) break;
                    if (lane == 0) {
                        span_continue(SEG, segs[(seg_it - 1) % kSegs], p.stretch);
                        mbar_arrive(SEG_FULL(seg_it % kSegs));
                    }
                    __syncwarp();
                    ++seg_it;
                }
                if (!ok) break;
            }
            if ((p.rec || (KIND && KIND != SPAN_PACKED)) && lane == 0) p.pieces[blockIdx.x] = pieces;
        } else if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            uint32_t kv_it = 0, q_it0 = 0, q_it1 = 0;
            bool ok = true;
            const int box = KIND ? min(p.page, 128) : 128;  // rows of a box
            while (ok) {
                ok = SEG_WAIT(span_warp_bwait);
                volatile SpanSeg &g = SEG;
                const int n = g.n, j0 = g.j0, head = g.head;
                if (!ok || n == 0) break;
                const bool dual = g.dual;
                // page of this lane's box of step x's tile; n_pages (outside the pool)
                // where no token of the item sees any of its keys
                const int *table = kPages ? p.table + (int64_t)g.seq * p.max_pages : nullptr;
                auto page_of = [&](int x) -> int {
                    if (!kPages || lane * box >= 128 || x >= n) return 0;
                    const int k0 = span_tile(g, j0 + x) * 128 + lane * box;
                    if (k0 > g.last || (k0 + box <= g.lo && k0 >= p.sinks)) return p.n_pages;
                    const int id = table[k0 >> p.page_log2];
                    return id < 0 || id >= p.n_pages ? p.n_pages : id;
                };
                auto load_tile = [&](const CUtensorMap *m, int x, int page) {
                    const uint32_t slot = kv_it % C::kSlots, ph = (kv_it / C::kSlots) & 1u;
                    ok = span_warp_bwait(BAR(SPKV_EMPTY + slot), ph ^ 1u, abort_flag, kSiteLoadKV);
                    if (!ok) return;
                    ++kv_it;
                    if (lane == 0) mbar_arrive_expect_tx(BAR(SPKV_FULL + slot), C::kTile);
                    __syncwarp();
                    const int tile = span_tile(g, j0 + x);
                    if (kPages) {
                        if (lane * box < 128) {
                            const int row = (tile * 128 + lane * box) & (p.page - 1);
                            const uint32_t dst = sKV + slot * C::kTile + (uint32_t)(lane * box) * 128u;
#pragma unroll
                            for (int db = 0; db < C::kNDB; ++db)
                                tma_load_4d(dst + db * C::kBlk, m, BAR(SPKV_FULL + slot), db * 64, head, row, page);
                        }
                    } else if (KIND == SPAN_PACKED) {  // rows of the next sequence, or zeros, behind this one's last
                        if (lane < C::kNDB)
                            tma_load_4d(sKV + slot * C::kTile + lane * C::kBlk, m, BAR(SPKV_FULL + slot), lane * 64, head,
                                        g.q0 + tile * 128, 0);
                    } else if (lane < C::kNDB) {
                        tma_load_4d(sKV + slot * C::kTile + lane * C::kBlk, m, BAR(SPKV_FULL + slot), lane * 64,
                                    head % p.Hl, tile * 128, head / p.Hl);
                    }
                };
                int pg0 = page_of(0), pg1 = page_of(1), pg2 = page_of(2);
                load_tile(&tm.k, 0, pg0);  // before Q, whose place is free only after the last S of the item before
                for (int i = 0; i < (dual ? 1 : 2) && ok; ++i) {
                    const int t = FEW ? (int)(seg_it & 1u) : i;  // few rows: items take the two tiles in turn
                    const uint32_t use = FEW ? seg_it >> 1 : t ? q_it1++ : q_it0++;
                    ok = span_warp_bwait(BAR(SPQ_EMPTY + t), (use & 1u) ^ 1u, abort_flag, kSiteLoadQ);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(BAR(SPQ_FULL + t), (uint32_t)C::kNDB * 128u * (uint32_t)(p.tile_tok * p.G));
                        const int tok = g.q0 + g.tok0 + i * p.tile_tok;
#pragma unroll
                        for (int db = 0; db < C::kNDB; ++db) {
                            const uint32_t dst = sQ + t * C::kQTile + db * C::kQBlk;
                            if (KIND)
                                tma_load_4d(dst, &tm.q, BAR(SPQ_FULL + t), db * 64, 0, head, tok);
                            else
                                tma_load_4d(dst, &tm.q, BAR(SPQ_FULL + t), db * 64, head % p.Hl, tok, head / p.Hl);
                        }
                    }
                }
                if (!ok) break;
                if (ok && dual && n > 1) load_tile(&tm.k, 1, pg1);
                for (int x = 0; ok && x < n; ++x) {
                    const int pg3 = page_of(x + 3);
                    load_tile(&tm.v, x, pg0);
                    const int la = dual ? 2 : 1;
                    if (ok && x + la < n) load_tile(&tm.k, x + la, dual ? pg2 : pg1);
                    pg0 = pg1;
                    pg1 = pg2;
                    pg2 = pg3;
                }
                if (ok) SEG_DONE();
            }
            if (!ok) {  // let copies already in flight land before the CTA exits
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) {
                }
            }
        } else if (KIND && warp == 3) {
            // ------------------------------------ V rows behind the last key: zeros
            uint32_t kv_it = 0, fph = 0;
            const int box = min(p.page, 128);
            while (SEG_WAIT(span_warp_bwait)) {
                const int n = SEG.n, rows = SEG.fix;
                if (n == 0) break;
                // the segment's first V tile follows its first one or two K tiles
                const uint32_t slot = (kv_it + (SEG.dual && n > 1 ? 2u : 1u)) % C::kSlots;
                kv_it += 2u * (uint32_t)n;
                if (rows >= 0) {
                    if (!span_warp_bwait(BAR(SPFIX_ASK), fph, abort_flag, kSiteFix)) break;  // the tile is in
                    fph ^= 1u;
                    for (int r = rows * 8 + lane; r < ((rows + box - 1) / box * box) * 8; r += 32)
#pragma unroll
                        for (int db = 0; db < C::kNDB; ++db)
                            st_shared_v4(sKV + slot * C::kTile + db * C::kBlk + (uint32_t)r * 16u, 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(SPFIX_DONE));
                }
                SEG_DONE();
            }
        } else if (warp == 1 && elect_one()) {  // (with lane == 0 ptxas does not know of the one thread: half as much code again)
            // -------------------------------------------------------- MMA issuer
            // few rows: M = 128 keys (or columns of V, bit 15: A MN-major), N = the rows
            constexpr uint32_t idS = idesc_bf16_f32(128, FEW ? FEW : 128, 0);
            constexpr uint32_t idO = FEW ? idesc_bf16_f32(128, FEW, 0) | 1u << 15 : idesc_bf16_f32(128, D, 1);
            const uint64_t dK = sdesc_sw128(0, 16, 1024);       // K-major, 128-byte rows
            const uint64_t dV = sdesc_sw128(0, C::kBlk, 1024);  // MN-major V, 64-column blocks kBlk apart
            auto issue_S = [&](int t, int qt, uint32_t slot) {
                const uint64_t qa = dK + (opaque(sQ + qt * C::kQTile) >> 4);
                const uint64_t ka = dK + (opaque(sKV + slot * C::kTile) >> 4);
                const uint32_t d = opaque(tmem + C::colS(t));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * C::kBlk + (kk & 3) * 32) >> 4;
                    const uint32_t q_off = ((kk >> 2) * C::kQBlk + (kk & 3) * 32) >> 4;
                    if (FEW)
                        tc_mma_ss(d, ka + off, qa + q_off, idS, kk > 0 ? 1u : 0u);
                    else
                        tc_mma_ss(d, qa + q_off, ka + off, idS, kk > 0 ? 1u : 0u);
                }
                tc_commit(BAR(SPS_FULL + t));
            };
            auto issue_PV = [&](int t, uint32_t slot, bool acc) {
                const uint64_t va = dV + (opaque(sKV + slot * C::kTile) >> 4);
                const uint32_t d = opaque(tmem + C::colO(t)), a = opaque(tmem + C::colS(t));
                const uint64_t pa = dK + (opaque(sStage + t * C::kPTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    if (FEW)
                        tc_mma_ss(d, va + (kk * 2048 >> 4), pa + (((kk >> 2) * C::kQBlk + (kk & 3) * 32) >> 4), idO,
                                  (acc || kk > 0) ? 1u : 0u);
                    else
                        tc_mma_ts(d, a + kk * 8, va + (kk * 2048 >> 4), idO, (acc || kk > 0) ? 1u : 0u);
                }
            };
            uint32_t kv_it = 0, q_it0 = 0, q_it1 = 0, pph0 = 0, pph1 = 0, fph = 0;
            bool ok = true, carried = false;  // carried: the segment's first S has been issued with the one before it
            enum : uint32_t { NEXT = 1, NEXT_S0 = 2, NEXT_LAST0 = 4, NEXT_S1 = 8, NEXT_LAST1 = 16, NEXT_Q = 32 };
            auto wait_kv = [&](uint32_t &slot) {
                slot = kv_it % C::kSlots;
                ok = ok && span_bwait(BAR(SPKV_FULL + slot), (kv_it / C::kSlots) & 1u, abort_flag, kSiteMmaKV);
                ++kv_it;
            };
            auto wait_p = [&](int t, bool first) {  // P_t is in (and, at a tile's first step, O_t is free)
                ok = span_bwait(BAR(SPP_FULL + t), t ? pph1 : pph0, abort_flag, kSiteMmaP);
                if (ok && first) ok = span_bwait(BAR(SPO_FREE + t), (seg_it & 1u) ^ 1u, abort_flag, kSiteMmaOFree);
                if (t)
                    pph1 ^= 1u;
                else
                    pph0 ^= 1u;
                tc_fence_after();
            };
            auto wait_v = [&](uint32_t &slot, bool fix) {
                wait_kv(slot);
                if (ok && fix) {
                    mbar_arrive(BAR(SPFIX_ASK));
                    ok = span_bwait(BAR(SPFIX_DONE), fph, abort_flag, kSiteFix);
                    fph ^= 1u;
                }
            };
            auto no_steps = [&](int t) {  // a tile or chain without a step in this segment
                ok = span_bwait(BAR(SPO_FREE + t), (seg_it & 1u) ^ 1u, abort_flag, kSiteMmaOFree);
                if (ok) tc_commit(BAR(SPO_FINAL + t));
            };
            while (ok) {
                ok = SEG_WAIT(span_bwait);
                volatile SpanSeg &g = SEG;
                const int n = g.n;
                if (!ok || n == 0) break;
                const bool fix = KIND && g.fix >= 0;
                uint32_t ks, vs;
                const int qb = FEW ? (int)(seg_it & 1u) : 0;  // the tile that holds Q (dual)
                if (FEW || g.dual) {
                    ok = span_bwait(BAR(SPQ_FULL + qb), (FEW ? seg_it >> 1 : q_it0++) & 1u, abort_flag, kSiteMmaQ);
                    // two chains: even steps in S_0, O_0, odd ones in S_1, O_1
#pragma unroll 1
                    for (int y = 0; y < n + 2; ++y) {  // S of step y, P V of step y - 2
                        const int t = y & 1;
                        if (y >= 2) {
                            wait_v(vs, fix && y == 2);
                            if (ok) wait_p(t, y < 4);
                            if (!ok) break;
                            issue_PV(t, vs, y >= 4);
                            tc_commit(BAR(SPKV_EMPTY + vs));
                            if (y >= n) tc_commit(BAR(SPO_FINAL + t));
                        }
                        if (y < n) {
                            wait_kv(ks);
                            if (!ok) break;
                            tc_fence_after();
                            issue_S(t, qb, ks);
                            tc_commit(BAR(SPKV_EMPTY + ks));
                            if (y + 1 == n) tc_commit(BAR(SPQ_EMPTY + qb));
                        }
                    }
                    if (ok && n == 1) no_steps(1);
                } else {
                    // steps (of the segment) of tile 0: from f0 on; of tile 1: below l1 and from m1 on
                    const int f0 = max(g.s0 - g.j0, 0), l1 = min(g.e1 - g.j0, n), m1 = max(g.nw - g.j0, 0);
                    auto on1 = [&](int x) { return x < l1 || x >= m1; };
                    const int first1 = l1 > 0 ? 0 : m1, last1 = m1 < n ? n - 1 : l1 - 1;  // last1 < 0: none
                    // Steps in the middle, which both tiles take, as they do the next, have a loop
                    // without decisions: the issuer's own instructions are on the chain of every
                    // step (S = 16384, window of 4096: 516 us, 581 without). It is entered for as few as
                    // four: items of 10 steps with 5 of them here take 63.4 us then, 64.2 from one step
                    // on, 65.0 from six; the mixed paged batch 62.3, 62.5, 63.1, and 66.0 from twelve.
                    const int mid0 = f0 + 1, mid1 = min(l1, n) - 2;  // short of the last S of either tile
                    for (int x = carried ? 0 : -1; x < n; ++x) {  // P V of step x, S of the step behind it
                        if (x == mid0 && mid1 - x >= kMidSteps) {
#pragma unroll 1
                            for (; x < mid1; ++x) {
                                vs = kv_it % C::kSlots;
                                ok = span_bwait(BAR(SPKV_FULL + vs), (kv_it / C::kSlots) & 1u, abort_flag, kSiteMmaKV) &&
                                     span_bwait(BAR(SPP_FULL + 0), pph0, abort_flag, kSiteMmaP);
                                if (!ok) break;
                                tc_fence_after();
                                issue_PV(0, vs, true);
                                ks = (kv_it + 1u) % C::kSlots;
                                ok = span_bwait(BAR(SPKV_FULL + ks), ((kv_it + 1u) / C::kSlots) & 1u, abort_flag, kSiteMmaKV);
                                if (!ok) break;
                                kv_it += 2u;
                                issue_S(0, 0, ks);
                                ok = span_bwait(BAR(SPP_FULL + 1), pph1, abort_flag, kSiteMmaP);
                                if (!ok) break;
                                pph0 ^= 1u;
                                pph1 ^= 1u;
                                tc_fence_after();
                                issue_PV(1, vs, true);
                                tc_commit(BAR(SPKV_EMPTY + vs));
                                issue_S(1, 1, ks);
                                tc_commit(BAR(SPKV_EMPTY + ks));
                            }
                            if (!ok) break;
                        }
                        // The step behind x: this segment's, or the next one's first where that is a pair too, whose
                        // scores the softmax then finds ready when it has done with this segment.
                        uint32_t next = 0;
                        if (x + 1 < n) {
                            next = NEXT | (x + 1 >= f0 ? NEXT_S0 : 0u) | (x + 2 == n ? NEXT_LAST0 : 0u) |
                                   (on1(x + 1) ? NEXT_S1 : 0u) |
                                   ((x < 0 ? last1 <= 0 : x + 1 == last1) ? NEXT_LAST1 : 0u) | (x < 0 ? NEXT_Q : 0u);
                        } else {
                            ok = span_bwait(SEG_FULL((seg_it + 1u) % kSegs), ((seg_it + 1u) / kSegs) & 1u, abort_flag, kSiteSeg);
                            if (!ok) break;
                            volatile SpanSeg &h = segs[(seg_it + 1u) % kSegs];
                            const int n2 = h.n;
                            if (n2 > 0 && !h.dual) {
                                const int j2 = h.j0, l2 = min(h.e1 - j2, n2), m2 = h.nw - j2;
                                next = NEXT | NEXT_Q | (h.s0 <= j2 ? NEXT_S0 : 0u) | (n2 == 1 ? NEXT_LAST0 : 0u) |
                                       (l2 > 0 || m2 <= 0 ? NEXT_S1 : 0u) |
                                       ((m2 < n2 ? n2 == 1 : l2 <= 1) ? NEXT_LAST1 : 0u);
                            }
                            carried = next != 0;
                        }
                        if (x >= 0) {
                            wait_v(vs, fix && x == 0);
                            if (!ok) break;
                            if (x >= f0) {
                                wait_p(0, x == f0);
                                if (!ok) break;
                                issue_PV(0, vs, x > f0);
                                if (x + 1 == n) tc_commit(BAR(SPO_FINAL + 0));
                            }
                        }
                        if (next) {
                            if (next & NEXT_Q) ok = span_bwait(BAR(SPQ_FULL + 0), q_it0++ & 1u, abort_flag, kSiteMmaQ);
                            wait_kv(ks);
                            if (!ok) break;
                            tc_fence_after();
                            if (next & NEXT_S0) issue_S(0, 0, ks);
                            if (next & NEXT_LAST0) tc_commit(BAR(SPQ_EMPTY + 0));  // after each tile's last S
                        }
                        if (x >= 0) {
                            if (on1(x)) {
                                wait_p(1, x == first1);
                                if (!ok) break;
                                issue_PV(1, vs, x > first1);
                                if (x == last1) tc_commit(BAR(SPO_FINAL + 1));
                            }
                            tc_commit(BAR(SPKV_EMPTY + vs));
                        }
                        if (next) {
                            if (next & NEXT_Q) ok = span_bwait(BAR(SPQ_FULL + 1), q_it1++ & 1u, abort_flag, kSiteMmaQ);
                            if (!ok) break;
                            if (next & NEXT_S1) issue_S(1, 1, ks);
                            if (next & NEXT_LAST1) tc_commit(BAR(SPQ_EMPTY + 1));
                            tc_commit(BAR(SPKV_EMPTY + ks));
                        }
                    }
                    if (ok && f0 >= n) no_steps(0);
                    if (ok && l1 <= 0 && m1 >= n) no_steps(1);
                }
                if (ok) SEG_DONE();
            }
            if (!ok) {  // wait (bounded) for MMAs in flight before tensor memory is released
                tc_commit(BAR(SP_DRAIN));
                uint32_t dummy = 0;
                const unsigned long long t0 = globaltimer_ns();
                while (!mbar_try_wait(BAR(SP_DRAIN), 0) && globaltimer_ns() - t0 < 200000000ull) ++dummy;
            }
        }
        __syncwarp();
    } else if (wg == 1 || wg == 2) {
        // ------------------------------------------------------------- softmax
        setmaxnreg_inc<C::kRegsSoftmax>();
        const int t = wg - 1;
        if constexpr (FEW > 0) {
            // One thread per key of the tile, its scores of all rows in registers. The rows'
            // maxima m (shared memory, common to the chain's 128 threads) follow the same
            // rules as below; when some weight passes kSpanRise all four warps take the
            // maxima anew. Sums are kept per thread and added up at the segment's end.
            const int kl = (warp & 3) * 32 + lane;
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lane_base + C::colS(t), tO = tmem + lane_base + C::colO(t);
            // P goes to [64-key block][row][key], 128-byte rows, 16-byte chunks swizzled by row
            const uint32_t p_at = sStage + t * C::kPTile + (uint32_t)(kl >> 6) * (FEW * 128u) + (uint32_t)(kl & 7) * 2u;
            const uint32_t chunk = (uint32_t)(kl & 63) >> 3;
            float *red = reinterpret_cast<float *>(sm + C::kOffRed) + t * 8 * FEW;  // [4][FEW], then m, its use, alpha
            float *m_s = red + 4 * FEW, *me_s = red + 5 * FEW, *al_s = red + 6 * FEW;
            volatile uint32_t *flags = misc + 2 + t;
            const float sl2 = p.scale_log2;
            uint32_t sph = 0;
            bool ok = true;
            volatile uint32_t *rise = reinterpret_cast<volatile uint32_t *>(red + 7 * FEW);  // by turns: the step that passed
            uint32_t cph = 0, stamp = 0;
            if (kl < 2) rise[kl] = 0u;
            auto sync = [&]() {  // the chain's four warps meet (bounded, unlike a named barrier)
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(SPCHAIN + t));
                ok = ok && span_warp_bwait(BAR(SPCHAIN + t), cph, abort_flag, kSiteSoftS);
                cph ^= 1u;
            };
            // v of all rows: the warps' results of `op` over their lanes to red, then a barrier.
            // Each exchange halves the rows a lane holds; it ends with one row, lane / (32 / FEW).
            auto over_keys = [&](float (&v)[FEW], auto op) {
#pragma unroll
                for (int n = FEW / 2, d = 16; n; n >>= 1, d >>= 1) {
                    const bool up = lane & d;
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
                        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, d));
                    }
                }
                if (FEW == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
                red[(warp & 3) * FEW + (FEW == 16 ? lane >> 1 : lane)] = v[0];
                sync();
            };
            while (ok) {
                ok = SEG_WAIT(span_warp_bwait);
                volatile SpanSeg &g = SEG;
                if (!ok || g.n == 0) break;
                const int rows = g.ntok * p.G;
                if (kl < FEW) m_s[kl] = -INFINITY;
                float l[FEW];
#pragma unroll
                for (int r = 0; r < FEW; ++r) l[r] = 0.f;
                bool fresh = true;  // some row has not seen a key
                int steps = (g.n + 1 - t) >> 1, c, c_end = g.hi - g.nw + 1;
                {
                    const int y = g.j0 + t, nw = g.nw;
                    c = y < nw ? g.hi - y : g.ns - 1 - (y - nw);
                    if (y >= nw) c_end = INT_MIN;
                }
#pragma unroll 1
                for (; steps > 0; --steps) {
                    const int c0 = c * 128;
                    const bool masked = c0 > g.all_hi[0] || (c0 < g.all_lo[0] && c0 + 128 > p.sinks);
                    c -= 2;
                    if (c < c_end) {
                        c += g.ns - c_end;
                        c_end = INT_MIN;
                    }
                    uint32_t by_row = ~0u;  // a tree's rows that see this thread's key; fetched before the scores are in
                    if (kIsTree<KIND> && masked) by_row = span_tree_rows<FEW>(p, g, c0 + kl);
                    ok = span_warp_bwait(BAR(SPS_FULL + t), sph, abort_flag, kSiteSoftS);
                    if (!ok) break;
                    sph ^= 1u;
                    tc_fence_after();
                    uint32_t s[FEW];
                    float e[FEW];
                    if constexpr (FEW == 16)
                        tmem_ld16(tS, s);
                    else
                        tmem_ld32(tS, s);
                    if (kIsTree<KIND> && masked) {
#pragma unroll
                        for (int r = 0; r < FEW; ++r) s[r] = (by_row >> r) & 1u ? s[r] : f2u(-INFINITY);
                    } else if (masked) {
                        // the key is seen by tokens key - right .. key + left (a sink: by all from there
                        // on), so by rows r0 <= r < r1 of the item
                        const int key = c0 + kl, at = key - g.pos0;
                        const int r0 = min(max(at - p.right, 0), FEW) * p.G;
                        const int r1 = key >= g.keys ? 0 : key < p.sinks ? FEW : min(max(at + p.left + 1, 0), FEW) * p.G;
#pragma unroll
                        for (int r = 0; r < FEW; ++r) s[r] = r >= r0 && r < r1 ? s[r] : f2u(-INFINITY);
                    }
                    bool by_max = fresh;
#pragma unroll 1
                    for (;;) {
                        if (by_max) {
                            float v[FEW];
#pragma unroll
                            for (int r = 0; r < FEW; ++r) v[r] = u2f(s[r]);
                            over_keys(v, [](float a, float b) { return fmaxf(a, b); });
                            if (!ok) break;
                            if ((warp & 3) == 0) {
                                bool unseen = false, up = false;
                                if (lane < FEW) {
                                    const float mx = fmaxf(fmaxf(red[lane], red[FEW + lane]),
                                                           fmaxf(red[2 * FEW + lane], red[3 * FEW + lane])) * sl2;
                                    const float old = m_s[lane];
                                    const float now = old == -INFINITY || mx > old + 4.0f ? mx : old;
                                    up = old != -INFINITY && now != old && lane < rows;
                                    unseen = now == -INFINITY && lane < rows;
                                    m_s[lane] = now;
                                    me_s[lane] = now == -INFINITY ? 0.f : now;
                                    al_s[lane] = up ? ex2_approx(old - now) : 1.f;
                                }
                                const uint32_t f = (__any_sync(0xffffffffu, unseen) ? 1u : 0u) |
                                                   (__any_sync(0xffffffffu, up) ? 2u : 0u);
                                if (lane == 0) *flags = f;
                            }
                            sync();
                            if (!ok) break;
                            const uint32_t f = *flags;
                            fresh = f & 1u;
                            if (f & 2u) {
                                // O^T is stable: the commit that signalled S_t covers the P V before
                                uint32_t o[FEW];
                                if constexpr (FEW == 16)
                                    tmem_ld16(tO, o);
                                else
                                    tmem_ld32(tO, o);
#pragma unroll
                                for (int r = 0; r < FEW; ++r) {
                                    l[r] *= al_s[r];
                                    o[r] = f2u(u2f(o[r]) * al_s[r]);
                                }
                                if constexpr (FEW == 16)
                                    tmem_st16(tO, o);
                                else
                                    tmem_st32(tO, o);
                                tmem_st_wait();
                            }
                        }
                        float top = 0.f;
#pragma unroll
                        for (int r = 0; r < FEW; ++r) {
                            e[r] = ex2_approx(fmaf(u2f(s[r]), sl2, -me_s[r]));
                            if (r < rows) top = fmaxf(top, e[r]);
                        }
                        if (by_max) break;
                        if (__any_sync(0xffffffffu, top > kSpanRise) && lane == 0) rise[stamp & 1u] = stamp + 1u;
                        sync();
                        if (!ok) break;
                        by_max = rise[stamp & 1u] == stamp + 1u;
                        ++stamp;
                        if (!by_max) break;
                    }
                    if (!ok) break;
#pragma unroll
                    for (int r = 0; r < FEW; r += 2) {
                        l[r] += e[r];
                        l[r + 1] += e[r + 1];
                        const uint32_t two = pack_bf16x2(e[r], e[r + 1]);
                        st_shared_u16(p_at + r * 128u + ((chunk ^ (r & 7)) << 4), two & 0xffffu);
                        st_shared_u16(p_at + (r + 1) * 128u + ((chunk ^ ((r + 1) & 7)) << 4), two >> 16);
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(SPP_FULL + t));
                }
                if (!ok) break;
                over_keys(l, [](float a, float b) { return a + b; });
                if (!ok) break;
                ok = span_warp_bwait(BAR(SPL_EMPTY + t), (seg_it & 1u) ^ 1u, abort_flag, kSiteSoftL);
                if (!ok) break;
                if (kl < FEW) {
                    row_ml[t * 256 + kl] = red[kl] + red[FEW + kl] + red[2 * FEW + kl] + red[3 * FEW + kl];
                    row_ml[t * 256 + 128 + kl] = m_s[kl];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(SPL_FULL + t));
                SEG_DONE();
                sync();  // red and m are free for the next segment
            }
        } else {
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lane_base + C::colS(t);
            const uint32_t tO = tmem + lane_base + C::colO(t);
            const int row = (warp & 3) * 32 + lane;
            const float sl2 = p.scale_log2;
            uint32_t sph = 0;
            bool ok = true;
            while (ok) {
                ok = SEG_WAIT(span_warp_bwait);
                volatile SpanSeg &g = SEG;
                if (!ok || g.n == 0) break;
                // lim: the row sum that calls for the row max again: none for a row that does
                // not exist, any for one that has not seen a key yet
                float m = -INFINITY, l = 0.f, lim;
                bool idle;
                {
                    const int rows = min(g.ntok - (g.dual ? 0 : t * p.tile_tok), p.tile_tok) * p.G;
                    lim = row < rows ? -1.f : INFINITY;
                    idle = (warp & 3) * 32 >= rows;  // no row of this warp exists
                }
                // This tile's (chain's) steps and K/V tiles: c, c - step, ... down to c_end, then
                // the sinks' from ns - 1 on.
                int steps, c, c_end = g.hi - g.nw + 1;
                {
                    const int n = g.n, j0 = g.j0, nw = g.nw;
                    int y = j0;  // the first step's
                    if (g.dual) {
                        steps = (n + 1 - t) >> 1;
                        y += t;
                    } else if (t == 0) {
                        y = max(j0, g.s0);
                        steps = j0 + n - y;
                    } else {
                        const int e1 = g.e1;
                        steps = max(0, min(e1, j0 + n) - j0) + max(0, j0 + n - max(nw, j0));
                        if (y >= e1) y = max(y, nw);
                        c_end = g.hi - e1 + 1;
                    }
                    c = y < nw ? g.hi - y : g.ns - 1 - (y - nw);
                    if (y >= nw) c_end = INT_MIN;
                }
                // Rows whose keys end in an earlier tile than the first see none in it, so the
                // maxima are taken over the first two steps (mixed paged batch 80.6 us; over the first one
                // 88.5; over three 80.6, and S = 1000 14.3 us instead of 14.2).
                const int settled = steps - 2;
#pragma unroll 1
                for (; steps > 0; --steps) {
                    const int c0 = c * 128;
                    const bool masked = c0 > g.all_hi[t] || (c0 < g.all_lo[t] && c0 + 128 > p.sinks);
                    c -= 1 + g.dual;
                    if (c < c_end) {
                        c += g.ns - c_end;
                        c_end = INT_MIN;
                    }
                    uint32_t bits_at[5] = {};  // a tree's words of this row for the tile; fetched before the scores are in
                    if (kIsTree<KIND> && masked && !idle) {
                        const int tok = min((g.dual ? 0 : t * p.tile_tok) + span_row_tok<KIND>(p, row), g.ntok - 1);
                        const int *m_row = p.mask + ((int64_t)g.q0 + g.tok0 + tok) * p.words;
                        const int w0 = (c0 - (g.pos0 - g.tok0)) >> 5;  // (rounded down)
#pragma unroll
                        for (int i = 0; i < 5; ++i) bits_at[i] = span_tree_word(m_row, p.words, w0 + i);
                    }
                    ok = span_warp_bwait(BAR(SPS_FULL + t), sph, abort_flag, kSiteSoftS);
                    if (!ok) break;
                    sph ^= 1u;
                    if (idle) {  // P keeps what S left there: only rows that do not exist read it
                        if (lane == 0) mbar_arrive(BAR(SPP_FULL + t));
                        continue;
                    }
                    tc_fence_after();
                    uint32_t sa[64], sb[64];  // this thread's row of S: columns 0-63, 64-127
#define SV(i) u2f((i) < 64 ? sa[(i) & 63] : sb[(i) & 63])
                    uint32_t pk[64];
                    float lstep = 0.f;
                    if (masked) {
                        // Masked scores become -inf in tensor memory, 32 columns at a time: a few
                        // instructions in a loop, where masking them in the registers below is 500
                        // that have to be fetched anew for the one or two tiles of an item with an
                        // edge in them.
                        // Places of this row's token and of the last key it may see:
                        const int pos = g.pos0 + (g.dual ? 0 : t * p.tile_tok) + span_row_tok<KIND>(p, row);
                        const int row_hi = min(pos + p.right, g.keys - 1);
#pragma unroll 1
                        for (int h = 0; h < 128; h += 32) {
                            uint32_t bits;
                            if (kIsTree<KIND>) {
                                bits = __funnelshift_r(bits_at[0], bits_at[1], c0 - (g.pos0 - g.tok0)) &
                                       span_mask_word(INT_MIN / 2, g.keys - 1 - c0, 0, h);
#pragma unroll
                                for (int i = 0; i < 4; ++i) bits_at[i] = bits_at[i + 1];
                            } else {
                                bits = span_mask_word(pos - p.left - c0, row_hi - c0, p.sinks - c0, h);
                            }
                            if (__all_sync(0xffffffffu, bits == ~0u)) continue;
                            if (__any_sync(0xffffffffu, bits)) {
                                uint32_t s[32];
                                tmem_ld32(tS + h, s);
#pragma unroll
                                for (int i = 0; i < 32; ++i) s[i] = (bits >> i) & 1u ? s[i] : f2u(-INFINITY);
                                tmem_st32(tS + h, s);
                            } else {
                                tmem_fill32(tS + h, f2u(-INFINITY));
                            }
                        }
                        tmem_st_wait();
                    }
                    auto row_max = [&]() {
                        float mx0 = fmaxf(u2f(sa[0]), u2f(sa[1])), mx1 = fmaxf(u2f(sa[2]), u2f(sa[3]));
                        float mx2 = fmaxf(u2f(sa[4]), u2f(sa[5])), mx3 = fmaxf(u2f(sa[6]), u2f(sa[7]));
#pragma unroll
                        for (int i = 8; i < 64; i += 8) {
                            mx0 = fmax3(mx0, u2f(sa[i + 0]), u2f(sa[i + 1]));
                            mx1 = fmax3(mx1, u2f(sa[i + 2]), u2f(sa[i + 3]));
                            mx2 = fmax3(mx2, u2f(sa[i + 4]), u2f(sa[i + 5]));
                            mx3 = fmax3(mx3, u2f(sa[i + 6]), u2f(sa[i + 7]));
                        }
#pragma unroll
                        for (int i = 0; i < 64; i += 8) {
                            mx0 = fmax3(mx0, u2f(sb[i + 0]), u2f(sb[i + 1]));
                            mx1 = fmax3(mx1, u2f(sb[i + 2]), u2f(sb[i + 3]));
                            mx2 = fmax3(mx2, u2f(sb[i + 4]), u2f(sb[i + 5]));
                            mx3 = fmax3(mx3, u2f(sb[i + 6]), u2f(sb[i + 7]));
                        }
                        return fmax3(mx0, mx1, fmaxf(mx2, mx3)) * sl2;
                    };
                    // p = exp2(s * scale*log2e - m); a row that has seen no key yet takes m = 0,
                    // its scores being -inf
                    auto exps = [&]() {
                        const float me = m == -INFINITY ? 0.f : m;
                        const uint64_t sc2 = f2pack(sl2, sl2), nm2 = f2pack(-me, -me);
                        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
                        for (int i = 0; i < 64; i += 2) {
                            const int e = 2 * i;
                            float e0, e1, e2, e3;
                            f2unpack(ffma2(f2pack(SV(e), SV(e + 1)), sc2, nm2), e0, e1);
                            f2unpack(ffma2(f2pack(SV(e + 2), SV(e + 3)), sc2, nm2), e2, e3);
                            e0 = ex2_approx(e0);
                            e1 = ex2_approx(e1);
                            e2 = ex2_approx(e2);
                            e3 = ex2_approx(e3);
                            acc0 = fadd2(acc0, f2pack(e0, e1));
                            acc1 = fadd2(acc1, f2pack(e2, e3));
                            pk[i] = pack_bf16x2(e0, e1);
                            pk[i + 1] = pack_bf16x2(e2, e3);
                        }
                        float a0, a1;
                        f2unpack(fadd2(acc0, acc1), a0, a1);
                        lstep = a0 + a1;
                    };
                    tmem_ld64x2(tS, sa, sb);
                    if (steps > settled) {
                        const float mx = row_max();
                        if (lim < 0.f && mx > -INFINITY) {
                            m = mx;
                            lim = kSpanRise;
                        }
                    }
                    exps();
                    // A row keeps its max while no row sum passes kSpanRise: p, l and O are floating
                    // point, so a maximum that lags by up to 2^14 costs no precision, and a first
                    // tile with only a few keys in it (a causal diagonal) seldom has to be put
                    // right. A row that sees its first key later yet (a piece that begins behind
                    // its window) gets its max here too. Until then its weights, sum and O are 0.
                    // Two-sided window S = 4096: 83.1 us with a limit of 2^4, 67.7 with 2^8, 63.3 to 63.4 with
                    // 2^12, 2^14, 2^16 and 2^24; S = 16384, window of 4096: 701, 512, and 510 to 518. Higher
                    // ones gain nothing and bring O closer to fp32's end.
                    if (steps < settled + 2 && __any_sync(0xffffffffu, lstep > lim)) {  // (at the first step m is exact)
                        tmem_ld64x2(tS, sa, sb);
                        const float mnew = row_max();
                        float alpha = 1.f;
                        if (mnew > m) {
                            alpha = ex2_approx(m - mnew);
                            m = mnew;
                            if (lim < 0.f) lim = kSpanRise;
                        }
                        if (__any_sync(0xffffffffu, alpha != 1.f)) {
                            // The commit that signalled S_t for this step also covers the
                            // previous O_t += P V, so O_t is stable here.
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(tO + c, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = f2u(u2f(o[i]) * alpha);
                                tmem_st32(tO + c, o);
                            }
                            l *= alpha;
                        }
                        exps();
                    }
                    l += lstep;
                    {
                        uint32_t h0[32], h1[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            h0[i] = pk[i];
                            h1[i] = pk[32 + i];
                        }
                        tmem_st32(tS, h0);
                        tmem_st32(tS + 32, h1);
                    }
#undef SV
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(SPP_FULL + t));
                }
                if (!ok) break;
                ok = span_warp_bwait(BAR(SPL_EMPTY + t), (seg_it & 1u) ^ 1u, abort_flag, kSiteSoftL);
                if (!ok) break;
                row_ml[t * 256 + row] = l;
                row_ml[t * 256 + 128 + row] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(SPL_FULL + t));
                SEG_DONE();
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        setmaxnreg_dec<C::kRegsEpilogue>();
        const int wq = warp & 3;
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const int row = wq * 32 + lane;
        const uint32_t stage = sStage + wq * C::kStageWarp;
        bool ok = true;
        while (ok) {
            ok = SEG_WAIT(span_warp_bwait);
            volatile SpanSeg &g = SEG;
            if (!ok || g.n == 0) break;
            // a segment among several of a part goes to the CTA's third record, and from there to its part's
            auto several = [&]() -> bool { return LONG && g.flags & (SPAN_ADD | SPAN_MORE); };
            const bool piece = g.flags;
            float *rec = p.rec + (size_t)(several() ? 2 * gridDim.x + blockIdx.x : g.slot) * R::kFloats;
            auto row_dst = [&](int t, int rows) -> int64_t {
                if (row >= rows) return -1;
                const int r = span_row_tok<KIND>(p, row);
                return span_out_offset<D, KIND>(p, g.head, g.q0, g.tok0 + t * p.tile_tok + r, KIND ? row - r * p.G : 0);
            };
            auto release_o = [&](int t) {  // O_t fully read: the next item may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(SPO_FREE + t));
            };
            // one tile's 32 columns from c0 on (f: its factors) to the output or the record
            auto emit = [&](int t, int c0, const float (&f)[32], int64_t dst, bool any_row) {
                if (!any_row) return;
                if (piece) {
                    if (dst < 0) return;
                    float4 *o4 = reinterpret_cast<float4 *>(rec) + (size_t)t * (D / 4) * 128;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        o4[(size_t)(c0 / 4 + q) * 128 + row] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
                    return;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    stage_chunk(stage, lane, (c0 % 64) / 8 + c, pack_bf16x2(f[8 * c + 0], f[8 * c + 1]),
                                pack_bf16x2(f[8 * c + 2], f[8 * c + 3]), pack_bf16x2(f[8 * c + 4], f[8 * c + 5]),
                                pack_bf16x2(f[8 * c + 6], f[8 * c + 7]));
                if ((c0 + 32) % 64 == 0)
                    flush_block<true>(p.out, stage, lane, dst, c0 / 64);
                else if (c0 + 32 == D)  // the half block of D = 96
                    flush_block<true, 4>(p.out, stage, lane, dst, c0 / 64);
            };
            auto take_ml = [&](int t, float &l, float &m) {
                ok = span_warp_bwait(BAR(SPO_FINAL + t), seg_it & 1u, abort_flag, kSiteEpiO) &&
                     span_warp_bwait(BAR(SPL_FULL + t), seg_it & 1u, abort_flag, kSiteEpiL);
                if (!ok) return;
                l = row_ml[t * 256 + row];
                m = row_ml[t * 256 + 128 + row];
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(SPL_EMPTY + t));
                tc_fence_after();
            };
            auto put_ml = [&](int t, float m, float l) {
                rec[R::kML + t * 256 + row] = m;
                rec[R::kML + t * 256 + 128 + row] = l;
            };
            // m and l of a row's segment with what its part's record holds (written by this thread): their
            // common maximum and sum, and the factors of either O
            auto join = [&](float m_part, float l_part, float &m, float &l, float &a, float &a_part) {
                const float top = fmaxf(m, m_part);
                a = m == -INFINITY ? 0.f : ex2_approx(m - top);
                a_part = m_part == -INFINITY ? 0.f : ex2_approx(m_part - top);
                l = a * l + a_part * l_part;
                m = top;
            };
            if constexpr (FEW > 0) {
                // one thread per column of the output, all rows
                ok = span_warp_bwait(BAR(SPO_FINAL + 0), seg_it & 1u, abort_flag, kSiteEpiO) &&
                     span_warp_bwait(BAR(SPO_FINAL + 1), seg_it & 1u, abort_flag, kSiteEpiO) &&
                     span_warp_bwait(BAR(SPL_FULL + 0), seg_it & 1u, abort_flag, kSiteEpiL) &&
                     span_warp_bwait(BAR(SPL_FULL + 1), seg_it & 1u, abort_flag, kSiteEpiL);
                if (!ok) break;
                tc_fence_after();
                const int rows = g.ntok * p.G, head = g.head, tok0 = g.tok0, q_row = g.q0;
                uint32_t o0[FEW], o1[FEW];
                if constexpr (FEW == 16) {
                    tmem_ld16(tmem + lane_base + C::colO(0), o0);
                    tmem_ld16(tmem + lane_base + C::colO(1), o1);
                } else {
                    tmem_ld32(tmem + lane_base + C::colO(0), o0);
                    tmem_ld32(tmem + lane_base + C::colO(1), o1);
                }
                release_o(0);
                release_o(1);
#pragma unroll
                for (int r = 0; r < FEW; ++r) {
                    if (r >= rows) break;
                    const float l0 = row_ml[r], m0 = row_ml[128 + r], l1 = row_ml[256 + r], m1 = row_ml[384 + r];
                    const float m = fmaxf(m0, m1);
                    const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - m), a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
                    const float l = a0 * l0 + a1 * l1;
                    float f = a0 > 0.f ? u2f(o0[r]) * a0 : 0.f;
                    f = a1 > 0.f ? fmaf(u2f(o1[r]), a1, f) : f;
                    if (row >= D) continue;
                    if (piece) {
                        rec[r * D + row] = f;
                        if (row == 0) {
                            rec[R::kML + r] = m;
                            rec[R::kML + 128 + r] = l;
                        }
                    } else {
                        const int tk = span_row_tok<KIND>(p, r);
                        p.out[span_out_offset<D, KIND>(p, head, q_row, tok0 + tk, r - tk * p.G) + row] =
                            (uint16_t)pack_bf16x2(l > 0.f ? f * (1.0f / l) : 0.f, 0.f);
                    }
                }
                if (several() && row < D) {
                    const int flags = g.flags;
                    // as below for tiles; each thread keeps maxima and sums of its own, behind O in the third record
                    float *part = p.rec + (size_t)g.slot * R::kFloats, *own = rec + FEW * D + row;
                    static_assert(FEW * D + 256 * FEW <= R::kML, "their place in the record");
#pragma unroll 1
                    for (int r = 0; r < rows; ++r, own += 256) {
                        const float l0 = row_ml[r], m0 = row_ml[128 + r], l1 = row_ml[256 + r], m1 = row_ml[384 + r];
                        float m = fmaxf(m0, m1), a = 1.f, a_part = 0.f;
                        float l = (m0 == -INFINITY ? 0.f : ex2_approx(m0 - m) * l0) + (m1 == -INFINITY ? 0.f : ex2_approx(m1 - m) * l1);
                        if (flags & SPAN_ADD) join(own[0], own[128], m, l, a, a_part);
                        float f = rec[r * D + row] * a;  // zero where no key has been seen
                        if (a_part > 0.f) f = fmaf(part[r * D + row], a_part, f);
                        own[0] = m;
                        own[128] = l;
                        if (flags & (SPAN_PIECE | SPAN_MORE)) {
                            part[r * D + row] = f;
                            if (row == 0) {
                                part[R::kML + r] = m;
                                part[R::kML + 128 + r] = l;
                            }
                        } else {
                            const int tk = span_row_tok<KIND>(p, r);
                            p.out[span_out_offset<D, KIND>(p, head, q_row, tok0 + tk, r - tk * p.G) + row] =
                                (uint16_t)pack_bf16x2(l > 0.f ? f * (1.0f / l) : 0.f, 0.f);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(BAR(SPL_EMPTY + 0));
                    mbar_arrive(BAR(SPL_EMPTY + 1));
                }
            } else if (g.dual) {
                float l0 = 0.f, m0 = 0.f, l1 = 0.f, m1 = 0.f;
                take_ml(0, l0, m0);
                if (ok) take_ml(1, l1, m1);
                if (!ok) break;
                const int rows = g.ntok * p.G;
                const int64_t dst = row_dst(0, rows);
                const bool any_row = wq * 32 < rows, two = g.n > 1;
                const float m = fmaxf(m0, m1);
                float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - m);
                float a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
                const float l = a0 * l0 + a1 * l1;
                if (!piece) {
                    const float inv = l > 0.f ? 1.0f / l : 0.f;
                    a0 *= inv;
                    a1 *= inv;
                } else if (dst >= 0) {
                    put_ml(0, m, l);
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    if (!any_row) continue;
                    uint32_t o[32];
                    float f[32];
                    tmem_ld32(tmem + lane_base + C::colO(0) + c0, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = a0 > 0.f ? u2f(o[i]) * a0 : 0.f;
                    if (two) {
                        tmem_ld32(tmem + lane_base + C::colO(1) + c0, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = a1 > 0.f ? fmaf(u2f(o[i]), a1, f[i]) : f[i];
                    }
                    emit(0, c0, f, dst, true);
                }
                release_o(0);
                release_o(1);
            } else {
                for (int t = 0; t < 2; ++t) {
                    float l = 0.f, m = 0.f;
                    take_ml(t, l, m);
                    if (!ok) break;
                    const int rows = min(g.ntok - t * p.tile_tok, p.tile_tok) * p.G;
                    const int64_t dst = row_dst(t, rows);
                    const bool any_row = wq * 32 < rows;
                    float inv = 1.f;
                    if (!piece)
                        inv = l > 0.f ? 1.0f / l : 0.f;
                    else if (dst >= 0)
                        put_ml(t, m, l);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        float f[32];
                        tmem_ld32(tmem + lane_base + C::colO(t) + c0, o);
                        if (c0 + 32 == D) release_o(t);
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = u2f(o[i]) * inv;
                        emit(t, c0, f, dst, any_row);
                    }
                }
            }
            if constexpr (LONG && FEW == 0) {
                if (ok && several()) {
                    // the rows' segment from the third record to their part's record or, the part being all
                    // of the item and this its last segment, to the output
#pragma unroll 1
                    for (int t = 0; t < (g.dual ? 1 : 2); ++t) {
                        const int64_t dst = row_dst(t, min(g.ntok - t * p.tile_tok, p.tile_tok) * p.G);
                        if (dst < 0) continue;
                        float *part = p.rec + (size_t)g.slot * R::kFloats;
                        const size_t ml = R::kML + t * 256 + row, at = (size_t)t * (D / 4) * 128 + row;
                        const int flags = g.flags;
                        float m = rec[ml], l = rec[ml + 128], a = 1.f, a_part = 0.f;
                        if (flags & SPAN_ADD) join(part[ml], part[ml + 128], m, l, a, a_part);
                        const bool out = !(flags & (SPAN_PIECE | SPAN_MORE));
                        const float inv = !out ? 1.f : l > 0.f ? 1.0f / l : 0.f;
                        part[ml] = m;
                        part[ml + 128] = l;
#pragma unroll 1
                        for (int c = 0; c < D / 4; ++c) {
                            const float4 x = reinterpret_cast<const float4 *>(rec)[at + c * 128];
                            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (a > 0.f) f = make_float4(x.x * a, x.y * a, x.z * a, x.w * a);  // (else there is no O)
                            float4 *o4 = reinterpret_cast<float4 *>(part) + at + c * 128;
                            if (a_part > 0.f) {
                                const float4 y = *o4;
                                f = make_float4(fmaf(y.x, a_part, f.x), fmaf(y.y, a_part, f.y), fmaf(y.z, a_part, f.z), fmaf(y.w, a_part, f.w));
                            }
                            if (!out)
                                *o4 = f;
                            else
                                *reinterpret_cast<uint2 *>(p.out + dst + 4 * c) =
                                    make_uint2(pack_bf16x2(f.x * inv, f.y * inv), pack_bf16x2(f.z * inv, f.w * inv));
                        }
                    }
                    __syncwarp();
                }
            }
            if (ok) SEG_DONE();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && misc[1]) atomicOr(&g_xs_error, misc[1]);  // a wait ran out
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
#undef BAR
#undef SEG_FULL
#undef SEG_EMPTY
#undef SEG
#undef SEG_WAIT
#undef SEG_DONE
}

// Adds up the pieces of the item whose first piece is CTA blockIdx.x's last
// segment: piece 0 in the record named by the CTA, piece i > 0 in the first
// record of CTA blockIdx.x + i (trees: + i * lanes), in that order. The pieces' loads go out several at
// a time (U), their latency being most of what this costs.
// Records hold neighbouring rows of 4 columns side by side, so a warp reads 32 rows
// of kPer such groups, block y 32 rows; the output rows are put together in shared
// memory and stored whole: 10 us for 152 items of 256 rows in two pieces, D = 128,
// against 17 with 8 bytes of a row at a time. With few rows the records hold whole
// rows, and a thread takes 4 columns of one.
template <int D, int KIND, int FEW>
__global__ void __launch_bounds__(256) span_merge_kernel(const __grid_constant__ SpanParams p) {
    using R = Rec<D>;
    constexpr int kPer = FEW ? 1 : D / 32, U = FEW ? 8 : 2;
    __shared__ uint2 rows_s[FEW ? 1 : 32][FEW ? 1 : D / 4 + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched early: the attention kernel is done from here on
    const SpanPieces s = p.pieces[blockIdx.x];
    if (s.pieces < 2) return;
    const int step = KIND == SPAN_TREE_LANES ? s.lanes : 1;  // CTAs from one piece to the next
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = FEW ? 0 : (int)blockIdx.y >> 2, row0 = FEW ? 0 : ((int)blockIdx.y & 3) * 32;  // this block's rows
    const int rows = min(s.ntok - t * p.tile_tok, p.tile_tok) * p.G - row0;
    const int i = (int)blockIdx.y * 256 + (int)threadIdx.x;
    const int r = FEW ? i / (D / 4) : lane, c4 = FEW ? i % (D / 4) : warp;  // and groups warp + 8, warp + 16, ...
    if (rows <= 0) return;
    const bool mine = r < rows;
    const size_t o_at = FEW ? (size_t)r * (D / 4) + c4 : ((size_t)t * (D / 4) + c4) * 128 + row0 + r;
    const size_t ml_at = R::kML + t * 256 + row0 + r;
    float M = -INFINITY, L = 0.f;
    float4 acc[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; mine && k0 < s.pieces; k0 += U) {
        float m[U], l[U];
        float4 o[U][kPer];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] = -INFINITY;
            if (k0 + u >= s.pieces) continue;
            const float *rec = p.rec + (size_t)(k0 + u == 0 ? s.slot : 2 * ((int)blockIdx.x + (k0 + u) * step)) * R::kFloats;
            m[u] = rec[ml_at];
            l[u] = rec[ml_at + 128];
#pragma unroll
            for (int j = 0; j < kPer; ++j) o[u][j] = reinterpret_cast<const float4 *>(rec)[o_at + (size_t)j * 8 * 128];
        }
        float top = M;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
        if (top == -INFINITY) continue;  // no key seen yet
        const float a = ex2_approx(M - top);
        M = top;
        L *= a;
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[j] = make_float4(acc[j].x * a, acc[j].y * a, acc[j].z * a, acc[j].w * a);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (m[u] == -INFINITY) continue;  // such a piece's O is not looked at
            const float b = ex2_approx(m[u] - top);
            L = fmaf(b, l[u], L);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                acc[j] = make_float4(fmaf(b, o[u][j].x, acc[j].x), fmaf(b, o[u][j].y, acc[j].y), fmaf(b, o[u][j].z, acc[j].z),
                                     fmaf(b, o[u][j].w, acc[j].w));
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    auto row_at = [&](int row) -> uint16_t * {
        const int tk = span_row_tok<KIND>(p, row);
        return p.out + span_out_offset<D, KIND>(p, s.head, s.q0, s.tok0 + t * p.tile_tok + tk, KIND ? row - tk * p.G : 0);
    };
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint2 x = make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
        if constexpr (FEW > 0) {
            if (mine) *reinterpret_cast<uint2 *>(row_at(r) + c4 * 4) = x;
        } else {
            rows_s[r][c4 + 8 * j] = x;
        }
    }
    if constexpr (FEW == 0) {
        __syncthreads();
        for (int q = warp; q < min(rows, 32); q += 8) {
            uint16_t *dst = row_at(row0 + q);
            if (lane < D / 4) *reinterpret_cast<uint2 *>(dst + lane * 4) = rows_s[q][lane];
        }
    }
}

template <int D, int KIND, int FEW, bool LONG>
static cudaError_t launch_span_one(const SpanMaps &maps, const SpanParams &p, int grid, cudaStream_t stream) {
    auto kern = span_attn_kernel<D, KIND, FEW, LONG>;
    static std::atomic<uint64_t> configured{0};  // devices where the shared-memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SpanCfg<D, KIND, FEW>::kSmemAlloc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    kern<<<grid, 512, SpanCfg<D, KIND, FEW>::kSmemAlloc, stream>>>(maps, p);
    e = cudaGetLastError();
    if (e == cudaErrorInvalidValue || e == cudaErrorLaunchOutOfResources) {
        // the limit was lost (for instance by a device reset): set it again once
        configured.fetch_and(~bit, std::memory_order_acq_rel);
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SpanCfg<D, KIND, FEW>::kSmemAlloc);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
        kern<<<grid, 512, SpanCfg<D, KIND, FEW>::kSmemAlloc, stream>>>(maps, p);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    if (p.rec) {
        // set up while the attention kernel still runs; it waits for its end itself
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)grid, (unsigned)p.merge_y);
        cfg.blockDim = dim3(256);
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, span_merge_kernel<D, KIND, FEW>, p);
    }
    return e;
}

template <int D, int KIND, int FEW>
static cudaError_t launch_span_form(const SpanMaps &maps, const SpanParams &p, int grid, cudaStream_t stream) {
    return p.stretch ? launch_span_one<D, KIND, FEW, true>(maps, p, grid, stream)
                     : launch_span_one<D, KIND, FEW, false>(maps, p, grid, stream);
}

#define XS_DEFINE_SPAN_ERROR_WORD(NAME)                                                                               \
    cudaError_t NAME(unsigned int *value, bool clear) {                                          \
        cudaError_t e = cudaMemcpyFromSymbol(value, g_xs_error, sizeof(unsigned int));                                \
        if (e == cudaSuccess && clear && *value) {                                                                    \
            const unsigned int zero = 0;                                                                              \
            e = cudaMemcpyToSymbol(g_xs_error, &zero, sizeof(unsigned int));                                          \
        }                                                                                                             \
        return e;                                                                                                     \
    }

#define XS_DEFINE_SPAN_ENTRY(D)                                                                                       \
    cudaError_t launch_span_d##D(const SpanMaps &maps, const SpanParams &p, int grid, cudaStream_t stream) {          \
        if (p.kind == SPAN_WHOLE) return launch_span_form<D, SPAN_WHOLE, 0>(maps, p, grid, stream);                   \
        if (p.few == 16) return launch_span_form<D, SPAN_PAGED, 16>(maps, p, grid, stream);                           \
        if constexpr (D > 64)                                                                                         \
            if (p.few == 32) return launch_span_form<D, SPAN_PAGED, 32>(maps, p, grid, stream);                       \
        return launch_span_form<D, SPAN_PAGED, 0>(maps, p, grid, stream);                                             \
    }                                                                                                                 \
    XS_DEFINE_SPAN_ERROR_WORD(read_error_word_span_d##D)

#define XS_DEFINE_SPAN_SERVE_ENTRY(D)                                                                                 \
    cudaError_t launch_span_serve_d##D(const SpanMaps &maps, const SpanParams &p, int grid, cudaStream_t stream) {    \
        if (p.kind == SPAN_PACKED) return launch_span_form<D, SPAN_PACKED, 0>(maps, p, grid, stream);                 \
        if (p.few == 16) return launch_span_form<D, SPAN_TREE, 16>(maps, p, grid, stream);                            \
        if (p.kind == SPAN_TREE_LANES) return launch_span_form<D, SPAN_TREE_LANES, 0>(maps, p, grid, stream);         \
        return launch_span_form<D, SPAN_TREE, 0>(maps, p, grid, stream);                                              \
    }                                                                                                                 \
    XS_DEFINE_SPAN_ERROR_WORD(read_error_word_span_serve_d##D)

}  // namespace xs
