"""The schedule of window and paged attention (`xs_span_schedule.cuh`) on the host: the device code itself, compiled
with g++, its warps run as 32 fibers that meet at every vote and shuffle.

Each CTA finds its part of the call's steps by itself, walks it stretch by stretch, and names the item whose first piece
it holds; the merge then adds up one record of each of the CTAs behind it. These tests run every CTA of a call and check
that each item's steps are covered once and in order, and that the records which the merge reads are those, and only
those, which the pieces of that item write in this call: the workspace needs no initialisation.
"""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "comm_comp_fusion_gb300", "csrc")
CUDA_INC = "/usr/local/cuda/include"

DRIVER = r"""
#include <cstdio>
#include <cstring>
#include <functional>
#include <vector>
#include <ucontext.h>
#include <cuda_runtime.h>
#undef __device__
#undef __forceinline__
#define __device__
#define __forceinline__ inline
using std::size_t;
struct Dim { unsigned x; };
static Dim block_, grid_, thread_, threads_;
#define blockIdx block_
#define gridDim grid_
#define threadIdx thread_
#define blockDim threads_
template <class T> static T min(T a, T b) { return b < a ? b : a; }
template <class T> static T max(T a, T b) { return a < b ? b : a; }
static int __ffs(int v) { return __builtin_ffs(v); }

// A warp: 32 fibers. A collective call leaves its value and yields; when a lane runs again, all lanes have left theirs.
struct Warp {
    ucontext_t main, lane[32];
    std::vector<char> stack[32];
    unsigned long long slot[2][32];
    int turn[32];
    bool done[32];
    std::function<void(int)> body;
    int at;
} W;
static unsigned long long meet(unsigned long long v, int (*from)(int, int), int arg) {
    const int me = W.at, t = W.turn[me];
    W.slot[t][me] = v;
    W.turn[me] ^= 1;
    swapcontext(&W.lane[me], &W.main);
    return W.slot[t][from(me, arg)];
}
template <class T> static T pass(T v, int (*from)(int, int), int arg) {
    unsigned long long x = 0;
    memcpy(&x, &v, sizeof v);
    x = meet(x, from, arg);
    memcpy(&v, &x, sizeof v);
    return v;
}
template <class T> static T __shfl_sync(unsigned, T v, int l) { return pass(v, [](int, int a) { return a & 31; }, l); }
template <class T> static T __shfl_xor_sync(unsigned, T v, int d) { return pass(v, [](int m, int a) { return m ^ a; }, d); }
template <class T> static T __shfl_up_sync(unsigned, T v, int d) { return pass(v, [](int m, int a) { return m < a ? m : m - a; }, d); }
static unsigned __ballot_sync(unsigned, int ok) {
    const int me = W.at, t = W.turn[me];
    meet(ok != 0, [](int m, int) { return m; }, 0);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= (unsigned)W.slot[t][i] << i;
    return r;
}
static void lane_main() {
    const int me = W.at;
    W.body(me);
    W.done[me] = true;
}
static void run_warp(std::function<void(int)> body) {
    W.body = body;
    for (int i = 0; i < 32; ++i) {
        W.stack[i].resize(1 << 16);
        getcontext(&W.lane[i]);
        W.lane[i].uc_stack.ss_sp = W.stack[i].data();
        W.lane[i].uc_stack.ss_size = W.stack[i].size();
        W.lane[i].uc_link = &W.main;
        makecontext(&W.lane[i], lane_main, 0);
        W.turn[i] = 0;
        W.done[i] = false;
    }
    for (bool any = true; any;) {
        any = false;
        for (int i = 0; i < 32; ++i)
            if (!W.done[i]) {
                W.at = i;
                swapcontext(&W.main, &W.lane[i]);
                any |= !W.done[i];
            }
    }
}

#include "xs_span_schedule.cuh"
using namespace xs;

template <bool PAGED> static void call(SpanParams &p) {
    const int chunks = ((PAGED ? p.N : p.n_pairs) + 31) / 32;
    std::vector<long long> sums(chunks);
    threads_.x = 32;
    if (chunks > 1)
        run_warp([&](int lane) {
            thread_.x = lane;  // one warp takes all chunks; read before the first yield
            span_chunk_sums<PAGED>(p, chunks, sums.data());
        });
    for (unsigned c = 0; c < grid_.x; ++c) {
        block_.x = c;
        SpanSched s[32];
        run_warp([&](int lane) { s[lane] = span_schedule<PAGED>(p, chunks, sums.data(), lane); });
        for (int i = 1; i < 32; ++i)
            if (memcmp(&s[i].rem, &s[0].rem, sizeof(long long)) || s[i].ctas != s[0].ctas || s[i].rounds != s[0].rounds ||
                (s[0].rem && (s[i].seq != s[0].seq || s[i].head != s[0].head || s[i].pair != s[0].pair || s[i].j != s[0].j)))
                std::printf("lanes differ in CTA %u\n", c);
        SpanWalk w;
        SpanPieces pieces{};
        span_walk_init<PAGED>(p, s[0], w);
        SpanSeg g;
        while (span_next<PAGED>(p, s[0], w, g)) {
            if (g.flags && g.j0 == 0) pieces = span_pieces_of(s[0], g);
            span_cut(g, p.stretch);
            for (bool more = true; more;) {
                std::printf("s %u %d %d %d %d %d %d %d %d\n", c, g.seq, g.head, g.tok0, g.j0, g.n, g.nw + g.ns, g.flags & 7, g.slot);
                const SpanSeg o = g;
                if ((more = o.flags & SPAN_MORE)) span_continue(g, o, p.stretch);
            }
        }
        span_cut(g, p.stretch);  // what ends the roles' loops
        if (g.n || g.flags) std::printf("CTA %u does not end\n", c);
        if (pieces.pieces) std::printf("p %u %d %d %d %d %d\n", c, pieces.seq, pieces.head, pieces.tok0, pieces.pieces, pieces.slot);
    }
}

int main() {
    int paged, grid, heads, item_tok, tile_tok, left, right, sinks, log2, stretch, S, N;
    static float rec[1];
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &paged, &grid, &heads, &item_tok, &tile_tok, &left, &right, &sinks, &log2, &stretch, &S, &N) == 12) {
        SpanParams p{};
        p.heads = heads;
        p.item_tok = item_tok;
        p.tile_tok = tile_tok;
        p.left = left < 0 ? 1 << 29 : left;
        p.right = right < 0 ? 1 << 29 : right;
        p.sinks = sinks;
        p.min_steps_log2 = log2;
        p.stretch = stretch;
        p.rec = rec;
        grid_.x = grid;
        std::vector<int> starts(1, 0), kv;
        if (paged) {
            p.N = N;
            p.page = 16;
            p.max_pages = 1 << 20;
            for (int i = 0; i < N; ++i) {
                int q, k;
                if (std::scanf("%d %d", &q, &k) != 2) return 1;
                starts.push_back(starts.back() + q);
                kv.push_back(k);
            }
            p.T = starts.back();
            p.q_start = starts.data();
            p.kv_len = kv.data();
            call<true>(p);
        } else {
            p.S = p.T = S;
            p.n_pairs = (S + 255) / 256;
            call<false>(p);
        }
        std::printf("end\n");
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA_INC, "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are missing")
    d = tmp_path_factory.mktemp("span")
    src, exe = d / "driver.cpp", d / "driver"
    src.write_text(DRIVER)
    subprocess.run([gxx, "-std=c++17", "-O2", "-w", "-I", CSRC, "-I", CUDA_INC, str(src), "-o", str(exe)], check=True)

    def run(text):
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        calls, cur = [], []
        for line in out.splitlines():
            if line == "end":
                calls.append(cur)
                cur = []
            else:
                cur.append(line)
        return calls
    return run


def steps_of(pos0, ntok, keys, left, right, sinks):
    """128-key tiles that some token at pos0 .. pos0 + ntok - 1 sees; one (masked) if there is none."""
    last = pos0 + ntok - 1
    hi = keys - 1 if right < 0 else min(keys - 1, last + right)
    if hi < 0:
        return 1
    lo = 0 if left < 0 else max(0, pos0 - left)
    tiles = set(range(lo // 128, hi // 128 + 1)) | set(range(0, -(-min(sinks, hi + 1) // 128)))
    return len(tiles)


PIECE, ADD, MORE = 1, 2, 4
WHOLE = 1 << 30


def verify(lines, items, grid, stretch=WHOLE):
    """items: {(seq, head, tok0): steps}."""
    parts, merges, open_, kept = {}, {}, {}, {}
    for line in lines:
        kind, *x = line.split()
        assert kind in "sp", line
        x = [int(v) for v in x]
        if kind == "s":
            cta, seq, head, tok0, j0, n, total, flags, slot = x
            item = seq, head, tok0
            assert items[item] == total and 1 <= n <= stretch
            assert 2 * cta <= slot <= 2 * cta + 1
            # the segments of a part follow one another and use one record, which no kept one has
            if flags & ADD:
                assert open_[cta][:3] == (item, j0, slot), line
            else:
                assert open_.get(cta) is None, line
                open_[cta] = (item, j0, slot, j0)
            begin = open_[cta][3]
            if flags != 0:
                assert slot not in kept, (line, kept[slot])
            if flags & MORE:
                assert n == stretch
                open_[cta] = (item, j0 + n, slot, begin)
                continue
            open_[cta] = None
            whole = begin == 0 and j0 + n == total
            assert bool(flags & PIECE) != whole, line
            parts.setdefault(item, []).append((cta, begin, j0 + n - begin, None if whole else slot))
            if not whole:
                kept[slot] = line
        else:
            cta, seq, head, tok0, pieces, slot = x
            merges[seq, head, tok0] = [slot] + [2 * (cta + i) for i in range(1, pieces)]
            assert cta + pieces <= grid
    assert set(parts) == set(items) and not any(open_.values())
    for item, segs in parts.items():
        segs.sort(key=lambda s: s[1])
        at = 0
        for _, j0, n, _ in segs:
            assert j0 == at, (item, segs)
            at += n
        assert at == items[item]
        if len(segs) == 1:
            assert item not in merges and segs[0][3] is None
            continue
        # the records the merge adds up are those that the pieces write, in order
        assert merges[item] == [s[3] for s in segs], (item, segs, merges[item])


def window_items(S, heads, left, right, sinks):
    return {(0, h, t): steps_of(t, min(256, S - t), S, left, right, sinks) for h in range(heads) for t in range(0, S, 256)}


def window(walk, cases, stretch=WHOLE):
    text = "".join(f"0 {grid} {heads} 256 128 {left} {right} {sinks} 2 {stretch} {S} 0\n"
                   for grid, heads, S, left, right, sinks in cases)
    for case, lines in zip(cases, walk(text)):
        grid, heads, S, left, right, sinks = case
        verify(lines, window_items(S, heads, left, right, sinks), grid, stretch)


def test_window_rests_smaller_than_the_grid(walk):
    """Whole items in rounds, then a rest of fewer steps than CTAs, among it items of two steps and more."""
    window(walk, [(152, 21 * 32, 256, -1, 0, 0),       # 4 rounds, 64 items of 2 steps left
                  (152, 23 * 16, 200, -1, 0, 0),
                  (152, 13 * 40, 256, -1, -1, 0),
                  (152, 73, 1280, 0, 0, 0),
                  (152, 152 * 2 + 61, 256, -1, 0, 0),  # the fewest items that are shared out
                  (152, 152 * 2 + 75, 300, 5, 5, 0),
                  (152, 152 * 3, 256, -1, 0, 0),       # nothing left
                  (7, 17, 256, -1, 0, 0), (7, 18, 129, -1, -1, 0), (1, 5, 700, 100, 0, 4), (2, 9, 512, 0, 0, 0)])
    window(walk, [(grid, heads, 256, -1, right, 0) for grid in (2, 3, 5, 10, 16) for heads in range(2 * grid, 4 * grid)
                  for right in (0, -1)])
    window(walk, [(grid, heads, 640, 0, 0, 0) for grid in (3, 7) for heads in range(grid, 4 * grid)])


def test_window_any_shape(walk):
    rng = random.Random(5)
    cases = []
    for _ in range(300):
        grid = rng.choice((1, 2, 3, 5, 8, 13, 20))
        S = rng.choice((rng.randint(1, 600), rng.randint(1, 3000), rng.randint(9000, 20000)))
        heads = rng.randint(1, max(1, rng.choice((grid // 2 + 1, 3 * grid, 6 * grid)) * 256 // max(S, 256)))
        left = rng.choice((-1, 0, rng.randint(0, 300), rng.randint(0, 4000)))
        right = rng.choice((-1, 0, 0, left, rng.randint(0, 1000)))
        cases.append((grid, heads, S, left, right, rng.choice((0, 0, 4, 128, 300))))
    for stretch in (WHOLE, 1, 3, 16):
        window(walk, cases, stretch)


def test_paged_any_batch(walk):
    rng = random.Random(6)
    text, wants = "", []
    for i in range(200):
        grid = rng.choice((1, 2, 5, 8, 20, 152 if i % 20 == 0 else 11))
        G, few = rng.choice(((1, 0), (1, 16), (4, 0), (4, 16), (3, 32), (16, 16), (7, 0), (128, 0)))
        tile = (few or 128) // G
        item = tile if few else 2 * tile
        heads, N = rng.randint(1, 6), rng.choice((1, 2, rng.randint(1, 9), rng.randint(30, 80)))
        left = rng.choice((-1, -1, 0, rng.randint(0, 700)))
        right, sinks = rng.choice((0, 0, -1, rng.randint(0, 300))), rng.choice((0, 4, 200))
        log2 = 0 if few else 1
        lens, stretch = [], rng.choice((WHOLE, WHOLE, 1, 2, 7, 30))
        for _ in range(N):
            q = rng.choice((0, 1, 1, rng.randint(1, 5), rng.randint(1, 3 * item)))
            lens.append((q, rng.choice((0, q, q + rng.randint(0, 300), q + rng.randint(0, 5000), rng.randint(0, q)))))
        text += f"1 {grid} {heads} {item} {tile} {left} {right} {sinks} {log2} {stretch} 0 {N} " + " ".join(f"{a} {b}" for a, b in lens) + "\n"
        wants.append((grid, stretch, {(n, h, t): steps_of(k - q + t, min(item, q - t), k, left, right, sinks)
                                       for n, (q, k) in enumerate(lens) for h in range(heads) for t in range(0, q, item)}))
    for (grid, stretch, items), lines in zip(wants, walk(text)):
        verify(lines, items, grid, stretch)
