"""The schedule of packed prompts and drafted trees on the host (see test_span_schedule.py): items count for their steps and
a constant, so that a CTA's part may end before an item's first step; the steps are covered once and the merge reads what
the pieces write all the same."""
import os
import random
import shutil
import subprocess

import pytest

from test_span_schedule import CSRC, CUDA_INC, DRIVER, WHOLE, steps_of, verify


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(CUDA_INC, "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are missing")
    d = tmp_path_factory.mktemp("weights")
    src, exe = d / "driver.cpp", d / "driver"
    code = DRIVER.replace("template <bool PAGED>", "template <int PAGED>").replace("sums(chunks)", "sums(2 * chunks)")
    code = code.replace("span_pieces_of(", "span_pieces_of<PAGED>(")
    code = code.replace("call<true>(p);", "if (std::scanf(\"%d\", &p.item_cost) != 1) return 1;\n"
                        "if (paged == 1) call<SPAN_PAGED>(p);\nif (paged == 2) call<SPAN_PACKED>(p);\nif (paged == 3) call<SPAN_TREE>(p);\nif (paged == 5) call<SPAN_TREE_LANES>(p);\n"
                        "if (paged == 4) { p.rec = nullptr; call<SPAN_PACKED>(p); }")
    code = code.replace("        SpanWalk w;", "        if (c == 0) std::printf(\"l %d\\n\", span_lanes<PAGED>(s[0]));\n        SpanWalk w;")
    assert "SPAN_TREE" in code and "2 * chunks" in code and "lanes" in code
    src.write_text(code)
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


def side_by_side(lines, grid):
    """With lanes, the CTAs of lane 0 first, then those of lane 1, ...: an item's pieces then lie in neighbouring ones."""
    lanes = int(lines[0].split()[1])
    assert lines[0][0] == "l" and 1 <= lanes <= 4
    out, per = [], grid // lanes
    at = lambda c: c % lanes * per + c // lanes  # noqa: E731
    for line in lines[1:]:
        x = line.split()
        if lanes > 1:
            c = int(x[1])
            assert c < per * lanes, "a CTA behind the lanes' has work"
            x[1] = str(at(c))
            x[-1] = str(2 * at(int(x[-1]) // 2) + int(x[-1]) % 2)
        out.append(" ".join(x))
    return lanes, out


@pytest.mark.parametrize("kind", (2, 3, 5))
@pytest.mark.parametrize("cost", (0, 1, 3, 40))
def test_weighted_any_batch(walk, kind, cost):
    rng = random.Random(10 * kind + cost)
    text, wants = "", []
    for i in range(150):
        grid = rng.choice((1, 2, 5, 8, 20, 152 if i % 20 == 0 else 11))
        G, few = rng.choice(((1, 0), (4, 0), (7, 0), (128, 0)) if kind == 2 else ((1, 0), (1, 16), (4, 0), (4, 16), (3, 32), (16, 16)))
        tile = (few or 128) // G
        item = tile if few else 2 * tile
        heads, N = rng.randint(1, 6), rng.choice((1, 2, rng.randint(1, 9), rng.randint(30, 80)))
        left, right, sinks = -1, -1, 0
        if kind == 2:
            left, right = rng.choice((-1, -1, 0, rng.randint(0, 700))), rng.choice((0, 0, -1, rng.randint(0, 300)))
            sinks = rng.choice((0, 4, 200))
        stretch, lens = rng.choice((WHOLE, WHOLE, 1, 2, 7, 30)), []
        for _ in range(N):
            q = rng.choice((0, 1, 1, rng.randint(1, 5), rng.randint(1, 3 * item), rng.randint(1, 6 * item)))
            lens.append((q, q if kind == 2 else rng.choice((0, q, q + rng.randint(0, 300), q + rng.randint(0, 5000), rng.randint(0, q)))))
        text += (f"{kind} {grid} {heads} {item} {tile} {left} {right} {sinks} {0 if few else 1} {stretch} 0 {N} "
                 + " ".join(f"{a} {b}" for a, b in lens) + f" {cost}\n")
        wants.append((grid, stretch, {(n, h, t): steps_of(k - q + t, min(item, q - t), k, left, right, sinks)
                                       for n, (q, k) in enumerate(lens) for h in range(heads) for t in range(0, q, item)}))
    calls = walk(text)
    assert len(calls) == len(wants)
    for (grid, stretch, items), lines in zip(wants, calls):
        verify(side_by_side(lines, grid)[1], items, grid, stretch)


def test_weights_even_out_item_changes(walk):
    """Many short prompts next to a long one: no CTA gets more than its share of steps and changes."""
    lens = [4000] + [100] * 60
    cost, grid = 3, 20
    items = {(n, h, t): steps_of(t, min(256, q - t), q, -1, 0, 0) for n, q in enumerate(lens) for h in range(2) for t in range(0, q, 256)}
    lines = walk(f"2 {grid} 2 256 128 -1 0 0 1 {WHOLE} 0 {len(lens)} " + " ".join(f"{q} {q}" for q in lens) + f" {cost}\n")[0]
    lines = side_by_side(lines, grid)[1]
    verify(lines, items, grid)
    units = [0] * grid
    for line in lines:
        if line[0] == "s":
            x = [int(v) for v in line.split()[1:]]
            units[x[0]] += x[5] + cost * (x[4] == 0)
    share = (sum(items.values()) + cost * len(items)) / grid
    assert max(units) <= share + cost + 1


def test_whole_items_without_workspace(walk):
    """Packed prompts without a workspace: every item whole, and no CTA more than its share of them."""
    rng = random.Random(3)
    text, wants = "", []
    for _ in range(60):
        grid, heads, N = rng.choice((1, 3, 20, 152)), rng.randint(1, 6), rng.choice((1, 3, 50))
        lens = [rng.choice((0, 1, rng.randint(1, 600))) for _ in range(N)]
        text += f"4 {grid} {heads} 64 32 -1 0 0 1 {WHOLE} 0 {N} " + " ".join(f"{q} {q}" for q in lens) + " 2\n"
        wants.append((grid, {(n, h, t): steps_of(t, min(64, q - t), q, -1, 0, 0)
                             for n, q in enumerate(lens) for h in range(heads) for t in range(0, q, 64)}))
    for (grid, items), lines in zip(wants, walk(text)):
        lines = side_by_side(lines, grid)[1]
        verify(lines, items, grid)
        count = [0] * grid
        for line in lines:
            assert line[0] == "s" and line.split()[5] == "0", line
            count[int(line.split()[1])] += 1
        assert max(count) <= -(-len(items) // grid)


def test_lanes_of_alike_trees(walk):
    """Trees of two to four items a key head: that many CTAs side by side, in step on the same keys."""
    rng = random.Random(8)
    text, wants = "", []
    for i in range(120):
        grid, heads, N = rng.choice((2, 3, 5, 20, 76, 152)), rng.randint(1, 6), rng.choice((1, 2, 16, 40))
        G, np = rng.choice(((1, 2), (4, 2), (8, 2), (8, 3), (8, 4), (16, 4), (8, 5)))
        tile = 128 // G
        item, stretch = 2 * tile, rng.choice((WHOLE, WHOLE, 3))
        lens = []
        for _ in range(N):
            q = rng.randint((np - 1) * item + 1, np * item) if rng.random() < 0.9 or N == 1 else 0
            lens.append((q, q + rng.randint(0, 3000)))
        if all(q == 0 for q, _ in lens):
            lens[0] = (np * item, np * item + 77)
        text += (f"5 {grid} {heads} {item} {tile} -1 -1 0 1 {stretch} 0 {N} " + " ".join(f"{a} {b}" for a, b in lens) + " 2\n")
        wants.append((grid, np, stretch, {(n, h, t): steps_of(k - q + t, min(item, q - t), k, -1, -1, 0)
                                           for n, (q, k) in enumerate(lens) for h in range(heads) for t in range(0, q, item)}))
    for (grid, np, stretch, items), lines in zip(wants, walk(text)):
        lanes, lines = side_by_side(lines, grid)
        assert lanes == (np if np <= min(4, grid) else 1)
        verify(lines, items, grid, stretch)
        if lanes > 1:  # lane r does what lane 0 does, with the items r
            per = grid // lanes
            of = [[(c - r * per, x[1], x[2], x[4], x[5]) for c, x in ((int(l.split()[1]), l.split()[1:]) for l in lines if l[0] == "s")
                   if c // per == r] for r in range(lanes)]
            assert all(o == of[0] for o in of)
