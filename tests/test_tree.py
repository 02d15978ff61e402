"""Drafted token trees: masks and positions from parents (xs_tree_mask), attention under masks of bits over the paged cache
(xs_attn_tree), against plain implementations in 64 bits; a speculative step with all operators in a row; refusals."""
import numpy as np
import pytest

from span_testlib import attend, bf16, check, values
from test_paged import Batch
from xs_testlib import from_dev, guarded, to_dev

I32 = np.int32


def random_parents(rng, n, late=2):
    """Parents of n tokens, each an earlier one or -1; `late` random ones' latest, so 1 makes bushes and many make chains."""
    return np.array([max(rng.integers(-1, i, late)) if i else -1 for i in range(n)], dtype=np.int64)


def closure(parents, most):
    """Masks [n, n] and depths of a tree, token by token; parents that are none count as -1, tokens from `most` on see
    nothing."""
    n = len(parents)
    seen, depth = np.zeros((n, n), bool), np.zeros(n, np.int64)
    for i in range(min(n, most)):
        p = int(parents[i])
        if 0 <= p < i:
            seen[i] = seen[p]
            depth[i] = depth[p] + 1
        seen[i, i] = True
    return seen, depth


def to_words(seen, words):
    """[n, m] truth values to [n, words] int32."""
    bits = np.zeros((seen.shape[0], words * 32), bool)
    m = min(seen.shape[1], words * 32)
    bits[:, :m] = seen[:, :m]
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32).astype(np.int64).astype(np.uint32).view(I32)


# ------------------------------------------------------------------ masks from parents

MASKS = [  # q_len, kv_len, words, spare, late
    ([1], [1], 1, 0, 1),
    ([8, 8, 8], [300, 8, 50], 1, 3, 2),
    ([5, 0, 32, 1, 33], [9, 4, 32, 900, 40], 1, 2, 2),          # one token more than bits
    ([64, 1, 250, 256, 300], [100, 1, 300, 256, 1000], 8, 0, 2),
    ([90, 96, 100], [2000, 96, 100], 3, 5, 1),
    ([256], [300], 8, 0, 60),                                    # nearly a chain
    ([7] * 400, [40] * 400, 2, 1, 2),
    ([14, 15, 16, 17, 18, 33, 34, 100, 255, 256], [300] * 10, 8, 2, 4000),   # chains
    ([32, 31, 17], [300] * 3, 1, 0, 4000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(MASKS)))
@pytest.mark.parametrize("with_pos", (True, False))
def test_tree_mask_matches_closure(case, with_pos):
    import torch
    import comm_comp_fusion_gb300 as xs
    q_len, kv_len, words, spare, late = MASKS[case]
    rng = np.random.default_rng(case)
    N, T = len(q_len), sum(q_len) + spare
    parents = np.concatenate([random_parents(rng, n, late) for n in q_len] + [np.zeros(spare, np.int64)])
    bad = rng.random(T) < 0.05  # what is no earlier token of the sequence: a root
    start = np.concatenate(([0], np.cumsum(q_len)))
    for n in range(N):
        for i in range(q_len[n]):
            if bad[start[n] + i]:
                parents[start[n] + i] = rng.choice((i, i + 1, -2, 2 ** 31 - 1, -2 ** 31))
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    mask, pos = guarded(T * words, torch.int32, 77), guarded(T, torch.int32, 77)
    xs.tree_mask(dev(parents), dev(start), dev(kv_len) if with_pos else None, mask, pos if with_pos else None, N, T, words)
    torch.cuda.synchronize()
    mask, pos = mask.cpu().numpy().reshape(T, words), pos.cpu().numpy()
    for n in range(N):
        rows = slice(start[n], start[n + 1])
        seen, depth = closure(parents[rows], 32 * words)
        assert np.array_equal(mask[rows], to_words(seen, words))
        assert np.array_equal(pos[rows], kv_len[n] - q_len[n] + depth if with_pos else np.full(q_len[n], 77))
    assert (mask[start[-1]:] == 77).all() and (pos[start[-1]:] == 77).all()


@pytest.mark.gpu
def test_tree_mask_ignores_bad_metadata_and_follows_a_graph():
    import torch
    import comm_comp_fusion_gb300 as xs
    N, T, words = 3, 9, 2
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    parents, start, kv = dev([-1, 0, 1, -1, 0, 0, -1, 0, 0]), dev([0, 3, 6, 9]), dev([50, 3, 10])
    mask, pos = guarded(T * words, torch.int32, 0), guarded(T, torch.int32, 0)
    for bad in ([9, 100, 10 ** 9, 2 ** 31 - 1], [-7, -3, -1, 0], [5, 5, 4, 2]):
        xs.tree_mask(parents, dev(bad), kv, mask, pos, N, T, words)
        torch.cuda.synchronize()
        assert not mask.any() and not pos.any()
    xs.tree_mask(parents, start, kv, mask, pos, N, T, words)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xs.tree_mask(parents, start, kv, mask, pos, N, T, words)
    parents.copy_(dev([-1, -1, 0, -1, 0, 1, -1, 0, -1]))
    kv.copy_(dev([3, -2, 1000]))
    start.copy_(dev([0, 3, 6, 8]))
    mask.fill_(5)
    g.replay()
    torch.cuda.synchronize()
    assert mask.view(T, words)[:, 0].tolist() == [1, 2, 5, 1, 3, 7, 1, 3, 5]
    assert mask.view(T, words)[:8, 1].tolist() == [0] * 8
    assert pos.tolist()[:8] == [0, 0, 1, -3, -2, -1, 998, 999]


# ------------------------------------------------------------------ attention

class Trees(Batch):
    """A cache whose sequences' new tokens are under masks of bits: random trees, or any bits (`dense`: their share)."""

    def __init__(self, q_len, kv_len, H, Hk, D, page, words, spare=0, seed=0, dense=None, **kw):
        import torch
        super().__init__(q_len, kv_len, H, Hk, D, page, spare, seed, **kw)
        rng = np.random.default_rng(seed + 500)
        self.words, self.bits = words, []
        rows = []
        for n in q_len:
            if dense is None:
                seen = closure(random_parents(rng, n), 32 * words)[0]
            else:
                seen = rng.random((n, 32 * words)) < dense  # bits past the new tokens among them: not looked at
            self.bits.append(seen)
            rows.append(to_words(seen, words))
        rows.append(rng.integers(-2 ** 31, 2 ** 31, (spare, words)).astype(I32))
        self.mask = torch.from_numpy(np.concatenate(rows)).cuda()
        self.ws = guarded(xs_size(self.N, self.T, H, Hk, D), torch.uint8)

    def call(self, out=None, **kw):
        import comm_comp_fusion_gb300 as xs
        return xs.attn_tree(self.dq, self.kp, self.vp, self.table, self.q_start, self.kv_len, self.mask,
                            self.out if out is None else out, self.N, self.T, self.H, self.Hk, self.D, self.page,
                            self.n_pages, self.max_pages, self.words, self.D ** -0.5, self.ws, **kw)

    def seen(self, n):
        ql, kl = self.q_len[n], self.kv[n]
        seen = np.zeros((ql, kl), bool)
        c = kl - ql
        seen[:, :max(c, 0)] = True
        for j in range(min(ql, 32 * self.words)):
            if c + j >= 0 and j < self.bits[n].shape[1]:
                seen[:, c + j] = self.bits[n][:, j]
        return seen

    def verify(self, what="", heads=None):
        import torch
        import comm_comp_fusion_gb300 as xs
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        got, G, t = from_dev(self.out).reshape(self.T, self.H, self.D), self.H // self.Hk, 0
        for n, ql in enumerate(self.q_len):
            seen = self.seen(n)
            for h in range(self.H) if self.H * ql < 9000 else sorted({0, 1, self.H // 3, self.H // 2, self.H - 1}):
                ref, bound = attend(self.q[t:t + ql, h], self.k[n][:, h // G], self.v[n][:, h // G], seen, self.D ** -0.5)
                check(got[t:t + ql, h], ref, bound, f"{what} sequence {n} head {h}")
                assert (got[t:t + ql, h][~seen.any(-1)] == 0).all()
            t += ql
        assert (got[t:] == 0xFFFF).all(), "rows of no sequence were written"


def xs_size(*a):
    import comm_comp_fusion_gb300 as xs
    return xs.attn_tree_workspace_size(*a)


TREES = [  # q_len, kv_len, H, Hk, D, page, words, spare, dense
    ([1], [1], 1, 1, 64, 16, 1, 0, None),
    ([8, 8, 8, 8], [300, 1200, 8, 129], 32, 8, 128, 16, 1, 0, None),
    ([3, 1, 2], [4100, 33, 900], 8, 2, 128, 64, 1, 2, None),               # few rows
    ([4, 4, 1, 3], [700, 1500, 131, 66], 4, 4, 96, 32, 1, 0, None),
    ([16], [2000], 4, 4, 64, 16, 1, 1, None),                              # 16 tokens of one head each
    ([7, 5, 8], [777, 128, 1290], 6, 2, 128, 256, 2, 0, None),             # tiles of 32 rows
    ([16] * 5, [5000, 16, 17, 300, 144], 16, 2, 128, 64, 1, 3, None),      # 128 rows a sequence and key head
    ([61, 7, 0, 33], [2000, 500, 40, 33], 24, 24, 64, 32, 2, 5, None),
    ([64, 64], [1000, 64], 16, 2, 128, 64, 2, 0, None),                    # 512 rows: several items
    ([130, 200, 256], [1130, 200, 3000], 4, 2, 96, 16, 8, 0, None),
    ([300, 40], [1000, 500], 4, 4, 64, 64, 8, 0, None),                    # more tokens than bits
    ([20, 50], [20, 50], 8, 8, 128, 1024, 1, 0, None),                     # no context; more tokens than bits
    ([40, 9], [39, 3], 4, 2, 64, 16, 2, 2, None),                          # fewer keys than new tokens
    ([12, 40, 100], [612, 40, 1000], 8, 2, 128, 32, 4, 1, 0.3),            # any bits
    ([2, 3], [2, 3], 16, 2, 64, 16, 1, 0, 0.2),                            # rows that see nothing
    ([2, 3, 1], [600, 3, 1], 4, 2, 128, 16, 1, 0, 0.0),                    # the context alone, or nothing
    ([90], [500], 128, 1, 64, 16, 3, 0, 0.5),                              # 128 heads a key head
    ([33], [160], 7, 1, 64, 32, 2, 0, 1.0),                                # seven heads a key head; every bit
    ([1] * 70, list(range(1, 1400, 20)), 4, 2, 64, 16, 1, 0, None),        # more sequences than a warp's lanes
    ([30] * 40, list(range(100, 2100, 50)), 8, 4, 128, 32, 1, 7, None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree_matches_64_bits(case):
    q_len, kv_len, H, Hk, D, page, words, spare, dense = TREES[case]
    b = Trees(q_len, kv_len, H, Hk, D, page, words, spare, seed=case, dense=dense)
    b.call()
    b.verify(what=str(TREES[case][2:]))
    b.out.fill_(-1)
    b.ws.fill_(255)
    b.call()
    b.verify(what="again, workspace of ones")


@pytest.mark.gpu
@pytest.mark.parametrize("D", (64, 96, 128))
@pytest.mark.parametrize("G,q_len", ((1, [13, 16, 3]), (5, [3, 1, 0]), (3, [10, 7, 8]), (16, [1, 2, 1]), (11, [4, 1, 1])))
def test_tree_few_rows(D, G, q_len):
    """Trees that do and do not fill the few-rows tiles, with the border of context and tree at places around a tile's."""
    for kv in ([2500, 129, 700], [128 + 13, 256 + 16, 3], [384 + 6, 250, 128]):
        b = Trees(q_len, kv, 2 * G, 2, D, 32, 1, spare=2, seed=G + D)
        b.call()
        b.verify(what=f"{kv}")


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,kv_len,H,Hk,D,page", (([64, 0, 61, 50], [3000, 9, 61, 2000], 16, 2, 128, 64), ([40] * 5, [700, 1500, 40, 41, 5000], 4, 1, 64, 16),
                                                      ([96, 90], [4000, 1100], 8, 1, 96, 32), ([128] * 3, [2500, 300, 129], 24, 3, 128, 128),
                                                      ([255, 250, 129], [3000, 250, 900], 4, 2, 64, 64), ([64] * 40, [64 + 37 * i for i in range(40)], 8, 1, 64, 16)))
@pytest.mark.parametrize("wide", (False, True))
def test_tree_alike_trees_side_by_side(q_len, kv_len, H, Hk, D, page, wide):
    """Trees of two to four items a key head each, whose items neighbouring CTAs take side by side, whole and in pieces."""
    import torch
    b = Trees(q_len, kv_len, H, Hk, D, page, 8, spare=1, seed=D + len(q_len))
    if wide:  # a table that could hold more than 2^18 keys
        t = torch.full((b.N, 2 ** 18 // page + 100), -5, dtype=torch.int32, device="cuda")
        t[:, :b.max_pages] = b.table
        b.table, b.max_pages = t, t.shape[1]
    b.ws.fill_(255)
    b.call()
    b.verify()
    first = from_dev(b.out).copy()
    b.out.fill_(-1)
    b.call()
    torch.cuda.synchronize()
    assert np.array_equal(first, from_dev(b.out))


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", (0, 1, 31, 32, 33, 95, 96, 97, 127, 128, 129, 250))
def test_tree_borders(ctx):
    """Every alignment of the tree's first bit in a tile of keys, for trees of one to four words."""
    for ql, H, words in ((5, 2, 1), (32, 4, 1), (64, 2, 2), (100, 4, 4), (128, 2, 4)):
        b = Trees([ql, 3], [ctx + ql, ctx + 3], H, 1, 64, 16, words, seed=ctx, dense=0.5)
        b.call()
        b.verify(what=f"{ql} {H}")


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,H,Hk", (([2, 3], 4, 2), ([20, 16], 16, 2), ([70, 9], 4, 2)))
@pytest.mark.parametrize("ramp", ((8.0, 0.0), (0.0, 8.0)))
def test_tree_rising_and_falling_keys(q_len, H, Hk, ramp):
    b = Trees(q_len, [1900, 900], H, Hk, 128, 32, 3, seed=4, ramp=ramp, dense=0.1)
    b.call()
    b.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,H,Hk,D", (([2, 1, 3], 8, 2, 128), ([16, 9], 16, 2, 64), ([70, 12], 4, 2, 96)))
def test_tree_wide_tables(q_len, H, Hk, D):
    """A table that could hold more than 2^18 keys a sequence, around ordinary lengths, in every form."""
    import torch
    b = Trees(q_len, [700, 2900, 130][:len(q_len)], H, Hk, D, 32, 3, spare=1, seed=D)
    wide = torch.full((b.N, 9000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :b.max_pages] = b.table
    b.table, b.max_pages = wide, 9000
    b.call()
    b.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,Hk,D,keys", ((3, 8, 2, 128, 2 ** 21 + 5), (16, 16, 2, 64, 2 ** 20 + 900), (40, 8, 1, 96, 2 ** 20 - 77)))
def test_tree_very_many_keys(T, H, Hk, D, keys):
    """Millions of keys before a tree, in every form. Values around 1; four pages stand for all before the tree, so a key's
    weight counts as often as it comes. The bound: that of span_testlib.attend, and 2^14 additions of a stretch that
    truncate by 2^-23 at most."""
    import torch
    import comm_comp_fusion_gb300 as xs
    page, own = 1024, 4096
    max_pages = -(-keys // page)
    rng = np.random.default_rng(keys)
    gen = torch.Generator(device="cuda").manual_seed(keys)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    n_pages = 6  # the last two hold the tree
    q, kp, vp = rand(T, H, D).bfloat16(), rand(n_pages, page, Hk, D).bfloat16(), (1 + 0.25 * rand(n_pages, page, Hk, D)).bfloat16()
    table = (torch.arange(max_pages, device="cuda") % 4).to(torch.int32)
    table[-2], table[-1] = 4, 5
    q_start, kv_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [keys]))
    seen = rng.random((T, T)) < 0.5
    words = (T + 31) // 32
    mask = torch.from_numpy(to_words(seen, words)).cuda()
    out = guarded(T * H * D)
    ws = guarded(xs_size(1, T, H, Hk, D), torch.uint8, 0xFF)
    xs.attn_tree(q, kp, vp, table, q_start, kv_len, mask, out, 1, T, H, Hk, D, page, n_pages, max_pages, words, D ** -0.5, ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got = from_dev(out).reshape(T, H, D)
    first = (max_pages - 2) * page                     # place of the two last pages
    j = torch.arange(own + 2 * page, device="cuda")
    often = torch.zeros((T, own + 2 * page), dtype=torch.float64, device="cuda")
    often[:, :own] = ((first - 1 - j[:own]) // own + 1).clamp(min=0).double()
    place = first + j[own:] - own
    often[:, own:] = (place < keys - T).double()
    for i in range(T):
        often[:, own + keys - T + i - first] = torch.from_numpy(seen[:, i].astype(np.float64)).cuda()
    for h in sorted({0, 1, H // 2, H - 1}):
        k, v = kp[:, :, h * Hk // H].reshape(-1, D).double(), vp[:, :, h * Hk // H].reshape(-1, D).double()
        qd = q[:, h].double()
        s = qd @ k.T * D ** -0.5
        w = often * (s - s.amax(-1, keepdim=True)).exp()
        w = w / w.sum(-1, keepdim=True)
        ref, a = w @ v, w @ v.abs()
        delta = 2.0 ** -18 * (qd.abs() @ k.abs().T * D ** -0.5).amax(-1, keepdim=True)
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * delta + 2.0 ** -9) * a
        check(got[:, h], ref.cpu().numpy(), bound.cpu().numpy(), f"head {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("N,rows", ((1000, 1), (65536, 1), (30000, 3)))
def test_tree_very_many_sequences(N, rows):
    """Thousands of short sequences with chains of up to two tokens: the schedule's sums over the whole batch."""
    import torch
    import comm_comp_fusion_gb300 as xs
    H, Hk, D, page, n_pages = 2 * rows, 2, 64, 16, 300
    gen = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda").bfloat16()  # noqa: E731
    kp, vp = rand(n_pages, page, Hk, D), rand(n_pages, page, Hk, D)
    q_len = torch.randint(0, 3, (N,), generator=gen, device="cuda")
    kv = torch.randint(2, 2 * page + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    table = torch.randint(0, n_pages, (N, 2), generator=gen, device="cuda", dtype=torch.int32)
    q_start = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), q_len.cumsum(0)))
    T = int(q_start[-1])
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), q_len)
    i = torch.arange(T, device="cuda") - q_start[seq]
    mask = torch.where(i == 0, 1, 2).to(torch.int32)   # the second token does not see the first
    q, out = rand(T, H, D), guarded(T * H * D)
    ws = guarded(xs_size(N, T, H, Hk, D), torch.uint8)
    xs.attn_tree(q, kp, vp, table, q_start.to(torch.int32), kv, mask, out, N, T, H, Hk, D, page, n_pages, 2, 1, 0.125, ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got = values(from_dev(out)).reshape(T, H, D)
    for a in range(0, T, 20000):
        r = slice(a, min(a + 20000, T))
        k = kp[table[seq[r]].long()].view(-1, 2 * page, Hk, D).double().repeat_interleave(rows, 2)
        v = vp[table[seq[r]].long()].view(-1, 2 * page, Hk, D).double().repeat_interleave(rows, 2)
        s = torch.einsum("thd,tkhd->thk", q[r].double(), k) * 0.125
        key, c = torch.arange(2 * page, device="cuda"), (kv[seq[r]] - q_len[seq[r]]).view(-1, 1)
        see = (key < c) | (key == c + i[r].view(-1, 1))
        w = s.masked_fill(~see.unsqueeze(1), -np.inf).softmax(-1)
        ref, b = (torch.einsum("thk,tkhd->thd", w, x).cpu().numpy() for x in (v, v.abs()))
        # the bound of span_testlib.attend; here scale sum |q k| is below 2^5, so the scores' share 2 delta is below 2^-12
        assert (np.abs(got[r] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * b + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,kv_len,H,Hk,D,page", (([1] * 4, [700, 90, 1500, 64], 8, 2, 128, 16), ([9, 300], [300, 900], 4, 2, 96, 64),
                                                      ([16, 1], [400, 33], 16, 2, 64, 32)))
def test_tree_of_a_triangle_is_causal(q_len, kv_len, H, Hk, D, page):
    """With masks of each token and all before it, xs_attn_tree computes what xs_attn_paged does (and in the same order
    of sums, so to the bit)."""
    import torch
    import comm_comp_fusion_gb300 as xs
    words = 8
    b = Trees(q_len, kv_len, H, Hk, D, page, words, seed=1)
    rows = []
    for n in q_len:
        rows.append(to_words(np.tril(np.ones((n, n), bool)), words))
    b.mask = torch.from_numpy(np.concatenate(rows)).cuda()
    b.bits = [np.tril(np.ones((n, n), bool)) for n in q_len]
    b.call()
    b.verify()
    if max(q_len) <= 32 * words:
        other = guarded(b.T * H * D)
        Batch.call(b, out=other)
        got, want = (values(from_dev(x)) for x in (b.out, other))
        assert np.abs(got - want).max() <= 2.0 ** -6 * np.abs(want).max()


@pytest.mark.gpu
def test_tree_spoiled_rows_stay_alone():
    """A row of q with NaN or an infinity spoils its own output alone."""
    import torch
    for q_len, H, Hk, D in (([3, 2], 8, 2, 128), ([40, 64], 4, 2, 64)):
        b = Trees(q_len, [500, 300], H, Hk, D, 32, 2, seed=9)
        bits, bad = b.qb.copy(), {(0, 0): 0x7FC1, (b.T - 1, 1): 0xFF80}
        for (t, h), x in bad.items():
            bits[t, h, ::5] = x
        b.dq = to_dev(bits)
        b.call()
        torch.cuda.synchronize()
        got, t = from_dev(b.out).reshape(b.T, H, D), 0
        for n, ql in enumerate(q_len):
            for h in range(H):
                ok = [i for i in range(ql) if (t + i, h) not in bad]
                ref, bound = attend(b.q[t:t + ql, h][ok], b.k[n][:, h // (H // Hk)], b.v[n][:, h // (H // Hk)], b.seen(n)[ok],
                                    D ** -0.5)
                check(got[t:t + ql, h][ok], ref, bound, f"sequence {n} head {h}")
            t += ql


@pytest.mark.gpu
def test_tree_graphs_and_streams():
    """Captured calls follow masks, lengths, starts and table, two of them in one workspace; two calls on two streams."""
    import torch
    a, c = Trees([4, 2, 5], [700, 300, 1000], 8, 2, 128, 16, 1, seed=7), Trees([60, 33], [500, 1200], 4, 4, 64, 32, 2, seed=8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, s in zip((a, c), streams):
            x.call(stream=s)
    torch.cuda.synchronize()
    a.verify()
    c.verify()
    c.ws = a.ws
    graphs = []
    for x in (a, c):
        x.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.call()
        graphs.append(g)
    full, rng = (a.k, a.v), np.random.default_rng(3)
    for kv in ([700, 300, 1000], [4, 290, 513], [128, 127, 640]):
        a.kv = kv
        a.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        a.k, a.v = ([x[:n] for x, n in zip(y, kv)] for y in full)
        a.bits = [rng.random((n, 32)) < 0.5 for n in a.q_len]
        a.mask.copy_(torch.from_numpy(np.concatenate([to_words(x, 1) for x in a.bits])))
        for x, g in zip((a, c), graphs):
            x.out.fill_(-1)
            g.replay()
            x.verify()


@pytest.mark.gpu
def test_tree_ignores_bad_metadata():
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Trees([2, 3, 40], [40, 60, 70], 4, 2, 64, 16, 2, spare=2, seed=1)
    b.kp.fill_(0)
    b.vp.fill_(0)
    good = b.table.clone(), b.q_start.clone(), b.kv_len.clone()
    for what in range(5):
        b.table, b.q_start, b.kv_len = (x.clone() for x in good)
        if what == 0:
            b.table.fill_(2 ** 31 - 1)
        elif what == 1:
            b.table.fill_(-1)
        elif what == 2:
            b.kv_len.copy_(torch.tensor([2 ** 31 - 1, -5, 10 ** 6], dtype=torch.int32))
        elif what == 3:
            b.q_start.copy_(torch.tensor([9, 100, 10 ** 9, 2 ** 31 - 1], dtype=torch.int32))
        else:
            b.q_start.copy_(torch.tensor([-7, -3, -1, 0], dtype=torch.int32))
        b.call()
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()


@pytest.mark.gpu
def test_tree_pool_past_32_bits():
    import torch
    Hk, D, page = 8, 128, 256
    n_pages = 2 ** 31 // (Hk * D * page) + 8
    kp, vp = (torch.empty(n_pages * page * Hk * D, dtype=torch.int16, device="cuda") for _ in range(2))
    b = Trees([17], [700], 16, Hk, D, page, 1, seed=2)
    last = torch.arange(n_pages - 1, n_pages - 4, -1, dtype=torch.int32, device="cuda")
    old = b.table[0, :3].clone()
    for dst, src in ((kp, b.kp), (vp, b.vp)):
        dst.view(n_pages, -1)[last.long()] = src.view(b.n_pages, -1)[old.long()]
    b.table[0, :3] = last
    b.kp, b.vp, b.n_pages = kp, vp, n_pages
    b.call()
    b.verify()


# ------------------------------------------------------------------ in a row

@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,D", ((8, 2, 128), (4, 4, 64)))
def test_speculative_step(H, Hk, D):
    """A drafted step with all operators in a row: a prompt turned into the cache and attended packed, then a tree whose
    masks and positions come from its parents. Each token's output equals that of the prompt followed by its own branch
    alone, in 64 bits."""
    import torch
    import comm_comp_fusion_gb300 as xs
    rng = np.random.default_rng(D)
    page, words, P, tree = 32, 1, [70, 33], [11, 6]
    N, row, scale = 2, (H + 2 * Hk) * D, D ** -0.5
    ax = xs.RopeAxes.powers((D,), halves=True)
    need = [-(-(p + t) // page) for p, t in zip(P, tree)]
    cols, n_pages = max(need), sum(need)
    table = np.full((N, cols), -1)
    ids = rng.permutation(n_pages)
    for n in range(N):
        table[n, :need[n]] = ids[sum(need[:n]):sum(need[:n + 1])]
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    dtable = dev(table)
    kp, vp = (torch.full((n_pages, page, Hk, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def rows(T):
        x = to_dev(bf16(rng, (T, row))[0]).view(torch.bfloat16)
        return x[:, :H * D], x[:, H * D:(H + Hk) * D], x[:, (H + Hk) * D:]

    T = sum(P)
    q, k, v = rows(T)
    start, kv = dev([0, P[0], T]), dev(P)
    qo, ko, out = guarded(T * H * D).view(torch.bfloat16), guarded(T * Hk * D).view(torch.bfloat16), guarded(T * H * D)
    xs.cache_append_rope(q, k, v, qo, kp, vp, dtable, start, kv, N, T, H, Hk, D, page, n_pages, cols, ax, k_out=ko)
    ws = guarded(xs.attn_packed_workspace_size(N, T, H, Hk, D), torch.uint8)
    xs.attn_packed(qo, ko, v, start, out, N, T, H, Hk, D, scale, workspace=ws)
    M = sum(tree)
    parents = [random_parents(rng, t) for t in tree]
    tq, tk, tv = rows(M)
    t_start, t_kv = dev([0, tree[0], M]), dev([p + t for p, t in zip(P, tree)])
    mask, pos = guarded(M * words, torch.int32, 0), guarded(M, torch.int32, 0)
    tqo, t_out = guarded(M * H * D).view(torch.bfloat16), guarded(M * H * D)
    xs.tree_mask(dev(np.concatenate(parents)), t_start, t_kv, mask, pos, N, M, words)
    xs.cache_append_rope(tq, tk, tv, tqo, kp, vp, dtable, t_start, t_kv, N, M, H, Hk, D, page, n_pages, cols, ax, pos=pos)
    ws2 = guarded(xs.attn_tree_workspace_size(N, M, H, Hk, D), torch.uint8)
    xs.attn_tree(tqo, kp, vp, dtable, t_start, t_kv, mask, t_out, N, M, H, Hk, D, page, n_pages, cols, words, scale, ws2)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got, t_got = from_dev(out).reshape(T, H, D), from_dev(t_out).reshape(M, H, D)
    num = lambda x, h: values(from_dev(x.contiguous().view(torch.int16))).reshape(-1, h, D)  # noqa: E731
    Q, K, V, TQ = num(qo, H), num(ko, Hk), num(v, Hk), num(tqo, H)
    pool_k, TV = num(kp, Hk).reshape(n_pages, page, Hk, D), num(tv, Hk)
    a = b = 0
    for n in range(N):
        places = np.arange(P[n], P[n] + tree[n])
        tk_n = pool_k[table[n, places // page], places % page]  # the turned keys of the tree, as they stand in the cache
        for h in range(H):
            g = h // (H // Hk)
            ref, bound = attend(Q[a:a + P[n], h], K[a:a + P[n], g], V[a:a + P[n], g], np.tril(np.ones((P[n], P[n]), bool)), scale)
            check(got[a:a + P[n], h], ref, bound, f"prompt {n} head {h}")
            for i in range(tree[n]):
                branch = [i]
                while parents[n][branch[0]] >= 0:
                    branch.insert(0, int(parents[n][branch[0]]))
                kk = np.concatenate((K[a:a + P[n], g], tk_n[branch, g]))
                vv = np.concatenate((V[a:a + P[n], g], TV[b:b + tree[n]][branch, g]))
                ref, bound = attend(TQ[b + i:b + i + 1, h], kk, vv, np.ones((1, len(kk)), bool), scale)
                check(t_got[b + i:b + i + 1, h], ref, bound, f"tree {n} token {i} head {h}")
                assert int(pos[b + i]) == P[n] + len(branch) - 1
        a, b = a + P[n], b + tree[n]


# ------------------------------------------------------------------ refusals

A = [0x10000000 * (i + 1) for i in range(12)]


def test_tree_refusals():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs

    def attn(**kw):
        a = dict(q=A[0], k_pages=A[1], v_pages=A[2], page_table=A[3], q_start=A[4], kv_len=A[5], mask=A[6], out=A[7], N=2, T=10,
                 H=8, Hk=2, D=128, page=16, n_pages=50, max_pages=20, words=2, scale=0.1, workspace=A[8],
                 workspace_bytes=1 << 27, check=False)
        a.update(kw)
        return xs.attn_tree(**a)

    def mask(**kw):
        a = dict(parents=A[0], q_start=A[1], kv_len=A[2], mask=A[3], pos=A[4], N=2, T=10, words=2, check=False)
        a.update(kw)
        return xs.tree_mask(**a)

    for name in ("q", "k_pages", "v_pages", "page_table", "q_start", "kv_len", "mask", "out"):
        assert attn(**{name: None}) == xs.XS_ERR_NULL
    for name in ("parents", "q_start", "mask", "kv_len"):
        assert mask(**{name: None}) == xs.XS_ERR_NULL
    assert mask(kv_len=None, pos=None, N=0) == xs.XS_OK
    for f in (attn, mask):
        for kw in (dict(N=-1), dict(T=-1), dict(N=65537), dict(T=(1 << 29) + 1), dict(words=0), dict(words=9), dict(words=-1)):
            assert f(**kw) == xs.XS_ERR_SHAPE, kw
        assert f(N=0) == xs.XS_OK and f(T=0) == xs.XS_OK
        assert f(mask=A[6] + 2) == xs.XS_ERR_ALIGN and f(q_start=A[10] + 1) == xs.XS_ERR_ALIGN
    for kw in (dict(H=7), dict(H=0), dict(Hk=0), dict(scale=0.0), dict(scale=float("nan")), dict(T=1 << 28), dict(n_pages=0)):
        assert attn(**kw) == xs.XS_ERR_SHAPE, kw
    for kw in (dict(D=256), dict(D=80), dict(page=48), dict(H=258)):
        assert attn(**kw) == xs.XS_ERR_UNSUPPORTED, kw
    for kw in (dict(q=A[0] + 2), dict(out=A[7] + 8), dict(kv_len=A[5] + 2), dict(page_table=A[3] + 1)):
        assert attn(**kw) == xs.XS_ERR_ALIGN, kw
    for name in ("q", "k_pages", "v_pages", "page_table", "q_start", "kv_len", "mask"):
        assert attn(**{name: A[7] + 16}) == xs.XS_ERR_ALIAS, name
    assert attn(workspace=None, workspace_bytes=0) == xs.XS_ERR_NULL
    for kw in (dict(workspace=None, workspace_bytes=8), dict(workspace=A[8] + 128), dict(workspace=A[7]), dict(workspace=A[6])):
        assert attn(**kw) == xs.XS_ERR_WORKSPACE, kw
    for out in ("mask", "pos"):
        for name in ("parents", "q_start", "kv_len"):
            assert mask(**{out: A[9], name: A[9] + 4}) == xs.XS_ERR_ALIAS
    assert mask(mask=A[9], pos=A[9] + 8) == xs.XS_ERR_ALIAS
    i, x, p = torch.zeros(64, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(2048, dtype=torch.bfloat16)
    for bad in (i.long(), i.float(), i[:3], i.view(32, 2)[:, 0]):
        with pytest.raises(ValueError, match="int32"):
            xs.tree_mask(bad, i, i, i, i, 1, 4, 1)
        with pytest.raises(ValueError, match="int32"):
            xs.tree_mask(i, i, i, bad, i, 1, 4, 1)
        with pytest.raises(ValueError, match="int32"):
            xs.attn_tree(x, p, p, i, i, i, bad, x, 1, 4, 2, 2, 64, 16, 1, 1, 1, 0.1)
    with pytest.raises(ValueError, match="bfloat16"):
        xs.attn_tree(x.half(), p, p, i, i, i, i, x, 1, 4, 2, 2, 64, 16, 1, 1, 1, 0.1)
    with pytest.raises(ValueError, match="workspace"):
        xs.attn_tree(A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], 2, 4, 4, 2, 64, 16, 50, 20, 1, 0.1,
                     torch.zeros(1, dtype=torch.uint8).expand(1 << 27))
    for bad in ((-1, 4, 4, 2, 64), (1, 4, 5, 2, 64), (1, 4, 4, 2, 80)):
        with pytest.raises(xs.XsError):
            xs.attn_tree_workspace_size(*bad)
    assert xs.attn_tree_workspace_size(0, 4, 4, 2, 64) == 0


@pytest.mark.gpu
def test_tree_small_workspace_and_host_memory_are_refused():
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Trees([3], [20], 2, 1, 64, 16, 1)
    b.ws = b.ws[:4096]
    assert b.call(check=False) == xs.XS_ERR_WORKSPACE
    b = Trees([3], [20], 2, 1, 64, 16, 1)
    b.mask = b.mask.cpu()
    assert b.call(check=False) == xs.XS_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (from_dev(b.out) == 0xFFFF).all()
