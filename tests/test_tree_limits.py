"""Attention of drafted trees (xs_attn_tree) with metadata that names nothing, by what it leaves in its output, and with
triangular masks next to xs_attn_paged."""
import numpy as np
import pytest

from span_testlib import attend, values
from test_paged import Batch
from test_tree import Trees, to_words
from xs_testlib import from_dev, guarded

BIG = 2 ** 31 - 1


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,kv_len,H,Hk", (([2, 3, 1], [40, 60, 70], 4, 2),        # few rows
                                               ([2, 3, 40], [40, 60, 70], 4, 2),       # one item a sequence
                                               ([70, 70, 70], [400, 70, 900], 4, 1),   # two side by side
                                               ([70, 20, 140], [400, 70, 900], 4, 1)))
def test_tree_bad_metadata_leaves_other_rows(q_len, kv_len, H, Hk):
    """Pools of zeros, so that every row of a sequence gets zeros whatever its keys; all other rows keep what they held."""
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Trees(q_len, kv_len, H, Hk, 64, 16, 2, spare=2, seed=1)
    b.kp.fill_(0)
    b.vp.fill_(0)
    good, T = (b.table, b.q_start, b.kv_len), b.T

    def run(what, start=None, **kw):
        b.table, b.q_start, b.kv_len = (x.clone() for x in good)
        for name, x in kw.items():
            getattr(b, name).copy_(torch.as_tensor(x, dtype=torch.int32).expand_as(getattr(b, name)))
        if start is not None:
            b.q_start.copy_(torch.tensor(start, dtype=torch.int32))
        b.out.fill_(-1)
        b.ws.fill_(255)
        b.call()
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        got = from_dev(b.out).reshape(T, H, 64)
        own = np.zeros(T, bool)
        for s, e in zip(b.q_start.tolist()[:-1], b.q_start.tolist()[1:]):
            own[min(max(s, 0), T):max(min(max(e, 0), T), min(max(s, 0), T))] = True
        assert (got[own] == 0).all(), f"{what}: rows of a sequence"
        assert (got[~own] == 0xFFFF).all(), f"{what}: rows of none"
        return int(own.sum())

    real = sum(q_len)
    assert run("as it was") == real
    assert run("pages past the pool", table=BIG) == real
    assert run("pages before the pool", table=-1) == real
    assert run("lengths past the table and below zero", kv_len=[BIG, -5, 10 ** 6]) == real
    assert run("no keys", kv_len=0) == real
    assert run("starts past the rows", [500, 600, 10 ** 9, BIG]) == 0
    assert run("starts before the rows", [-7, -3, -1, 0]) == 0
    assert run("starts that fall", [T, 4, 4, 1]) == 0
    assert run("the first sequence up to the last row", [T - 1, 10 ** 6, 10 ** 9, BIG]) == 1


TRIANGLES = [  # q_len, kv_len, H, Hk, D, page
    ([1] * 4, [700, 90, 1500, 64], 8, 2, 128, 16),        # few rows
    ([3, 4], [1500, 600], 8, 2, 64, 16),
    ([16, 1], [400, 33], 16, 2, 64, 32),                   # a tile of 128 rows, and of 8
    ([9, 30], [300, 900], 4, 2, 96, 64),
    ([40, 128], [2500, 128], 2, 2, 128, 128),              # no context
    ([10, 10], [1000, 500], 4, 2, 128, 32),                # 20 rows: xs_attn_paged takes tiles of 32
    ([9, 256], [300, 900], 4, 2, 96, 64),                  # as many tokens as there are bits; several items
    ([100, 256, 3], [1100, 256, 50], 8, 2, 64, 16),
    ([200], [5000], 1, 1, 128, 16),                        # two tiles, which xs_attn_paged ends at different keys
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(TRIANGLES)))
def test_tree_of_a_triangle_next_to_paged(case):
    """Masks of each token and all before it are causal attention, which xs_attn_paged computes with a schedule and edges of
    its own. Each output is within its row's bound of the 64-bit one, so the two differ by twice that at most."""
    import torch
    q_len, kv_len, H, Hk, D, page = TRIANGLES[case]
    b = Trees(q_len, kv_len, H, Hk, D, page, 8, seed=case)
    b.bits = [np.tril(np.ones((n, n), bool)) for n in q_len]
    b.mask = torch.from_numpy(np.concatenate([to_words(x, 8) for x in b.bits])).cuda()
    b.call()
    b.verify()
    other = guarded(b.T * H * D)
    Batch.call(b, out=other)
    torch.cuda.synchronize()
    got, want = (values(from_dev(x)).reshape(b.T, H, D) for x in (b.out, other))
    t = 0
    for n, m in enumerate(q_len):
        for h in range(H):
            g = h // (H // Hk)
            bound = attend(b.q[t:t + m, h], b.k[n][:, g], b.v[n][:, g], b.seen(n), D ** -0.5)[1]
            assert (np.abs(got - want)[t:t + m, h] <= 2 * bound).all(), (n, h)
        t += m
