"""Drafted trees of several items a key head (xs_attn_tree): side by side where all have as many, one after the other where
they differ, in very large batches, and in a captured call that goes from the one to the other."""
import numpy as np
import pytest

from test_tree import Trees, to_words
from xs_testlib import from_dev


def lanes_of(b):
    """The lanes of the last call, from its cut items' records at the workspace's end (SpanPieces, 8 words: pieces first,
    lanes last); None where nothing was cut."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    torch.cuda.synchronize()
    rec = b.ws.view(torch.int32)[-8 * sms:].view(sms, 8)
    lanes = rec[rec[:, 0] > 1][:, 7].unique().tolist()
    assert len(lanes) <= 1
    return lanes[0] if lanes else None


CASES = [  # q_len, kv_len, H, Hk, D, page, lanes
    ([70] * 5, [700, 1500, 70, 71, 5000], 4, 1, 64, 16, 2),            # 64 tokens an item: two items each
    ([65, 128, 100], [900, 128, 4000], 8, 2, 128, 64, 2),
    ([160, 130], [2160, 700], 4, 1, 96, 32, 3),
    ([64, 0, 50], [3000, 9, 2000], 16, 2, 128, 64, 2),                  # a sequence without new tokens counts for nothing
    ([64, 10, 96], [2064, 900, 1500], 16, 2, 128, 32, 1),              # unlike: two, one and three items
    ([33, 32, 32], [1033, 500, 2000], 16, 2, 64, 16, 1),               # all but one of one item
    ([128, 129, 120], [1128, 700, 130], 8, 1, 96, 128, 1),             # four items and five
    ([160] * 3, [1200, 160, 161], 8, 1, 64, 16, 1),                     # five items each
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_lanes_follow_the_batch(case):
    q_len, kv_len, H, Hk, D, page, lanes = CASES[case]
    b = Trees(q_len, kv_len, H, Hk, D, page, 8, spare=1, seed=case)
    assert b.T > b.N * 2 * (128 // (H // Hk))  # more than an item a sequence on average: what the host looks at
    b.ws.fill_(255)
    b.call()
    b.verify(what=str(CASES[case]))
    got = lanes_of(b)
    assert got == lanes, got
    first = from_dev(b.out).copy()
    b.out.fill_(-1)
    b.call()
    b.verify(what="again")
    assert np.array_equal(first, from_dev(b.out))


@pytest.mark.gpu
@pytest.mark.parametrize("N", (1024, 1025, 1100))
def test_lanes_of_very_many_trees(N):
    """Trees alike, in as many sequences as the lanes are looked for, and in more."""
    rng = np.random.default_rng(N)
    q_len = [int(x) for x in rng.integers(17, 25, N)]  # 16 tokens an item: two items each
    b = Trees(q_len, [int(q + x) for q, x in zip(q_len, rng.integers(0, 200, N))], 16, 1, 64, 16, 1, seed=N)
    b.ws.fill_(255)
    b.call()
    b.verify()
    assert lanes_of(b) in (None, 2 if N <= 1024 else 1)


@pytest.mark.gpu
def test_lanes_in_a_captured_call():
    """The number of lanes is found on the device: a captured call goes from trees alike to unlike ones and back."""
    import torch
    b = Trees([70, 70, 70], [1000, 500, 300], 4, 1, 64, 16, 8, seed=3)
    b.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call()
    rng = np.random.default_rng(5)
    for q_len, lanes in (([70, 70, 70], 2), ([20, 130, 60], 1), ([65, 65, 80], 2), ([210, 0, 0], 4), ([1, 1, 190], 1), ([0, 100, 110], 2),
                         ([70, 70, 70], 2)):
        b.q_len = q_len
        b.q_start.copy_(torch.tensor(np.concatenate(([0], np.cumsum(q_len))), dtype=torch.int32))
        b.bits = [rng.random((n, 256)) < 0.4 for n in q_len]
        b.mask[:sum(q_len)] = torch.from_numpy(np.concatenate([to_words(x, 8) for x in b.bits if len(x)])).cuda()
        b.out.fill_(-1)
        g.replay()
        b.verify(what=f"{q_len}")
        assert lanes_of(b) in (None, lanes), q_len
