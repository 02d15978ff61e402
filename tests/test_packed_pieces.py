"""Packed prompts of more than 1024 tokens (xs_attn_packed): items cut in pieces that meet in the workspace, in captured
calls, in a workspace that two of them share, on two streams, with peaked scores and with rows of q that are not finite.
(Shorter calls of few items take whole items and leave the workspace alone.)"""
import numpy as np
import pytest

from span_testlib import attend, check, seen_mask
from test_packed import NAN, Prompts
from xs_testlib import from_dev


def cut_items(b):
    """How many items the last call cut: each CTA's record at the workspace's end says in how many pieces the item lies
    whose first piece it has (SpanPieces, 8 words, the first of them)."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    torch.cuda.synchronize()
    return int((b.ws.view(torch.int32)[-8 * sms:].view(sms, 8)[:, 0] > 1).sum())


def restart(b, lens):
    """Other prompts in the same rows."""
    import torch
    b.lens = lens
    b.q_start.copy_(torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32))




@pytest.mark.gpu
def test_pieces_are_met_where_the_tests_below_want_them():
    """On either side of the limit: 1024 tokens leave the workspace as it was, 1025 cut items."""
    for lens, cut in (([1000, 24], False), ([1000, 25], True)):
        b = Prompts(lens, 4, 2, 128, seed=4)
        b.ws.fill_(0)
        b.call()
        b.verify()
        assert (cut_items(b) > 0) == cut == bool((b.ws != 0).any())


@pytest.mark.gpu
def test_packed_pieces_in_graphs_and_on_streams():
    """Captured calls of cut items follow starts that move the cuts; two of them, and short ones between, share a
    workspace; two at a time on two streams with one each."""
    import torch
    a, c = Prompts([900, 150, 600, 0, 0, 0, 0, 0], 4, 2, 128, seed=7, spare=30), Prompts([1500, 5], 4, 4, 64, seed=8, fused=True)
    short = Prompts([300, 50, 200], 4, 2, 128, seed=9, spare=3)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, s in zip((a, c), streams):
            x.call(stream=s)
    torch.cuda.synchronize()
    a.verify(what="two streams")
    c.verify(what="two streams")
    assert cut_items(a) and cut_items(c)
    c.ws = short.ws = a.ws
    a.ws.fill_(255)
    graphs = []
    for x in (a, c, short):
        x.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.call()
        graphs.append(g)
    for lens in ([900, 150, 600, 0, 0, 0, 0, 0], [0, 0, 1650, 0, 0, 0, 0, 0], [206] * 8, [1, 2, 3, 1500, 0, 129, 7, 8], [0] * 8,
                 [1, 0, 0, 0, 0, 0, 0, 1649]):
        restart(a, lens)
        for x in (a, c, short):
            x.out.fill_(-1)
        for g in graphs:  # nothing between them but the stream's order
            g.replay()
        for x in (a, c, short):
            x.verify(what=f"replayed {lens}")


@pytest.mark.gpu
@pytest.mark.parametrize("sigma", (4.0, 0.0))
@pytest.mark.parametrize("span", ((-1, 0, 0), (-1, -1, 0), (400, 60, 9)))
def test_packed_pieces_of_peaked_and_equal_scores(sigma, span):
    b = Prompts([1300, 129, 40], 8, 2, 128, seed=3, sigma=sigma)
    b.ws.fill_(255)
    b.call(*span)
    b.verify(*span)
    assert cut_items(b)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,D", ((4, 2, 128), (4, 4, 96), (8, 1, 64)))
def test_packed_pieces_next_to_spoiled_rows_of_q(H, Hk, D):
    """A row of q that is not finite spoils its own output alone, where it lies in a cut item too."""
    import torch
    b = Prompts([1200, 40, 300], H, Hk, D, seed=3)
    bad = {(0, 0): NAN, (600, 3): 0x7F80, (1199, 1): 0xFF80, (1200, 2): NAN, (1539, 0): 0x7F80}
    for (t, h), x in bad.items():
        b.q.view(b.T, H, D)[t, h, ::7] = int(np.uint16(x).view(np.int16))
    b.call()
    assert cut_items(b)
    got, t = from_dev(b.out).reshape(b.T, H, D), 0
    for m in b.lens:
        for h in range(H):
            ok = [i for i in range(m) if (t + i, h) not in bad]
            ref, bound = attend(b.val["q"][t:t + m, h][ok], b.val["k"][t:t + m, h * Hk // H], b.val["v"][t:t + m, h * Hk // H],
                                seen_mask(np.arange(m)[ok], m, -1, 0, 0), D ** -0.5)
            check(got[t:t + m, h][ok], ref, bound, f"head {h}")
        t += m
