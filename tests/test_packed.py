"""Attention over whole prompts packed one after the other (xs_attn_packed), against 64 bits; refusals."""
import numpy as np
import pytest

from span_testlib import attend, bf16, check, seen_mask, values
from xs_testlib import from_dev, guarded, to_dev

NAN = 0x7FC1


class Prompts:
    """Packed sequences; rows of none hold NaN, as do the gaps between rows that lie apart."""

    def __init__(self, lens, H, Hk, D, spare=0, seed=0, fused=False, before=0, sigma=1.0):
        import torch
        import comm_comp_fusion_gb300 as xs
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.Hk, self.D, self.before = lens, H, Hk, D, before
        self.N, self.T = len(lens), before + sum(lens) + spare
        real = slice(before, before + sum(lens))
        self.val, bits = {}, {}
        for name, h in (("q", H), ("k", Hk), ("v", Hk)):
            b, x = bf16(rng, (self.T, h, D), sigma if name != "v" else 1.0)
            bits[name] = np.full_like(b, NAN)
            bits[name][real] = b[real]
            self.val[name] = x
        if fused:
            row = to_dev(np.concatenate([bits["q"], bits["k"], np.full((self.T, 1, D), NAN, np.uint16), bits["v"]], 1))
            self.q, self.k, self.v = row[:, :H], row[:, H:H + Hk], row[:, H + Hk + 1:]
        else:
            self.q, self.k, self.v = (to_dev(bits[n]) for n in "qkv")
        start = before + np.concatenate(([0], np.cumsum(lens)))
        self.q_start = torch.tensor(start, dtype=torch.int32, device="cuda")
        self.out = guarded(self.T * H * D)
        self.ws = guarded(xs.attn_packed_workspace_size(self.N, self.T, H, Hk, D), torch.uint8)

    def call(self, left=-1, right=0, sinks=0, **kw):
        import comm_comp_fusion_gb300 as xs
        return xs.attn_packed(self.q, self.k, self.v, self.q_start, self.out, self.N, self.T, self.H, self.Hk, self.D,
                              self.D ** -0.5, left, right, sinks, self.ws, **kw)

    def verify(self, left=-1, right=0, sinks=0, what=""):
        import torch
        import comm_comp_fusion_gb300 as xs
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        got = from_dev(self.out).reshape(self.T, self.H, self.D)
        G, t = self.H // self.Hk, self.before
        assert (got[:t] == 0xFFFF).all()
        for n, m in enumerate(self.lens):
            seen, r = seen_mask(np.arange(m), m, left, right, sinks), slice(t, t + m)
            for h in range(self.H) if self.H * m < 4000 else sorted({0, self.H // 3, self.H - 1}):
                ref, bound = attend(self.val["q"][r, h], self.val["k"][r, h // G], self.val["v"][r, h // G], seen, self.D ** -0.5)
                check(got[r, h], ref, bound, f"{what} sequence {n} head {h}")
                assert (got[r, h][~seen.any(-1)] == 0).all()
            t += m
        assert (got[t:] == 0xFFFF).all(), "rows of no sequence were written"


CASES = [  # lengths, H, Hk, D, spare, one projection, (left, right, sinks)
    ([1], 1, 1, 64, 0, False, (-1, 0, 0)),
    ([1, 1, 1], 8, 2, 128, 5, True, (-1, 0, 0)),
    ([17, 300, 128, 129], 8, 8, 64, 0, False, (-1, 0, 0)),
    ([127, 0, 1, 256, 257], 4, 2, 128, 3, True, (-1, 0, 0)),
    ([500, 3, 1000], 6, 2, 96, 0, True, (-1, 0, 0)),              # three heads a key head
    ([33, 70, 400], 7, 1, 64, 1, False, (-1, 0, 0)),              # seven heads a key head: 126 rows of a tile
    ([250, 90], 128, 1, 64, 0, False, (-1, 0, 0)),                # 128 heads a key head: a token a tile
    ([900, 100], 32, 8, 128, 2, True, (-1, 0, 0)),
    ([400, 60, 130], 4, 4, 128, 0, False, (-1, -1, 0)),           # everything
    ([400, 60, 130], 4, 2, 96, 0, True, (-1, 40, 0)),
    ([1000, 129], 4, 2, 128, 9, False, (255, 0, 4)),
    ([1000, 129], 4, 1, 64, 0, True, (100, 37, 0)),
    ([800, 300, 1], 5, 1, 128, 0, False, (130, 0, 140)),
    ([50, 20], 4, 4, 64, 0, False, (0, 0, 0)),                    # itself alone
    ([7] * 90, 4, 2, 64, 2, False, (-1, 0, 0)),                   # more sequences than a warp's lanes
    ([1100, 1000, 900, 1200], 40, 40, 64, 0, False, (-1, 0, 0)),
    ([2100], 16, 16, 128, 0, True, (-1, 0, 0)),
    ([1500, 700], 24, 24, 64, 0, False, (300, 0, 0)),
    (list(range(1, 200, 3)), 6, 6, 96, 4, False, (-1, 0, 0)),
    ([9, 0, 12] * 20, 3, 1, 64, 0, True, (-1, 0, 0)),             # whole items of more sequences than a warp's lanes
    ([1024], 4, 1, 128, 0, False, (-1, 0, 0)),                    # the longest call of whole items, and one more token
    ([1000, 25], 4, 1, 128, 0, True, (-1, 0, 0)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_packed_matches_64_bits(case):
    lens, H, Hk, D, spare, fused, span = CASES[case]
    b = Prompts(lens, H, Hk, D, spare, case, fused)
    b.call(*span)
    b.verify(*span, what=str(CASES[case][1:]))
    first = from_dev(b.out).copy()
    b.out.fill_(-1)
    b.ws.fill_(255)
    b.call(*span)
    b.verify(*span, what="again, workspace of ones")
    assert np.array_equal(first, from_dev(b.out))


@pytest.mark.gpu
@pytest.mark.parametrize("D", (64, 96, 128))
@pytest.mark.parametrize("H,Hk", ((2, 2), (4, 1), (6, 2), (32, 2)))
def test_packed_lengths_around_tiles(D, H, Hk):
    """Lengths around multiples of the tiles of keys and of tokens, each next to a sequence of large values."""
    G = H // Hk
    lens = sorted({1, 2, 127, 128, 129, 128 // G, 128 // G + 1, 256 // G - 1, 256 // G, 256 // G + 1, 255, 256, 257, 385})
    b = Prompts(lens, H, Hk, D, spare=1, seed=D + H, fused=True)
    for span in ((-1, 0, 0), (-1, -1, 0), (60, 5, 3)):
        b.out.fill_(-1)
        b.call(*span)
        b.verify(*span, what=f"{span}")


@pytest.mark.gpu
def test_packed_sequences_do_not_touch():
    """One sequence of infinities and NaN between two others, and rows of none before and behind: the others' outputs
    are those of a call without it."""
    import torch
    for lens, H, Hk, D in (([300, 200, 129], 4, 2, 64), ([1, 5, 90], 8, 1, 128), ([513, 2, 700], 4, 4, 96)):
        b = Prompts(lens, H, Hk, D, spare=40, before=3, seed=2)
        a, e = 3 + lens[0], 3 + lens[0] + lens[1]
        for x in (b.q, b.k, b.v):
            x.view(b.T, -1)[a:e] = torch.tensor([0x7F80, NAN, -128], dtype=torch.int16, device="cuda").repeat(x.numel() // b.T)[
                :x.numel() // b.T]
        b.call()
        torch.cuda.synchronize()
        got = from_dev(b.out).reshape(b.T, H, D).copy()
        for n, (t, m) in enumerate(((3, lens[0]), (e, lens[2]))):
            for h in range(H):
                r = slice(t, t + m)
                ref, bound = attend(b.val["q"][r, h], b.val["k"][r, h // (H // Hk)], b.val["v"][r, h // (H // Hk)],
                                    seen_mask(np.arange(m), m, -1, 0, 0), D ** -0.5)
                check(got[r, h], ref, bound, f"sequence {n} head {h}")
        assert (got[:3] == 0xFFFF).all() and (got[e + lens[2]:] == 0xFFFF).all()


@pytest.mark.gpu
def test_packed_spoiled_rows_of_q_stay_alone():
    import torch
    b = Prompts([300, 40], 4, 2, 128, seed=3)
    bad = {(0, 0): NAN, (150, 3): 0x7F80, (339, 1): 0xFF80}
    for (t, h), x in bad.items():
        b.q.view(b.T, 4, 128)[t, h, ::7] = int(np.uint16(x).view(np.int16))
    b.call()
    torch.cuda.synchronize()
    got, t = from_dev(b.out).reshape(b.T, 4, 128), 0
    for m in b.lens:
        for h in range(4):
            ok = [i for i in range(m) if (t + i, h) not in bad]
            ref, bound = attend(b.val["q"][t:t + m, h][ok], b.val["k"][t:t + m, h // 2], b.val["v"][t:t + m, h // 2],
                                seen_mask(np.arange(m)[ok], m, -1, 0, 0), 128 ** -0.5)
            check(got[t:t + m, h][ok], ref, bound, f"head {h}")
        t += m


@pytest.mark.gpu
@pytest.mark.parametrize("sigma", (4.0, 0.0))
def test_packed_peaked_and_equal_scores(sigma):
    b = Prompts([700, 129, 40], 8, 2, 128, seed=3, sigma=sigma)
    b.call()
    b.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("N,H", ((1000, 2), (65536, 1)))
def test_packed_very_many_sequences(N, H):
    """Thousands of short sequences, empty ones among them."""
    import torch
    import comm_comp_fusion_gb300 as xs
    D = 64
    gen = torch.Generator(device="cuda").manual_seed(N)
    lens = torch.randint(0, 5, (N,), generator=gen, device="cuda")
    start = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), lens.cumsum(0)))
    T = int(start[-1]) + 3
    q, k, v = (torch.randn((T, H, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    out = guarded(T * H * D)
    ws = guarded(xs.attn_packed_workspace_size(N, T, H, H, D), torch.uint8)
    xs.attn_packed(q, k, v, start.to(torch.int32), out, N, T, H, H, D, 0.125, workspace=ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got = values(from_dev(out)).reshape(T, H, D)[:-3]
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), lens)
    t = torch.arange(T - 3, device="cuda")
    at = t.view(-1, 1) - torch.arange(5, device="cuda")  # a token and the four before it
    ok = at >= start[seq].view(-1, 1)
    kk, vv = (x[at.clamp(min=0)].double() for x in (k, v))
    s = torch.einsum("thd,tjhd->thj", q[:-3].double(), kk) * 0.125
    w = s.masked_fill(~ok.unsqueeze(1), -np.inf).softmax(-1)
    ref, a = (torch.einsum("thj,tjhd->thd", w, x).cpu().numpy() for x in (vv, vv.abs()))
    # the bound of span_testlib.attend; here scale sum |q k| is below 2^5, so the scores' share 2 delta is below 2^-12
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * a + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("span", ((-1, 0, 0), (1500, 0, 100)))
def test_packed_long_prompts_sampled(span):
    """Long prompts: one row of every 301 against 64 bits."""
    import torch
    b = Prompts([9001, 5000], 8, 2, 128, seed=15, fused=True)
    b.call(*span)
    torch.cuda.synchronize()
    got, t = from_dev(b.out).reshape(b.T, 8, 128), 0
    for m in b.lens:
        rows = np.arange(m - 1, 0, -301)
        for h in range(0, 8, 3):
            ref, bound = attend(b.val["q"][t + rows, h], b.val["k"][t:t + m, h // 4], b.val["v"][t:t + m, h // 4],
                                seen_mask(rows, m, *span), 128 ** -0.5)
            check(got[t + rows, h], ref, bound, f"h={h}")
        t += m


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,Hk,D,span", (([2 ** 18 + 4000, 700], 2, 1, 64, (-1, 0, 0)), ([300, 2 ** 18 + 129], 1, 1, 128, (-1, -1, 0)),
                                              ([2 ** 18 + 70000], 3, 1, 96, (2 ** 18 + 1000, 0, 200))))
def test_packed_very_long_prompt(lens, H, Hk, D, span):
    """Prompts of more than 2^18 tokens: sums in tensor memory truncate, so they are taken in stretches. Values around 1,
    where that shows. The bound: that of span_testlib.attend, and 2^14 additions of a stretch that truncate by 2^-23 at
    most."""
    import torch
    import comm_comp_fusion_gb300 as xs
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    q, k, v = rand(T, H, D).bfloat16(), rand(T, Hk, D).bfloat16(), (1 + 0.25 * rand(T, Hk, D)).bfloat16()
    start = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    out = guarded(T * H * D)
    ws = guarded(xs.attn_packed_workspace_size(len(lens), T, H, Hk, D), torch.uint8, 0xFF)
    xs.attn_packed(q, k, v, start, out, len(lens), T, H, Hk, D, D ** -0.5, *span, workspace=ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got, t = from_dev(out).reshape(T, H, D), 0
    for m in lens:
        rows = torch.cat((torch.arange(m - 1, 0, -m // 11, device="cuda"), torch.tensor([0, 1, m - 2], device="cuda")))
        j = torch.arange(m, device="cuda").view(1, -1)
        i = rows.view(-1, 1)
        seen = torch.ones((len(rows), m), dtype=torch.bool, device="cuda")
        if span[1] >= 0:
            seen &= j <= i + span[1]
        if span[0] >= 0:
            seen &= (j >= i - span[0]) | (j < span[2])
        for h in range(H):
            kd, vd, qd = (x[t:t + m, g].double() for x, g in ((k, h * Hk // H), (v, h * Hk // H), (q, h)))
            qd = qd[rows]
            w = (qd @ kd.T * D ** -0.5).masked_fill(~seen, -np.inf).softmax(-1)
            ref, a = w @ vd, w @ vd.abs()
            delta = 2.0 ** -18 * (qd.abs() @ kd.abs().T * D ** -0.5).amax(-1, keepdim=True)
            bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * delta + 2.0 ** -9) * a
            check(got[t + rows.cpu().numpy(), h], ref.cpu().numpy(), bound.cpu().numpy(), f"head {h}")
        t += m


@pytest.mark.gpu
def test_packed_graphs_and_streams():
    """A captured call follows starts that change between replays, two of them in one workspace; two on two streams."""
    import torch
    a, c = Prompts([300, 50, 200], 4, 2, 128, seed=7, spare=30), Prompts([600, 5], 4, 4, 64, seed=8, fused=True)
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
    for lens in ([300, 50, 200], [1, 549, 0], [128, 129, 255]):
        a.lens = lens
        a.q_start.copy_(torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32))
        for x, g in zip((a, c), graphs):
            x.out.fill_(-1)
            g.replay()
            x.verify()


@pytest.mark.gpu
def test_packed_ignores_bad_starts():
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Prompts([30, 40, 60], 4, 2, 64, spare=2, seed=1)
    for bad in ([500, 600, 10 ** 9, 2 ** 31 - 1], [-7, -3, -1, 0], [90, 50, 20, 3]):
        b.q_start.copy_(torch.tensor(bad, dtype=torch.int32))
        b.call()
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        assert (from_dev(b.out) == 0xFFFF).all()
    b.q_start.copy_(torch.tensor([-9, 30, 70, 10 ** 6], dtype=torch.int32))  # cut to the packed rows
    b.lens = [30, 40, 62]
    for n in "qkv":
        getattr(b, n).view(b.T, -1)[130:] = to_dev(np.zeros(2, np.uint16)).view(2, 1)
        b.val[n][130:] = 0
    b.call()
    b.verify()


@pytest.mark.gpu
def test_packed_rows_past_32_bits():
    """Rows of a projection more than 2^31 elements from its first."""
    import torch
    b = Prompts([3, 300], 2, 1, 64, seed=6)
    stride = 2 ** 23
    wide = torch.zeros((b.T - 1) * stride + 256, dtype=torch.int16, device="cuda")
    row = torch.as_strided(wide, (b.T, 256), (stride, 1))
    row[:, :128], row[:, 128:192], row[:, 192:] = b.q.view(b.T, -1), b.k.view(b.T, -1), b.v.view(b.T, -1)
    b.q, b.k, b.v = row[:, :128], row[:, 128:192], row[:, 192:]
    b.call()
    b.verify()


# ------------------------------------------------------------------ refusals

A = [0x10000000 * (i + 1) for i in range(12)]


def test_packed_refusals():
    import __graft_entry__
    __graft_entry__.build()
    import ctypes
    import torch
    import comm_comp_fusion_gb300 as xs

    def call(**kw):
        a = dict(q=A[0], k=A[1], v=A[2], q_start=A[3], out=A[4], N=2, T=10, H=8, Hk=2, D=128, scale=0.1, workspace=A[5],
                 workspace_bytes=1 << 27, check=False)
        a.update(kw)
        return xs.attn_packed(**a)

    for name in ("q", "k", "v", "q_start", "out"):
        assert call(**{name: None}) == xs.XS_ERR_NULL
    for kw in (dict(N=-1), dict(T=-1), dict(N=65537), dict(T=(1 << 29) + 1), dict(H=7), dict(H=0), dict(Hk=0), dict(T=1 << 28),
               dict(scale=-1.0), dict(scale=float("inf")), dict(left=-2), dict(right=-3), dict(sinks=-1)):
        assert call(**kw) == xs.XS_ERR_SHAPE, kw
    for kw in (dict(D=256), dict(D=32), dict(H=258)):
        assert call(**kw) == xs.XS_ERR_UNSUPPORTED, kw
    for kw in (dict(q=A[0] + 8), dict(k=A[1] + 2), dict(v=A[2] + 4), dict(out=A[4] + 8), dict(q_start=A[3] + 2)):
        assert call(**kw) == xs.XS_ERR_ALIGN, kw
    for name in ("q", "k", "v", "q_start"):
        assert call(**{name: A[4] + 16}) == xs.XS_ERR_ALIAS, name
    assert call(workspace=None, workspace_bytes=0) == xs.XS_ERR_NULL
    for kw in (dict(workspace=None, workspace_bytes=8), dict(workspace=A[5] + 128), dict(workspace=A[4]), dict(workspace=A[0])):
        assert call(**kw) == xs.XS_ERR_WORKSPACE, kw
    assert call(N=0) == xs.XS_OK and call(T=0) == xs.XS_OK and call(T=0, workspace=None, workspace_bytes=0) == xs.XS_OK

    def raw(strides):
        return xs.lib.xs_attn_packed(A[0], A[1], A[2], *strides, A[3], A[4], 2, 10, 8, 2, 128, 0.1, -1, 0, 0, A[5], 1 << 27, None)
    for strides in ((1016, 0, 0), (1028, 0, 0), (0, 255, 0), (0, 0, -256), (0, 1 << 31, 0)):
        assert raw(strides) == xs.XS_ERR_SHAPE, strides
    n = ctypes.c_size_t(7)
    for T, H, Hk, D in ((4, 258, 2, 64), (4, 7, 2, 64), (4, 0, 2, 64), (1 << 27, 16, 16, 64), (4, 4, 2, 80)):
        assert xs.lib.xs_attn_packed_workspace_size(2, T, H, Hk, D, ctypes.byref(n)) == call(T=T, H=H, Hk=Hk, D=D) != xs.XS_OK
    assert n.value == 7 and xs.attn_packed_workspace_size(0, 4, 4, 2, 64) == 0
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    for kw in (dict(q=x.float()), dict(q=x[:3]), dict(k=x[:, ::2, ::2]), dict(v=x.expand(2, 4, 2, 64)[:, :, :1])):
        a = dict(q=x, k=x, v=x)
        a.update(kw)
        with pytest.raises(ValueError):
            xs.attn_packed(a["q"], a["k"], a["v"], i, x, 1, 4, 2, 2, 64, 0.1)
    with pytest.raises(ValueError, match="int32"):
        xs.attn_packed(x, x, x, i.long(), x, 1, 4, 2, 2, 64, 0.1)
    with pytest.raises(ValueError, match="workspace"):
        xs.attn_packed(A[0], A[1], A[2], A[3], A[4], 2, 10, 8, 2, 128, 0.1, workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 27))


@pytest.mark.gpu
def test_packed_small_workspace_and_host_memory_are_refused():
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Prompts([20], 2, 1, 64)
    b.ws = b.ws[:4096]
    assert b.call(check=False) == xs.XS_ERR_WORKSPACE
    b = Prompts([20], 2, 1, 64)
    b.q_start = b.q_start.cpu()
    assert b.call(check=False) == xs.XS_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (from_dev(b.out) == 0xFFFF).all()
