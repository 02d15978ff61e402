"""Attention through a sliding window with sinks (xs_attn_window, xs_attn_window_a2a): against 64 bits, the schedules
against each other, graphs and streams, and refusals."""
import numpy as np
import pytest

from span_testlib import attend, bf16, check, head_to_tokens, seen_mask, seq_to_tokens, tokens_to_head, values
from xs_testlib import from_dev, guarded, to_dev

# B, S, H, D, P, left, right, sinks, sigma of q and k
CASES = [
    (1, 1, 1, 64, 1, 0, 0, 0, 1.0),            # one token sees itself
    (1, 5, 2, 128, 1, 2, 0, 1, 1.0),
    (2, 100, 4, 96, 2, 30, 0, 4, 1.0),         # below one tile
    (1, 128, 2, 64, 1, 127, 0, 0, 1.0),
    (1, 129, 3, 128, 3, 0, 0, 0, 1.0),         # only the diagonal: out = v
    (1, 256, 2, 128, 2, 0, 0, 200, 1.0),       # sinks past the first tile
    (1, 384, 2, 64, 1, 128, 0, 0, 1.0),        # odd tile count
    (1, 1000, 4, 64, 4, 255, 0, 4, 1.0),       # ragged
    (1, 1000, 4, 96, 2, 63, 63, 0, 1.0),       # two-sided
    (2, 777, 2, 128, 1, 300, 17, 130, 1.0),
    (1, 640, 2, 128, 2, 5, 500, 0, 1.0),       # mostly to the right
    (1, 900, 2, 128, 1, -1, 0, 0, 1.0),        # causal
    (1, 900, 2, 128, 1, -1, -1, 0, 1.0),       # everything
    (1, 900, 2, 64, 1, 40, -1, 7, 1.0),        # no right end
    (1, 1500, 2, 128, 1, 200, 0, 3, 4.0),      # peaked scores
    (1, 2176, 8, 128, 8, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1.0),
    (1, 1280, 40, 64, 4, 400, 0, 64, 1.0),     # more items than SMs
    (1, 2048, 48, 64, 2, 300, 0, 3, 1.0),      # several items a CTA: whole rounds, then half an item each
    (1, 2560, 31, 64, 1, 200, 100, 0, 1.0),    # whole rounds, a little more than one item each left
    (2, 1024, 76, 64, 4, 150, 0, 0, 1.0),      # whole rounds and nothing left (152 SMs)
    (1, 2304, 40, 64, 1, -1, 0, 0, 1.0),       # items of unlike lengths: no rounds
]


def run(case, q, k, v, scale, workspace=True, fill=None):
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D, P, left, right, sinks, _ = case
    n = B * S * H * D
    head, fused, serial = (guarded(n) for _ in range(3))
    ws = None
    if workspace:
        ws = guarded(xs.attn_window_workspace_size(B, S, H, D, P), torch.uint8, fill)
    xs.attn_window(q, k, v, head, B, S, H, D, P, scale, left, right, sinks, ws)
    xs.attn_window_a2a(q, k, v, fused, B, S, H, D, P, scale, left, right, sinks, ws)
    xs.a2a_permute(head, serial, B, S, H, D, P)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    f = from_dev(fused)
    assert np.array_equal(f, from_dev(serial))
    h = head_to_tokens(from_dev(head).reshape(P, B, S, H // P, D))
    assert np.array_equal(h, seq_to_tokens(f.reshape(P, B, S // P, H, D)))
    return h


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_window_matches_64_bits(case):
    B, S, H, D, P, left, right, sinks, sigma = case
    rng = np.random.default_rng(S * 7 + D)
    (qb, q), (kb, k) = bf16(rng, (B, S, H, D), sigma), bf16(rng, (B, S, H, D), sigma)
    vb, v = bf16(rng, (B, S, H, D))
    dev = [to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)]
    seen = seen_mask(np.arange(S), S, left, right, sinks)
    for ws, fill in ((True, None), (True, 0xFF), (False, None)):
        got = run(case, *dev, D ** -0.5, ws, fill)
        for b in range(B):
            for h in range(H) if S * H < 9000 else sorted({0, 1, H // 3, H // 2, 2 * H // 3, H - 2, H - 1}):
                ref, bound = attend(q[b, :, h], k[b, :, h], v[b, :, h], seen, D ** -0.5)
                check(got[b, :, h], ref, bound, f"{case} b={b} h={h} ws={ws}")
    if left == right == sinks == 0:
        assert np.array_equal(got, vb)


@pytest.mark.gpu
def test_window_rows_that_are_not_finite_stay_alone():
    """A row of q with NaN or an infinity spoils its own output alone."""
    B, S, H, D, P = 1, 1500, 3, 128, 1
    case = (B, S, H, D, P, 400, 30, 4, 1.0)
    rng = np.random.default_rng(8)
    (qb, q), (kb, k), (vb, v) = (bf16(rng, (B, S, H, D)) for _ in range(3))
    bad = {(0, 0): 0x7FC1, (700, 1): 0x7F80, (701, 2): 0xFF80, (1499, 2): 0x7FC1}
    for (t, h), x in bad.items():
        qb[0, t, h, 3::5] = x
    for ws in (True, False):
        got = run(case, *[to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)], D ** -0.5, ws)
        for h in range(H):
            ok = np.array([t for t in range(S) if (t, h) not in bad])
            ref, bound = attend(q[0, ok, h], k[0, :, h], v[0, :, h], seen_mask(ok, S, 400, 30, 4), D ** -0.5)
            check(got[0, ok, h], ref, bound, f"h={h} ws={ws}")


@pytest.mark.gpu
def test_window_rising_keys():
    """Scores that grow along the sequence: the running maximum moves in every tile, in the window and past the sinks."""
    B, S, H, D, P = 1, 1100, 2, 128, 1
    case = (B, S, H, D, P, 500, 0, 40, 1.0)
    rng = np.random.default_rng(2)
    q = np.abs(bf16(rng, (B, S, H, D))[1])
    k = np.abs(bf16(rng, (B, S, H, D))[1]) * np.linspace(0.0, 6.0, S).reshape(1, S, 1, 1)
    import torch
    t = lambda x: torch.from_numpy(np.asarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    qb, kb = t(q), t(k)
    vb, v = bf16(rng, (B, S, H, D))
    got = run(case, *[to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)], D ** -0.5)
    seen = seen_mask(np.arange(S), S, 500, 0, 40)
    for h in range(H):
        ref, bound = attend(values(qb)[0, :, h], values(kb)[0, :, h], v[0, :, h], seen, D ** -0.5)
        check(got[0, :, h], ref, bound, f"h={h}")


@pytest.mark.gpu
def test_window_falling_keys_after_far_first_tile():
    """Large scores only among keys that leave the window: what they set must not push later rows' weights to zero."""
    B, S, H, D, P = 1, 700, 1, 64, 1
    case = (B, S, H, D, P, 150, 0, 0, 1.0)
    rng = np.random.default_rng(4)
    (qb, q), (kb, k), (vb, v) = (bf16(rng, (B, S, H, D)) for _ in range(3))
    q = np.abs(q)
    k = k.copy()
    k[:, :130] = np.abs(k[:, :130]) * 8.0
    k[:, 130:] = -np.abs(k[:, 130:]) * 8.0     # scores of several hundred below the first tile's
    import torch
    t = lambda x: torch.from_numpy(np.asarray(x, np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    qb, kb = t(q), t(k)
    got = run(case, *[to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)], 1.0)
    ref, bound = attend(values(qb)[0, :, 0], values(kb)[0, :, 0], v[0, :, 0], seen_mask(np.arange(S), S, 150, 0, 0), 1.0)
    check(got[0, :, 0], ref, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("case", ((2, 4, 3, 96, 1, 726, 10, 4), (1, 68, 16, 128, 4, 35, 0, 200), (3, 257, 30, 64, 1, -1, 0, 0),
                                  (1, 1000, 30, 128, 5, 300, 300, 4), (2, 900, 19, 96, 1, 200, 40, 0), (1, 1, 152, 64, 1, 0, 0, 0)))
def test_window_small_calls_take_whole_items(case):
    """No more items than SMs, none much longer than the others' share: no item is cut, so the bits are those without a
    workspace, which are near 64 bits. (Three batches of 30 heads and two items are more than the SMs: some are cut.)"""
    import torch
    B, S, H, D, P, left, right, sinks = case
    rng = np.random.default_rng(S + 3 * D)
    (qb, q), (kb, k), (vb, v) = (bf16(rng, (B, S, H, D)) for _ in range(3))
    dev = [to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)]
    whole = run((*case, 1.0), *dev, D ** -0.5, False, None)
    got = run((*case, 1.0), *dev, D ** -0.5, True, 0xFF)
    if B * H * -(-S // 256) <= torch.cuda.get_device_properties(0).multi_processor_count:
        np.testing.assert_array_equal(got, whole)
    seen = seen_mask(np.arange(S), S, left, right, sinks)
    for h in range(0, H, max(1, H // 4)):
        ref, bound = attend(q[0, :, h], k[0, :, h], v[0, :, h], seen, D ** -0.5)
        for bits in (got, whole):
            check(bits[0, :, h], ref, bound, f"{case} h={h}")


@pytest.mark.gpu
@pytest.mark.parametrize("span", ((3000, 0, 70), (-1, 0, 0), (1500, 2500, 0)))
def test_window_long_sampled(span):
    """A long ragged sequence: items of many K/V tiles, one row of every query tile against 64 bits."""
    B, S, H, D, P = 1, 12040, 6, 128, 2
    rng = np.random.default_rng(77)
    (qb, q), (kb, k), (vb, v) = (bf16(rng, (B, S, H, D)) for _ in range(3))
    got = run((B, S, H, D, P, *span, 1.0), *[to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)], D ** -0.5)
    for h in range(H):
        rows = np.minimum(np.arange(0, S, 128) + rng.integers(0, 128, -(-S // 128)), S - 1)
        ref, bound = attend(q[0, rows, h], k[0, :, h], v[0, :, h], seen_mask(rows, S, *span), D ** -0.5)
        check(got[0, rows, h], ref, bound, f"{span} h={h}")


@pytest.mark.gpu
def test_window_unlimited_is_causal_and_full_attention():
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D, P = 1, 1152, 4, 128, 2
    rng = np.random.default_rng(6)
    qb, kb, vb = (bf16(rng, (P, B, S, H // P, D))[0] for _ in range(3))
    q, k, v = to_dev(qb), to_dev(kb), to_dev(vb)
    n = qb.size
    for right, call in ((0, xs.attn_causal), (-1, xs.attn)):
        a, b = guarded(n), guarded(n)
        xs.attn_window(q, k, v, a, B, S, H, D, P, D ** -0.5, -1, right)
        call(q, k, v, b, B, S, H, D, P, D ** -0.5)
        torch.cuda.synchronize()
        x, y = values(from_dev(a)), values(from_dev(b))
        # two roundings of one result: a step of 2^-7 apart at most, and each call's weights rounded by 2^-8
        assert (np.abs(x - y) <= 2.0 ** -7 * np.abs(y) + 2.0 ** -7).all()


@pytest.mark.gpu
def test_window_graphs_share_a_workspace():
    """Two captured calls that use one workspace in turn, replayed several times with changing inputs, among eager ones."""
    import torch
    import comm_comp_fusion_gb300 as xs
    D, scale = 128, 128 ** -0.5
    shapes = [(1, 1500, 6, 700, 0, 4), (2, 800, 2, 100, 100, 0)]
    size = max(xs.attn_window_workspace_size(B, S, H, D, 1) for B, S, H, *_ in shapes)
    ws = guarded(size, torch.uint8)
    rng = np.random.default_rng(8)
    jobs = []
    for B, S, H, left, right, sinks in shapes:
        q, k, v = (to_dev(bf16(rng, (1, B, S, H, D))[0]) for _ in range(3))
        out, want = guarded(q.numel()), guarded(q.numel())
        call = lambda o, q=q, k=k, v=v, B=B, S=S, H=H, w=(left, right, sinks): xs.attn_window(  # noqa: E731
            q, k, v, o, B, S, H, D, 1, scale, *w, ws)
        call(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        jobs.append((g, q, out, want, call))
    for turn in range(3):
        for g, q, out, want, call in jobs:
            q.copy_(to_dev(bf16(rng, tuple(q.shape))[0]))
            out.fill_(-1)
            g.replay()
            call(want)
            assert np.array_equal(from_dev(out), from_dev(want)), turn


@pytest.mark.gpu
def test_window_on_two_streams_at_once():
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D = 1, 2000, 8, 64
    rng = np.random.default_rng(12)
    q, k, v = (to_dev(bf16(rng, (1, B, S, H, D))[0]) for _ in range(3))
    size = xs.attn_window_workspace_size(B, S, H, D, 1)
    outs, wss, want = [guarded(q.numel()) for _ in range(2)], [guarded(size, torch.uint8) for _ in range(2)], guarded(q.numel())
    xs.attn_window(q, k, v, want, B, S, H, D, 1, 0.125, 300, 0, 4, wss[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(4):
        for s, o, w in zip(streams, outs, wss):
            xs.attn_window(q, k, v, o, B, S, H, D, 1, 0.125, 300, 0, 4, w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(from_dev(o), from_dev(want))


@pytest.mark.gpu
@pytest.mark.parametrize("case", ((21, 256, 32, 64, 1, -1, 0, 0), (23, 200, 16, 96, 1, -1, 0, 0), (13, 256, 40, 64, 2, -1, -1, 0),
                                  (1, 1280, 73, 64, 1, 0, 0, 0), (2, 256, 160, 64, 1, -1, -1, 0), (5, 300, 31, 128, 1, 70, 0, 0)))
def test_window_rest_of_fewer_steps_than_sms(case):
    """Whole rounds, then items of two or three steps whose steps are fewer than the CTAs (152 SMs): every head, with
    a workspace that holds NaN or finite leftovers of another call, which no result may depend on."""
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D, P, left, right, sinks = case
    rng = np.random.default_rng(S + B)
    (qb, q), (kb, k), (vb, v) = (bf16(rng, (B, S, H, D)) for _ in range(3))
    dev = [to_dev(tokens_to_head(x, P)) for x in (qb, kb, vb)]
    ws = guarded(xs.attn_window_workspace_size(B, S, H, D, P), torch.uint8)
    outs = []
    for fill in (0xFF, 0x3C):
        ws.fill_(fill)
        out = guarded(B * S * H * D)
        xs.attn_window(*dev, out, B, S, H, D, P, D ** -0.5, left, right, sinks, ws)
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        outs.append(head_to_tokens(from_dev(out).reshape(P, B, S, H // P, D)))
    seen = seen_mask(np.arange(S), S, left, right, sinks)
    for b in range(B):
        for h in range(H):
            ref, bound = attend(q[b, :, h], k[b, :, h], v[b, :, h], seen, D ** -0.5)
            check(outs[0][b, :, h], ref, bound, f"{case} b={b} h={h}")
    assert np.array_equal(outs[0], outs[1])


@pytest.mark.gpu
@pytest.mark.parametrize("S,H,span", ((2 ** 20 + 77, 1, (-1, 0, 0)), (1300001, 1, (290000, 0, 500)), (530000, 2, (-1, -1, 0))))
def test_window_of_very_many_keys(S, H, span):
    """Items of thousands of K/V tiles, whose sums are taken in stretches: values around 1, of which a single sum in tensor
    memory loses what its additions truncate (2^-23 at most each, 2^14 of them in a stretch: 2^-9 more than the bound of
    span_testlib.attend)."""
    import torch
    import comm_comp_fusion_gb300 as xs
    D = 64
    gen = torch.Generator(device="cuda").manual_seed(S)
    q, k, v = (torch.randn(1, 1, S, H, D, generator=gen, device="cuda") for _ in range(3))
    q, k, v = q.bfloat16(), k.bfloat16(), (1 + 0.25 * v).bfloat16()
    out = guarded(q.numel())
    ws = guarded(xs.attn_window_workspace_size(1, S, H, D, 1), torch.uint8, 0xFF)
    xs.attn_window(q, k, v, out, 1, S, H, D, 1, D ** -0.5, *span, ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got = from_dev(out).reshape(S, H, D)
    for i in (0, 255, S // 3, S // 2 + 1, S - 300, S - 1):
        lo = 0 if span[0] < 0 else max(0, i - span[0])
        hi = S if span[1] < 0 else i + 1
        at = torch.cat((torch.arange(min(span[2], lo)), torch.arange(lo, hi))).cuda()
        for h in range(H):
            qd, kd, vd = (x.double().cpu().numpy() for x in (q[0, 0, i:i + 1, h], k[0, 0, at, h], v[0, 0, at, h]))
            ref, bound = attend(qd, kd, vd, np.ones((1, len(at)), bool), D ** -0.5)
            check(got[i:i + 1, h], ref, bound + 2.0 ** -9 * np.abs(ref), f"row {i} head {h}")


@pytest.mark.gpu
def test_window_of_very_many_keys_scatters():
    """The same with the All-to-All, whole items and pieces: bit for bit the permuted one."""
    import torch
    import comm_comp_fusion_gb300 as xs
    S, H, D, P = 2 ** 18 + 2048, 2, 64, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(P, 1, S, H // P, D, generator=gen, device="cuda").bfloat16() for _ in range(3))
    ws = guarded(xs.attn_window_workspace_size(1, S, H, D, P), torch.uint8, 0xFF)
    head, fused, serial = (guarded(q.numel()) for _ in range(3))
    xs.attn_window(q, k, v, head, 1, S, H, D, P, D ** -0.5, -1, -1, 0, ws)
    xs.attn_window_a2a(q, k, v, fused, 1, S, H, D, P, D ** -0.5, -1, -1, 0, ws)
    xs.a2a_permute(head, serial, 1, S, H, D, P)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    assert torch.equal(fused, serial)
    got = head_to_tokens(from_dev(head).reshape(P, 1, S, H // P, D))
    for i in (0, 130000, S - 1):
        for h in range(H):
            x = [y[h, 0, :, 0].double().cpu().numpy() for y in (q, k, v)]
            ref, bound = attend(x[0][i:i + 1], x[1], x[2], np.ones((1, S), bool), D ** -0.5)
            check(got[0, i:i + 1, h], ref, bound, f"row {i} head {h}")


def test_window_without_workspace_takes_no_more_keys_than_it_can_add_up():
    import __graft_entry__
    __graft_entry__.build()
    import comm_comp_fusion_gb300 as xs

    def f(S, left, right, sinks, ws=None, nb=None):
        return xs.attn_window(Q, Q + (1 << 33), Q + (2 << 33), Q + (3 << 33), 1, S, 1, 64, 1, 0.1, left, right, sinks, ws, nb,
                              check=False)

    M = 1 << 20
    for S, *span in ((M + 1, -1, 0, 0), (1 << 24, -1, -1, 0), (2 * M, M, 0, 0), (3 * M, 100, 0, M), (1 << 24, 0, M, 0)):
        assert f(S, *span) == xs.XS_ERR_WORKSPACE and "2^20" in xs.last_error()
        assert f(S, *span, Q + (4 << 33), 1 << 28) != xs.XS_ERR_WORKSPACE or _gpu()
    for S, *span in ((M, -1, -1, 0), (1 << 24, 1000, 1000, 100000), (2 * M, M - 512, 0, 0)):
        assert f(S, *span) in (xs.XS_ERR_CUDA, xs.XS_ERR_UNSUPPORTED)   # no device, or addresses of nothing


def _gpu():
    import torch
    return torch.cuda.is_available()


Q, K, V, O, W = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000


def test_window_refusals():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs

    for fn in (xs.attn_window, xs.attn_window_a2a):
        def f(q=Q, k=K, v=V, o=O, B=1, S=256, H=8, D=64, P=4, scale=0.125, left=5, right=0, sinks=0, ws=None, nb=None):
            return fn(q, k, v, o, B, S, H, D, P, scale, left, right, sinks, ws, nb, check=False)

        assert f(q=0) == xs.XS_ERR_NULL and f(o=0) == xs.XS_ERR_NULL
        assert f(H=6) == xs.XS_ERR_SHAPE and f(S=130) == xs.XS_ERR_SHAPE and f(B=-1) == xs.XS_ERR_SHAPE
        assert f(left=-2) == xs.XS_ERR_SHAPE and f(right=-2) == xs.XS_ERR_SHAPE and f(sinks=-1) == xs.XS_ERR_SHAPE
        assert f(D=256) == xs.XS_ERR_UNSUPPORTED and f(D=72) == xs.XS_ERR_UNSUPPORTED
        assert f(scale=0.0) == xs.XS_ERR_SHAPE and f(scale=float("nan")) == xs.XS_ERR_SHAPE
        assert f(k=K + 4) == xs.XS_ERR_ALIGN and f(o=V + 64) == xs.XS_ERR_ALIAS
        assert f(ws=None, nb=16) == xs.XS_ERR_WORKSPACE and f(ws=W + 16, nb=1 << 20) == xs.XS_ERR_WORKSPACE
        assert f(ws=O, nb=1 << 20) == xs.XS_ERR_WORKSPACE and "out" in xs.last_error()
        assert f(B=0) == xs.XS_OK and f(S=0) == xs.XS_OK
        if not torch.cuda.is_available():
            assert f() in (xs.XS_ERR_CUDA, xs.XS_ERR_UNSUPPORTED)
    with pytest.raises(xs.XsError):
        xs.attn_window_workspace_size(1, 256, 8, 256, 4)
    with pytest.raises(xs.XsError):
        xs.attn_window_workspace_size(1, 255, 8, 64, 4)
    assert xs.attn_window_workspace_size(0, 256, 8, 64, 4) == 0
    t = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        xs.attn_window(t.transpose(1, 2), t, t, t, 1, 8, 2, 64, 1, 0.1)
    with pytest.raises(ValueError):
        xs.attn_window(t, t, t, t.float(), 1, 8, 2, 64, 1, 0.1)


@pytest.mark.gpu
def test_window_small_workspace_is_refused():
    import torch
    import comm_comp_fusion_gb300 as xs
    t = guarded(256 * 64)
    o = guarded(256 * 64)
    ws = guarded(4096, torch.uint8)
    assert xs.attn_window(t, t, t, o, 1, 256, 1, 64, 1, 0.1, 3, 0, 0, ws, check=False) == xs.XS_ERR_WORKSPACE
    host = torch.zeros(256 * 64, dtype=torch.int16)
    assert xs.attn_window(host, t, t, o, 1, 256, 1, 64, 1, 0.1, 3, 0, 0, check=False) == xs.XS_ERR_UNSUPPORTED
