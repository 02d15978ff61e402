"""Rotary positions (xs_rope): against a 64-bit rotation, its inverse and gradient, the layouts, and its refusals."""
import numpy as np
import pytest

from span_testlib import bf16, head_to_tokens, seq_to_tokens, tokens_to_head, tokens_to_seq, values
from xs_testlib import from_dev, guarded, to_dev


def rotate(x, pos, axes, freqs, halves, inverse):
    """x [B][S][H][D], pos [B][S][A]: (result, bound) in 64 bits.

    The bound: half a bf16 step of the result, 2^-8 of it, and the fp32 arithmetic before it: the angle in half turns is
    rounded to fp32 (2^-24 of at most pi), the sine and cosine are good to 2 ulp, the products and sum to 2^-23: under
    2^-20 (|a| + |b|)."""
    out, bound = x.copy(), np.zeros_like(x)
    begin = f0 = 0
    for a, d in enumerate(axes):
        f = np.asarray(freqs[f0:f0 + d // 2])
        i = np.arange(d // 2)
        i0 = begin + (i if halves else 2 * i)
        i1 = i0 + (d // 2 if halves else 1)
        # in extended precision: a place of 2^31 times a frequency needs more than 53 bits for an exact angle
        ang = (pos[..., a, None].astype(np.longdouble) * f.astype(np.longdouble))
        two_pi = np.longdouble("6.283185307179586476925286766559005768394")
        ang = (ang - np.rint(ang / two_pi) * two_pi).astype(np.float64)[:, :, None, :]
        c, s = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
        p, q = x[..., i0], x[..., i1]
        out[..., i0], out[..., i1] = p * c - q * s, p * s + q * c
        e = 2.0 ** -20 * (np.abs(p) + np.abs(q))
        bound[..., i0], bound[..., i1] = e, e
        begin, f0 = begin + d, f0 + d // 2
    rot = np.zeros(x.shape[-1])
    rot[:begin] = 2.0 ** -8
    return out, bound + np.abs(out) * rot


CASES = [  # B, S, H, Hk, D, P, axes, halves, inverse, seq_in, seq_out, farthest place
    (1, 1, 1, 1, 64, 1, (64,), False, False, False, False, 10),
    (3, 1, 8, 2, 128, 1, (128,), True, False, False, False, 200000),
    (1, 37, 4, 4, 128, 1, (44, 42, 42), False, False, True, False, 60),
    (2, 96, 8, 4, 64, 4, (16, 32), True, False, True, False, 1000),
    (1, 250, 4, 2, 96, 2, (32, 32, 32), True, True, False, True, 1000),
    (2, 24, 6, 6, 96, 3, (2, 4, 6, 8), False, True, True, True, 1000),
    (1, 513, 2, 1, 256, 1, (256,), True, False, False, False, 2 ** 31 - 1),
    (1, 1304, 8, 8, 128, 8, (32, 48, 48), True, False, True, False, 2 ** 31 - 1),
    (5, 700, 3, 0, 128, 1, (126,), False, False, False, False, 2 ** 31 - 1),
    (2, 64, 40, 8, 128, 4, (16,), True, False, False, False, 5000),
    # few heads, many tokens: more tokens share a block
    (1, 39001, 1, 0, 64, 1, (64,), False, False, False, False, 100000),
    (1, 19999, 2, 1, 96, 1, (32, 16), True, False, False, True, 1000),
    (2, 10028, 4, 4, 128, 2, (44, 42, 42), False, True, True, False, 90),
    (1, 9731, 1, 1, 256, 1, (256,), True, False, True, True, 2 ** 31 - 1),
]


def setup(case, seed=0):
    B, S, H, Hk, D, P, axes, halves, inverse, seq_in, seq_out, far = case
    rng = np.random.default_rng(1000 * seed + S + D)
    freqs = [500.0 ** (-2.0 * i / d) for d in axes for i in range(d // 2)]
    pos = rng.integers(-far if far > 100 else 0, far, (B, S, len(axes)), endpoint=True).astype(np.int32)
    qb, q = bf16(rng, (B, S, H, D))
    kb, k = bf16(rng, (B, S, max(Hk, 1), D))
    return freqs, pos, (qb, q), (kb, k)


def lay(x, P, seq):
    return tokens_to_seq(x, P) if seq else tokens_to_head(x, P)


def unlay(x, B, S, H, D, P, seq):
    return seq_to_tokens(x.reshape(P, B, S // P, H, D)) if seq else head_to_tokens(x.reshape(P, B, S, H // P, D))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_rope_matches_64_bits(case):
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, Hk, D, P, axes, halves, inverse, seq_in, seq_out, far = case
    freqs, pos, (qb, q), (kb, k) = setup(case)
    qo, ko = guarded(B * S * H * D), guarded(max(1, B * S * Hk * D))
    dq, dk = to_dev(lay(qb, P, seq_in)), to_dev(lay(kb, P, seq_in)) if Hk else None
    xs.rope(dq, dk, qo, ko if Hk else None, torch.from_numpy(pos).cuda(), B, S, H, Hk, D, P,
            xs.RopeAxes(axes, freqs, halves=halves), seq_in=seq_in, seq_out=seq_out, inverse=inverse)
    for got, x, xb, h in ((qo, q, qb, H), (ko, k, kb, Hk)):
        if not h:
            continue
        got = unlay(from_dev(got), B, S, h, D, P, seq_out)
        ref, bound = rotate(x, pos, axes, freqs, halves, inverse)
        off = np.abs(values(got) - ref) - bound
        assert (off <= 0).all(), (off.max(), np.unravel_index(off.argmax(), off.shape))
        assert np.array_equal(got[..., sum(axes):], xb[..., sum(axes):])


@pytest.mark.gpu
def test_rope_shared_positions_in_place_and_stream():
    """pos of one batch serves all; in place gives the bits of the separate call; on another stream."""
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, Hk, D, P, axes = 3, 50, 4, 2, 128, 2, (32, 32, 64)
    rng = np.random.default_rng(3)
    ax = xs.RopeAxes.powers(axes, theta=100.0, halves=True)
    pos = torch.from_numpy(rng.integers(0, 900, (1, S, 3)).astype(np.int32)).cuda()
    qb, kb = bf16(rng, (P, B, S, H // P, D))[0], bf16(rng, (P, B, S, Hk // P, D))[0]
    q, k = to_dev(qb), to_dev(kb)
    qo, ko = guarded(qb.size), guarded(kb.size)
    xs.rope(q, k, qo, ko, pos.expand(B, S, 3).contiguous(), B, S, H, Hk, D, P, ax)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        xs.rope(q, k, q, k, pos, B, S, H, Hk, D, P, ax)
    s.synchronize()
    assert np.array_equal(from_dev(q).ravel(), from_dev(qo)) and np.array_equal(from_dev(k).ravel(), from_dev(ko))


@pytest.mark.gpu
@pytest.mark.parametrize("halves", (False, True))
def test_rope_folds_the_all_to_all(halves):
    """Sequence partition in, head partition out: bit for bit the rotation followed by the inverse permute."""
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D, P = 2, 128, 8, 128, 4
    rng = np.random.default_rng(9)
    ax = xs.RopeAxes.powers((32, 48, 48), halves=halves)
    pos = torch.from_numpy(rng.integers(0, 64, (B, S, 3)).astype(np.int32)).cuda()
    q, k = to_dev(bf16(rng, (P, B, S // P, H, D))[0]), to_dev(bf16(rng, (P, B, S // P, H, D))[0])
    n = B * S * H * D
    one, two, mid, mid2, want = (guarded(n) for _ in range(5))
    xs.rope(q, k, one, two, pos, B, S, H, H, D, P, ax, seq_in=True, seq_out=False)
    xs.rope(q, k, mid, mid2, pos, B, S, H, H, D, P, ax, seq_in=True, seq_out=True)
    xs.a2a_permute_inverse(mid, want, B, S, H, D, P)
    assert np.array_equal(from_dev(one), from_dev(want))
    xs.a2a_permute_inverse(mid2, want, B, S, H, D, P)
    assert np.array_equal(from_dev(two), from_dev(want))


@pytest.mark.gpu
@pytest.mark.parametrize("halves", (False, True))
def test_rope_gradient(halves):
    """The inverse call is the gradient: against the transposed rotation in 64 bits, and against differences of
    f(x) = sum g rope(x) along random directions (f is linear, so the central difference is exact up to the outputs'
    rounding, 2^-8 of each |rope(x)| at either end)."""
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D, axes = 1, 40, 2, 64, (16, 32)
    rng = np.random.default_rng(21)
    ax = xs.RopeAxes.powers(axes, halves=halves)
    pos = rng.integers(-500, 500, (B, S, 2)).astype(np.int32)
    dpos = torch.from_numpy(pos).cuda()
    (gb, g), (xb, x) = bf16(rng, (B, S, H, D)), bf16(rng, (B, S, H, D))

    def call(bits, inverse):
        out = guarded(bits.size)
        xs.rope(to_dev(bits), None, out, None, dpos, B, S, H, 0, D, 1, ax, inverse=inverse)
        return values(from_dev(out).reshape(bits.shape))

    grad = call(gb, True)
    ref, bound = rotate(g, pos, axes, ax.freqs, halves, True)
    assert (np.abs(grad - ref) <= bound).all()
    for seed in range(3):
        d = np.sign(np.random.default_rng(seed).standard_normal(x.shape)) * 0.5  # x +- d is exact in bf16 only roughly:
        up, down = (to_bits(x + d), to_bits(x - d))                              # so the ends are what they round to
        step = values(up) - values(down)
        yu, yd = call(up, False), call(down, False)
        diff = float((g * (yu - yd)).sum())
        slack = float((np.abs(g) * (np.abs(yu) + np.abs(yd))).sum()) * (2.0 ** -8 + 2.0 ** -18)
        slack += float((np.abs(step) * bound).sum())
        assert abs(diff - float((grad * step).sum())) <= slack


def to_bits(x):
    import torch
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


@pytest.mark.gpu
def test_rope_copies_what_it_does_not_turn():
    """Elements past the axes keep every bit, infinities and NaN among them, and do not touch their neighbours."""
    import torch
    import comm_comp_fusion_gb300 as xs
    for halves, rot in ((False, 22), (True, 32)):
        B, S, H, D = 1, 9, 2, 64
        rng = np.random.default_rng(1)
        bits, x = bf16(rng, (B, S, H, D))
        bits = bits.copy()
        bits[..., rot:] = rng.integers(0, 1 << 16, bits[..., rot:].shape)
        bits[..., rot] = 0x7F80
        bits[..., rot + 1] = 0x7FC1
        x = x.copy()
        x[..., rot:] = 0
        pos = rng.integers(0, 99, (B, S, 1)).astype(np.int32)
        ax = xs.RopeAxes.powers((rot,), halves=halves)
        out = guarded(bits.size)
        xs.rope(to_dev(bits), None, out, None, torch.from_numpy(pos).cuda(), B, S, H, 0, D, 1, ax)
        got = from_dev(out).reshape(bits.shape)
        ref, bound = rotate(x, pos, (rot,), ax.freqs, halves, False)
        assert np.array_equal(got[..., rot:], bits[..., rot:])
        assert (np.abs(values(got[..., :rot]) - ref[..., :rot]) <= bound[..., :rot]).all()


@pytest.mark.gpu
def test_rope_captured_follows_its_positions():
    import torch
    import comm_comp_fusion_gb300 as xs
    B, S, H, D = 1, 20, 2, 128
    rng = np.random.default_rng(5)
    ax = xs.RopeAxes.powers((128,))
    q = to_dev(bf16(rng, (B, S, H, D))[0])
    pos = torch.zeros((B, S, 1), dtype=torch.int32, device="cuda")
    out, want = guarded(q.numel()), guarded(q.numel())
    xs.rope(q, None, out, None, pos, B, S, H, 0, D, 1, ax)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xs.rope(q, None, out, None, pos, B, S, H, 0, D, 1, ax)
    for first in (7, 100000):
        pos.copy_(torch.arange(first, first + S, dtype=torch.int32).view(B, S, 1))
        g.replay()
        xs.rope(q, None, want, None, pos, B, S, H, 0, D, 1, ax)
        assert np.array_equal(from_dev(out), from_dev(want))


Q, K, QO, KO, POS = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000


def test_rope_refusals():
    import __graft_entry__
    __graft_entry__.build()
    import comm_comp_fusion_gb300 as xs

    def f(q=Q, k=K, qo=QO, ko=KO, pos=POS, B=2, S=64, H=8, Hk=8, D=128, P=4, axes=(64, 32), freqs=None, halves=False,
          nb=None, **kw):
        ax = xs.RopeAxes(axes, freqs if freqs is not None else [0.5] * (sum(axes) // 2), halves=halves)
        return xs.rope(q, k, qo, ko, pos, B, S, H, Hk, D, P, ax, pos_batches=nb, check=False, **kw)

    assert f(q=0) == xs.XS_ERR_NULL and f(pos=0) == xs.XS_ERR_NULL and f(k=0) == xs.XS_ERR_NULL
    assert f(H=6) == xs.XS_ERR_SHAPE and f(Hk=6) == xs.XS_ERR_SHAPE and f(S=63) == xs.XS_ERR_SHAPE
    assert f(Hk=-4) == xs.XS_ERR_SHAPE and f(H=1 << 17, P=1) == xs.XS_ERR_SHAPE
    assert f(D=80) == xs.XS_ERR_UNSUPPORTED
    assert f(axes=(3, 2), freqs=[0.1] * 2) == xs.XS_ERR_SHAPE and "axis_dims[0]" in xs.last_error()
    assert f(axes=(64, 66)) == xs.XS_ERR_SHAPE
    assert f(axes=(64, 64, 2)) == xs.XS_ERR_SHAPE and "add up" in xs.last_error()
    assert f(axes=(2,) * 5) == xs.XS_ERR_SHAPE and "n_axes" in xs.last_error()
    assert f(axes=()) == xs.XS_ERR_SHAPE
    assert f(axes=(24,), halves=True) == xs.XS_ERR_UNSUPPORTED
    assert f(freqs=[float("nan")] * 48) == xs.XS_ERR_SHAPE and f(freqs=[2e6] * 48) == xs.XS_ERR_SHAPE
    assert f(nb=3) == xs.XS_ERR_SHAPE
    assert f(q=Q + 8) == xs.XS_ERR_ALIGN and f(ko=KO + 2) == xs.XS_ERR_ALIGN and f(pos=POS + 1) == xs.XS_ERR_ALIGN
    assert f(qo=Q + 16) == xs.XS_ERR_ALIAS and f(qo=K) == xs.XS_ERR_ALIAS and f(ko=Q) == xs.XS_ERR_ALIAS
    assert f(qo=KO) == xs.XS_ERR_ALIAS and f(ko=POS) == xs.XS_ERR_ALIAS and f(qo=POS - 16) == xs.XS_ERR_ALIAS
    assert f(qo=Q, seq_in=True) == xs.XS_ERR_ALIAS       # in place needs the same layout
    assert f(B=0) == xs.XS_OK and f(S=0, Hk=0, k=0, ko=0) == xs.XS_OK
    for kw in (dict(qo=Q, ko=K), dict(qo=Q, seq_in=True, P=1)):  # fine: only a missing GPU may stop these
        if not _gpu():
            assert f(**kw) in (xs.XS_ERR_CUDA, xs.XS_ERR_UNSUPPORTED)
    with pytest.raises(ValueError):
        xs.RopeAxes((4, 4), [1.0])


def _gpu():
    import torch
    return torch.cuda.is_available()


def test_rope_tensor_checks():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs
    ax = xs.RopeAxes.powers((64,))
    q, pos = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 1, dtype=torch.int32)
    bad = [(q.transpose(1, 2), q, pos), (q.float(), q, pos), (q[:, :3], q, pos), (q, q.float(), pos), (q, q, pos.long())]
    for a, b, c in bad:
        with pytest.raises(ValueError):
            xs.rope(a, None, b, None, c, 1, 4, 2, 0, 64, 1, ax)
