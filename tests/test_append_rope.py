"""Rotary positions on the way into the paged cache (xs_cache_append_rope): against 64 bits, and to the bit against the
rotary call followed by the append; rows of a projection; refusals."""
import numpy as np
import pytest

from span_testlib import bf16, values
from test_rope import rotate
from xs_testlib import from_dev, guarded, to_dev

CASES = [  # q_len, kv_len, H, Hk, D, page, spare, axes, halves, positions given, one projection, k_out
    ([1], [1], 1, 1, 64, 16, 0, (64,), False, False, False, False),
    ([1] * 8, [300, 17, 16, 1, 999, 64, 65, 128], 32, 8, 128, 16, 0, (128,), True, False, True, False),
    ([1] * 5, [9, 70, 33, 5, 1], 5, 1, 96, 32, 4, (96,), True, False, True, True),
    ([5, 0, 40, 1], [5, 9, 100, 64], 6, 3, 96, 32, 7, (32, 48), False, True, False, True),
    ([300, 77], [1000, 77], 8, 4, 128, 64, 0, (44, 42, 42), False, True, True, False),
    ([16] * 30, list(range(16, 1500, 50)), 8, 2, 64, 16, 3, (64,), True, True, True, True),
    ([2] * 40, list(range(2, 82, 2)), 40, 40, 128, 1024, 1, (16,), True, False, False, False),  # few elements turn
    ([700, 0, 1300], [700, 0, 9000], 2, 1, 64, 256, 5, (64,), True, False, True, True),         # many tokens a block
    ([4000, 3500], [4000, 8000], 4, 2, 96, 128, 0, (96,), False, False, True, False),
    ([33, 2], [33, 40], 0, 2, 128, 16, 1, (128,), True, False, False, False),                   # keys and values alone
    ([3, 1], [70, 9], 200, 100, 64, 16, 0, (32, 32), True, True, True, True),                   # many heads
    ([25, 3], [25, 90], 12, 4, 96, 16, 2, (16, 48), True, True, True, False),
    ([9, 40], [3, 39], 4, 2, 128, 16, 2, (128,), True, False, False, True),                     # places before the sequence
]


class Step:
    def __init__(self, case, seed=0):
        import torch
        (self.q_len, self.kv, self.H, self.Hk, self.D, self.page, self.spare, self.axes, self.halves, given, fused,
         keep) = case
        H, Hk, D = self.H, self.Hk, self.D
        rng = np.random.default_rng(seed)
        self.N, self.T = len(self.q_len), sum(self.q_len) + self.spare
        need = [-(-n // self.page) for n in self.kv]
        self.max_pages, self.n_pages = max(max(need), 1) + 1, sum(need) + 2
        ids, at = rng.permutation(self.n_pages), 0
        self.table = rng.choice(np.array([-1, -2 ** 31, 2 ** 31 - 1, self.n_pages]), (self.N, self.max_pages))
        for n, m in enumerate(need):
            self.table[n, :m] = ids[at:at + m]
            at += m
        self.places = np.concatenate([np.arange(k - q, k) for q, k in zip(self.q_len, self.kv)] + [np.zeros(self.spare, int)])
        self.seq = np.repeat(np.arange(self.N + 1), self.q_len + [self.spare])
        self.pos = None
        if given:
            self.pos = rng.integers(-2 ** 31, 2 ** 31 - 1, (self.T, len(self.axes)), endpoint=True).astype(np.int32)
        self.freqs = [500.0 ** (-2.0 * i / d) for d in self.axes for i in range(d // 2)]
        self.ax = None
        bits = bf16(rng, (self.T, H + 2 * Hk, D))[0]
        self.qb, self.kb, self.vb = bits[:, :H], bits[:, H:H + Hk], bits[:, H + Hk:]
        if fused:
            row = to_dev(bits)
            self.q, self.k, self.v = row[:, :H], row[:, H:H + Hk], row[:, H + Hk:]
        else:
            self.q, self.k, self.v = to_dev(self.qb), to_dev(self.kb), to_dev(self.vb)
        if not H:
            self.q = None
        self.q_out = guarded(self.T * H * D) if H else None
        self.k_out = guarded(self.T * Hk * D) if keep else None
        self.old = [bf16(rng, (self.n_pages, self.page, Hk, D))[0] for _ in range(2)]
        self.kp, self.vp = guarded(self.old[0].size), guarded(self.old[0].size)
        self.reset()
        self.dtable = torch.from_numpy(self.table.astype(np.int32)).cuda()
        self.q_start = torch.tensor(np.concatenate(([0], np.cumsum(self.q_len))), dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        self.dpos = None if self.pos is None else torch.from_numpy(self.pos).cuda()

    def reset(self):
        for pool, old in zip((self.kp, self.vp), self.old):
            pool.copy_(to_dev(old).view(-1))
        for out in (self.q_out, self.k_out):
            if out is not None:
                out.fill_(-1)

    def call(self, **kw):
        import comm_comp_fusion_gb300 as xs
        self.ax = self.ax or xs.RopeAxes(self.axes, self.freqs, halves=self.halves)
        a = dict(q=self.q, k=self.k, v=self.v, q_out=self.q_out, k_pages=self.kp, v_pages=self.vp, page_table=self.dtable,
                 q_start=self.q_start, kv_len=self.kv_len, N=self.N, T=self.T, H=self.H, Hk=self.Hk, D=self.D,
                 page=self.page, n_pages=self.n_pages, max_pages=self.max_pages, axes=self.ax, pos=self.dpos,
                 k_out=self.k_out)
        a.update(kw)
        return xs.cache_append_rope(**a)

    def turned(self, x):
        """(result, bound) in 64 bits of x [T, heads, D]."""
        pos = self.places.reshape(-1, 1) if self.pos is None else self.pos
        ref, bound = rotate(values(x)[None], pos[None], self.axes, self.freqs, self.halves, False)
        return ref[0], bound[0]

    def verify(self):
        import torch
        torch.cuda.synchronize()
        real = self.T - self.spare
        rows = np.full(self.T, -1)
        for t in range(real):
            p = self.places[t]
            if p >= 0:
                rows[t] = self.table[self.seq[t], p // self.page] * self.page + p % self.page
        for out, bits in ((self.q_out, self.qb), (self.k_out, self.kb)):
            if out is None:
                continue
            got = from_dev(out).reshape(bits.shape)
            ref, bound = self.turned(bits)
            off = np.abs(values(got[:real]) - ref[:real]) - bound[:real]
            assert (off <= 0).all(), off.max()
            assert np.array_equal(got[:real, :, sum(self.axes):], bits[:real, :, sum(self.axes):])
            assert (got[real:] == 0xFFFF).all(), "rows of no sequence were written"
        written = rows >= 0
        for pool, old, bits in ((self.kp, self.old[0], self.kb), (self.vp, self.old[1], self.vb)):
            got, want = from_dev(pool).reshape(-1, self.Hk, self.D), old.reshape(-1, self.Hk, self.D)
            rest = np.ones(got.shape[0], bool)
            rest[rows[written]] = False
            assert np.array_equal(got[rest], want[rest]), "other rows of the pool changed"
            if pool is self.vp:
                assert np.array_equal(got[rows[written]], bits[written])
            else:
                ref, bound = self.turned(bits)
                off = np.abs(values(got[rows[written]]) - ref[written]) - bound[written]
                assert (off <= 0).all(), off.max()
                if self.k_out is not None:
                    kept = from_dev(self.k_out).reshape(bits.shape)
                    assert np.array_equal(kept[written], got[rows[written]])


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_rope_matches_64_bits(case):
    s = Step(CASES[case], seed=case)
    s.call()
    s.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("case", (1, 3, 5, 7))
def test_append_rope_equals_rope_then_append(case):
    """To the bit; and the same call again gives the same bits."""
    import torch
    import comm_comp_fusion_gb300 as xs
    s = Step(CASES[case], seed=20 + case)
    s.spare, s.T = 0, s.T - s.spare
    s.call()
    got = [from_dev(x).copy() for x in (s.q_out[:s.T * s.H * s.D], s.kp, s.vp)]
    s.reset()
    pos = torch.from_numpy(s.places[:s.T].astype(np.int32)).cuda() if s.pos is None else s.dpos[:s.T].contiguous()
    q, k, v = (x[:s.T].contiguous() for x in (s.q, s.k, s.v))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    xs.rope(q, k, qo, ko, pos, 1, s.T, s.H, s.Hk, s.D, 1, s.ax)
    xs.cache_append(ko, v, s.kp, s.vp, s.dtable, s.q_start, s.kv_len, s.N, s.T, s.Hk, s.D, s.page, s.n_pages, s.max_pages)
    for a, b in zip(got, (qo, s.kp, s.vp)):
        assert np.array_equal(a, from_dev(b).reshape(a.shape))
    s.reset()
    s.call()
    for a, b in zip(got, (s.q_out[:s.T * s.H * s.D], s.kp, s.vp)):
        assert np.array_equal(a, from_dev(b))


@pytest.mark.gpu
def test_append_rope_in_place_other_stream_and_graph():
    """q and k turned in place; on another stream; a captured call follows lengths, table and positions."""
    import torch
    s = Step(CASES[3], seed=40)
    s.q_out, s.k_out = guarded(s.qb.size), guarded(s.kb.size)
    s.q, s.k = s.q_out, s.k_out
    stream = torch.cuda.Stream()

    def fill():
        s.reset()
        s.q_out.copy_(to_dev(s.qb).view(-1))
        s.k_out.copy_(to_dev(s.kb).view(-1))

    def verify():
        for out, bits in ((s.q_out, s.qb), (s.k_out, s.kb)):
            kept = from_dev(out).reshape(bits.shape)[s.T - s.spare:]
            assert np.array_equal(kept, bits[s.T - s.spare:])
            out.view(s.T, -1)[s.T - s.spare:] = -1
        s.verify()

    fill()
    torch.cuda.synchronize()
    s.call(stream=stream)
    torch.cuda.synchronize()
    verify()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    for kv in ([5, 9, 100, 64], [96, 0, 40, 1]):
        s.kv = kv
        s.table = np.array([[0, 1, 2, 9, -1], [-1] * 5, [3, 4, 5, 6, -1], [7, 8, -1, -1, -1]])
        s.places = np.concatenate([np.arange(k - q, k) for q, k in zip(s.q_len, s.kv)] + [np.zeros(s.spare, int)])
        s.dtable.copy_(torch.from_numpy(s.table.astype(np.int32)))
        s.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        fill()
        g.replay()
        torch.cuda.synchronize()
        verify()


@pytest.mark.gpu
def test_append_rope_ignores_bad_metadata():
    """Table entries, starts and lengths that lead outside the pool, the table or the packed rows touch nothing there."""
    import torch
    s = Step(([2, 3, 2], [40, 60, 20], 4, 2, 64, 16, 2, (64,), True, False, True, True), seed=3)
    good = s.dtable.clone(), s.q_start.clone(), s.kv_len.clone()
    for what in range(5):
        s.reset()
        s.dtable, s.q_start, s.kv_len = (x.clone() for x in good)
        if what == 0:
            s.dtable.fill_(2 ** 31 - 1)
        elif what == 1:
            s.dtable.fill_(-1)
        elif what == 2:
            s.kv_len.copy_(torch.tensor([2 ** 31 - 1, -5, 10 ** 6], dtype=torch.int32))
            s.dtable.fill_(s.n_pages)
        elif what == 3:
            s.q_start.copy_(torch.tensor([9, 100, 10 ** 9, 2 ** 31 - 1], dtype=torch.int32))
        else:
            s.q_start.copy_(torch.tensor([-7, -3, -1, 0], dtype=torch.int32))
        s.call()
        torch.cuda.synchronize()
        for pool, old in zip((s.kp, s.vp), s.old):
            assert np.array_equal(from_dev(pool), old.reshape(-1))
        if what >= 3:
            assert (from_dev(s.q_out) == 0xFFFF).all() and (from_dev(s.k_out) == 0xFFFF).all()


@pytest.mark.gpu
def test_append_rope_lengths_past_the_table():
    """A kv_len past the table's end counts as its end, as in the plain append."""
    import torch
    s = Step(([3, 2], [64, 60], 2, 1, 64, 16, 0, (64,), True, False, False, False), seed=5)
    s.dtable = s.dtable[:, :4].contiguous()   # 64 keys
    s.table, s.max_pages = s.table[:, :4], 4
    s.kv_len.copy_(torch.tensor([1000, 60], dtype=torch.int32))
    s.call()
    s.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("D,page", ((128, 256), (64, 16)))
def test_append_rope_pool_past_32_bits(D, page):
    """Pages more than 2^31 elements into the pool, and rows of a projection more than 2^31 elements apart."""
    import torch
    Hk, T = 8, 5
    s = Step(([T], [T + 9], 8, Hk, D, page, 0, (D,), True, False, False, False), seed=7)
    n_pages = 2 ** 31 // (Hk * D * page) + 4
    kp, vp = (torch.zeros(n_pages * page * Hk * D, dtype=torch.int16, device="cuda") for _ in range(2))
    table = torch.full_like(s.dtable, n_pages - 1)
    stride = 2 ** 29 + 64
    wide = torch.zeros((T - 1) * stride + 8 * D, dtype=torch.int16, device="cuda")
    far = torch.as_strided(wide, (T, 8 * D), (stride, 1))
    far.copy_(s.q.view(T, -1))
    s.call(q=far, k_pages=kp, v_pages=vp, page_table=table, n_pages=n_pages)
    torch.cuda.synchronize()
    got = from_dev(s.q_out).reshape(s.qb.shape)
    ref, bound = s.turned(s.qb)
    assert (np.abs(values(got) - ref) <= bound).all()
    rows = vp.view(n_pages, page, Hk, D)[n_pages - 1, 9:9 + T]
    assert np.array_equal(from_dev(rows), s.vb)
    assert not vp.view(n_pages, -1)[:n_pages - 1].any()
    rows = from_dev(kp.view(n_pages, page, Hk, D)[n_pages - 1, 9:9 + T])
    ref, bound = s.turned(s.kb)
    assert (np.abs(values(rows) - ref) <= bound).all()


# ------------------------------------------------------------------ refusals

A = [0x10000000 * (i + 1) for i in range(12)]


def _refusal(xs, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], q_out=A[3], k_pages=A[4], v_pages=A[5], page_table=A[6], q_start=A[7], kv_len=A[8], N=2,
             T=4, H=4, Hk=2, D=64, page=16, n_pages=50, max_pages=20, axes=xs.RopeAxes.powers((64,)), pos=None, k_out=None,
             check=False)
    a.update(kw)
    return xs.cache_append_rope(**a)


def test_append_rope_refusals():
    import __graft_entry__
    __graft_entry__.build()
    import comm_comp_fusion_gb300 as xs
    for name in ("k", "v", "k_pages", "v_pages", "page_table", "q_start", "kv_len", "q", "q_out"):
        assert _refusal(xs, **{name: None}) == xs.XS_ERR_NULL, name
    for kw in (dict(N=-1), dict(T=-1), dict(H=-1), dict(Hk=0), dict(n_pages=0), dict(max_pages=0), dict(N=65537),
               dict(T=(1 << 29) + 1), dict(H=65536), dict(T=1 << 28, H=8), dict(max_pages=1 << 26)):
        assert _refusal(xs, **kw) == xs.XS_ERR_SHAPE, kw
    for kw in (dict(D=80), dict(D=256), dict(page=8), dict(page=24), dict(page=2048)):
        assert _refusal(xs, **kw) == xs.XS_ERR_UNSUPPORTED, kw
    assert _refusal(xs, axes=xs.RopeAxes.powers((32, 32))) == xs.XS_ERR_NULL          # which place is whose axis?
    assert _refusal(xs, axes=xs.RopeAxes.powers((128,))) == xs.XS_ERR_SHAPE
    assert _refusal(xs, axes=xs.RopeAxes.powers((24,), halves=True)) == xs.XS_ERR_UNSUPPORTED
    assert _refusal(xs, axes=xs.RopeAxes((64,), [float("nan")] * 32)) == xs.XS_ERR_SHAPE
    for name in ("q", "k", "v", "q_out", "k_out", "k_pages", "v_pages"):
        assert _refusal(xs, **{name: A[10] + 8}) == xs.XS_ERR_ALIGN, name
    for name in ("page_table", "q_start", "kv_len", "pos"):
        assert _refusal(xs, **{name: A[10] + 2}) == xs.XS_ERR_ALIGN, name
    for out in ("q_out", "k_out", "k_pages", "v_pages"):
        for name in ("q", "k", "v", "page_table", "q_start", "kv_len", "pos", "q_out", "k_out", "k_pages", "v_pages"):
            if name != out and (out, name) not in (("q_out", "q"), ("k_out", "k")):
                assert _refusal(xs, **{out: A[10], name: A[10] + 16}) == xs.XS_ERR_ALIAS, (out, name)
    assert _refusal(xs, q=A[3] + 16) == xs.XS_ERR_ALIAS
    assert _refusal(xs, k=A[1], k_out=A[1] + 16) == xs.XS_ERR_ALIAS
    ax = xs.RopeAxes.powers((64,))

    def raw(strides=(0, 0, 0), flags=0, q_out=A[3]):
        return xs.lib.xs_cache_append_rope(A[0], A[1], A[2], *strides, q_out, None, A[4], A[5], A[6], A[7], A[8], None, 2, 4, 4,
                                           2, 64, 16, 50, 20, 1, ax._dims, ax._freqs, flags, None)
    for strides in ((255, 0, 0), (260, 0, 0), (0, 120, 0), (0, 0, 1 << 31), (-256, 0, 0)):
        assert raw(strides) == xs.XS_ERR_SHAPE
    assert raw(flags=2) == xs.XS_ERR_SHAPE
    assert raw((512, 0, 0), q_out=A[0]) == xs.XS_ERR_ALIAS        # in place, but the rows have gaps
    assert xs.lib.xs_cache_append_rope(A[0], A[1], A[2], 0, 0, 0, A[3], None, A[4], A[5], A[6], A[7], A[8], None, 0, 4, 4, 2, 64,
                                       16, 50, 20, 1, ax._dims, ax._freqs, 0, None) == xs.XS_OK  # nothing to do


def test_append_rope_types_and_rows():
    """Types are checked; rows may lie apart, but not overlap or have gaps within."""
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs
    ax = xs.RopeAxes.powers((64,))
    x, i = torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.int32)
    pool = torch.zeros(16 * 2 * 64, dtype=torch.bfloat16)

    def call(q=None, k=None, o=None, j=i):
        return xs.cache_append_rope(x[:, :4] if q is None else q, x[:, 4:6] if k is None else k, x[:, 6:],
                                    x.clone() if o is None else o, pool, pool.clone(), i, j, i, 1, 4, 4, 2, 64, 16, 1, 1, ax,
                                    check=False)
    assert call() == xs.XS_ERR_UNSUPPORTED or call() == xs.XS_ERR_CUDA    # host tensors get as far as the device checks
    for kw in (dict(q=x[:, :4].half()), dict(q=x.half()[:, :4]), dict(o=x.half())):
        with pytest.raises(ValueError, match="bfloat16"):
            call(**kw)
    with pytest.raises(ValueError, match="int32"):
        call(j=i.long())
    for bad in (x[:2, :4], x[:, ::2], x[:, :4, ::2], x[:, :4].transpose(0, 1), x[:1, :4].expand(4, 4, 64), x[:, :4].flatten(0, 1)[:15]):
        with pytest.raises(ValueError, match="contiguous"):
            call(q=bad)
