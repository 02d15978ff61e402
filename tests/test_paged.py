"""The paged cache: writing new tokens into pages (xs_cache_append) and attention of new tokens over it (xs_attn_paged),
against 64 bits; the operators in a row as a serving loop calls them; refusals."""
import numpy as np
import pytest

from span_testlib import attend, bf16, check, seen_mask, values
from xs_testlib import from_dev, guarded, to_dev

NAN = 0x7FC1


class Batch:
    """A cache with scattered pages. Whatever no sequence owns holds NaN; table entries past a sequence's pages hold
    numbers far outside the pool."""

    def __init__(self, q_len, kv_len, H, Hk, D, page, spare=0, seed=0, sigma=1.0, evict=0, ramp=None):
        import torch
        rng = np.random.default_rng(seed)
        self.q_len, self.kv, self.H, self.Hk, self.D, self.page = q_len, kv_len, H, Hk, D, page
        self.N, self.T = len(q_len), sum(q_len) + spare
        need = [-(-n // page) for n in kv_len]
        self.max_pages, self.n_pages = max(max(need), 1) + 1, sum(need) + 2
        ids = rng.permutation(self.n_pages)
        table = rng.choice(np.array([-1, -2 ** 31, 2 ** 31 - 1, self.n_pages]), (self.N, self.max_pages))
        kp = np.full((self.n_pages, page, Hk, D), NAN, np.uint16)
        vp = np.full((self.n_pages, page, Hk, D), NAN, np.uint16)
        self.k, self.v, at = [], [], 0
        for n in range(self.N):
            kb, k = bf16(rng, (kv_len[n], Hk, D), sigma)
            if ramp:  # keys that point along the queries, longer from `ramp[1]` to `ramp[0]` times along the sequence
                import torch
                long = np.linspace(ramp[0], ramp[1], max(kv_len[n], 1)).reshape(-1, 1, 1)
                kb = torch.from_numpy((np.abs(k) * long).astype(np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)
                k = values(kb)
            vb, v = bf16(rng, (kv_len[n], Hk, D))
            self.k.append(k)
            self.v.append(v)
            for j in range(need[n]):
                i = int(ids[at])
                at += 1
                table[n, j] = i
                m = min(page, kv_len[n] - j * page)
                kp[i, :m], vp[i, :m] = kb[j * page:j * page + m], vb[j * page:j * page + m]
            for j in range(evict):  # pages that a window has passed: their entries may hold anything
                table[n, j] = (-7, 2 ** 31 - 1)[j % 2]
        self.qb, self.q = bf16(rng, (self.T, H, D), sigma)
        if ramp:
            self.qb = self.qb & 0x7FFF
            self.q = np.abs(self.q)
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.q_start = torch.tensor(np.concatenate(([0], np.cumsum(q_len))), dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
        self.dq, self.kp, self.vp = to_dev(self.qb), to_dev(kp), to_dev(vp)
        self.out = guarded(self.T * H * D)
        import comm_comp_fusion_gb300 as xs
        self.ws = guarded(xs.attn_paged_workspace_size(self.N, self.T, H, Hk, D), torch.uint8)

    def call(self, left=-1, right=0, sinks=0, out=None, **kw):
        import comm_comp_fusion_gb300 as xs
        return xs.attn_paged(self.dq, self.kp, self.vp, self.table, self.q_start, self.kv_len,
                             self.out if out is None else out, self.N, self.T, self.H, self.Hk, self.D, self.page,
                             self.n_pages, self.max_pages, self.D ** -0.5, left, right, sinks, self.ws, **kw)

    def verify(self, left=-1, right=0, sinks=0, what=""):
        import torch
        import comm_comp_fusion_gb300 as xs
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        got = from_dev(self.out).reshape(self.T, self.H, self.D)
        G, t = self.H // self.Hk, 0
        for n, (ql, kl) in enumerate(zip(self.q_len, self.kv)):
            pos = np.arange(kl - ql, kl)
            seen = seen_mask(pos, kl, left, right, sinks)
            for h in range(self.H) if self.H * ql < 9000 else sorted({0, 1, self.H // 3, self.H // 2, self.H - 1}):
                ref, bound = attend(self.q[t:t + ql, h], self.k[n][:, h // G], self.v[n][:, h // G], seen, self.D ** -0.5)
                check(got[t:t + ql, h], ref, bound, f"{what} sequence {n} head {h}")
                assert (got[t:t + ql, h][~seen.any(-1)] == 0).all()
            t += ql
        assert (got[t:] == 0xFFFF).all(), "rows of no sequence were written"


CASES = [  # q_len, kv_len, H, Hk, D, page, spare, (left, right, sinks)
    ([1], [1], 1, 1, 64, 16, 0, (-1, 0, 0)),
    ([1], [1], 8, 1, 128, 16, 3, (-1, 0, 0)),
    ([1, 1, 1], [17, 128, 129], 8, 2, 128, 16, 0, (-1, 0, 0)),
    ([1] * 5, [300, 5, 1111, 64, 257], 6, 2, 96, 32, 2, (-1, 0, 0)),      # three heads a key head
    ([1] * 3, [4100, 33, 900], 32, 8, 128, 64, 0, (-1, 0, 0)),
    ([1], [20000], 4, 4, 64, 128, 0, (-1, 0, 0)),                          # split many times
    ([1] * 70, list(range(1, 1400, 20)), 2, 1, 64, 16, 0, (-1, 0, 0)),     # more sequences than a warp's lanes
    ([1, 1], [3000, 2000], 16, 1, 64, 16, 0, (255, 0, 4)),                 # window with sinks
    ([5, 0, 2, 0], [5, 77, 600, 0], 4, 2, 128, 16, 1, (-1, 0, 0)),         # no new tokens, empty sequences
    ([33], [33], 7, 1, 64, 32, 0, (-1, 0, 0)),                             # seven heads a key head: 126 rows of a tile
    ([300], [1000], 4, 4, 128, 64, 5, (-1, 0, 0)),
    ([257, 1, 128], [257, 700, 1500], 8, 4, 96, 256, 9, (-1, 0, 0)),
    ([200, 64], [900, 64], 10, 2, 64, 16, 0, (100, 0, 30)),
    ([200, 64], [900, 500], 4, 2, 128, 1024, 0, (100, 37, 0)),             # two-sided window
    ([150], [650], 4, 2, 128, 16, 0, (-1, -1, 0)),                         # a chunk that sees all of itself
    ([9, 40], [3, 39], 4, 2, 128, 16, 2, (-1, 0, 0)),                      # fewer keys than new tokens: rows without any
    ([9], [0], 4, 2, 64, 16, 0, (-1, -1, 0)),
    ([3], [400], 128, 1, 64, 16, 0, (-1, 0, 0)),                           # 128 heads a key head
    ([600], [2500], 5, 1, 128, 32, 0, (700, 0, 140)),
    ([700, 0, 900, 1, 640], [1500, 40, 1500, 1300, 1290], 32, 32, 64, 16, 3, (-1, 0, 0)),   # whole rounds, then a rest
    ([500, 512], [1100, 1000], 76, 76, 64, 64, 0, (255, 0, 0)),            # two items a CTA, nothing left (152 SMs)
    ([1500], [1500], 24, 24, 64, 128, 0, (-1, 0, 0)),                      # items of unlike lengths
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_paged_matches_64_bits(case):
    q_len, kv_len, H, Hk, D, page, spare, span = CASES[case]
    b = Batch(q_len, kv_len, H, Hk, D, page, spare, seed=case)
    b.call(*span)
    b.verify(*span, what=str(CASES[case][2:]))
    b.out.fill_(-1)
    b.ws.fill_(255)
    b.call(*span)
    b.verify(*span, what="again, workspace of ones")


@pytest.mark.gpu
@pytest.mark.parametrize("D", (64, 96, 128))
def test_paged_passed_pages_may_hold_anything(D):
    """Pages that no token's window reaches are not looked at, whatever their table entries say."""
    b = Batch([3], [1000], 4, 2, D, 16, seed=5, evict=55)   # the first key seen is 997 - 100 = 897, page 56
    b.call(100, 0, 0)
    b.verify(100, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("N,rows", ((1000, 1), (65536, 1), (40000, 3)))
def test_paged_very_many_sequences(N, rows):
    """Thousands of short sequences, many without new tokens: the schedule's sums over the whole batch."""
    import torch
    import comm_comp_fusion_gb300 as xs
    H, Hk, D, page, n_pages = 2 * rows, 2, 64, 16, 300
    gen = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda").bfloat16()  # noqa: E731
    kp, vp = rand(n_pages, page, Hk, D), rand(n_pages, page, Hk, D)
    q_len = torch.randint(0, 2, (N,), generator=gen, device="cuda")
    kv = torch.randint(1, 2 * page + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    table = torch.randint(0, n_pages, (N, 2), generator=gen, device="cuda", dtype=torch.int32)
    q_start = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), q_len.cumsum(0))).to(torch.int32)
    T = int(q_start[-1])
    q, out = rand(T, H, D), guarded(T * H * D)
    ws = guarded(xs.attn_paged_workspace_size(N, T, H, Hk, D), torch.uint8)
    xs.attn_paged(q, kp, vp, table, q_start, kv, out, N, T, H, Hk, D, page, n_pages, 2, 0.125, workspace=ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got = values(from_dev(out)).reshape(T, H, D)
    seqs = q_len.nonzero().view(-1)
    k = kp[table[seqs].long()].view(T, 2 * page, Hk, D).double().repeat_interleave(rows, 2)
    v = vp[table[seqs].long()].view(T, 2 * page, Hk, D).double().repeat_interleave(rows, 2)
    s = torch.einsum("thd,tkhd->thk", q.double(), k) * 0.125
    s = s.masked_fill(torch.arange(2 * page, device="cuda") >= kv[seqs].view(T, 1, 1), -np.inf)
    w = s.softmax(-1)
    ref, a = (torch.einsum("thk,tkhd->thd", w, x).cpu().numpy() for x in (v, v.abs()))
    # the bound of span_testlib.attend; here scale sum |q k| is below 2^5, so the scores' share 2 delta is below 2^-12
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * a + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("q_len", ([1, 1], [90, 40]))
def test_paged_sequences_share_pages(q_len):
    """Two sequences with the same first pages (a common prefix), and one page named twice in a row of the table."""
    b = Batch(q_len, [600, 500], 4, 2, 128, 64, seed=12)
    b.table[1, :5] = b.table[0, :5]
    b.table[0, 6] = b.table[0, 7]
    b.k[1][:320], b.v[1][:320] = b.k[0][:320], b.v[0][:320]
    b.k[0][384:448], b.v[0][384:448] = b.k[0][448:512], b.v[0][448:512]
    b.call()
    b.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,kv_len,H,Hk,D", (([1] * 4, [700, 90, 1500, 64], 8, 2, 128), ([6, 3, 2], [400, 300, 5], 6, 2, 64),
                                                 ([300, 1], [900, 700], 4, 2, 96), ([140], [3000], 2, 1, 128)))
def test_paged_rows_that_are_not_finite_stay_alone(q_len, kv_len, H, Hk, D):
    """A row of q with NaN or an infinity spoils its own output alone, whole and split, in every form."""
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Batch(q_len, kv_len, H, Hk, D, 32, seed=D)
    bad = {(0, 0): NAN, (b.T // 2, H - 1): 0x7F80, (b.T - 1, 1): 0xFF80}
    bits = b.qb.copy()
    for (t, h), x in bad.items():
        bits[t, h, ::7] = x
    b.dq = to_dev(bits)
    b.call()
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got, t = from_dev(b.out).reshape(b.T, H, D), 0
    for n, (ql, kl) in enumerate(zip(q_len, kv_len)):
        for h in range(H):
            ok = [i for i in range(ql) if (t + i, h) not in bad]
            seen = seen_mask(np.arange(kl - ql, kl)[ok], kl, -1, 0, 0)
            if ok:
                ref, bound = attend(b.q[t:t + ql, h][ok], b.k[n][:, h // (H // Hk)], b.v[n][:, h // (H // Hk)], seen, D ** -0.5)
                check(got[t:t + ql, h][ok], ref, bound, f"sequence {n} head {h}")
        t += ql


@pytest.mark.gpu
def test_paged_starts_behind_the_first_row():
    """Packed rows before q_start[0] and behind q_start[N] belong to no sequence."""
    b = Batch([3, 2], [200, 90], 4, 2, 64, 16, spare=6, seed=14)
    b.q_start += 4
    b.call()
    whole = from_dev(b.out).reshape(b.T, 4, 64)
    assert (whole[:4] == 0xFFFF).all() and (whole[9:] == 0xFFFF).all()
    b.out = to_dev(np.concatenate((whole[4:9], whole[9:], whole[:4])))
    b.q = np.concatenate((b.q[4:], b.q[:4]))
    b.verify()


@pytest.mark.gpu
def test_paged_long_chunk_sampled():
    """A chunk over a long cache: items of many K/V tiles in pieces, one row of every 60 against 64 bits."""
    import torch
    b = Batch([1000], [30000], 8, 2, 128, 128, seed=15)
    b.call()
    torch.cuda.synchronize()
    got = from_dev(b.out).reshape(b.T, 8, 128)
    rows = np.arange(0, 1000, 60)
    for h in range(8):
        ref, bound = attend(b.q[rows, h], b.k[0][:, h // 4], b.v[0][:, h // 4], seen_mask(29000 + rows, 30000, -1, 0, 0),
                            128 ** -0.5)
        check(got[rows, h], ref, bound, f"h={h}")


@pytest.mark.gpu
def test_paged_on_two_streams_at_once():
    import torch
    a, c = Batch([1] * 6, [900] * 6, 8, 2, 128, 16, seed=16), Batch([300, 20], [1500, 700], 4, 4, 64, 32, seed=17)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for x, s in zip((a, c), streams):
            x.call(stream=s)
    torch.cuda.synchronize()
    a.verify()
    c.verify()


@pytest.mark.gpu
def test_paged_peaked_scores():
    b = Batch([1, 40], [2000, 700], 8, 2, 128, 16, seed=3, sigma=4.0)
    b.call()
    b.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,H,Hk", (([1, 1], 4, 2), ([2, 3], 16, 2), ([70, 1], 4, 2)))
@pytest.mark.parametrize("ramp", ((8.0, 0.0), (0.0, 8.0)))
def test_paged_rising_and_falling_keys(q_len, H, Hk, ramp):
    """Scores that grow by hundreds along the sequence or against it: the running maxima move in every tile."""
    b = Batch(q_len, [1900, 900], H, Hk, 128, 32, seed=4, ramp=ramp)
    b.call()
    b.verify()


@pytest.mark.gpu
@pytest.mark.parametrize("D", (64, 96, 128))
@pytest.mark.parametrize("G,q_len", ((1, [1, 1, 1]), (5, [3, 1, 0]), (16, [1, 1, 1]), (11, [4, 1, 1]), (32, [1, 1, 1])))
def test_paged_few_rows(D, G, q_len):
    """Groups that do and do not fill the few-rows tiles, sequences of more tokens than one tile among them, and a
    window whose pieces begin behind it."""
    for page, span in ((16, (-1, 0, 0)), (256, (300, 0, 2)), (64, (40, 3, 200))):
        b = Batch(q_len, [2500, 129, 700], 2 * G, 2, D, page, spare=2, seed=G + D)
        b.call(*span)
        b.verify(*span, what=f"{page} {span}")


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,G,spare", (([1] * 30 + [50] + [1] * 30, 4, 0), ([60] + [1] * 20, 5, 3), ([1] * 9 + [0, 17], 8, 0),
                                           ([1] * 12, 4, 150), ([1] * 12, 4, 400)))
@pytest.mark.parametrize("D", (64, 96, 128))
def test_paged_chunk_among_single_tokens(D, q_len, G, spare):
    """A chunk of many few-rows tiles in a batch of single tokens, and single tokens with many rows of no sequence: the
    form follows the average, the results do not."""
    kv = [n + 37 * i % 500 for i, n in enumerate(q_len)]
    kv[q_len.index(max(q_len))] += 700
    for span in ((-1, 0, 0), (90, 5, 3)):
        b = Batch(q_len, kv, 2 * G, 2, D, 32, spare=spare, seed=D + G)
        b.call(*span)
        b.verify(*span, what=f"{span}")


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,kv_len,H,Hk,D", (([1, 1, 1], [700, 2900, 1], 8, 2, 128), ([6, 3, 0, 5], [400, 1300, 70, 5], 6, 2, 64),
                                                 ([5, 5], [3000, 2000], 8, 2, 96), ([300, 1], [1900, 700], 4, 2, 96),
                                                 ([140, 9], [3000, 3], 6, 2, 128), ([257, 600], [900, 1500], 4, 4, 64)))
def test_paged_wide_tables(q_len, kv_len, H, Hk, D):
    """A table that could hold more than 2^18 keys a sequence, around ordinary lengths, in every form, without and with a
    window."""
    import torch
    b = Batch(q_len, kv_len, H, Hk, D, 32, spare=1, seed=D)
    wide = torch.full((b.N, 9000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :b.max_pages] = b.table
    b.table, b.max_pages = wide, 9000
    for span in ((-1, 0, 0), (-1, -1, 0), (300, 0, 4)):
        b.ws.fill_(255)
        b.out.fill_(-1)
        b.call(*span)
        b.verify(*span, what=f"{span}")


@pytest.mark.gpu
def test_paged_graph_follows_lengths():
    """A captured call follows table, lengths and starts that change between replays; two captured calls take turns in
    one workspace."""
    import torch
    b = Batch([1, 1, 1], [700, 300, 1000], 8, 2, 128, 16, seed=7)
    c = Batch([60, 5], [500, 1200], 8, 2, 128, 32, seed=8)
    c.ws = b.ws
    graphs = []
    for x in (b, c):
        x.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.call()
        graphs.append(g)
    for kv in ([700, 300, 1000], [1, 290, 513], [128, 127, 640]):
        b.kv = kv
        b.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        full = (b.k, b.v)
        b.k, b.v = ([a[:n] for a, n in zip(x, kv)] for x in full)
        for x, g in zip((b, c), graphs):
            x.out.fill_(-1)
            g.replay()
            x.verify()
        b.k, b.v = full


@pytest.mark.gpu
def test_paged_pool_past_32_bits():
    """Pages more than 2^31 elements into the pool."""
    import torch
    import comm_comp_fusion_gb300 as xs
    Hk, D, page = 8, 128, 256
    n_pages = 2 ** 31 // (Hk * D * page) + 8
    kp, vp = (torch.empty(n_pages * page * Hk * D, dtype=torch.int16, device="cuda") for _ in range(2))
    b = Batch([7], [700], 16, Hk, D, page, seed=2)
    last = torch.arange(n_pages - 1, n_pages - 4, -1, dtype=torch.int32, device="cuda")
    old = b.table[0, :3].clone()
    for dst, src in ((kp, b.kp), (vp, b.vp)):
        dst.view(n_pages, -1)[last.long()] = src.view(b.n_pages, -1)[old.long()]
    b.table[0, :3] = last
    b.kp, b.vp, b.n_pages = kp, vp, n_pages
    b.call()
    b.verify()
    k = to_dev(bf16(np.random.default_rng(0), (7, Hk, D))[0])
    xs.cache_append(k, k, kp, vp, b.table, b.q_start, b.kv_len, 1, 7, Hk, D, page, n_pages, b.max_pages)
    rows = vp.view(n_pages, page, Hk * D)[int(last[2]), 700 - 512 - 7:700 - 512]
    assert torch.equal(rows.reshape(-1), k.reshape(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,Hk,D,keys", ((1, 152, 152, 64, 2 ** 23 - 77), (1, 190, 190, 128, 2 ** 21 + 5),
                                           (3, 304, 38, 96, 2 ** 22 + 1), (100, 170, 170, 64, 2 ** 21 - 9),
                                           (256, 160, 160, 64, 2 ** 22 - 300), (200, 152, 152, 128, 2 ** 20 + 900),
                                           (2, 2432, 19, 96, 2 ** 21 - 1)))
def test_paged_very_many_keys(T, H, Hk, D, keys):
    """Millions of keys a sequence in every form, whole items and pieces: sums in tensor memory truncate, so they are taken
    in stretches. Values around 1, where that shows. Four pages stand for all, so a key's weight counts as often as it
    comes. The bound: that of span_testlib.attend, and 2^14 additions of a stretch that truncate by 2^-23 at most."""
    import torch
    import comm_comp_fusion_gb300 as xs
    page, n_pages = 1024, 4
    max_pages, own = -(-keys // page), n_pages * page
    gen = torch.Generator(device="cuda").manual_seed(keys)
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    q, kp, vp = rand(T, H, D).bfloat16(), rand(n_pages, page, Hk, D).bfloat16(), (1 + 0.25 * rand(n_pages, page, Hk, D)).bfloat16()
    table = (torch.arange(max_pages, device="cuda") % n_pages).to(torch.int32)
    q_start, kv_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [keys]))
    out = guarded(T * H * D)
    ws = guarded(xs.attn_paged_workspace_size(1, T, H, Hk, D), torch.uint8, 0xFF)
    xs.attn_paged(q, kp, vp, table, q_start, kv_len, out, 1, T, H, Hk, D, page, n_pages, max_pages, D ** -0.5, workspace=ws)
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    got = from_dev(out).reshape(T, H, D)
    j, pos = torch.arange(own, device="cuda"), torch.arange(keys - T, keys, device="cuda")
    often = ((pos.view(-1, 1) - j) // own + 1).double()
    for h in sorted({0, 1, H // 5, H // 3, H // 2, 2 * H // 3, 4 * H // 5, H - 2, H - 1}):
        k, v = kp[:, :, h * Hk // H].reshape(own, D).double(), vp[:, :, h * Hk // H].reshape(own, D).double()
        qd = q[:, h].double()
        s = qd @ k.T * D ** -0.5
        w = often * (s - s.amax(-1, keepdim=True)).exp()
        w = w / w.sum(-1, keepdim=True)
        ref, a = w @ v, w @ v.abs()
        delta = 2.0 ** -18 * (qd.abs() @ k.abs().T * D ** -0.5).amax(-1, keepdim=True)
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * delta + 2.0 ** -9) * a
        check(got[:, h], ref.cpu().numpy(), bound.cpu().numpy(), f"head {h}")


# ------------------------------------------------------------------ append

APPEND = [  # q_len, kv_len, Hk, D, page, spare
    ([1], [1], 1, 64, 16, 0),
    ([1, 1, 1], [17, 16, 300], 8, 128, 16, 2),
    ([5, 0, 40, 1], [5, 9, 100, 64], 3, 96, 32, 7),
    ([300, 77], [1000, 77], 4, 128, 64, 0),
    ([1] * 100, list(range(1, 301, 3)), 1, 64, 16, 0),
    ([2] * 40, list(range(2, 82, 2)), 40, 128, 1024, 1),     # more than 512 chunks a token
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_writes_exactly_its_rows(case):
    import torch
    import comm_comp_fusion_gb300 as xs
    q_len, kv_len, Hk, D, page, spare = APPEND[case]
    b = Batch(q_len, kv_len, Hk, Hk, D, page, spare, seed=case)
    rng = np.random.default_rng(99)
    kb, vb = bf16(rng, (b.T, Hk, D))[0], bf16(rng, (b.T, Hk, D))[0]
    kp, vp = guarded(b.kp.numel()), guarded(b.vp.numel())
    kp.copy_(b.kp.view(-1))
    vp.copy_(b.vp.view(-1))
    xs.cache_append(to_dev(kb), to_dev(vb), kp, vp, b.table, b.q_start, b.kv_len, b.N, b.T, Hk, D, page, b.n_pages,
                    b.max_pages)
    torch.cuda.synchronize()
    table = b.table.cpu().numpy()
    for got, old, new in ((kp, b.kp, kb), (vp, b.vp, vb)):
        want, t = from_dev(old).reshape(b.n_pages, page, Hk, D).copy(), 0
        for n in range(b.N):
            for i in range(q_len[n]):
                place = kv_len[n] - q_len[n] + i
                want[table[n, place // page], place % page] = new[t + i]
            t += q_len[n]
        assert np.array_equal(from_dev(got).reshape(want.shape), want)


@pytest.mark.gpu
def test_append_and_attention_ignore_bad_metadata():
    """Table entries, starts and lengths that lead outside the pool, the table or the packed rows touch nothing."""
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Batch([2, 3, 2], [40, 60, 20], 4, 2, 64, 16, spare=2, seed=1)
    kp, vp = guarded(b.kp.numel()), guarded(b.vp.numel())
    kp.fill_(0)
    vp.fill_(0)
    new = to_dev(bf16(np.random.default_rng(0), (b.T, 2, 64))[0])
    good = b.table.clone(), b.q_start.clone(), b.kv_len.clone()
    for what in range(5):
        b.table, b.q_start, b.kv_len = (x.clone() for x in good)
        if what == 0:
            b.table.fill_(2 ** 31 - 1)
        elif what == 1:
            b.table.fill_(-1)
        elif what == 2:
            b.kv_len.copy_(torch.tensor([2 ** 31 - 1, -5, 10 ** 6], dtype=torch.int32))
            b.table.fill_(b.n_pages)
        elif what == 3:
            b.q_start.copy_(torch.tensor([9, 100, 10 ** 9, 2 ** 31 - 1], dtype=torch.int32))
        else:
            b.q_start.copy_(torch.tensor([-7, -3, -1, 0], dtype=torch.int32))
        xs.cache_append(new, new, kp, vp, b.table, b.q_start, b.kv_len, b.N, b.T, 2, 64, 16, b.n_pages, b.max_pages)
        b.call()
        torch.cuda.synchronize()
        assert xs.device_status() == xs.XS_OK, xs.last_error()
        assert not kp.any() and not vp.any()


@pytest.mark.gpu
@pytest.mark.parametrize("q_len,G", (([3, 2, 2], 2), ([40, 2, 60], 2)))
def test_lengths_past_the_table_count_as_its_end(q_len, G):
    """A kv_len of more keys than the table holds is cut to them, by the append and the attention alike: the new tokens
    stand at the table's last places, are written there and seen there. A negative one counts as none."""
    import torch
    import comm_comp_fusion_gb300 as xs
    Hk, D, page = 2, 64, 16
    for over in (1, 5, page, 2 ** 31 - 1 - 96):
        b = Batch(q_len, [96, 90, 0], G * Hk, Hk, D, page, spare=2, seed=over % 1000)
        b.max_pages = 6   # 96 keys
        b.table = b.table[:, :6].contiguous()
        b.kv_len = torch.tensor([96 + over, 90, -over], dtype=torch.int32, device="cuda")
        (kb, k), (vb, v) = (bf16(np.random.default_rng(1), (b.T, Hk, D)) for _ in range(2))
        old, table = [from_dev(x).reshape(b.n_pages, page, Hk, D) for x in (b.kp, b.vp)], b.table.cpu().numpy()
        kp, vp = guarded(b.kp.numel()), guarded(b.vp.numel())
        kp.copy_(b.kp.view(-1))
        vp.copy_(b.vp.view(-1))
        xs.cache_append(to_dev(kb), to_dev(vb), kp, vp, b.table, b.q_start, b.kv_len, b.N, b.T, Hk, D, page, b.n_pages, 6)
        b.kp, b.vp = kp, vp
        b.call()
        torch.cuda.synchronize()
        for got, want, new, own in ((kp, old[0], kb, b.k), (vp, old[1], vb, b.v)):
            want, t = want.copy(), 0
            for n in range(2):
                for i in range(q_len[n]):
                    place = b.kv[n] - q_len[n] + i
                    want[table[n, place // page], place % page] = new[t + i]
                    own[n][place] = values(new[t + i])
                t += q_len[n]
            assert (from_dev(got).reshape(want.shape) == want).all(), over
        b.verify(what=f"over by {over}")


# ------------------------------------------------------------------ in a row

@pytest.mark.gpu
@pytest.mark.parametrize("span", ((-1, 0, 0), (150, 0, 4)))
def test_serving_loop_equals_whole_sequence(span):
    """A prompt in chunks and then single tokens, each step turning q and k, appending and attending over the cache,
    against rotary positions and windowed attention over the whole sequences at once."""
    import torch
    import comm_comp_fusion_gb300 as xs
    N, S, H, D, page = 2, 430, 4, 128, 16
    steps = [200, 129, 90] + [1] * 11
    assert sum(steps) == S
    rng = np.random.default_rng(31)
    (qb, _), (kb, _), (vb, _) = (bf16(rng, (N, S, H, D)) for _ in range(3))
    ax = xs.RopeAxes.powers((D,), halves=True)
    pos = torch.arange(S, dtype=torch.int32, device="cuda").view(1, S, 1)
    q, k, v = to_dev(qb), to_dev(kb), to_dev(vb)
    qr, kr, want = (guarded(q.numel()) for _ in range(3))
    xs.rope(q, k, qr, kr, pos, N, S, H, H, D, 1, ax)
    xs.attn_window(qr, kr, v, want, N, S, H, D, 1, D ** -0.5, *span)
    max_pages = -(-S // page)
    n_pages = N * max_pages
    kp, vp = guarded(n_pages * page * H * D), guarded(n_pages * page * H * D)   # NaN to begin with
    table = torch.randperm(n_pages, device="cuda").to(torch.int32).view(N, max_pages)
    got = torch.zeros((N, S, H, D), dtype=torch.int16, device="cuda")
    done = 0
    for n_new in steps:
        T = N * n_new
        part = [x.view(N, S, H, D)[:, done:done + n_new].reshape(T, H, D).contiguous() for x in (q, k, v)]
        at = pos[:, done:done + n_new].expand(N, n_new, 1).contiguous()
        xs.rope(part[0], part[1], part[0], part[1], at, 1, T, H, H, D, 1, ax, pos_batches=1)
        q_start = torch.arange(0, T + 1, n_new, dtype=torch.int32, device="cuda")
        kv_len = torch.full((N,), done + n_new, dtype=torch.int32, device="cuda")
        xs.cache_append(part[1], part[2], kp, vp, table, q_start, kv_len, N, T, H, D, page, n_pages, max_pages)
        out = guarded(T * H * D)
        ws = guarded(xs.attn_paged_workspace_size(N, T, H, H, D), torch.uint8)
        xs.attn_paged(part[0], kp, vp, table, q_start, kv_len, out, N, T, H, H, D, page, n_pages, max_pages, D ** -0.5,
                      *span, workspace=ws)
        got[:, done:done + n_new] = out.view(N, n_new, H, D)
        done += n_new
    torch.cuda.synchronize()
    assert xs.device_status() == xs.XS_OK, xs.last_error()
    qv, kv_ = (values(from_dev(x).reshape(N, S, H, D)) for x in (qr, kr))
    vv = values(vb)
    seen = seen_mask(np.arange(S), S, *span)
    for bits in (from_dev(got), from_dev(want).reshape(N, S, H, D)):
        for n in range(N):
            for h in range(H):
                ref, bound = attend(qv[n, :, h], kv_[n, :, h], vv[n, :, h], seen, D ** -0.5)
                check(bits[n, :, h], ref, bound, f"sequence {n} head {h}")


# ------------------------------------------------------------------ refusals

Q, KP, VP, TAB, QS, KL, O, W = (0x10000000 * i for i in range(1, 9))


def test_paged_refusals():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs

    def attn(q=Q, kp=KP, tab=TAB, qs=QS, o=O, N=2, T=10, H=8, Hk=2, D=128, page=16, n_pages=50, max_pages=20, scale=0.1,
             left=-1, right=0, sinks=0, ws=W, nb=1 << 27):
        return xs.attn_paged(q, kp, VP, tab, qs, KL, o, N, T, H, Hk, D, page, n_pages, max_pages, scale, left, right,
                             sinks, ws, nb, check=False)

    def app(q=Q, kp=KP, tab=TAB, qs=QS, o=O, **kw):
        a = dict(N=2, T=10, Hk=2, D=128, page=16, n_pages=50, max_pages=20)
        a.update({n: x for n, x in kw.items() if n in a})
        return xs.cache_append(q, o, kp, VP, tab, qs, KL, a["N"], a["T"], a["Hk"], a["D"], a["page"], a["n_pages"],
                               a["max_pages"], check=False)

    for f in (attn, app):
        assert f(q=0) == xs.XS_ERR_NULL and f(tab=0) == xs.XS_ERR_NULL and f(qs=0) == xs.XS_ERR_NULL
        assert f(N=-1) == xs.XS_ERR_SHAPE and f(T=-1) == xs.XS_ERR_SHAPE and f(Hk=0) == xs.XS_ERR_SHAPE
        assert f(n_pages=0) == xs.XS_ERR_SHAPE and f(max_pages=0) == xs.XS_ERR_SHAPE
        assert f(max_pages=1 << 27) == xs.XS_ERR_SHAPE and f(n_pages=2 ** 31 - 1, page=1024) == xs.XS_ERR_SHAPE
        assert f(T=2 ** 31 - 1) == xs.XS_ERR_SHAPE and f(N=(1 << 16) + 1) == xs.XS_ERR_SHAPE
        assert f(D=256) == xs.XS_ERR_UNSUPPORTED and f(page=8) == xs.XS_ERR_UNSUPPORTED
        assert f(page=48) == xs.XS_ERR_UNSUPPORTED and f(page=2048) == xs.XS_ERR_UNSUPPORTED
        assert f(q=Q + 2) == xs.XS_ERR_ALIGN and f(kp=KP + 8) == xs.XS_ERR_ALIGN and f(tab=TAB + 2) == xs.XS_ERR_ALIGN
        assert f(N=0) == xs.XS_OK and f(T=0) == xs.XS_OK
        if not torch.cuda.is_available():
            assert f() in (xs.XS_ERR_CUDA, xs.XS_ERR_UNSUPPORTED)
    assert app(kp=Q) == xs.XS_ERR_ALIAS and app(kp=VP + 16) == xs.XS_ERR_ALIAS and app(tab=KP + 64) == xs.XS_ERR_ALIAS
    assert attn(o=Q + 16) == xs.XS_ERR_ALIAS and attn(o=KP) == xs.XS_ERR_ALIAS and attn(tab=O) == xs.XS_ERR_ALIAS
    assert attn(H=7) == xs.XS_ERR_SHAPE and attn(H=0) == xs.XS_ERR_SHAPE and attn(H=258) == xs.XS_ERR_UNSUPPORTED
    assert attn(scale=-1.0) == xs.XS_ERR_SHAPE and attn(scale=float("inf")) == xs.XS_ERR_SHAPE
    assert attn(left=-2) == xs.XS_ERR_SHAPE and attn(right=-9) == xs.XS_ERR_SHAPE and attn(sinks=-1) == xs.XS_ERR_SHAPE
    assert attn(ws=None, nb=0) == xs.XS_ERR_NULL and attn(ws=None, nb=8) == xs.XS_ERR_WORKSPACE
    assert attn(ws=W + 128) == xs.XS_ERR_WORKSPACE and attn(ws=O) == xs.XS_ERR_WORKSPACE
    assert attn(ws=None, nb=0, N=0) == xs.XS_OK
    for bad in ((-1, 4, 4, 2, 64), (1, 4, 5, 2, 64), (1, 4, 4, 0, 64), (1, 4, 4, 2, 80)):
        with pytest.raises(xs.XsError):
            xs.attn_paged_workspace_size(*bad)
    assert xs.attn_paged_workspace_size(0, 4, 4, 2, 64) == 0
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool, i = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for a, p, tab in ((t[:, :1], pool, i), (t, pool.float(), i), (t, pool[:1], i), (t, pool, i.long())):
        with pytest.raises(ValueError):
            xs.attn_paged(a, p, pool, tab, i, i, t, 1, 4, 2, 2, 64, 16, 2, 1, 0.1)
        with pytest.raises(ValueError):
            xs.cache_append(a, t, p, pool, tab, i, i, 1, 4, 2, 64, 16, 2, 1)


@pytest.mark.gpu
def test_paged_small_workspace_and_host_memory_are_refused():
    import torch
    import comm_comp_fusion_gb300 as xs
    b = Batch([1], [20], 2, 1, 64, 16)
    b.ws = b.ws[:4096]
    assert b.call(check=False) == xs.XS_ERR_WORKSPACE
    b = Batch([1], [20], 2, 1, 64, 16)
    b.kv_len = b.kv_len.cpu()
    assert b.call(check=False) == xs.XS_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (from_dev(b.out) == 0xFFFF).all()


def test_types_are_checked():
    """float16 values are not taken as bf16, nor floats as places, numbers of pages or lengths; bf16 bits are."""
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    ax = xs.RopeAxes.powers((64,))

    def calls(x, o, i):
        return [lambda: xs.rope(x, x, o, o, i, 1, 4, 2, 2, 64, 1, ax, check=False),
                lambda: xs.attn_window(x, x, x, o, 1, 4, 2, 64, 1, 0.1, check=False),
                lambda: xs.attn_window_a2a(x, x, x, o, 1, 4, 2, 64, 1, 0.1, check=False),
                lambda: xs.cache_append(x, x, o, o, i, i, i, 1, 4, 2, 64, 2, 1, 1, check=False),
                lambda: xs.attn_paged(x, x, x, i, i, i, o, 1, 4, 2, 2, 64, 2, 1, 1, 0.1, check=False)]

    for bad in (calls(x.half(), x, i), calls(x, x.half(), i)):
        for call in bad:
            with pytest.raises(ValueError, match="bfloat16"):
                call()
    for k in (0, 3, 4):
        for wrong in (i.float(), i.view(torch.float32)):
            with pytest.raises(ValueError, match="int32"):
                calls(x, x, wrong)[k]()
    for bits in (torch.int16, torch.uint16):
        for call in calls(x.view(bits), x.view(bits), i):
            assert call() != xs.XS_OK  # these are host tensors, or one buffer twice: refused behind the types


def test_workspace_sizes_refuse_what_the_calls_refuse():
    import __graft_entry__
    __graft_entry__.build()
    import ctypes
    import comm_comp_fusion_gb300 as xs
    n = ctypes.c_size_t(7)
    for T, H, Hk in ((4, 258, 2), (4, 7, 2), (4, 0, 2), (1 << 27, 16, 16)):
        want = xs.attn_paged(Q, KP, VP, TAB, QS, KL, O, 2, T, H, Hk, 64, 16, 50, 20, 0.1, workspace=W, workspace_bytes=1 << 27,
                             check=False)
        assert want in (xs.XS_ERR_SHAPE, xs.XS_ERR_UNSUPPORTED)
        assert xs.lib.xs_attn_paged_workspace_size(2, T, H, Hk, 64, ctypes.byref(n)) == want
    for B, S, H, D, P in ((1, (1 << 24) + 128, 1, 64, 1), (1, 128, 1, 256, 1), (1, 129, 2, 64, 2)):
        want = xs.attn_window(Q, KP, VP, O, B, S, H, D, P, 0.1, check=False)
        assert want in (xs.XS_ERR_SHAPE, xs.XS_ERR_UNSUPPORTED)
        assert xs.lib.xs_attn_window_workspace_size(B, S, H, D, P, ctypes.byref(n)) == want
    assert n.value == 7


def test_workspace_tensors_are_contiguous():
    import __graft_entry__
    __graft_entry__.build()
    import torch
    import comm_comp_fusion_gb300 as xs
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 27), torch.zeros(64, 2, dtype=torch.float32).t()):
        with pytest.raises(ValueError, match="workspace"):
            xs.attn_window(Q, KP, VP, O, 1, 128, 1, 64, 1, 0.1, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            xs.attn_paged(Q, KP, VP, TAB, QS, KL, O, 2, 4, 4, 2, 64, 16, 50, 20, 0.1, workspace=ws)
