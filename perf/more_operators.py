"""The operators of a serving step around the paged cache, as a program calls them: new tokens' queries, keys and values
turned by their positions on the way into the cache, the masks of drafted token trees and attention of such trees over the
cache, and attention over whole prompts packed one after the other.

`run` computes each operator in plain torch operations; with `own` set it calls the library. `exact` gives the same
results in 64 bits."""
import math

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # rotate and append: one new token of each of 8 sequences, projected as one [q k v] row, at its own place
        dict(name="rope append 8 single tokens", op="append", N=8, H=32, Hk=8, D=128, page=16, q_min=1, q_max=1,
             kv_min=200, kv_max=6000, axes="128", theta=10000.0, halves=True, tree=False, fused=True, keep=False, spare=0),
        # rotate and append: drafted trees, whose tokens' positions follow their depth, some padded rows behind them
        dict(name="rope append 48 trees of up to 21", op="append", N=48, H=24, Hk=8, D=96, page=32, q_min=5, q_max=21,
             kv_min=100, kv_max=4000, axes="96", theta=500000.0, halves=True, tree=True, fused=True, keep=False, spare=37),
        # rotate and append: prompts into their pages, rotated keys kept in a row too for the prompt's own attention
        dict(name="rope append 8 prompts", op="append", N=8, H=32, Hk=8, D=128, page=64, q_min=700, q_max=4096,
             kv_min=4096, kv_max=8192, axes="128", theta=10000.0, halves=False, tree=False, fused=True, keep=True, spare=0),
        # masks and positions of a few small trees, once a step of a small batch
        dict(name="tree mask 4 trees of 8", op="mask", N=4, q_min=8, q_max=8, kv_min=300, kv_max=1200, words=1, spare=0),
        # the same for a large batch with large trees
        dict(name="tree mask 256 trees of up to 250", op="mask", N=256, q_min=60, q_max=250, kv_min=100, kv_max=20000,
             words=8, spare=100),
        # tree attention: four short sequences with eight drafted tokens each, where the latency counts
        dict(name="tree 4 of 8 tokens short", op="tree", N=4, H=32, Hk=8, D=128, page=16, q_min=8, q_max=8, kv_min=300,
             kv_max=1200, words=1, spare=0),
        # tree attention: chains of up to three drafted tokens (the smallest trees) over long caches
        dict(name="tree 32 of up to 3 tokens long", op="tree", N=32, H=40, Hk=8, D=128, page=64, q_min=1, q_max=3,
             kv_min=4000, kv_max=16384, words=1, spare=5),
        # tree attention: ordinary trees, no shared heads, ragged
        dict(name="tree 9 of up to 61 tokens", op="tree", N=9, H=24, Hk=24, D=64, page=32, q_min=7, q_max=61, kv_min=500,
             kv_max=8000, words=2, spare=19),
        # tree attention: a large batch of large trees over long caches
        dict(name="tree 16 of 64 tokens long", op="tree", N=16, H=64, Hk=8, D=128, page=64, q_min=64, q_max=64,
             kv_min=4000, kv_max=16384, words=2, spare=0),
        # prompts: a few short ones, where the latency counts
        dict(name="packed 4 short prompts", op="packed", N=4, H=8, Hk=8, D=64, q_min=17, q_max=300, left=-1, right=0,
             sinks=0, fused=False, spare=0),
        # prompts: an ordinary batch, ragged, shared heads, straight from one [q k v] projection
        dict(name="packed 12 prompts", op="packed", N=12, H=32, Hk=8, D=128, q_min=130, q_max=4001, left=-1, right=0,
             sinks=0, fused=True, spare=11),
        # prompts: one long prompt
        dict(name="packed one prompt of 16384", op="packed", N=1, H=40, Hk=8, D=128, q_min=16384, q_max=16384, left=-1,
             right=0, sinks=0, fused=False, spare=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("append", "mask", "tree", "tree", "packed", "packed"))
    D = rng.choice((64, 96, 128))
    Hk = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "append":
        H = Hk * rng.choice((1, 1, 2, 3, 4, 5, 8))
        tree = rng.random() < 0.4
        N = _log_int(rng, 1, 100)
        most = max(1, 800000 // (N * (H + 2 * Hk)))
        q_max = _log_int(rng, 1, min(most, 64 if tree else 4000))
        kv_max = rng.randint(q_max, q_max + max(1, 200000 // (N * Hk)))
        halves = rng.random() < 0.5
        step = 16 if halves else 2
        axes = [step * rng.randint(1, D // step)] if rng.random() < 0.7 or tree else [D // 2, D // 4 // step * step]
        return dict(op=op, N=N, H=H, Hk=Hk, D=D, page=page, q_min=rng.randint(1, q_max), q_max=q_max,
                    kv_min=rng.randint(q_max, kv_max), kv_max=kv_max, axes=",".join(map(str, axes)),
                    theta=rng.choice((100.0, 10000.0, 500000.0)), halves=halves, tree=tree, fused=rng.random() < 0.6,
                    keep=rng.random() < 0.4, spare=rng.randint(0, 20))
    if op == "mask":
        q_max = _log_int(rng, 1, 256)
        return dict(op=op, N=_log_int(rng, 1, 256), q_min=rng.randint(1, q_max), q_max=q_max, kv_min=q_max,
                    kv_max=rng.randint(q_max, 20000), words=rng.randint((q_max + 31) // 32, 8), spare=rng.randint(0, 40))
    if op == "tree":
        H = Hk * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
        q_max = _log_int(rng, 1, 130)
        N = _log_int(rng, 1, 40)
        kv_max = max(q_max, _log_int(rng, 20, min(16000, max(400, 250000000 // (N * H * q_max)))))
        return dict(op=op, N=N, H=H, Hk=Hk, D=D, page=page, q_min=rng.randint(1, q_max), q_max=q_max,
                    kv_min=rng.randint(q_max, kv_max), kv_max=kv_max, words=rng.randint((q_max + 31) // 32, 5),
                    spare=rng.randint(0, 9))
    H = Hk * rng.choice((1, 1, 2, 3, 4, 5, 8))
    N = _log_int(rng, 1, 60)
    q_max = _log_int(rng, 1, max(300, min(9000, int(math.sqrt(4.0e9 / (N * H))))))
    left = rng.choice((-1, -1, -1, _log_int(rng, 1, 3000) - 1))
    return dict(op=op, N=N, H=H, Hk=Hk, D=D, q_min=rng.randint(1, q_max), q_max=q_max, left=left,
                right=rng.choice((0, 0, 0, -1, _log_int(rng, 1, 300))), sinks=0 if left < 0 else rng.choice((0, 4, 130)),
                fused=rng.random() < 0.5, spare=rng.randint(0, 20))


def _spread(lo, hi, N, mix):
    """N values over lo .. hi, in mixed order."""
    return [lo + (hi - lo) * ((n * mix + N - 1) % N) // max(1, N - 1) for n in range(N)]


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence, spread over the case's ranges."""
    N = case["N"]
    q = _spread(case["q_min"], case["q_max"], N, 5 if N % 5 else 7)
    if case["op"] == "packed":
        return q, q
    return q, [max(a, b) for a, b in zip(q, _spread(case["kv_min"], case["kv_max"], N, 3 if N % 3 else 1))]


def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _freqs(case):
    return [case["theta"] ** (-2.0 * i / a) for a in _axes(case) for i in range(a // 2)]


# ------------------------------------------------------------------ inputs

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(BF16)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _qkv(case, T, gen):
    """q [T, H, D], k and v [T, Hk, D]: of one projection's rows, or tensors of their own."""
    H, Hk, D = case["H"], case["Hk"], case["D"]
    if case["fused"]:
        row = _normal((T, H + 2 * Hk, D), gen)
        return row[:, :H], row[:, H:H + Hk], row[:, H + Hk:]
    return _normal((T, H, D), gen), _normal((T, Hk, D), gen), _normal((T, Hk, D), gen)


def _parents(lengths, gen):
    """Of each drafted token the one it follows (-1: the sequence's last token), always an earlier one; the later of two
    random ones, which makes trees with long branches. [N, most]"""
    i = torch.arange(max(lengths), device="cuda", dtype=torch.float64)
    u = torch.rand((2, len(lengths), max(lengths)), generator=gen, device="cuda", dtype=torch.float64).amax(0)
    return (u * (i + 1)).floor().clamp(max=i).to(torch.int32) - 1


def _packed_rows(x, lengths):
    return torch.cat([x[n, :m] for n, m in enumerate(lengths)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, N = case["op"], case["N"]
    ql, kl = _lengths(case)
    T = sum(ql) + case["spare"]
    st = {"case": case, "T": T, "q_start": _starts(ql), "kv_len": torch.tensor(kl, dtype=torch.int32, device="cuda")}
    if op == "mask":
        rows = _packed_rows(_parents(ql, gen), ql)
        st["kv_len"] += torch.randint(0, 1000, (N,), generator=gen, device="cuda", dtype=torch.int32)
        st["parents"] = torch.cat((rows, torch.zeros(case["spare"], dtype=torch.int32, device="cuda")))
        st["mask"] = torch.zeros((T, case["words"]), dtype=torch.int32, device="cuda")
        st["pos"] = torch.zeros(T, dtype=torch.int32, device="cuda")
        return st
    H, Hk, D = case["H"], case["Hk"], case["D"]
    if op == "packed":
        st["q"], st["k"], st["v"] = _qkv(case, T, gen)
        st["out"] = torch.zeros((T, H, D), dtype=BF16, device="cuda")
        if own:
            import comm_comp_fusion_gb300 as xs
            st["ws"] = torch.empty(xs.attn_packed_workspace_size(N, T, H, Hk, D), dtype=torch.uint8, device="cuda")
        return st
    # a paged cache: every sequence's pages lie scattered in the pool
    page = case["page"]
    need = [-(-n // page) for n in kl]
    st["cols"], st["n_pages"] = max(need), sum(need) + 3
    order = torch.randperm(st["n_pages"], generator=gen, device="cuda").to(torch.int32)
    table = torch.full((N, st["cols"]), -1, dtype=torch.int32, device="cuda")
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = order[at:at + m]
        at += m
    st["table"] = table
    st["k_pages"] = _normal((st["n_pages"], page, Hk, D), gen)
    st["v_pages"] = _normal((st["n_pages"], page, Hk, D), gen)
    if op == "append":
        st["q"], st["k"], st["v"] = _qkv(case, T, gen)
        st["q_out"] = torch.zeros((T, H, D), dtype=BF16, device="cuda")
        st["k_out"] = torch.zeros((T, Hk, D), dtype=BF16, device="cuda") if case["keep"] else None
        n_axes = len(_axes(case))
        st["pos"] = None  # tokens stand at their places in the sequence
        if case["tree"] or n_axes > 1:
            pos = torch.randint(0, max(kl) + 1, (T, n_axes), generator=gen, device="cuda", dtype=torch.int32)
            if case["tree"]:  # behind the cached ones, by their depth
                depth = _plain_masks(_parents(ql, gen))[1]
                first = torch.tensor([b - a for a, b in zip(ql, kl)], device="cuda").view(N, 1)
                pos[:sum(ql), 0] = _packed_rows(first + depth, ql).to(torch.int32)
            st["pos"] = pos
        st["freqs"] = torch.tensor(_freqs(case), dtype=torch.float64, device="cuda")
        if own:
            import comm_comp_fusion_gb300 as xs
            st["axes"] = xs.RopeAxes(_axes(case), _freqs(case), halves=case["halves"])
        return st
    st["q"] = _normal((T, H, D), gen)
    st["out"] = torch.zeros((T, H, D), dtype=BF16, device="cuda")
    seen = _plain_masks(_parents(ql, gen))[0]
    words = _packed_rows(_words(seen, case["words"]), ql)
    st["mask"] = torch.cat((words, torch.zeros((case["spare"], case["words"]), dtype=torch.int32, device="cuda")))
    if own:
        import comm_comp_fusion_gb300 as xs
        st["ws"] = torch.empty(xs.attn_tree_workspace_size(N, T, H, Hk, D), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _plain_masks(parents):
    """Which tokens of its tree each token sees (itself and those it follows) [N, M, M], and its depth [N, M]."""
    M = parents.shape[1]
    j = torch.arange(M, device=parents.device)
    reach = (j.view(1, M, 1) == j).float() + (parents.unsqueeze(-1) == j).float()  # in at most one step
    for _ in range(max(0, M - 1).bit_length()):  # in at most twice as many
        reach = (torch.matmul(reach, reach) > 0).float()
    seen = reach > 0
    return seen, seen.sum(-1) - 1


def _words(seen, words):
    """Bits of 32-bit words: [N, M, M] -> [N, M, words] int32."""
    N, M, _ = seen.shape
    full = torch.zeros((N, M, words * 32), dtype=torch.int64, device=seen.device)
    full[..., :M] = seen.long()
    w = (full.view(N, M, words, 32) << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _bits(words):
    """[T, words] int32 -> [T, 32 * words] truth values."""
    at = torch.arange(32, device=words.device)
    return ((words.long().unsqueeze(-1) >> at) & 1).flatten(1) > 0


def _tokens(st):
    """Of each packed row: its sequence, its place among the new tokens, and whether it belongs to any sequence."""
    qs = st["q_start"].long()
    t = torch.arange(st["T"], device=qs.device)
    seq = (torch.searchsorted(qs, t, right=True) - 1).clamp(0, qs.numel() - 2)
    return seq, t - qs[seq], t < qs[-1]


def _plain_append(st):
    c, page = st["case"], st["case"]["page"]
    axes, dev = _axes(c), st["q"].device
    seq, i, real = _tokens(st)
    qs = st["q_start"].long()
    place = st["kv_len"].long()[seq] - (qs[seq + 1] - qs[seq]) + i
    pos = place.unsqueeze(-1) if st["pos"] is None else st["pos"]
    axis_of = torch.repeat_interleave(torch.arange(len(axes), device=dev), torch.tensor([a // 2 for a in axes], device=dev),
                                      output_size=sum(axes) // 2)
    angle = pos.double()[:, axis_of] * st["freqs"]  # [T, pairs], in 64 bits: positions may be far
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    pair = torch.arange(sum(axes) // 2, device=dev)
    begin = torch.tensor([sum(axes[:n]) for n in range(len(axes))], device=dev)[axis_of]
    dim = torch.tensor(axes, device=dev)[axis_of]
    within = pair - begin // 2
    first = begin + (within if c["halves"] else 2 * within)
    second = first + (dim // 2 if c["halves"] else 1)

    def turn(x):
        y = x.float()
        a, b = y[..., first], y[..., second]
        z = y.clone()
        z[..., first] = a * cos - b * sin
        z[..., second] = a * sin + b * cos
        return z.to(BF16)

    some = real.view(-1, 1, 1)
    q, k = turn(st["q"]), turn(st["k"])
    row = st["table"].long()[seq, (place // page).clamp(0, st["cols"] - 1)] * page + place % page
    row = torch.where(real, row, row[0])  # rows of no sequence write what row 0 writes
    for new, pool in ((k, st["k_pages"]), (st["v"], st["v_pages"])):
        pool.view(-1, c["Hk"], c["D"])[row] = torch.where(some, new, new[:1])
    done = [torch.where(some, q, st["q_out"]), st["k_pages"], st["v_pages"]]
    return done + [torch.where(some, k, st["k_out"])] if c["keep"] else done


def _plain_tree_mask(st):
    c = st["case"]
    qs, M = st["q_start"].long(), st["case"]["q_max"]
    rows = (qs[:-1].view(-1, 1) + torch.arange(M, device=qs.device)).clamp(max=st["T"] - 1)
    seen, depth = _plain_masks(st["parents"][rows])  # rows of the next sequence come behind the own ones, which none sees
    seq, i, real = _tokens(st)
    i = i.clamp(0, M - 1)
    first = st["kv_len"].long() - (qs[1:] - qs[:-1])
    mask = torch.where(real.view(-1, 1), _words(seen, c["words"])[seq, i], st["mask"])
    return mask, torch.where(real, first[seq] + depth[seq, i], st["pos"].long()).to(torch.int32)


def _softmax_product(scores, seen, v):
    """Softmax over the seen places of each row (zeros where a row sees nothing), times v."""
    s = torch.where(seen, scores, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_tree(st):
    c, page, cols = st["case"], st["case"]["page"], st["cols"]
    N, H, Hk, D = c["N"], c["H"], c["Hk"], c["D"]
    G, M = H // Hk, c["q_max"]
    qs, kl = st["q_start"].long(), st["kv_len"].long()
    first = kl - (qs[1:] - qs[:-1])
    pages = st["table"].long().clamp(min=0)
    m = torch.arange(M, device=qs.device)
    rows = (qs[:-1].view(N, 1) + m).clamp(max=st["T"] - 1)
    q = st["q"][rows].float().view(N, M, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * M, D)
    key = torch.arange(cols * page, device=qs.device)
    new = (key.view(1, -1) - first.view(N, 1))  # [N, keys]: which new token a key is, negative before them
    bits = _bits(st["mask"])[rows]              # [N, M, 32 words]
    at = new.clamp(0, bits.shape[-1] - 1).unsqueeze(1).expand(N, M, cols * page)
    seen = (new < 0).unsqueeze(1) | (bits.gather(2, at) & (new < bits.shape[-1]).unsqueeze(1))
    seen = seen & (key < kl.view(N, 1)).unsqueeze(1)
    o = torch.empty((N, Hk, G, M, D), device=q.device)
    for h in range(Hk):  # one key head's scores at a time
        k = st["k_pages"][:, :, h][pages].view(N, cols * page, D).float()
        v = st["v_pages"][:, :, h][pages].view(N, cols * page, D).float()
        scores = (torch.matmul(q[:, h], k.transpose(-1, -2)) * D ** -0.5).view(N, G, M, cols * page)
        o[:, h] = _softmax_product(scores, seen.unsqueeze(1), v.unsqueeze(1))
    o = o.permute(0, 3, 1, 2, 4).reshape(N, M, H, D).to(BF16)
    seq, i, real = _tokens(st)
    return torch.where(real.view(-1, 1, 1), o[seq, i.clamp(0, M - 1)], st["out"])


def _seen(i, j, left, right, sinks):
    """Whether token i sees token j: within the window to the left or among the sinks, and not past its right end."""
    ok = torch.ones_like(i - j, dtype=torch.bool)
    if left >= 0:
        ok = ok & ((j >= i - left) | (j < sinks))
    if right >= 0:
        ok = ok & (j <= i + right)
    return ok


def _plain_packed(st):
    c = st["case"]
    Hk, D, G = c["Hk"], c["D"], c["H"] // c["Hk"]
    done, t = [], 0
    for n in _lengths(c)[0]:
        q = st["q"][t:t + n].float().view(n, Hk, G, D).permute(1, 2, 0, 3)  # [Hk, G, n, D]
        k, v = (st[x][t:t + n].float().transpose(0, 1) for x in "kv")       # [Hk, n, D]
        i = torch.arange(n, device=q.device)
        seen = _seen(i.view(-1, 1), i.view(1, -1), c["left"], c["right"], c["sinks"])
        o = []
        for h in range(Hk):  # one key head's scores at a time
            scores = torch.matmul(q[h], k[h].T) * D ** -0.5
            o.append(_softmax_product(scores, seen, v[h]))
        done.append(torch.stack(o).permute(2, 0, 1, 3).reshape(n, c["H"], D).to(BF16))
        t += n
    return torch.cat(done + [st["out"][t:]])


_PLAIN = {"append": _plain_append, "mask": _plain_tree_mask, "tree": _plain_tree, "packed": _plain_packed}


# ------------------------------------------------------------------ the library

def _own(st):
    import comm_comp_fusion_gb300 as xs
    c, T = st["case"], st["T"]
    if c["op"] == "append":
        xs.cache_append_rope(st["q"], st["k"], st["v"], st["q_out"], st["k_pages"], st["v_pages"], st["table"],
                             st["q_start"], st["kv_len"], c["N"], T, c["H"], c["Hk"], c["D"], c["page"], st["n_pages"],
                             st["cols"], st["axes"], pos=st["pos"], k_out=st["k_out"])
        done = [st["q_out"], st["k_pages"], st["v_pages"]]
        return done + [st["k_out"]] if c["keep"] else done
    if c["op"] == "mask":
        xs.tree_mask(st["parents"], st["q_start"], st["kv_len"], st["mask"], st["pos"], c["N"], T, c["words"])
        return st["mask"], st["pos"]
    if c["op"] == "tree":
        xs.attn_tree(st["q"], st["k_pages"], st["v_pages"], st["table"], st["q_start"], st["kv_len"], st["mask"], st["out"],
                     c["N"], T, c["H"], c["Hk"], c["D"], c["page"], st["n_pages"], st["cols"], c["words"], c["D"] ** -0.5,
                     st["ws"])
        return st["out"]
    xs.attn_packed(st["q"], st["k"], st["v"], st["q_start"], st["out"], c["N"], T, c["H"], c["Hk"], c["D"], c["D"] ** -0.5,
                   c["left"], c["right"], c["sinks"], st["ws"])
    return st["out"]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def _pairs_seen(n, left, right, sinks):
    """Sum over the tokens of a sequence of n of the keys that each sees."""
    total = 0
    for p in range(n):
        hi = n - 1 if right < 0 else min(n - 1, p + right)
        lo = 0 if left < 0 else max(0, p - left)
        total += hi - lo + 1 + max(0, min(sinks, lo))
    return total


def work(case):
    ql, kl = _lengths(case)
    T = sum(ql)
    if case["op"] == "mask":  # parents in, masks and positions out
        return {"bytes": T * (8 + 4 * case["words"]), "flops": 0}
    H, Hk, D = case["H"], case["Hk"], case["D"]
    if case["op"] == "append":
        moved = 2 * H + 4 * Hk + (Hk if case["keep"] else 0)
        n_pos = len(_axes(case)) if case["tree"] or len(_axes(case)) > 1 else 0
        return {"bytes": T * (2 * moved * D + 4 * n_pos), "flops": 3 * T * (H + Hk) * sum(_axes(case))}
    if case["op"] == "tree":  # all cached tokens, and of the drafted ones about the depth of a random tree
        seen = sum(a * (b - a + min(a, 1 + 2 * math.log(a))) for a, b in zip(ql, kl))
        return {"bytes": T * (4 * H * D + 4 * case["words"]) + 4 * sum(kl) * Hk * D, "flops": int(4 * seen * H * D)}
    seen = sum(_pairs_seen(n, case["left"], case["right"], case["sinks"]) for n in ql)
    return {"bytes": T * (4 * H + 4 * Hk) * D, "flops": 4 * seen * H * D}


# ------------------------------------------------------------------ 64 bits

def _exact_append(case, st, ql, kl):
    page, dev = case["page"], st["q"].device
    real = sum(ql)
    if st["pos"] is None:
        place = torch.cat([torch.arange(b - a, b, device=dev) for a, b in zip(ql, kl)]).view(-1, 1)
    else:
        place = st["pos"][:real]

    def turn(x):
        y, begin, done, n = x[:real].double(), 0, [], 0
        for axis, dim in enumerate(_axes(case)):
            f = torch.tensor(_freqs(case)[n:n + dim // 2], dtype=torch.float64, device=dev)
            n += dim // 2
            angle = place[:, axis].double().unsqueeze(-1) * f
            unit = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
            part = y[..., begin:begin + dim]
            two = part.unflatten(-1, (2, dim // 2)).transpose(-1, -2) if case["halves"] else part.unflatten(-1, (dim // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(two.contiguous()) * unit)
            done.append((z.transpose(-1, -2) if case["halves"] else z).flatten(-2))
            begin += dim
        return torch.cat(done + [y[..., begin:]], -1)

    q, k = turn(st["q"]), turn(st["k"])
    kp, vp, t = st["k_pages"].double(), st["v_pages"].double(), 0
    for n in range(case["N"]):
        at = torch.arange(kl[n] - ql[n], kl[n], device=dev)
        ids = st["table"][n].long()[at // page]
        kp[ids, at % page] = k[t:t + ql[n]]
        vp[ids, at % page] = st["v"][t:t + ql[n]].double()
        t += ql[n]
    done = [torch.cat((q, st["q_out"][real:].double())), kp, vp]
    return done + [torch.cat((k, st["k_out"][real:].double()))] if case["keep"] else done


def _exact_mask(case, st, ql, kl):
    """Token by token, on the host."""
    parents, mask, pos = st["parents"].tolist(), st["mask"].tolist(), st["pos"].tolist()
    t = 0
    for a, b in zip(ql, kl):
        bits, depth = [], []
        for i in range(a):
            p = parents[t + i]
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
            for w in range(case["words"]):
                x = bits[i] >> 32 * w & 0xFFFFFFFF
                mask[t + i][w] = x - (1 << 32) if x >> 31 else x
            pos[t + i] = b - a + depth[i]
        t += a
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (mask, pos))


def _rows_exact(q, k, v, hide, scale):
    """Rows q [g, m, D] over keys k, v [keys, D], without those that `hide` [m, keys] names."""
    w = (q @ k.T * scale).masked_fill(hide, -math.inf).softmax(-1)
    return w.nan_to_num(0.0) @ v


def exact(case, seed):
    st = prepare(case, seed)
    ql, kl = _lengths(case)
    if case["op"] == "append":
        return _exact_append(case, st, ql, kl)
    if case["op"] == "mask":
        return _exact_mask(case, st, ql, st["kv_len"].tolist())
    G, scale, t = case["H"] // case["Hk"], case["D"] ** -0.5, 0
    out = st["out"].double()
    for n in range(case["N"]):
        a, b = ql[n], kl[n]
        if case["op"] == "tree":
            ids = st["table"][n, :-(-b // case["page"])].long()
            k, v = (st[x][ids].flatten(0, 1)[:b] for x in ("k_pages", "v_pages"))
            words = st["mask"][t:t + a].long()
            drafted = torch.stack([words[:, j >> 5] >> (j & 31) & 1 for j in range(a)], -1)
            hide = torch.cat((torch.zeros((a, b - a), dtype=torch.bool, device=k.device), drafted == 0), -1)
        else:
            k, v = st["k"][t:t + a], st["v"][t:t + a]
        for h in range(case["Hk"]):
            kh, vh = k[:, h].double(), v[:, h].double()
            q = st["q"][t:t + a, h * G:(h + 1) * G].double().transpose(0, 1)
            for m in range(0, a, 2048):
                rows = slice(m, min(m + 2048, a))
                if case["op"] == "tree":
                    o = _rows_exact(q[:, rows], kh, vh, hide[rows], scale)
                else:  # the keys that any of these rows sees, but for the sinks before them
                    i = torch.arange(rows.start, rows.stop, device=k.device).view(-1, 1)
                    hi = a if case["right"] < 0 else min(a, rows.stop + case["right"])
                    lo = 0 if case["left"] < 0 or case["sinks"] else max(0, rows.start - case["left"])
                    j = torch.arange(lo, hi, device=k.device).view(1, -1)
                    gone = torch.zeros((rows.stop - rows.start, hi - lo), dtype=torch.bool, device=k.device)
                    if case["right"] >= 0:
                        gone |= j - i > case["right"]
                    if case["left"] >= 0:
                        gone |= (i - j > case["left"]) & (j >= case["sinks"])
                    o = _rows_exact(q[:, rows], kh[lo:hi], vh[lo:hi], gone, scale)
                out[t + rows.start:t + rows.stop, h * G:(h + 1) * G] = o.transpose(0, 1)
        t += a
    return out
