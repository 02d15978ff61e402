"""The operators around the fused attention, as a program calls them: rotary positions with several axes,
attention through a sliding window with sinks, and the paged key/value cache of a serving loop (writing new tokens into
its pages, attention of a chunk of new tokens over it).

`run` computes each operator in plain torch operations; with `own` set it calls the library. `exact` gives the same
results in 64 bits."""
import math

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # rotary: q and k of eight single new tokens of a causal model (one axis, pairs half a head apart)
        dict(name="rope 8 single tokens", op="rope", B=8, S=1, H=32, Hk=8, D=128, P=1, axes="128", theta=10000.0,
             halves=True, inverse=False, seq_in=False, seq_out=False, far=131072),
        # rotary: the DiT workload's q and k, (time, height, width), on their way from the sequence to the head partition
        dict(name="rope DiT S=4096 to heads", op="rope", B=1, S=4096, H=24, Hk=24, D=128, P=8, axes="44,42,42",
             theta=10000.0, halves=False, inverse=False, seq_in=True, seq_out=False, far=0),
        # rotary: the largest workload, turned back (the gradient of q and k), in the sequence partition
        dict(name="rope B=2 S=16384 H=40 back", op="rope", B=2, S=16384, H=40, Hk=40, D=128, P=4, axes="32,48,48",
             theta=256.0, halves=True, inverse=True, seq_in=True, seq_out=True, far=0),
        # window: a short ragged causal sequence with four sinks
        dict(name="window S=1000 causal sinks", op="window", B=1, S=1000, H=8, D=64, P=4, left=255, right=0, sinks=4,
             a2a=False),
        # window: the DiT workload with every token seeing its neighbours on both sides, scattered to the ranks
        dict(name="window DiT S=4096 two-sided", op="window", B=1, S=4096, H=24, D=128, P=8, left=512, right=512,
             sinks=0, a2a=True),
        # window: a long causal sequence, 4096 keys and the first 64
        dict(name="window S=16384 causal sinks", op="window", B=1, S=16384, H=24, D=128, P=8, left=4095, right=0,
             sinks=64, a2a=False),
        # cache: one new token of each of 64 sequences
        dict(name="append 64 single tokens", op="append", N=64, Hk=8, D=128, page=16, q_min=1, q_max=1, kv_min=200,
             kv_max=2000, spare=3),
        # cache: prompts written into their pages, ragged
        dict(name="append 8 prompts", op="append", N=8, Hk=8, D=128, page=64, q_min=700, q_max=4096, kv_min=4096,
             kv_max=8192, spare=0),
        # paged attention: one new token of four short sequences, where the latency counts
        dict(name="paged 4 single tokens short", op="paged", N=4, H=32, Hk=8, D=128, page=16, q_min=1, q_max=1,
             kv_min=300, kv_max=1200, left=-1, right=0, sinks=0, spare=0),
        # paged attention: one new token of 32 long sequences
        dict(name="paged 32 single tokens long", op="paged", N=32, H=64, Hk=8, D=128, page=64, q_min=1, q_max=1,
             kv_min=4000, kv_max=32768, left=-1, right=0, sinks=0, spare=0),
        # paged attention: single tokens and prompt chunks in one batch, a window with sinks, padded rows at the end
        dict(name="paged mixed batch window", op="paged", N=9, H=24, Hk=24, D=64, page=32, q_min=1, q_max=500,
             kv_min=500, kv_max=8000, left=2047, right=0, sinks=4, spare=19),
        # paged attention: two long prompt chunks over a long cache
        dict(name="paged 2 chunks of 2048", op="paged", N=2, H=32, Hk=8, D=128, page=128, q_min=2048, q_max=2048,
             kv_min=16000, kv_max=18001, left=-1, right=0, sinks=0, spare=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("rope", "window", "append", "paged", "paged"))
    if op == "rope":
        D = rng.choice((64, 96, 128, 256))
        P = rng.choice((1, 2, 4, 8))
        Hl = rng.randint(1, 5)
        Hk = P * Hl
        H = Hk * rng.choice((1, 1, 2, 3))
        B = rng.randint(1, 3)
        Sl = _log_int(rng, 1, max(1, (1 << 26) // (P * B * (H + Hk) * D)))
        halves = rng.random() < 0.5
        step = 16 if halves else 2
        n = rng.randint(1, 3)
        axes, left = [], D
        for _ in range(n):
            a = step * rng.randint(1, max(1, left // step // (n - len(axes))))
            axes.append(a)
            left -= a
        return dict(op=op, B=B, S=P * Sl, H=H, Hk=Hk, D=D, P=P, axes=",".join(map(str, axes)),
                    theta=rng.choice((100.0, 256.0, 10000.0, 500000.0)), halves=halves, inverse=rng.random() < 0.4,
                    seq_in=rng.random() < 0.5, seq_out=rng.random() < 0.5, far=rng.choice((0, 0, 1000, 1000000)))
    if op == "window":
        D = rng.choice((64, 96, 128))
        P = rng.choice((1, 2, 4))
        H = P * rng.randint(1, 4)
        B = rng.randint(1, 2)
        S = P * _log_int(rng, 1, 8192 // P)
        left = _log_int(rng, 1, 6000) - 1
        return dict(op=op, B=B, S=S, H=H, D=D, P=P, left=left, right=rng.choice((0, 0, left, _log_int(rng, 1, 2000))),
                    sinks=rng.choice((0, 1, 4, 64, 200)), a2a=rng.random() < 0.5)
    D = rng.choice((64, 96, 128))
    page = rng.choice((16, 32, 64, 128, 256))
    Hk = rng.choice((1, 2, 3, 4, 8))
    if op == "append":
        N = _log_int(rng, 1, 100)
        kv_max = _log_int(rng, 20, 400000 // (N * Hk) + 20)
        q_max = _log_int(rng, 1, min(kv_max, 3000))
        return dict(op=op, N=N, Hk=Hk, D=D, page=page, q_min=rng.randint(1, q_max), q_max=q_max,
                    kv_min=rng.randint(q_max, kv_max), kv_max=kv_max, spare=rng.randint(0, 20))
    H = Hk * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    decode = rng.random() < 0.5
    N = _log_int(rng, 1, 64 if decode else 6)
    kv_max = _log_int(rng, 20, 20000 if decode else 9000)
    q_max = rng.choice((1, 1, 1, 4)) if decode else _log_int(rng, 2, min(kv_max, 900))
    left = rng.choice((-1, -1, _log_int(rng, 1, 5000) - 1))
    return dict(op=op, N=N, H=H, Hk=Hk, D=D, page=page, q_min=rng.randint(1, q_max), q_max=q_max,
                kv_min=rng.randint(q_max, kv_max), kv_max=kv_max, left=left,
                right=rng.choice((0, 0, 0, -1, _log_int(rng, 1, 300))), sinks=0 if left < 0 else rng.choice((0, 4, 130)),
                spare=rng.randint(0, 9))


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence, spread over the case's ranges."""
    N = case["N"]

    def spread(lo, hi, mix):
        return [lo + (hi - lo) * ((n * mix + N - 1) % N) // max(1, N - 1) for n in range(N)]

    q = spread(case["q_min"], case["q_max"], 5 if N % 5 else 7)
    kv = [max(a, b) for a, b in zip(q, spread(case["kv_min"], case["kv_max"], 3 if N % 3 else 1))]
    return q, kv


def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _freqs(case):
    return [case["theta"] ** (-2.0 * i / a) for a in _axes(case) for i in range(a // 2)]


# ------------------------------------------------------------------ inputs

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(BF16)


def _head_shape(B, S, H, D, P):
    return (P, B, S, H // P, D)


def _seq_shape(B, S, H, D, P):
    return (P, B, S // P, H, D)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "rope":
        B, S, H, Hk, D, P = (case[k] for k in ("B", "S", "H", "Hk", "D", "P"))
        shape_in = _seq_shape if case["seq_in"] else _head_shape
        shape_out = _seq_shape if case["seq_out"] else _head_shape
        st["q"], st["k"] = _normal(shape_in(B, S, H, D, P), gen), _normal(shape_in(B, S, Hk, D, P), gen)
        n = len(_axes(case))
        if n == 1:  # the tokens' places in their sequences, each from a start of its own
            first = torch.randint(0, case["far"] + 1, (B, 1, 1), generator=gen, device="cuda")
            pos = first + torch.arange(S, device="cuda").view(1, S, 1)
        else:  # frames of a grid, rows and columns within each
            w = max(1, int(math.sqrt(S / 8)))
            s = torch.arange(S, device="cuda")
            first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda")
            grid = [first + (s // (w * w)).view(1, S), ((s // w) % w).expand(B, S), (s % w).expand(B, S)]
            pos = torch.stack(grid[:n], -1)
        st["pos"] = pos.to(torch.int32).contiguous()
        st["freqs"] = torch.tensor(_freqs(case), dtype=torch.float64, device="cuda")
        if own:
            import comm_comp_fusion_gb300 as xs
            st["axes"] = xs.RopeAxes(_axes(case), _freqs(case), halves=case["halves"])
            st["q_out"] = torch.empty(shape_out(B, S, H, D, P), dtype=BF16, device="cuda")
            st["k_out"] = torch.empty(shape_out(B, S, Hk, D, P), dtype=BF16, device="cuda")
        return st
    if case["op"] == "window":
        B, S, H, D, P = (case[k] for k in ("B", "S", "H", "D", "P"))
        for name in "qkv":
            st[name] = _normal(_head_shape(B, S, H, D, P), gen)
        if own:
            import comm_comp_fusion_gb300 as xs
            st["out"] = torch.empty((_seq_shape if case["a2a"] else _head_shape)(B, S, H, D, P), dtype=BF16, device="cuda")
            st["ws"] = torch.empty(xs.attn_window_workspace_size(B, S, H, D, P), dtype=torch.uint8, device="cuda")
        return st
    # a paged cache: every sequence's pages lie scattered in the pool
    N, Hk, D, page = (case[k] for k in ("N", "Hk", "D", "page"))
    ql, kl = _lengths(case)
    T = sum(ql) + case["spare"]
    need = [-(-n // page) for n in kl]
    cols, n_pages = max(need), sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    starts = [sum(need[:n]) for n in range(N)]
    idx = torch.tensor(starts, device="cuda").view(N, 1) + torch.arange(cols, device="cuda").view(1, cols)
    held = torch.arange(cols, device="cuda").view(1, cols) < torch.tensor(need, device="cuda").view(N, 1)
    table = order[idx.clamp(max=n_pages - 1)]
    st["table"] = torch.where(held, table, torch.full_like(table, -1)).contiguous()
    st["q_start"] = torch.tensor([sum(ql[:n]) for n in range(N + 1)], dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(kl, dtype=torch.int32, device="cuda")
    st["T"], st["n_pages"], st["cols"] = T, n_pages, cols
    st["k_pages"] = _normal((n_pages, page, Hk, D), gen)
    st["v_pages"] = _normal((n_pages, page, Hk, D), gen)
    if case["op"] == "append":
        st["k"], st["v"] = _normal((T, Hk, D), gen), _normal((T, Hk, D), gen)
        return st
    st["q"] = _normal((T, case["H"], D), gen)
    st["out"] = torch.zeros((T, case["H"], D), dtype=BF16, device="cuda")
    if own:
        import comm_comp_fusion_gb300 as xs
        st["ws"] = torch.empty(xs.attn_paged_workspace_size(N, T, case["H"], Hk, D), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _from_layout(x, seq):
    """[P, B, ...] of either partition -> [B, S, H, D]."""
    P, B, s, h, D = x.shape
    return x.permute(1, 0, 2, 3, 4).reshape(B, P * s, h, D) if seq else x.permute(1, 2, 0, 3, 4).reshape(B, s, P * h, D)


def _to_layout(x, P, seq):
    B, S, H, D = x.shape
    y = x.view(B, P, S // P, H, D).permute(1, 0, 2, 3, 4) if seq else x.view(B, S, P, H // P, D).permute(2, 0, 1, 3, 4)
    return y.contiguous()


def _plain_rope(st):
    c = st["case"]
    axes, dev = _axes(c), st["q"].device
    axis_of = torch.repeat_interleave(torch.arange(len(axes), device=dev), torch.tensor([a // 2 for a in axes], device=dev),
                                      output_size=sum(axes) // 2)
    angle = st["pos"].double()[..., axis_of] * st["freqs"]  # [B, S, pairs], in 64 bits: positions may be far
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    if c["inverse"]:
        sin = -sin
    i = torch.arange(sum(axes) // 2, device=dev)
    begin = torch.tensor([sum(axes[:n]) for n in range(len(axes))], device=dev)[axis_of]
    dim = torch.tensor(axes, device=dev)[axis_of]
    within = i - begin // 2
    first = begin + (within if c["halves"] else 2 * within)
    second = first + (dim // 2 if c["halves"] else 1)

    def turn(x):
        y = _from_layout(x, c["seq_in"]).float()
        a, b = y[..., first], y[..., second]
        z = y.clone()
        z[..., first] = a * cos - b * sin
        z[..., second] = a * sin + b * cos
        return _to_layout(z.to(BF16), c["P"], c["seq_out"])

    return turn(st["q"]), turn(st["k"])


def _softmax_product(scores, seen, v):
    """Softmax over the seen places of each row (zeros where a row sees nothing), times v."""
    s = torch.where(seen, scores, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))


def _seen(pos, key, left, right, sinks):
    """Whether the token at `pos` sees key place `key`: within the window to the left or among the sinks, and not
    past the window's right end."""
    ok = torch.ones_like(pos - key, dtype=torch.bool)
    if left >= 0:
        ok = ok & ((key >= pos - left) | (key < sinks))
    if right >= 0:
        ok = ok & (key <= pos + right)
    return ok


def _plain_window(st):
    c = st["case"]
    q, k, v = (_from_layout(st[n], False).float().transpose(1, 2) for n in "qkv")  # [B, H, S, D]
    i = torch.arange(c["S"], device=q.device)
    scores = torch.matmul(q, k.transpose(-1, -2)) * c["D"] ** -0.5
    o = _softmax_product(scores, _seen(i.view(-1, 1), i.view(1, -1), c["left"], c["right"], c["sinks"]), v)
    return _to_layout(o.to(BF16).transpose(1, 2), c["P"], c["a2a"])


def _tokens(st):
    """Of each packed row: its sequence, its place among the new tokens, and whether it belongs to any sequence."""
    qs = st["q_start"].long()
    t = torch.arange(st["T"], device=qs.device)
    seq = (torch.searchsorted(qs, t, right=True) - 1).clamp(0, qs.numel() - 2)
    return seq, t - qs[seq], t < qs[-1]


def _plain_append(st):
    c, page = st["case"], st["case"]["page"]
    seq, i, real = _tokens(st)
    qs = st["q_start"].long()
    place = st["kv_len"].long()[seq] - (qs[seq + 1] - qs[seq]) + i
    row = st["table"].long()[seq, (place // page).clamp(0, st["cols"] - 1)] * page + place % page
    row = torch.where(real, row, row[0])  # rows of no sequence write what row 0 writes
    for new, pool in ((st["k"], st["k_pages"]), (st["v"], st["v_pages"])):
        pool.view(-1, c["Hk"], c["D"])[row] = torch.where(real.view(-1, 1, 1), new, new[:1])
    return st["k_pages"], st["v_pages"]


def _plain_paged(st):
    c, page, cols = st["case"], st["case"]["page"], st["cols"]
    N, H, Hk, D = c["N"], c["H"], c["Hk"], c["D"]
    G, M = H // Hk, c["q_max"]
    qs, kl = st["q_start"].long(), st["kv_len"].long()
    ql = qs[1:] - qs[:-1]
    pages = st["table"].long().clamp(min=0)
    k = st["k_pages"][pages].view(N, cols * page, Hk, D).float().transpose(1, 2)  # [N, Hk, keys, D]
    v = st["v_pages"][pages].view(N, cols * page, Hk, D).float().transpose(1, 2)
    m = torch.arange(M, device=qs.device)
    q = st["q"][(qs[:-1].view(N, 1) + m).clamp(max=st["T"] - 1)].float()  # [N, M, H, D]
    q = q.view(N, M, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * M, D)
    scores = (torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5).view(N, Hk, G, M, cols * page)
    key = torch.arange(cols * page, device=qs.device).view(1, 1, -1)
    pos = (kl - ql).view(N, 1, 1) + m.view(1, M, 1)
    seen = _seen(pos, key, c["left"], c["right"], c["sinks"]) & (key < kl.view(N, 1, 1))
    o = _softmax_product(scores, seen.view(N, 1, 1, M, cols * page), v.unsqueeze(2))  # [N, Hk, G, M, D]
    o = o.permute(0, 3, 1, 2, 4).reshape(N, M, H, D).to(BF16)
    seq, i, real = _tokens(st)
    return torch.where(real.view(-1, 1, 1), o[seq, i.clamp(0, M - 1)], st["out"])


_PLAIN = {"rope": _plain_rope, "window": _plain_window, "append": _plain_append, "paged": _plain_paged}


# ------------------------------------------------------------------ the library

def _own(st):
    import comm_comp_fusion_gb300 as xs
    c = st["case"]
    if c["op"] == "rope":
        xs.rope(st["q"], st["k"], st["q_out"], st["k_out"], st["pos"], c["B"], c["S"], c["H"], c["Hk"], c["D"], c["P"],
                st["axes"], seq_in=c["seq_in"], seq_out=c["seq_out"], inverse=c["inverse"])
        return st["q_out"], st["k_out"]
    if c["op"] == "window":
        call = xs.attn_window_a2a if c["a2a"] else xs.attn_window
        call(st["q"], st["k"], st["v"], st["out"], c["B"], c["S"], c["H"], c["D"], c["P"], c["D"] ** -0.5, c["left"],
             c["right"], c["sinks"], st["ws"])
        return st["out"]
    if c["op"] == "append":
        xs.cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["q_start"], st["kv_len"], c["N"],
                        st["T"], c["Hk"], c["D"], c["page"], st["n_pages"], st["cols"])
        return st["k_pages"], st["v_pages"]
    xs.attn_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["q_start"], st["kv_len"], st["out"], c["N"],
                  st["T"], c["H"], c["Hk"], c["D"], c["page"], st["n_pages"], st["cols"], c["D"] ** -0.5, c["left"],
                  c["right"], c["sinks"], st["ws"])
    return st["out"]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def _pairs_seen(pos0, n, keys, left, right, sinks):
    """Sum over the tokens at pos0 .. pos0+n-1 of the keys each sees, and the keys that any of them sees."""
    total = 0
    for p in range(pos0, pos0 + n):
        hi = keys - 1 if right < 0 else min(keys - 1, p + right)
        lo = 0 if left < 0 else max(0, p - left)
        s = min(sinks, lo, hi + 1)
        total += max(0, hi - lo + 1) + max(0, s)
    hi = keys - 1 if right < 0 else min(keys - 1, pos0 + n - 1 + right)
    lo = 0 if left < 0 else max(0, pos0 - left)
    return total, max(0, hi - lo + 1) + max(0, min(sinks, lo))


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        n = case["B"] * case["S"] * (case["H"] + case["Hk"])
        rot = sum(_axes(case))
        return {"bytes": n * D * 4 + case["B"] * case["S"] * 4 * len(_axes(case)), "flops": 3 * n * rot}
    if case["op"] == "window":
        heads = case["B"] * case["H"]
        seen, _ = _pairs_seen(0, case["S"], case["S"], case["left"], case["right"], case["sinks"])
        return {"bytes": heads * case["S"] * D * 8, "flops": 4 * heads * seen * D}
    ql, kl = _lengths(case)
    if case["op"] == "append":
        return {"bytes": 8 * sum(ql) * case["Hk"] * D, "flops": 0}
    seen = [_pairs_seen(b - a, a, b, case["left"], case["right"], case["sinks"]) for a, b in zip(ql, kl)]
    return {"bytes": 4 * sum(ql) * case["H"] * D + 4 * sum(s[1] for s in seen) * case["Hk"] * D,
            "flops": 4 * sum(s[0] for s in seen) * case["H"] * D}


# ------------------------------------------------------------------ 64 bits

def _exact_rope(case, st):
    def turn(x):
        y = _from_layout(x, case["seq_in"]).double()
        begin, done, n = 0, [], 0
        for axis, dim in enumerate(_axes(case)):
            f = torch.tensor(_freqs(case)[n:n + dim // 2], dtype=torch.float64, device=y.device)
            n += dim // 2
            angle = st["pos"][..., axis].double().unsqueeze(-1) * f * (-1.0 if case["inverse"] else 1.0)
            unit = torch.polar(torch.ones_like(angle), angle).unsqueeze(2)
            part = y[..., begin:begin + dim]
            two = part.unflatten(-1, (2, dim // 2)).transpose(-1, -2) if case["halves"] else part.unflatten(-1, (dim // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(two.contiguous()) * unit)
            done.append((z.transpose(-1, -2) if case["halves"] else z).flatten(-2))
            begin += dim
        done.append(y[..., begin:])
        return _to_layout(torch.cat(done, -1), case["P"], case["seq_out"])

    return turn(st["q"]), turn(st["k"])


def _exact_rows(q, k, v, pos, keys, case):
    """Rows q [g, m, D] at places pos [m] over keys 0 .. keys-1 of k, v [keys, D], in blocks of rows."""
    out = torch.zeros_like(q)
    left, right, sinks = case["left"], case["right"], case["sinks"]
    for a in range(0, q.shape[1], 1024):
        p = pos[a:a + 1024]
        first, last = int(p[0]), int(p[-1])
        lo = 0 if left < 0 else max(0, first - left)
        hi = keys if right < 0 else min(keys, last + right + 1)
        at = torch.cat((torch.arange(0, min(sinks, lo, max(hi, 0)), device=q.device),
                        torch.arange(lo, max(hi, lo), device=q.device)))
        if not at.numel():
            continue
        d = at.view(1, -1) - p.view(-1, 1)
        hide = torch.zeros_like(d, dtype=torch.bool)
        if right >= 0:
            hide |= d > right
        if left >= 0:
            hide |= (d < -left) & (at.view(1, -1) >= sinks)
        w = (q[:, a:a + 1024] @ k[at].T * case["D"] ** -0.5).masked_fill(hide, -math.inf).softmax(-1)
        out[:, a:a + 1024] = w.nan_to_num(0.0) @ v[at]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    if case["op"] == "window":
        q, k, v = (_from_layout(st[n], False).double() for n in "qkv")
        pos = torch.arange(case["S"], device=q.device)
        o = torch.empty_like(q)
        for b in range(case["B"]):
            for h in range(case["H"]):
                o[b, :, h] = _exact_rows(q[b, :, h].unsqueeze(0), k[b, :, h], v[b, :, h], pos, case["S"], case)[0]
        return _to_layout(o, case["P"], case["a2a"])
    ql, kl = _lengths(case)
    page, t = case["page"], 0
    if case["op"] == "append":
        k, v = st["k_pages"].double(), st["v_pages"].double()
        for n in range(case["N"]):
            place = torch.arange(kl[n] - ql[n], kl[n], device=k.device)
            at = st["table"][n].long()[place // page]
            k[at, place % page] = st["k"][t:t + ql[n]].double()
            v[at, place % page] = st["v"][t:t + ql[n]].double()
            t += ql[n]
        return k, v
    G = case["H"] // case["Hk"]
    out = st["out"].double()
    for n in range(case["N"]):
        ids = st["table"][n, :-(-kl[n] // page)].long()
        k, v = (st[x][ids].flatten(0, 1)[:kl[n]] for x in ("k_pages", "v_pages"))
        pos = torch.arange(kl[n] - ql[n], kl[n], device=k.device)
        for h in range(case["Hk"]):
            q = st["q"][t:t + ql[n], h * G:(h + 1) * G].double().transpose(0, 1)
            o = _exact_rows(q, k[:, h].double(), v[:, h].double(), pos, kl[n], case)
            out[t:t + ql[n], h * G:(h + 1) * G] = o.transpose(0, 1)
        t += ql[n]
    return out
