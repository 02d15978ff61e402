"""64-bit references and derived tolerances for the rotary, window and paged-cache tests (numpy, no library code)."""
import numpy as np

import xsgen


def bf16(rng, shape, sigma=1.0):
    """N(0, sigma) rounded to bf16: (uint16 bits, float64 values)."""
    import torch
    t = torch.from_numpy(np.asarray(rng.standard_normal(shape) * sigma, dtype=np.float32)).to(torch.bfloat16)
    bits = t.view(torch.int16).numpy().view(np.uint16)
    return bits, xsgen.bf16_bits_to_f32(bits).astype(np.float64)


def values(bits):
    return xsgen.bf16_bits_to_f32(np.asarray(bits)).astype(np.float64)


def seen_mask(pos, keys, left, right, sinks):
    """[rows, keys]: which keys the tokens at places `pos` see."""
    i, j = np.asarray(pos).reshape(-1, 1), np.arange(keys).reshape(1, -1)
    m = np.ones((i.shape[0], keys), dtype=bool)
    if right >= 0:
        m &= j <= i + right
    if left >= 0:
        m &= (j >= i - left) | (j < sinks)
    return m


def attend(q, k, v, seen, scale):
    """One head in 64 bits: (out, bound). q [rows, D], k and v [keys, D].

    The bound on a bf16 result's error, per element: the output's own rounding, half a step, 2^-8 |o|; the weights'
    rounding to bf16 before the product with V, at most 2^-8 each, so 2^-8 sum_j w_j |v_j|; and the scores' fp32 sums, off
    by at most 2^-18 of scale sum |q k| (D <= 256 terms, each rounded at 2^-23 or truncated at 2^-22, plus the
    exponential's 2^-22), which changes each weight and their sum by twice that share."""
    rows, D = q.shape
    if k.shape[0] == 0:
        return np.zeros((rows, D)), np.zeros((rows, D))
    s = np.where(seen, (q @ k.T) * scale, -np.inf)
    top = s.max(-1, keepdims=True)
    e = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = e.sum(-1, keepdims=True)
    w = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
    o, a = w @ v, w @ np.abs(v)
    delta = 2.0 ** -18 * np.where(seen, (np.abs(q) @ np.abs(k).T) * scale, 0.0).max(-1, keepdims=True)
    return o, 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * delta) * a + 1e-30


def check(got, ref, bound, what=""):
    got = values(got)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (f"{what}: {np.count_nonzero(over > 0)} of {over.size} values are off by more than their bound, "
                               f"the worst by {over.max():.3e} at {np.unravel_index(over.argmax(), over.shape)}")


def head_to_tokens(x):
    """Head-partitioned [P][B][S][Hl][D] -> [B][S][H][D]."""
    P, B, S, Hl, D = x.shape
    return x.transpose(1, 2, 0, 3, 4).reshape(B, S, P * Hl, D)


def tokens_to_head(x, P):
    B, S, H, D = x.shape
    return np.ascontiguousarray(x.reshape(B, S, P, H // P, D).transpose(2, 0, 1, 3, 4))


def seq_to_tokens(x):
    """Sequence-partitioned [P][B][Sl][H][D] -> [B][S][H][D]."""
    P, B, Sl, H, D = x.shape
    return x.transpose(1, 0, 2, 3, 4).reshape(B, P * Sl, H, D)


def tokens_to_seq(x, P):
    B, S, H, D = x.shape
    return np.ascontiguousarray(x.reshape(B, P, S // P, H, D).transpose(1, 0, 2, 3, 4))
