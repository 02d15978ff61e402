"""Empty calls (no batch, no token, no sequence) with tensors, which have no address when they hold nothing: fine, and
nothing is enqueued, so this runs without a GPU. A pointer that is missing from a call with work stays refused."""
import ctypes

import pytest
import torch


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.fixture(scope="module")
def xs():
    import __graft_entry__
    __graft_entry__.build()
    import comm_comp_fusion_gb300 as xs
    return xs


H, Hk, D, PAGE, PAGES, COLS = 4, 2, 64, 16, 5, 3


@pytest.mark.parametrize("N,T", ((2, 0), (0, 0), (0, 7)))
def test_serving_calls_without_work(xs, N, T):
    """A step with no new token, and one with no sequence (rows of none may be there all the same)."""
    assert bf(0, H, D).data_ptr() == 0  # what this is about
    ax, start, kv, table = xs.RopeAxes.powers((D,)), i32(N + 1), i32(N), i32(N, COLS)
    kp, vp = bf(PAGES, PAGE, Hk, D), bf(PAGES, PAGE, Hk, D)
    q, k, v, qo, ko, out = bf(T, H, D), bf(T, Hk, D), bf(T, Hk, D), bf(T, H, D), bf(T, Hk, D), bf(T, H, D)
    row = bf(T, (H + 2 * Hk) * D)
    mask, pos, parents = i32(T, 1), i32(T), i32(T)
    cache = (N, T, H, Hk, D, PAGE, PAGES, COLS)
    for cols in ((q, k, v), (row[:, :H * D], row[:, H * D:(H + Hk) * D], row[:, (H + Hk) * D:])):
        assert xs.cache_append_rope(*cols, qo, kp, vp, table, start, kv, *cache, ax) == xs.XS_OK
        assert xs.cache_append_rope(*cols, qo, kp, vp, table, start, kv, *cache, ax, pos=pos, k_out=ko) == xs.XS_OK
        assert xs.attn_packed(*cols, start, out, N, T, H, Hk, D, 0.1) == xs.XS_OK
    two = xs.RopeAxes.powers((32, 32))
    assert xs.cache_append_rope(q, k, v, qo, kp, vp, table, start, kv, *cache, two, pos=i32(T, 2)) == xs.XS_OK
    assert xs.cache_append(k, v, kp, vp, table, start, kv, N, T, Hk, D, PAGE, PAGES, COLS) == xs.XS_OK
    assert xs.attn_paged(q, kp, vp, table, start, kv, out, *cache, 0.1) == xs.XS_OK
    assert xs.tree_mask(parents, start, kv, mask, pos, N, T, 1) == xs.XS_OK
    assert xs.tree_mask(parents, start, None, mask, None, N, T, 1) == xs.XS_OK
    assert xs.attn_tree(q, kp, vp, table, start, kv, mask, out, *cache, 1, 0.1) == xs.XS_OK


@pytest.mark.parametrize("B,S", ((0, 128), (1, 0)))
def test_whole_sequence_calls_without_work(xs, B, S):
    q, k, v, out = (bf(1, B, S, H, D) for _ in range(4))
    few = bf(1, B, S, Hk, D)
    args = (q, k, v, out, B, S, H, D, 1, 0.1)
    for fn in (xs.attn, xs.attn_a2a, xs.attn_ws, xs.attn_a2a_ws, xs.attn_causal, xs.attn_causal_a2a, xs.attn_window,
               xs.attn_window_a2a, xs.ulysses_attn):
        assert fn(*args, *((None, 0) if fn in (xs.attn_ws, xs.attn_a2a_ws) else ())) == xs.XS_OK, fn.__name__
    for fn in (xs.a2a_permute, xs.a2a_permute_inverse):
        assert fn(q, out, B, S, H, D, 1) == xs.XS_OK, fn.__name__
    assert xs.attn_a2a_noalloc(*args) == xs.XS_OK
    assert xs.attn_a2a_trace(q, k, v, out, B, S, H, 128, 1, 0.1, torch.zeros(0, dtype=torch.uint8)) == xs.XS_OK
    for fn in (xs.attn_q8, xs.attn_a2a_q8, xs.attn_qkv8, xs.attn_a2a_qkv8):
        assert fn(q, k, v, out, B, S, H, 128, 1, 0.1) == xs.XS_OK, fn.__name__
    host = torch.zeros(0, dtype=torch.bfloat16)
    for fn in (xs.attn_host, xs.attn_a2a_host):
        assert fn(host, host, host, host, *args) == xs.XS_OK, fn.__name__
    ax = xs.RopeAxes.powers((D,))
    assert xs.rope(q, few, out, few.clone(), i32(1, S, 1), B, S, H, Hk, D, 1, ax) == xs.XS_OK
    assert xs.rope(q, None, out, None, i32(B, S, 1), B, S, H, 0, D, 1, ax) == xs.XS_OK


def test_the_other_checks_hold_for_empty_calls(xs):
    """What is wrong with an empty call's sizes, or with the pointers that it does have, is still refused."""
    q, kv, i = bf(0, H, D), bf(0, Hk, D), i32(3)
    pool, ax = bf(PAGES, PAGE, Hk, D), xs.RopeAxes.powers((D,))
    assert xs.attn_packed(q, kv, kv, i, q, 2, 0, H, Hk, 80, 0.1, check=False) == xs.XS_ERR_UNSUPPORTED
    assert xs.attn_packed(q, kv, kv, i.data_ptr() + 2, q, 2, 0, H, Hk, D, 0.1, check=False) == xs.XS_ERR_ALIGN
    assert xs.attn_packed(q, kv, kv, i, q, 2, 0, H, Hk, D, -0.1, check=False) == xs.XS_ERR_SHAPE
    assert xs.cache_append_rope(q, kv, kv, q, pool, pool, i32(2, COLS), i, i, 2, 0, H, Hk, D, PAGE, PAGES, COLS, ax,
                                check=False) == xs.XS_ERR_ALIAS
    assert xs.tree_mask(q.data_ptr(), i, i, None, None, 2, -1, 1, check=False) == xs.XS_ERR_NULL
    assert xs.tree_mask(i, i, i, i32(9), None, 2, 0, 9, check=False) == xs.XS_ERR_SHAPE
    for name in ("axis_dims", "freqs"):  # host arrays: never empty
        ptr = {"axis_dims": ctypes.addressof(ax._dims), "freqs": ctypes.addressof(ax._freqs)}
        ptr[name] = None
        assert xs.lib.xs_cache_append_rope(None, None, None, 0, 0, 0, None, None, None, None, None, None, None, None, 0, 0, H, Hk, D,
                                           PAGE, PAGES, COLS, 1, ptr["axis_dims"], ptr["freqs"], 0, None) == xs.XS_ERR_NULL


def test_missing_pointers_of_calls_with_work_stay_refused(xs):
    A = [0x10000000 * (i + 1) for i in range(12)]
    for at in range(4):
        ptr = [None if i == at else A[i] for i in range(4)]
        assert xs.attn(*ptr, 1, 128, H, D, 1, 0.1, check=False) == xs.XS_ERR_NULL
        assert xs.attn_window(*ptr, 1, 128, H, D, 1, 0.1, check=False) == xs.XS_ERR_NULL
        assert xs.attn_packed(*ptr, A[5], 1, 9, H, Hk, D, 0.1, workspace=A[6], workspace_bytes=1 << 27, check=False) == xs.XS_ERR_NULL
    assert xs.a2a_permute(None, A[0], 1, 128, H, D, 1, check=False) == xs.XS_ERR_NULL
    assert xs.cache_append(None, *A[:6], 1, 9, Hk, D, PAGE, PAGES, COLS, check=False) == xs.XS_ERR_NULL
    assert xs.tree_mask(A[0], A[1], None, A[2], A[3], 1, 9, 1, check=False) == xs.XS_ERR_NULL
    two = xs.RopeAxes.powers((32, 32))
    assert xs.cache_append_rope(*A[:9], 1, 9, H, Hk, D, PAGE, PAGES, COLS, two, check=False) == xs.XS_ERR_NULL  # pos
