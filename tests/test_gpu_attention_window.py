"""Attention over the 4-bit cache through a window against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests import lowbit_plain as low
from tests import step_plain as plain
from tests.test_gpu_attention_cache4 import _case, _i32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _run(q, pages, table, start, count=None, **kw):
    B, T, Hq, D = q.shape
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, T, Hq), 7.0, device=DEV)
    sv.attention_cache4(q, pages, _i32(table), _i32(start), count=None if count is None else _i32(count),
                        out=out, lse=lse, **kw)
    return out, lse


def _check(q, pages, table, start, count, window, sinks, got, sees=None, depth=None):
    out, lse = (x.double().cpu().numpy() for x in got)
    B, T, Hq, D = q.shape
    H = pages.shape[1]
    a, pool = q.double().cpu().numpy(), pages.cpu().numpy()
    for b in range(B):
        n = T if count is None else count[b]
        if not low.fits(start[b], n, T, table.shape[1]):
            assert np.isnan(out[b]).all() and np.isnan(lse[b]).all()
            continue
        assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()
        see = plain.window_sees(start[b], n, T, sees or (lambda i, j: j <= i), depth and depth[b], sees is not None,
                                window, sinks)
        k, v, _ = plain.held(pool, table[b], start[b] + n, D)
        for i in range(n):
            for h in range(Hq):
                want = plain.attend(a[b, i, h], k[:, h // (Hq // H)], v[:, h // (Hq // H)], see[i], D ** -0.5)
                assert np.isnan(want[1]) == np.isnan(lse[b, i, h])
                if np.isnan(want[1]):
                    assert np.isnan(out[b, i, h]).all()
                    continue
                assert (np.abs(out[b, i, h] - want[0]) <= want[2]).all(), (b, i, h)
                assert lse[b, i, h] == want[1] or abs(lse[b, i, h] - want[1]) <= want[3], (b, i, h)


def _forget(table, start, T, window, sinks):
    """The table without the pages that no token sees."""
    table = table.copy()
    for b, s in enumerate(start):
        for p in range(table.shape[1]):
            if p * 64 >= sinks and (p + 1) * 64 <= s - window + 1:
                table[b, p] = (-1, 1 << 30)[p % 2]
    return table


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (63, 0), (64, 64), (65, 65), (200, 4), (129, 130),
                                          (1 << 30, 0), (2147483647, 2147483647)])
def test_chains(D, window, sinks):
    start = [0, 1, 64, 130, 511]
    q, pages, table = _case(1, 5, 5, 4, 2, D, start)
    table = _forget(table, start, 5, window, sinks)
    _check(q, pages, table, start, None, window, sinks, _run(q, pages, table, start, window=window, sinks=sinks))


@pytest.mark.parametrize("D,T,Hq,H", [(64, 1, 1, 1), (64, 33, 2, 1), (128, 1, 8, 2), (128, 7, 7, 1), (256, 3, 8, 2), (128, 70, 1, 1)])
def test_rows_and_counts(D, T, Hq, H):
    """Windows shorter than the new tokens, with fewer tokens than the call has columns."""
    start, count = [700, 3, 0, 127, 64], [T, 1, T, 0, max(1, T - 1)]
    q, pages, table = _case(2, 5, T, Hq, H, D, start)
    for window, sinks in ((5, 2), (40, 0), (400, 70)):
        t = _forget(table, start, T, window, sinks)
        _check(q, pages, t, start, count, window, sinks, _run(q, pages, t, start, count, window=window, sinks=sinks))


@pytest.mark.parametrize("window,sinks", [(1, 0), (8, 3), (100, 4)])
@pytest.mark.parametrize("T", [4, 21, 40])
def test_trees(T, window, sinks):
    """Cached tokens by depth, new ones by the mask alone; depths for all and for each sequence,
    those outside 0 .. T - 1 as the nearer end, none at all."""
    start = [0, 90, 300]
    rs = np.random.default_rng(T)
    par = [-1] + [int(rs.integers(0, i)) for i in range(1, T)]
    see = np.zeros((T, T), bool)
    for i in range(T):
        see[i] = see[par[i]] if i else see[i]
        see[i, i] = True
    q, pages, table = _case(3, 3, T, 4, 2, 64, start)
    table = _forget(table, start, T, window, sinks)
    mask, depth = sv.tree_mask(par).to(DEV), sv.tree_depths(par)
    wild = torch.tensor([[-5] + [T + 9] * (T - 1), [0] * T, list(range(T))], dtype=torch.int32)
    for d in (depth, wild, None):
        got = _run(q, pages, table, start, mask=mask, depth=None if d is None else d.to(DEV), window=window, sinks=sinks)
        rows = None if d is None else [d[b % len(d)].tolist() for b in range(3)]
        _check(q, pages, table, start, None, window, sinks, got, lambda i, j: see[i, j], rows)


@pytest.mark.parametrize("B,T,Hq,H,D,window,sinks", [(8, 21, 512, 64, 128, 100, 5), (8, 30, 256, 64, 128, 1500, 0),
                                                     (8, 27, 256, 64, 128, 40, 70), (3, 21, 32, 4, 256, 40000, 0),
                                                     (2, 33, 8, 2, 256, 1 << 20, 9), (4, 70, 2, 2, 256, 30000, 1)])
def test_shared_pages(B, T, Hq, H, D, window, sinks):
    """Shapes whose pages the waves of a workgroup share (heads of 128: more than 96 rows and 512
    sequences times kv heads; of 256: more than 64 rows and wide tables), as chains and as trees."""
    start = [(b * 131) % 700 for b in range(B)]
    slack = 5200 // (B * H) * 4 if D == 256 else 0
    q, pages, table = _case(8, B, T, Hq, H, D, start)
    table = np.concatenate([_forget(table, start, T, window, sinks), np.full((B, slack), -1, np.int32)], 1)
    keep = [(b, i, h) for b in range(B) for i in range(T) for h in range(Hq) if (b * 7 + i * 5 + h) % 97 == 0]
    rs = np.random.default_rng(T)
    par = [-1] + [int(rs.integers(0, i)) for i in range(1, T)]
    see = np.zeros((T, T), bool)
    for i in range(T):
        see[i] = see[par[i]] if i else see[i]
        see[i, i] = True
    count = [T - b % 3 for b in range(B)]
    for kw, rule, depth in ((dict(), None, None),
                            (dict(mask=sv.tree_mask(par).to(DEV), depth=sv.tree_depths(par).to(DEV)),
                             lambda i, j: see[i, j], sv.tree_depths(par)[0].tolist())):
        got = _run(q, pages, table, start, count, window=window, sinks=sinks, **kw)
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
        a, pool, held = q.double().cpu().numpy(), pages.cpu().numpy(), {}
        out, lse = (x.double().cpu().numpy() for x in got)
        for b in range(B):
            assert (out[b, count[b]:] == 7).all() and (lse[b, count[b]:] == 7).all()
            held[b] = plain.held(pool, table[b], start[b] + count[b], D)[:2] + (
                plain.window_sees(start[b], count[b], T, rule or (lambda i, j: j <= i), depth, rule is not None, window, sinks),)
        for b, i, h in keep:
            if i < count[b]:
                k, v, sees = held[b]
                want = plain.attend(a[b, i, h], k[:, h // (Hq // H)], v[:, h // (Hq // H)], sees[i], D ** -0.5)
                assert (np.abs(out[b, i, h] - want[0]) <= want[2]).all(), (b, i, h)
                assert abs(lse[b, i, h] - want[1]) <= want[3], (b, i, h)


@pytest.mark.parametrize("B,T,Hq,H,D", [(4, 3, 48, 48, 64), (4, 12, 96, 48, 128), (4, 2, 48, 48, 256)])
def test_windows_of_many_pages_not_cut(B, T, Hq, H, D):
    """Four times as many segments as pages, more than 20 of those."""
    start, window, sinks = [1700, 0, 900, 2300], 1500, 70
    count = [T, T, 0, max(1, T - 1)]
    q, pages, table = _case(19, B, T, Hq, H, D, start)
    table = _forget(table, start, T, window, sinks)
    got = _run(q, pages, table, start, count, window=window, sinks=sinks)
    some = [0, 1, 2, Hq - 1]  # query heads that are looked at, each with its kv head
    _check(q[:, :, some].contiguous(), pages[:, [h // (Hq // H) for h in some]].contiguous(), table, start, count, window,
           sinks, tuple(x[:, :, some] for x in got))


def test_rows_that_see_nothing():
    T, start = 3, [200, 0]
    q, pages, table = _case(4, 2, T, 2, 1, 128, start)
    none = torch.zeros(1, T, 1, dtype=torch.int32, device=DEV)
    out, lse = _run(q, pages, table, start, mask=none, window=1)
    assert (out == 0).all() and (lse == -float("inf")).all()
    out, lse = _run(q, pages, table, start, mask=none, window=1, sinks=1)
    _check(q, pages, table, start, None, 1, 1, (out, lse), lambda i, j: False)


def test_a_wide_window_is_no_window():
    for T, start, slack in ((5, [0, 77, 1900, 640], 0), (9, [3000], 20)):
        q, pages, table = _case(5, len(start), T, 8, 2, 128, start, slack=slack)
        plain_out = _run(q, pages, table, start)
        for window, sinks in ((max(start) + T, 0), (1, max(start) + T), (1 << 29, 5)):
            got = _run(q, pages, table, start, window=window, sinks=sinks)
            # the same sums, cut elsewhere: the outputs' rounding and the bounds of both
            assert torch.allclose(got[1], plain_out[1], rtol=2.0 ** -20, atol=2.0 ** -18)
            assert (got[0].float() - plain_out[0].float()).abs().max() <= 2.0 ** -6 * 4


def test_long_cache():
    """A window over the end of 140,000 tokens, cut over workgroups or whole, in pages of which most
    are nobody's."""
    D, H = 64, 2
    for W, sinks in ((1500, 4), (100, 0), (2500, 700)):
        T, s = 3, 140_001
        cols = -(-(s + T) // 64)
        keep = [p for p in range(cols) if p * 64 < sinks or (p + 1) * 64 > s - W + 1]
        rs = np.random.default_rng(W)
        table = np.full((1, cols), -1, np.int32)
        table[0, keep] = rs.permutation(len(keep))
        pages = sv.cache4_alloc(len(keep), H, D, DEV)
        k, v = (torch.randn(1, 64 * len(keep), H, D, device=DEV) for _ in range(2))
        sv.cache4_write(pages, _i32([list(range(len(keep)))]), _i32([0]), k, v)
        q = torch.randn(1, T, 4, D, device=DEV).bfloat16()
        got = _run(q, pages, table, [s], window=W, sinks=sinks)
        # the positions that are read, as a short cache of their own
        see = plain.window_sees(s, T, T, lambda i, j: j <= i, None, False, W, sinks)
        pos = np.concatenate([np.arange(p * 64, min(p * 64 + 64, s + T)) for p in keep])
        kk, vv, _ = plain.held(pages.cpu().numpy(), table[0, keep], len(pos), D)
        for i in range(T):
            for h in range(4):
                want = plain.attend(q[0, i, h].double().cpu().numpy(), kk[:, h // 2], vv[:, h // 2], see[i, pos], D ** -0.5)
                assert (np.abs(got[0][0, i, h].double().cpu().numpy() - want[0]) <= want[2]).all()
                assert abs(float(got[1][0, i, h]) - want[1]) <= want[3]


def test_bad_sequences_and_pages():
    """Ill-formed sequences, and a page outside the pool that a token does see, are NaN; one that none
    sees is not looked at."""
    T, start, count = 2, [-1, 300, 300, 0, 400], [2, 2, 2, 3, -2]
    q, pages, table = _case(6, 5, T, 2, 1, 64, [300] * 5)
    table[1, 2] = -1        # positions 128 .. 191
    table[2, 4] = 1 << 20   # 256 .. 319
    got = _run(q, pages, table, start, count, window=90, sinks=4)
    nan = torch.isnan(got[0]).flatten(1)
    assert nan[[0, 2, 3, 4]].all() and not nan[1].any()
    got = _run(q, pages, table, [0, 300, 0, 0, 0], [0, 2, 0, 0, 0], window=150, sinks=0)
    assert torch.isnan(got[0][1]).all()


def test_nan_reaches_only_what_sees_it():
    T, H, D, start = 3, 1, 128, [300]
    q, pages, table = _case(7, 1, T, 1, H, D, start)
    k = torch.zeros(1, 1, H, D, device=DEV)
    k[..., 3] = float("inf")
    sv.cache4_write(pages, _i32(table), _i32([200]), k, torch.ones_like(k))
    # position 200 is in the window of the token at 300 only
    got = _run(q, pages, table, start, window=101)
    assert torch.isnan(got[0][0, 0]).all() and not torch.isnan(got[0][0, 1:]).any()
    got = _run(q, pages, table, start, window=50, sinks=200)
    assert not torch.isnan(got[0]).any()
    got = _run(q, pages, table, start, window=50, sinks=201)
    assert torch.isnan(got[0]).all()
