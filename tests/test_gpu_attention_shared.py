"""Attention of branches behind shared prefixes against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests import lowbit_plain as low
from tests import step_plain as plain
from tests.test_gpu_attention_cache4 import _i32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# Columns of a prefix's table with which its pages are shared: calls go by the tables' width, and
# with narrow ones each branch of a small call reads its prefix itself.
WIDE = 6000


def _case(seed, B, fan, T, Hq, H, D, start, prefix, slack=0, wide=0):
    """q, a pool of random values, the branches' tables and their prefixes', `slack` columns wider
    than they need be, the prefixes' `wide` columns more."""
    rs = np.random.default_rng([seed, B, T, Hq, D])
    P = max(1, -(-(max(start) + T) // 64))
    PP = max(1, -(-max(prefix) // 64))
    n = B * P + len(prefix) * PP + 2
    order = rs.permutation(n).astype(np.int32)
    table, ptable = order[: B * P].reshape(B, P), order[B * P: B * P + len(prefix) * PP].reshape(-1, PP)
    pages = sv.cache4_alloc(n, H, D, DEV)
    g = torch.Generator(DEV).manual_seed(seed + B)
    k, v = (torch.randn(1, n * 64, H, D, generator=g, device=DEV) for _ in range(2))
    sv.cache4_write(pages, _i32([list(range(n))]), _i32([0]), k, v)
    q = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    table, ptable = (np.concatenate([x, np.full((len(x), n), -1, np.int32)], 1) for x, n in ((table, slack), (ptable, slack + wide)))
    return q, pages, table, ptable


def _run(q, pages, table, start, ptable, prefix, fan, count=None, **kw):
    B, T, Hq, D = q.shape
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, T, Hq), 7.0, device=DEV)
    sv.attention_cache4_shared(q, pages, _i32(table), _i32(start), _i32(ptable), _i32(prefix), fan=fan,
                               count=None if count is None else _i32(count), out=out, lse=lse, **kw)
    return out, lse


def _check(q, pages, table, start, ptable, prefix, fan, got, count=None, sees=None, rows=None):
    out, lse = (x.double().cpu().numpy() for x in got)
    B, T, Hq, D = q.shape
    H = pages.shape[1]
    a, pool = q.double().cpu().numpy(), pages.cpu().numpy()
    for g in range(len(prefix)):
        p_ok = 0 <= prefix[g] <= 64 * ptable.shape[1]
        pk, pv, good = plain.held(pool, ptable[g], prefix[g] if p_ok else 0, D)
        for b in range(g * fan, min(B, g * fan + fan)):
            n = T if count is None else count[b]
            if not low.fits(start[b], n, T, table.shape[1]):
                assert np.isnan(out[b]).all() and np.isnan(lse[b]).all()
                continue
            assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()
            k, v, own = plain.held(pool, table[b], start[b] + n, D)
            if not (p_ok and good and own):
                assert np.isnan(out[b, :n]).all() and np.isnan(lse[b, :n]).all()
                continue
            see = plain.window_sees(start[b], n, T, sees or (lambda i, j: j <= i), None, True, 1 << 40, 0)
            see = np.concatenate([np.ones((n, len(pk)), bool), see], 1)
            k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
            for i in range(n):
                for h in range(Hq):
                    if rows is not None and not rows(b, i, h):
                        continue
                    kv = h // (Hq // H)
                    want = plain.attend(a[b, i, h], k[:, kv], v[:, kv], see[i], D ** -0.5, 2.0 ** -20)
                    assert np.isnan(want[1]) == np.isnan(lse[b, i, h])
                    if np.isnan(want[1]):
                        assert np.isnan(out[b, i, h]).all()
                        continue
                    off = np.abs(out[b, i, h] - want[0])
                    assert (off <= want[2]).all(), (b, i, h, (off / want[2]).max())
                    assert lse[b, i, h] == want[1] or abs(lse[b, i, h] - want[1]) <= want[3], (b, i, h)


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,fan,T,Hq,H,start,prefix", [
    (1, 1, 1, 1, 1, [0], [1]),
    (1, 4, 1, 4, 2, [3], [0]),                             # fewer branches than fan; an empty prefix
    (4, 4, 1, 8, 2, [0, 1, 63, 64], [777]),
    (5, 2, 3, 7, 1, [0, 5, 130, 64, 9], [63, 64, 65]),     # a last group of one
    (6, 3, 5, 8, 2, [0] * 6, [0, 128]),                    # 60 rows
    (9, 9, 9, 8, 2, [7, 0, 1, 2, 3, 64, 65, 66, 300], [350]),  # 324 rows
    (33, 16, 2, 4, 4, list(range(33)), [31, 95, 33]),
])
def test_branches(D, B, fan, T, Hq, H, start, prefix, wide):
    q, pages, table, ptable = _case(1, B, fan, T, Hq, H, D, start, prefix, wide=wide)
    _check(q, pages, table, start, ptable, prefix, fan, _run(q, pages, table, start, ptable, prefix, fan))


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_counts_and_wide_tables(D, wide):
    """Fewer new tokens than columns, none at all, tables wide enough for pages to be cut."""
    B, fan, T = 7, 3, 6
    start, count, prefix = [0, 70, 3, 1, 0, 200, 5], [6, 0, 1, 3, 0, 2, 6], [1000, 65, 300]
    q, pages, table, ptable = _case(2, B, fan, T, 8, 2, D, start, prefix, 21, wide)
    _check(q, pages, table, start, ptable, prefix, fan, _run(q, pages, table, start, ptable, prefix, fan, count), count)


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("T", [5, 21, 40])
def test_trees(T, wide):
    rs = np.random.default_rng(T)
    par = [-1] + [int(rs.integers(0, i)) for i in range(1, T)]
    see = np.zeros((T, T), bool)
    for i in range(T):
        see[i] = see[par[i]] if i else see[i]
        see[i, i] = True
    start, prefix = [0, 30, 64, 2, 0], [100, 0, 190]
    q, pages, table, ptable = _case(3, 5, 2, T, 4, 1, 64, start, prefix, wide=wide)
    got = _run(q, pages, table, start, ptable, prefix, 2, mask=sv.tree_mask(par).to(DEV))
    _check(q, pages, table, start, ptable, prefix, 2, got, sees=lambda i, j: see[i, j])


@pytest.mark.parametrize("wide", [0, WIDE])
def test_rows_that_see_nothing_of_their_own(wide):
    T, start, prefix = 3, [0, 0, 0, 0], [70, 0]
    q, pages, table, ptable = _case(4, 4, 2, T, 2, 1, 128, start, prefix, wide=wide)
    none = torch.zeros(1, T, 1, dtype=torch.int32, device=DEV)
    got = _run(q, pages, table, start, ptable, prefix, 2, mask=none)
    _check(q, pages, table, start, ptable, prefix, 2, got, sees=lambda i, j: False)
    assert (got[0][2:] == 0).all() and (got[1][2:] == -float("inf")).all()


@pytest.mark.parametrize("wide", [0, 3 * WIDE])
def test_bad_prefixes_sequences_and_pages(wide):
    B, fan, T = 10, 2, 2
    start, count, prefix = [0, 3, 0, 0, 5, -1, 9, 1, 0, 0], [2, 2, 2, 2, 2, 2, 3, 2, 2, 2], [100, -1, 60, 9, 1 << 24]
    q, pages, table, ptable = _case(5, B, fan, T, 2, 1, 64, [70] * B, [130] * 5, wide=wide)
    ptable[0, 2] = -7   # behind the prefix's end: not looked at
    ptable[2, 0] = 1 << 28
    table[7, 0] = -1
    got = _run(q, pages, table, start, ptable, prefix, fan, count)
    _check(q, pages, table, start, ptable, prefix, fan, got, count)
    nan = torch.isnan(got[0]).flatten(1).any(1).tolist()
    assert nan == [False, False, True, True, True, True, True, True, True, True]


@pytest.mark.parametrize("wide", [0, WIDE])
def test_noise_behind_a_prefix_and_nan_in_it(wide):
    D, T, fan = 128, 2, 3
    start, prefix = [0] * 6, [70, 70]
    q, pages, table, ptable = _case(6, 6, fan, T, 4, 2, D, start, prefix, wide=wide)
    raw = pages.cpu().numpy()
    rs = np.random.default_rng(1)
    for g in range(2):
        for x in range(70, 128):
            for at in low.offsets(x % 64, D):
                raw[ptable[g, 1], :, at] = 255 if g else rs.integers(0, 256, (len(at), 2))
    pages = torch.from_numpy(raw).to(DEV)
    k = torch.zeros(1, 1, 2, D, device=DEV)
    k[0, 0, 1, 0] = float("nan")
    sv.cache4_write(pages, _i32(ptable[1:]), _i32([69]), k, torch.ones_like(k))
    q[0, 1, 0, 5] = float("nan")
    got = _run(q, pages, table, start, ptable, prefix, fan)
    nan = torch.isnan(got[0]).any(-1)
    want = torch.zeros(6, T, 4, dtype=torch.bool)
    want[3:, :, 2:] = want[0, 1, 0] = True
    assert torch.equal(nan.cpu(), want) and torch.equal(torch.isnan(got[1]).cpu(), want)
    _check(q, pages, table, start, ptable, prefix, fan, got)


@pytest.mark.parametrize("D,B,fan,T,Hq,H,prefix", [
    (128, 64, 8, 5, 32, 8, [1500 + 313 * (g % 8) for g in range(8)]),   # 160 rows a head
    (64, 96, 96, 2, 4, 4, [5000]),
    (256, 12, 6, 9, 14, 2, [37, 1155]),                                  # 378 rows a head
    (128, 300, 300, 1, 8, 1, [2500]),                                    # 2,400 rows
    (64, 40, 40, 7, 8, 1, [801]),                                        # 2,240 rows
    (128, 3, 3, 1, 2, 1, [9000]),                                        # six rows, a long prefix
])
def test_many_rows_and_long_prefixes(D, B, fan, T, Hq, H, prefix):
    start = [(b * 37) % 150 for b in range(B)]
    q, pages, table, ptable = _case(7, B, fan, T, Hq, H, D, start, prefix)
    got = _run(q, pages, table, start, ptable, prefix, fan)
    _check(q, pages, table, start, ptable, prefix, fan, got, rows=lambda b, i, h: (b * 7 + i * 3 + h) % 11 == 0)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()


# Shapes whose prefixes are shared, in blocks of rows or, heads of 128 with more than 96 rows and
# 512 (prefix, kv head) pairs and heads of 256 with more than 64 rows and wide tables, by the waves of
# a workgroup; the first one by each branch, 6,656 segments of few pages.  (B, fan, T, Hq, H, D, slack
# of the tables: wide ones are cut, and those of up to 20 columns not)
SHARED = [(104, 13, 2, 256, 64, 128, 0), (104, 13, 2, 256, 64, 128, 17), (103, 13, 2, 256, 64, 128, 21),
          (40, 5, 9, 256, 64, 128, 70), (70, 7, 5, 192, 64, 128, 40), (12, 6, 9, 14, 2, 256, 400), (7, 7, 3, 8, 2, 256, 2200),
          (9, 3, 22, 8, 8, 256, 200), (24, 2, 17, 128, 64, 256, 40), (48, 12, 3, 128, 64, 256, 17),
          (32, 16, 4, 128, 64, 64, 17), (40, 10, 2, 256, 64, 128, 17), (32, 8, 1, 128, 64, 256, 17)]


@pytest.mark.parametrize("B,fan,T,Hq,H,D,slack", SHARED)
def test_shared_pages(B, fan, T, Hq, H, D, slack):
    n = -(-B // fan)
    start = [(b * 23) % 90 for b in range(B)]
    prefix = [(0, 1, 64, 65, 97, 127, 128, 190)[(g * 5 + 3) % 8] for g in range(n)]
    q, pages, table, ptable = _case(11, B, fan, T, Hq, H, D, start, prefix, slack)
    got = _run(q, pages, table, start, ptable, prefix, fan)
    _check(q, pages, table, start, ptable, prefix, fan, got, rows=lambda b, i, h: (b * 7 + i * 5 + h) % 61 == 0)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    again = _run(q, pages, table, start, ptable, prefix, fan)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("B,fan,T,Hq,H,D,slack", [(12, 6, 9, 14, 2, 256, 400), (18, 6, 9, 14, 2, 128, 400),
                                                    (12, 6, 9, 14, 2, 128, 2)])
def test_shared_pages_of_live_rows(B, fan, T, Hq, H, D, slack):
    """Fewer new tokens than columns: rows of one tile up to all, none at all, and counts that fit no
    call, whose sequences are NaN and whose neighbours are not."""
    n = -(-B // fan)
    start, prefix = [(b * 23) % 90 for b in range(B)], [130 - g for g in range(n)]
    q, pages, table, ptable = _case(12, B, fan, T, Hq, H, D, start, prefix, slack)
    for counts in ([(b * 5) % (T + 1) for b in range(B)], [1] + [0] * (B - 1), [0] * B, [T] * B,
                   [T + 1, -1, 3, 0, T, 1] * (B // 6)):
        got = _run(q, pages, table, start, ptable, prefix, fan, counts)
        _check(q, pages, table, start, ptable, prefix, fan, got, counts, rows=lambda b, i, h: (b + i + h) % 7 == 0)


@pytest.mark.parametrize("fan,D", [(64, 64), (65, 64), (64, 256), (65, 128)])
def test_counts_around_64_branches(fan, D):
    """Live rows are counted through up to 64 branches; above that all rows have their place."""
    B, T, start, prefix = 2 * fan - 3, 3, [7] * (2 * fan - 3), [200, 66]
    counts = [(b * 7) % 4 for b in range(B)]
    q, pages, table, ptable = _case(13, B, fan, T, 4, 1, D, start, prefix, slack=600)
    got = _run(q, pages, table, start, ptable, prefix, fan, counts)
    _check(q, pages, table, start, ptable, prefix, fan, got, counts, rows=lambda b, i, h: (b + i + h) % 5 == 0)


@pytest.mark.parametrize("case", [(104, 13, 2, 256, 64, 128), (24, 6, 9, 14, 2, 256)])
def test_shared_pages_bad_ones_and_noise(case):
    """An ill-formed prefix, a page outside the pool, noise behind a prefix's end and a NaN in one."""
    B, fan, T, Hq, H, D = case
    n = -(-B // fan)
    prefix, start = ([70, 1 << 20, 130, 70] + [70] * n)[:n], [5] * B
    q, pages, table, ptable = _case(14, B, fan, T, Hq, H, D, start, [130] * n, 400 if D == 256 else 17)
    ptable[2, 1] = -3
    raw = pages.cpu().numpy()
    for x in range(70, 128):
        for at in low.offsets(x % 64, D):
            raw[ptable[0, 1], :, at] = 255
    pages = torch.from_numpy(raw).to(DEV)
    if n > 3:
        k = torch.zeros(1, 1, H, D, device=DEV)
        k[0, 0, 1, 0] = float("nan")
        sv.cache4_write(pages, _i32(ptable[3:4]), _i32([69]), k, torch.ones_like(k))
    got = _run(q, pages, table, start, ptable, prefix, fan)
    nan = torch.isnan(got[0]).any(-1).cpu()
    want = torch.zeros(B, T, Hq, dtype=torch.bool)
    want[fan: 3 * fan] = True
    want[3 * fan: 4 * fan, :, Hq // H: 2 * (Hq // H)] = True
    assert torch.equal(nan, want) and torch.equal(torch.isnan(got[1]).cpu(), want)
    _check(q, pages, table, start, ptable, prefix, fan, got, rows=lambda b, i, h: (b + i + h) % 53 == 0)


@pytest.mark.parametrize("case", [(104, 13, 2, 256, 64, 128, 0), (104, 13, 2, 256, 64, 128, 17), (24, 6, 9, 14, 2, 256, 400)])
def test_shared_pages_and_rows_of_any_magnitude(case):
    """Rows whose scores pass 2^24 or F32's range beside ordinary ones in one tile."""
    B, fan, T, Hq, H, D, slack = case
    start, prefix = [3] * B, [150] * (-(-B // fan))
    q, pages, table, ptable = _case(17, B, fan, T, Hq, H, D, start, prefix, slack)
    size = torch.ones(B, 1, Hq, 1, device=DEV)
    size[1::5, :, ::3], size[2::5, :, 1::3], size[3::5, :, ::2] = 1e8, 3e37, 1e-30
    got = _run((q.float() * size).bfloat16(), pages, table, start, ptable, prefix, fan)
    usual = (size[:, 0, :, 0] == 1).cpu().numpy()
    _check(q, pages, table, start, ptable, prefix, fan, got, rows=lambda b, i, h: usual[b, h] and (b * 7 + i * 5 + h) % 61 == 0)
    far = (size[:, 0, :, 0] == 1e8)[:, None].expand(B, T, Hq)
    assert torch.isfinite(got[0][far]).all() and (got[0][far].abs() <= 8).all()


# Branches with so many (branch, kv head, block of rows) that a wave has one by itself, for few pages
# and for more, or a workgroup, behind short prefixes (wide: 0) and behind shared ones; 1 to 4 tiles.
@pytest.mark.parametrize("wide", [0, 100])
@pytest.mark.parametrize("B,fan,T,Hq,H,D,slack", [
    (33, 4, 1, 32, 32, 64, 0), (40, 3, 5, 160, 32, 64, 0), (66, 5, 10, 128, 32, 64, 25), (33, 2, 15, 128, 32, 64, 3),
    (33, 4, 1, 64, 32, 128, 0), (33, 4, 7, 96, 32, 128, 5), (66, 4, 10, 128, 32, 128, 20), (20, 2, 2, 16, 16, 128, 30),
    (33, 3, 2, 32, 32, 256, 0), (24, 4, 5, 128, 32, 256, 25), (12, 3, 3, 32, 16, 256, 45)])
def test_many_segments(B, fan, T, Hq, H, D, slack, wide):
    n = -(-B // fan)
    start = [(b * 29) % 120 for b in range(B)]
    prefix = [(0, 1, 64, 65, 97, 127, 128)[(g * 5 + 3) % 7] for g in range(n)]
    count = [(b * 3 + 1) % (T + 1) for b in range(B)]
    q, pages, table, ptable = _case(18, B, fan, T, Hq, H, D, start, prefix, slack, wide)
    table[3, 0] = -1
    for counts in (None, count):
        got = _run(q, pages, table, start, ptable, prefix, fan, counts)
        _check(q, pages, table, start, ptable, prefix, fan, got, counts, rows=lambda b, i, h: (b * 7 + i * 5 + h) % 83 == 0)


def test_captured_with_shared_pages():
    B, fan, T, Hq, H, D = 104, 13, 2, 256, 64, 128
    start, prefix = [3] * B, [100 + g for g in range(8)]
    q, pages, table, ptable = _case(15, B, fan, T, Hq, H, D, start, prefix, 21)
    args = [q, pages, _i32(table), _i32(start), _i32(ptable), _i32(prefix)]
    want = sv.attention_cache4_shared(*args, fan=fan, return_lse=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.attention_cache4_shared(*args, fan=fan, return_lse=True)
    for _ in range(4):
        got[0].zero_()
        got[1].zero_()
        g.replay()
        other = sv.attention_cache4_shared(*args, fan=fan, return_lse=True)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(z, y) for x, y, z in zip(got, want, other))


def test_another_stream():
    B, fan, T, Hq, H, D = 6, 3, 2, 8, 2, 64
    start, prefix = [9] * B, [100, 64]
    q, pages, table, ptable = _case(16, B, fan, T, Hq, H, D, start, prefix)
    args = [q, pages, _i32(table), _i32(start), _i32(ptable), _i32(prefix)]
    want = sv.attention_cache4_shared(*args, fan=fan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.attention_cache4_shared(*args, fan=fan, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("wide", [0, 3 * WIDE])
def test_far_scores(wide):
    """Scores of ordinary and of large magnitude side by side, in the prefix and behind it."""
    D, T, fan = 64, 1, 4
    start, prefix = [3] * 4, [200]
    q, pages, table, ptable = _case(8, 4, fan, T, 2, 1, D, start, prefix, wide=wide)
    q = q * torch.tensor([1.0, 1e4, 1e9, 1e-9], device=DEV).view(4, 1, 1, 1).bfloat16()
    got = _run(q, pages, table, start, ptable, prefix, fan)
    _check(q, pages, table, start, ptable, prefix, fan, got, rows=lambda b, i, h: b in (0, 3))
    # one position outweighs all others: its value, or the mean of those whose scores round alike
    assert torch.isfinite(got[0]).all() and (got[0].abs() <= 64).all()


@pytest.mark.parametrize("wide", [0, WIDE])
def test_agrees_with_one_cache(wide):
    """A prefix of whole pages with each branch's own pages behind it, as one table."""
    B, fan, T, Hq, H, D, n = 12, 4, 4, 8, 2, 128, 512
    start, prefix = [(b * 29) % 90 for b in range(B)], [n] * 3
    q, pages, table, ptable = _case(9, B, fan, T, Hq, H, D, start, prefix, wide=wide)
    got = _run(q, pages, table, start, ptable, prefix, fan)
    one = np.concatenate([np.repeat(ptable[:, : n // 64], fan, 0), table], 1)
    out, lse = sv.attention_cache4(q, pages, _i32(one), _i32([n + s for s in start]), return_lse=True)
    assert (got[1] - lse).abs().max() <= 2.0 ** -17
    assert (got[0].float() - out.float()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("wide", [0, WIDE])
def test_same_outputs_every_time_and_strided(wide):
    B, fan, T, Hq, H, D = 16, 8, 3, 8, 2, 128
    start, prefix = [11] * B, [1999, 2345]
    q, pages, table, ptable = _case(10, B, fan, T, Hq, H, D, start, prefix, wide=wide)
    want = _run(q, pages, table, start, ptable, prefix, fan)
    wide = torch.zeros(T, B, Hq + 3, D + 8, dtype=torch.bfloat16, device=DEV)
    wide[:, :, :Hq, :D] = q.transpose(0, 1)
    view = wide[:, :, :Hq, :D].transpose(0, 1)
    target = torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    ws = torch.full((sv.lib().spec_attention_cache4_shared_workspace(B, T, Hq, H, D, fan) + 512,), 255,
                    dtype=torch.uint8, device=DEV)
    off = -ws.data_ptr() % 256
    for _ in range(3):
        sv.attention_cache4_shared(view, pages, _i32(table), _i32(start), _i32(ptable), _i32(prefix), fan=fan, out=target,
                                   workspace=ws[off:])
        assert torch.equal(target, want[0])
