"""Attention over the 4-bit cache against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests import lowbit_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _case(seed, B, T, Hq, H, D, start, spare=2, slack=0):
    """q, a pool with random pages of well-formed values, and tables."""
    rs = np.random.default_rng([seed, B, T, Hq, D])
    P = max(1, -(-(max(start) + T) // 64)) + slack
    n = B * P + spare
    table = rs.permutation(n)[: B * P].reshape(B, P).astype(np.int32)
    pages = sv.cache4_alloc(n, H, D, DEV)
    k, v = (torch.tensor(rs.normal(0, 1, (1, n * 64, H, D)), dtype=torch.float32, device=DEV) for _ in range(2))
    sv.cache4_write(pages, _i32([list(range(n))]), _i32([0]), k, v)
    q = torch.tensor(rs.normal(0, 1, (B, T, Hq, D)), dtype=torch.float32).bfloat16().to(DEV)
    return q, pages, table


def _check(q, pages, table, start, count, sees, got, scale=None, old=7.0):
    out, lse = got
    B, T, Hq, D = q.shape
    n = [T] * B if count is None else count
    want = plain.attention(q.double().cpu().numpy(), pages.cpu().numpy(), table, start, n, sees,
                           plain.inv_sqrt(D) if scale is None else scale)
    for x, w, bound in ((out, want[0], want[2]), (lse, want[1], want[3])):
        x = x.double().cpu().numpy()
        for b in range(B):
            keep = n[b] if plain.fits(start[b], n[b], T, table.shape[1]) else T
            a, y, t = x[b, :keep], w[b, :keep], bound[b, :keep]
            assert np.array_equal(np.isnan(a), np.isnan(y))
            fine = np.isfinite(y)
            assert np.array_equal(a[~fine], y[~fine], equal_nan=True)
            off = np.abs(a[fine] - y[fine])
            assert (off <= t[fine]).all(), (b, (off / t[fine]).max())
            if old is not None:
                assert (x[b, keep:] == old).all()


def _run(q, pages, table, start, count=None, **kw):
    B, T, Hq, D = q.shape
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, T, Hq), 7.0, device=DEV)
    sv.attention_cache4(q, pages, _i32(table), _i32(start), count=None if count is None else _i32(count),
                        out=out, lse=lse, **kw)
    return out, lse


def _chain(b, i, j):
    return j <= i


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,Hq,H,start", [
    (1, 1, 1, 1, [0]),              # one token, nothing cached
    (1, 1, 4, 4, [1]),
    (2, 1, 8, 2, [62, 63]),         # a page's end
    (2, 5, 8, 2, [64, 300]),        # rows past a tile of 16
    (3, 3, 7, 1, [0, 5, 130]),      # seven heads to a kv head
    (1, 9, 16, 2, [700]),           # more pages than waves; several workgroups to a sequence
    (2, 33, 4, 1, [31, 95]),        # several blocks of rows
])
def test_chain(D, B, T, Hq, H, start):
    q, pages, table = _case(1, B, T, Hq, H, D, start)
    _check(q, pages, table, start, None, _chain, _run(q, pages, table, start))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_counts_leave_rows_as_they_were(D):
    start, count = [0, 3, 60, 128, 0], [0, 4, 1, 3, 2]
    q, pages, table = _case(2, 5, 4, 4, 2, D, start)
    _check(q, pages, table, start, count, _chain, _run(q, pages, table, start, count))


@pytest.mark.parametrize("start", [[0, 0], [40, 127], [50, 64], [1, 33]])
@pytest.mark.parametrize("T", [4, 21, 40, 70])
def test_trees(T, start):
    """Trees across page and word borders, one mask for all and one for each."""
    rs = np.random.default_rng(T)
    par = [[-1] + [int(rs.integers(0, i)) for i in range(1, T)] for _ in range(2)]
    q, pages, table = _case(3, 2, T, 4, 2, 64, start)
    anc = []
    for p in par:
        s = np.zeros((T, T), bool)
        for i in range(T):
            s[i] = s[p[i]] if i else s[i]
            s[i, i] = True
        anc.append(s)
    one = sv.tree_mask(par[0]).to(DEV)
    _check(q, pages, table, start, None, lambda b, i, j: anc[0][i, j], _run(q, pages, table, start, mask=one))
    both = torch.cat([sv.tree_mask(p) for p in par]).to(DEV)
    _check(q, pages, table, start, [T, T - 2], lambda b, i, j: anc[b][i, j],
           _run(q, pages, table, start, [T, T - 2], mask=both))
    wide = torch.full((2, T, both.shape[2] + 3), -1, dtype=torch.int32, device=DEV)
    wide[:, :, : both.shape[2]] = both
    again = _run(q, pages, table, start, mask=wide[:, :, : both.shape[2]])
    assert all(torch.equal(x, y) for x, y in zip(again, _run(q, pages, table, start, mask=both)))


def test_rows_that_see_nothing():
    T, start = 6, [0, 0, 2]
    q, pages, table = _case(4, 3, T, 2, 1, 128, start)
    see = np.zeros((T, T), bool)
    see[1, 0] = see[4, 2] = see[4, 4] = True
    words = torch.tensor([[[int(sum(1 << j for j in range(T) if see[i, j]))] for i in range(T)]],
                         dtype=torch.int32, device=DEV)
    _check(q, pages, table, start, None, lambda b, i, j: see[i, j], _run(q, pages, table, start, mask=words))


def test_nan_reaches_the_rows_that_see_it_and_no_other():
    """Positions held as NaN, non-finite queries, and pages whose unwritten positions hold bytes
    of any kind, NaN exponents among them."""
    T, H, D, start = 4, 2, 128, [70, 3]
    q, pages, table = _case(5, 2, T, 4, H, D, start)
    rs = np.random.default_rng(5)
    raw = pages.cpu().numpy()
    for b in range(2):  # everything behind the last token: noise, then all exponents 255
        for x in range(start[b] + T, table.shape[1] * 64):
            for at in plain.offsets(x % 64, D):
                raw[table[b, x // 64], :, at] = 255 if b else rs.integers(0, 256, (len(at), H))
    pages = torch.from_numpy(raw).to(DEV)
    k = torch.zeros(2, 1, H, D, device=DEV)
    k[0, 0, 1, 5], k[1, 0, 0, 9] = float("inf"), float("nan")
    v = torch.ones(2, 1, H, D, device=DEV)
    sv.cache4_write(pages, _i32(table), _i32([start[0] + 2, start[1] + 1]), k, v)
    q[0, 1, 3, 17] = float("nan")
    q[1, 0, 2, 1] = float("inf")
    got = _run(q, pages, table, start)
    nan = torch.isnan(got[0]).all(-1)
    assert torch.equal(nan, torch.isnan(got[0]).any(-1)) and torch.equal(nan, torch.isnan(got[1]))
    want = torch.zeros(2, T, 4, dtype=torch.bool)
    want[0, 2:, 2:] = True   # kv head 1 of sequence 0 from its new token 2 on
    want[1, 1:, :2] = True   # kv head 0 of sequence 1 from its new token 1 on
    want[0, 1, 3] = want[1, 0, 2] = True
    assert torch.equal(nan.cpu(), want)
    q2, fine = q.clone(), ~want
    q2[0, 1, 3, 17] = q2[1, 0, 2, 1] = 0
    w = plain.attention(q2.double().cpu().numpy(), pages.cpu().numpy(), table, start, [T] * 2, _chain,
                        plain.inv_sqrt(D))
    for x, y, t in ((got[0], w[0], w[2]), (got[1], w[1], w[3])):
        off = np.abs(x.double().cpu().numpy() - y)[fine.numpy()]
        assert (off <= t[fine.numpy()]).all()


def test_ill_formed_sequences_are_nan():
    start, count = [-1, 5, 5, 10, 64, 2 ** 31 - 1], [2, -1, 5, 3, 3, 3]
    q, pages, table = _case(6, 6, 4, 2, 1, 128, [64])
    table[3, 0], table[4, 0] = len(pages), -1  # pages outside the pool, the second a cached one
    _check(q, pages, table, start, count, _chain, _run(q, pages, table, start, count))


def test_scores_of_any_size():
    """A running maximum that keeps rising, scores far apart, and keys of any exponent."""
    D, T, start = 128, 2, [640]
    q, pages, table = _case(7, 1, T, 2, 1, D, start)
    ramp = torch.linspace(-30, 30, 642, device=DEV)
    u = torch.nn.functional.normalize(torch.randn(D, device=DEV), dim=0)
    k = (ramp[:, None] * u * 11).view(1, 642, 1, D)
    v = torch.randn(1, 642, 1, D, device=DEV)
    for sign in (1, -1):
        sv.cache4_write(pages, _i32(table), _i32([0]), sign * k, v)
        q[:] = u.bfloat16()
        got = _run(q, pages, table, start, scale=1.0)
        _check(q, pages, table, start, None, _chain, got, scale=1.0)
    sv.cache4_write(pages, _i32(table), _i32([0]), k * 1e30, v * 1e30)
    got = _run(q * 1e-30, pages, table, start, scale=1.0)
    _check(q * 1e-30, pages, table, start, None, _chain, got, scale=1.0)


def test_strides_scale_streams_and_repeats():
    start = [100, 7]
    q, pages, table = _case(8, 2, 3, 8, 2, 128, start, slack=2)
    want = _run(q, pages, table, start, scale=0.3)
    _check(q, pages, table, start, None, _chain, want, scale=0.3)
    wide = torch.randn(2, 8, 3, 256, device=DEV).bfloat16()
    wide[..., 128:] = q.transpose(1, 2)
    out = torch.zeros(2, 3, 16, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(2, 3, 8, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    sv.attention_cache4(wide.transpose(1, 2)[..., 128:], pages, _i32(table), _i32(start), scale=0.3,
                        out=out[:, :, ::2], lse=lse, stream=st)
    st.synchronize()
    assert torch.equal(out[:, :, ::2], want[0]) and torch.equal(lse, want[1])
    assert (out[:, :, 1::2] == 0).all()
    for _ in range(3):  # the same bits each time
        again = _run(q, pages, table, start, scale=0.3)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    only = sv.attention_cache4(q, pages, _i32(table), _i32(start), scale=0.3)
    assert torch.equal(only, want[0])


@pytest.mark.parametrize("B,T,Hq,H,D,lo,hi", [(64, 6, 32, 8, 128, 0, 700), (300, 2, 4, 2, 64, 0, 200),
                                              (1, 3, 8, 8, 128, 20011, 20011), (1100, 1, 2, 1, 64, 0, 70)])
def test_larger_batches(B, T, Hq, H, D, lo, hi):
    """Many sequences and long ones, on the device in 64 bits: the plain form is checked above on
    small ones, here the values come from cache4_read."""
    rs = np.random.default_rng(B)
    start = rs.integers(lo, hi + 1, B)
    q, pages, table = _case(9, B, T, Hq, H, D, list(start))
    out, lse = _run(q, pages, table, start)
    L = int(start.max()) + T
    K, V = sv.cache4_read(pages, _i32(table), _i32([0] * B), table.shape[1] * 64, D, dtype=torch.float32)
    K, V = (x[:, :L].double().repeat_interleave(Hq // H, 2) for x in (K, V))
    s = torch.einsum("bihd,bxhd->bihx", q.double(), K) / D ** 0.5
    see = torch.arange(L, device=DEV)[None, None] <= _i32(start)[:, None, None] + torch.arange(T, device=DEV)[:, None]
    s = s.masked_fill(~see[:, :, None], -float("inf"))
    p = torch.softmax(s, -1)
    want, mag = torch.einsum("bihx,bxhd->bihd", p, V), torch.einsum("bihx,bxhd->bihd", p, V.abs())
    few = 2.0 ** -16 + L * 2.0 ** -24  # scores stay below 2^7: (D + 2) 2^-24 of their magnitudes
    off = (out.double() - want).abs()
    assert (off <= (2.0 ** -8 + few) * (mag * (1 + 2.0 ** -8) + want.abs())).all()
    assert ((lse.double() - torch.logsumexp(s, -1)).abs() <= 2 * few + 2.0 ** -18).all()


def test_captured_calls():
    """Two graphs captured on one stream and replayed on two at once, with new lengths between the
    replays: their scratch is their own."""
    q, pages, table = _case(10, 4, 5, 8, 2, 128, [900] * 4)
    t, n = _i32(table), len(pages)
    jobs = []
    for seed in range(2):
        qq = q if seed == 0 else q.flip(0).contiguous()
        start = _i32([900, 0, 333, 64])
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            sv.attention_cache4(qq, pages, t, start, return_lse=True)
        torch.cuda.current_stream().wait_stream(s)
        with torch.cuda.graph(g):
            out = sv.attention_cache4(qq, pages, t, start, return_lse=True)
        jobs.append((qq, start, g, out, torch.cuda.Stream()))
    for lengths in ([900, 0, 333, 64], [1, 2, 3, 4], [512, 700, 0, 900], [900, 0, 333, 64]):
        for _, start, *_ in jobs:
            start.copy_(_i32(lengths))
        torch.cuda.synchronize()
        for _, _, g, _, st in jobs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for qq, start, _, out, _ in jobs:
            want = sv.attention_cache4(qq, pages, t, start, return_lse=True)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert len(pages) == n


@pytest.mark.parametrize("B,T,Hq,H,D,lo,hi,kind", [
    (40, 6, 16, 2, 128, 0, 1500, "chain"),     # sequences of one page beside ones over several workgroups
    (24, 21, 16, 4, 64, 1000, 1400, "tree"),   # two blocks of rows to a head
    (5, 9, 16, 8, 256, 900, 2200, "chain"),    # few segments, each over many workgroups
    (33, 2, 2, 2, 64, 0, 1300, "counts"),      # some without a new token
    (33, 2, 2, 2, 64, 0, 2600, "counts"),
    (7, 3, 16, 1, 256, 900, 3000, "chain"),    # three blocks of rows to a head of 256
    (3, 40, 8, 2, 128, 0, 9000, "tree"),
    (70, 3, 4, 2, 128, 1100, 1500, "faults"),  # ill-formed ones and pages outside the pool between them
    (6, 3, 8, 2, 128, 3000, 6000, "faults"),
])
def test_sequences_cut_over_workgroups(B, T, Hq, H, D, lo, hi, kind):
    rs = np.random.default_rng([B, T, D])
    start = rs.integers(lo, hi + 1, B)
    q, pages, table = _case(11, B, T, Hq, H, D, list(start))
    count, see = [T] * B, np.tril(np.ones((T, T), bool))[None].repeat(B, 0)
    kw, gone = {}, []
    if kind == "tree":
        par = [-1] + [int(rs.integers(0, i)) for i in range(1, T)]
        one = np.zeros((T, T), bool)
        for i in range(T):
            one[i] = one[par[i]] if i else one[i]
            one[i, i] = True
        see, kw["mask"] = one[None].repeat(B, 0), sv.tree_mask(par).to(DEV)
    if kind == "counts":
        count = rs.integers(0, T + 1, B).tolist()
    if kind == "faults":
        count = rs.integers(0, T + 1, B).tolist()
        gone = [0, 2, B - 1]
        start[0], count[2], count[B - 1] = -1, T + 1, 2
        table[B - 1, int(start[B - 1]) // 128] = len(pages)
    out, lse = _run(q, pages, table, list(start), count if "mask" not in kw else None, **kw)
    new = [T if b in gone[:2] else count[b] for b in range(B)]
    live = torch.arange(T, device=DEV)[None] < _i32(new)[:, None]
    assert (out[~live] == 7).all() and (lse[~live] == 7).all()
    for b in gone:
        assert torch.isnan(out[b][live[b]]).all() and torch.isnan(lse[b][live[b]]).all()
        live[b] = False
        table[b], start[b] = 0, 0
    K, V = sv.cache4_read(pages, _i32(table), _i32([0] * B), table.shape[1] * 64, D, dtype=torch.float32)
    L = int((start + T).max())
    x = torch.arange(L, device=DEV)[None, None] - _i32(start)[:, None, None]
    sees = (x < 0) | (torch.gather(torch.tensor(see, device=DEV), 2, x.clamp(0, T - 1).expand(B, T, L)) & (x < T))
    for b in range(B):
        kb, vb = (y[b, :L].double().repeat_interleave(Hq // H, 1).transpose(0, 1).contiguous() for y in (K, V))
        qb = q[b].double().transpose(0, 1).contiguous()  # [Hq][T][D]
        s = (qb @ kb.transpose(1, 2).contiguous() / D ** 0.5).masked_fill(~sees[b][None], -float("inf"))
        p = torch.softmax(s, -1)
        want, mag = p @ vb, p @ vb.abs()
        most = (qb.abs() @ kb.abs().transpose(1, 2).contiguous()).max() / D ** 0.5
        few = most * 2 * (D + 2) * 2.0 ** -24 + 2.0 ** -21 + L * 2.0 ** -24
        off = (out[b].double().transpose(0, 1) - want).abs()
        ok = off <= (2.0 ** -8 + few) * (mag * (1 + 2.0 ** -8) + want.abs())
        assert ok[:, live[b]].all(), b
        l = torch.logsumexp(s, -1)
        ok = (lse[b].double().t() - l).abs() <= few + l.abs() * 2.0 ** -21
        assert ok[:, live[b]].all(), b


@pytest.mark.parametrize("T,Hq,H,D", [(256, 2, 1, 64), (1, 128, 1, 128), (2, 96, 2, 256)])
def test_many_rows_to_a_head(T, Hq, H, D):
    start = [70]
    q, pages, table = _case(12, 1, T, Hq, H, D, start)
    _check(q, pages, table, start, None, _chain, _run(q, pages, table, start))


def test_a_pool_past_32_bits():
    """Records past 4 GiB of a pool, read and written there as in a small one."""
    B, T, Hq, H, D, start = 2, 3, 16, 8, 256, [1200, 70]
    q, pages, table = _case(13, B, T, Hq, H, D, start)
    n, P = 40000, table.shape[1]
    big = torch.empty(n, H, 68 * D, dtype=torch.uint8, device=DEV)
    far = n - 1 - np.arange(B * P).reshape(B, P)
    big[torch.tensor(far, device=DEV).view(-1)] = pages[torch.tensor(table, device=DEV).long().view(-1)]
    k, v = (torch.randn(B, T, H, D, device=DEV).bfloat16() for _ in range(2))
    for pool, t in ((pages, table), (big, far)):
        sv.cache4_write(pool, _i32(t), _i32(start), k, v)
    for a, b in zip(_run(q, pages, table, start), _run(q, big, far, start)):
        assert torch.equal(a, b)
    for a, b in zip(sv.cache4_read(pages, _i32(table), _i32(start), T, D),
                    sv.cache4_read(big, _i32(far), _i32(start), T, D)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("start", [[0, 5], [1100, 70]])
def test_no_new_tokens(start):
    q, pages, table = _case(14, 2, 2, 2, 1, 64, start)
    out, lse = _run(q, pages, table, start, [0, 0])
    assert (out == 7).all() and (lse == 7).all()
    K = torch.ones(2, 2, 1, 64, device=DEV)
    before = pages.clone()
    sv.cache4_write(pages, _i32(table), _i32(start), K, K, count=_i32([0, 0]))
    assert torch.equal(pages, before)


@pytest.mark.parametrize("Hq,H,start", [(1024, 1024, [5]), (16384, 1, [2])])
def test_the_most_heads(Hq, H, start):
    q, pages, table = _case(15, 1, 1, Hq, H, 64, start)
    _check(q, pages, table, start, None, _chain, _run(q, pages, table, start))


def test_the_most_heads_over_cut_pages():
    """Every kv head holds the same values as the first: so do its query heads' outputs."""
    H, start = 1024, [1290]
    q, one, table = _case(15, 1, 1, 2, 1, 64, start)
    got = _run(q.repeat(1, 1, H, 1), one.expand(-1, H, -1).contiguous(), table, start)
    _check(q, one, table, start, None, _chain, tuple(x[:, :, :2].contiguous() for x in got))
    for x in got:
        x = x.view(H, 2, -1)
        assert (x - x[:1]).abs().max() <= 2.0 ** -7  # cut at other pages: a step of bf16 below 2


def test_the_most_sequences():
    """65,536 sequences, without and with new tokens, on pages that many of them share."""
    B, D = 65536, 64
    rs = np.random.default_rng(16)
    q, pages, _ = _case(16, 1, 1, 1, 1, D, [0], spare=2)
    n = len(pages)
    q = torch.tensor(rs.normal(0, 1, (B, 1, 1, D)), dtype=torch.float32).bfloat16().to(DEV)
    table, start, count = rs.integers(0, n, (B, 1)), rs.integers(0, 63, B), rs.integers(0, 2, B)
    out, lse = _run(q, pages, table, list(start), list(count))
    K, V = sv.cache4_read(pages, _i32(np.arange(n)[:, None]), _i32([0] * n), 64, D, dtype=torch.float32)
    for b0 in range(0, B, 8192):
        part = slice(b0, b0 + 8192)
        t, c = torch.tensor(table[part, 0], device=DEV), torch.tensor(count[part], device=DEV).bool()
        k, v = K[t, :, 0].double(), V[t, :, 0].double()
        s = (k * q[part, :, 0].double()).sum(-1) / D ** 0.5
        s = s.masked_fill(torch.arange(64, device=DEV) > torch.tensor(start[part], device=DEV)[:, None], -float("inf"))
        p = torch.softmax(s, -1)[..., None]
        want, mag = (p * v).sum(1), (p * v.abs()).sum(1)
        most = (k.abs() * q[part, :, 0].double().abs()).sum(-1).max() / D ** 0.5
        few = most * 2 * (D + 2) * 2.0 ** -24 + 2.0 ** -21 + 64 * 2.0 ** -24
        off = (out[part, 0, 0].double() - want).abs()
        assert (off <= (2.0 ** -8 + few) * (mag * (1 + 2.0 ** -8) + want.abs()))[c].all()
        l = torch.logsumexp(s, -1)
        assert ((lse[part, 0, 0].double() - l).abs() <= few + l.abs() * 2.0 ** -21)[c].all()
        assert (out[part][~c] == 7).all() and (lse[part][~c] == 7).all()


@pytest.mark.parametrize("B,T,Hq,H,D,lo,hi", [(64, 6, 32, 8, 128, 100, 2000), (1, 9, 32, 8, 128, 20000, 20000),
                                              (16, 21, 32, 4, 128, 37, 2000), (48, 40, 8, 8, 64, 0, 1500),
                                              (8, 4, 16, 4, 256, 0, 3000)])
def test_two_streams_at_once(B, T, Hq, H, D, lo, hi):
    """The same bits from every call, whatever runs beside it."""
    start = np.random.default_rng(17).integers(lo, hi + 1, B)
    q, pages, table = _case(17, B, T, Hq, H, D, list(start))
    t, s = _i32(table), _i32(start)
    want = sv.attention_cache4(q, pages, t, s, return_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [sv.attention_cache4(q, pages, t, s, return_lse=True, stream=st) for st in streams]
        torch.cuda.synchronize()
        for out, lse in got:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
