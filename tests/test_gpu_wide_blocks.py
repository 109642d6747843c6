"""Attention of many rows of a kv head, in several blocks, by kernels whose waves share each page: the
last block has every size at which two waves hold the same rows.  All rows of a call against the
formula in 64 bits, whole and cut over workgroups, and each call twice."""
import pytest
import torch

import draft_token_verification_11_amd as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool(n, H, D, g):
    """n pages of random values."""
    pages = sv.cache4_alloc(n, H, D, DEV)
    k, v = (torch.randn(1, n * 64, H, D, generator=g, device=DEV) for _ in range(2))
    sv.cache4_write(pages, _i32([list(range(n))]), _i32([0]), k, v)
    return pages


def _held(pages, table, lens, D):
    """K and V [rows of the table][max(lens)][H][D] of the first lens[b] positions of each row."""
    return sv.cache4_read(pages, table.contiguous(), _i32([0] * len(lens)), max(1, max(lens)), D, count=_i32(lens), dtype=torch.float32)


def _rows_agree(got, q, k, v, see, more=0.0):
    """Rows q [n][Hq][D] of a sequence, each over those of k, v [L][H][D] that `see` [n][L] names, within
    the bounds of tests/step_plain.py's `attend` (derived in tests/lowbit_plain.py's `attention`)."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    a = q.double().view(n, H, Hq // H, D).transpose(0, 1).reshape(H, -1, D)  # [H][n G][D]
    kt, vh = k.double().permute(1, 2, 0).contiguous(), v.double().transpose(0, 1).contiguous()
    see = see[:, None].expand(n, Hq // H, L).reshape(1, -1, L)
    s = (torch.matmul(a, kt) * D ** -0.5).masked_fill(~see, -torch.inf)
    size = (torch.matmul(a.abs(), kt.abs()) * D ** -0.5).masked_fill(~see, 0).amax(-1)
    m, lse = s.amax(-1), torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    want = torch.matmul(p, vh)
    few = size * (D + 2) * 2.0 ** -23 + 2.0 ** -21 + see.sum(-1) * 2.0 ** -24 + more
    bound = (2.0 ** -8 + few)[..., None] * (torch.matmul(p, vh.abs()) * (1 + 2.0 ** -8) + want.abs()) + 1e-38
    back = lambda x: x.view(H, n, Hq // H, -1).transpose(0, 1).reshape(n, Hq, -1)  # noqa: E731
    assert ((got[0].double() - back(want)).abs() <= back(bound)).all()
    assert ((got[1].double() - back(lse)[..., 0]).abs() <= back(few + (lse.abs() + m.abs()) * 2.0 ** -22)[..., 0]).all()


def _twice(call, shape):
    """The outputs of a call, once it has given the same ones again; rows that it leaves are 7."""
    got = []
    for _ in range(2):
        out = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full(shape[:-1], 7.0, device=DEV)
        call(out=out, lse=lse)
        got.append((out, lse))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    return got[0]


def _tiles(rows, D):
    """Blocks of rows, and the last one's tiles of 16: blocks of up to 12 or 8, as even as can be."""
    t, most = -(-rows // 16), 12 if D == 128 else 8
    blocks = -(-t // most)
    return blocks, t - (blocks - 1) * -(-t // blocks)


# 512 (sequence, kv head) pairs of heads of 128, fewer of 256: (B, Hq, H, D, T, tiles of the last block)
@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("B,Hq,H,D,T,last", [
    (8, 1024, 64, 128, 133, 1), (8, 512, 64, 128, 243, 2), (8, 512, 64, 128, 221, 3), (8, 512, 64, 128, 222, 3),
    (8, 1024, 64, 128, 111, 3), (8, 512, 64, 128, 199, 4), (8, 512, 64, 128, 177, 5), (8, 512, 64, 128, 201, 5),
    (8, 512, 64, 128, 225, 5), (8, 448, 64, 128, 202, 5), (8, 512, 64, 128, 121, 6), (8, 512, 64, 128, 256, 8),
    (8, 128, 16, 256, 130, 1), (8, 128, 16, 256, 100, 2), (8, 128, 16, 256, 101, 3), (16, 128, 16, 256, 50, 4)])
def test_windows(B, Hq, H, D, T, last, cut):
    assert _tiles(T * Hq // H, D)[1] == last
    g = torch.Generator(DEV).manual_seed(T + Hq)
    start, count = [(b * 131) % 500 for b in range(B)], [T - 5 * (b % 4 == 3) for b in range(B)]
    P = -(-(max(start) + T) // 64)
    pages = _pool(B * P, H, D, g)
    order = torch.randperm(B * P, generator=g, device=DEV).to(torch.int32).view(B, P)
    # tables of up to 20 columns are not cut, nor are those of up to 72 with as many segments
    table = torch.cat([order, torch.full((B, 80 if cut else 0), -1, dtype=torch.int32, device=DEV)], 1)
    window, sinks = (1 << 20, 0) if cut else (150, 70)
    q = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    out, lse = _twice(lambda **kw: sv.attention_cache4(q, pages, table, _i32(start), count=_i32(count), window=window, sinks=sinks,
                                                       **kw), (B, T, Hq, D))
    for b, (s, n) in enumerate(zip(start, count)):
        k, v = _held(pages, order[b : b + 1], [s + n], D)
        at, x = s + torch.arange(n, device=DEV)[:, None], torch.arange(s + n, device=DEV)
        _rows_agree((out[b, :n], lse[b, :n]), q[b, :n], k[0], v[0], (x <= at) & ((x > at - window) | (x < sinks)))
        assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()


# Eight prefixes of 64 kv heads of 128, which are shared by the sizes: (fan, T, columns of the prefixes'
# tables, some rows not live, tiles of the last block).  Tables of up to 20 columns are not cut.
@pytest.mark.parametrize("fan,T,cols,counted,last", [
    (266, 1, 18, False, 1), (244, 1, 18, False, 2), (222, 1, 18, False, 3), (200, 1, 18, False, 4), (178, 1, 18, False, 5),
    (204, 1, 18, False, 6), (222, 1, 60, False, 3), (178, 1, 60, False, 5), (45, 5, 120, False, 5), (101, 2, 50, True, 5),
    (111, 2, 50, True, 3)])
def test_prefixes(fan, T, cols, counted, last):
    H, G, D, prefixes = 64, 8, 128, 8
    assert _tiles(fan * T * G, D)[1] == last
    B, Hq = prefixes * fan - 3, H * G
    g = torch.Generator(DEV).manual_seed(fan + T)
    start, count = [(b * 5) % 7 for b in range(B)], [(b * 3 + 1) % (T + 1) if counted else T for b in range(B)]
    lens = [(190, 64, 1, 129, 65, 128, 0, 77)[p] for p in range(prefixes)]
    n = B + 3 * prefixes
    pages = _pool(n, H, D, g)
    order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    table, some = order[:B, None], order[B:].view(prefixes, 3)
    ptable = torch.cat([some, torch.full((prefixes, cols - 3), -1, dtype=torch.int32, device=DEV)], 1)
    q = torch.randn(B, T, Hq, D, generator=g, device=DEV).bfloat16()
    out, lse = _twice(lambda **kw: sv.attention_cache4_shared(
        q, pages, table, _i32(start), ptable, _i32(lens), fan=fan, count=_i32(count) if counted else None, **kw), (B, T, Hq, D))
    pk, pv = _held(pages, some, lens, D)
    for b0 in range(0, B, fan):
        p, mine = b0 // fan, range(b0, min(B, b0 + fan))
        ok, ov = _held(pages, table[b0 : mine[-1] + 1], [start[b] + count[b] for b in mine], D)
        for b in mine:
            s, m = start[b], count[b]
            assert (out[b, m:] == 7).all() and (lse[b, m:] == 7).all()
            if m == 0:
                continue
            k, v = (torch.cat([x[p, : lens[p]], y[b - b0, : s + m]]) for x, y in ((pk, ok), (pv, ov)))
            x = torch.arange(lens[p] + s + m, device=DEV) - lens[p] - s
            _rows_agree((out[b, :m], lse[b, :m]), q[b, :m], k, v, x <= torch.arange(m, device=DEV)[:, None], 2.0 ** -20)
