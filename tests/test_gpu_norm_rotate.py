"""Norms of queries and keys with their rotation against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests import step_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _freq(n, base=10000.0):
    return (base ** (-torch.arange(n, dtype=torch.float64) / max(1, n))).float().to(DEV)


def _check(x, y, weight, eps, freq, pos, interleaved, count=None, old=0.0):
    """Against the formula.  In F32 a norm is off by 2^-20 at most (the sum of D squares as 8 and
    then log2 D / 8 additions, the mean, halved by the root; the root's reciprocal to a unit in the
    last place; the product and the weight), an angle's cosine and sine by 2^-21 (the turn's part
    rounded to 2^-25, times 2 pi, and two units in the last place), their products by 2^-23: 2^-19 of
    the magnitudes that an element is made of, and the output's rounding."""
    B, T = x.shape[:2]
    w = None if weight is None else weight.double().cpu().numpy()
    f = None if freq is None else freq.cpu().numpy()
    a, got = x.double().cpu().numpy(), y.double().cpu().numpy()
    for b in range(B):
        n = T if count is None else count[b]
        for i in range(n):
            want, size = plain.rotate(a[b, i], w, eps, f, pos(b, i), interleaved)
            off = np.abs(got[b, i] - want)
            bound = size * 2.0 ** -19 * (1 + HALF[y.dtype]) + np.abs(want) * HALF[y.dtype] + 2.0 ** -126
            assert (off <= bound).all(), (b, i, (off / bound).max())
        assert (got[b, n:] == old).all()


@pytest.mark.parametrize("D,rot", [(16, 16), (64, 64), (64, 32), (80, 80), (96, 48), (128, 128), (128, 0),
                                   (128, 16), (192, 192), (256, 256), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,to", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_heads(D, rot, interleaved, dtype, to):
    rs = torch.Generator().manual_seed(D + rot)
    B, T, Hq, H = 2, 3, 7, 2
    qkv = (torch.randn(B, T, Hq + 2 * H, D, generator=rs) * 2).to(dtype).to(DEV)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H]
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=rs)).to(dtype).to(DEV) for _ in range(2))
    start, freq = [5, 131003], _freq(rot // 2) if rot else None
    yq, yk = sv.norm_rotate(q, k, _i32(start), eps=1e-6, q_weight=wq, k_weight=wk, inv_freq=freq,
                            interleaved=interleaved, out_dtype=to)
    assert yq.dtype == yk.dtype == to
    for x, y, w in ((q, yq, wq), (k, yk, wk)):
        _check(x, y, w, 1e-6, freq, lambda b, i: start[b] + i, interleaved)


@pytest.mark.parametrize("B,T,Hq,H", [(1, 1, 1, 0), (1, 1, 0, 1), (1, 1, 33, 1), (3, 1, 64, 8), (1, 300, 4, 4),
                                      (70, 2, 5, 1), (2, 2500, 3, 1)])
def test_sizes(B, T, Hq, H):
    rs = torch.Generator().manual_seed(B * T)
    start = [(7919 * b) % 100000 for b in range(B)]
    q = torch.randn(B, T, Hq, 64, generator=rs).bfloat16().to(DEV) if Hq else None
    k = torch.randn(B, T, H, 64, generator=rs).bfloat16().to(DEV) if H else None
    got = sv.norm_rotate(q, k, _i32(start), eps=1e-5, inv_freq=_freq(32))
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
        else:
            _check(x, y, None, 1e-5, _freq(32), lambda b, i: start[b] + i, False)


def test_no_norm_no_rotation_is_a_copy():
    q = torch.randn(2, 3, 4, 64, device=DEV)
    k = torch.randn(2, 3, 1, 64, device=DEV)
    yq, yk = sv.norm_rotate(q, k, _i32([0, 0]))
    assert torch.equal(yq, q) and torch.equal(yk, k)
    yq, _ = sv.norm_rotate(q, None, _i32([0, 9]), out_dtype=BF16)
    assert torch.equal(yq, q.bfloat16())


@pytest.mark.parametrize("interleaved", [False, True])
def test_depths_counts_and_far_positions(interleaved):
    """Positions of a tree's depths, one for all and one for each; rows behind a sequence's last
    token stay; positions up to 2^30 keep their angles, whose F32 products would be off by turns."""
    B, T, D = 3, 6, 128
    start, count = [0, 1 << 30, 999_999], [6, 4, 0]
    depth = torch.tensor([[0, 1, 1, 2, 2, 2], [0, 0, 5, -3, 7, 1], [0] * 6], dtype=torch.int32)
    q, k = torch.randn(B, T, 3, D, device=DEV), torch.randn(B, T, 2, D, device=DEV)
    for dep in (depth, depth[1:2], None):
        at = (lambda b, i: start[b] + i) if dep is None else (lambda b, i: start[b] + int(dep[b % len(dep), i]))
        out = [torch.full_like(q, 7.0), torch.full_like(k, 7.0)]
        got = sv.norm_rotate(q, k, _i32(start), eps=1e-6, inv_freq=_freq(64), interleaved=interleaved,
                             count=_i32(count), depth=None if dep is None else dep.to(DEV), out=out)
        assert got[0] is out[0] and got[1] is out[1]
        for x, y in zip((q, k), out):
            _check(x, y, None, 1e-6, _freq(64), at, interleaved, count, old=7.0)
        fresh = sv.norm_rotate(q, k, _i32(start), eps=1e-6, inv_freq=_freq(64), interleaved=interleaved,
                               count=_i32(count), depth=None if dep is None else dep.to(DEV))
        assert all((f[b, count[b]:] == 0).all() and torch.equal(f[b, :count[b]], o[b, :count[b]])
                   for f, o in zip(fresh, out) for b in range(B))


def test_counts_outside_the_call_become_nan():
    q = torch.randn(3, 2, 2, 64, device=DEV)
    for interleaved in (False, True):
        y, _ = sv.norm_rotate(q, None, _i32([0, 0, 0]), eps=1e-6, inv_freq=_freq(32), count=_i32([-1, 2, 3]),
                              interleaved=interleaved)
        assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all() and torch.isfinite(y[1]).all()


def test_in_place_over_the_projection():
    qkv = torch.randn(2, 5, 8, 128, device=DEV).bfloat16()
    old, start = qkv.clone(), _i32([3, 70])
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    want = sv.norm_rotate(q, k, start, eps=1e-6, inv_freq=_freq(64))
    got = sv.norm_rotate(q, k, start, eps=1e-6, inv_freq=_freq(64), out=(q, k))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(qkv[:, :, 6:], old[:, :, 6:])


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e30])
@pytest.mark.parametrize("scale", [1.0, 1e-19, 1e-37, 1e19, 3e37])
def test_magnitudes(scale, eps):
    """Squares that leave F32's range on the way."""
    x = torch.randn(1, 1, 4, 128, generator=torch.Generator().manual_seed(1)) * scale
    y, _ = sv.norm_rotate(x.to(DEV), None, _i32([0]), eps=eps)
    want, size = plain.rotate(x[0, 0].double().numpy(), None, eps, None, 0, False)
    # a reciprocal root or a product below the normal range is off by half its smallest step
    bound = size * 2.0 ** -20 + 2.0 ** -126
    assert (np.abs(y[0, 0].double().cpu().numpy() - want) <= bound).all()


def test_non_finite_values_stay_in_their_heads():
    q = torch.ones(1, 3, 4, 64, device=DEV)
    q[0, 0, 1, 5], q[0, 1, 2, 7], q[0, 2, 3] = float("nan"), float("inf"), 0.0
    y, _ = sv.norm_rotate(q, None, _i32([2]), eps=0.0)
    y = y.cpu()
    assert torch.isnan(y[0, 0, 1]).all()
    # x / inf is 0, inf / inf is not a number, and neither is 0 / 0
    assert torch.isnan(y[0, 1, 2, 7]) and (y[0, 1, 2, :7] == 0).all()
    assert torch.isnan(y[0, 2, 3]).all()
    fine = torch.ones(1, 3, 4, dtype=torch.bool)
    fine[0, 0, 1] = fine[0, 1, 2] = fine[0, 2, 3] = False
    assert ((y[fine] - 1).abs() <= 2.0 ** -20).all()


def test_rows_past_4_gib_apart():
    """Strides whose offsets pass 32 bits."""
    n = (1 << 31) + 4096
    big = torch.zeros(n, dtype=BF16, device=DEV)
    q = torch.as_strided(big, (2, 1, 2, 64), (1 << 31, 64, 64, 1))
    q.copy_(torch.randn(2, 1, 2, 64))
    y, _ = sv.norm_rotate(q, None, _i32([1, 2]), eps=1e-6, inv_freq=_freq(32))
    _check(q, y, None, 1e-6, _freq(32), lambda b, i: 1 + b + i, False)


def test_another_stream():
    q = torch.randn(4, 6, 8, 128, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = sv.norm_rotate(q, None, _i32([1, 2, 3, 4]), eps=1e-6, inv_freq=_freq(64), stream=s)
    s.synchronize()
    assert torch.equal(y, sv.norm_rotate(q, None, _i32([1, 2, 3, 4]), eps=1e-6, inv_freq=_freq(64))[0])
