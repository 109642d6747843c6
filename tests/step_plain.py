"""Plain 64-bit forms of the serving step around the cached pass, written from
the definitions in include/specverify_step.h: norms with rotation, attention
over positions of the 4-bit cache that a rule names, and pages reserved and
given back.  Test infrastructure (numpy and lists, on the CPU)."""
import numpy as np

from tests import lowbit_plain as low

PAGE = low.PAGE


def held(pages, row, n, D):
    """K and V [n][H][D] of a sequence's first n positions; NaN where its page is bad or what it
    holds is; and whether all its pages are good."""
    H, G = pages.shape[1], D // 32
    k, v = np.full((n, H, D), np.nan), np.full((n, H, D), np.nan)
    good = True
    at = [low.offsets(t, D) for t in range(PAGE)]
    where = [np.stack([x[i] for x in at]) for i in range(4)]  # [64][bytes]
    for p in range(-(-n // PAGE)):
        if not 0 <= row[p] < len(pages):
            good = False
            continue
        m = min(PAGE, n - p * PAGE)
        rec = pages[row[p]].astype(np.int64)  # [H][68 D]
        kc, ke, vc, ve = (rec[:, w[:m]].transpose(1, 0, 2) for w in where)
        for c, e, x in ((kc, ke, k), (vc, ve, v)):
            codes = np.stack([c & 15, c >> 4], -1).reshape(m, H, D)
            y = np.where(codes >= 8, -1.0, 1.0) * low.E2M1[codes % 8]
            with np.errstate(over="ignore"):
                y = y * np.repeat(2.0 ** (e.astype(np.float64) - 127), 32, -1)
            x[p * PAGE: p * PAGE + m] = np.where((ke[:, :, :1] == 255), np.nan, y)
    return k, v, good


def attend(q, k, v, see, scale, more=0.0):
    """(out, lse, bounds of both) of one new token's head q [D] over positions k, v [L][D], of which
    it sees `see`; the bounds are derived in lowbit_plain.attention; `more`: further relative error
    of the probabilities (where two parts are joined: a factor exp2 and two roundings each, 2^-21)."""
    D = len(q)
    if not see.any():
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    ks, vs = k[see], v[see]
    if np.isnan(ks).any() or np.isnan(q).any():
        return np.full(D, np.nan), np.nan, np.zeros(D), 0.0
    s = ks @ q * scale
    e = (np.abs(ks) @ np.abs(q) * scale).max() * (D + 2) * 2.0 ** -24
    m = s.max()
    p = np.exp(s - m)
    lse = m + np.log(p.sum())
    p /= p.sum()
    out = p @ vs
    few = e * 2 + 2.0 ** -21 + len(s) * 2.0 ** -24 + more
    bo = (2.0 ** -8 + few) * (p @ np.abs(vs)) * (1 + 2.0 ** -8) + (2.0 ** -8 + few) * np.abs(out) + 1e-38
    return out, lse, bo, few + np.abs(lse) * 2.0 ** -22 + np.abs(m) * 2.0 ** -22


def window_sees(start, n, T, sees, depth, masked, window, sinks):
    """[n][start + n]: which positions each new token sees."""
    x = np.arange(start + n)
    got = np.zeros((n, start + n), bool)
    for i in range(n):
        at = start + (min(max(int(depth[i]), 0), T - 1) if depth is not None else i)
        near = (x > at - window) | (x < sinks)
        got[i] = near & (x < start)
        new = np.array([sees(i, j) for j in range(n)], bool)
        got[i, start:] = new if masked else new & near[start:]
    return got


def rotate(x, weight, eps, inv_freq, pos, interleaved):
    """(y, sum of the magnitudes that an element of y is made of) of heads x [..., D] (float64) at
    one position."""
    D = x.shape[-1]
    y = x
    if eps is not None:
        with np.errstate(all="ignore"):
            y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        if weight is not None:
            y = y * weight
    size = np.abs(y)
    if inv_freq is not None:
        n = len(inv_freq)
        a = np.float64(pos) * inv_freq.astype(np.float64)
        c, s = np.cos(a), np.sin(a)
        u, v = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        y, size = y.copy(), size.copy()
        yu, yv = y[..., u].copy(), y[..., v].copy()
        y[..., u], y[..., v] = yu * c - yv * s, yv * c + yu * s
        size[..., u] = size[..., v] = np.abs(yu) + np.abs(yv)
    return y, size


def reserve(table, held_, need, free, count):
    """The call on lists of lists, in place: table rows, held, free (its capacity long); returns the
    new free count."""
    cols, cap = len(table[0]), len(free)
    want = []
    for b in range(len(table)):
        w = -(-need[b] // PAGE)
        want.append(w if need[b] >= 0 and 0 <= held_[b] <= cols and w <= cols else held_[b])
    back = [(b, p) for b in range(len(table)) for p in range(want[b], held_[b])]
    if not 0 <= count <= count + len(back) <= cap:
        return count
    for b, p in reversed(back):
        free[count] = table[b][p]
        table[b][p] = -1
        count += 1
    for b in range(len(table)):
        held_[b] = min(held_[b], want[b])
    for b in range(len(table)):
        miss = want[b] - held_[b]
        if miss > count:
            break
        for p in range(held_[b], want[b]):
            count -= 1
            table[b][p] = free[count]
        held_[b] = want[b]
    return count
