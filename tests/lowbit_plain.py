"""Plain 64-bit forms of the target's pass in few bits, written from the
definitions in include/specverify_lowbit.h: the 4-bit cache's records byte by
byte, attention over their values, and the 8-bit head.  Test infrastructure
(numpy, on the CPU)."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([i * 2.0 ** -9 for i in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])
PAGE = 64


def exponent(amax, top):
    """Exponent byte of the smallest power of two >= 2^-126 whose top-fold holds amax."""
    p = -126
    while top * 2.0 ** p < amax:
        p += 1
    return p + 127


def nearest(x, grid):
    """Index of the grid value nearest to each |x|, ties to the even index."""
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    dl, dh = a - grid[hi - 1], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, hi - 1)


def group4(x):
    """(codes, exponent byte) of one group of 32 finite values."""
    e = exponent(np.abs(x).max(), 6.0)
    c = nearest(x * 2.0 ** (127 - e), E2M1)
    return c + 8 * np.signbit(x), e


def token4(k, v):
    """((codes, exponents) of k, of v) [D], [D / 32] of one (token, head)."""
    G = len(k) // 32
    if not (np.isfinite(k).all() and np.isfinite(v).all()):
        z = np.zeros(len(k), int)
        return (z, np.full(G, 255)), (z, np.full(G, 1))
    got = []
    for x in (k, v):
        parts = [group4(x[32 * g: 32 * g + 32].astype(np.float64)) for g in range(G)]
        got.append((np.concatenate([c for c, _ in parts]).astype(int),
                    np.array([e for _, e in parts])))
    return got[0], got[1]


def value4(codes, e):
    x = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes % 8]
    return x * np.repeat(2.0 ** (e.astype(np.float64) - 127), 32)


def offsets(t, D):
    """Byte offsets in a record of token t: key codes, key exponents, value codes, value exponents."""
    G = D // 32
    j, g = np.arange(D // 2), np.arange(G)
    kc = t * (D // 2) + j
    ke = 32 * D + (g * 16 + t % 16) * 4 + t // 16
    vc = 32 * D + 64 * G + (((t // 16 * 4 + t % 16 // 4) * 16 + j // G) * 4 + t % 4) * G + j % G
    ve = 64 * D + 64 * G + ((t // 16 * 4 + t % 16 // 4) * G + g) * 4 + t % 4
    return kc, ke, vc, ve


def store(pages, table, b, h, pos, k, v):
    """Writes one (token, head) into pages [n][H][68 D] (a dropped one where the page is bad)."""
    D, page = len(k), table[b, pos // PAGE]
    if not 0 <= page < len(pages):
        return
    (kc, ke), (vc, ve) = token4(k, v)
    for at, x in zip(offsets(pos % PAGE, D), (kc[0::2] + 16 * kc[1::2], ke, vc[0::2] + 16 * vc[1::2], ve)):
        pages[page, h, at] = x


def fetch(pages, table, b, h, pos, D):
    """(k, v) [D] of one (position, head): NaN where its page is bad or it is held as NaN."""
    page = table[b, pos // PAGE]
    if not 0 <= page < len(pages):
        return np.full(D, np.nan), np.full(D, np.nan)
    kc, ke, vc, ve = (pages[page, h, at].astype(int) for at in offsets(pos % PAGE, D))
    if ke[0] == 255:
        return np.full(D, np.nan), np.full(D, np.nan)
    return tuple(value4(np.stack([c & 15, c >> 4], -1).reshape(-1), e) for c, e in ((kc, ke), (vc, ve)))


def fits(start, n, T, cols):
    return start >= 0 and 0 <= n <= T and start + n <= cols * PAGE


def attention(q, pages, table, start, count, sees, scale):
    """(out, lse, bound of out, bound of lse): q [B][T][Hq][D] float64; sees(b, i, j): whether new
    token i sees new token j.  Rows past count[b] are None-marked by NaN in the bounds.

    Bounds: scores carry D roundings of the fp32 sum and one of the product with c, each 2^-24 of
    the summed magnitudes (e); a probability then e + 2^-22 (exp2 and the running maximum's
    factors) and, for the second product, 2^-8 of bf16; the sums over L positions L 2^-24; out is
    rounded to bf16 once, 2^-8."""
    B, T, Hq, D = q.shape
    H = pages.shape[1]
    out, lse = np.zeros(q.shape), np.zeros((B, T, Hq))
    bo, bl = np.full(q.shape, np.nan), np.full((B, T, Hq), np.nan)
    for b in range(B):
        n = int(count[b])
        if not fits(int(start[b]), n, T, table.shape[1]):
            out[b], lse[b], bo[b], bl[b] = np.nan, np.nan, 0, 0
            continue
        L = int(start[b]) + n
        bad = any(not 0 <= table[b, p] < len(pages) for p in range(-(-L // PAGE)))
        for h in range(H if n else 0):
            kv = [fetch(pages, table, b, h, x, D) for x in range(L)]
            K, V = np.array([x[0] for x in kv]), np.array([x[1] for x in kv])
            for i in range(n):
                see = np.array([x < start[b] or sees(b, i, x - start[b]) for x in range(L)], bool)
                for g in range(Hq // H):
                    at = (b, i, h * (Hq // H) + g)
                    if bad:
                        out[at], lse[at], bo[at], bl[at] = np.nan, np.nan, 0, 0
                        continue
                    if not see.any():
                        out[at], lse[at], bo[at], bl[at] = 0, -np.inf, 0, 0
                        continue
                    s = K[see] @ q[at] * scale
                    e = (np.abs(K[see]) @ np.abs(q[at]) * scale).max() * (D + 2) * 2.0 ** -24
                    m = s.max()
                    p = np.exp(s - m)
                    lse[at] = m + np.log(p.sum())
                    p /= p.sum()
                    out[at] = p @ V[see]
                    few = e * 2 + 2.0 ** -21 + L * 2.0 ** -24
                    bo[at] = (2.0 ** -8 + few) * (p @ np.abs(V[see])) * (1 + 2.0 ** -8) + \
                        (2.0 ** -8 + few) * np.abs(out[at]) + 1e-38
                    bl[at] = few + np.abs(lse[at]) * 2.0 ** -22 + np.abs(m) * 2.0 ** -22
    return out, lse, bo, bl


def block8(x):
    """(e4m3 values over the scale, scale) of one block; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    p = 2.0 ** (exponent(np.abs(x[fine]).max() if fine.any() else 0.0, 448.0) - 127)
    y = np.full(x.shape, np.nan)
    y[fine] = np.sign(x[fine]) * E4M3[nearest(x[fine] / p, E4M3)]
    return y, p


def quantize8(w):
    V, d = w.shape
    q, s = np.zeros((V, d)), np.zeros((-(-V // 128), -(-d // 128)))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            a = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
            q[a], s[i, j] = block8(w[a])
    return q, s


def head8(hidden, q, scale):
    """(logits, sum of magnitudes) of hidden [M][d]."""
    M, d = hidden.shape
    h = np.zeros((M, d))
    for m in range(M):
        for j in range(0, d, 128):
            y, p = block8(hidden[m, j:j + 128])
            h[m, j:j + 128] = y * p
    w = q * np.repeat(np.repeat(scale, 128, 0)[: len(q)], 128, 1)[:, :d]
    return h @ w.T, np.abs(h) @ np.abs(w).T


def inv_sqrt(D):
    return 1.0 / math.sqrt(D)
