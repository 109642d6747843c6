"""The operators around a target's cached pass, as measured: norms of queries and keys with the
position rotation, attention over the 4-bit cache through a sliding window with a few first tokens
that stay visible, attention of branches that share a long prefix, and the pages of each sequence
reserved and given back on the GPU, with the slots of its new tokens.

``run`` computes each in elementary torch operations, or, with ``own`` set, through
``draft_token_verification_11_amd``.

The cache: pages of 64 tokens, one record of 68 D bytes per (page, kv head).  D values of a token
form D / 32 groups; a group is held as 4-bit e2m1 codes and one power of two 2^(e - 127).  The
record holds, in this order,
  the key codes      [64 tokens][D / 2 bytes], the even element in a byte's low half,
  the key exponents  [D / 32 groups][16][4]: token t at [t % 16][t / 16],
  the value codes    [4][4][16][4][D / 32 bytes]: token t at [t / 16][t % 16 / 4][.][t % 4], the
                     third axis over sixteenths of D,
  the value exponents [4][4][D / 32 groups][4]: token t at [t / 16][t % 16 / 4][.][t % 4].
"""
import math

import torch

own = False

PAGE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of one sequence, far into a long text, wide heads of which a quarter is rotated
        dict(name="rotate_one", op="rotate", B=1, T=1, Hq=16, Hkv=4, D=256, rot=64, pairs=1, weights=True, lo=131003, hi=131003, ragged=False, tree=0, dtype="float32"),
        # a serving step: the last token and five drafts of 64 sequences, queries and keys out of one projection
        dict(name="rotate_step", op="rotate", B=64, T=6, Hq=32, Hkv=8, D=128, rot=128, pairs=0, weights=True, lo=1500, hi=4091, ragged=True, tree=0, dtype="bfloat16"),
        # whole prompts
        dict(name="rotate_prompt", op="rotate", B=4, T=8191, Hq=32, Hkv=8, D=128, rot=128, pairs=0, weights=True, lo=0, hi=1, ragged=False, tree=0, dtype="bfloat16"),
        # one sequence decoding a single token behind 131,000: its window and four first tokens
        dict(name="window_one", op="window", B=1, T=1, Hq=32, Hkv=8, D=64, lo=131003, hi=131003, window=1024, sinks=4, tree=0, ragged=False),
        # a window layer of a serving step: five drafts and the last token, ragged lengths
        dict(name="window_batch", op="window", B=64, T=6, Hq=32, Hkv=8, D=128, lo=1500, hi=4091, window=1024, sinks=4, tree=0, ragged=False),
        # candidate trees of 21 nodes under a wide window, some sequences shorter than it
        dict(name="window_tree", op="window", B=16, T=21, Hq=64, Hkv=8, D=128, lo=37, hi=8155, window=4001, sinks=100, tree=4, ragged=False),
        # four samples of one prompt, their first tokens: latency
        dict(name="prefix_one", op="prefix", B=4, fan=4, T=1, Hq=32, Hkv=8, D=128, plo=777, phi=777, lo=0, hi=40, tree=0, ragged=False),
        # branch fan-out: 64 requests of eight branches, four drafts each, which differ in what follows the prompt
        dict(name="prefix_branches", op="prefix", B=512, fan=8, T=5, Hq=32, Hkv=8, D=128, plo=1500, phi=4091, lo=0, hi=100, tree=0, ragged=True),
        # a whole batch behind one long common instruction, heads of 64 without sharing
        dict(name="prefix_system", op="prefix", B=96, fan=96, T=2, Hq=16, Hkv=16, D=64, plo=16411, phi=16411, lo=100, hi=2045, tree=0, ragged=False),
        # few requests of six branches with a tree of nine candidates each, heads of 256 in sevens
        dict(name="prefix_wide", op="prefix", B=24, fan=6, T=9, Hq=28, Hkv=4, D=256, plo=37, phi=8155, lo=3, hi=130, tree=3, ragged=False),
        # a step's pages: 64 sequences make room for six tokens, some have ended, and back
        dict(name="reserve_step", op="reserve", B=64, T=6, cols=512, lo=1500, hi=30000, ends=0.05),
        # many sequences, whose prompts are taken in and given back
        dict(name="reserve_prompts", op="reserve", B=4093, T=1000, cols=160, lo=0, hi=9000, ends=0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotate", "window", "window", "prefix", "prefix", "reserve"])
    if op == "reserve":
        B, T = _log(rng, 1, 4093), _log(rng, 1, 1000)
        hi = _log(rng, 1, min(30000, 36_000_000 // B))
        return dict(op=op, B=B, T=T, cols=-(-(hi + T) // PAGE) + rng.randint(0, 30), lo=rng.randint(0, hi), hi=hi, ends=rng.choice([0.0, 0.05, 0.3]))
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 4, 7, 8])
    tree = rng.choice([0, 0, 2, 4])
    if op == "rotate":
        D = 16 * rng.choice([4, 5, 6, 8, 8, 12, 16])
        B, dtype = _log(rng, 1, 128), rng.choice(["bfloat16", "bfloat16", "float32"])
        T = max(1, min(_log(rng, 1, 8191), (167_000_000 if dtype == "bfloat16" else 83_000_000) // (B * Hkv * (G + 1) * D)))
        hi = _log(rng, 1, 1_000_000)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, rot=16 * rng.randint(0, D // 16) if rng.random() < 0.4 else D, pairs=rng.choice([0, 0, 1]),
                    weights=rng.random() < 0.8, lo=rng.randint(0, hi), hi=hi, ragged=rng.random() < 0.3, tree=tree if T < 64 else 0, dtype=dtype)
    D = rng.choice([64, 128, 128, 256])
    if op == "window":
        B = _log(rng, 1, 128)
        window, sinks = _log(rng, 16, 8000), rng.choice([0, 1, 4, 4, 100])
        window = max(16, min(window, 120_000_000 // (B * Hkv * D)))
        T = max(1, min(_log(rng, 1, 33), 30_000_000 // (B * Hkv * G * window)))
        hi = _log(rng, 1, 140000)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, lo=rng.randint(0, hi), hi=hi, window=window, sinks=sinks, tree=tree, ragged=rng.random() < 0.3)
    fan, groups, T = _log(rng, 1, 100), _log(rng, 1, 64), _log(rng, 1, 21)
    groups = max(1, min(groups, 512 // fan))
    B = max(1, fan * groups - rng.randint(0, fan - 1))
    phi = min(_log(rng, 1, 32000), 240_000_000 // (groups * Hkv * D))
    phi = max(1, min(phi, 28_000_000_000 // (B * T * Hkv * G * D)))
    hi = max(1, min(_log(rng, 1, 2000), 100_000_000 // (B * Hkv * D), 100_000_000 // (B * T * Hkv * G)))
    return dict(op=op, B=B, fan=fan, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, plo=rng.randint(0, phi), phi=phi, lo=rng.randint(0, hi), hi=hi, tree=tree, ragged=rng.random() < 0.3)


def _spread(n, lo, hi):
    """n lengths over [lo, hi], out of order."""
    return [lo + (hi - lo) * ((b * 37 + 11) % n) // max(1, n - 1) if n > 1 else hi for b in range(n)]


def _counts(case):
    """New tokens of each sequence."""
    return [1 + (b * 7) % case["T"] if case["ragged"] else case["T"] for b in range(case["B"])]


def _parents(T, fan):
    return [-1] + [(i - 1) // fan if fan else i - 1 for i in range(1, T)]


def _depths(T, fan):
    """How far each new token is behind the first one: its place in a chain, or its depth in a tree."""
    parents, depth = _parents(T, fan), [0] * T
    for i in range(1, T):
        depth[i] = depth[parents[i]] + 1
    return depth


def _layout(D, device):
    """Where each byte of [key codes | key exponents | value codes | value exponents], each token by
    token, stands in a record."""
    G, t = D // 32, torch.arange(PAGE, device=device).view(PAGE, 1)
    j, g = torch.arange(D // 2, device=device), torch.arange(G, device=device)
    kc = t * (D // 2) + j
    ks = PAGE * D // 2 + g * PAGE + (t % 16) * 4 + t // 16
    quad = (t // 16) * 4 + (t % 16) // 4
    vc = PAGE * D // 2 + PAGE * G + quad * (2 * D) + (j // G) * (4 * G) + (t % 4) * G + j % G
    vs = PAGE * D + PAGE * G + quad * (4 * G) + g * 4 + t % 4
    return [x.reshape(PAGE, -1) for x in (kc, ks, vc, vs)]


def _two(e):
    """2^(e - 127) of the integers e in [1, 254], in float32."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _codes(x):
    """4-bit codes (two to a byte) and exponent bytes of x [..., D], in 32 bits."""
    D = x.shape[-1]
    x = x.float().reshape(*x.shape[:-1], D // 32, 32)
    amax = x.abs().amax(-1)
    e = (((amax.view(torch.int32) + 0x3FFFFF) >> 23) - 2).clamp_min(1)
    y = x.abs() * _two(254 - e).unsqueeze(-1)
    c = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    c = (c + 8 * torch.signbit(x).to(torch.uint8)).reshape(*x.shape[:-2], D // 2, 2)
    return c[..., 0] + 16 * c[..., 1], e.to(torch.uint8)


def _values(code, e):
    """float32 values [..., D] of code bytes [..., D / 2] and exponent bytes [..., D / 32]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    x = table[torch.stack((code & 15, code >> 4), -1).long()].reshape(*e.shape, 32)
    return (x * _two(e).unsqueeze(-1)).flatten(-2)


def _filled(n, case, g):
    """n pages of random keys, a few channels of them loud, and values."""
    dev, H, D = "cuda", case["Hkv"], case["D"]
    pages = torch.empty(n, H, 68 * D, dtype=torch.uint8, device=dev)
    loud = 1 + 3 * (torch.rand(H, D, generator=g, device=dev) < 0.03)
    at = torch.cat([x.reshape(-1) for x in _layout(D, dev)])
    step = max(1, (1 << 26) // (PAGE * H * D))
    for a in range(0, n, step):
        m = min(step, n - a)
        k = torch.randn(m, PAGE, H, D, generator=g, device=dev) * loud
        v = torch.randn(m, PAGE, H, D, generator=g, device=dev)
        parts = [y.transpose(1, 2).reshape(m, H, -1) for x in (k, v) for y in _codes(x)]
        pages[a : a + m, :, at] = torch.cat(parts, -1)
    return pages


def _mask(case, device):
    """Which of the new tokens each one attends to (itself and those before it on its path), as bits
    of 32-bit words [1][T][ceil(T / 32)]; None for a chain."""
    if not case["tree"]:
        return None
    T, parents = case["T"], _parents(case["T"], case["tree"])
    words = [[0] * (-(-T // 32)) for _ in range(T)]
    for i in range(T):
        if i:
            words[i] = list(words[parents[i]])
        words[i][i // 32] |= 1 << (i % 32)
    signed = [[w - (1 << 32) if w >> 31 else w for w in row] for row in words]
    return torch.tensor([signed], dtype=torch.int32, device=device)


def _first_seen(case, start):
    """The first position that the window of a sequence's first new token reaches."""
    return max(0, start - case["window"] + 1)


def prepare(case, seed):
    dev, g = "cuda", torch.Generator("cuda")
    g.manual_seed(seed)
    s, B, T = dict(case=case), case["B"], case["T"]
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    starts = _spread(B, case["lo"], case["hi"])
    if case["op"] == "reserve":
        cols = case["cols"]
        gone = torch.rand(B, generator=g, device=dev) < case["ends"]
        length = put(starts)
        new = 1 + torch.randint(0, T, (B,), generator=g, device=dev, dtype=torch.int32)
        s["before"], s["need"] = length, torch.where(gone, 0, length + new)
        s["start"] = torch.where(gone, 0, length)
        s["count"] = torch.where(gone, 0, new)
        s["held"] = (length + PAGE - 1) // PAGE
        first, room = [], 0
        for n in starts:
            first.append(room)
            room += -(-n // PAGE)
        s["n_pages"] = n_pages = room + B * -(-T // PAGE) + 5
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        at = put(first)[:, None] + torch.arange(cols, device=dev, dtype=torch.int32)
        mine = torch.arange(cols, device=dev) < s["held"][:, None]
        s["table"] = torch.where(mine, order[at.clamp_max(n_pages - 1).long()], -1)
        # the pool's pages that are nobody's, the next to be taken last
        s["free"] = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        s["free"][: n_pages - room] = order[room:]
        s["free_count"] = put([n_pages - room])
        return s
    H, D, counts = case["Hkv"], case["D"], _counts(case)
    s["start"], s["count"] = put(starts), put(counts) if case["ragged"] else None
    s["depth"] = put([_depths(T, case["tree"])]) if case["tree"] else None
    if case["op"] == "rotate":
        dtype, Hq, rot = getattr(torch, case["dtype"]), case["Hq"], case["rot"]
        # the projection's output: queries, keys and values of a position side by side
        qkv = torch.empty(B, T, Hq + 2 * H, D, dtype=dtype, device=dev)
        for b in range(B):
            qkv[b] = torch.randn(T, Hq + 2 * H, D, generator=g, device=dev) * 1.7
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq : Hq + H]
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / max(1, rot)).float() if rot else None
        s["weights"] = [(1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dtype) if case["weights"] else None for _ in range(2)]
        s["out"] = [torch.zeros(B, T, n, D, dtype=dtype, device=dev) for n in (Hq, H)]
        return s
    lens = [a + T for a in starts]
    P = max(-(-n // PAGE) for n in lens)
    if case["op"] == "window":
        # pages that no new token sees are nobody's any more
        keep = [[p for p in range(-(-n // PAGE)) if p * PAGE < case["sinks"] or (p + 1) * PAGE > _first_seen(case, a)] for a, n in zip(starts, lens)]
    else:
        keep = [list(range(-(-n // PAGE))) for n in lens]
        prefixes = _spread(-(-B // case["fan"]), case["plo"], case["phi"])
        s["prefix_len"] = put(prefixes)
        keep += [list(range(-(-n // PAGE))) for n in prefixes]
        P = max(P, max(1, max(-(-n // PAGE) for n in prefixes)))
    n = sum(map(len, keep)) + 3
    order, at, rows = torch.randperm(n, generator=g, device=dev).tolist(), 0, []
    for pages in keep:
        row = [-1] * P
        for p in pages:
            row[p] = order[at]
            at += 1
        rows.append(row)
    tables = put(rows)
    own_cols = max(-(-m // PAGE) for m in lens)
    s["table"] = tables[:B, :own_cols].contiguous()
    if case["op"] == "prefix":
        s["prefix_table"] = tables[B:, : max(1, max(-(-m // PAGE) for m in prefixes))].contiguous()
    s["pages"] = _filled(n, case, g)
    s["q"] = (torch.randn(B, T, case["Hq"], D, generator=g, device=dev) * 0.8).bfloat16()
    s["mask"] = _mask(case, dev)
    s["out"] = torch.zeros(B, T, case["Hq"], D, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros(B, T, case["Hq"], device=dev)
    return s


# --- the plain forms ------------------------------------------------------------------------------


def _live(s):
    """Which new tokens there are [B][T]."""
    c = s["case"]
    i = torch.arange(c["T"], device=s["start"].device)
    return i < (s["count"][:, None] if s["count"] is not None else torch.full_like(s["start"], c["T"])[:, None])


def _places(s):
    """How far each new token is behind start [1][T]."""
    return s["depth"].long() if s["depth"] is not None else torch.arange(s["case"]["T"], device=s["start"].device)[None]


def _normed(x, weight, eps):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x if weight is None else x * weight.float()


def _turned(x, cos, sin, pairs):
    """x [B][T][H][D] with its first 2 n values turned by the angles of cos, sin [B][T][1][n]."""
    n = cos.shape[-1]
    a, b = (x[..., 0 : 2 * n : 2], x[..., 1 : 2 * n : 2]) if pairs else (x[..., :n], x[..., n : 2 * n])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((y, x[..., 2 * n :]), -1)


def _plain_rotate(s):
    c = s["case"]
    pos = s["start"].long()[:, None] + _places(s)
    q, k = (_normed(x, w, 1e-6) for x, w in zip((s["q"], s["k"]), s["weights"]))
    if c["rot"]:
        angle = pos.double()[..., None, None] * s["inv_freq"].double()  # far positions: 64 bits
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q, k = (_turned(x, cos, sin, c["pairs"]) for x in (q, k))
    live = _live(s)[..., None, None]
    return tuple(torch.where(live, x.to(o.dtype), o) for x, o in zip((q, k), s["out"]))


def _at(pages, table, pos, D):
    """K and V [B][N][H][D] in float32 of positions pos [B][N]."""
    H = pages.shape[1]
    page = table.long().gather(1, pos // PAGE)
    rec = (page.clamp_min(0)[:, :, None] * H + torch.arange(H, device=pages.device)) * pages.shape[2]
    parts = [pages.view(-1)[rec[..., None] + x[pos % PAGE][:, :, None, :]] for x in _layout(D, pages.device)]
    return _values(parts[0], parts[1]), _values(parts[2], parts[3])


def _take(pages, table, D):
    """K and V [B][64 max_pages][Hkv][D] in float32 of the sequences' pages."""
    rec = pages[table.clamp_min(0).long()]  # [B][P][H][bytes]
    got = [rec[..., x.reshape(-1)].unflatten(-1, x.shape).transpose(2, 3).flatten(1, 2) for x in _layout(D, pages.device)]
    return _values(got[0], got[1]), _values(got[2], got[3])


def _new_seen(s, at):
    """Which of the new tokens at places at [B][L] (from start on) each new token sees [B][T][L]."""
    T = s["case"]["T"]
    i = torch.arange(T, device=at.device)
    if s["mask"] is None:
        return (at[:, None, :] >= 0) & (at[:, None, :] <= i[:, None])
    to = at.clamp(0, T - 1)
    words = s["mask"][0][:, to // 32].permute(1, 0, 2)  # [B][T][L]
    return (at[:, None, :] >= 0) & (at[:, None, :] < T) & ((words >> (to % 32)[:, None, :]) & 1).bool()


def _scores(q, k, scale):
    """[B][H][R][L] of q [B][R][H][D], k [B][L][H][D]."""
    return torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1).contiguous()) * scale


def _told(s, out, lse):
    """What the call leaves in out [B][T][Hq][D] and lse: rows past a sequence's new tokens stay."""
    live = _live(s)[..., None]
    return torch.where(live[..., None], out.bfloat16(), s["out"]), torch.where(live, lse, s["lse"])


def _plain_window(s):
    c, start = s["case"], s["start"].long()[:, None]
    B, T, Hq, H, D, W = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["window"]
    # the first tokens, and all that some window may reach
    first = torch.arange(c["sinks"], device=start.device).expand(B, -1)
    reach = start - W + 1 + torch.arange(W - 1 + T, device=start.device)
    pos = torch.cat((first, reach), 1)  # [B][L]
    once = torch.cat((first >= 0, reach >= c["sinks"]), 1)
    k, v = _at(s["pages"], s["table"], pos.clamp(0, s["table"].shape[1] * PAGE - 1), D)
    L, G = pos.shape[1], Hq // H
    at = pos - start
    old = (at < 0)[:, None, :] & ((pos < c["sinks"])[:, None, :] | (at[:, None, :] > _places(s)[:, :, None] - W))
    new = _new_seen(s, at)
    if s["mask"] is None:
        i = torch.arange(T, device=start.device)
        new = new & ((i[:, None] - at[:, None, :] < W) | (pos < c["sinks"])[:, None, :])
    count = s["count"].long()[:, None] if s["count"] is not None else T
    see = (old | (new & (at < count)[:, None, :])) & once[:, None, :] & (pos >= 0)[:, None, :]
    q = s["q"].float().reshape(B, T, H, G, D).transpose(2, 3).reshape(B, T * G, H, D)
    score = _scores(q, k, 1 / math.sqrt(D)).view(B, H, T, G, L).masked_fill(~see[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, H, T * G, L), v.transpose(1, 2).contiguous()).view(B, H, T, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out)).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return _told(s, out, lse)


def _plain_prefix(s):
    c = s["case"]
    B, T, Hq, H, D, fan = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["fan"]
    n, G = s["prefix_len"].shape[0], Hq // H
    dev, scale = s["q"].device, 1 / math.sqrt(D)
    q = torch.zeros(n * fan, T, Hq, D, device=dev)
    q[:B] = s["q"].float()
    q = q.view(n * fan, T, H, G, D).transpose(2, 3)  # [branches][T][G][H][D]
    # the prefix, once for the rows of all its branches
    k, v = _take(s["pages"], s["prefix_table"], D)
    score = _scores(q.reshape(n, fan * T * G, H, D), k, scale)
    score = score.masked_fill((torch.arange(k.shape[1], device=dev) >= s["prefix_len"][:, None])[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e38)
    p = torch.exp(score - top)
    branch = lambda x: x.view(n, H, fan, T * G, -1).transpose(1, 2).reshape(n * fan, H, T * G, -1)[:B]  # noqa: E731
    top, total, out = branch(top), branch(p.sum(-1, keepdim=True)), branch(torch.matmul(p, v.transpose(1, 2).contiguous()))
    # each branch's own tokens
    k, v = _take(s["pages"], s["table"], D)
    at = torch.arange(k.shape[1], device=dev) - s["start"].long()[:, None]
    count = s["count"].long()[:, None] if s["count"] is not None else T
    see = (at < 0)[:, None, :] | (_new_seen(s, at) & (at < count)[:, None, :])
    score = _scores(q[:B].reshape(B, T * G, H, D), k, scale).view(B, H, T, G, -1)
    score = score.masked_fill(~see[:, None, :, None, :], -math.inf).view(B, H, T * G, -1)
    both = torch.maximum(top, score.amax(-1, keepdim=True))
    old, p = torch.exp(top - both), torch.exp(score - both)
    total = total * old + p.sum(-1, keepdim=True)
    out = (out * old + torch.matmul(p, v.transpose(1, 2).contiguous())) / total
    lse = (both + torch.log(total)).view(B, H, T, G).transpose(1, 2).reshape(B, T, Hq)
    return _told(s, out.view(B, H, T, G, D).transpose(1, 2).reshape(B, T, Hq, D), lse)


def _plain_reserve(table, held, need, free, free_count):
    """The sequences' pages brought to what `need` tokens take: what is too many goes back behind the
    free ones, the first page last; what is missing is taken from their end, the sequences in turn
    until one of them finds too few."""
    cols = torch.arange(table.shape[1], device=table.device)
    held, want, n = held.long()[:, None], ((need.long() + PAGE - 1) // PAGE)[:, None], free_count.long()
    give, take = (held - want).clamp_min(0), (want - held).clamp_min(0)
    upto = torch.cumsum(take, 0)
    full = n + give.sum()
    served = (take > 0) & (upto <= full)
    back = (cols >= want) & (cols < held)
    place = full - 1 - (torch.cumsum(give, 0) - give + cols - want)
    stack = torch.cat((free, free[:1]))
    stack = stack.scatter(0, torch.where(back, place, free.shape[0]).reshape(-1), table.reshape(-1))[:-1]
    fresh = served & (cols >= held) & (cols < want)
    place = full - 1 - (upto - take + cols - held)
    table = torch.where(back, -1, torch.where(fresh, stack[torch.where(fresh, place, 0)], table))
    left = full - (take * served).sum()
    return table, torch.where((give > 0) | served, want, held).squeeze(1).int(), stack, left.view(1).int()


def _plain_slots(s, table):
    """The slot in the pool of each new token [B][T], -1 where there is none."""
    i = torch.arange(s["case"]["T"], device=table.device)
    pos = s["start"].long()[:, None] + i
    page = table.long().gather(1, (pos // PAGE).clamp_max(table.shape[1] - 1))
    return torch.where((i < s["count"][:, None]) & (page >= 0), page * PAGE + pos % PAGE, -1)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import draft_token_verification_11_amd as sv

        if op == "rotate":
            sv.norm_rotate(s["q"], s["k"], s["start"], eps=1e-6, q_weight=s["weights"][0], k_weight=s["weights"][1], inv_freq=s["inv_freq"],
                           interleaved=bool(s["case"]["pairs"]), count=s["count"], depth=s["depth"], out=s["out"])
            return tuple(s["out"])
        if op == "window":
            return sv.attention_cache4(s["q"], s["pages"], s["table"], s["start"], count=s["count"], mask=s["mask"], depth=s["depth"], window=s["case"]["window"],
                                       sinks=s["case"]["sinks"], out=s["out"], lse=s["lse"])
        if op == "prefix":
            return sv.attention_cache4_shared(s["q"], s["pages"], s["table"], s["start"], s["prefix_table"], s["prefix_len"], fan=s["case"]["fan"], count=s["count"],
                                              mask=s["mask"], out=s["out"], lse=s["lse"])
        sv.cache4_reserve(s["table"], s["held"], s["need"], s["free"], s["free_count"])
        slots = sv.cache4_slots(s["table"], s["start"], s["case"]["T"], s["n_pages"], count=s["count"])
        sv.cache4_reserve(s["table"], s["held"], s["before"], s["free"], s["free_count"])
        return slots, s["table"], s["held"], s["free"], s["free_count"]
    if op == "rotate":
        return _plain_rotate(s)
    if op == "window":
        return _plain_window(s)
    if op == "prefix":
        return _plain_prefix(s)
    got = _plain_reserve(s["table"], s["held"], s["need"], s["free"], s["free_count"])
    slots = _plain_slots(s, got[0])
    s["table"], s["held"], s["free"], s["free_count"] = _plain_reserve(got[0], got[1], s["before"], got[2], got[3])
    return slots, s["table"], s["held"], s["free"], s["free_count"]


def work(case):
    B, T, starts = case["B"], case["T"], _spread(case["B"], case["lo"], case["hi"])
    if case["op"] == "reserve":
        # lengths and pages held, read and written by each call, a page's entry read and written where
        # it changes hands, there and back, and the slots
        pages = sum(-(-a // PAGE) for a in starts) * case["ends"] + (1 - case["ends"]) * B * T / 2 / PAGE
        return dict(bytes=2 * B * 12 + 2 * pages * 8 + B * 12 + B * T * 8, flops=0)
    counts, H, D, Hq = _counts(case), case["Hkv"], case["D"], case["Hq"]
    if case["op"] == "rotate":
        each = 2 if case["dtype"] == "bfloat16" else 4
        return dict(bytes=sum(counts) * (Hq + H) * D * 2 * each, flops=sum(counts) * (Hq + H) * (4 * D + 3 * case["rot"]))
    token = H * (D + D // 16)  # bytes of a cached token's keys and values
    depth = _depths(T, case["tree"])
    # new tokens that each new one sees: its path in a tree, all before it in a chain
    seen = lambda n: sum(d + 1 for d in depth[:n])  # noqa: E731
    pairs = cached = 0
    if case["op"] == "window":
        W, S = case["window"], case["sinks"]
        for a, n in zip(starts, counts):
            for d in depth[:n]:
                low = max(0, a + d - W + 1)  # the first cached token in the window
                pairs += max(0, a - low) + min(S, low, a)
            low = _first_seen(case, a)
            pairs, cached = pairs + seen(n), cached + a + n - low + min(S, low)
    else:
        fan, prefixes = case["fan"], _spread(-(-B // case["fan"]), case["plo"], case["phi"])
        for b, (a, n) in enumerate(zip(starts, counts)):
            pairs, cached = pairs + n * (a + prefixes[b // fan]) + seen(n), cached + a + n
        cached += sum(prefixes)
    rows = sum(counts) * Hq
    return dict(bytes=cached * token + rows * (4 * D + 4), flops=4 * D * pairs * Hq)


# --- the definitions in 64 bits -------------------------------------------------------------------


def _held(pages, table, n, D):
    """K and V [n][H][D] in float64 of a sequence's first n positions (zeros where it has no page)."""
    P, H, G, half = -(-n // PAGE), pages.shape[1], D // 32, 32 * D
    rec = pages[table[:P].clamp_min(0).long()]  # [P][H][68 D]
    kc = rec[..., :half].reshape(P, H, PAGE, D // 2)
    ks = rec[..., half : half + 2 * D].reshape(P, H, G, 16, 4).permute(0, 1, 4, 3, 2).reshape(P, H, PAGE, G)
    vc = rec[..., half + 2 * D : 66 * D].reshape(P, H, 16, 16, 4, G).permute(0, 1, 2, 4, 3, 5).reshape(P, H, PAGE, D // 2)
    vs = rec[..., 66 * D :].reshape(P, H, 16, G, 4).permute(0, 1, 2, 4, 3).reshape(P, H, PAGE, G)
    sixteen = torch.tensor([sign * v for sign in (1.0, -1.0) for v in E2M1], dtype=torch.float64, device=pages.device)
    got = []
    for code, e in ((kc, ks), (vc, vs)):
        x = sixteen[torch.stack([code % 16, code // 16], dim=-1).long()].reshape(P, H, PAGE, G, 32)
        x = x * ((e.long() + 896) << 52).view(torch.float64)[..., None] * (table[:P] >= 0).view(P, 1, 1, 1, 1)
        got.append(x.reshape(P, H, PAGE, D).transpose(1, 2).reshape(P * PAGE, H, D)[:n])
    return got


def _path(T, fan):
    """[T][T]: whether new token i sees new token j."""
    parents, sees = _parents(T, fan), torch.zeros(T, T, dtype=torch.bool)
    for i in range(T):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = parents[j]
    return sees.to("cuda")


def exact(case, seed):
    if case["op"] == "reserve":
        return None  # whole numbers
    s, dev, T, starts, counts = prepare(case, seed), "cuda", case["T"], _spread(case["B"], case["lo"], case["hi"]), _counts(case)
    depth = torch.tensor(_depths(T, case["tree"]), device=dev)
    if case["op"] == "rotate":
        got, rot = [], case["rot"]
        for x, w in zip((s["q"], s["k"]), s["weights"]):
            y = torch.zeros(x.shape, dtype=torch.float64, device=dev)
            for b, (a, n) in enumerate(zip(starts, counts)):
                z = x[b, :n].double()
                z = z / (z.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6).sqrt()
                if w is not None:
                    z = z * w.double()
                y[b, :n] = z
                if rot:
                    turn = torch.polar(torch.ones(1, 1, dtype=torch.float64, device=dev), (a + depth[:n, None]).double() * s["inv_freq"].double())[:, None]
                    part = z[..., :rot].unflatten(-1, (-1, 2) if case["pairs"] else (2, -1))
                    part = part if case["pairs"] else part.transpose(-1, -2)
                    part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
                    y[b, :n, :, :rot] = (part if case["pairs"] else part.transpose(-1, -2)).flatten(-2)
            got.append(y)
        return tuple(got)
    B, Hq, H, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.zeros(B, T, Hq, dtype=torch.float64, device=dev)
    path, kept = _path(T, case["tree"]), {}
    for b, (a, n) in enumerate(zip(starts, counts)):
        k, v = _held(s["pages"], s["table"][b], a + n, D)
        ban = torch.zeros(n, a + n, dtype=torch.bool, device=dev)
        ban[:, a:] = ~path[:n, :n]
        if case["op"] == "window":
            x = torch.arange(a + n, device=dev)
            far = (a + depth[:n, None] - x >= case["window"]) & (x >= case["sinks"])
            ban = ban | (far & (x < a)) if case["tree"] else ban | far
        else:
            if b // case["fan"] not in kept:
                g = b // case["fan"]
                kept = {g: _held(s["pages"], s["prefix_table"][g], int(s["prefix_len"][g]), D)}
            pk, pv = kept[b // case["fan"]]
            k, v = torch.cat((pk, k)), torch.cat((pv, v))
            ban = torch.cat((torch.zeros(n, pk.shape[0], dtype=torch.bool, device=dev), ban), 1)
        q = s["q"][b, :n].double().reshape(n, H, Hq // H, D)
        z = torch.einsum("nhgd,lhd->nhgl", q, k) / math.sqrt(D)
        z = z.masked_fill(ban[:, None, None, :], -math.inf)
        lse[b, :n] = torch.logsumexp(z, -1).reshape(n, Hq)
        out[b, :n] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(z, -1), v).reshape(n, Hq, D)
    return out, lse
