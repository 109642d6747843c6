"""Host-side checks of the serving step's calls (no GPU needed): the header and its symbols, sizes,
refusals before any HIP call, the binding's own checks, and the plain forms the GPU tests compare with."""
import ctypes
import os
import random
import re
import subprocess

import numpy as np
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests import lowbit_plain as low
from tests import step_plain as plain
from tests.test_lowbit_host import BAD_CACHES, BAD_HEADS, _cache, _heads

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "specverify_step.h")
HIPCC, CLANG = "/opt/rocm/bin/hipcc", "/opt/rocm/lib/llvm/bin/clang++"
OK, BAD, UNSUP, WS = sv.SPEC_OK, sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_UNSUPPORTED, sv.SPEC_ERR_WORKSPACE
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4098)


def test_header_and_symbols():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(spec_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(["spec_norm_rotate", "spec_attention_cache4_window", "spec_attention_cache4_window_workspace",
                            "spec_attention_cache4_shared_workspace", "spec_attention_cache4_shared", "spec_cache4_reserve", "spec_cache4_reserve_workspace",
                            "spec_cache4_slots"])
    out = subprocess.run(["nm", "-D", "--defined-only", sv.library_path()], capture_output=True, text=True,
                         check=True).stdout.split()
    assert all(n in out for n in names)


@pytest.mark.parametrize("lang", ["c", "c++"])
def test_header_compiles(tmp_path, lang):
    src = tmp_path / ("t.c" if lang == "c" else "t.cpp")
    src.write_text('#include "specverify_step.h"\nint main(void) { return (int)sizeof(spec_rotate_t) - 64; }\n')
    subprocess.run(["gcc" if lang == "c" else "g++", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), "-o",
                    str(tmp_path / "t"), str(src)], check=True)
    assert subprocess.run([str(tmp_path / "t")]).returncode == 0
    assert ctypes.sizeof(sv.spec_rotate_t) == 64


def _rotate(q=None, qo=None, Hq=4, k=None, ko=None, H=2, B=2, T=3, start=P, count=None, how=None, **kw):
    h = sv.spec_rotate_t(128, 128, 0, 1, 1e-6, 1, 4096, 4096, 4096, None, 0)
    for name, x in kw.items():
        setattr(h, name, x)
    d = dict(seq=4096, pos=1024, head=128)
    return sv.lib().spec_norm_rotate(q or _heads(**d), qo or _heads(**d), Hq, k or _heads(**d), ko or _heads(**d), H,
                                     None if how == 0 else ctypes.byref(h), B, T, start, count, None)


def test_rotate_refusals():
    for kw, want in BAD_HEADS:
        kw = dict(dict(seq=4096, pos=1024, head=128), **kw)
        assert _rotate(q=_heads(**kw)) == want and _rotate(ko=_heads(**kw)) == want, kw
    for kw in (dict(seq=0), dict(pos=64), dict(head=64)):  # written rows share no elements
        kw = dict(dict(seq=4096, pos=1024, head=128), **kw)
        assert _rotate(qo=_heads(**kw)) == BAD and _rotate(ko=_heads(**kw)) == BAD, kw
    none = _heads(ptr=0)
    assert _rotate(Hq=0, H=0) == BAD and _rotate(Hq=-1) == BAD and _rotate(H=-1) == BAD
    assert _rotate(Hq=16384, H=1) == UNSUP and _rotate(Hq=0, q=none, qo=none, H=2, B=0) == BAD
    assert _rotate(how=0) == BAD and _rotate(B=0) == BAD and _rotate(T=0) == BAD and _rotate(start=None) == BAD
    assert _rotate(start=ODD) == BAD and _rotate(count=ODD) == BAD and _rotate(B=65537) == UNSUP
    for d in (0, 8, 24, 272, -16):
        assert _rotate(head_dim=d, rotary_dim=0, inv_freq=None) == UNSUP, d
    assert _rotate(rotary_dim=144) == BAD and _rotate(rotary_dim=-16) == BAD and _rotate(rotary_dim=24) == UNSUP
    assert _rotate(inv_freq=None) == BAD and _rotate(rotary_dim=0) == BAD and _rotate(inv_freq=4098) == BAD
    assert _rotate(interleaved=2) == BAD and _rotate(norm=2) == BAD and _rotate(norm=-1) == BAD
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _rotate(eps=eps) == BAD
    assert _rotate(norm=0) == BAD  # weights without a norm
    assert _rotate(weight_dtype=2) == UNSUP and _rotate(q_weight=4104) == BAD and _rotate(k_weight=4104) == BAD
    assert _rotate(depth=4098) == BAD and _rotate(depth=4096, depth_stride=-1) == BAD
    d = dict(seq=4096, pos=1024, head=128)
    assert _rotate(q=_heads(dtype=0, **d)) == BAD and _rotate(qo=_heads(dtype=0, **d)) == BAD


def _window(c=None, q=None, B=2, T=3, Hq=4, start=P, count=None, mask=P, ms=0, mp=1, depth=None, ds=0, window=5, sinks=1,
            scale=0.1, out=None, lse=None, w=ctypes.c_void_p(1 << 20), wb=1 << 30):
    return sv.lib().spec_attention_cache4_window(c or _cache(), q or _heads(pos=512), B, T, Hq, start, count, mask, ms, mp,
                                                 depth, ds, window, sinks, scale, out or _heads(pos=512), lse, w, wb, None)


def _shared(c=None, table=P, stride=4, cols=4, length=P, fan=2, q=None, B=2, T=3, Hq=4, start=P, count=None, mask=None, ms=0,
            mp=1, scale=0.1, out=None, lse=None, w=ctypes.c_void_p(1 << 20), wb=1 << 40):
    return sv.lib().spec_attention_cache4_shared(c or _cache(), table, stride, cols, length, fan, q or _heads(pos=512), B, T,
                                                 Hq, start, count, mask, ms, mp, scale, out or _heads(pos=512), lse, w, wb,
                                                 None)


@pytest.mark.parametrize("call", [_window, _shared])
def test_attention_refusals(call):
    for kw, want in BAD_CACHES:
        assert call(c=_cache(**kw)) == want, kw
    for kw, want in BAD_HEADS:
        kw = dict(dict(pos=512), **kw)
        assert call(q=_heads(**kw)) == want and call(out=_heads(**kw)) == want, kw
    assert call(q=_heads(dtype=0, pos=512)) == UNSUP and call(out=_heads(dtype=0, pos=512)) == UNSUP
    for kw in (dict(seq=0), dict(pos=64), dict(head=64)):
        assert call(out=_heads(**dict(dict(pos=512), **kw))) == BAD
    assert call(Hq=3) == BAD and call(Hq=0) == BAD and call(T=257) == UNSUP and call(B=0) == BAD
    for s in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=s) == BAD, s
    assert call(mask=ODD) == BAD and call(mask=P, ms=-1) == BAD and call(mask=P, mp=-1) == BAD
    assert call(lse=ODD) == BAD and call(start=None) == BAD and call(count=ODD) == BAD
    assert call(w=None) == WS and call(wb=16) == WS and call(w=ctypes.c_void_p((1 << 20) + 16)) == WS


def test_window_refusals():
    assert _window(window=0) == BAD and _window(window=-5) == BAD and _window(sinks=-1) == BAD
    L = sv.lib()
    for T in (3, 100):
        need = L.spec_attention_cache4_window_workspace(2, T, 4, 2, 128)
        assert need > 0 and _window(T=T, wb=need - 1, q=_heads(seq=1 << 16, pos=512), out=_heads(seq=1 << 16, pos=512)) == WS
    for bad in [(0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 257, 8, 8, 128), (1, 1, 9, 8, 128), (1, 1, 8, 8, 80)]:
        assert L.spec_attention_cache4_window_workspace(*bad) == 0, bad
    assert _window(depth=ODD) == BAD and _window(depth=P, ds=-1) == BAD and _window(depth=P, mask=None) == BAD


def test_shared_refusals():
    assert _shared(fan=0) == BAD and _shared(fan=-3) == BAD
    assert _shared(table=None) == BAD and _shared(table=ODD) == BAD and _shared(stride=3) == BAD and _shared(cols=0) == BAD
    assert _shared(cols=(1 << 24) + 1, stride=1 << 25) == UNSUP
    assert _shared(length=None) == BAD and _shared(length=ODD) == BAD
    need = sv.lib().spec_attention_cache4_shared_workspace(2, 3, 4, 2, 128, 2)
    assert need > 2 * 3 * 4 * 128 * 4 and _shared(wb=need - 1) == WS
    # rows of a prefix past 2^30
    big = dict(B=65536, T=256, Hq=128, fan=65536, c=_cache(heads=128), q=_heads(seq=1 << 22, pos=1 << 14),
               out=_heads(seq=1 << 22, pos=1 << 14))
    assert _shared(wb=1 << 60, **big) == UNSUP
    L = sv.lib()
    for bad in [(0, 1, 8, 8, 128, 1), (1, 0, 8, 8, 128, 1), (1, 257, 8, 8, 128, 1), (1, 1, 9, 8, 128, 1), (1, 1, 8, 8, 80, 1),
                (1, 1, 8, 8, 128, 0), (1, 1, 8, 8, 128, -1), (65536, 256, 128, 128, 128, 65536)]:
        assert L.spec_attention_cache4_shared_workspace(*bad) == 0, bad
    for fan in (1, 7, 2147483647):
        assert L.spec_attention_cache4_shared_workspace(3, 2, 8, 2, 64, fan) > 0


def test_pages_refusals():
    L = sv.lib()

    def reserve(table=P, stride=4, cols=4, held=P, need=P, B=2, free=P, cap=8, count=P, w=P, wb=1 << 20):
        return L.spec_cache4_reserve(table, stride, cols, held, need, B, free, cap, count, w, wb, None)

    for name in ("table", "held", "need", "free", "count"):
        assert reserve(**{name: None}) == BAD and reserve(**{name: ODD}) == BAD
    assert reserve(stride=3) == BAD and reserve(cols=0) == BAD and reserve(B=0) == BAD and reserve(cap=0) == BAD
    for B in (129, 5000, 65536):
        need = L.spec_cache4_reserve_workspace(B)
        assert need > 8 * B and reserve(B=B, wb=need - 1) == WS
        assert reserve(B=B, w=None) == WS and reserve(B=B, w=ctypes.c_void_p(4096 + 16)) == WS
    assert [L.spec_cache4_reserve_workspace(B) for B in (1, 128, 0, -1, 65537)] == [0] * 5
    assert reserve(B=65537) == UNSUP and reserve(cols=(1 << 24) + 1, stride=1 << 25) == UNSUP

    def slots(table=P, stride=4, cols=4, n=8, B=2, T=3, start=P, count=None, out=P):
        return L.spec_cache4_slots(table, stride, cols, n, B, T, start, count, out, None)

    for name in ("table", "start", "out"):
        assert slots(**{name: None}) == BAD and slots(**{name: ODD}) == BAD
    assert slots(count=ODD) == BAD and slots(out=ctypes.c_void_p(4100)) == BAD and slots(n=0) == BAD
    assert slots(stride=3) == BAD and slots(cols=0) == BAD and slots(B=0) == BAD and slots(T=0) == BAD
    assert slots(B=65537) == UNSUP and slots(T=(1 << 24) + 1) == UNSUP and slots(B=65536, T=1 << 24) == UNSUP


def test_binding_refusals():
    """Tensors of the wrong kind or place raise before any launch."""
    q, s = torch.zeros(2, 3, 4, 64), torch.zeros(2, dtype=torch.int32)
    for bad in (None, q.long(), q[0]):
        with pytest.raises((TypeError, ValueError)):
            sv.norm_rotate(bad, bad, s)
    with pytest.raises(ValueError, match="device memory"):
        sv.norm_rotate(q, None, s)
    with pytest.raises(ValueError, match="device memory"):
        sv.cache4_reserve(torch.zeros(2, 3, dtype=torch.int32), s, s, s, s[:1])
    with pytest.raises(TypeError):
        sv.cache4_slots(torch.zeros(2, 3), s, 3, 8)
    b = q.bfloat16()
    pages, table = torch.zeros(4, 2, 68 * 64, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        sv.attention_cache4(b, pages, table, s, window=4)
    with pytest.raises(ValueError, match="device memory"):
        sv.attention_cache4_shared(b, pages, table, s, table[:1], s[:1], fan=2)


def test_tree_depths():
    assert sv.tree_depths([-1, 0, 0, 1, 3]).tolist() == [[0, 1, 1, 2, 3]]
    assert sv.tree_depths(torch.tensor([-1])).tolist() == [[0]]
    for bad in ([], [0], [-1, 1], [-1, -1], [-1, 0, 5]):
        with pytest.raises(ValueError):
            sv.tree_depths(bad)


def test_plain_positions_against_bytes():
    """step_plain.held against lowbit_plain.fetch, one position at a time."""
    rs = np.random.default_rng(0)
    pages = np.zeros((3, 2, 68 * 64), np.uint8)
    row = np.array([2, 0, 7])
    for pos in range(128):
        for h in range(2):
            x = rs.normal(0, 1, 64)
            low.store(pages, row[None], 0, h, pos, x * (np.nan if pos == 5 else 1), rs.normal(0, 1, 64))
    k, v, good = plain.held(pages, row, 140, 64)
    assert not good and np.isnan(k[128:]).all()
    for pos in range(128):
        for h in range(2):
            want = low.fetch(pages, row[None], 0, h, pos, 64)
            assert np.array_equal(k[pos, h], want[0], equal_nan=True) and np.isnan(k[pos, h, 0]) == (pos == 5)
            assert pos == 5 or np.array_equal(v[pos, h], want[1])


def test_plain_rotation():
    """A turn keeps a pair's length, and turns add up."""
    rs = np.random.default_rng(1)
    x, f = rs.normal(0, 1, (3, 64)), np.float32(10000.0) ** (-np.arange(16, dtype=np.float32) / 16)
    for pairs in (False, True):
        y, _ = plain.rotate(x, None, None, f, 5, pairs)
        z, _ = plain.rotate(y, None, None, f, 7, pairs)
        assert np.allclose(z, plain.rotate(x, None, None, f, 12, pairs)[0])
        assert np.array_equal(y[:, 32:], x[:, 32:]) and np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(plain.rotate(x[:, :2] * [1, 0], None, None, np.array([np.pi / 2]), 1, False)[0][:, 1], x[:, 0])


def test_plain_reserve_keeps_every_page():
    r = random.Random(1)
    for _ in range(50):
        B, cols, n = r.randint(1, 6), r.randint(1, 5), r.randint(1, 20)
        rows, held, free, count = [[-1] * cols for _ in range(B)], [0] * B, list(range(n)), n
        for _ in range(6):
            old = [list(x) for x in rows], list(held), list(free[:count])
            count = plain.reserve(rows, held, [r.randint(0, 64 * cols) for _ in range(B)], free, count)
            taken = [x for b in range(B) for x in rows[b][:held[b]]]
            assert sorted(taken + free[:count]) == list(range(n))
            assert all(x == -1 for b in range(B) for x in rows[b][held[b]:])
            back = plain.reserve(rows, held, [64 * x for x in old[1]], free, count)
            assert (rows, held, free[:back]) == old
            count = back


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="no ROCm toolchain")
def test_host_code_under_asan_ubsan(tmp_path):
    """Every refusal at the ends of the arguments' ranges, under sanitizers on the host side."""
    csrc, inc = os.path.join(ROOT, "draft_token_verification_11_amd", "csrc"), os.path.join(ROOT, "include")
    exe, objs = str(tmp_path / "step_san"), []
    for name in ("sv_step.hip", "sv_shared.hip"):
        objs.append(str(tmp_path / (name + ".o")))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-c", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang",
                        "-target-feature", "-Xclang", "-packed-fp32-ops", "-Xarch_host", "-fsanitize=address",
                        "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", "-I", inc, "-I",
                        csrc, "-o", objs[-1], os.path.join(csrc, name)], check=True, capture_output=True)
    objs.append(str(tmp_path / "drv.o"))
    subprocess.run([CLANG, "-c", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", inc, "-o", objs[-1], os.path.join(ROOT, "tests", "sanitize_step.cpp")], check=True)
    subprocess.run([CLANG, "-fsanitize=address,undefined", "-o", exe] + objs +
                   ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0 and "runtime error" not in report and "AddressSanitizer" not in report, report
    assert "sanitized step validation ok" in report
