"""Builds libspecverify.so for gfx950 with hipcc, in the package directory."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspecverify.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = [os.path.join(CSRC, n) for n in ("sv_abi.hip", "sv_lowbit.hip", "sv_step.hip", "sv_shared.hip")]
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # keep hand-written and compiler-made packed fp32 arithmetic out of the code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _hipcc(args) -> str:
    """Runs hipcc; what it says, or an error."""
    res = subprocess.run([HIPCC] + args, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature"
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed (%d):\n%s" % (res.returncode, msgs))
    return msgs


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as work:
        objects = [os.path.join(work, os.path.basename(x) + ".o") for x in SOURCES]
        steps = [FLAGS + ["-I", INCLUDE, "-I", CSRC, "-c", "-o", o, x] for x, o in zip(SOURCES, objects)]
        with ThreadPoolExecutor(len(steps)) as pool:  # the sources side by side
            done = list(pool.map(_hipcc, steps))
        done.append(_hipcc(["--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objects))
    if verbose and any(m.strip() for m in done):
        print("\n".join(m for m in done if m.strip()))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
