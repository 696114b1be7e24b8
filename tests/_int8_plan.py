"""Which form of the product kernel sizes take: csrc/int8_plan.cuh, compiled for the host."""

import functools
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X = {"f32": 0, "bf16": 1, "i8": 3}


@functools.lru_cache(maxsize=None)
def _program():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no host C++ compiler")
    d = tempfile.mkdtemp()
    exe = os.path.join(d, "int8_plan")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-x", "c++",
                    "-I", os.path.join(ROOT, "mixture_experts_ffn_14_b200", "csrc"),
                    os.path.join(ROOT, "tests", "int8_plan_host_check.cpp"), "-o", exe], check=True)
    with open(exe, "rb") as f:
        code = f.read()
    shutil.rmtree(d)
    return code


def plans(sizes):
    """[(form, tile rows, CTAs per tile, workspace bytes)] of sizes (R, K, N, experts, x type, gated)."""
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "int8_plan")
        with open(exe, "wb") as f:
            f.write(_program())
        os.chmod(exe, 0o700)
        lines = "".join(f"{R} {K} {N} {n} {X[x]} {int(pair)}\n" for R, K, N, n, x, pair in sizes)
        out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.split("\n")
    got = [tuple(int(v) for v in line.split()) for line in out if line]
    assert len(got) == len(sizes)
    return [("split" if s else "stream" if rows < 256 else "pair", rows, s, ws) for rows, s, ws in got]


def form(R, K, N, n=1, x="bf16", pair=False):
    return plans([(R, K, N, n, x, pair)])[0][:3]


# Products that between them run every form: (form, tile rows, R, K, N, rows of each expert, gated).
CASES = [
    ("split", 64, 60, 1040, 2064, [20, 0, 40], False),
    ("split", 128, 333, 1040, 2064, [333], True),
    ("stream", 64, 200, 1040, 8208, [1, 64, 65, 0, 70], True),
    ("stream", 128, 290, 1040, 8208, [100, 128, 2, 60], False),
    ("pair", 256, 1600, 1040, 2064, [1, 512, 1087], True),
    # 512-row tiles: more of them than CTA pairs, so that the accumulators are taken up again; last
    # tiles with rows in their first half alone, which take one accumulator, not two; K blocks fewer
    # than the ring's four stages, as many, and more
    ("pair", 512, 3300, 1040, 8208, [1100, 700, 1500], False),
    ("pair", 512, 3300, 1040, 8208, [1100, 700, 1500], True),
    ("pair", 512, 3300, 512, 8208, [512, 1, 256, 257, 2274], True),
    ("pair", 512, 3300, 272, 16400, [512, 1, 256, 257, 2274], False),
    ("pair", 512, 3300, 640, 8208, [512, 0, 1024, 200, 1500], True),
    ("pair", 512, 2500, 112, 16400, [100, 2400], True),
]
