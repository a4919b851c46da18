"""moe_linear and moe_decode refuse an out that overlaps an input, and a
workspace that overlaps a buffer, before any HIP call: workgroups store out
while others still read the inputs.  No GPU."""

import ctypes
import os
import random
import shutil
import subprocess
import textwrap

import pytest

from mixture_experts_moe_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_moe_amd", "csrc")
F32, BF16, E4 = B.MOE_DTYPE_F32, B.MOE_DTYPE_BF16, B.MOE_DTYPE_E4M3FN
OVERLAP = -11


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B._LIB_PATH):
        from mixture_experts_moe_amd import build
        build.build()
    return B.lib()


def at(i):
    """The i-th of addresses far apart, never dereferenced."""
    return (i + 1) << 44


def linear(lib, d, **kw):
    p = dict(x=at(0), w=at(1), scale=None, bias=at(3), res=at(4), out=at(5), ws=at(6))
    p.update(kw)
    return lib.moe_linear(ctypes.byref(d), p["x"], p["w"], p["scale"], p["bias"], p["res"],
                          p["out"], p["ws"], 1 << 40, None)


def desc(M=40, N=64, K=64, ldx=0, ldw=0, ldr=0, ldo=0, act=BF16, w=BF16, gated=0, mode=0):
    return B.moe_linear_desc(M, N, K, ldx, ldw, ldr, ldo, act, w, 0, gated, mode, 0)


ROW = 64 * 2  # bytes of a row of 64 bf16


@pytest.mark.parametrize("kw,ptrs", [
    # x += f(x): the residual is out, and out is x
    (dict(), dict(x=at(5), res=at(5))),
    (dict(), dict(x=at(5), res=None)),
    # out begins in x's last row, x in out's last row
    (dict(), dict(out=at(0) + 39 * ROW)),
    (dict(), dict(out=at(0) - 39 * ROW)),
    # the weight: its last row (of 64; gated: of 128), its padded row
    (dict(), dict(out=at(1) + 63 * ROW)),
    (dict(gated=1), dict(out=at(1) + 127 * ROW)),
    (dict(ldw=4096), dict(out=at(1) + 63 * 8192 + 64)),
    (dict(w=E4, mode=2), dict(out=at(1) + 63 * 64, scale=at(2))),
    # scales (one per row of W, or one), biases
    (dict(w=E4, mode=2), dict(scale=at(5) + 40 * ROW - 16)),
    (dict(w=E4, mode=2), dict(out=at(2) + 63 * 4 - 12, scale=at(2))),
    (dict(w=E4, mode=1), dict(out=at(2), scale=at(2))),
    (dict(gated=1), dict(out=at(3) + 127 * 4 - 12)),
    # the residual, but not the same rows
    (dict(), dict(out=at(4) + ROW)),
    (dict(), dict(out=at(4) - ROW)),
    (dict(ldr=72), dict(res=at(5))),
    (dict(ldo=72), dict(res=at(5))),
    (dict(ldr=128, ldo=128), dict(res=at(5) + 112)),
    # column slices of a wider matrix that share columns
    (dict(ldx=128, ldo=128), dict(x=at(5) + 112)),
    (dict(ldx=128, ldo=128), dict(x=at(5) + 256 - 112)),
    # rows of other lengths between each other
    (dict(ldx=128, ldo=256), dict(x=at(5) + 128 + 16)),
    # a workspace in a buffer (K is split)
    (dict(M=48, N=256, K=8192), dict(ws=at(5) + 512)),
    (dict(M=48, N=256, K=8192), dict(ws=at(0) + 48 * 8192 * 2 - 256)),
    (dict(M=48, N=256, K=8192), dict(ws=at(1))),
    (dict(M=48, N=256, K=8192), dict(ws=at(3))),
    (dict(M=48, N=256, K=8192), dict(out=at(6) + 256)),
])
def test_linear(lib, kw, ptrs):
    assert linear(lib, desc(**kw), **ptrs) == OVERLAP


SZ = dict(T=4, d=128, E=8, I=192)


def decode(lib, w=BF16, mode=0, schedule="auto", **kw):
    p = dict(x=at(0), wg=at(1), w13=at(2), w2=at(3), s13=at(4), s2=at(5), res=at(6), out=at(7),
             ws=at(8))
    p.update(kw)
    d = B.make_desc(SZ["T"], SZ["d"], SZ["E"], SZ["I"], BF16, w, 0, None, schedule)
    sc = B.moe_scales(mode, 0, p["s13"], p["s2"]) if w == E4 else None
    return lib.moe_decode(ctypes.byref(d), p["x"], p["wg"], p["w13"], p["w2"], 2,
                          ctypes.byref(sc) if sc is not None else None, p["res"], p["out"],
                          p["ws"], 1 << 40, None)


@pytest.mark.parametrize("schedule", ["auto", "static", "queue"])
@pytest.mark.parametrize("kw", [
    dict(x=at(7), res=at(7)), dict(x=at(7), res=None),
    dict(out=at(0) + 3 * 256), dict(out=at(0) - 3 * 256),
    dict(out=at(1) + 8 * 128 * 4 - 16), dict(out=at(2) + 8 * 384 * 128 * 2 - 16),
    dict(out=at(3) + 8 * 128 * 192 * 2 - 16), dict(out=at(6) + 256), dict(out=at(6) - 256),
    dict(w=E4, mode=2, out=at(2) + 8 * 384 * 128 - 16),
    dict(w=E4, mode=2, out=at(4) + 8 * 384 * 4 - 16), dict(w=E4, mode=2, out=at(5) + 8 * 128 * 4 - 16),
    dict(w=E4, mode=1, out=at(4) + 16), dict(w=E4, mode=1, out=at(5) + 16),
    dict(ws=at(7)), dict(ws=at(0)), dict(ws=at(2) + 256), dict(ws=at(6)), dict(out=at(8) + 1024),
])
def test_decode(lib, kw, schedule):
    assert decode(lib, schedule=schedule, **kw) == OVERLAP


def test_status_text():
    assert "overlap" in B.strerror(OVERLAP)
    assert B.MOE_ERR_OVERLAP == OVERLAP


SOURCE = textwrap.dedent(r"""
    #include <cstdio>
    #include "overlap.h"
    int main() {
      long long a[4], b[4];
      while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld", a, a + 1, a + 2, a + 3, b, b + 1,
                        b + 2, b + 3) == 8)
        std::printf("%d\n", moe::rows_overlap(moe::Rows{(uintptr_t)a[0], a[1], a[2], a[3]},
                                              moe::Rows{(uintptr_t)b[0], b[1], b[2], b[3]}));
      return 0;
    }
""")


def test_rows_overlap_against_sets_of_bytes(tmp_path):
    """Two matrices of any starts, rows, lengths and steps: exactly when some
    byte is in both."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "overlap.cpp"
    src.write_text(SOURCE)
    exe = tmp_path / "overlap"
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    rng = random.Random(7)

    def matrix():
        rows, n = rng.choice((0, 1, 1, 2, 3, 7, 12)), rng.randint(0 if rng.random() < 0.1 else 1, 6)
        step = max(n, 1) + rng.choice((0, 1, 3, 8, 20))
        if rows == 1 and rng.random() < 0.3:
            step = rng.randint(1, 4)        # one row may have any step
        return 1000 + rng.randint(0, 60), rows, n, step

    def held(m):
        return {m[0] + i * m[3] + c for i in range(m[1]) for c in range(m[2])}

    cases = []
    for _ in range(20000):
        a, b = matrix(), matrix()
        if rng.random() < 0.4:
            b = (b[0], b[1], min(b[2], a[3]), a[3])     # the same step
        cases.append((a, b))
    # far apart in steps, many rows
    for at_, step in ((5, 64), (40, 64), (5, 96), (48, 160)):
        cases.append(((1000, 300, 32, 64), (1000 + at_, 40, 8, step)))
    text = "\n".join(" ".join(map(str, a + b)) for a, b in cases)
    got = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    want = [bool(held(a) & held(b)) for a, b in cases]
    got = [l == "1" for l in got.split()]
    assert len(got) == len(want) and 0.2 < sum(want) / len(want) < 0.8
    wrong = [c for c, g, w in zip(cases, got, want) if g != w]
    assert not wrong, wrong[:3]


def test_the_texts_of_refused_shapes_name_these_calls(lib):
    """17 tokens and no output features are refused with a text that says why."""
    d = B.make_desc(17, 128, 8, 128, BF16, BF16)
    n = ctypes.c_size_t()
    assert lib.moe_decode_workspace_bytes(ctypes.byref(d), 2, ctypes.byref(n)) == -2
    assert lib.moe_linear_workspace_bytes(ctypes.byref(desc(N=0)), ctypes.byref(n)) == -2
    assert "moe_decode: T <= 16" in B.strerror(-2) and "moe_linear: 0 <= M" in B.strerror(-2)
    assert "moe_linear_workspace_bytes" in B.strerror(-6)
