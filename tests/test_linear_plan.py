"""moe_linear's choice of kernel, from the library's own rule on the CPU: the
GPU tests' sizes reach every kernel that it chooses, and what it chooses fits
a launch and the workspace that the library reports."""

import ctypes
import math
import os
import random

import pytest

from linear_plan_tool import linear_plans
from mixture_experts_moe_amd import binding as B
from test_gpu_linear import FMTS, LARGE, SHAPES
from test_gpu_linear_kernels import KERNELS


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def sizes(n, seed=1):
    """Sizes of 1..4096 tokens and 64..14336 rows and K, aligned and not."""
    rng = random.Random(seed)
    for _ in range(n):
        step = rng.choice((1, 8, 16, 64))
        N, K = (max(step, log_uniform(rng, 64, 14336) // step * step) for _ in range(2))
        yield (rng.choice(FMTS), log_uniform(rng, 1, 4096), N, K, rng.random() < 0.5,
               rng.choice((0, 0, 16, 5)), rng.choice((0, 0, 0, 3)))


def kernel(case, plan):
    """What makes another kernel of the tile's code."""
    stream = (plan.aligned,) if plan.tile.startswith("stream") else ()
    return (case[0], plan.tile, bool(case[4]), plan.splits > 1, *stream)


def test_the_value_tests_reach_every_kernel():
    tested = [(f, M, N, K, g, 0, 0) for f in FMTS for g in (False, True) for M, N, K in SHAPES]
    tested += [(f, M, N, K, g, 0, 0) for f, M, N, K, g in LARGE + KERNELS]
    reached = {kernel(c, p) for c, p in zip(tested, linear_plans(tested))}
    drawn = list(sizes(40000))
    missing = {}
    for c, p in zip(drawn, linear_plans(drawn)):
        if kernel(c, p) not in reached:
            missing.setdefault(kernel(c, p), (c, p))
    assert not missing, list(missing.values())[:5]


def test_copied_rows_are_tested_for_every_type():
    """x alone, and x and W."""
    tested = [(f, M, N, K, g, 0, 0) for f, M, N, K, g in LARGE + KERNELS]
    tested += [("bf16", M, N, K, False, 3, 0) for M, N, K in [(600, 2100, 520), (16, 96, 1024)]]
    got = {(c[0], p.pack_x, p.pack_w) for c, p in zip(tested, linear_plans(tested))}
    assert {(f, 1, 1) for f in FMTS} | {("bf16", 1, 0)} <= got


def test_plans_fit_a_launch():
    """At most 2^32 threads, K ranges that cover K in whole stages, and no
    range left empty, up to the documented limits."""
    rng = random.Random(2)
    cases = []
    while len(cases) < 20000:
        M, N, K = log_uniform(rng, 1, 1 << 28), log_uniform(rng, 1, 1 << 20), log_uniform(rng, 1, 1 << 20)
        if M * N <= 1 << 34:
            cases.append((rng.choice(FMTS), M, N, K, rng.random() < 0.5, rng.choice((0, 5)), 0))
    rows = {"stream4": 16, "stream16": 16, "stream16pair": 32, "256": 256, "128": 128, "128pair": 128,
            "128x64": 128, "128x64pair": 128, "64": 64, "staged128": 128, "staged64": 64}
    tokens = {"256": 256, "128": 128, "128pair": 128, "128x64": 64, "128x64pair": 64, "64": 64,
              "staged128": 128, "staged64": 64}
    for c, p in zip(cases, linear_plans(cases)):
        fmt, M, N, K, gated = c[:5]
        ch = rows[p.tile] // (2 if gated else 1)
        groups = -(-N // ch) * (-(-M // tokens[p.tile]) if M > 16 else 1)
        threads = 256 if rows[p.tile] == 64 else 512
        assert (groups + 7) * threads < 1 << 32, (c, p)
        assert p.splits >= 1 and p.splits * p.ksplit >= K > (p.splits - 1) * p.ksplit, (c, p)
        if p.splits > 1:
            assert p.ksplit % (32 if fmt == "f32" else 64) == 0, (c, p)
            assert M * -(-N // 4) + 256 < 1 << 32, (c, p)       # the launch that adds the ranges
        unit = {"f32": 4, "bf16": 8, "e4m3fn": 16}[fmt]
        if p.pack_x or p.pack_w:
            assert p.kpack % unit == 0 and K <= p.kpack < K + unit, (c, p)
            xu = p.kpack // (4 if fmt == "f32" else 8)
            units = M * xu * p.pack_x + (2 if gated else 1) * N * (p.kpack // unit) * p.pack_w
            assert units + 256 < 1 << 32, (c, p)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B._LIB_PATH):
        from mixture_experts_moe_amd import build
        build.build()
    return B.lib()


def test_the_library_reports_the_plans_workspace(lib):
    code = {"f32": (B.MOE_DTYPE_F32, B.MOE_DTYPE_F32, 0), "bf16": (B.MOE_DTYPE_BF16, B.MOE_DTYPE_BF16, 0),
            "e4m3fn": (B.MOE_DTYPE_BF16, B.MOE_DTYPE_E4M3FN, 2)}
    cases = list(sizes(500, seed=3)) + [("bf16", 48, 256, 8192, False, 0, 0)]
    plans = linear_plans(cases)
    for c, p in zip(cases, plans):
        fmt, M, N, K, gated, xp, wp = c
        act, w, mode = code[fmt]
        n = ctypes.c_size_t()
        d = B.moe_linear_desc(M, N, K, K + xp, K + wp, 0, 0, act, w, 0, int(gated), mode, 0)
        assert lib.moe_linear_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
        assert n.value == p.workspace, (c, p)


def test_a_split_products_workspace_is_checked(lib):
    """48 tokens against a long K: split, so that there is a workspace to check."""
    fake = 1 << 20
    d = B.moe_linear_desc(48, 256, 8192, 0, 0, 0, 0, B.MOE_DTYPE_BF16, B.MOE_DTYPE_BF16, 0, 0, 0, 0)
    n = ctypes.c_size_t()
    assert lib.moe_linear_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value >= 2 * 48 * 256 * 4

    def call(ws, nbytes):
        return lib.moe_linear(ctypes.byref(d), fake, fake, None, None, None, fake, ws, nbytes, None)
    assert call(None, 1 << 40) == -6
    assert call(fake, n.value - 1) == -6
    assert call(fake + 16, 1 << 40) == -5
