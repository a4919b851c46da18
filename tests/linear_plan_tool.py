"""moe_linear's choice of kernel for given sizes, from the library's own
``csrc/linear_plan.h`` compiled with the host compiler (no GPU, no HIP)."""

import os
import shutil
import subprocess
import tempfile
import textwrap
from collections import namedtuple

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_moe_amd", "csrc")

TILES = ("stream4", "stream16", "stream16pair", "256", "128", "128pair", "128x64", "128x64pair",
         "64", "staged128", "staged64")
Plan = namedtuple("Plan", "tile splits ksplit pack_x pack_w kpack aligned workspace")

SOURCE = textwrap.dedent(r"""
    #include <cstdio>
    #include <cstring>
    #include "linear_plan.h"
    int main() {
      char fmt[16];
      long long M, N, K, ldx, ldw;
      int gated;
      while (std::scanf("%15s %lld %lld %lld %d %lld %lld", fmt, &M, &N, &K, &gated, &ldx, &ldw) == 7) {
        moe::LinearArgs a{};
        a.M = M;
        a.N = (int)N;
        a.K = (int)K;
        a.gated = gated;
        a.R = gated ? 2 * a.N : a.N;
        a.ldx = ldx;
        a.ldw = ldw;
        a.ldr = a.ldo = N;
        a.act_dtype = std::strcmp(fmt, "f32") ? moe::kDtypeBF16 : moe::kDtypeF32;
        a.w_dtype = !std::strcmp(fmt, "f32") ? moe::kDtypeF32
                    : !std::strcmp(fmt, "bf16") ? moe::kDtypeBF16 : moe::kDtypeE4M3FN;
        moe::linear_plan(&a);
        const size_t ws = moe::linear_workspace(&a, nullptr);
        std::printf("%d %d %d %d %d %d %d %zu\n", a.tile, a.splits, a.ksplit, a.pack_x, a.pack_w,
                    a.kpack, a.aligned, ws);
      }
      return 0;
    }
""")


def linear_plans(cases):
    """The Plan of each (fmt, M, N, K, gated, xpad, wpad): columns by which a
    row of x and of w is longer than K in memory."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    with tempfile.TemporaryDirectory(prefix="moe_plan_") as d:
        src, exe = os.path.join(d, "plan.cpp"), os.path.join(d, "plan")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, src, "-o", exe],
                       check=True)
        text = "\n".join(f"{f} {M} {N} {K} {int(g)} {K + xp} {K + wp}" for f, M, N, K, g, xp, wp in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    rows = [list(map(int, l.split())) for l in out.splitlines()]
    assert len(rows) == len(cases)
    return [Plan(TILES[r[0]], *r[1:]) for r in rows]
