"""moe_linear's refusals: the C entry point on the host before any HIP call,
and the binding on tensor metadata.  No GPU."""

import ctypes
import os

import pytest
import torch

from mixture_experts_moe_amd import binding as B

F32, BF16, E4 = B.MOE_DTYPE_F32, B.MOE_DTYPE_BF16, B.MOE_DTYPE_E4M3FN
FAKE = 1 << 20            # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B._LIB_PATH):
        from mixture_experts_moe_amd import build
        build.build()
    return B.lib()


def desc(M=4, N=64, K=128, ldx=0, ldw=0, ldr=0, ldo=0, act=BF16, w=BF16, fn=0, gated=0, mode=0,
         reserved=0):
    return B.moe_linear_desc(M, N, K, ldx, ldw, ldr, ldo, act, w, fn, gated, mode, reserved)


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(M=0), 0), (dict(M=-1), -2), (dict(N=0), -2), (dict(K=0), -2),
    (dict(M=1, N=1, K=1), 0), (dict(N=(1 << 20) + 1), -2), (dict(K=(1 << 20) + 1), -2),
    (dict(M=(1 << 28) + 1, N=1), -2), (dict(M=1 << 20, N=(1 << 14) + 1), -2),
    (dict(M=1 << 20, N=1 << 14), 0),
    (dict(ldx=127), -2), (dict(ldx=128), 0), (dict(ldw=127), -2), (dict(ldr=63), -2),
    (dict(ldo=63), -2), (dict(ldo=(1 << 20) + 1), -2), (dict(ldx=-1), -2),
    (dict(act=F32), -4), (dict(act=F32, w=F32), 0), (dict(act=E4, w=E4), -4),
    (dict(act=F32, w=E4, mode=2), -4), (dict(w=E4), -4), (dict(w=E4, mode=1), 0),
    (dict(w=E4, mode=2), 0), (dict(w=E4, mode=3), -4), (dict(mode=1), -4),
    (dict(fn=5), -9), (dict(fn=-1), -9), (dict(gated=2), -9), (dict(reserved=1), -9),
])
def test_descriptor(lib, kw, status):
    n = ctypes.c_size_t()
    assert lib.moe_linear_workspace_bytes(ctypes.byref(desc(**kw)), ctypes.byref(n)) == status


def call(lib, d, x=FAKE, w=FAKE, scale=None, bias=None, res=None, out=FAKE, ws=FAKE, n=1 << 40):
    return lib.moe_linear(ctypes.byref(d), x, w, scale, bias, res, out, ws, n, None)


def test_pointers(lib):
    d = desc()
    assert lib.moe_linear(None, FAKE, FAKE, None, None, None, FAKE, None, 0, None) == -1
    assert lib.moe_linear_workspace_bytes(ctypes.byref(d), None) == -1
    assert call(lib, d, x=None) == -1
    assert call(lib, d, w=None) == -1
    assert call(lib, d, out=None) == -1
    assert call(lib, d, x=FAKE + 8) == -5
    assert call(lib, d, bias=FAKE + 4) == -5
    assert call(lib, d, res=FAKE + 2) == -5
    assert call(lib, d, scale=FAKE) == -4                # bf16 weights take no scale
    assert call(lib, desc(w=E4, mode=2)) == -1           # e4m3fn weights need one
    assert call(lib, desc(w=E4, mode=2), scale=FAKE + 4) == -5
    # no tokens: nothing is looked at
    assert call(lib, desc(M=0), x=None, w=None, out=None, ws=None, n=0) == 0


def test_workspace(lib):
    """A few tokens against a long K: split, with a workspace that is checked."""
    d = desc(M=48, N=256, K=8192)
    n = ctypes.c_size_t()
    assert lib.moe_linear_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
    if n.value:
        assert call(lib, d, ws=None) == -6
        assert call(lib, d, n=n.value - 1) == -6
        assert call(lib, d, ws=FAKE + 16) == -5


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("exc,match,kw", [
    (ValueError, r"x must be \[M, K\]", dict(x=meta(4, 2, 64))),
    (ValueError, "w must be", dict(w=meta(32, 63))),
    (ValueError, "activation must be", dict(activation="tanh")),
    (ValueError, "even number", dict(w=meta(33, 64), gated=True)),
    (TypeError, "activations must be", dict(x=meta(4, 64, dtype=torch.float16))),
    (TypeError, "weights must be", dict(w=meta(32, 64, dtype=torch.float16))),
    (ValueError, "need a scale", dict(w=meta(32, 64, dtype=torch.uint8))),
    (ValueError, "scale must be", dict(w=meta(32, 64, dtype=torch.uint8),
                                       scale=meta(31, dtype=torch.float32))),
    (ValueError, "only for e4m3fn", dict(scale=meta(32, dtype=torch.float32))),
    (ValueError, "bias must be", dict(bias=meta(32))),
    (ValueError, "bias must be", dict(bias=meta(16, dtype=torch.float32))),
    (TypeError, "residual must be", dict(residual=meta(4, 32, dtype=torch.float32))),
    (ValueError, "residual must be", dict(residual=meta(4, 31))),
    (TypeError, "out must be", dict(out=meta(4, 32, dtype=torch.float32))),
    (ValueError, "out must be", dict(out=meta(5, 32))),
    (ValueError, "dense rows", dict(x=meta(64, 4).t())),
    (ValueError, "on the GPU", dict()),
])
def test_binding_checks(lib, exc, match, kw):
    args = dict(x=meta(4, 64), w=meta(32, 64))
    args.update(kw)
    with pytest.raises(exc, match=match):
        B.moe_linear(args.pop("x"), args.pop("w"), **args)


def test_rows_that_overlap_are_refused():
    """A stride shorter than the row (an expanded row has 0) would be read as dense."""
    x, w = torch.zeros(1, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="overlap"):
        B.moe_linear(x.expand(20, 64), w)
    with pytest.raises(ValueError, match="overlap"):
        B.moe_linear(torch.zeros(20, 64), w[:1].expand(8, 64))
    with pytest.raises(ValueError, match="overlap"):
        B.moe_linear(torch.zeros(100).as_strided((4, 64), (8, 1)), w)
    with pytest.raises(ValueError, match="overlap"):
        B.moe_linear(torch.zeros(20, 64), w, residual=torch.zeros(1, 8).expand(20, 8))
    with pytest.raises(ValueError, match="overlap"):
        B.moe_linear(torch.zeros(20, 64), w, out=torch.zeros(1, 8).expand(20, 8))
