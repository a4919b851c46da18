"""moe_decode's refusals, on the host before any HIP call.  No GPU."""

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


def desc(T=4, d=128, E=8, I=128, act=BF16, w=BF16, bm=0, q=None, schedule="auto"):
    return B.make_desc(T, d, E, I, act, w, bm, q, schedule)


@pytest.mark.parametrize("kw,k,status", [
    (dict(), 2, 0), (dict(T=0), 2, 0), (dict(T=16), 2, 0), (dict(T=17), 2, -2), (dict(T=-1), 2, -2),
    (dict(d=100), 2, -2), (dict(I=96), 2, -2), (dict(E=1025), 2, -2), (dict(E=1024), 64, 0),
    (dict(), 9, -3), (dict(), 0, -3), (dict(act=F32), 2, -4), (dict(act=F32, w=F32), 2, 0),
    (dict(w=E4), 2, 0), (dict(bm=16), 2, -8), (dict(d=256, I=256, w=E4, q="mx_e4m3"), 2, -9),
    (dict(schedule="static"), 2, 0), (dict(schedule="queue"), 2, 0),
])
def test_descriptor(lib, kw, k, status):
    n = ctypes.c_size_t()
    assert lib.moe_decode_workspace_bytes(ctypes.byref(desc(**kw)), k, ctypes.byref(n)) == status
    if status == 0:
        assert (n.value > 0) == (kw.get("T", 4) > 0)


def call(lib, d, k=2, x=FAKE, wg=FAKE, w13=FAKE, w2=FAKE, scales=None, res=None, out=FAKE, ws=FAKE,
         n=1 << 40):
    return lib.moe_decode(ctypes.byref(d), x, wg, w13, w2, k,
                          ctypes.byref(scales) if scales is not None else None, res, out, ws, n,
                          None)


def test_pointers(lib):
    d = desc()
    assert lib.moe_decode_workspace_bytes(ctypes.byref(d), 2, None) == -1
    assert lib.moe_decode_workspace_bytes(None, 2, None) == -1
    for name in ("x", "wg", "w13", "w2", "out"):
        assert call(lib, d, **{name: None}) == -1
        assert call(lib, d, **{name: FAKE + 8}) == -5
    assert call(lib, d, res=FAKE + 4) == -5
    assert call(lib, d, ws=None) == -6
    assert call(lib, d, n=16) == -6
    assert call(lib, d, ws=FAKE + 16) == -5
    assert call(lib, desc(w=E4)) == -1                    # e4m3fn weights need scales
    assert call(lib, desc(T=17)) == -2
    assert call(lib, desc(T=0), x=None, wg=None, w13=None, w2=None, out=None, ws=None, n=0) == 0


def test_binding_checks(lib):
    x = torch.empty(4, 128, dtype=torch.bfloat16, device="meta")
    wg = torch.empty(4, 128, device="meta")
    w13 = torch.empty(4, 256, 128, dtype=torch.bfloat16, device="meta")
    w2 = torch.empty(4, 128, 128, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="out must match x"):
        B.moe_decode(x, wg, w13, w2, 2, out=x[:3])
    with pytest.raises(ValueError, match="residual must match x"):
        B.moe_decode(x, wg, w13, w2, 2, residual=x.float())
    with pytest.raises(ValueError, match="residual must match x"):
        B.moe_decode(x, wg, w13, w2, 2, residual=x[:3])
    with pytest.raises(ValueError, match="on the GPU"):
        B.moe_decode(x, wg, w13, w2, 2)
