"""Buffers of moe_linear and moe_decode that lie between or beside each other
without sharing an element are accepted; the refused ones leave them alone."""

import pytest
import torch

from mixture_experts_moe_amd import binding as B
from mixture_experts_moe_amd import synth

pytestmark = pytest.mark.gpu


def rand(*shape, seed=1, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("M", [1, 3, 16, 40, 300])
def test_column_slices_of_one_matrix(M):
    """x, the residual and out as neighbouring columns of the same rows."""
    K, N = 128, 72
    w, buf = rand(N, K, seed=2), rand(M, K + 2 * N)
    x, r, out = buf[:, :K], buf[:, K:K + N], buf[:, K + N:]
    want = B.moe_linear(x.clone(), w, activation="silu", residual=r.clone())
    before = buf.clone()
    B.moe_linear(x, w, activation="silu", residual=r, out=out)
    assert torch.equal(out, want) and torch.equal(buf[:, :K + N], before[:, :K + N])
    assert B.moe_linear(x, w, activation="silu", residual=r, out=r) is r
    assert torch.equal(r, want) and torch.equal(x, before[:, :K])


@pytest.mark.parametrize("M", [2, 40])
def test_rows_of_different_strides_between_each_other(M):
    K, N = 64, 32
    w, buf = rand(N, K, seed=2), rand(2 * M, K + N)
    x, out = buf[:M, :K], buf[::2, K:]          # out's rows behind every other row of x
    want = B.moe_linear(x.clone(), w)
    assert torch.equal(B.moe_linear(x, w, out=out), want)


@pytest.mark.parametrize("M", [3, 40])
def test_linear_refuses_an_out_that_is_x(M):
    x, w = rand(M, 64), rand(64, 64, seed=2)
    before = x.clone()
    for kw in (dict(out=x), dict(out=x, residual=x)):
        with pytest.raises(B.MoEError) as e:
            B.moe_linear(x, w, **kw)
        assert e.value.status == B.MOE_ERR_OVERLAP
    torch.cuda.synchronize()
    assert torch.equal(x, before)
    assert torch.isfinite(B.moe_linear(x, w, residual=x).float()).all()


@pytest.mark.parametrize("schedule", ["auto", "static", "queue"])
@pytest.mark.parametrize("T", [1, 9])
def test_decode(T, schedule):
    cfg = dict(T=T, d=256, E=8, k=2, I=192, act="bf16", w="bf16", x_std=1.0, w_std=0.05, skew=False)
    inp = synth.make_inputs(cfg, device="cuda", seed=3)
    buf = rand(3 * T, 256)
    x, r, out = buf[:T], buf[T:2 * T], buf[2 * T:]
    x.copy_(inp.x)
    args = (inp.w_gate, inp.w13, inp.w2, 2)
    want = B.moe_decode(inp.x, *args, residual=r.clone())
    B.moe_decode(x, *args, residual=r, out=out, schedule=schedule)
    assert torch.equal(out, want) and torch.equal(x, inp.x)
    for kw in (dict(out=x), dict(out=x, residual=x), dict(out=buf[T - 1:2 * T - 1], residual=r)):
        with pytest.raises(B.MoEError) as e:
            B.moe_decode(x, *args, schedule=schedule, **kw)
        assert e.value.status == B.MOE_ERR_OVERLAP
    torch.cuda.synchronize()
    assert torch.equal(x, inp.x) and torch.equal(out, want)
