"""The norm's gradient at the lower end of its range: rows so small that r = 1 /
sqrt(mean(h^2) + eps) is finite and r^2 is not.

Tolerance, with u = 2^-24.  As for rows of ordinary size: a row's sum of squares
is off by (c + 24) u of itself, c = max(32, d / 1024 + 8) terms in a chain, r by
half of that and 4 u more (er), and mean(g h) by (c + 26 + 3) u of the mean of
magnitudes.  Here the squares are subnormal besides: each of the d fused additions
and the division by d are off by up to 2^-150 where their results are below 2^-126
(sums of such numbers are exact), 2 * 2^-150 / mean(h^2) of the mean in all, half
of that of r.  dx is rounded once to its type."""

import numpy as np
import pytest
import torch

from mixture_experts_moe_amd import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]
WIDTHS = [24, 1500, 4096, 40001]        # a wave, a workgroup, the widest in registers, read twice


def randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check(dx, dw, dy, h, w, eps):
    d = h.shape[1]
    c = max(32, d / 1024 + 8)
    h64, g = h.double(), dy.double() * w.double()
    m = h64.pow(2).mean(dim=1, keepdim=True)
    r = (m + float(np.float32(eps))).rsqrt()
    er = ((c + 24) / 2 + 4) * U + torch.where(m > 0, 2.0 ** -150 / m, torch.zeros_like(m))
    mean = (g * h64).mean(dim=1, keepdim=True)
    second = h64 * (r * r * mean)
    want = (g - second) * r
    size = (g.abs() + second.abs()) * r
    of_mean = (c + 29) * U * (h64.abs() * r * r * (g * h64).abs().mean(dim=1, keepdim=True)) * r
    tol = (3 * er + 8 * U) * size + of_mean
    tol = tol * 1.01 + torch.finfo(h.dtype).eps / 2 * (want.abs() + tol) + 1e-37
    assert dx.isfinite().all()
    assert ((dx.double() - want).abs() <= tol).all(), float(((dx.double() - want).abs() / tol).max())
    terms = (dy.double() * h64 * r).abs()
    tolw = ((64 + 3) * U * terms + er * terms).sum(dim=0) * 1.01 + 1e-37
    assert ((dw.double() - (dy.double() * h64 * r).sum(dim=0)).abs() <= tolw).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_small_rows_without_eps(d, dtype):
    print(f"norm backward, rows of 1e-20, {d} {dtype}", flush=True)
    scale = torch.tensor([[1e-20], [3e-20], [1e-19], [1e-18], [1.0]], device="cuda")
    h = randn(d, 5, d, dtype=dtype, scale=scale)
    dy, w = randn(d + 1, 5, d, dtype=dtype), randn(d + 2, d)
    dx, dw = B.moe_rmsnorm_backward(dy, h, w, 0.0)
    check(dx, dw, dy, h, w, 0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", WIDTHS)
def test_rows_of_zeros_with_a_tiny_eps(d, dtype):
    """dx = w dy / sqrt(eps), 1e20 times dy."""
    print(f"norm backward, zeros, {d} {dtype}", flush=True)
    h = torch.zeros((3, d), dtype=dtype, device="cuda")
    dy, w = randn(d + 3, 3, d, dtype=dtype), randn(d + 4, d)
    dx, dw = B.moe_rmsnorm_backward(dy, h, w, 1e-40)
    check(dx, dw, dy, h, w, 1e-40)
    assert not dw.any()
