"""The activations of moe_linear's epilogues, value by value, in their tails.

Every sum is exact (one product with 1, or zero sums and the bias), so what is
left is the function's own error and the one rounding of the result.

Tolerance, all relative to the exact value y: half a step of the result's type
(eps / 2), and twice the bound d on the function's error in fp32:

 silu        z / (1 + e^-z).  bf16: e^-u as exp2(-u log2 e): the constant
             (2^-25) and the product (2^-24) put 1.5 |u| 2^-24 on the
             exponential, exp2 and the reciprocal one unit (2^-23) each, the
             sum and the product half of one: d = |u| 2^-23 + 2^-21, u = z.
             fp32: expf and the division, d = 2^-21.
 gelu_tanh   z / (1 + e^-u), u = 2 sqrt(2/pi) (z + 0.044715 z^3): at most six
             roundings of 2^-24 in u besides, all terms of one sign:
             d = |u| 2^-21 + 2^-21.
 gelu        z Phi(z).  bf16: e^(-z^2/2) times a polynomial: two roundings in
             the exponent besides those of e^-u, 3.5 z^2/2 2^-24 in all; the
             fit 1.1e-6 and the polynomial's sums 2^-21: d = z^2 2^-23 + 2^-19.
             fp32: erfcf of an argument off by 1.5 2^-24 of itself, whose
             logarithm's slope there is at most z^2 + 2: d = z^2 2^-23 + 2^-20.

A factor y / z below the smallest normal number (2^-126; e^-u overflows just
beyond) and results below it may be flushed to zero: (|z| + 1) 2^-126 besides.
"""

import math

import pytest
import torch

from mixture_experts_moe_amd import binding as B
from test_gpu_linear import FMTS, FNS, act64

pytestmark = pytest.mark.gpu

# M, N, K: the epilogues of the streaming kernels (up to 4 and 16 tokens), of the
# small tiles, of the launch that adds the K ranges, and of the 256 x 256 tile
SIZES = [(4, 3584, 64), (12, 3584, 64), (40, 3584, 64), (40, 512, 4096), (1024, 3584, 512),
         (4096, 3584, 4096)]


def points(n, generator, whole_range):
    """n values of z: bf16 numbers, or fp32 ones just beside them; |z| from
    2^-6 to 13, smaller powers of two and values up to 60."""
    codes = torch.arange(0x3C80, 0x4150, device="cuda", dtype=torch.int32)     # 2^-6 .. 13
    z = (codes << 16).view(torch.float32)
    z = torch.cat([z, torch.exp2(-torch.arange(7, 41, device="cuda").float()),
                   torch.arange(13, 61, device="cuda").float()])
    z = torch.cat([z, -z])
    if whole_range:
        z = z * (1 + 2.0 ** -8 * (torch.rand(z.shape, generator=generator, device="cuda") - 0.5))
    pick = torch.randperm(z.numel(), generator=generator, device="cuda")
    return z[pick][torch.arange(n, device="cuda") % z.numel()].contiguous()


def exact(z, fn):
    """fn(z) in 64 bits without cancellation for large negative z."""
    z = z.double()
    if fn == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if fn == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return act64(z, fn)


def bound(z, fn, f32):
    z = z.double().abs()
    if fn == "silu":
        return (0 if f32 else z * 2.0 ** -23) + 2.0 ** -21
    if fn == "gelu_tanh":
        return 1.5957691216057308 * (z + 0.044715 * z ** 3) * 2.0 ** -21 + 2.0 ** -21
    if fn == "gelu":
        return z * z * 2.0 ** -23 + (2.0 ** -20 if f32 else 2.0 ** -19)
    return 0 * z


def operands(M, N, K, fmt, gated, z, carrier):
    """(x, w, bias, scale) whose gate sums are exactly z for every token, and
    whose up sums are 1."""
    R = 2 * N if gated else N
    act = torch.float32 if fmt == "f32" else torch.bfloat16
    v = torch.cat([z, torch.ones_like(z)]) if gated else z
    x = torch.zeros((M, K), dtype=act, device="cuda")
    w = torch.zeros((R, K), dtype=act, device="cuda")
    bias = scale = None
    at = K - 1 if M % 8 else 0          # the one k that is not zero
    x[:, at] = 1
    if fmt == "e4m3fn":
        w = torch.zeros((R, K), dtype=torch.uint8, device="cuda")
        scale = torch.ones(R, device="cuda")
    if carrier == "bias":
        bias = v
    elif fmt == "e4m3fn":
        w[:, at] = 0x38                 # 1.0
        scale = v
    else:
        w[:, at] = v.to(act)
        assert torch.equal(w[:, at].float(), v)
    return x, w, bias, scale


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("carrier", ["sum", "bias"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_tails(M, N, K, carrier, gated, fmt, fn):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    z = points(N, g, whole_range=carrier == "bias" or fmt != "bf16")
    x, w, bias, scale = operands(M, N, K, fmt, gated, z, carrier)
    out = B.moe_linear(x, w, bias=bias, scale=scale, activation=fn, gated=gated)
    y = exact(z, fn)
    tol = (torch.finfo(out.dtype).eps / 2 + 2 * bound(z, fn, fmt == "f32")) * y.abs()
    tol = tol + (z.double().abs() + 1) * 2.0 ** -126
    err = (out.double() - y).abs()
    bad = err > tol
    at = bad.any(dim=0).nonzero().flatten()[:4]
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()}; z {z[at].tolist()} gives "
                           f"{out[bad.any(dim=1).nonzero()[0, 0], at].tolist()} for {y[at].tolist()}")


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(3, 48, 64), (12, 48, 64), (40, 48, 64), (40, 48, 8192),
                                   (600, 1200, 64)])
def test_infinities_nan_and_the_largest_values(M, N, K, gated, fmt, fn):
    """A NaN sum gives NaN, +inf +inf, and -inf what the formula's arithmetic
    gives or its limit; the largest finite values the function's own; none
    touches the channels beside it."""
    inf, nan = float("inf"), float("nan")
    special = torch.tensor([nan, inf, -inf, 3e38, -3e38, 1e20, -1e20, 0.0, -0.0], device="cuda")
    n = special.numel()
    z = torch.ones(N, device="cuda")
    z[1:1 + 2 * n:2] = special
    x, w, bias, scale = operands(M, N, K, fmt, gated, z, "bias")
    if gated:
        bias[N + 40] = nan
    out = B.moe_linear(x, w, bias=bias, scale=scale, activation=fn, gated=gated).float()
    assert (out == out[:1]).logical_or(torch.isnan(out) & torch.isnan(out[:1])).all()
    got = out[0, 1:1 + 2 * n:2].tolist()
    assert math.isnan(got[0]) and got[1] == inf
    if fn is None:
        assert got[2] == -inf
    else:
        assert math.isnan(got[2]) or got[2] == 0
    big, low = 3e38, {None: -3e38}.get(fn, 0.0)
    assert got[3] == pytest.approx(big, rel=2.0 ** -8) and got[4] == pytest.approx(low, rel=2.0 ** -8)
    big, low = 1e20, {None: -1e20}.get(fn, 0.0)
    assert got[5] == pytest.approx(big, rel=2.0 ** -8) and got[6] == pytest.approx(low, rel=2.0 ** -8)
    assert got[7] == 0 and got[8] == 0
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[1:1 + 2 * n:2] = False
    if gated:
        assert torch.isnan(out[:, 40]).all()
        rest[40] = False
    one = exact(torch.ones(1), fn).item()
    assert ((out[:, rest] - one).abs() <= 2.0 ** -8 * one + 2.0 ** -19).all()
