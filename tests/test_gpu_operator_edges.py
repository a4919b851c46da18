"""Calls of the operators around the layer that their documentation allows and that
lie at its edges."""

import pytest
import torch

from mixture_experts_moe_amd import binding as B

pytestmark = pytest.mark.gpu


def randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("outputs", ["y", "both"])
def test_a_norm_over_its_input_returns_no_sum(outputs):
    """Without a residual sum is x; where y replaced x there is no such tensor."""
    x, w = randn(1, 6, 200, dtype=torch.bfloat16), randn(2, 200)
    want = B.moe_rmsnorm(x, w, outputs=outputs)
    assert want.sum is x
    z = x.clone()
    got = B.moe_rmsnorm(z, w, outputs=outputs, out=z[:, :])
    assert got.sum is None and torch.equal(z, want.y)
    other = torch.empty_like(x)
    assert B.moe_rmsnorm(x, w, outputs=outputs, out=other).sum is x
    # with a residual sum is a tensor of its own, or the one given
    res = randn(3, 6, 200, dtype=torch.bfloat16)
    h = (x.double() + res.double()).to(torch.bfloat16)
    z = x.clone()
    got = B.moe_rmsnorm(z, w, residual=res, outputs=outputs, out=z)
    assert torch.equal(got.sum, h) and torch.equal(got.y, B.moe_rmsnorm(h, w).y)


@pytest.mark.parametrize("K", [1, 64, 200])
def test_experts_of_one_weight_row(K):
    """w [E, 1, K], the first rows of wider experts: rows that lie an expert apart."""
    E, rows = 4, 5
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randint(-128, 128, (E, rows, K), generator=g, device="cuda").to(torch.int8)
    w = wide[:, :1]
    x = torch.randint(-128, 128, (40, K), generator=g, device="cuda").to(torch.int8)
    at = torch.tensor([0, 7, 7, 30, 40], dtype=torch.int32, device="cuda")
    one, ones = torch.ones(E, device="cuda"), torch.ones(40, device="cuda")
    out = B.moe_linear_i8(x, ones, w, one, offsets=at, out_dtype=torch.float32)
    for e in range(E):
        s = slice(int(at[e]), int(at[e + 1]))
        assert torch.equal(out[s].double(), x[s].double() @ w[e].double().t()), e
