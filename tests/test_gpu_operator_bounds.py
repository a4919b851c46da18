"""The operators around the layer run together, held to bounds that are derived element
by element (operator_bounds.py; test_operator_bounds.py shows on the CPU that results
with a mistake leave them)."""

import pytest
import torch

import operator_bounds as ob
from mixture_experts_moe_amd import binding as B

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,E,k", [(60, 130, 5, 3), (33, 1030, 4, 2), (5, 64, 8, 8), (1, 4096, 8, 2),
                                     (1500, 520, 16, 8), (40, 8200, 6, 2)])
def test_gradients_of_a_block(T, d, E, k, dtype):
    """norm -> permute -> an expert that scales each row -> unpermute into the stream, and back."""
    print(f"block {T}x{d} experts {E} top {k} {dtype}", flush=True)
    g = gen(T + d)
    x, res, dout = (randn(g, T, d, dtype=dtype) for _ in range(3))
    w, c = rand(g, d) + 0.5, rand(g, E) + 0.5
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    gates = torch.softmax(randn(g, T, k), 1)

    n = B.moe_rmsnorm(x, w, EPS, residual=res)
    h = x.double() + res.double()
    assert ((n.sum.double() - h).abs() <= (ob.half(dtype) + ob.U) * h.abs()).all()
    p = B.moe_permute(n.y, ids, E)
    scale = c[ids.flatten()[p.row_slot.long()].long()][:, None]
    rows = (p.rows.float() * scale).to(dtype)
    out = B.moe_unpermute(rows, p.slot_row, weights=gates, residual=n.sum)
    drows, dgates = B.moe_unpermute_backward(dout, rows, p.slot_row, gates)
    dy = B.moe_unpermute((drows.float() * scale).to(dtype), p.slot_row)
    dx, dw = B.moe_rmsnorm_backward(dy, n.sum, w, EPS, dsum=dout)

    got = {"out": out, "dgates": dgates, "dx": dx, "dweight": dw}
    want = ob.block(n.sum, w, c, ids, gates, dout, EPS, dtype)
    assert {name: ob.outside(got[name], want[name]) for name in want} == dict.fromkeys(want, 0.0)


@pytest.mark.parametrize("T", [5, 300])
def test_the_layer_from_its_parts(T):
    """route, permute, each expert's products, unpermute, and what moe_forward computes in one
    call, both against 64 bits."""
    d, I, E, k = 256, 128, 8, 2
    g = gen(T)
    x = randn(g, T, d)
    gate, w13, w2 = randn(g, E, d) * 0.1, randn(g, E, 2 * I, d) * 0.05, randn(g, E, d, I) * 0.05
    _, ids, gates = B.moe_route(x, gate, k)
    p = B.moe_permute(x, ids, E)
    at = p.offsets.tolist()
    y = torch.empty_like(p.rows)
    for e in range(E):
        if at[e] < at[e + 1]:
            r = slice(at[e], at[e + 1])
            h = B.moe_linear(p.rows[r], w13[e], activation="silu", gated=True)
            B.moe_linear(h, w2[e], out=y[r])
    want = ob.layer(x, ids, gates, w13, w2)
    assert ob.outside(B.moe_unpermute(y, p.slot_row, weights=gates), want) == 0
    assert ob.outside(B.moe_forward(x, gate, w13, w2, k), want) == 0


@pytest.mark.parametrize("T,d", [(3, 50), (4, 1500), (2, 5000)])
def test_backward_against_differences(T, d):
    """The slope between the norm's own results on both sides of x, and of the weight.  dy leans
    towards the norm's result and v towards x, so that the gradient's second term counts."""
    g = gen(T * d)
    x, res, ds = (randn(g, T, d) for _ in range(3))
    w, q = rand(g, d) + 0.5, randn(g, d)
    dy = randn(g, T, d) + (x + res) * 0.5

    def norm(xx, ww, rr):
        n = B.moe_rmsnorm(xx, ww, EPS, residual=rr)
        return n.y, n.sum

    def backward(dy, h, w, dsum):
        return B.moe_rmsnorm_backward(dy, h, w, EPS, dsum=dsum)

    got = ob.slopes(norm, backward, x, res, w, dy, ds, randn(g, T, d) + x + res,
                    q + (dy * (x + res)).mean(0), 2.0 ** -5)
    for name, (diff, bound) in got.items():
        assert abs(diff) <= bound, (name, diff, bound)
