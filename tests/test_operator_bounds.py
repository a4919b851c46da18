"""The bounds of operator_bounds.py on the CPU: plain 32-bit forms that round where the
library does stay inside them, and forms with a planted mistake do not."""

import pytest
import torch

import operator_bounds as ob

EPS = 1e-6
DTYPES = [torch.float32, torch.bfloat16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g).to(dtype)


# ------------------------------------------------------------ the norm, in fp32

def norm(x, w, res=None):
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    f = h.float()
    return (f * (1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)) * w).to(x.dtype), h


def backward(dy, h, w, dsum, plant=None):
    dy, f = dy.float(), h.float()
    r = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    g = dy if plant == "weight" else dy * w
    k = r * (g * f).mean(1, keepdim=True)
    dx = (g - (0 if plant == "second term" else f * r * k)) * r
    if plant != "dsum":
        dx = dx + dsum.float()
    if plant == "no dx":
        dx = torch.zeros_like(dx)
    dw = (dy * f * (1 if plant == "r" else r)).sum(0)
    if plant == "no dweight":
        dw = torch.zeros_like(dw)
    if plant == "last row":
        dw = (dy * f * r)[:-1].sum(0)
    return dx.to(h.dtype), dw


# ------------------------------------------------------------ a block and its gradients

def block_inputs(T, d, E, k, dtype, seed):
    g = gen(seed)
    x, res, dout = (randn(g, T, d, dtype=dtype) for _ in range(3))
    w, c = torch.rand(d, generator=g) + 0.5, torch.rand(E, generator=g) + 0.5
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    return x, res, dout, w, c, ids, torch.softmax(randn(g, T, k), 1)


def plain_block(x, res, dout, w, c, ids, gates, dtype, plant=None):
    """Step by step as the library does it, without sorting the rows."""
    y, h = norm(x, w, res)
    ce = c[ids.long()][:, :, None]
    rows = (y[:, None, :].float() * ce).to(dtype)
    used = slice(0, -1) if plant == "last slot" else slice(None)
    out = (gates[:, used, None] * rows[:, used].float()).sum(1)
    out = (out if plant == "residual" else out + h.float()).to(dtype)
    dgates = (dout.float()[:, None, :] * rows.float()).sum(2)
    if plant == "dgates of y":
        dgates = (dout.float()[:, None, :] * y.float()[:, None, :]).sum(2).expand_as(gates)
    drows = (gates[:, :, None] * dout.float()[:, None, :]).to(dtype)
    dperm = drows if plant == "expert" else (drows.float() * ce).to(dtype)
    dy = dperm.float()[:, :1 if plant == "one slot" else None].sum(1).to(dtype)
    dx, dw = backward(dy, h, w, dout, plant)
    if plant == "five percent":
        dx = dx * 1.05
    return h, {"out": out, "dgates": dgates, "dx": dx, "dweight": dw}


SIZES = [(60, 130, 5, 3), (33, 1030, 4, 2), (5, 64, 8, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,E,k", SIZES)
def test_a_plain_block_is_inside(T, d, E, k, dtype):
    inputs = block_inputs(T, d, E, k, dtype, T)
    h, got = plain_block(*inputs, dtype)
    want = ob.block(h, inputs[3], inputs[4], inputs[5], inputs[6], inputs[2], EPS, dtype)
    assert {n: ob.outside(got[n], want[n]) for n in want} == dict.fromkeys(want, 0.0)


# a mistake, and the results that it shows in
PLANTS = [("second term", ["dx"]), ("dsum", ["dx"]), ("no dx", ["dx"]), ("weight", ["dx"]),
          ("five percent", ["dx"]), ("r", ["dweight"]), ("no dweight", ["dweight"]),
          ("last row", ["dweight"]), ("residual", ["out"]), ("last slot", ["out"]),
          ("dgates of y", ["dgates"]), ("expert", ["dx", "dweight"]),
          ("one slot", ["dx", "dweight"])]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,E,k", SIZES)
@pytest.mark.parametrize("plant,shows", PLANTS)
def test_a_block_with_a_mistake_is_not(plant, shows, T, d, E, k, dtype):
    inputs = block_inputs(T, d, E, k, dtype, T)
    h, got = plain_block(*inputs, dtype, plant)
    want = ob.block(h, inputs[3], inputs[4], inputs[5], inputs[6], inputs[2], EPS, dtype)
    for n in shows:                     # (one element outside fails the library's test)
        assert ob.outside(got[n], want[n]) > 0, n


# ------------------------------------------------------------ the layer from its parts

def layer_inputs(T, d, I, E, k, seed):
    g = gen(seed)
    x = randn(g, T, d)
    w13, w2 = randn(g, E, 2 * I, d) * 0.05, randn(g, E, d, I) * 0.05
    gates, ids = torch.topk(torch.softmax(randn(g, T, E), 1), k)
    return x, ids.to(torch.int32), gates / gates.sum(1, keepdim=True), w13, w2


def plain_layer(x, ids, gates, w13, w2, plant=None):
    I = w2.shape[2]
    out = torch.zeros_like(x)
    for j in range(ids.shape[1] - (plant == "last slot")):
        e = ids[:, j].long()
        z = torch.bmm(w13[e], x[:, :, None])[:, :, 0]
        a, b = (z[:, I:], z[:, :I]) if plant == "halves" else (z[:, :I], z[:, I:])
        hid = (a if plant == "function" else a / (1 + torch.exp(-a))) * b
        y = torch.bmm(w2[e], hid[:, :, None])[:, :, 0]
        out += (1 if plant == "gates" else gates[:, j:j + 1]) * y
    return out * 0 if plant == "zeros" else out * 1.01 if plant == "one percent" else out


@pytest.mark.parametrize("plant", [None, "zeros", "last slot", "halves", "function", "gates",
                                   "one percent"])
def test_layer(plant):
    inputs = layer_inputs(60, 256, 128, 8, 2, 7)
    share = ob.outside(plain_layer(*inputs, plant), ob.layer(*inputs))
    assert share > 0 if plant else share == 0, share


# ------------------------------------------------------------ slopes

def slope_inputs(T, d, seed):
    """dy leans towards the norm's result and v towards x, so that the gradient's second term is
    as large as its first."""
    g = gen(seed)
    x, res, ds = (randn(g, T, d) for _ in range(3))
    w, q = torch.rand(d, generator=g) + 0.5, randn(g, d)
    dy = randn(g, T, d) + (x + res) * 0.5
    return x, res, w, dy, ds, randn(g, T, d) + x + res, q + (dy * (x + res)).mean(0)


@pytest.mark.parametrize("plant", [None, "second term", "dsum", "no dx", "weight", "r", "no dweight"])
@pytest.mark.parametrize("T,d", [(3, 50), (4, 1500)])
def test_slopes(T, d, plant):
    x, res, w, dy, ds, v, q = slope_inputs(T, d, T)
    got = ob.slopes(norm, lambda *a: backward(*a, plant), x, res, w, dy, ds, v, q, 2.0 ** -5)
    hit = {None: None, "r": "dweight", "no dweight": "dweight"}.get(plant, "dx")
    for name, (diff, bound) in got.items():
        assert (abs(diff) > 4 * bound) if name == hit else (abs(diff) <= bound), (name, diff, bound)
