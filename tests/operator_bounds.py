"""What a block of the operators around the layer may be off by, element by element:
64-bit results of the values that each step was given, and the roundings that the
steps make, each times the magnitudes that it meets.  Device and implementation are
the caller's, so that the same bounds hold the library's results and, on the CPU,
those of plain 32-bit forms with and without a planted mistake.

U = 2^-24 is half a step of fp32 and half(t) of the type t.  Sums of n terms in a
chain are off by n U of the sum of magnitudes; chain(d) counts the terms that a
thread of the norm adds, 22 more follow over the workgroup."""

import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def chain(d):
    return max(32, d / 1024 + 8)


def e_norm(d):
    """Relative error of h r w in fp32: half of its sum of squares', and six roundings."""
    return ((chain(d) + 24) / 2 + 6) * U


def silu(z):
    return z * torch.sigmoid(z)


def norm64(h, w, eps):
    """(y, r) of h in 64 bits."""
    r = (h.double().pow(2).mean(dim=1, keepdim=True) + eps).rsqrt()
    return h.double() * r * w.double(), r


def norm_gradient(dy, h, w, eps, dsum, dtype, dy_err=None):
    """{"dx", "dweight": (value, bound)} of the norm's gradient in 64 bits, for a dy of which each
    element is off by at most dy_err."""
    d = h.shape[1]
    dy, h, w = dy.double(), h.double(), w.double()
    err = torch.zeros_like(dy) if dy_err is None else dy_err
    _, r = norm64(h, w, eps)
    er = ((chain(d) + 24) / 2 + 4) * U
    g = dy * w
    second = h * (r * r * (g * h).mean(dim=1, keepdim=True))
    dx = (g - second) * r + dsum.double()
    # of dy; of the norm's sums; of the products; of the sum with dsum and the result's rounding
    ge = err * w.abs()
    tol = (ge + h.abs() * r * r * (ge * h.abs()).mean(dim=1, keepdim=True)) * r
    tol = tol + (3 * er + 8 * U) * (g.abs() + ge + second.abs()) * r
    tol = tol + (chain(d) + 29) * U * h.abs() * r ** 3 * ((g.abs() + ge) * h.abs()).mean(dim=1, keepdim=True)
    tol = tol * 1.01 + 2 * U * (dx.abs() + dsum.double().abs())
    tol = tol + half(dtype) * (dx.abs() + tol) + 1e-37
    terms = (dy * h * r).abs()
    tolw = (err * (h * r).abs()).sum(dim=0) + (h.shape[0] / 512 + 64 + er / U + 3) * U * (
        terms + err * (h * r).abs()).sum(dim=0)
    return {"dx": (dx, tol), "dweight": ((dy * h * r).sum(dim=0), tolw * 1.01 + 1e-37)}


def block(h, w, c, ids, gates, dout, eps, dtype):
    """{name: (value, bound)} of a block whose stream is h = x + residual as it was rounded:

        y = norm(h) w,  rows = y c[e] of every slot's expert e,  out = h + sum of gates rows

    and, for the gradient dout of out, of what reaches gates, h ("dx") and w ("dweight") through
    the library's steps, each of which rounds its rows to dtype."""
    T, k = ids.shape
    d, ht = h.shape[1], half(dtype)
    y, _ = norm64(h, w, eps)
    ce, gd, do = c.double()[ids.long()], gates.double(), dout.double()
    rows = y[:, None, :] * ce[:, :, None]
    # y, its rows and the scaled rows: two roundings to dtype, y's own error and a product
    rel = (1 + ht) ** 2 * (1 + e_norm(d)) * (1 + U) - 1
    row_err = rel * rows.abs()
    out = h.double() + (gd[:, :, None] * rows).sum(1)
    S = h.double().abs() + (gd[:, :, None] * (rows.abs() + row_err)).sum(1)
    tol = (gd[:, :, None] * row_err).sum(1) + (k + 2) * U * S
    tol = tol + ht * (out.abs() + tol) + 1e-37
    prod = do[:, None, :] * rows
    tolg = (do.abs()[:, None, :] * row_err).sum(2) + (d / 256 + 26) * U * (
        do.abs()[:, None, :] * (rows.abs() + row_err)).sum(2) + 1e-37
    # the rows' gradient, times c, summed over the slots: three roundings to dtype
    scale = (gd * ce).sum(1, keepdim=True)
    dy = do * scale
    dy_err = ((1 + ht) ** 3 * (1 + (k + 3) * U) - 1) * dy.abs() + 1e-37
    want = {"out": (out, tol), "dgates": (prod.sum(2), tolg)}
    want.update(norm_gradient(dy, h, w, eps, dout, dtype, dy_err))
    return want


def layer(x, ids, gates, w13, w2):
    """(value, bound) of the routed layer in fp32: sum over a token's experts of gate * w2 (silu(w1 x)
    * (w3 x)), sums of d and I products in any order."""
    T, d = x.shape
    I = w2.shape[2]
    value = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(value)
    xd = x.double()
    for j in range(ids.shape[1]):
        e = ids[:, j].long()
        a13, a2 = w13[e].double(), w2[e].double()
        z = (a13 * xd[:, None, :]).sum(2)
        ez = (d + 2) * U * (a13 * xd[:, None, :]).abs().sum(2)
        zg, zu, eg, eu = z[:, :I], z[:, I:], ez[:, :I], ez[:, I:]
        f = silu(zg)
        # slope at most 1.13; e^-z and the quotient, and z's rounding in the exponent
        ef = 1.13 * eg + (8 + 4 * zg.abs()) * U * f.abs()
        hidden = f * zu
        eh = ef * (zu.abs() + eu) + f.abs() * eu + 2 * U * hidden.abs()
        g = gates[:, j].double()[:, None]
        yd = (a2 * hidden[:, None, :]).sum(2)
        size = (a2.abs() * (hidden.abs() + eh)[:, None, :]).sum(2)
        ey = (a2.abs() * eh[:, None, :]).sum(2) + (I + 2) * U * size
        value = value + g * yd
        tol = tol + g * (ey + (ids.shape[1] + 4) * U * size)
    return value, tol * 1.01 + 1e-37


def outside(got, want):
    """The share of elements that are further from the value than its bound."""
    value, tol = want
    return float((~((got.double() - value).abs() <= tol)).double().mean())


def slopes(norm, backward, x, res, w, dy, ds, v, q, step, eps=1e-6):
    """{name: (difference, bound)}: the slope of f = <dy, y> + <ds, sum> between norm's own results
    on both sides of x along v (and of w along q), less the one that backward's dx (dweight) has.

    Both are taken along what the rounded points really differ by.  What they may be apart by: the
    curvature that 64 bits have between the same points, to the digit (w: f is linear, none), the
    errors of the two y, and those of dx (dweight)."""
    d = x.shape[1]
    mid = norm(x, w, res)[1]
    dx, dw = backward(dy, mid, w, ds)
    exact = norm_gradient(dy, mid, w, eps, ds, x.dtype)

    def ends(xx, ww):
        y, h = norm(xx, ww, res)
        y64 = norm64(h, ww, eps)[0]
        f = [(dy.double() * t.double()).sum() + (ds.double() * h.double()).sum() for t in (y, y64)]
        return h.double(), ww.double(), f, (e_norm(d) + U) * (dy.double() * y64).abs().sum()

    def apart(a, b, got, exact, along):
        (_, _, fa, na), (_, _, fb, nb) = a, b
        move = along(a) - along(b)
        curve = (fa[1] - fb[1]) - (exact[0] * move).sum()
        diff = (fa[0] - fb[0]) - (got.double() * move).sum() - curve
        return float(diff / (2 * step)), float((na + nb + (exact[1] * move.abs()).sum()) / (2 * step))

    return {"dx": apart(ends(x + step * v, w), ends(x - step * v, w), dx, exact["dx"], lambda t: t[0]),
            "dweight": apart(ends(x, w + step * q), ends(x, w - step * q), dw, exact["dweight"],
                             lambda t: t[1])}
