"""moe_decode against the layer in 64 bits.

Tolerance, element by element, from where the kernels round: a sum over K is
at most n = K/4 + 64 accumulations (fp32 operands: 2K + 64), each off by at
most 2^-23 of the sum of magnitudes; h is rounded to the activation type
(half a step, eps/2) and SiLU good to 8 units of 2^-24; a gate is off by the
logits' errors on both sides of its quotient and a few units of 2^-24; the
output is rounded once.  Tokens whose selection is closer than the logits'
errors are left out.
"""

import pytest
import torch

from mixture_experts_moe_amd import binding as B
from mixture_experts_moe_amd import synth

pytestmark = pytest.mark.gpu


def real(w, s, e):
    if w.dtype != torch.uint8:
        return w[e].double()
    v = w[e].view(torch.float8_e4m3fn).double()
    return v * (s[e].double()[:, None] if s.dim() == 2 else s[e].double())


def reference(inp, residual=None):
    """(out, tolerance, usable tokens) in 64 bits."""
    x, k, I = inp.x.double(), inp.top_k, inp.I
    f32 = inp.act == "f32"
    eps = 2.0 ** -24 if f32 else 2.0 ** -8      # half a step
    u = 2.0 ** -23
    n1 = (2 * inp.d if f32 else inp.d / 4) + 64
    n2 = (2 * I if f32 else I / 4) + 64
    wg = inp.w_gate.double()
    logits, el = x @ wg.t(), (2 * inp.d + 64) * 2.0 ** -24 * (x.abs() @ wg.abs().t())
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    gates = torch.softmax(top[:, :k], dim=1)
    worst = el.amax(dim=1)
    usable = torch.ones(inp.T, dtype=torch.bool, device=x.device)
    if k < inp.E:
        gap = top[:, k - 1] - top[:, k]
        usable = (gap > 2 * worst) | (gap == 0)         # equal rows give equal logits
    eg = torch.expm1(4 * worst) + 16 * 2.0 ** -24       # relative
    out = residual.double().clone() if residual is not None else torch.zeros_like(x)
    tol = torch.zeros_like(x)
    for e in sorted(set(ids[:, :k].flatten().tolist())):
        t, j = (ids[:, :k] == e).nonzero(as_tuple=True)
        w13, w2 = real(inp.w13, inp.s13, e), real(inp.w2, inp.s2, e)
        z, ez = x[t] @ w13.t(), n1 * u * (x[t].abs() @ w13.abs().t())
        g, up = z[:, :I], z[:, I:]
        y = g * torch.sigmoid(g)
        ey = 1.1 * ez[:, :I] + 8 * 2.0 ** -24 * y.abs()
        h = y * up
        eh = ey * up.abs() + (y.abs() + ey) * ez[:, I:]
        eh = eh + eps * (h.abs() + eh) + 1e-37
        o = h @ w2.t()
        eo = eh @ w2.abs().t() + (n2 + 8 * inp.E) * u * ((h.abs() + eh) @ w2.abs().t())
        gate = gates[t, j][:, None]
        out.index_add_(0, t, gate * o)
        tol.index_add_(0, t, gate * (eo + eg[t][:, None] * (o.abs() + eo)))
    tol = tol * (1 + 2.0 ** -8) + (eps + 2.0 ** -22) * (out.abs() + tol) + 1e-37
    return out, tol, usable


def check(got, inp, residual=None, least=0.8):
    want, tol, usable = reference(inp, residual)
    assert usable.float().mean() > least
    assert torch.isfinite(got.float()).all()
    err = (got.double() - want).abs()[usable]
    worst = float((err / tol[usable]).max())
    assert worst <= 1, f"{worst:.3g} of the tolerance"


def layer(T, d, E, k, I, w, seed=0, **kw):
    cfg = dict(T=T, d=d, E=E, k=k, I=I, act="f32" if w == "f32" else "bf16", w=w, x_std=1.0,
               w_std=0.05, skew=False)
    return synth.make_inputs(cfg, device="cuda", seed=seed, **kw)


def decode(inp, **kw):
    sc = (inp.s13, inp.s2) if inp.w == "e4m3fn" else None
    return B.moe_decode(inp.x, inp.w_gate, inp.w13, inp.w2, inp.top_k, sc, **kw)


def rand_like(x, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(x.shape, generator=g, device="cuda").to(x.dtype)


CASES = [(1, 64, 1, 1, 64), (2, 64, 2, 1, 64), (16, 256, 8, 2, 512), (3, 128, 4, 4, 192),
         (5, 320, 32, 4, 448), (7, 192, 5, 5, 64), (9, 64, 1024, 64, 64), (16, 128, 1, 1, 128),
         (12, 512, 64, 8, 256), (8, 1024, 16, 2, 1088), (4, 2048, 128, 8, 768),
         (16, 2880, 32, 4, 2880), (1, 4096, 8, 2, 4096), (16, 64, 300, 64, 320)]


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3fn"])
@pytest.mark.parametrize("T,d,E,k,I", CASES)
def test_values(T, d, E, k, I, w):
    print(f"decode T={T} d={d} E={E} k={k} I={I} {w}", flush=True)
    inp = layer(T, d, E, k, I, w)
    res = rand_like(inp.x) if T % 2 else None
    check(decode(inp, residual=res), inp, res)


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3fn"])
@pytest.mark.parametrize("T,d,E,k,I", [(1, 7168, 4, 2, 128), (4, 5120, 8, 2, 192),
                                       (13, 7168, 6, 3, 64), (16, 8192, 4, 1, 128),
                                       (2, 4160, 16, 4, 64)])
def test_more_output_rows_than_four_per_unit(T, d, E, k, I, w):
    """Workgroups with several groups of four rows of W2, evenly and not.

    The bound on a logit's error grows with d squared: (2d + 64) 2^-24 of
    sum |x||w| = 0.032 d, twice 0.2 at d = 7168, while a logit's deviation is
    0.05 sqrt(d) = 4.2 and the kept and the first dropped of six lie about 1.2
    apart: about a third of the tokens are left out, more than the fifth that
    the smaller layers allow.
    """
    print(f"decode wide T={T} d={d} E={E} k={k} I={I} {w}", flush=True)
    inp = layer(T, d, E, k, I, w)
    check(decode(inp), inp, least=0.3)


@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(T):
    inp = layer(T, 256, 6, 3, 192, "bf16", seed=T)
    check(decode(inp), inp)


@pytest.mark.parametrize("T", [1, 6, 16])
def test_one_scale_per_expert(T):
    inp = layer(T, 192, 8, 2, 256, "e4m3fn", scale_mode="tensor")
    check(decode(inp), inp)


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3fn"])
@pytest.mark.parametrize("T,d,E,k,I", [(1, 512, 8, 2, 1024), (4, 2048, 64, 8, 512),
                                       (7, 320, 16, 4, 448), (16, 1024, 32, 4, 704)])
def test_schedules_give_the_same_bits(T, d, E, k, I, w):
    """Waiting for the other workgroups' h, computing what is missing at once,
    and the two halves as launches of their own."""
    inp = layer(T, d, E, k, I, w)
    res = rand_like(inp.x)
    want = decode(inp, residual=res)
    for schedule in ("static", "queue", "auto"):
        for _ in range(3):
            assert torch.equal(decode(inp, residual=res, schedule=schedule), want), schedule


@pytest.mark.parametrize("T", [1, 3, 10, 16])
def test_ties_go_to_the_lower_expert(T):
    """Identical router rows: experts 2, 5 and 6 tie for every token."""
    inp = layer(T, 256, 8, 3, 128, "bf16")
    inp.w_gate[5] = inp.w_gate[2]
    inp.w_gate[6] = inp.w_gate[2]
    check(decode(inp), inp)


def test_nan_logit_ranks_last_and_stays_with_its_token():
    inp = layer(6, 128, 4, 2, 128, "bf16")
    want, tol, usable = reference(inp)
    inp.x[3, 7] = float("nan")
    got = decode(inp)
    assert torch.isnan(got[3].float()).all()
    usable[3] = False
    assert ((got.double() - want).abs() <= tol)[usable].all()


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3fn"])
@pytest.mark.parametrize("T", [2, 11])
def test_out_may_be_the_residual(T, w):
    inp = layer(T, 320, 8, 2, 256, w)
    res = rand_like(inp.x)
    want = decode(inp, residual=res)
    assert decode(inp, residual=res, out=res) is res
    assert torch.equal(res, want)


@pytest.mark.parametrize("w", ["f32", "bf16", "e4m3fn"])
@pytest.mark.parametrize("T", [1, 5, 16])
def test_agrees_with_moe_forward(T, w):
    inp = layer(T, 512, 8, 2, 512, w)
    sc = (inp.s13, inp.s2) if w == "e4m3fn" else None
    other = B.moe_forward(inp.x, inp.w_gate, inp.w13, inp.w2, inp.top_k, sc)
    _, tol, usable = reference(inp)
    err = (decode(inp).double() - other.double()).abs()[usable]
    assert (err <= 2 * tol[usable]).all()


@pytest.mark.parametrize("w,T", [("bf16", 1), ("e4m3fn", 4), ("bf16", 12), ("f32", 7)])
def test_replays_of_a_graph_equal_eager_calls(w, T):
    inp = layer(T, 768, 16, 4, 512, w)
    out = torch.empty_like(inp.x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(inp, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        decode(inp, out=out)
    for i in range(4):
        inp.x.copy_(rand_like(inp.x, seed=20 + i))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, decode(inp))


def test_workspace_contents_do_not_matter_and_calls_follow_each_other():
    a, b = layer(2, 512, 8, 2, 512, "bf16"), layer(13, 320, 16, 4, 448, "bf16", seed=3)
    want = [decode(a), decode(b)]
    n = max(B.moe_decode_workspace_bytes(
        B.make_desc(i.T, i.d, i.E, i.I, B.MOE_DTYPE_BF16, B.MOE_DTYPE_BF16), i.top_k)
        for i in (a, b))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        for i, inp in enumerate((a, b)):
            assert torch.equal(decode(inp, workspace=ws), want[i])


def test_two_streams_at_once():
    a, b = layer(1, 1024, 8, 2, 2048, "bf16"), layer(16, 1024, 32, 4, 1024, "e4m3fn", seed=3)
    want = [decode(a), decode(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, inp in enumerate((a, b)):
            got[i].append(decode(inp, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("w", ["bf16", "e4m3fn"])
@pytest.mark.parametrize("T", [1, 8])
def test_with_a_shared_expert(T, w):
    """As a block uses them together: the shared expert's products put their
    sum onto the residual stream, and the routed experts add to that."""
    inp = layer(T, 512, 16, 4, 256, w)
    stream = rand_like(inp.x)
    g = torch.Generator(device="cuda").manual_seed(9)
    sw13 = (torch.randn((2 * 384, 512), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    sw2 = (torch.randn((512, 384), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    h = B.moe_linear(inp.x, sw13, activation="silu", gated=True)
    r = B.moe_linear(h, sw2, residual=stream)
    out = decode(inp, residual=r, out=r)
    z = inp.x.double() @ sw13.double().t()
    hs = z[:, :384] * torch.sigmoid(z[:, :384]) * z[:, 384:]
    shared = hs @ sw2.double().t()
    base = stream.double() + shared
    want, tol, usable = reference(inp, base)
    # the shared expert's h and the sum it leaves are rounded to bf16
    tol = tol + 2.0 ** -8 * (hs.abs() @ sw2.double().abs().t() + base.abs()) * 1.02 + 1e-4
    assert ((out.double() - want).abs() <= tol)[usable].all()


def test_no_tokens():
    inp = layer(1, 64, 2, 1, 64, "bf16")
    assert B.moe_decode(inp.x[:0], inp.w_gate, inp.w13, inp.w2, 1).shape == (0, 64)


def test_workspaces_that_will_not_do_are_refused():
    inp = layer(3, 128, 8, 2, 64, "bf16")
    want = decode(inp)
    n = B.moe_decode_workspace_bytes(B.make_desc(3, 128, 8, 64, B.MOE_DTYPE_BF16, B.MOE_DTYPE_BF16), 2)
    for ws in (torch.empty(n, dtype=torch.uint8),
               torch.empty(n - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)):
        with pytest.raises(ValueError):
            decode(inp, workspace=ws)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(decode(inp, workspace=ws), want)
