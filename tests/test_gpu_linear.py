"""moe_linear against the product in 64 bits.

Tolerance.  A channel sum is a chain of fp32 MFMA accumulations, each wrong
by at most one unit of 2^-23 of the running sum of magnitudes S = |x| . |w|^T
(the matrix core may truncate); for bf16 and e4m3fn operands (exact products)
an MFMA adds 16 or more k at once or four at a time, for fp32 one at a time
with a rounded product, so at most n = K/4 + 64 (fp32: 2K + 64) errors of
2^-23 S, plus one 2^-23 S each for the scale and the bias.  The activations
have slopes of at most 1.13 (gated: the product rule), are themselves good to
8 units of 2^-24, and the result is rounded once to the output type: half a
step, eps/2 of its magnitude.
"""

import ctypes
import math

import pytest
import torch

from mixture_experts_moe_amd import binding as B

pytestmark = pytest.mark.gpu

FNS = [None, "relu", "silu", "gelu", "gelu_tanh"]
FMTS = ["f32", "bf16", "e4m3fn"]


def act64(z, fn):
    if fn == "relu":
        return z.clamp_min(0.0)
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu":
        return z * torch.special.ndtr(z)
    if fn == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def w64(w):
    return w.view(torch.float8_e4m3fn).double() if w.dtype == torch.uint8 else w.double()


def check(out, x, w, fn, gated, bias, scale, residual):
    xd, wd = x.double(), w64(w)
    K = x.shape[1]
    z, S = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if scale is not None:
        z, S = z * scale.double(), S * scale.double().abs()
    if bias is not None:
        z, S = z + bias.double(), S + bias.double().abs()
    n = (2 * K if x.dtype == torch.float32 else K / 4) + 64
    ez = n * 2.0 ** -23 * S
    N = z.shape[1] // 2 if gated else z.shape[1]
    y, ey = act64(z[:, :N], fn), 1.13 * ez[:, :N]
    ey = ey + 8 * 2.0 ** -24 * y.abs()
    if gated:
        up, eu = z[:, N:], ez[:, N:]
        ey = ey * up.abs() + (y.abs() + ey) * eu
        y = y * up
    if residual is not None:
        y = y + residual.double()
    tol = ey * (1 + 2.0 ** -8) + (torch.finfo(out.dtype).eps / 2 + 2.0 ** -22) * y.abs() + 1e-37
    err = (out.double() - y).abs()
    assert torch.isfinite(out.float()).all()
    bad = err > tol
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside: worst "
                           f"{float((err / tol).max()):.3g} of the tolerance at "
                           f"{bad.nonzero()[0].tolist()}")


def inputs(M, N, K, fmt, gated=False, bias=True, residual=True, per_tensor=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + M + 7 * N + 13 * K)
    R = 2 * N if gated else N
    adt = torch.float32 if fmt == "f32" else torch.bfloat16
    x = torch.randn((M, K), generator=g, device="cuda").to(adt)
    w = torch.randn((R, K), generator=g, device="cuda") * 0.1
    scale = None
    if fmt == "bf16":
        w = w.to(torch.bfloat16)
    elif fmt == "e4m3fn":
        scale = (torch.rand((1 if per_tensor else R,), generator=g, device="cuda") + 0.5) * 0.1
        w = (w * 10).to(torch.float8_e4m3fn).view(torch.uint8)
    b = torch.randn((R,), generator=g, device="cuda") if bias else None
    r = torch.randn((M, N), generator=g, device="cuda").to(adt) if residual else None
    return x, w, b, scale, r


SHAPES = [(1, 1, 1), (1, 5, 3), (2, 4, 64), (3, 64, 64), (5, 130, 520), (8, 256, 1024),
          (16, 100, 256), (16, 1030, 2100), (17, 33, 65), (33, 512, 1024), (64, 64, 8),
          (77, 1001, 777), (128, 128, 4096), (130, 260, 520), (257, 300, 64), (300, 515, 1000),
          (512, 640, 320)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_values(M, N, K, gated, fmt):
    print(f"linear {M}x{N}x{K} gated={gated} {fmt}", flush=True)
    fn = FNS[(M + N + K) % len(FNS)]
    x, w, b, scale, r = inputs(M, N, K, fmt, gated, bias=(N + K) % 3 > 0, residual=M % 2 > 0)
    out = B.moe_linear(x, w, bias=b, activation=fn, gated=gated, scale=scale, residual=r)
    check(out, x, w, fn, gated, b, scale, r)


# Larger products: every tile size with whole and split K, tiles that end past
# M and N, K that ends inside a stage, and rows that are copied to be aligned
# (K not a multiple of 16 bytes).
LARGE = [("bf16", 975, 12755, 720, False), ("bf16", 422, 13115, 736, True),
         ("bf16", 129, 10887, 7328, False), ("bf16", 139, 6384, 4976, True),
         ("bf16", 1310, 8982, 802, False), ("bf16", 901, 6272, 670, True),
         ("bf16", 1452, 1869, 6279, False), ("e4m3fn", 3302, 4264, 1040, False),
         ("e4m3fn", 2977, 1397, 1568, True), ("e4m3fn", 147, 14600, 8176, False),
         ("e4m3fn", 986, 10000, 1813, False), ("e4m3fn", 770, 3175, 7162, True),
         ("bf16", 459, 4097, 64, False), ("bf16", 73, 11581, 64, True),
         ("bf16", 68, 1458, 5712, False), ("bf16", 1738, 2320, 72, False),
         ("bf16", 307, 6585, 64, True), ("bf16", 1954, 133, 5376, False),
         ("bf16", 65, 2998, 2640, True), ("bf16", 42, 15235, 496, True),
         ("bf16", 21, 10198, 1840, False), ("bf16", 5386, 694, 240, False),
         ("bf16", 167, 9540, 64, True), ("bf16", 22, 8468, 2528, True),
         ("bf16", 998, 4305, 82, False), ("bf16", 138, 12673, 67, True),
         ("bf16", 72, 4765, 4897, False), ("bf16", 2660, 3356, 70, False),
         ("e4m3fn", 238, 8849, 64, True), ("e4m3fn", 5617, 179, 2848, False),
         ("e4m3fn", 1118, 2836, 64, False), ("e4m3fn", 20, 5305, 1184, True),
         ("e4m3fn", 1097, 1954, 710, False), ("e4m3fn", 217, 8283, 67, True),
         ("e4m3fn", 96, 12901, 3078, False), ("f32", 197, 12707, 64, False),
         ("f32", 67, 4606, 528, True), ("f32", 962, 3901, 64, True),
         ("f32", 2075, 211, 7616, False), ("f32", 284, 12322, 68, False),
         ("f32", 19, 9381, 544, True), ("f32", 328, 8656, 69, False),
         ("f32", 71, 3071, 607, True), ("f32", 26, 65, 155, False)]


@pytest.mark.parametrize("fmt,M,N,K,gated", LARGE)
def test_large_products(M, N, K, gated, fmt):
    print(f"linear large {M}x{N}x{K} gated={gated} {fmt}", flush=True)
    fn = FNS[(M + N + K) % len(FNS)]
    x, w, b, scale, r = inputs(M, N, K, fmt, gated, bias=(N + K) % 3 > 0, residual=M % 2 > 0)
    out = B.moe_linear(x, w, bias=b, activation=fn, gated=gated, scale=scale, residual=r)
    check(out, x, w, fn, gated, b, scale, r)


@pytest.mark.parametrize("xpad,wpad", [(3, 0), (0, 3)])
@pytest.mark.parametrize("M,N,K", [(2, 300, 512), (6, 520, 512), (16, 96, 1024), (600, 2100, 520),
                                   (1300, 4200, 328)])
def test_one_operand_of_unaligned_rows(M, N, K, xpad, wpad):
    x, w, b, _, r = inputs(M, N, K, "bf16")
    _, xv = padded(x, xpad, float("nan"))
    _, wv = padded(w, wpad, float("nan"))
    out = B.moe_linear(xv, wv, bias=b, activation="relu", residual=r)
    check(out, x, w, "relu", False, b, None, r)


def test_operands_beyond_32_bit_offsets():
    """Rows 2^20 elements apart, more than 2^32 elements after the first."""
    M, N, K, ld = 4200, 136, 64, 1 << 20
    x, w, b, _, r = inputs(M, N, K, "bf16")
    xb = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    xb[:, :K] = x
    ob = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    out = B.moe_linear(xb[:, :K], w, bias=b, residual=r, out=ob[:, :N])
    check(out, x, w, None, False, b, None, r)
    del xb, ob
    wb = torch.empty((2 * M, ld), dtype=torch.bfloat16, device="cuda")
    for m in (3, 70):
        x, w, b, _, r = inputs(m, M, K, "bf16", gated=True)
        wb[:, :K] = w
        out = B.moe_linear(x, wb[:, :K], bias=b, gated=True, residual=r)
        check(out, x, w, None, True, b, None, r)


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [4, 40])
def test_each_activation_far_from_zero(M, gated, fn):
    """Sums of up to about +-100: the tails of every activation."""
    x, w, b, _, r = inputs(M, 48, 96, "f32", gated)
    w = w * 30
    out = B.moe_linear(x, w, bias=b, activation=fn, gated=gated, residual=r)
    check(out, x, w, fn, gated, b, None, r)


@pytest.mark.parametrize("M", [3, 80])
def test_one_scale_for_the_whole_weight(M):
    x, w, b, scale, r = inputs(M, 96, 256, "e4m3fn", per_tensor=True)
    out = B.moe_linear(x, w, bias=b, scale=scale, residual=r)
    check(out, x, w, None, False, b, scale, r)


def padded(t, cols, fill):
    """The same matrix as a view of rows `cols` elements longer."""
    p = torch.full((t.shape[0], t.shape[1] + cols), fill, dtype=t.dtype, device=t.device)
    p[:, :t.shape[1]] = t
    return p, p[:, :t.shape[1]]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("pad", [1, 8, 64])
@pytest.mark.parametrize("M,N,K", [(1, 48, 100), (7, 50, 72), (16, 300, 264), (70, 90, 136),
                                   (300, 260, 328)])
def test_rows_longer_than_their_length(M, N, K, pad, fmt):
    """What lies between the rows (NaN here) is neither used nor written."""
    print(f"linear strided {M}x{N}x{K} pad={pad} {fmt}", flush=True)
    x, w, b, scale, r = inputs(M, N, K, fmt, True)
    nan = float("nan")
    _, xv = padded(x, pad, nan)
    _, wv = padded(w, pad, 0x7F if fmt == "e4m3fn" else nan)
    _, rv = padded(r, pad, nan)
    buf = torch.full((M, N + pad), 7.0, dtype=x.dtype, device="cuda")
    out = B.moe_linear(xv, wv, bias=b, activation="silu", gated=True, scale=scale, residual=rv,
                       out=buf[:, :N])
    assert out.data_ptr() == buf.data_ptr()
    check(out, x, w, "silu", True, b, scale, r)
    assert (buf[:, N:] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (5, 70, 130), (40, 256, 512), (290, 300, 256)])
def test_bad_tokens_and_channels_stay_their_own(M, N, K):
    """A NaN or infinite token, or weight row, reaches its own row or column only."""
    x, w, b, _, _ = inputs(M, N, K, "bf16")
    clean = B.moe_linear(x, w, bias=b)
    x2, w2 = x.clone(), w.clone()
    x2[M // 2, K - 1] = float("nan")
    w2[N - 3, 0] = float("inf")
    got = B.moe_linear(x2, w2, bias=b)
    rows = [m for m in range(M) if m != M // 2]
    cols = [n for n in range(N) if n != N - 3]
    assert torch.isnan(got[M // 2]).all()
    assert not torch.isfinite(got[:, N - 3]).any()
    if rows:
        assert torch.equal(got[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 128, 512), (9, 96, 3000), (48, 128, 4096), (200, 136, 640)])
def test_out_may_be_the_residual(M, N, K, fmt):
    x, w, b, scale, r = inputs(M, N, K, fmt)
    want = B.moe_linear(x, w, bias=b, activation="gelu", scale=scale, residual=r)
    r2 = r.clone()
    got = B.moe_linear(x, w, bias=b, activation="gelu", scale=scale, residual=r2, out=r2)
    assert got is r2 and torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 2048), (16, 640, 4096), (48, 256, 8192),
                                   (300, 520, 1024), (1800, 4100, 999), (2048, 4096, 1024)])
def test_same_bits_every_time_and_in_a_graph(M, N, K):
    x, w, b, _, r = inputs(M, N, K, "bf16")
    want = B.moe_linear(x, w, bias=b, residual=r)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.moe_linear(x, w, bias=b, residual=r, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_linear(x, w, bias=b, residual=r, out=out)
    x1 = x.clone()
    for i in range(3):
        x.copy_(x1 * (i + 1))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, B.moe_linear(x, w, bias=b, residual=r))


def test_two_streams_with_their_own_workspaces():
    a = inputs(48, 256, 8192, "bf16")
    b = inputs(40, 512, 6144, "bf16")
    want = [B.moe_linear(t[0], t[1], bias=t[2], residual=t[4]) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, t in enumerate((a, b)):
            got[i].append(B.moe_linear(t[0], t[1], bias=t[2], residual=t[4], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_no_tokens():
    x, w, b, _, r = inputs(4, 64, 64, "bf16")
    assert B.moe_linear(x[:0], w, bias=b, residual=r[:0]).shape == (0, 64)


def test_workspaces_that_will_not_do_are_refused():
    x, w, _, _, _ = inputs(48, 256, 8192, "bf16")           # K is split
    desc = B.moe_linear_desc(48, 256, 8192, 0, 0, 0, 0, B.MOE_DTYPE_BF16, B.MOE_DTYPE_BF16, 0, 0, 0, 0)
    n = ctypes.c_size_t()
    assert B.lib().moe_linear_workspace_bytes(ctypes.byref(desc), n) == 0 and n.value > 0
    for ws in (torch.empty(n.value, dtype=torch.uint8),
               torch.empty(n.value - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(1, dtype=torch.uint8, device="cuda").expand(n.value)):
        with pytest.raises(ValueError):
            B.moe_linear(x, w, workspace=ws)
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    assert torch.equal(B.moe_linear(x, w, workspace=ws), B.moe_linear(x, w))


def test_one_row_of_a_wider_matrix():
    """One row (and one column) may have any stride."""
    x, w, b, _, _ = inputs(1, 40, 64, "f32")
    out = B.moe_linear(x.expand(1, 64), w, bias=b)
    check(out, x, w, None, False, b, None, None)
    x, w, b, _, _ = inputs(30, 40, 1, "f32")
    wide = torch.randn((30, 7), device="cuda")
    wide[:, :1] = x
    check(B.moe_linear(wide[:, :1], w, bias=b), x, w, None, False, b, None, None)
