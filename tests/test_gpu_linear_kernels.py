"""moe_linear against the product in 64 bits at sizes that reach the kernels
which the cases of test_gpu_linear.py leave out (test_linear_plan.py holds the
two lists against the library's choice; tolerance as there)."""

import pytest

from mixture_experts_moe_amd import binding as B
from test_gpu_linear import FNS, check, inputs, padded

pytestmark = pytest.mark.gpu

# format, M, N, K, gated
KERNELS = [("bf16", 65, 1440, 7360, False), ("bf16", 17, 8128, 3264, True),
           ("bf16", 17, 1228, 6128, True), ("bf16", 132, 5504, 2304, False),
           ("bf16", 21, 8224, 2512, True), ("bf16", 130, 5593, 7192, True),
           ("bf16", 68, 12505, 2422, False), ("bf16", 65, 2068, 8557, True),
           ("e4m3fn", 259, 13568, 64, False), ("e4m3fn", 67, 2752, 8192, True),
           ("e4m3fn", 17, 6016, 2176, False), ("e4m3fn", 67, 12864, 64, True),
           ("e4m3fn", 18, 4944, 1200, True), ("e4m3fn", 137, 11072, 9152, False),
           ("e4m3fn", 131, 5504, 8640, True), ("e4m3fn", 259, 14054, 69, False),
           ("e4m3fn", 2732, 73, 10663, False), ("e4m3fn", 65, 2768, 6392, True),
           ("e4m3fn", 119, 9648, 1776, True), ("e4m3fn", 6, 4133, 66, False),
           ("e4m3fn", 5, 4224, 64, False), ("e4m3fn", 16, 4500, 2320, False),
           ("e4m3fn", 9, 7001, 1033, False), ("e4m3fn", 5, 2068, 77, True),
           ("e4m3fn", 5, 2176, 64, True), ("e4m3fn", 11, 2301, 4112, True),
           ("e4m3fn", 16, 3500, 1111, True), ("f32", 74, 2816, 2112, False),
           ("f32", 71, 12528, 64, True), ("f32", 66, 4368, 528, True),
           ("f32", 706, 10048, 64, False), ("f32", 66, 1112, 10696, True),
           ("f32", 17, 5488, 1360, False), ("f32", 149, 8256, 64, True),
           ("f32", 67, 2812, 2089, False), ("f32", 646, 2301, 65, True),
           ("f32", 72, 751, 2167, True), ("f32", 5, 69, 77, False),
           ("f32", 8, 1392, 4913, True),
           ("f32", 533, 508, 199, False), ("f32", 737, 172, 193, True),
           ("f32", 1400, 2100, 1999, False), ("bf16", 2633, 80, 4688, False),
           ("bf16", 19, 3824, 2000, True), ("bf16", 68, 5440, 2512, False),
           ("bf16", 17, 5040, 1488, True), ("f32", 67, 8296, 688, False),
           ("f32", 72, 9104, 2176, False), ("f32", 66, 4424, 2240, True),
           ("f32", 17, 8304, 792, False), ("f32", 71, 8320, 880, False),
           ("f32", 66, 4112, 864, True), ("f32", 589, 11910, 67, False),
           ("f32", 65, 8230, 865, False), ("f32", 669, 5362, 67, True),
           ("f32", 81, 4222, 875, True), ("f32", 1700, 2301, 2501, True),
           ("f32", 1500, 3796, 2842, False), ("f32", 457, 12368, 280, False),
           ("f32", 200, 13312, 288, True), ("f32", 649, 10455, 215, False),
           ("f32", 66, 3264, 4863, False), ("f32", 68, 4468, 1677, True)]


@pytest.mark.parametrize("fmt,M,N,K,gated", KERNELS)
def test_values(M, N, K, gated, fmt):
    print(f"linear kernels {M}x{N}x{K} gated={gated} {fmt}", flush=True)
    fn = FNS[(M + N + K) % len(FNS)]
    x, w, b, scale, r = inputs(M, N, K, fmt, gated, bias=(N + K) % 3 > 0, residual=M % 2 > 0)
    out = B.moe_linear(x, w, bias=b, activation=fn, gated=gated, scale=scale, residual=r)
    check(out, x, w, fn, gated, b, scale, r)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "e4m3fn"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("opad,rpad", [(0, 0), (4, 0), (0, 4), (4, 8), (2, 0), (8, 2)])
@pytest.mark.parametrize("M,N,K", [(7, 52, 64), (40, 100, 128), (300, 260, 1024), (1500, 1300, 128)])
def test_rows_of_every_alignment_leave_whole(M, N, K, opad, rpad, gated, fmt):
    """Vectors of eight, of four and single elements of out and the residual;
    what lies between out's rows stays."""
    print(f"linear rows {M}x{N}x{K} +{opad} +{rpad} gated={gated} {fmt}", flush=True)
    x, w, b, scale, r = inputs(M, N, K, fmt, gated)
    _, rv = padded(r, rpad, float("nan"))
    buf, out = padded(r, opad, 7.0)
    B.moe_linear(x, w, bias=b, activation="relu", gated=gated, scale=scale, residual=rv, out=out)
    check(out, x, w, "relu", gated, b, scale, r)
    assert (buf[:, N:] == 7.0).all()
