"""Measured cases of two operators that stand beside the fused MoE layer.

``linear``: a dense product with its epilogue, the layer's own kind of product
without routing (shared experts, dense feed-forward layers, projections):

    z = (x . W^T) * scale + bias          W [R, K], R = N, or 2N when gated
    y = act(z)                            or act(z[:, :N]) * z[:, N:] when gated
    out = y + residual                    [M, N]

``decode``: the whole MoE layer for at most 16 tokens, with a residual:

    logits = x . W_gate^T; the top_k largest per token (ties to the lower
    index); gates = softmax over the selected logits
    out = residual + sum_j gate_j * W2_e(j) (SiLU(W1_e(j) x) * (W3_e(j) x))

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits (the router's logits in 64: the selection compares values that can lie
close together); with ``own`` true it calls the library.
"""

import math

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3fn"
SIZE = {BF16: 2, F32: 4, E4M3: 1}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _linear(name, M, N, K, w, act="none", gated=False, bias=False, residual=False, pad=0):
    """pad: columns by which a row of x is longer than K in memory."""
    return dict(name=name, op="linear", M=M, N=N, K=K, w=w, act=act, gated=gated, bias=bias,
                residual=residual, pad=pad)


def _decode(name, T, d, E, k, I, w, residual=True):
    return dict(name=name, op="decode", T=T, d=d, E=E, k=k, I=I, w=w, residual=residual)


def listed():
    return [
        # the up projection of the smallest configured layer, one token: only latency counts
        _linear("linear_f32_token", 1, 512, 256, F32, act="gelu", bias=True),
        # a dense down projection of one decoded token at the decode configuration's sizes, added
        # to the residual stream: a pure read of the weights
        _linear("linear_bf16_token", 1, 4096, 14336, BF16, residual=True),
        # the gate/up product of a shared expert beside 256 fine-grained ones, eight decoded tokens
        _linear("linear_e4m3_gated_8", 8, 2048, 7168, E4M3, act="silu", gated=True),
        # the gate/up product of a dense layer for a full decode batch
        _linear("linear_bf16_gated_64", 64, 14336, 4096, BF16, act="silu", gated=True),
        # a biased product over a ragged prefill batch, x a slice of wider rows
        _linear("linear_bf16_ragged", 333, 2880, 2880, BF16, act="gelu_tanh", bias=True,
                residual=True, pad=64),
        # sizes that no tile divides and rows that are not 16-byte aligned
        _linear("linear_bf16_odd", 77, 1001, 777, BF16, act="relu", bias=True),
        # a shared expert's down projection over a prefill batch, weights in 8 bits
        _linear("linear_e4m3_prefill", 2048, 7168, 2048, E4M3, residual=True),
        # the gate/up product of a dense layer over a prefill batch: bound by the matrix cores
        _linear("linear_bf16_gated_prefill", 4096, 14336, 4096, BF16, act="silu", gated=True),
        # the smallest configured layer
        _decode("decode_f32_tiny", 16, 256, 8, 2, 512, F32, residual=False),
        # one decoded token through a layer of few large experts
        _decode("decode_bf16_token", 1, 4096, 8, 2, 14336, BF16),
        # four decoded tokens through a layer of many small experts, weights in 8 bits
        _decode("decode_e4m3_4", 4, 7168, 256, 8, 2048, E4M3),
        # sixteen tokens, sizes that are no powers of two
        _decode("decode_bf16_16", 16, 2880, 32, 4, 2880, BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limit = max(_flops(c) for c in listed())
    while True:
        if rng.random() < 0.6:
            gated = rng.random() < 0.4
            act = rng.choice(ACTS)
            w = rng.choice((BF16, BF16, E4M3, F32))
            step = rng.choice((1, 8, 16, 64))       # 1: any size, rows mostly not 16-byte aligned
            N, K = (max(step, _log(rng, 64, 14336) // step * step) for _ in range(2))
            case = _linear(None, _log(rng, 1, 4096), N, K, w, act, gated, rng.random() < 0.5,
                           rng.random() < 0.5, rng.choice((0, 0, 16, 5)))
            if _flops(case) > limit / (8 if w == F32 else 1):
                continue
        else:
            w = rng.choice((BF16, E4M3, F32))
            E = _log(rng, 4, 256)
            d, I = (max(64, _log(rng, 128, 8192) // 64 * 64) for _ in range(2))
            case = _decode(None, rng.randint(1, 16), d, E, rng.randint(1, min(8, E)), I, w,
                           rng.random() < 0.5)
            if E * 3 * d * I * SIZE[w] > 12e9 or case["T"] * case["k"] * 3 * d * I > 3e9:
                continue
        del case["name"]
        return case


def _flops(c):
    if c["op"] == "linear":
        return 2.0 * c["M"] * c["N"] * (2 if c["gated"] else 1) * c["K"]
    return 2.0 * c["T"] * (c["E"] * c["d"] + c["k"] * 3 * c["d"] * c["I"])


def work(case):
    w, act = SIZE[case["w"]], 4 if case["w"] == F32 else 2
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        rows = N * (2 if case["gated"] else 1)
        nbytes = M * K * act + rows * K * w + M * N * act
        nbytes += rows * 4 * ((case["w"] == E4M3) + case["bias"]) + M * N * act * case["residual"]
    else:
        T, d, E, k, I = (case[n] for n in ("T", "d", "E", "k", "I"))
        used = E * (1.0 - (1.0 - k / E) ** T)       # experts that T independent tokens touch
        nbytes = used * (3 * d * I * w + (4 * (2 * I + d) if case["w"] == E4M3 else 0))
        nbytes += E * d * 4 + T * d * act * (2 + case["residual"])
    return {"bytes": float(nbytes), "flops": _flops(case)}


# ------------------------------------------------------------------ inputs

def _gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(1_000_003 * (seed + 1))
    return g


def _weights(rows, K, fmt, g, dev):
    """N(0, 0.02) rows in the stored format, and their scales (e4m3fn: one per row, the row's
    largest magnitude on the format's largest value)."""
    a = torch.randn((rows, K), generator=g, device=dev) * 0.02
    if fmt == F32:
        return a, None
    if fmt == BF16:
        return a.to(torch.bfloat16), None
    scale = a.abs().amax(dim=1).clamp_min(1e-30) / 448.0
    return (a / scale[:, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = _gen(seed, dev)
    fmt = case["w"]
    adt = torch.float32 if fmt == F32 else torch.bfloat16
    s = {"case": dict(case)}

    def acts(rows, cols):
        return torch.randn((rows, cols), generator=g, device=dev).to(adt)

    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        rows = N * (2 if case["gated"] else 1)
        s["x"] = acts(M, K + case["pad"])[:, :K]
        s["w"], s["scale"] = _weights(rows, K, fmt, g, dev)
        s["bias"] = torch.randn((rows,), generator=g, device=dev) * 0.1 if case["bias"] else None
        s["residual"] = acts(M, N) if case["residual"] else None
        return s
    T, d, E, I = case["T"], case["d"], case["E"], case["I"]
    s["x"] = acts(T, d)
    s["residual"] = acts(T, d) if case["residual"] else None
    s["w_gate"] = torch.randn((E, d), generator=g, device=dev) * 0.02
    wdt = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.uint8}[fmt]
    s["w13"] = torch.empty((E, 2 * I, d), dtype=wdt, device=dev)
    s["w2"] = torch.empty((E, d, I), dtype=wdt, device=dev)
    s["scales"] = None
    if fmt == E4M3:
        s["scales"] = (torch.empty((E, 2 * I), device=dev), torch.empty((E, d), device=dev))
    for e in range(E):
        for n, (t, rows, K) in enumerate(((s["w13"], 2 * I, d), (s["w2"], d, I))):
            q, sc = _weights(rows, K, fmt, g, dev)
            t[e] = q
            if sc is not None:
                s["scales"][n][e] = sc
    return s


# ------------------------------------------------------------------ one pass

def _real(w, scale):
    """Stored weights as 32-bit values."""
    if w.dtype == torch.uint8:
        return w.view(torch.float8_e4m3fn).float() * scale[..., None]
    return w.float()


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * (-1.0 / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ _real(s["w"], s["scale"]).t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z[:, :c["N"]], c["act"]) * z[:, c["N"]:] if c["gated"] else _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _plain_decode(s):
    c, x = s["case"], s["x"]
    k, I = c["k"], c["I"]
    logits = x.double() @ s["w_gate"].double().t()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = torch.exp(top - top[:, :1])
    gates = (w / w.sum(dim=1, keepdim=True)).float()
    rows = []
    for t in range(c["T"]):
        xt, y = x[t].float(), 0.0
        for j in range(k):
            e = ids[t, j:j + 1]
            s13, s2 = (None, None) if s["scales"] is None else (q.index_select(0, e)[0]
                                                                for q in s["scales"])
            z = _real(s["w13"].index_select(0, e)[0], s13) @ xt
            h = _act(z[:I], "silu") * z[I:]
            y = y + gates[t, j] * (_real(s["w2"].index_select(0, e)[0], s2) @ h)
        rows.append(y)
    out = torch.stack(rows)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(x.dtype)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain_linear(s) if c["op"] == "linear" else _plain_decode(s)
    from mixture_experts_moe_amd import binding as moe
    if c["op"] == "linear":
        return moe.moe_linear(s["x"], s["w"], scale=s["scale"], bias=s["bias"],
                              activation=None if c["act"] == "none" else c["act"],
                              gated=c["gated"], residual=s["residual"])
    return moe.moe_decode(s["x"], s["w_gate"], s["w13"], s["w2"], c["k"], s["scales"],
                          residual=s["residual"])


# ------------------------------------------------------------------ 64 bits

def _f64(w, scale):
    """Stored weights in 64 bits; e4m3fn codes decoded from their bits."""
    if w.dtype != torch.uint8:
        return w.double()
    b = torch.arange(256, device=w.device)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    value = torch.where(b >= 128, -mag, mag)
    return value[w.long()] * scale.double().unsqueeze(-1)


def _act64(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "linear":
        N, step = case["N"], 2048
        out = torch.empty((case["M"], N), dtype=torch.float64, device=x.device)
        for n in range(0, N, step):         # output columns n .. n + step
            parts = []
            for off in (0, N) if case["gated"] else (0,):
                r = slice(off + n, off + min(N, n + step))
                z = torch.matmul(x, _f64(s["w"][r], None if s["scale"] is None else s["scale"][r]).T)
                parts.append(z + s["bias"][r].double() if s["bias"] is not None else z)
            y = _act64(parts[0], case["act"])
            out[:, n:n + step] = y * parts[1] if case["gated"] else y
        return out + s["residual"].double() if s["residual"] is not None else out
    I, k = case["I"], case["k"]
    out = s["residual"].double() if s["residual"] is not None else torch.zeros_like(x)
    logits = (x @ s["w_gate"].double().T).tolist()
    chosen = {}                              # expert -> [(token, gate)]
    for t, row in enumerate(logits):
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        total = math.fsum(math.exp(row[e] - row[order[0]]) for e in order)
        for e in order:
            chosen.setdefault(e, []).append((t, math.exp(row[e] - row[order[0]]) / total))
    for e, users in sorted(chosen.items()):
        tok = [t for t, _ in users]
        s13, s2 = (None, None) if s["scales"] is None else (q[e] for q in s["scales"])
        z = x[tok] @ _f64(s["w13"][e], s13).T
        y = (_act64(z[:, :I], "silu") * z[:, I:]) @ _f64(s["w2"][e], s2).T
        for n, (t, gate) in enumerate(users):
            out[t] += gate * y[n]
    return out
