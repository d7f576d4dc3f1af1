"""The operators around the Gated DeltaNet layer, as cases that can be timed.

A hybrid model's block around the layer is: add the residual, RMSNorm, project
to the layer's streams; then the layer; then its gated RMSNorm, project back
and add the residual.  The operators are the two norms (with an output in
8 bits and one scale per token where the product that reads it runs in 8 bits)
and the product with its epilogue:

  add_rmsnorm    s = x + residual;  y = s / sqrt(mean(s^2) + eps) * (offset + w)
  gated_quant    y = o / sqrt(mean over a head of o^2 + eps) * w * SiLU(z)
  linear         y = act(sx_t sw_n sum_k x_tk w_nk + bias_n) + residual_tn

and 8 bits: scale_t = max_j |y_tj| / 448, q = y / scale_t rounded to e4m3.

``run`` computes them in elementary torch operations where ``own`` is false,
and calls the package where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 2.0 ** -126                      # the smallest scale: a row of zeros keeps a finite 1 / scale
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
EPS = 1e-6


def listed():
    return [
        # one request's next token, before the layer
        {"name": "norm 1x2048 bf16", "op": "add_rmsnorm", "tokens": 1, "hidden": 2048, "dtype": "bf16", "out": "bf16", "offset": 0.0, "residual": True},
        # a decode step of 256 sequences, the product behind it in 8 bits
        {"name": "norm 256x2048 e4m3", "op": "add_rmsnorm", "tokens": 256, "hidden": 2048, "dtype": "bf16", "out": "e4m3", "offset": 1.0, "residual": True},
        # the eight prompts of the varlen prefill (20,668 tokens)
        {"name": "norm 20668x2048 e4m3", "op": "add_rmsnorm", "tokens": 20668, "hidden": 2048, "dtype": "bf16", "out": "e4m3", "offset": 0.0, "residual": True},
        # fp32 activations, an odd width, a first block without a residual
        {"name": "norm 1237x1111 f32", "op": "add_rmsnorm", "tokens": 1237, "hidden": 1111, "dtype": "f32", "out": "f32", "offset": 1.0, "residual": False},
        # the layer's output of a decode step, for the output projection in 8 bits
        {"name": "gated 256x32x128", "op": "gated_quant", "tokens": 256, "heads": 32, "dim": 128, "dtype": "bf16"},
        # the layer's output of the varlen prefill
        {"name": "gated 20668x32x128", "op": "gated_quant", "tokens": 20668, "heads": 32, "dim": 128, "dtype": "bf16"},
        # one token into the layer's q|k|v stream: the weights are read for one row
        {"name": "linear 1x2048x8192 bf16", "op": "linear", "tokens": 1, "n_in": 2048, "n_out": 8192, "dtype": "bf16", "out": "bf16", "bias": False, "act": "none", "residual": False},
        # a decode step's projection into the q|k|v stream, in 8 bits
        {"name": "linear 256x2048x8192 e4m3", "op": "linear", "tokens": 256, "n_in": 2048, "n_out": 8192, "dtype": "e4m3", "out": "bf16", "bias": False, "act": "none", "residual": False},
        # a decode step's output projection, the residual added in the epilogue
        {"name": "linear 256x4096x2048 bf16", "op": "linear", "tokens": 256, "n_in": 4096, "n_out": 2048, "dtype": "bf16", "out": "bf16", "bias": False, "act": "none", "residual": True},
        # odd sizes everywhere, every part of the epilogue
        {"name": "linear 777x1003x1331 bf16", "op": "linear", "tokens": 777, "n_in": 1003, "n_out": 1331, "dtype": "bf16", "out": "bf16", "bias": True, "act": "gelu", "residual": True},
        # the varlen prefill's projection into the q|k|v stream
        {"name": "linear 20668x2048x8192 bf16", "op": "linear", "tokens": 20668, "n_in": 2048, "n_out": 8192, "dtype": "bf16", "out": "bf16", "bias": True, "act": "none", "residual": False},
        # the varlen prefill's output projection in 8 bits, with the residual
        {"name": "linear 20668x4096x2048 e4m3", "op": "linear", "tokens": 20668, "n_in": 4096, "n_out": 2048, "dtype": "e4m3", "out": "bf16", "bias": False, "act": "none", "residual": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["add_rmsnorm", "gated_quant", "linear", "linear"])
    tokens = _log(rng, 1, 20668)
    if op == "add_rmsnorm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        out = rng.choice([dtype, "e4m3"])
        hidden = _log(rng, 33, 8192)
        if rng.random() < 0.5:                                  # half of them whole vectors
            hidden = max(64, hidden // 64 * 64)
        tokens = min(tokens, 20668 * 2048 * 2 // (hidden * SIZE[dtype]))
        return {"op": op, "tokens": tokens, "hidden": hidden, "dtype": dtype, "out": out,
                "offset": rng.choice([0.0, 1.0]), "residual": rng.random() < 0.7}
    if op == "gated_quant":
        heads, dim = rng.randint(1, 32), rng.choice([16, 32, 64, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        tokens = min(tokens, 20668 * 32 * 128 * 2 // (heads * dim * SIZE[dtype]))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "dtype": dtype}
    n_in, n_out = _log(rng, 64, 8192), _log(rng, 33, 12288)
    if rng.random() < 0.5:
        n_in, n_out = max(64, n_in // 64 * 64), max(64, n_out // 64 * 64)
    tokens = max(1, min(tokens, 20668 * 2048 * 8192 // (n_in * n_out)))
    return {"op": op, "tokens": tokens, "n_in": n_in, "n_out": n_out, "dtype": rng.choice(["bf16", "e4m3"]),
            "out": "bf16", "bias": rng.random() < 0.5,
            "act": rng.choice(["none", "silu", "gelu"]), "residual": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs --

def _quantise_rows(v):
    """e4m3 rows and their fp32 scales, as a user's weights and activations come in 8 bits."""
    scale = (v.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
    return (v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def _padded(v):
    """v with its rows on 16-byte boundaries, as a view of a wider buffer where its width is odd."""
    n = 16 // v.element_size()
    width = -(-v.shape[1] // n) * n
    if width == v.shape[1]:
        return v
    wide = torch.zeros(v.shape[0], width, dtype=torch.uint8 if v.dtype == E4M3 else v.dtype, device=v.device)
    wide = wide.view(v.dtype)
    wide[:, :v.shape[1]] = v
    return wide[:, :v.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    T, s = case["tokens"], dict(case)
    dt = TYPES[case["dtype"]]
    if case["op"] == "add_rmsnorm":
        H = case["hidden"]
        s["x"] = randn(T, H).to(dt)
        s["res"] = (3 * randn(T, H)).to(dt) if case["residual"] else None
        s["w"] = rand(H) + 0.5 - case["offset"]
        s["y"] = torch.empty(T, H, dtype=TYPES[case["out"]], device=DEV)
        s["ys"] = torch.empty(T, device=DEV) if case["out"] == "e4m3" else None
        s["ro"] = torch.empty(T, H, dtype=dt, device=DEV) if case["residual"] else None
    elif case["op"] == "gated_quant":
        hv, dv = case["heads"], case["dim"]
        s["o"] = (0.2 * randn(T, hv, dv)).to(dt)
        s["z"] = randn(T, hv, dv).to(dt)
        s["w"] = rand(dv) + 0.5
        s["y"] = torch.empty(T, hv, dv, dtype=E4M3, device=DEV)
        s["ys"] = torch.empty(T, device=DEV)
    else:
        K, N, out = case["n_in"], case["n_out"], TYPES[case["out"]]
        x, w = randn(T, K), randn(N, K) * K ** -0.5
        s["sx"] = s["sw"] = None
        if case["dtype"] == "e4m3":
            (x, s["sx"]), (w, s["sw"]) = _quantise_rows(x), _quantise_rows(w)
        else:
            x, w = x.to(dt), w.to(dt)
        s["x"], s["w"] = _padded(x), _padded(w)
        s["b"] = 0.5 * randn(N) if case["bias"] else None
        s["res"] = (2 * randn(T, N)).to(out) if case["residual"] else None
        s["y"] = torch.empty(T, N, dtype=out, device=DEV)
    if own:
        import gated_deltanet_linear_10_gb300 as gdn
        s["gdn"] = gdn
    return s


# ------------------------------------------------------------ plain form --

def _plain_quant(y, rows):
    """y in 32 bits -> e4m3 values and one scale per row of the [rows, -1] view."""
    flat = y.reshape(rows, -1)
    scale = (flat.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
    return (flat / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(y.shape), scale


def _plain(s):
    if s["op"] == "add_rmsnorm":
        v = s["x"].float()
        if s["res"] is not None:
            v = v + s["res"].float()
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * (s["offset"] + s["w"])
        got = {"y": y.to(TYPES[s["out"]])}
        if s["out"] == "e4m3":
            got["y"], got["scale"] = _plain_quant(y, s["tokens"])
        if s["res"] is not None:
            got["residual"] = v.to(s["x"].dtype)
        return got
    if s["op"] == "gated_quant":
        o, z = s["o"].float(), s["z"].float()
        y = o * torch.rsqrt((o * o).mean(2, keepdim=True) + EPS) * s["w"] * (z / (1 + torch.exp(-z)))
        q, scale = _plain_quant(y, s["tokens"])
        return {"y": q, "scale": scale}
    v = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["sx"] is not None:
        v = v * (s["sx"][:, None] * s["sw"])
    if s["b"] is not None:
        v = v + s["b"]
    if s["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    elif s["act"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if s["res"] is not None:
        v = v + s["res"].float()
    return {"y": v.to(TYPES[s["out"]])}


def run(state):
    s = state
    if not own:
        return _plain(s)
    if s["op"] == "add_rmsnorm":
        y, scale, res = s["gdn"].gdn_add_rmsnorm(s["x"], s["w"], residual=s["res"], eps=EPS, weight_offset=s["offset"],
                                                 y=s["y"], y_scale=s["ys"], residual_out=s["ro"])
        got = {"y": y}
        if scale is not None:
            got["scale"] = scale
        if res is not None:
            got["residual"] = res
        return got
    if s["op"] == "gated_quant":
        y, scale = s["gdn"].gdn_gated_rmsnorm_quant(s["o"], s["z"], s["w"], eps=EPS, y=s["y"], y_scale=s["ys"])
        return {"y": y, "scale": scale}
    return {"y": s["gdn"].gdn_linear(s["x"], s["w"], x_scale=s["sx"], weight_scale=s["sw"], bias=s["b"], act=s["act"],
                                     residual=s["res"], y=s["y"])}


# ------------------------------------------------- the work and 64 bits --

def work(case):
    """Each input read once, each output written once; a multiply-add counts two."""
    T = case["tokens"]
    if case["op"] == "add_rmsnorm":
        n, e = T * case["hidden"], SIZE[case["dtype"]]
        moved = n * (e + SIZE[case["out"]]) + case["hidden"] * 4
        moved += 2 * n * e if case["residual"] else 0
        moved += 4 * T if case["out"] == "e4m3" else 0
        return {"bytes": moved, "flops": 6 * n}
    if case["op"] == "gated_quant":
        n = T * case["heads"] * case["dim"]
        return {"bytes": n * (2 * SIZE[case["dtype"]] + 1) + 4 * T + 4 * case["dim"], "flops": 12 * n}
    K, N, e = case["n_in"], case["n_out"], SIZE[case["dtype"]]
    moved = (T + N) * K * e + T * N * SIZE[case["out"]]
    moved += 4 * N if case["bias"] else 0
    moved += T * N * SIZE[case["out"]] if case["residual"] else 0
    moved += 4 * (T + N) if case["dtype"] == "e4m3" else 0
    return {"bytes": moved, "flops": 2 * T * N * K}


def _exact_scaled(y):
    """y [T, n] in 64 bits -> the values that 8 bits are to hold, and the scales."""
    top = y.abs().max(dim=1).values
    scale = torch.maximum(top / E4M3_MAX, torch.full_like(top, TINY))
    return y / scale.unsqueeze(1), scale


def exact(case, seed):
    """The formulas in 64 bits, before the rounding to the outputs' types."""
    s = prepare(case, seed)
    T = case["tokens"]
    if case["op"] == "add_rmsnorm":
        a = s["x"].double()
        if case["residual"]:
            a += s["res"].double()
        rms = torch.sqrt(torch.einsum("th,th->t", a, a) / case["hidden"] + EPS)
        y = a / rms[:, None] * (s["w"].double() + case["offset"])
        if case["out"] == "e4m3":
            q, scale = _exact_scaled(y)
            got = {"y": q, "scale": scale}
        else:
            got = {"y": y}
        if case["residual"]:
            got["residual"] = a
        return got
    if case["op"] == "gated_quant":
        o, z = s["o"].double(), s["z"].double()
        rms = torch.sqrt(torch.einsum("thd,thd->th", o, o) / case["dim"] + EPS)
        y = o / rms[:, :, None] * s["w"].double() * z * torch.sigmoid(z)
        q, scale = _exact_scaled(y.reshape(T, -1))
        return {"y": q.reshape(y.shape), "scale": scale}
    x, w = s["x"].double(), s["w"].double()
    if case["dtype"] == "e4m3":
        x, w = x * s["sx"].double()[:, None], w * s["sw"].double()[:, None]
    y = torch.einsum("tk,nk->tn", x, w)
    if case["bias"]:
        y = y + s["b"].double()[None]
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
    if case["residual"]:
        y = y + s["res"].double()
    return {"y": y}
