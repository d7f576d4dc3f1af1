"""The operators of a mixture-of-experts MLP and of 8-bit weights with a scale
for each block of 128, as cases that can be timed.

A block of the hybrid model ends in an MLP of many small experts, of which each
token takes a few.  With r a row of the pairs (token, choice) sorted by expert:

  route       ids, w = the top k of softmax(logits_t);  the pairs' order
  quant       scale_tb = max_{j in block b} |v_tj| / 448, q = v / scale in e4m3;
              v = x, or SiLU(x[:n]) x[n:]
  experts     y_r = W_e x_{rows[r]}        for offsets[e] <= r < offsets[e + 1]
  linear      y_tn = sum_b sx_tb sw_{n/128,b} sum_{k in b} x_tk w_nk
  combine     y_t = residual_t + sum_j w_tj x_{slots[t][j]}

where b runs over blocks of 128 in k; the experts' products take bf16, or e4m3
with the block scales of ``linear``.

``run`` computes them in elementary torch operations where ``own`` is false,
and calls the package where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
TINY = 2.0 ** -126                      # the smallest scale: a block of zeros keeps a finite 1 / scale
B = 128                                 # values that share a scale
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # a decode step of 256 sequences: 10 of 512 experts for each
        {"name": "route 256x512 top 10 f32", "op": "route", "tokens": 256, "experts": 512, "top": 10, "dtype": "f32", "renorm": True},
        # the eight prompts of the varlen prefill (20,668 tokens); logits in bf16 have ties
        {"name": "route 20668x512 top 10 bf16", "op": "route", "tokens": 20668, "experts": 512, "top": 10, "dtype": "bf16", "renorm": True},
        # fp32 activations of an odd width before a projection in 8 bits
        {"name": "quant 777x1111 f32", "op": "quant", "rows": 777, "n": 1111, "dtype": "f32", "glu": False},
        # the prefill's gate and up products, on their way into the down product
        {"name": "quant 206680x512 glu bf16", "op": "quant", "rows": 206680, "n": 512, "dtype": "bf16", "glu": True},
        # one request's next token through its ten experts
        {"name": "experts 1x10/512 2048x1024 e4m3", "op": "experts", "tokens": 1, "top": 10, "experts": 512, "n_in": 2048, "n_out": 1024, "dtype": "e4m3", "gather": True},
        # a decode step's gate and up products: every expert's weights for a few rows
        {"name": "experts 256x10/512 2048x1024 e4m3", "op": "experts", "tokens": 256, "top": 10, "experts": 512, "n_in": 2048, "n_out": 1024, "dtype": "e4m3", "gather": True},
        # bf16 experts, rows in place, odd sizes everywhere
        {"name": "experts 1237x4/60 1003x777 bf16", "op": "experts", "tokens": 1237, "top": 4, "experts": 60, "n_in": 1003, "n_out": 777, "dtype": "bf16", "gather": False},
        # the prefill's gate and up products
        {"name": "experts 20668x10/512 2048x1024 e4m3", "op": "experts", "tokens": 20668, "top": 10, "experts": 512, "n_in": 2048, "n_out": 1024, "dtype": "e4m3", "gather": True},
        # a decode step's projection into the q|k|v stream
        {"name": "linear 256x2048x8192", "op": "linear", "tokens": 256, "n_in": 2048, "n_out": 8192, "out": "bf16"},
        # the varlen prefill's projection into the q|k|v stream
        {"name": "linear 20668x2048x8192", "op": "linear", "tokens": 20668, "n_in": 2048, "n_out": 8192, "out": "bf16"},
        # a decode step's ten rows of each token, back into the residual stream
        {"name": "combine 256x10x2048 bf16", "op": "combine", "tokens": 256, "top": 10, "hidden": 2048, "dtype": "bf16", "residual": True},
        # the prefill's
        {"name": "combine 20668x10x2048 bf16", "op": "combine", "tokens": 20668, "top": 10, "hidden": 2048, "dtype": "bf16", "residual": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quant", "experts", "experts", "linear", "combine"])
    tokens = _log(rng, 1, 20668)
    if op == "route":
        experts = _log(rng, 8, 512)
        return {"op": op, "tokens": tokens, "experts": experts, "top": rng.randint(1, min(10, experts)),
                "dtype": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.7}
    if op == "quant":
        n, dtype, glu = _log(rng, 33, 8192), rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5
        if rng.random() < 0.5:
            n = max(B, n // B * B)
        rows = max(1, min(10 * tokens, 206680 * 512 * 4 // (n * SIZE[dtype] * (1 + glu))))
        return {"op": op, "rows": rows, "n": n, "dtype": dtype, "glu": glu}
    if op == "combine":
        hidden, dtype = _log(rng, 33, 8192), rng.choice(["bf16", "bf16", "f32"])
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        top = rng.randint(1, 10)
        tokens = max(1, min(tokens, 20668 * 10 * 2048 * 2 // (top * hidden * SIZE[dtype])))
        return {"op": op, "tokens": tokens, "top": top, "hidden": hidden, "dtype": dtype, "residual": rng.random() < 0.7}
    n_in, n_out = _log(rng, 64, 4096), _log(rng, 33, 8192)
    if rng.random() < 0.5:
        n_in, n_out = max(B, n_in // B * B), max(64, n_out // 64 * 64)
    if op == "linear":
        tokens = max(1, min(tokens, 20668 * 2048 * 8192 // (n_in * n_out)))
        return {"op": op, "tokens": tokens, "n_in": n_in, "n_out": n_out, "out": rng.choice(["bf16", "f32"])}
    experts = max(2, min(_log(rng, 4, 512), 512 * 2048 * 1024 // (n_in * n_out)))
    top, dtype = rng.randint(1, min(10, experts)), rng.choice(["bf16", "e4m3"])
    tokens = max(1, min(tokens, 20668 * 10 * 2048 * 512 // (n_in * n_out * top)))
    return {"op": op, "tokens": tokens, "top": top, "experts": experts, "n_in": n_in, "n_out": n_out, "dtype": dtype,
            "gather": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs --

def _up(n, m):
    return -(-n // m) * m


def _quantise(v, rows):
    """[..., n, k] in e4m3 with one scale for each [rows, 128] block of it."""
    *lead, n, k = v.shape
    w = torch.nn.functional.pad(v, (0, _up(k, B) - k, 0, _up(n, rows) - n))
    w = w.view(*lead, _up(n, rows) // rows, rows, _up(k, B) // B, B)
    scale = (w.abs().amax((-3, -1)) / E4M3_MAX).clamp_min(TINY)
    q = (w / scale[..., :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return q.view(*lead, _up(n, rows), _up(k, B))[..., :n, :k], scale


def _padded(v):
    """v with its rows on 16-byte boundaries, as a view of a wider buffer where its width is odd; packed but for that."""
    width = _up(v.shape[-1], 16 // v.element_size())
    wide = torch.zeros(*v.shape[:-1], width, dtype=torch.uint8 if v.dtype == E4M3 else v.dtype, device=v.device)
    wide = wide.view(v.dtype)
    wide[..., :v.shape[-1]] = v
    return wide[..., :v.shape[-1]]


def _choices(randn, tokens, experts, top):
    """Each token's experts, some asked for more than others, and the pairs sorted by expert."""
    ids = (randn(tokens, experts) + 0.5 * randn(experts)).topk(top, dim=1).indices
    order = ids.flatten().sort(stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(ids.flatten(), minlength=experts).cumsum(0)
    return order, offsets


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s, op = dict(case), case["op"]
    dt = TYPES[case.get("dtype", "e4m3")]
    if op == "route":
        s["logits"] = (randn(s["tokens"], s["experts"]) + 0.5 * randn(s["experts"])).to(dt)
    elif op == "quant":
        s["x"] = randn(s["rows"], s["n"] * (2 if s["glu"] else 1)).to(dt)
    elif op == "combine":
        T, k, H = s["tokens"], s["top"], s["hidden"]
        s["x"] = randn(T * k, H).to(dt)
        s["w"] = torch.softmax(randn(T, k), 1)
        s["slots"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
        s["res"] = (3 * randn(T, H)).to(dt) if s["residual"] else None
    else:
        T, K, N = s["tokens"], s["n_in"], s["n_out"]
        s["sx"] = s["sw"] = s["rows"] = None
        if op == "linear":
            (x, s["sx"]), (w, s["sw"]) = _quantise(randn(T, K), 1), _quantise(randn(N, K) * K ** -0.5, B)
        else:
            order, s["offsets"] = _choices(randn, T, s["experts"], s["top"])
            rows = s["offsets"][1:] - s["offsets"][:-1]
            s["most"], s["used"] = int(rows.max()), rows.nonzero().flatten()     # rows of the busiest expert, experts with any
            if s["gather"]:
                s["rows"] = (order // s["top"]).to(torch.int32)
            x, w = randn(T if s["gather"] else T * s["top"], K), randn(s["experts"], N, K) * K ** -0.5
            if s["dtype"] == "e4m3":
                (x, s["sx"]), (w, s["sw"]) = _quantise(x, 1), _quantise(w, B)
            else:
                x, w = x.to(dt), w.to(dt)
        s["x"], s["w"] = _padded(x), _padded(w)
    return s


# ------------------------------------------------------------ plain form --

def _spread(scale, rows, n, k):
    """A scale of each [rows, 128] block for every element of [n, k]."""
    return scale.repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(B, -1)[..., :k]


def _plain(s):
    op = s["op"]
    if op == "route":
        T, E, k = s["tokens"], s["experts"], s["top"]
        v, ids = s["logits"].float().sort(dim=1, descending=True, stable=True)
        p = torch.exp(v - v[:, :1])
        w = p[:, :k] / (p[:, :k] if s["renorm"] else p).sum(1, keepdim=True)
        ids = ids[:, :k]
        by, order = ids.flatten().sort(stable=True)
        slots = torch.empty_like(order)
        slots[order] = torch.arange(T * k, device=DEV)
        offsets = torch.searchsorted(by, torch.arange(E + 1, device=DEV))
        return {"ids": ids.int(), "weights": w, "offsets": offsets.int(), "rows": (order // k).int(), "slots": slots.view(T, k).int()}
    if op == "quant":
        x, R, n = s["x"].float(), s["rows"], s["n"]
        if s["glu"]:
            gate, up = x[:, :n], x[:, n:]
            x = gate / (1 + torch.exp(-gate)) * up
        v = torch.zeros(R, _up(n, B), device=DEV)
        v[:, :n] = x
        v = v.view(R, -1, B)
        scale = (v.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
        q = (v / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        return {"y": q.view(R, -1)[:, :n].contiguous(), "scale": scale}
    if op == "combine":
        y = (s["x"].float()[s["slots"].long()] * s["w"][:, :, None]).sum(1)
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(s["x"].dtype)}
    x, w, sw, K, N = s["x"].float(), s["w"], s["sw"], s["n_in"], s["n_out"]
    if op == "experts":
        w = (w.view(torch.uint8) if w.dtype == E4M3 else w)[s["used"]].view(w.dtype)
        sw = sw if sw is None else sw[s["used"]]
    w = w.float()
    if s["sx"] is not None:
        x, w = x * _spread(s["sx"], 1, x.shape[0], K), w * _spread(sw, B, N, K)
    if op == "linear":
        return {"y": torch.matmul(x, w.t()).to(TYPES[s["out"]])}
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    R = x.shape[0]
    at = torch.arange(R, device=DEV)
    e = torch.searchsorted(s["offsets"][1:][s["used"]].long(), at, right=True)
    at = at - s["offsets"][s["used"]][e]
    packed = torch.zeros(w.shape[0], s["most"], K, device=DEV)
    packed[e, at] = x
    return {"y": torch.matmul(packed, w.transpose(1, 2))[e, at].to(torch.bfloat16)}


def run(state):
    s = state
    if not own:
        return _plain(s)
    import gated_deltanet_linear_10_gb300 as gdn
    op = s["op"]
    if op == "route":
        ids, w, offsets, rows, slots = gdn.gdn_moe_route(s["logits"], s["top"], renormalize=s["renorm"])
        return {"ids": ids, "weights": w, "offsets": offsets, "rows": rows, "slots": slots}
    if op == "quant":
        y, scale = gdn.gdn_block_quant(s["x"], glu=s["glu"])
        return {"y": y, "scale": scale}
    if op == "combine":
        return {"y": gdn.gdn_moe_combine(s["x"], s["slots"], s["w"], residual=s["res"])}
    if op == "linear":
        return {"y": gdn.gdn_linear_block(s["x"], s["w"], s["sx"], s["sw"], y_dtype=TYPES[s["out"]])}
    return {"y": gdn.gdn_grouped_linear(s["x"], s["w"], s["offsets"], rows=s["rows"], x_scale=s["sx"], weight_scale=s["sw"])}


# ------------------------------------------------- the work and 64 bits --

def work(case):
    """Each input read once, each output written once; a multiply-add counts two."""
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top"]
        return {"bytes": T * E * SIZE[case["dtype"]] + 16 * T * k + 4 * (E + 1), "flops": 2 * T * E}
    if op == "quant":
        n, m = case["rows"] * case["n"], 2 if case["glu"] else 1
        return {"bytes": n * (m * SIZE[case["dtype"]] + 1) + 4 * case["rows"] * (_up(case["n"], B) // B), "flops": (9 if case["glu"] else 3) * n}
    if op == "combine":
        T, k, H, e = case["tokens"], case["top"], case["hidden"], SIZE[case["dtype"]]
        return {"bytes": T * H * e * (k + 1 + case["residual"]) + 8 * T * k, "flops": 2 * T * k * H}
    T, K, N, kb = case["tokens"], case["n_in"], case["n_out"], _up(case["n_in"], B) // B
    if op == "linear":
        return {"bytes": (T + N) * K + T * N * SIZE[case["out"]] + 4 * kb * (T + _up(N, B) // B), "flops": 2 * T * N * K}
    E, k, e = case["experts"], case["top"], SIZE[case["dtype"]]
    used = E * (1 - (1 - k / E) ** T)                                # experts that some token asks for, all alike
    xs, R = T if case["gather"] else T * k, T * k
    moved = xs * K * e + used * N * K * e + R * N * 2 + 4 * (E + 1) + (4 * R if case["gather"] else 0)
    moved += 4 * kb * (xs + used * (_up(N, B) // B)) if case["dtype"] == "e4m3" else 0
    return {"bytes": moved, "flops": 2 * R * N * K}


def _blocks64(q, scale, rows):
    """The values in 64 bits that 8-bit [n, k] with a scale for each [rows, 128] block stands for."""
    n, k = q.shape
    i = torch.arange(n, device=DEV) // rows
    j = torch.arange(k, device=DEV) // B
    return q.double() * scale.double()[i][:, j]


def exact(case, seed):
    """The formulas in 64 bits, before the rounding to the outputs' types."""
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        x = s["logits"].double()
        w, top = torch.softmax(x, 1), case["top"]
        w = w.sort(dim=1, descending=True).values[:, :top]
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": None, "weights": w, "offsets": None, "rows": None, "slots": None}
    if op == "quant":
        x, n = s["x"].double(), case["n"]
        if case["glu"]:
            x = x[:, :n] * torch.sigmoid(x[:, :n]) * x[:, n:]
        scale = torch.stack([b.abs().max(1).values for b in x.split(B, dim=1)], 1) / E4M3_MAX
        scale = torch.maximum(scale, torch.full_like(scale, TINY))
        return {"y": torch.cat([b / scale[:, i:i + 1] for i, b in enumerate(x.split(B, dim=1))], 1), "scale": scale}
    if op == "combine":
        y = s["res"].double() if case["residual"] else torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=DEV)
        for j in range(case["top"]):
            y = y + s["w"][:, j:j + 1].double() * s["x"].index_select(0, s["slots"][:, j].long()).double()
        return {"y": y}
    x = s["x"].double() if s["sx"] is None else _blocks64(s["x"], s["sx"], 1)
    if op == "linear":
        return {"y": torch.einsum("tk,nk->tn", x, _blocks64(s["w"], s["sw"], B))}
    y = torch.empty(case["tokens"] * case["top"], case["n_out"], dtype=torch.float64, device=DEV)
    ends = s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            w = s["w"][e].double() if s["sw"] is None else _blocks64(s["w"][e], s["sw"][e], B)
            y[a:b] = torch.einsum("tk,nk->tn", x[a:b] if s["rows"] is None else x[s["rows"][a:b].long()], w)
    return {"y": y}
