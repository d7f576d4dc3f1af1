"""The mixture-of-experts operators and the block-scaled product in 64 bits, in
plain torch on the tensors' own device, with the bounds that the kernels'
arithmetic gives; and inputs for them."""
import torch

from tests import block64 as b64

E4M3 = b64.E4M3


def up(n, m):
    return -(-n // m) * m


def quantise_blocks(v, rows):
    """fp32 [..., n, k] -> e4m3 and one fp32 scale for each [rows, 128] block."""
    *lead, n, k = v.shape
    if n == 0:
        return v.to(E4M3), torch.empty(*lead, 0, up(k, 128) // 128, device=v.device)
    w = torch.nn.functional.pad(v, (0, up(k, 128) - k, 0, up(n, rows) - n))
    w = w.view(*lead, up(n, rows) // rows, rows, up(k, 128) // 128, 128)
    scale = (w.abs().amax((-3, -1)) / 448).clamp_min(2.0 ** -126)
    q = (w / scale[..., :, None, :, None]).clamp(-448, 448).to(E4M3)
    return q.view(*lead, up(n, rows), up(k, 128))[..., :n, :k], scale


def padded(v, fill, extra=0):
    """v with its last dimension on 16-byte boundaries (and `extra` 16-byte pieces
    more); what lies behind a row is `fill`."""
    per = 16 // v.element_size()
    wide = torch.full((*v.shape[:-1], up(v.shape[-1], per) + extra * per), fill, device=v.device).to(v.dtype)
    raw = torch.uint8 if v.dtype == E4M3 else v.dtype
    wide.view(raw)[..., :v.shape[-1]] = v.view(raw)
    return wide[..., :v.shape[-1]]


def blocks(q, scale, rows):
    """What 8-bit [n, k] with a scale for each [rows, 128] block stands for, in 64 bits."""
    n, k = q.shape
    i = torch.arange(n, device=q.device) // rows
    j = torch.arange(k, device=q.device) // 128
    return q.double() * scale.double()[i][:, j]


def product(x, w, sx=None, sw=None):
    """(y, size): x [T, k] @ w [n, k].T and sum_k |x w|, what the sum's rounding scales with."""
    x = x.double() if sx is None else blocks(x, sx, 1)
    w = w.double() if sw is None else blocks(w, sw, 128)
    return x @ w.t(), x.abs() @ w.abs().t()


def grouped(x, w, offsets, rows, sx=None, sw=None):
    """(y, size) of the rows up to offsets[E]; an index out of range is a row of zeros."""
    ends = offsets.tolist()
    n = ends[-1]
    y = torch.zeros(n, w.shape[1], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        at = torch.arange(a, b, device=x.device) if rows is None else rows[a:b].long()
        keep = (at >= 0) & (at < x.shape[0])
        at = at[keep]
        if a == b or not len(at):
            continue
        raw = x.view(torch.uint8)[at].view(E4M3) if x.dtype == E4M3 else x[at]
        v, s = product(raw, w[e], None if sx is None else sx[at], None if sw is None else sw[e])
        y[a:b][keep], size[a:b][keep] = v, s
    return y, size


def sum_bound(k, e4m3):
    """As the linear product's, relative to sum |x w|; with block scales each block of
    128 adds one more fp32 product, sum and scale, under one error of 2^-22."""
    return b64.sum_bound(k, e4m3) + (k / 128 + 1) * 2.0 ** -22 * e4m3


def check_product(y, ref, size, k, e4m3, what=""):
    half = b64.HALF[y.dtype]
    tol = size * sum_bound(k, e4m3) * (1 + half) + ref.abs() * (half + 2.0 ** -23) + 1e-37
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def route(logits, top, renorm):
    """ids, weights (64 bits), offsets, rows, slots on the CPU."""
    x = logits.cpu().float()
    T, E = x.shape
    v, ids = x.sort(dim=1, descending=True, stable=True)
    v, ids = v.double(), ids[:, :top]
    p = torch.exp(v - v[:, :1])
    w = p[:, :top] / (p[:, :top] if renorm else p).sum(1, keepdim=True)
    w[v[:, 0] == -float("inf")] = 0.0
    flat = ids.flatten()
    by, order = flat.sort(stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1))
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * top)
    return ids.int(), w, offsets.int(), (order // top).int(), slots.view(T, top).int()


def check_weights(got, want, logits, ids, what=""):
    """The difference to the largest logit, d, is rounded once and multiplied by log2 e
    (each 2^-24 of d), the power of two and the division take a few ulp and a sum over
    the experts under 42 roundings: 2^-24 (64 + 4 |d|) of the weight."""
    x = logits.cpu().double()
    d = x.gather(1, ids.long()) - x.max(1, keepdim=True).values
    tol = want * (64 + 4 * torch.nan_to_num(d.abs(), nan=0.0, posinf=0.0)) * 2.0 ** -24 + 1e-37
    bad = ~((got.cpu().double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} weights off, first at {bad.nonzero()[0].tolist()}"


def combine(x, slots, w, res):
    """(y, size)"""
    on = (slots >= 0) & (slots < x.shape[0])
    v = x.double()[slots.long().clamp(0, x.shape[0] - 1)]
    v = torch.where(on[:, :, None], v * w.double()[:, :, None], torch.zeros((), dtype=torch.float64, device=x.device))
    y, size = v.sum(1), v.abs().sum(1)
    return (y, size) if res is None else (y + res.double(), size + res.double().abs())


def check_combine(y, ref, size, top, what=""):
    """top multiply-adds and the residual's addition, each 2^-24 of what was summed."""
    half = b64.HALF[y.dtype]
    tol = size * (top + 1) * 2.0 ** -24 * (1 + half) + ref.abs() * half + 1e-37
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def glu(x):
    x = x.double()
    n = x.shape[1] // 2
    return x[:, :n] * torch.sigmoid(x[:, :n]) * x[:, n:]


def check_block_quant(q, scale, ref, rel, what=""):
    """q [T, n], scale [T, ceil(n / 128)] against ref [T, n] in 64 bits."""
    T, n = ref.shape
    pad = lambda t: torch.nn.functional.pad(t, (0, up(n, 128) - n)).reshape(-1, 128)  # noqa: E731
    b64.check_quant(pad(q.double()), scale.flatten(), pad(ref), rel, what)
