"""The block operators (residual RMSNorm, 8-bit outputs, linear product) in 64
bits, in plain torch on the tensors' own device, and the bounds that the
kernels' arithmetic gives.

Half a step of a type relative to the value is finfo.eps / 2: bf16 2^-8, fp32
2^-24, e4m3 2^-4.  e4m3 has subnormals below 2^-6, in steps of 2^-9.
"""
import torch

E4M3 = torch.float8_e4m3fn
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, E4M3: 2.0 ** -4}


def add_rmsnorm(x, res, w, eps, offset):
    s = x.double() if res is None else x.double() + res.double()
    return s, s / (s.pow(2).mean(1, keepdim=True) + eps).sqrt() * (offset + w.double())


def gated_norm(o, z, w, eps):
    o, z = o.double(), z.double()
    return o / (o.pow(2).mean(2, keepdim=True) + eps).sqrt() * w.double() * z * torch.sigmoid(z)


def scale_of(y):
    """y [T, n] in 64 bits -> the scale of each row."""
    return (y.abs().amax(1) / 448).clamp_min(2.0 ** -126)


def linear(x, w, sx, sw, bias, act, res):
    """(y, size) where size = sum_k |x w| |sx sw|, what the sum's rounding scales with."""
    x, w = x.double(), w.double()
    v, size = x @ w.t(), x.abs() @ w.abs().t()
    if sx is not None:
        v, size = v * sx.double()[:, None], size * sx.double()[:, None]
    if sw is not None:
        v, size = v * sw.double(), size * sw.double()
    if bias is not None:
        v = v + bias.double()
        size = size + bias.double().abs()
    if act == "silu":
        v = v * torch.sigmoid(v)
    elif act == "gelu":
        v = v * 0.5 * torch.erfc(-v * 0.5 ** 0.5)
    return (v if res is None else v + res.double()), size


# The norms: a thread adds at most 64 squares, the block 10 more sums (halved
# by the root), then the division by n, rsqrt (2 ulp), three products and the
# reciprocal of the scale: under 64 half steps of fp32.
NORM = 64 * 2.0 ** -24
# SiLU adds the fast exponential, 2 + 1.173 |z| ulp of 2^-23, and the fast
# division, 2 ulp: under 32 half steps for |z| <= 8.
GATED = NORM + 32 * 2.0 ** -24


def check_near(got, ref, rel, half, what=""):
    """|got - ref| <= |ref| (rel + half (1 + rel)), element by element."""
    tol = ref.abs() * (rel + half * (1 + rel)) + 1e-37
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def check_quant(q, scale, ref, rel, what=""):
    """q, scale against ref [T, n] in 64 bits: the scale to `rel`, each value to half an e4m3 step."""
    want = scale_of(ref)
    check_near(scale, want, rel, 0.0, what + " scale")
    got = q.double().reshape(ref.shape) * want[:, None]
    tol = ref.abs() * (2.0 ** -4 + 2 * rel) + want[:, None] * 2.0 ** -10 * (1 + 2 * rel)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def sum_bound(n_in, e4m3=False):
    """Of the tensor cores' fp32 sum over k, relative to sum |x w|: the products
    are exact, every step of 16 (bf16) or 32 (e4m3) of them is added to the
    accumulator with an error of at most 2^-22 of what was summed, and the
    epilogue's scale, bias and activation (slope at most 1.13, a few ulp) add
    less than 16 such errors."""
    return (n_in / (32 if e4m3 else 16) + 17) * 1.13 * 2.0 ** -22


def check_linear(y, ref, size, n_in, e4m3=False, what=""):
    half = HALF[y.dtype]
    err = (y.double() - ref).abs()
    tol = size * sum_bound(n_in, e4m3) * (1 + half) + ref.abs() * (half + 2.0 ** -23) + 1e-37
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def quantise(v):
    """fp32 rows -> e4m3 rows and scales, as inputs of the 8-bit product."""
    scale = (v.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    return (v / scale[:, None]).clamp(-448, 448).to(E4M3), scale
