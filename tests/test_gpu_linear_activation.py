"""The activations of gdn_linear alone, on products of zero, so that act(bias) is
what is rounded: their error over the whole range against 64 bits, and the same
bits for a token in any row, whichever channels share a word with it."""
import pytest
import torch

from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _act(v, act):
    return v * torch.sigmoid(v) if act == "silu" else v * 0.5 * torch.erfc(-v * 0.5 ** 0.5)


def _of_bias(T, b, act, out):
    """act(b) in T rows: the products are zero."""
    x, w = torch.zeros(T, 8, dtype=BF16, device=DEV), torch.zeros(b.numel(), 8, dtype=BF16, device=DEV)
    y = gdn().gdn_linear(x, w, bias=b, act=act, y_dtype=out)
    torch.cuda.synchronize()
    status_clean()
    return y


# |act(v)| is kept to 2^-19 (1 + v^2 / 16) of itself.  The power of two takes an
# argument of |v| log2(e) (SiLU) or v^2 log2(e) / 2 (GELU), rounded twice: 2^-23 of
# it times ln 2, 6e-8 v^2 for GELU; the instruction's own 2^-22 of the result.  The
# shared reciprocal: 5 half steps (2^-24), doubled by GELU's polynomial in it (slope
# at most 1.95); its fit 2.7e-7, 8 steps of Horner's rule 2e-7, 3 more products.
# 1.5e-6 + 6e-8 v^2 in all.
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [3, 100, 2100])
def test_error_over_the_range(T, act, out):
    b = torch.cat([torch.linspace(-12.5, 12.5, 6001), torch.linspace(-1, 1, 2003), torch.tensor([1e-30, -1e-30, 0.0])]).to(DEV)
    y = _of_bias(T, b, act, out).double()
    ref = _act(b.double(), act)
    tol = ref.abs() * (2.0 ** -19 * (1 + b.double() ** 2 / 16) + (2.0 ** -8 if out == BF16 else 0.0)) + 1e-37
    bad = ~((y - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first at bias {float(b[bad.nonzero()[0][1]])}"


def _before(act, mid):
    """The fp32 v with act(v) nearest mid, for mid past the minimum of act."""
    lo, hi = torch.full_like(mid, -0.7), torch.full_like(mid, 60.0)
    for _ in range(80):
        m = (lo + hi) / 2
        low = _act(m, act) < mid
        lo, hi = torch.where(low, m, lo), torch.where(low, hi, m)
    return hi.float()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N", [4095, 8191])
def test_same_bits_in_every_row(act, N):
    """Packed rows of an odd width start between two words or on one, in turn.  The
    biases of the channels in front of the 32nd ones put act(bias) next to the middle
    between two bf16 values, where one fp32 step decides."""
    g = torch.Generator(device=DEV).manual_seed(N)
    b = torch.randn(N, generator=g, device=DEV)
    at = torch.arange(31, N - 1, 32, device=DEV)
    near = torch.rand(at.numel(), generator=g, device=DEV, dtype=torch.float64) * 4 + 0.1
    bits = near.to(BF16).view(torch.int16).int() << 16        # a bf16 value, and half a step more
    v = _before(act, (bits + 0x8000).view(F32).double())
    step = torch.arange(at.numel(), device=DEV) % 8 - 4       # some fp32 steps around it
    b[at] = (v.view(torch.int32) + step.int()).view(F32)
    y = _of_bias(2100, b, act, BF16)
    assert bits_equal(y, y[:1].expand(2100, N).contiguous())
