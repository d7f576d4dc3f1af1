"""What gdn_block_quant promises of its last step: each 8-bit value is the rounding of a
number that near to the quotient, and SiLU is off by its fast functions' errors
alone, at gates of any size."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3
INF, NAN = float("inf"), float("nan")
VALUES = torch.arange(127, dtype=torch.uint8).view(E4M3).double()       # of e4m3, from 0 to 448
MIDDLES = (VALUES[1:] + VALUES[:-1]) / 2


def _rounded_within(got, q, rel):
    """Which of `got` is a rounding to e4m3 of a number within `rel` of q (64 bits)."""
    a, y = q.abs(), got.double()
    lo = VALUES.to(q.device)[torch.searchsorted(MIDDLES.to(q.device), a * (1 - rel), right=False)]
    hi = VALUES.to(q.device)[torch.searchsorted(MIDDLES.to(q.device), a * (1 + rel), right=True)]
    return (y.abs() >= lo) & (y.abs() <= hi) & (y * q >= 0)


def _near_the_middles(seed, T, n, exponents):
    """Blocks of any scale, of values half way between two steps of e4m3 or a few fp32 steps beside."""
    g = torch.Generator().manual_seed(seed)
    rows = []
    for t in range(T):
        row = []
        for c in range(0, n, 128):
            m = min(128, n - c)
            top = torch.ldexp(1 + torch.rand((), generator=g), torch.tensor(exponents[t % len(exponents)]))
            scale = torch.clamp_min(top * (1.0 / 448), 2.0 ** -126)
            x = MIDDLES.float()[torch.randint(0, len(MIDDLES), (m,), generator=g)] * scale
            x = (x.view(torch.int32) + torch.randint(-2, 3, (m,), generator=g, dtype=torch.int32)).clamp_min(0).view(F32)
            x = torch.minimum(x, top) * (1 - 2 * torch.randint(0, 2, (m,), generator=g)).float()
            x[torch.randint(0, m, (1,), generator=g)] = top
            row.append(x)
        rows.append(torch.cat(row))
    return torch.stack(rows)


@pytest.mark.parametrize("n", [8, 250, 256, 1000])
@pytest.mark.parametrize("exponents", [[0, 3, -5, 20], [-126, -125, -118, -117, -100, -88, -60, -52, -51], [60, 100, 126, 127]])
def test_the_quotient(n, exponents):
    """The scale's reciprocal and the value's product with it, 2^-24 each (and a part of their product)."""
    x = _near_the_middles(n, 300, n, exponents)
    y, scale = gdn().gdn_block_quant(x.to(DEV))
    torch.cuda.synchronize()
    status_clean()
    scale = scale.cpu()
    ok = _rounded_within(y.cpu().float(), x.double() / scale.double().repeat_interleave(128, 1)[:, :n], 1.001 * 2.0 ** -23)
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()}, first {x[~ok][0].item()!r}: {y.cpu().float()[~ok][0]}"
    # the scale: the largest value's product with 1 / 448, both rounded
    pad = torch.nn.functional.pad(x.double(), (0, -n % 128)).view(-1, 128)
    b64.check_near(scale.flatten(), b64.scale_of(pad), 1.001 * 2.0 ** -23, 0.0, "scale")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_gated_quotient(dtype):
    """The product's error, as below, and the quotient's, 2^-23."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = (2 * torch.randn(3000, 1024, generator=g, device=DEV)).to(dtype)
    y, scale = gdn().gdn_block_quant(x, glu=True)
    again, _ = gdn().gdn_block_quant(x, glu=True)
    torch.cuda.synchronize()
    assert bits_equal(y.float(), again.float())
    rel = (5 + 1.2 * x[:, :512].double().abs()) * 2.0 ** -23
    ok = _rounded_within(y.float(), m64.glu(x) / scale.double().repeat_interleave(128, 1), rel + 1.001 * 2.0 ** -23)
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 8])
def test_silu_at_any_gate(n, dtype):
    """A value alone in its block, which its scale therefore is, times 448.

    Of the product's error, in ulp of 2^-23 of it: the fast exponential 2 + 1.173 |g|, its sum with 1
    a half, the fast division 2, the product with the other half a half: 5 + 1.2 |g|; of the
    scale's, 1.  Below -87.3 the division gives 0 for what is at most 1.1e-36 of the other half."""
    if dtype == BF16:
        gate = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
        gate = gate[gate.isfinite()]
    else:
        g = torch.Generator().manual_seed(1)
        gate = torch.cat([-100 + 200 * torch.rand(100000, generator=g), torch.randn(100000, generator=g),
                          torch.exp2(-120 + 240 * torch.rand(20000, generator=g)) * (1 - 2 * torch.randint(0, 2, (20000,), generator=g)),
                          torch.tensor([80.0, -80.0, -87.3, -87.4, -88.7, -88.8, -104.0])])
    for up in (1.0, -0.3, 11.0):
        x = torch.zeros(len(gate), 2 * n, dtype=dtype)
        x[:, n - 1], x[:, 2 * n - 1] = gate, up
        x = x.to(DEV)
        y, scale = gdn().gdn_block_quant(x, glu=True)
        torch.cuda.synchronize()
        a, b = x[:, n - 1].double(), x[:, 2 * n - 1].double()
        v = a * torch.sigmoid(a) * b
        want = (v.abs() / 448).clamp_min(2.0 ** -126)
        held = v.abs() < 3.4e38                          # (the product with `up` may leave fp32)
        tol = want * (6 + 1.2 * a.abs().clamp_max(100)) * 2.0 ** -23 + 1.1e-36 * b.abs() / 448 * (a < -87)
        bad = held & ~((scale[:, 0].double() - want).abs() <= tol)
        assert not bad.any(), f"{int(bad.sum())} of {len(gate)}, first at {gate[bad.cpu()][0].item()!r}"
        # and what is held in 8 bits is the largest value
        last = y[:, n - 1].float()
        big = held & (a > -87) & (v.abs() >= 2.0 ** -126 * 449)
        assert torch.all(last[big].abs() == 448) and torch.all((last * v.float())[held] >= 0)
    status_clean()


def test_no_finite_values():
    """Infinite gates and values: the formula's own."""
    gate = torch.tensor([INF, -INF, NAN, INF, 1.0, -1.0], device=DEV)
    up = torch.tensor([2.0, 2.0, 2.0, -2.0, INF, INF], device=DEV)
    want = torch.tensor([INF, NAN, NAN, INF, INF, INF], device=DEV)
    for n in (1, 8):
        x = torch.zeros(len(gate), 2 * n, device=DEV)
        x[:, 0], x[:, n] = gate, up
        y, scale = gdn().gdn_block_quant(x, glu=True)
        torch.cuda.synchronize()
        assert bits_equal(scale[:, 0].nan_to_num(nan=-1.0, posinf=INF), want.nan_to_num(nan=-1.0, posinf=INF))
        assert torch.all(y[:, 0].float().isnan())
        if n > 1:                                        # beside an infinite value all others are 0
            assert torch.all(y[want == INF][:, 1:].float() == 0) and torch.all(y[want.isnan()].float().isnan())
    status_clean()
