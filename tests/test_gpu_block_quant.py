"""gdn_block_quant on the GPU against 64 bits."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3
NAN = float("nan")


def _x(seed, T, n, dtype, glu):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, 2 * n if glu else n, generator=g, device=DEV).to(dtype)


def _check(x, glu, y, scale, what=""):
    # the scale's product and reciprocal, or with the gate the fast SiLU too
    ref = m64.glu(x) if glu else x.double()
    m64.check_block_quant(y, scale, ref, b64.GATED if glu else 4 * 2.0 ** -24, what)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 128), (1, 2048), (2, 127), (3, 129), (5, 8), (7, 136), (33, 1000), (64, 256),
                                 (100, 333), (257, 512), (1000, 130), (3000, 64), (19, 4096), (2, 12288), (5000, 384),
                                 (777, 1111), (50, 24), (9, 120)])
def test_sizes(T, n, glu, dtype):
    x = _x(T + n, T, n, dtype, glu)
    guard = torch.full((T + 1, n), 3.0, device=DEV).to(E4M3)
    sguard = torch.full((T + 1, -(-n // 128)), 7.0, device=DEV)
    y, scale = gdn().gdn_block_quant(x, glu=glu, y=guard[:T], y_scale=sguard[:T])
    torch.cuda.synchronize()
    status_clean()
    _check(x, glu, y, scale)
    assert torch.all(guard[T].float() == 3.0) and torch.all(sguard[T] == 7.0)
    y2, scale2 = gdn().gdn_block_quant(x, glu=glu)
    assert y2.stride(0) % 16 == 0 or T == 1
    assert bits_equal(y2.float(), y.float()) and bits_equal(scale2, scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n", [256, 264, 300, 301])
def test_strided(n, glu, dtype):
    T = 40
    x = _x(n, T, n, dtype, glu)
    want, wscale = gdn().gdn_block_quant(x, glu=glu)
    for off, pad in ((0, 8), (1, 2), (8, 8), (3, 0), (4, 4)):
        wide = torch.full((T, x.shape[1] + off + pad), NAN, dtype=dtype, device=DEV)
        wide[:, off:off + x.shape[1]] = x
        out = torch.full((T, n + off + pad), 3.0, device=DEV).to(E4M3)
        y, scale = gdn().gdn_block_quant(wide[:, off:off + x.shape[1]], glu=glu, y=out[:, off:off + n])
        torch.cuda.synchronize()
        assert bits_equal(y.float(), want.float()) and bits_equal(scale, wscale)
        o = out.float()
        assert torch.all(o[:, :off] == 3.0) and torch.all(o[:, off + n:] == 3.0)


@pytest.mark.parametrize("n", [256, 250])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_zeros_nans_and_range(n, dtype):
    x = _x(3, 8, n, dtype, False)
    x[0] = 0
    x[1, 5] = NAN
    x[2, :128] *= 1e-30
    x[3] *= 1e30
    x[4, 200] = 3e38
    x[5] = 1e-38
    y, scale = gdn().gdn_block_quant(x)
    torch.cuda.synchronize()
    assert torch.all(y[0].float() == 0) and torch.all(scale[0] == 2.0 ** -126)
    assert torch.isnan(scale[1, 0]) and torch.all(torch.isnan(y[1, :128].float()))
    keep = torch.tensor([0, 2, 3, 4, 5, 6, 7], device=DEV)
    _check(x[keep], False, y.float()[keep], scale[keep])
    _check(x[1:2, 128:], False, y[1:2, 128:], scale[1:2, 1:])


def test_gate_far_out():
    """Gates of any size: SiLU goes to 0 or to the gate."""
    gate = torch.tensor([-1e30, -1000.0, -200.0, -104.0, -88.0, -20.0, -1.0, 0.0, 1.0, 20.0, 88.0, 104.0, 200.0, 1000.0], device=DEV)
    up = torch.full_like(gate, 0.5)
    # one block each, so that every value sets its own scale
    x = torch.stack([gate, up], 1)
    y, scale = gdn().gdn_block_quant(x, glu=True)
    torch.cuda.synchronize()
    got = y.float().flatten().double() * scale.flatten().double()
    ref = m64.glu(x).flatten()
    assert torch.all(((got - ref).abs() <= ref.abs() * (2.0 ** -4 + 2.0 ** -12) + 1e-35))


def test_no_rows_other_stream_and_graph():
    assert gdn().gdn_block_quant(torch.empty(0, 40, device=DEV))[0].shape == (0, 40)
    x = _x(1, 500, 640, BF16, True)
    want, wscale = gdn().gdn_block_quant(x, glu=True)
    y, scale = torch.empty_like(want), torch.empty_like(wscale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gdn().gdn_block_quant(x, glu=True, y=y, y_scale=scale)
    torch.cuda.synchronize()
    assert bits_equal(y.float(), want.float()) and bits_equal(scale, wscale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn().gdn_block_quant(x, glu=True, y=y, y_scale=scale)
    x.copy_(_x(2, 500, 640, BF16, True))
    graph.replay()
    torch.cuda.synchronize()
    _check(x, True, y, scale)


def test_far_rows():
    """Rows of x and y past 2^31 elements."""
    T, n = 2 ** 31 // 8192 + 5, 8192
    x = torch.zeros(T, n, dtype=BF16, device=DEV)
    x[-5:] = _x(4, 5, n, BF16, False)
    y, scale = gdn().gdn_block_quant(x)
    near, nscale = gdn().gdn_block_quant(x[-5:].contiguous())
    torch.cuda.synchronize()
    assert bits_equal(y[-5:].float(), near.float()) and bits_equal(scale[-5:], nscale)
