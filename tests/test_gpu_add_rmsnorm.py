"""gdn_add_rmsnorm and gdn_gated_rmsnorm_quant on the GPU against the formulas
in 64 bits: widths from one element to the largest, odd ones, strided,
misaligned and in-place rows, both output forms, rows of zeros, NaNs and
infinities, rows behind the last one, another stream, and graph replay."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(DEV)


def _check(x, res, w, offset, out, eps=1e-6, **kw):
    y, scale, ro = gdn().gdn_add_rmsnorm(x, w, residual=res, eps=eps, weight_offset=offset,
                                         y_dtype=out, **kw)
    torch.cuda.synchronize()
    return y, scale, ro


@pytest.mark.parametrize("hidden", [1, 7, 8, 33, 100, 512, 1111, 2048, 4095, 4096, 4104, 8192, 8193, 16383,
                                    16384])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, E4M3), (F32, F32), (F32, E4M3)])
def test_widths(dtype, out, hidden):
    T = 5
    x, res = _rand(hidden, T, hidden).to(dtype), _rand(hidden + 1, T, hidden, scale=3).to(dtype)
    w = _rand(hidden + 2, hidden)
    for r, offset in ((res, 0.0), (None, 1.0)):
        y, scale, ro = _check(x, r, w, offset, out)
        s, ref = b64.add_rmsnorm(x, r, w, 1e-6, offset)
        if out == E4M3:
            b64.check_quant(y, scale, ref, b64.NORM, "y")
        else:
            assert scale is None and y.dtype == out
            b64.check_near(y, ref, b64.NORM, b64.HALF[out], "y")
        if r is None:
            assert ro is None
        else:
            b64.check_near(ro, s, 2.0 ** -24, b64.HALF[dtype], "residual_out")


@pytest.mark.parametrize("T", [1, 2, 151, 1217, 5000])
@pytest.mark.parametrize("out", [BF16, E4M3])
def test_rows(T, out):
    """From one row to more rows than the grid has CTAs."""
    x, res, w = _rand(T, T, 264).to(BF16), _rand(T + 1, T, 264).to(BF16), _rand(2, 264)
    y, scale, ro = _check(x, res, w, 1.0, out)
    s, ref = b64.add_rmsnorm(x, res, w, 1e-6, 1.0)
    b64.check_near(ro, s, 2.0 ** -24, b64.HALF[BF16], "residual_out")
    if out == E4M3:
        b64.check_quant(y, scale, ref, b64.NORM, "y")
    else:
        b64.check_near(y, ref, b64.NORM, b64.HALF[BF16], "y")


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, E4M3), (F32, E4M3), (F32, F32)])
@pytest.mark.parametrize("off,pad", [(8, 16), (1, 3), (4, 8)])
def test_strided_rows_and_what_lies_between(dtype, out, off, pad):
    """Views into wider buffers, on and off 16-byte boundaries: the same
    values as packed rows, and nothing outside the views is written."""
    T, H = 9, 96
    wide = lambda seed: _rand(seed, T + 1, H + off + pad).to(dtype)  # noqa: E731
    xw, rw, row = wide(1), wide(2), wide(3)
    yw = _rand(4, T + 1, H + off + pad).to(BF16).to(out)
    cut = lambda t: t[:T, off:off + H]  # noqa: E731
    sc = torch.full((T + 2,), -7.0, device=DEV)
    w = _rand(5, H)
    row0, yw0 = row.clone(), yw.clone()
    x, res = cut(xw), cut(rw)
    y, scale, ro = _check(x, res, w, 0.0, out, y=cut(yw), residual_out=cut(row),
                          y_scale=sc[1:T + 1] if out == E4M3 else None)
    p, pscale, pro = _check(x.contiguous(), res.contiguous(), w, 0.0, out)
    s, ref = b64.add_rmsnorm(x, res, w, 1e-6, 0.0)
    b64.check_near(ro, s, 2.0 ** -24, b64.HALF[dtype], "residual_out")
    if out == E4M3:
        b64.check_quant(y.float(), scale, ref, b64.NORM, "y")
        assert sc[0] == -7 and sc[T + 1] == -7
    else:
        b64.check_near(y, ref, b64.NORM, b64.HALF[out], "y")
    assert torch.equal(ro, pro)
    raw = torch.uint8 if out == E4M3 else out
    for now, before in ((row, row0), (yw.view(raw), yw0.view(raw))):
        assert torch.equal(now[T], before[T])
        assert torch.equal(now[:, :off], before[:, :off])
        assert torch.equal(now[:, off + H:], before[:, off + H:])


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, E4M3), (F32, E4M3), (F32, F32)])
@pytest.mark.parametrize("H", [1, 5, 9, 77, 2047, 2050, 2052])
def test_many_rows_of_odd_widths(H, dtype, out):
    """More rows than CTAs, packed rows that start anywhere within 16 bytes."""
    T = 3001
    x, res, w = _rand(H, T, H).to(dtype), _rand(H + 1, T, H).to(dtype), _rand(2, H)
    y, scale, ro = _check(x, res, w, 1.0, out)
    s, ref = b64.add_rmsnorm(x, res, w, 1e-6, 1.0)
    b64.check_near(ro, s, 2.0 ** -24, b64.HALF[dtype], "residual_out")
    if out == E4M3:
        b64.check_quant(y.float(), scale, ref, b64.NORM, "y")
    else:
        b64.check_near(y, ref, b64.NORM, b64.HALF[out], "y")


@pytest.mark.parametrize("offs", [(0, 1, 0, 0), (1, 1, 1, 2), (3, 3, 3, 3), (2, 2, 5, 2), (0, 0, 0, 4)])
@pytest.mark.parametrize("out", [BF16, E4M3])
def test_rows_that_start_unlike_each_other(offs, out):
    """x, the residual, residual_out and y at columns of their own of wider buffers,
    alike or not: the bits of packed copies, nothing else written."""
    T, H = 600, 203
    wide = [_rand(i, T, H + 8).to(BF16) for i in range(3)]
    x, res, row = (b[:, o:o + H] for b, o in zip(wide, offs))
    yw = torch.zeros(T, H + 8, dtype=BF16, device=DEV).to(out)
    y, w = yw[:, offs[3]:offs[3] + H], _rand(9, H)
    row0 = wide[2].clone()
    sc = torch.empty(T, device=DEV) if out == E4M3 else None
    _check(x, res, w, 0.0, out, y=y, residual_out=row, y_scale=sc)
    s, ref = b64.add_rmsnorm(x, res, w, 1e-6, 0.0)
    b64.check_near(row, s, 2.0 ** -24, b64.HALF[BF16], "residual_out")
    if out == E4M3:
        b64.check_quant(y.float(), sc, ref, b64.NORM, "y")
    else:
        b64.check_near(y, ref, b64.NORM, b64.HALF[BF16], "y")
    raw = yw.view(torch.uint8) if out == E4M3 else yw
    for buf, before, o in ((wide[2], row0, offs[2]), (raw, torch.zeros_like(raw), offs[3])):
        assert torch.equal(buf[:, :o], before[:, :o]) and torch.equal(buf[:, o + H:], before[:, o + H:])


@pytest.mark.parametrize("hidden", [2048, 1111])
def test_in_place(hidden):
    """residual_out over residual and y over x: the bits of separate buffers."""
    x, res, w = _rand(1, 40, hidden).to(BF16), _rand(2, 40, hidden).to(BF16), _rand(3, hidden)
    y, _, ro = _check(x, res, w, 0.0, None)
    x2, r2 = x.clone(), res.clone()
    y2, _, ro2 = _check(x2, r2, w, 0.0, None, y=x2, residual_out=r2)
    assert y2.data_ptr() == x2.data_ptr() and ro2.data_ptr() == r2.data_ptr()
    assert bits_equal(y2, y) and bits_equal(ro2, ro)
    x3 = x.clone()                                  # the sum over x, the norm over the residual
    r3 = res.clone()
    y3, _, ro3 = _check(x3, r3, w, 0.0, None, y=r3, residual_out=x3)
    assert bits_equal(y3, y) and bits_equal(ro3, ro)


@pytest.mark.parametrize("hidden", [2048, 77])
def test_zero_and_nan_rows(hidden):
    """Rows of zeros give zeros with the smallest scale; a NaN or an infinity
    stays in its row; values near the type's ends keep their scale."""
    x = _rand(1, 6, hidden).to(BF16)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] *= 1e-15                                    # mean of squares far below eps
    x[4] *= 1e15
    w = _rand(2, hidden).abs() + 0.5
    y, scale, _ = _check(x, None, w, 0.0, E4M3)
    yb, _, _ = _check(x, None, w, 0.0, None)
    assert torch.all(y[0].float() == 0) and scale[0] == 2.0 ** -126 and torch.all(yb[0] == 0)
    for r in (1, 2):
        assert torch.isnan(scale[r]) and torch.all(torch.isnan(y[r].float()))
    assert torch.all(torch.isnan(yb[1])) and torch.isnan(yb[2, 5])
    _, ref = b64.add_rmsnorm(x, None, w, 1e-6, 0.0)
    live = [3, 4, 5]
    b64.check_quant(y[live].float(), scale[live], ref[live], b64.NORM, "y")
    b64.check_near(yb[live], ref[live], b64.NORM, b64.HALF[BF16], "y")


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    y, scale, ro = gdn().gdn_add_rmsnorm(x, _rand(1, 64), residual=x, y_dtype=E4M3)
    assert y.shape == (0, 64) and scale.shape == (0,) and ro.shape == (0, 64)
    o = torch.empty(0, 2, 32, dtype=BF16, device=DEV)
    q, qs = gdn().gdn_gated_rmsnorm_quant(o, o, _rand(1, 32))
    assert q.shape == (0, 2, 32) and qs.shape == (0,)


@pytest.mark.parametrize("hidden", [128, 77])
def test_rows_past_32_bit_offsets(hidden):
    T, step = 3, 2 ** 30 + 64
    buf = torch.empty(step * (T - 1) + 4096, dtype=BF16, device=DEV)
    far = lambda off: buf.as_strided((T, hidden), (step, 1), off)  # noqa: E731
    x, res, w = _rand(1, T, hidden).to(BF16), _rand(2, T, hidden).to(BF16), _rand(3, hidden)
    xf, rf = far(0), far(256)
    xf.copy_(x)
    rf.copy_(res)
    y, _, ro = gdn().gdn_add_rmsnorm(xf, w, residual=rf, y=far(512), residual_out=rf)
    p, _, pro = gdn().gdn_add_rmsnorm(x, w, residual=res)
    torch.cuda.synchronize()
    assert bits_equal(y.contiguous(), p) and bits_equal(ro.contiguous(), pro)


# ------------------------------------------------- the gated norm in 8 bits --

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dv", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hv", [1, 3, 32])
def test_gated_quant(dtype, dv, hv):
    T = 11
    o, zw = _rand(dv, T, hv, dv, scale=0.3).to(dtype), _rand(dv + 1, T, hv * dv + 24).to(dtype)
    w = _rand(3, dv).abs() + 0.5
    for off in (8, 4):                              # on and (bf16) off 16-byte boundaries
        z = zw[:, off:off + hv * dv].unflatten(1, (hv, dv))
        y, scale = gdn().gdn_gated_rmsnorm_quant(o, z, w)
        torch.cuda.synchronize()
        b64.check_quant(y.float().reshape(T, -1), scale,
                        b64.gated_norm(o, z, w, 1e-6).reshape(T, -1), b64.GATED, "y")


@pytest.mark.parametrize("T", [1, 257, 3000])
def test_gated_quant_rows(T):
    """And against the library's own gated norm: one e4m3 step of its bf16 values."""
    hv, dv = 4, 128
    o, z, w = _rand(1, T, hv, dv).to(BF16), _rand(2, T, hv, dv).to(BF16), _rand(3, dv).abs() + 0.5
    guard = torch.zeros(T + 1, hv, dv, dtype=E4M3, device=DEV)
    sg = torch.full((T + 1,), 5.0, device=DEV)
    y, scale = gdn().gdn_gated_rmsnorm_quant(o, z, w, y=guard[:T], y_scale=sg[:T])
    plain = gdn().gdn_gated_rmsnorm(o, z, w)
    torch.cuda.synchronize()
    assert sg[T] == 5.0 and torch.all(guard[T].float() == 0)
    ref = b64.gated_norm(o, z, w, 1e-6).reshape(T, -1)
    b64.check_quant(y.float().reshape(T, -1), scale, ref, b64.GATED, "y")
    got = y.double().reshape(T, -1) * scale.double()[:, None]
    near = plain.double().reshape(T, -1)
    tol = near.abs() * (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -10) + scale.double()[:, None] * 2.0 ** -9
    assert torch.all((got - near).abs() <= tol)


def test_gated_quant_zero_and_nan_tokens():
    hv, dv = 4, 64
    o, z, w = _rand(1, 4, hv, dv).to(BF16), _rand(2, 4, hv, dv).to(BF16), _rand(3, dv)
    o[0] = 0
    z[1] = 0
    o[2, 1, 7] = float("nan")
    y, scale = gdn().gdn_gated_rmsnorm_quant(o, z, w)
    torch.cuda.synchronize()
    for t in (0, 1):
        assert torch.all(y[t].float() == 0) and scale[t] == 2.0 ** -126
    assert torch.isnan(scale[2]) and torch.all(torch.isnan(y[2].float()))
    ref = b64.gated_norm(o[3:], z[3:], w, 1e-6).reshape(1, -1)
    b64.check_quant(y[3:].float().reshape(1, -1), scale[3:], ref, b64.GATED, "y")


def test_other_stream_and_graph():
    """The calls run on the current stream and replay from a graph on new inputs."""
    T, H, hv, dv = 33, 512, 4, 128
    x, res, w = _rand(1, T, H).to(BF16), _rand(2, T, H).to(BF16), _rand(3, H)
    z, w2 = _rand(4, T, hv, dv).to(BF16), _rand(5, dv)
    y, ys = torch.empty(T, H, dtype=E4M3, device=DEV), torch.empty(T, device=DEV)
    ro = torch.empty_like(x)
    q, qs = torch.empty(T, hv, dv, dtype=E4M3, device=DEV), torch.empty(T, device=DEV)

    def both():
        gdn().gdn_add_rmsnorm(x, w, residual=res, y=y, y_scale=ys, residual_out=ro)
        gdn().gdn_gated_rmsnorm_quant(ro.view(T, hv, dv), z, w2, y=q, y_scale=qs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (y.view(torch.uint8), ys, ro, q.view(torch.uint8), qs)]
    b64.check_quant(y.float(), ys, b64.add_rmsnorm(x, res, w, 1e-6, 0.0)[1], b64.NORM, "y")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    x0 = x.clone()
    x.copy_(x0 * 2)
    graph.replay()
    b64.check_quant(y.float(), ys, b64.add_rmsnorm(x, res, w, 1e-6, 0.0)[1], b64.NORM, "replayed y")
    x.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (y.view(torch.uint8), ys, ro, q.view(torch.uint8), qs)):
        assert torch.equal(a, b)
    status_clean()


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, E4M3), (F32, E4M3), (F32, F32)])
@pytest.mark.parametrize("H", [131, 203, 1111, 4095, 8191])
@pytest.mark.parametrize("pad", [0, 6])
def test_what_lies_beside_a_row_stays_out(H, dtype, out, pad):
    """NaNs in other rows and between the rows, which share 16 bytes with a row's ends."""
    T, off = 400, 3 if pad else 0
    xw, rw = (torch.full((T, H + pad), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    x, res, w = xw[:, off:off + H], rw[:, off:off + H], _rand(1, H)
    x.copy_(_rand(2, T, H))
    res.copy_(_rand(3, T, H))
    x[1::3] = float("nan")
    res[0] = float("inf")
    row = torch.full((T, H + pad), float("nan"), dtype=dtype, device=DEV)[:, off:off + H]
    yw = torch.zeros(T, H + pad, device=DEV).to(out)
    y, scale, ro = gdn().gdn_add_rmsnorm(x, w, residual=res, y=yw[:, off:off + H], residual_out=row)
    torch.cuda.synchronize()
    good = torch.ones(T, dtype=torch.bool, device=DEV)
    good[1::3] = False
    good[0] = False
    s, ref = b64.add_rmsnorm(x[good], res[good], w, 1e-6, 0.0)
    b64.check_near(ro[good], s, 2.0 ** -24, b64.HALF[dtype], "residual_out")
    if out == E4M3:
        b64.check_quant(y.float()[good], scale[good], ref, b64.NORM, "y")
    else:
        b64.check_near(y[good], ref, b64.NORM, b64.HALF[out], "y")
    assert torch.all(torch.isnan(y.float()[1::3]))
