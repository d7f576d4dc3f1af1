"""gdn_linear on the GPU against the product in 64 bits: sizes around every
tile edge, odd numbers of channels, both operand types and output types, every
part of the epilogue, strided and in-place outputs, rows behind the last one,
NaNs that stay in their rows and columns, another stream, graph replay."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3


def _padded(v, fill):
    """v with rows on 16-byte boundaries; what lies behind a row is `fill`."""
    n = 16 // v.element_size()
    width = -(-v.shape[1] // n) * n
    wide = torch.full((v.shape[0], width), fill, dtype=F32, device=v.device).to(v.dtype)
    raw = torch.uint8 if v.dtype == E4M3 else v.dtype
    wide.view(raw)[:, :v.shape[1]] = v.view(raw)
    return wide[:, :v.shape[1]]


def _case(seed, T, K, N, dtype, bias=False, residual=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, w, sx, sw = r(T, K), r(N, K) * K ** -0.5, None, None
    if dtype == E4M3:
        (x, sx), (w, sw) = b64.quantise(x), b64.quantise(w)
    else:
        x, w = x.to(dtype), w.to(dtype)
    # NaN behind the rows: it must not be read into the product
    return (_padded(x, float("nan")), _padded(w, float("nan")), sx, sw, r(N) if bias else None,
            r(T, N).to(residual) if residual else None)


def _run(seed, T, K, N, dtype, out=BF16, bias=False, act="none", residual=False, what=""):
    x, w, sx, sw, b, res = _case(seed, T, K, N, dtype, bias, out if residual else None)
    guard = torch.full((T + 1, N), 7.0, dtype=out, device=DEV)
    y = gdn().gdn_linear(x, w, x_scale=sx, weight_scale=sw, bias=b, act=act, residual=res, y=guard[:T])
    torch.cuda.synchronize()
    status_clean()
    assert torch.all(guard[T] == 7.0)
    ref, size = b64.linear(x, w, sx, sw, b, act, res)
    b64.check_linear(y, ref, size, K, dtype == E4M3, f"{what} T={T} K={K} N={N} {dtype}")
    return y


SIZES = [(1, 64, 1), (1, 1, 33), (1, 2048, 128), (2, 8, 129), (15, 100, 127), (16, 128, 256), (17, 192, 64),
         (31, 1000, 300), (32, 256, 128), (33, 320, 100), (64, 512, 512), (65, 65, 65), (127, 63, 200),
         (128, 2048, 384), (129, 129, 129), (200, 4096, 250), (255, 640, 96), (256, 1024, 1024),
         (257, 257, 257), (300, 1003, 331), (511, 96, 700), (512, 2000, 520), (513, 4100, 40),
         (1025, 513, 1030), (2100, 64, 2050), (1, 8192, 4096), (7, 12288, 136), (260, 16, 3100)]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_sizes(T, K, N, dtype):
    _run(T + K + N, T, K, N, dtype, bias=True)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("T,K,N", [(3, 264, 200), (70, 200, 136), (300, 400, 333), (640, 256, 640)])
def test_epilogue(T, K, N, act, out, dtype):
    for bias in (False, True):
        for residual in (False, True):
            _run(T + bias, T, K, N, dtype, out, bias, act, residual, f"{act} {bias} {residual}")


@pytest.mark.parametrize("T", [5, 100, 700])
def test_scales_are_optional(T):
    x, w, sx, sw, _, _ = _case(T, T, 160, 144, E4M3)
    for a, b in ((None, None), (sx, None), (None, sw)):
        y = gdn().gdn_linear(x, w, x_scale=a, weight_scale=b, y_dtype=F32)
        ref, size = b64.linear(x, w, a, b, None, "none", None)
        b64.check_linear(y, ref, size, 160, True)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,N,off,pad", [(9, 120, 3, 2), (9, 128, 64, 64), (300, 200, 8, 16), (700, 333, 1, 1)])
def test_strided_outputs(T, N, off, pad, out):
    """y as columns of a wider buffer, residual as columns of another: the
    bits of packed ones, nothing outside written."""
    K = 136
    x, w, _, _, b, res = _case(N, T, K, N, BF16, True, out)
    wide = torch.full((T + 1, N + off + pad), 3.0, dtype=out, device=DEV)
    rwide = torch.full((T, N + off + pad), float("nan"), dtype=out, device=DEV)
    y, r = wide[:T, off:off + N], rwide[:, off:off + N]
    r.copy_(res)
    gdn().gdn_linear(x, w, bias=b, residual=r, y=y)
    p = gdn().gdn_linear(x, w, bias=b, residual=res, y_dtype=out)
    torch.cuda.synchronize()
    assert bits_equal(y.contiguous(), p)
    ref, size = b64.linear(x, w, None, None, b, "none", res)
    b64.check_linear(p, ref, size, K)
    assert torch.all(wide[T] == 3.0) and torch.all(wide[:, :off] == 3.0) and torch.all(wide[:, off + N:] == 3.0)


@pytest.mark.parametrize("T,N", [(4, 256), (130, 264), (700, 520), (300, 333)])
def test_residual_in_place(T, N):
    x, w, _, _, _, res = _case(T, T, 200, N, BF16, False, BF16)
    want = gdn().gdn_linear(x, w, residual=res)
    y = res.clone()
    got = gdn().gdn_linear(x, w, residual=y, y=y)
    torch.cuda.synchronize()
    assert got.data_ptr() == y.data_ptr() and bits_equal(y, want)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("T,N", [(20, 200), (300, 300), (900, 640)])
def test_nan_stays_in_its_row_and_column(T, N, dtype):
    x, w, sx, sw, b, _ = _case(T, T, 144, N, dtype, True)
    raw = lambda t: t.view(torch.uint8 if dtype == E4M3 else torch.int16)  # noqa: E731
    nan = 0x7F if dtype == E4M3 else 0x7FC0
    clean = gdn().gdn_linear(x, w, x_scale=sx, weight_scale=sw, bias=b)
    raw(x)[T // 2, 100] = nan
    raw(w)[N // 3, 5] = nan
    y = gdn().gdn_linear(x, w, x_scale=sx, weight_scale=sw, bias=b)
    torch.cuda.synchronize()
    assert torch.all(torch.isnan(y[T // 2])) and torch.all(torch.isnan(y[:, N // 3]))
    keep_t, keep_n = torch.arange(T, device=DEV) != T // 2, torch.arange(N, device=DEV) != N // 3
    assert bits_equal(y[keep_t][:, keep_n], clean[keep_t][:, keep_n])


@pytest.mark.parametrize("T,K,N", [(1, 2048, 512), (256, 4096, 2048), (3000, 512, 700)])
def test_same_bits_again(T, K, N):
    x, w, _, _, _, res = _case(1, T, K, N, BF16, False, BF16)
    first = gdn().gdn_linear(x, w, residual=res)
    for _ in range(3):
        assert bits_equal(gdn().gdn_linear(x, w, residual=res), first)


def test_no_rows_and_wide_fp32_rows():
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    w = torch.zeros(32, 64, dtype=BF16, device=DEV)
    assert gdn().gdn_linear(x, w).shape == (0, 32)


@pytest.mark.parametrize("T", [8, 256, 1500])
def test_other_streams_at_once_and_graph(T):
    """Two calls on two streams at once, and a captured call replayed on new inputs."""
    K, N = 512, 640
    a = _case(1, T, K, N, BF16, True, BF16)
    b = _case(2, T, K, N, E4M3, False, BF16)
    ya, yb = torch.empty(T, N, dtype=BF16, device=DEV), torch.empty(T, N, dtype=BF16, device=DEV)
    go = lambda c, y: gdn().gdn_linear(c[0], c[1], x_scale=c[2], weight_scale=c[3], bias=c[4],  # noqa: E731
                                       residual=c[5], y=y)
    wa, wb = go(a, ya.clone()), go(b, yb.clone())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            go(a, ya)
        with torch.cuda.stream(s2):
            go(b, yb)
    torch.cuda.synchronize()
    assert bits_equal(ya, wa) and bits_equal(yb, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(a, ya)
        go(b, yb)
    a[0].copy_(-a[0])
    graph.replay()
    torch.cuda.synchronize()
    ref, size = b64.linear(a[0], a[1], None, None, a[4], "none", a[5])
    b64.check_linear(ya, ref, size, K)
    assert bits_equal(yb, wb)
    status_clean()


@pytest.mark.parametrize("T,N", [(2, 96), (2, 90), (130, 96)])
def test_rows_past_32_bit_offsets(T, N):
    """Rows of x, y and the residual that lie more than 2^31 elements behind the first."""
    K = 128
    x, w, _, _, _, res = _case(T, T, K, N, BF16, False, BF16)
    step = 2 ** 31 // (T - 1) // 64 * 64 + 64
    buf = torch.empty(step * (T - 1) + 4096, dtype=BF16, device=DEV)
    far = lambda off, n: buf.as_strided((T, n), (step, 1), off)  # noqa: E731
    xf, rf, yf = far(0, K), far(256, N), far(512, N)
    xf.copy_(x)
    rf.copy_(res)
    y = gdn().gdn_linear(xf, w, residual=rf, y=yf)
    p = gdn().gdn_linear(x, w, residual=res)
    torch.cuda.synchronize()
    assert bits_equal(y.contiguous(), p)


def test_first_call_of_a_size_inside_a_capture():
    """What a call asks the device once (shared memory, clusters) may be asked during a capture."""
    K, N = 640, 896
    a, b = _case(1, 40, K, N, E4M3), _case(2, 600, K, N, E4M3)
    ya, yb = (torch.empty(t, N, dtype=F32, device=DEV) for t in (40, 600))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, y in ((a, ya), (b, yb)):
            gdn().gdn_linear(c[0], c[1], x_scale=c[2], weight_scale=c[3], y=y)
    graph.replay()
    torch.cuda.synchronize()
    for c, y in ((a, ya), (b, yb)):
        ref, size = b64.linear(c[0], c[1], c[2], c[3], None, "none", None)
        b64.check_linear(y, ref, size, K, True)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N", [1331, 1330, 1332, 1336, 1344])
@pytest.mark.parametrize("yoff,roff", [(0, 0), (1, 1), (1, 0), (2, 6), (4, 4), (8, 8)])
def test_many_tokens_rows_that_start_anywhere(N, yoff, roff, out):
    """y and the residual as columns of wider buffers, at every alignment of the
    rows (alike or not), odd and even strides: 64 bits, and nothing else written."""
    T, K = 2030, 72
    x, w, _, _, b, res = _case(N, T, K, N, BF16, True, out)
    for pad in (0, 1, 2, 8):
        if yoff == 0 and pad == 0:
            continue                                   # packed rows are test_sizes'
        wide = torch.full((T, N + yoff + pad), 3.0, dtype=out, device=DEV)
        rwide = torch.full((T, N + roff + pad), float("nan"), dtype=out, device=DEV)
        y, r = wide[:, yoff:yoff + N], rwide[:, roff:roff + N]
        r.copy_(res)
        gdn().gdn_linear(x, w, bias=b, act="silu", residual=r, y=y)
        torch.cuda.synchronize()
        ref, size = b64.linear(x, w, None, None, b, "silu", res)
        b64.check_linear(y, ref, size, K, what=f"pad {pad}")
        assert torch.all(wide[:, :yoff] == 3.0) and torch.all(wide[:, yoff + N:] == 3.0)
    plain = gdn().gdn_linear(x, w, bias=b, act="silu", y_dtype=out)
    again = torch.full((T, N + yoff + 1), 3.0, dtype=out, device=DEV)
    gdn().gdn_linear(x, w, bias=b, act="silu", y=again[:, yoff:yoff + N])
    torch.cuda.synchronize()
    assert bits_equal(again[:, yoff:yoff + N].contiguous(), plain)
    status_clean()


@pytest.mark.parametrize("N", [1331, 1330, 1332, 1344])
def test_many_tokens_residual_in_place(N):
    T, K = 5000, 40
    x, w, _, _, _, res = _case(N, T, K, N, BF16, False, BF16)
    want = gdn().gdn_linear(x, w, residual=res)
    y = res.clone()
    gdn().gdn_linear(x, w, residual=y, y=y)
    torch.cuda.synchronize()
    assert bits_equal(y, want)
    ref, size = b64.linear(x, w, None, None, None, "none", res)
    b64.check_linear(want, ref, size, K)


@pytest.mark.parametrize("T,K,N,dtype", [(20000, 64, 512, BF16), (9000, 300, 2050, E4M3), (1300, 136, 8193, BF16)])
def test_many_tiles(T, K, N, dtype):
    """Several tiles for every pair, the last ones narrower, with every part of the epilogue."""
    for act, residual in (("none", True), ("gelu", False)):
        _run(T, T, K, N, dtype, BF16, True, act, residual)


@pytest.mark.parametrize("N", [33, 35, 63, 65, 95, 97, 127, 129, 191, 223, 255, 257, 287, 321, 1025, 1055, 1057, 1087])
def test_many_tokens_odd_widths(N):
    """Packed rows of an odd width start on 2 and on 4 bytes in turn; their ends fall
    anywhere in the pieces that a warp writes."""
    for act, residual in (("none", False), ("silu", True)):
        y = _run(N, 2100, 40, N, BF16, BF16, True, act, residual)
    x, w, _, _, b, res = _case(N, 2100, 40, N, BF16, True, BF16)
    buf = res.clone()
    gdn().gdn_linear(x, w, bias=b, act="silu", residual=buf, y=buf)
    torch.cuda.synchronize()
    assert bits_equal(buf, y)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [5, 100, 2100])
def test_activations_far_out(T, act, out):
    """Values of any size in any channel leave the channels beside them alone."""
    K, far = 64, [1e30, -1e30, 3e38, -3e38, 1e4, -1e4, 200.0, -200.0, 90.0, -90.0, 45.0, -45.0, 20.0, -20.0,
                  float("inf"), float("-inf"), float("nan")]
    x, w, _, _, b, _ = _case(T, T, K, 4 * len(far), BF16, True)
    for i, v in enumerate(far):                          # far, near, near, far
        b[4 * i] = b[4 * i + 3] = v
    y = gdn().gdn_linear(x, w, bias=b, act=act, y_dtype=out)
    torch.cuda.synchronize()
    status_clean()
    finite = torch.isfinite(b)
    ref, size = b64.linear(x, w[finite], None, None, b[finite], act, None)
    b64.check_linear(y[:, finite], ref, size, K)
    near = b.abs() < 10
    ref, size = b64.linear(x, w[near], None, None, b[near], act, None)
    b64.check_linear(y[:, near], ref, size, K)
    assert torch.all(y[:, b == float("inf")] == float("inf"))
    assert torch.all(torch.isnan(y[:, torch.isnan(b)]))
    if act == "silu":                                    # its limit
        assert torch.all(y[:, b == float("-inf")].abs() <= 1e-17)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N", [1, 2, 33, 131, 333, 1004])
@pytest.mark.parametrize("T", [1, 33, 100, 128])
def test_few_tokens_odd_widths(T, N, out):
    """Rows that are no vectors of 8 channels, with every part of the epilogue, k cut
    over a cluster or not, and the residual in place."""
    for K in (40, 1500):
        y = _run(T + N, T, K, N, BF16, out, True, "gelu", True)
        x, w, _, _, b, res = _case(T + N, T, K, N, BF16, True, out)
        for off in (0, 1, 2):                              # columns of a wider buffer
            wide = torch.full((T, N + off + 5), 3.0, dtype=out, device=DEV)
            wide[:, off:off + N] = res
            cut = wide[:, off:off + N]
            gdn().gdn_linear(x, w, bias=b, act="gelu", residual=cut, y=cut)
            torch.cuda.synchronize()
            assert bits_equal(cut.contiguous(), y)
            assert torch.all(wide[:, :off] == 3.0) and torch.all(wide[:, off + N:] == 3.0)
