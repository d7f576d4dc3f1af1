"""The products grouped by expert and the product with block scales on the GPU
against 64 bits: sizes around every tile edge, experts of any number of rows,
gathered rows, both operand and output types, strides, what is left alone."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3
NAN = float("nan")


def _operands(seed, n_x, E, K, N, dtype, extra=0):
    """x, w, sx, sw; what lies between the rows is NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x, w = torch.randn(n_x, K, generator=g, device=DEV), torch.randn(E, N, K, generator=g, device=DEV) * K ** -0.5
    sx = sw = None
    if dtype == E4M3:
        # blocks of different sizes, so that a scale of another block shows
        x = x * torch.exp2(torch.randint(-3, 4, (n_x, m64.up(K, 128) // 128), generator=g, device=DEV).float()).repeat_interleave(128, 1)[:, :K]
        (x, sx), (w, sw) = m64.quantise_blocks(x, 1), m64.quantise_blocks(w, 128)
        sw = sw.contiguous()
    else:
        x, w = x.to(dtype), w.to(dtype)
    return m64.padded(x, NAN, extra), m64.padded(w, NAN, extra), sx, sw


def _offsets(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return o.to(DEV)


def _run(seed, counts, K, N, dtype, out=BF16, gather=None, behind=0, what="", x_case=None):
    """gather: None, or the number of rows of x that the rows are taken from."""
    E, R = len(counts), sum(counts) + behind
    x, w, sx, sw = _operands(seed, R if gather is None else gather, E, K, N, dtype) if x_case is None else x_case
    offsets, rows = _offsets(counts), None
    if gather is not None:
        g = torch.Generator(device=DEV).manual_seed(seed + 1)
        rows = torch.randint(0, gather, (R,), generator=g, device=DEV, dtype=torch.int32)
    guard = torch.full((R + 1, N), 7.0, dtype=out, device=DEV)
    y = gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw, y=guard[:R])
    torch.cuda.synchronize()
    status_clean()
    assert torch.all(guard[sum(counts):] == 7.0)
    ref, size = m64.grouped(x, w, offsets, rows, sx, sw)
    m64.check_product(y[:sum(counts)], ref, size, K, dtype == E4M3, f"{what} {counts[:8]} K={K} N={N} {dtype} {out}")
    return y


def _block(seed, T, K, N, out=BF16):
    x, w, sx, sw = _operands(seed, T, 1, K, N, E4M3)
    guard = torch.full((T + 1, N), 7.0, dtype=out, device=DEV)
    y = gdn().gdn_linear_block(x, w[0], sx, sw[0], y=guard[:T])
    torch.cuda.synchronize()
    status_clean()
    assert torch.all(guard[T] == 7.0)
    m64.check_product(y, *m64.product(x, w[0], sx, sw[0]), K, True, f"T={T} K={K} N={N}")
    return y


SIZES = [(1, 64, 1), (1, 1, 33), (1, 2048, 128), (2, 8, 129), (15, 100, 127), (16, 128, 256), (17, 192, 64),
         (31, 1000, 300), (32, 256, 128), (33, 320, 100), (64, 512, 512), (65, 65, 65), (127, 63, 200),
         (128, 2048, 384), (129, 129, 129), (200, 4096, 250), (255, 640, 96), (256, 1024, 1024),
         (257, 257, 257), (300, 1003, 331), (511, 96, 700), (512, 2000, 520), (513, 4100, 40),
         (1025, 513, 1030), (2100, 64, 2050), (1, 8192, 4096), (7, 12288, 136), (260, 16, 3100), (3000, 2048, 300)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_block_sizes(T, K, N, out):
    _block(T + K + N, T, K, N, out)


COUNTS = {"one": [1], "ones": [1] * 10, "none": [0, 0, 0], "ends": [0, 5, 0, 0, 40, 0], "few": [3, 0, 7, 1, 2, 9, 16, 17, 31, 33],
          "edges": [127, 128, 129, 1, 0, 255, 256, 257, 64, 65], "skew": [900, 1, 0, 2, 3], "many": [5] * 300 + [0] * 20 + [11],
          "big": [700, 0, 1300, 40], "1024": [2, 0, 1, 1] * 256}


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("name", COUNTS)
def test_counts(name, dtype):
    counts = COUNTS[name]
    for K, N, out in ((200, 136, BF16), (384, 77, F32)):
        for gather in (None, 97):
            _run(len(counts), counts, K, N, dtype, out, gather, what=name)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("K,N", [(1, 1), (16, 8), (63, 64), (64, 65), (127, 127), (128, 128), (129, 129), (500, 256), (1000, 257),
                                 (2048, 1024), (513, 511), (4104, 130), (130, 4100)])
def test_sizes(K, N, dtype):
    for gather in (None, 50):
        _run(K + N, [3, 0, 40, 130, 300, 1], K, N, dtype, gather=gather)
        _run(K + N, [2, 9, 1, 0, 5], K, N, dtype, F32, gather=gather)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("N", [1400, 1411, 1664, 1665, 2048, 2178])
def test_many_rows_an_expert(N, dtype, out):
    """Tiles on pairs of CTAs: channels that end in either half of a tile, k of one block and of many, ragged rows."""
    for counts, K in (([300, 0, 513, 700, 129, 1, 128, 255], 200), ([1, 2000, 0, 0, 31], 64), ([900, 900], 1160)):
        _run(N, counts, K, N, dtype, out)
        _run(N, counts, K, N, dtype, out, gather=77)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("off,pad", [(0, 8), (8, 0), (1, 3), (2, 2)])
def test_many_rows_an_expert_strided(off, pad, dtype):
    counts, K, N = [300, 0, 513, 700, 129, 1, 128, 255], 144, 1672
    R = sum(counts)
    x, w, sx, sw = _operands(N, 90, len(counts), K, N, dtype)
    rows = torch.randint(-1, 90, (R,), device=DEV, dtype=torch.int32)
    want = gdn().gdn_grouped_linear(x, w, _offsets(counts), rows=rows, x_scale=sx, weight_scale=sw)
    ref, size = m64.grouped(x, w, _offsets(counts), rows, sx, sw)
    m64.check_product(want, ref, size, K, dtype == E4M3)
    assert torch.all(want[rows < 0] == 0)
    wide = torch.full((R + 1, N + off + pad), 3.0, dtype=BF16, device=DEV)
    gdn().gdn_grouped_linear(x, w, _offsets(counts), rows=rows, x_scale=sx, weight_scale=sw, y=wide[:R, off:off + N])
    torch.cuda.synchronize()
    status_clean()
    assert bits_equal(wide[:R, off:off + N].contiguous(), want)
    assert torch.all(wide[R] == 3.0) and torch.all(wide[:, :off] == 3.0) and torch.all(wide[:, off + N:] == 3.0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("counts", [[5, 0, 3], [200, 0, 500]])
def test_rows_behind_the_last_and_bad_rows(counts, dtype):
    _run(3, counts, 160, 72, dtype, behind=9)
    _run(3, counts, 160, 72, dtype, behind=300, gather=40)
    R, n_x, K, N = sum(counts), 20, 160, 72
    x, w, sx, sw = _operands(4, n_x, len(counts), K, N, dtype)
    w.view(torch.uint8 if dtype == E4M3 else torch.int16)[2] = 0x7F if dtype == E4M3 else 0x7FC0     # NaN weights
    offsets = _offsets(counts)
    rows = torch.randint(0, n_x, (R,), device=DEV, dtype=torch.int32)
    rows[1], rows[R - 2] = -1, -2 ** 31
    y = gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw)
    torch.cuda.synchronize()
    status_clean()
    assert torch.all(y[1] == 0) and torch.all(y[R - 2] == 0) and torch.all(torch.isnan(y[R - 1]))
    rows[0], rows[R - 1] = n_x, 2 ** 31 - 1
    z = gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw)
    torch.cuda.synchronize()
    assert gdn().gdn_get_device_status(clear=True) == gdn().DEVSTAT_BAD_INDEX
    assert torch.all(z[0] == 0) and torch.all(z[R - 1] == 0) and bits_equal(z[1:counts[0]], y[1:counts[0]])


@pytest.mark.parametrize("R", [40, 2000])
@pytest.mark.parametrize("bad", [[0, 5, 3, 30], [0, 10, 20, 2001], [-1, 5, 6, 7], [0, -3, 20, 30]])
def test_bad_offsets_write_nothing(bad, R):
    x, w, _, _ = _operands(1, R, 3, 64, 96, BF16)
    y = torch.full((R, 96), 7.0, dtype=BF16, device=DEV)
    gdn().gdn_grouped_linear(x, w, torch.tensor(bad, dtype=torch.int32, device=DEV), y=y)
    torch.cuda.synchronize()
    assert gdn().gdn_get_device_status(clear=True) == gdn().DEVSTAT_BAD_SEQLEN
    assert torch.all(y == 7.0)


def test_first_expert_need_not_start_at_zero():
    """Rows in front of offsets[0] are left as they were too."""
    for R, offs in ((40, [6, 6, 30, 33]), (2000, [130, 700, 700, 1900])):
        x, w, _, _ = _operands(1, R, 3, 64, 96, BF16)
        y = torch.full((R, 96), 7.0, dtype=BF16, device=DEV)
        offsets = torch.tensor(offs, dtype=torch.int32, device=DEV)
        gdn().gdn_grouped_linear(x, w, offsets, y=y)
        torch.cuda.synchronize()
        status_clean()
        ref, size = m64.grouped(x, w, offsets, None)
        m64.check_product(y[offs[0]:offs[-1]], ref[offs[0]:], size[offs[0]:], 64, False)
        assert torch.all(y[:offs[0]] == 7.0) and torch.all(y[offs[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("counts", [[4, 9, 0, 1], [300, 0, 513, 20]])
@pytest.mark.parametrize("N", [128, 130, 131, 256, 264])
def test_strided_outputs_and_operands(counts, N, out, dtype):
    K, R = 136, sum(counts)
    x, w, sx, sw = _operands(N, R, len(counts), K, N, dtype)
    offsets = _offsets(counts)
    want = gdn().gdn_grouped_linear(x, w, offsets, x_scale=sx, weight_scale=sw, y_dtype=out)
    xp, wp, _, _ = _operands(N, R, len(counts), K, N, dtype, extra=3)
    raw = torch.uint8 if dtype == E4M3 else dtype
    far = torch.full((len(counts), N + 2, wp.stride(1)), NAN, device=DEV).to(dtype)       # experts apart
    far.view(raw)[:, :N, :K] = w.view(raw)
    for xx, ww in ((xp, wp), (x, far[:, :N, :K])):
        for off, pad in ((0, 0), (1, 2), (8, 8), (3, 0), (2, 6)):
            wide = torch.full((R + 1, N + off + pad), 3.0, dtype=out, device=DEV)
            y = wide[:R, off:off + N]
            gdn().gdn_grouped_linear(xx, ww, offsets, x_scale=sx, weight_scale=sw, y=y)
            torch.cuda.synchronize()
            ref, size = m64.grouped(x, w, offsets, None, sx, sw)
            m64.check_product(y, ref, size, K, dtype == E4M3)
            assert bits_equal(y.contiguous(), want)
            assert torch.all(wide[R] == 3.0) and torch.all(wide[:, :off] == 3.0) and torch.all(wide[:, off + N:] == 3.0)
    status_clean()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("counts", [[20, 11], [300, 500]])
def test_nan_stays_in_its_row_and_channel(counts, dtype):
    K, N, R = 144, 200, sum(counts)
    x, w, sx, sw = _operands(2, R, 2, K, N, dtype)
    offsets = _offsets(counts)
    go = lambda: gdn().gdn_grouped_linear(x, w, offsets, x_scale=sx, weight_scale=sw)  # noqa: E731
    clean = go()
    raw = lambda t: t.view(torch.uint8 if dtype == E4M3 else torch.int16)  # noqa: E731
    nan = 0x7F if dtype == E4M3 else 0x7FC0
    raw(x)[3, 100] = nan
    raw(w)[1, 70, 5] = nan
    y = go()
    torch.cuda.synchronize()
    a = counts[0]
    assert torch.all(torch.isnan(y[3])) and torch.all(torch.isnan(y[a:, 70]))
    keep = torch.arange(R, device=DEV) != 3
    assert bits_equal(y[:a][keep[:a]], clean[:a][keep[:a]])
    chan = torch.arange(N, device=DEV) != 70
    assert bits_equal(y[a:][:, chan], clean[a:][:, chan])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("total,K,N", [(10, 2048, 512), (400, 512, 640), (5000, 256, 300)])
def test_same_bits_streams_and_graph(total, K, N, dtype):
    """The same bits again and on two streams at once; a captured call on other rows, offsets and inputs."""
    E, n_x = 20, 333
    g = torch.Generator().manual_seed(total)

    def offs():
        return torch.cat([torch.zeros(1), torch.sort(torch.randint(0, total + 1, (E - 1,), generator=g)).values,
                          torch.tensor([total])]).to(torch.int32).to(DEV)
    x, w, sx, sw = _operands(total, n_x, E, K, N, dtype)
    offsets, rows = offs(), torch.randint(0, n_x, (total,), generator=g).to(torch.int32).to(DEV)
    go = lambda y: gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw, y=y)  # noqa: E731
    new = lambda: torch.empty(total, N, dtype=BF16, device=DEV)  # noqa: E731
    first = go(new())
    for _ in range(3):
        assert bits_equal(go(new()), first)
    ya, yb = new(), new()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for s, y in ((s1, ya), (s2, yb)):
            with torch.cuda.stream(s):
                go(y)
    torch.cuda.synchronize()
    assert bits_equal(ya, first) and bits_equal(yb, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(ya)
        go(yb)
    offsets.copy_(offs())
    rows.copy_(torch.randint(0, n_x, (total,), generator=g).to(torch.int32))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    status_clean()
    m64.check_product(ya, *m64.grouped(x, w, offsets, rows, sx, sw), K, dtype == E4M3)
    assert bits_equal(ya, yb)


def test_a_row_does_not_depend_on_the_others():
    """The same row among other ones, in a call of the same sizes."""
    K, N, n_x = 700, 200, 64
    for dtype in (BF16, E4M3):
        for R in (40, 1500):
            x, w, sx, sw = _operands(R, n_x, 3, K, N, dtype)
            rows = torch.randint(0, n_x, (R,), device=DEV, dtype=torch.int32)
            a = gdn().gdn_grouped_linear(x, w, _offsets([R - 30, 10, 20]), rows=rows, x_scale=sx, weight_scale=sw)
            other = rows.clone()
            other[:R - 30] = -1
            other[-3:] = 5
            b = gdn().gdn_grouped_linear(x, w, _offsets([R - 30, 10, 20]), rows=other, x_scale=sx, weight_scale=sw)
            torch.cuda.synchronize()
            assert bits_equal(a[R - 30:-3], b[R - 30:-3])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_no_expert_has_rows(dtype):
    _run(5, [0, 0, 0], 160, 72, dtype, behind=5)
    _run(5, [0, 0, 0], 160, 72, dtype, behind=700, gather=9)


def test_no_rows():
    x, w, _, _ = _operands(1, 8, 2, 64, 32, BF16)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    assert gdn().gdn_grouped_linear(x, w, _offsets([0, 0]), rows=empty).shape == (0, 32)
    assert gdn().gdn_grouped_linear(x[:0], w, _offsets([0, 0])).shape == (0, 32)
    q, s = m64.quantise_blocks(torch.ones(32, 64, device=DEV), 128)
    assert gdn().gdn_linear_block(q[:0], q.contiguous(), torch.empty(0, 1, device=DEV), s).shape == (0, 32)


@pytest.mark.parametrize("T", [2, 200])
def test_rows_past_32_bit_offsets(T):
    """Rows of x, w and y that lie more than 2^31 elements behind the first."""
    K, N = 128, 96
    x, w, _, _ = _operands(T, T, 2, K, N, BF16)
    counts = [T // 2, T - T // 2]
    step = 2 ** 31 // (T - 1) // 64 * 64 + 64
    buf = torch.empty(step * (T - 1) + 4096, dtype=BF16, device=DEV)
    xf, yf = buf.as_strided((T, K), (step, 1), 0), buf.as_strided((T, N), (step, 1), 256)
    wbuf = torch.empty(2 ** 31 + N * K, dtype=BF16, device=DEV)
    wf = wbuf.as_strided((2, N, K), (2 ** 31, K, 1), 0)
    xf.copy_(x)
    wf.copy_(w)
    y = gdn().gdn_grouped_linear(xf, wf, _offsets(counts), y=yf)
    p = gdn().gdn_grouped_linear(x, w, _offsets(counts))
    torch.cuda.synchronize()
    m64.check_product(p, *m64.grouped(x, w, _offsets(counts), None), K, False)
    assert bits_equal(y.contiguous(), p)


@pytest.mark.parametrize("T,k,E,K,N,dtype", [(2100, 8, 64, 512, 700, E4M3), (1500, 4, 16, 300, 1024, BF16), (256, 10, 512, 256, 256, E4M3),
                                             (20000, 2, 8, 128, 264, E4M3)])
def test_many_tiles(T, k, E, K, N, dtype):
    g = torch.Generator().manual_seed(T)
    counts = torch.bincount(torch.randint(0, E, (T * k,), generator=g), minlength=E).tolist()
    _run(T, counts, K, N, dtype, gather=T)
    _run(T, counts, K, N, dtype, F32)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("N", [700, 701, 704, 1022, 129])
def test_about_a_hundred_rows_an_expert(N, dtype, out):
    """Tiles of up to 128 rows: full, ragged and nearly empty ones, rows of y on 16 bytes, on words and on neither."""
    counts = [128, 97, 33, 128, 1, 0, 129, 250, 64, 100, 127, 5]
    for K in (300, 1152):
        for gather in (None, 77):
            _run(N + K, counts, K, N, dtype, out, gather)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("N,off,pad", [(704, 8, 8), (704, 1, 3), (702, 2, 2), (701, 0, 3)])
def test_about_a_hundred_rows_strided_and_left_out(N, off, pad, dtype, out):
    counts, K = [128, 97, 33, 128, 1, 0, 129, 250, 64, 100, 127, 5], 520
    R = sum(counts)
    x, w, sx, sw = _operands(N + off, 90, len(counts), K, N, dtype)
    rows = torch.randint(-1, 90, (R,), device=DEV, dtype=torch.int32)
    rows[::37] = -1
    go = lambda r, y=None: gdn().gdn_grouped_linear(x, w, _offsets(counts), rows=r, x_scale=sx, weight_scale=sw, y_dtype=out, y=y)  # noqa: E731
    want = go(rows.clamp_min(0))
    want[rows < 0] = 0
    wide = torch.full((R + 1, off + N + pad), 9.0, dtype=out, device=DEV)
    go(rows, wide[:R, off:off + N])
    torch.cuda.synchronize()
    status_clean()
    assert bits_equal(wide[:R, off:off + N].contiguous(), want)
    assert torch.all(wide[:R, :off] == 9.0) and torch.all(wide[:R, off + N:] == 9.0) and torch.all(wide[R] == 9.0)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,K,N", [(1, 4096, 2048), (16, 7168, 512), (5, 16384, 256), (1, 1024, 1), (3, 1025, 130), (70, 5800, 300),
                                   (40, 3333, 129), (128, 9000, 640), (150, 2100, 1000), (300, 6700, 129), (512, 16384, 256),
                                   (97, 12289, 8), (64, 4096, 2048), (1000, 8192, 264)])
def test_k_in_parts(T, K, N, out):
    """Few tiles and many blocks: clusters share a tile's blocks, in parts that start anywhere; the same bits again,
    on two streams and in a graph."""
    y = _block(T + K, T, K, N, out)
    x, w, sx, sw = _operands(T + K, T, 1, K, N, E4M3)
    go = lambda t: gdn().gdn_linear_block(x, w[0], sx, sw[0], y=t)  # noqa: E731
    ys = [torch.zeros_like(y) for _ in range(3)]
    torch.cuda.synchronize()
    for t, s in zip(ys, [torch.cuda.Stream(), torch.cuda.Stream()]):
        with torch.cuda.stream(s):
            for _ in range(3):
                go(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(ys[2])
    ys[2].zero_()
    graph.replay()
    torch.cuda.synchronize()
    status_clean()
    assert all(bits_equal(t, y) for t in ys)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("counts", [[1, 0, 0, 1, 0, 2], [0, 0, 0], [20, 20], [3], [0, 40, 0, 0, 0], [120, 0, 9], [1] * 9])
def test_few_rows_and_k_in_parts(counts, dtype, out):
    """Clusters that share a tile's blocks, more of them than there are tiles; rows left out and behind the last."""
    for K, N in ((2048, 256), (1100, 129), (5000, 250)):
        for gather in (None, 11):
            _run(K + N, counts, K, N, dtype, out, gather, behind=3 if sum(counts) else 7)
    K, N, R = 3000, 264, max(1, sum(counts))
    x, w, sx, sw = _operands(3, 5, len(counts), K, N, dtype)
    rows = (torch.arange(R, device=DEV, dtype=torch.int32) % 6 - 1).contiguous()
    go = lambda r: gdn().gdn_grouped_linear(x, w, _offsets(counts), rows=r, x_scale=sx, weight_scale=sw,  # noqa: E731
                                            y=torch.full((R, N), 5.0, dtype=out, device=DEV))
    got, want = go(rows), go(rows.clamp_min(0))
    want[:sum(counts)][rows[:sum(counts)] < 0] = 0
    torch.cuda.synchronize()
    status_clean()
    assert bits_equal(got, want)
