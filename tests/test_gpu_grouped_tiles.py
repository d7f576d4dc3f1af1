"""Every kernel that a grouped or block-scaled product may take, by its tile and by the
parts that k is cut into: which one a call gets is otherwise an estimate's choice.  Both
operand types, rows gathered and in place, either output, rows of y on 16 bytes and off."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3
NAN = float("nan")
KERNELS = [(rows, cut) for rows in (16, 32, 64, 128) for cut in range(4)] + [(256, 0)]


@pytest.fixture(params=KERNELS, ids=lambda k: f"{k[0]}rows{1 << k[1]}parts")
def kernel(request):
    gdn().gdn_debug_set_grouped_tile(*request.param)
    yield request.param
    gdn().gdn_debug_set_grouped_tile()


def _operands(seed, n_x, E, K, N, dtype):
    """x, w, sx, sw; what lies between the rows is NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x, w = torch.randn(n_x, K, generator=g, device=DEV), torch.randn(E, N, K, generator=g, device=DEV) * K ** -0.5
    sx = sw = None
    if dtype == E4M3:
        # blocks of different sizes, so that a scale of another block shows
        kb = m64.up(K, 128) // 128
        x = x * torch.exp2(torch.randint(-3, 4, (n_x, kb), generator=g, device=DEV).float()).repeat_interleave(128, 1)[:, :K]
        (x, sx), (w, sw) = m64.quantise_blocks(x, 1), m64.quantise_blocks(w, 128)
        sw = sw.contiguous()
    else:
        x, w = x.to(dtype), w.to(dtype)
    return m64.padded(x, NAN), m64.padded(w, NAN), sx, sw


def _least(cut, dtype):
    """The least n_in with a block for each part, and a value of the last."""
    return (1 << cut) * (128 if dtype == E4M3 else 64) - 1


def _run(counts, K, N, dtype, out, gather, off=0):
    E, R, behind = len(counts), sum(counts), 5
    n_x = 61 if gather else R + behind
    x, w, sx, sw = _operands(K + N + R, n_x, E, K, N, dtype)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    rows = None
    if gather:
        rows = torch.randint(0, n_x, (R + behind,), device=DEV, dtype=torch.int32, generator=torch.Generator(device=DEV).manual_seed(R))
        rows[::11] = -1
    wide = torch.full((R + behind + 1, off + N + off), 7.0, dtype=out, device=DEV)
    y = wide[:R + behind, off:off + N]
    go = lambda t: gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw, y=t)  # noqa: E731
    go(y)
    torch.cuda.synchronize()
    status_clean()
    ref, size = m64.grouped(x, w, offsets, rows, sx, sw)
    m64.check_product(y[:R], ref, size, K, dtype == E4M3, f"{counts[:8]} K={K} N={N} {dtype} {out} {gather}")
    assert torch.all(wide[R:] == 7.0) and torch.all(wide[:, :off] == 7.0) and torch.all(wide[:, off + N:] == 7.0)
    if gather:
        assert torch.all(y[:R][rows[:R] < 0] == 0)
    again = torch.full_like(wide, 7.0)
    go(again[:R + behind, off:off + N])
    torch.cuda.synchronize()
    assert bits_equal(again, wide)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_every_kernel(kernel, dtype, gather):
    cut = kernel[1]
    counts = [5, 0, 33, 130, 1, 64, 257]
    # a block a part, parts that start off and on multiples of four blocks
    for K in (_least(cut, dtype), 1100, 3584, 3333):
        for out in (BF16, F32):
            _run(counts, K, 264, dtype, out, gather)
            _run(counts, K, 129, dtype, out, gather)
    _run(counts, 1152, 264, dtype, BF16, gather, off=1)
    _run(counts, 1152, 262, dtype, BF16, gather, off=2)
    _run([1], 1152, 1, dtype, BF16, gather)
    _run([0, 300, 0], 1152, 72, dtype, F32, gather)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_more_tiles_than_the_device_holds(kernel, dtype, gather):
    """Several tiles for a CTA where k is whole, several waves of clusters where it is not."""
    _run([70, 128, 0, 3, 255] * 12 + [1000], 1030, 520, dtype, BF16, gather)


@pytest.mark.parametrize("T", [1, 31, 200])
def test_dense(kernel, T):
    for K, N, out in ((_least(kernel[1], E4M3), 300, BF16), (2100, 1000, F32), (4096, 131, BF16)):
        x, w, sx, sw = _operands(T + K, T, 1, K, N, E4M3)
        guard = torch.full((T + 1, N), 7.0, dtype=out, device=DEV)
        y = gdn().gdn_linear_block(x, w[0], sx, sw[0], y=guard[:T])
        torch.cuda.synchronize()
        status_clean()
        m64.check_product(y, *m64.product(x, w[0], sx, sw[0]), K, True, f"T={T} K={K} N={N}")
        assert torch.all(guard[T] == 7.0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_fewer_blocks_than_parts(kernel, dtype):
    rows, cut = kernel
    if cut == 0:
        return
    x, w, sx, sw = _operands(1, 40, 2, _least(cut, dtype) // 2, 72, dtype)
    offsets = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    with pytest.raises(gdn().GdnError, match="UNSUPPORTED"):
        gdn().gdn_grouped_linear(x, w, offsets, x_scale=sx, weight_scale=sw)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_streams_and_graph(kernel, dtype):
    """Two streams at once, and a captured call on other rows and offsets."""
    counts, K, N, n_x = [9, 40, 0, 129, 20], 1100, 136, 50
    R = sum(counts)
    x, w, sx, sw = _operands(R, n_x, 5, K, N, dtype)
    offsets = torch.tensor([0, 9, 49, 49, 178, 198], dtype=torch.int32, device=DEV)
    rows = torch.randint(0, n_x, (R,), device=DEV, dtype=torch.int32)
    go = lambda t: gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw, y=t)  # noqa: E731
    ys = [torch.zeros(R, N, dtype=BF16, device=DEV) for _ in range(3)]
    go(ys[2])
    torch.cuda.synchronize()
    for t in ys[:2]:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(3):
                go(t)
    torch.cuda.synchronize()
    assert bits_equal(ys[0], ys[2]) and bits_equal(ys[1], ys[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(ys[0])
        go(ys[1])
    offsets.copy_(torch.tensor([0, 0, 100, 101, 101, 198], dtype=torch.int32))
    rows.copy_(torch.randint(-1, n_x, (R,), dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    status_clean()
    m64.check_product(ys[0], *m64.grouped(x, w, offsets, rows, sx, sw), K, dtype == E4M3)
    assert bits_equal(ys[0], ys[1])
