"""The router and the combination of a mixture of experts on the GPU: every choice
and every place against a stable sort, the weights and the sums in 64 bits."""
import pytest
import torch

from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def _logits(seed, T, E, dtype, step=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = 2 * torch.randn(T, E, generator=g, device=DEV)
    if step:                                            # few values, so that most are tied
        x = (x / step).round() * step
    return x.to(dtype)


def _check(logits, top, renorm=True, what=""):
    got = gdn().gdn_moe_route(logits, top, renormalize=renorm)
    torch.cuda.synchronize()
    status_clean()
    want = m64.route(logits, top, renorm)
    for name, a, b in zip(("ids", "", "offsets", "rows", "slots"), got, want):
        if name:
            assert torch.equal(a.cpu(), b), f"{what} {name}"
    m64.check_weights(got[1], want[1], logits, want[0], what)
    return got


@pytest.mark.parametrize("T", [0, 1, 2, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257, 511, 512, 513, 1000, 5000])
@pytest.mark.parametrize("E,top", [(512, 10), (60, 4), (1, 1), (33, 33 - 1)])
def test_tokens(T, E, top):
    _check(_logits(T + E, T, E, F32), top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,top", [(38912, 24, 3), (38913, 24, 3), (70000, 16, 2), (160001, 9, 1), (40000, 1024, 30)])
def test_runs_of_more_than_a_word_of_tokens(T, E, top, dtype):
    _check(_logits(T, T, E, dtype), top)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [1, 2, 3, 8, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 511, 512, 513,
                               777, 1000, 1023, 1024])
def test_experts(E, dtype):
    for top in {1, min(E, 2), min(E, 7), min(E, 10), min(E, 32)}:
        for renorm in (True, False):
            _check(_logits(E + top, 70, E, dtype), top, renorm, f"top {top}")
        _check(_logits(E + top, 600, E, dtype), top, False, f"many, top {top}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,top", [(5, 512, 10), (300, 512, 10), (2000, 512, 10), (700, 100, 32), (64, 1024, 32), (90, 48, 6)])
def test_ties_go_to_the_lowest_index(T, E, top, dtype):
    for step in (0.25, 1.0, 4.0, 100.0):
        _check(_logits(T, T, E, dtype, step), top, what=f"step {step}")
    x = _logits(T, T, E, dtype, 1.0)
    _check(torch.where(x == 0, torch.where(torch.arange(E, device=DEV) % 2 == 0, -0.0, 0.0).to(dtype), x), top, what="-0")


@pytest.mark.parametrize("T", [7, 200, 900])
@pytest.mark.parametrize("renorm", [True, False])
def test_closed_experts_nans_and_infinities(T, renorm):
    E, top = 96, 6
    x = _logits(T, T, E, F32)
    x[0] = -INF                                         # no expert is open: weights 0
    x[1, 3:] = -INF                                     # three are
    x[2, ::2] = torch.finfo(F32).min                    # a mask of the type's lowest value
    x[3] = torch.finfo(F32).min
    x[4, 50] = 1e30
    got = _check(x, top, renorm)
    assert torch.all(got[1][0] == 0) and torch.all(got[1][1, 3:] == 0)
    y = x.clone()
    y[5, 70], y[5, 20] = NAN, NAN
    y[6, 9] = INF
    ids, w, offsets, rows, slots = (t.cpu() for t in gdn().gdn_moe_route(y, top, renormalize=renorm))
    want = m64.route(y, top, renorm)
    for a, b in zip((ids, offsets, rows, slots), (want[0], want[2], want[3], want[4])):
        assert torch.equal(a, b)
    assert ids[5, :2].tolist() == [20, 70] and ids[6, 0] == 9
    assert torch.all(torch.isnan(w[5])) and torch.isnan(w[6, 0])
    keep = torch.ones(T, dtype=torch.bool)
    keep[5] = keep[6] = False
    assert bits_equal(w[keep], got[1].cpu()[keep])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,pad,off", [(40, 64, 64, 0), (700, 64, 3, 1), (700, 500, 12, 4), (9, 7, 1, 3), (100, 512, 512, 8)])
def test_strided_logits(T, E, pad, off, dtype):
    wide = torch.full((T, E + pad + off), INF, dtype=dtype, device=DEV)
    wide[:, off:off + E] = _logits(T, T, E, dtype)
    _check(wide[:, off:off + E], min(E, 8))


def test_the_same_expert_for_all():
    for T in (50, 512, 513, 4000):
        x = torch.zeros(T, 40, device=DEV)
        x[:, 17], x[:, 39] = 5.0, 4.0
        ids, _, offsets, rows, slots = _check(x, 2)
        assert torch.equal(rows.cpu(), torch.arange(T, dtype=torch.int32).repeat(2))


def test_route_far_logits():
    """Rows that lie more than 2^31 elements apart."""
    E = 64
    buf = torch.empty(2 ** 31 + 4096, dtype=BF16, device=DEV)
    x = buf.as_strided((2, E), (2 ** 31 + 64, 1), 0)
    x.copy_(_logits(3, 2, E, BF16))
    _check(x, 5)


@pytest.mark.parametrize("T", [40, 300, 3000])
def test_route_outputs_given_streams_and_graph(T):
    E, top = 128, 8
    a, b = _logits(1, T, E, F32), _logits(2, T, E, BF16, 0.5)
    wa, wb = gdn().gdn_moe_route(a, top), gdn().gdn_moe_route(b, top)
    ga, gb = ([torch.empty_like(t) for t in w] for w in (wa, wb))
    need = gdn().gdn_moe_route_workspace_size(T, E)
    spaces = [torch.empty(max(need, 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
    go = lambda x, o, ws: gdn().gdn_moe_route(x, top, True, *o, workspace=ws)  # noqa: E731
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            go(a, ga, spaces[0])
        with torch.cuda.stream(s2):
            go(b, gb, spaces[1])
    torch.cuda.synchronize()
    for got, want in zip(ga + gb, [*wa, *wb]):
        assert bits_equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                       # one workspace: the calls follow each other
        go(a, ga, spaces[0])
        go(b, gb, spaces[0])
    a.copy_(_logits(7, T, E, F32))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    want = m64.route(a, top, True)
    for i in (0, 2, 3, 4):
        assert torch.equal(ga[i].cpu(), want[i])
    for got, w in zip(gb, wb):
        assert bits_equal(got, w)
    status_clean()


def test_route_writes_nothing_else():
    T, E, top = 333, 50, 5
    x = _logits(T, T, E, F32)
    bufs = [torch.full((n + 8,), 77, dtype=d, device=DEV) for n, d in
            ((T * top, torch.int32), (T * top, F32), (E + 1, torch.int32), (T * top, torch.int32), (T * top, torch.int32))]
    out = [b[:-8] for b in bufs]
    gdn().gdn_moe_route(x, top, True, out[0].view(T, top), out[1].view(T, top), out[2], out[3], out[4].view(T, top))
    torch.cuda.synchronize()
    for b in bufs:
        assert torch.all(b[-8:] == 77)


# ------------------------------------------------------------- combination --

def _combine_case(seed, T, top, H, dtype, residual, R=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    R = T * top if R is None else R
    x = torch.randn(R, H, generator=g, device=DEV).to(dtype)
    slots = torch.randint(0, R, (T, top), generator=g, device=DEV, dtype=torch.int32)
    w = torch.rand(T, top, generator=g, device=DEV)
    res = (3 * torch.randn(T, H, generator=g, device=DEV)).to(dtype) if residual else None
    return x, slots, w, res


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,top,H", [(1, 1, 1), (1, 10, 2048), (2, 3, 33), (7, 2, 8), (30, 8, 1000), (100, 16, 257), (257, 10, 2048),
                                     (1000, 4, 64), (3, 33, 4096), (64, 5, 12), (5, 40, 100), (2000, 10, 24)])
def test_combine_sizes(T, top, H, dtype):
    for residual in (False, True):
        x, slots, w, res = _combine_case(T + H, T, top, H, dtype, residual)
        guard = torch.full((T + 1, H), 7.0, dtype=dtype, device=DEV)
        y = gdn().gdn_moe_combine(x, slots, w, residual=res, y=guard[:T])
        torch.cuda.synchronize()
        status_clean()
        m64.check_combine(y, *m64.combine(x, slots, w, res), top)
        assert torch.all(guard[T] == 7.0)
        if residual:
            buf = res.clone()
            gdn().gdn_moe_combine(x, slots, w, residual=buf, y=buf)
            assert bits_equal(buf, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_combine_leaves_out_and_flags(dtype):
    x, slots, w, res = _combine_case(5, 20, 4, 72, dtype, True)
    slots[3, 1] = -1
    slots[4] = -5
    x[0] = NAN                                          # a row that nobody asks for
    slots[slots == 0] = 1
    y = gdn().gdn_moe_combine(x, slots, w, residual=res)
    torch.cuda.synchronize()
    status_clean()
    m64.check_combine(y, *m64.combine(x, slots, w, res), 4)
    assert bits_equal(y[4], res[4])
    slots[6, 2] = x.shape[0]
    slots[7, 0] = 2 ** 31 - 1
    y = gdn().gdn_moe_combine(x, slots, w, residual=res)
    torch.cuda.synchronize()
    assert gdn().gdn_get_device_status(clear=True) == gdn().DEVSTAT_BAD_INDEX
    m64.check_combine(y, *m64.combine(x, slots, w, res), 4)


@pytest.mark.parametrize("H", [40, 43, 44])
def test_combine_strided(H):
    T, top = 50, 6
    for dtype in (F32, BF16):
        x, slots, w, res = _combine_case(H, T, top, H, dtype, True)
        want = gdn().gdn_moe_combine(x, slots, w, residual=res)
        for off, pad in ((0, 8), (1, 4), (8, 8), (3, 0)):
            cut = lambda t: torch.full((t.shape[0], H + off + pad), 9.0, dtype=dtype, device=DEV)  # noqa: E731
            xw, rw, yw = cut(x), cut(res), cut(res)
            xw[:, off:off + H], rw[:, off:off + H] = x, res
            gdn().gdn_moe_combine(xw[:, off:off + H], slots, w, residual=rw[:, off:off + H], y=yw[:, off:off + H])
            torch.cuda.synchronize()
            assert bits_equal(yw[:, off:off + H].contiguous(), want)
            assert torch.all(yw[:, :off] == 9.0) and torch.all(yw[:, off + H:] == 9.0)


def test_combine_of_no_rows_and_no_tokens():
    x = torch.empty(0, 16, device=DEV)
    slots, w = torch.full((3, 2), -1, dtype=torch.int32, device=DEV), torch.ones(3, 2, device=DEV)
    assert torch.all(gdn().gdn_moe_combine(x, slots, w) == 0)
    assert gdn().gdn_moe_combine(x, slots[:0], w[:0]).shape == (0, 16)


def test_combine_far_rows():
    """Rows of x past 2^31 elements."""
    R, H = 2 ** 31 // 4096 + 9, 4096
    x = torch.empty(R, H, dtype=BF16, device=DEV)
    x[-9:] = torch.randn(9, H, device=DEV).to(BF16)
    slots = torch.arange(R - 9, R, dtype=torch.int32, device=DEV).view(3, 3)
    w = torch.rand(3, 3, device=DEV)
    y = gdn().gdn_moe_combine(x, slots, w)
    near = gdn().gdn_moe_combine(x[-9:].contiguous(), slots - (R - 9), w)
    torch.cuda.synchronize()
    assert bits_equal(y, near)


@pytest.mark.parametrize("top", [-1, 0, 9])
def test_route_refuses_a_number_of_choices(top):
    with pytest.raises(gdn().GdnError):
        gdn().gdn_moe_route(torch.zeros(4, 8, device=DEV), top)
