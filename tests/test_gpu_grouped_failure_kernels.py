"""Failure path of every kernel of the grouped and block-scaled products on the GPU,
without a fault: loads are left out and the wait limit is 1 ms, so that the waits for
them run out.  Whatever was left out, the call reports GDN_DEVSTAT_TIMEOUT, and what it
wrote are finished sums: a tile is either as it was or right."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.test_gpu_grouped_failure import CASES

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3
KERNELS = [(rows, cut) for rows in (16, 32, 64, 128) for cut in range(4)] + [(256, 0)]


def _check(counts, K, N, dtype, gather, drop):
    E, R = len(counts), sum(counts)
    n_x = 50 if gather else R
    g = torch.Generator(device=DEV).manual_seed(R + N)
    x, w = torch.randn(n_x, K, generator=g, device=DEV), torch.randn(E, N, K, generator=g, device=DEV) * K ** -0.5
    sx = sw = None
    if dtype == E4M3:
        (x, sx), (w, sw) = m64.quantise_blocks(x, 1), m64.quantise_blocks(w, 128)
        sw = sw.contiguous()
    else:
        x, w = x.to(dtype), w.to(dtype)
    x, w = m64.padded(x, 0.0), m64.padded(w, 0.0)
    rows = torch.randint(0, n_x, (R,), generator=g, device=DEV, dtype=torch.int32) if gather else None
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    ref, size = m64.grouped(x, w, offsets, rows, sx, sw)
    guard = torch.full((R + 1, N), 700.0, dtype=F32, device=DEV)
    go = lambda: gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw, y=guard[:R])  # noqa: E731
    if E == 1:
        go = lambda: gdn().gdn_linear_block(x, w[0], sx, sw[0], y=guard[:R])  # noqa: E731
    status_clean()
    gdn().gdn_debug_set_wait_limit(1_000_000, drop_linear_loads=drop)      # 1 ms
    try:
        go()
        torch.cuda.synchronize()
        st = gdn().gdn_get_device_status(clear=True)
    finally:
        gdn().gdn_debug_set_wait_limit(0)
    assert st == gdn().DEVSTAT_TIMEOUT, f"status {st:#x}"
    left = guard == 700.0
    assert left.any() and (drop == 2 or left.all()) and left[R].all()
    # (the bound of values that are there, and of none where the guard is)
    held = torch.where(left[:R], ref, guard[:R].double()).to(F32)
    m64.check_product(held, ref, size, K, dtype == E4M3, f"drop {drop}")
    go()
    torch.cuda.synchronize()
    status_clean()
    m64.check_product(guard[:R], ref, size, K, dtype == E4M3)
    assert guard[R].eq(700.0).all()


@pytest.mark.parametrize("drop", [1, 2])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: f"{k[0]}rows{1 << k[1]}parts")
def test_every_kernel(kernel, dtype, gather, drop):
    """Two blocks of k a part at least, and several tiles a pair, so that something is left out behind the first."""
    gdn().gdn_debug_set_grouped_tile(*kernel)
    try:
        if kernel[0] == 256:
            _check([5000, 3000, 0, 4000], 640, 1024, dtype, gather, drop)
        else:
            _check([70, 0, 3, 200], 2100, 300, dtype, gather, drop)
    finally:
        gdn().gdn_debug_set_grouped_tile()


@pytest.mark.parametrize("drop", [1, 2])
@pytest.mark.parametrize("counts,K,N,dtype,gather", CASES)
def test_chosen_kernels(counts, K, N, dtype, gather, drop):
    _check(counts, K, N, dtype, gather, drop)
