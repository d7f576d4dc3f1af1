"""Failure path of the grouped and block-scaled products on the GPU, without a
fault: loads are left out and the wait limit is 1 ms, so that the waits for them run
out.  The call must return, report GDN_DEVSTAT_TIMEOUT and nothing else, write
nothing outside its rows and leave the context usable: the same call with the
defaults restored is right."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3


# one tile and several for a CTA, tiles of 16 to 128 rows and of pairs, rows gathered or in place
CASES = [([3] * 10, 1024, 512, E4M3, True), ([3] * 10, 1024, 512, BF16, False), ([4] * 300, 512, 1024, E4M3, True),
         ([100], 2048, 512, E4M3, False), ([60, 61, 50, 64], 1000, 3000, BF16, True), ([256], 2048, 8192, E4M3, False),
         ([700, 0, 513, 900], 512, 4096, E4M3, True), ([700, 0, 513, 900], 512, 4003, BF16, True),
         ([5000], 640, 4096, E4M3, False), ([3000, 3000], 512, 2048, BF16, False)]


@pytest.mark.parametrize("drop", [1, 2])
@pytest.mark.parametrize("counts,K,N,dtype,gather", CASES)
def test_waits_run_out_and_the_context_survives(counts, K, N, dtype, gather, drop):
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
    guard = torch.full((R + 1, N), 7.0, dtype=BF16, device=DEV)
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
    # with the first tile of a pair kept, one tile for each leaves nothing out
    assert st == gdn().DEVSTAT_TIMEOUT or (drop == 2 and st == 0), f"status {st:#x}"
    assert torch.all(guard[R] == 7.0)
    if drop == 1:
        assert st == gdn().DEVSTAT_TIMEOUT and torch.all(guard == 7.0)
    go()
    torch.cuda.synchronize()
    status_clean()
    ref, size = m64.grouped(x, w, offsets, rows, sx, sw)
    m64.check_product(guard[:R], ref, size, K, dtype == E4M3)
    assert torch.all(guard[R] == 7.0)


def test_a_call_may_take_longer_than_the_limit():
    """The limit is one of each wait: a call of some 300 us at 100 us ends as usual."""
    T, K, N = 20000, 2048, 8192
    g = torch.Generator(device=DEV).manual_seed(3)
    x, sx = m64.quantise_blocks(torch.randn(T, K, generator=g, device=DEV), 1)
    w, sw = m64.quantise_blocks(torch.randn(N, K, generator=g, device=DEV), 128)
    want = gdn().gdn_linear_block(x.contiguous(), w.contiguous(), sx, sw)
    gdn().gdn_debug_set_wait_limit(100_000)
    try:
        y = gdn().gdn_linear_block(x.contiguous(), w.contiguous(), sx, sw)
        torch.cuda.synchronize()
        status_clean()
    finally:
        gdn().gdn_debug_set_wait_limit(0)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
