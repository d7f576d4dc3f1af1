"""Failure path of gdn_linear on the GPU, without a fault: loads are left out and
the wait limit is 1 ms, so that its waits run out.  The call must return, report
GDN_DEVSTAT_TIMEOUT and nothing else, write nothing that did not come and leave
the context usable: the same call with the defaults restored is right."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3


# k in one, two to four, and eight for few tokens; many tokens with one tile and with
# several for a pair, with columns' scales (barriers of the epilogue's warps) and without
@pytest.mark.parametrize("T,K,N,dtype,out,bias", [
    (8, 512, 40000, BF16, BF16, True), (256, 4096, 2048, BF16, BF16, False), (8, 8192, 128, BF16, F32, True),
    (100, 2048, 512, E4M3, BF16, True), (512, 2048, 8192, BF16, BF16, True), (4096, 512, 4096, BF16, BF16, True),
    (4096, 512, 4096, BF16, BF16, False), (4000, 640, 4003, E4M3, F32, True)])
@pytest.mark.parametrize("drop", [1, 2])
def test_waits_run_out_and_the_context_survives(T, K, N, dtype, out, bias, drop):
    g = torch.Generator(device=DEV).manual_seed(T + N)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, w, sx, sw, b = r(T, K), r(N, K) * K ** -0.5, None, None, r(N) if bias else None
    if dtype == E4M3:
        (x, sx), (w, sw) = b64.quantise(x), b64.quantise(w)
    else:
        x, w = x.to(dtype), w.to(dtype)
    res = r(T, N).to(out)
    act = "silu" if bias else "none"
    guard = torch.full((T + 1, N), 7.0, dtype=out, device=DEV)
    go = lambda y: gdn().gdn_linear(x, w, x_scale=sx, weight_scale=sw, bias=b, act=act, residual=res, y=y)  # noqa: E731
    status_clean()
    gdn().gdn_debug_set_wait_limit(1_000_000, drop_linear_loads=drop)      # 1 ms
    try:
        go(guard[:T])
        torch.cuda.synchronize()
        st = gdn().gdn_get_device_status(clear=True)
    finally:
        gdn().gdn_debug_set_wait_limit(0)
    # 512 tokens are one tile for a pair: nothing is left out behind it
    assert st == (0 if drop == 2 and T == 512 else gdn().DEVSTAT_TIMEOUT), f"status {st:#x}"
    assert torch.all(guard[T] == 7.0)
    if drop == 1:
        assert torch.all(guard == 7.0)

    go(guard[:T])
    torch.cuda.synchronize()
    status_clean()
    ref, size = b64.linear(x, w, sx, sw, b, act, res)
    b64.check_linear(guard[:T], ref, size, K, dtype == E4M3)
    assert torch.all(guard[T] == 7.0)


def test_two_kernel_limit_leaves_the_product_alone():
    """The prefill's part of the control does not reach the loads of the product."""
    x, w = (torch.ones(4, 64, dtype=BF16, device=DEV) for _ in range(2))
    gdn().gdn_debug_set_wait_limit(0, drop_prep_loads=True)
    try:
        y = gdn().gdn_linear(x, w)
        torch.cuda.synchronize()
    finally:
        gdn().gdn_debug_set_wait_limit(0)
    assert torch.all(y == 64)
    status_clean()


def test_a_call_may_take_longer_than_the_limit():
    """The limit is one of each wait: a call of some 400 us at 100 us ends as usual."""
    T, K, N = 20000, 2048, 8192
    g = torch.Generator(device=DEV).manual_seed(3)
    x, w = (torch.randn(n, K, generator=g, device=DEV).to(BF16) for n in (T, N))
    want = gdn().gdn_linear(x, w)
    gdn().gdn_debug_set_wait_limit(100_000)
    try:
        y = gdn().gdn_linear(x, w)
        torch.cuda.synchronize()
        status_clean()
    finally:
        gdn().gdn_debug_set_wait_limit(0)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
