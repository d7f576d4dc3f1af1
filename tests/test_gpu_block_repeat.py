"""The block operators again and again on the same inputs, with calls on other inputs
between them and nothing waited for: the same bits every time."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, b64.E4M3


def _state(op, T, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if op == "norm":
        x, res, w = r(T, 2048).to(BF16), r(T, 2048).to(BF16), r(2048)
        y, ys, ro = torch.empty(T, 2048, dtype=E4M3, device=DEV), torch.empty(T, device=DEV), torch.empty_like(x)
        return (lambda: gdn().gdn_add_rmsnorm(x, w, residual=res, y=y, y_scale=ys, residual_out=ro)), (y, ys, ro)
    if op == "gated":
        o, z, w = r(T, 32, 128).to(BF16), r(T, 32, 128).to(BF16), r(128)
        y, ys = torch.empty(T, 32, 128, dtype=E4M3, device=DEV), torch.empty(T, device=DEV)
        return (lambda: gdn().gdn_gated_rmsnorm_quant(o, z, w, y=y, y_scale=ys)), (y, ys)
    (x, sx), (w, sw), res = b64.quantise(r(T, 1024)), b64.quantise(r(1031, 1024)), r(T, 1031).to(BF16)
    y = torch.empty(T, 1031, dtype=BF16, device=DEV)
    return (lambda: gdn().gdn_linear(x, w, x_scale=sx, weight_scale=sw, act="gelu", residual=res, y=y)), (y,)


@pytest.mark.parametrize("T", [1, 256, 6000])
@pytest.mark.parametrize("op", ["norm", "gated", "linear"])
def test_same_bits_between_other_calls(op, T):
    (go, out), (other, _) = _state(op, T, 1), _state(op, T, 2)
    bits = lambda: [t.view(torch.uint8).clone() for t in out]  # noqa: E731
    go()
    first = bits()
    for k in range(30):
        for t in out:
            t.view(torch.uint8).fill_(0x55)
        for _ in range(k % 3):
            other()
        go()
        other()
        assert all(torch.equal(a, b) for a, b in zip(first, bits())), f"call {k}"
    status_clean()
