"""What gdn_linear_block promises of a row among others: the same bits in a call of the
same sizes, whatever the other rows hold; in calls of other sizes a sum within the
product's bound, whose order over k the sizes choose."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, E4M3 = torch.float32, b64.E4M3
SIZES = [1, 7, 16, 17, 33, 64, 65, 100, 256, 300, 1000]


def _operands(T, K, N):
    g = torch.Generator(device=DEV).manual_seed(K)
    x, sx = m64.quantise_blocks(torch.randn(T, K, generator=g, device=DEV), 1)
    w, sw = m64.quantise_blocks(torch.randn(N, K, generator=g, device=DEV) * K ** -0.5, 128)
    return x.contiguous(), sx, w.contiguous(), sw


@pytest.mark.parametrize("K,N", [(4096, 2048), (2048, 8192), (16384, 256)])
def test_other_values(K, N):
    x, sx, w, sw = _operands(1000, K, N)
    for T in SIZES:
        a = gdn().gdn_linear_block(x[:T], w, sx[:T], sw, y_dtype=F32)
        other, scales = x.clone(), sx.clone()
        keep = torch.arange(T, device=DEV) % 3 == 0
        other.view(torch.uint8)[:T][~keep] = 0x7F        # NaN
        scales[:T][~keep] = 1e30
        b = gdn().gdn_linear_block(other[:T], w, scales[:T], sw, y_dtype=F32)
        torch.cuda.synchronize()
        assert bits_equal(a[keep], b[keep])
    status_clean()


@pytest.mark.parametrize("K,N", [(4096, 2048), (2048, 8192), (16384, 256)])
def test_other_sizes(K, N):
    x, sx, w, sw = _operands(1000, K, N)
    ref, size = m64.product(x, w, sx, sw)
    for T in SIZES:
        y = gdn().gdn_linear_block(x[:T], w, sx[:T], sw, y_dtype=F32)
        torch.cuda.synchronize()
        m64.check_product(y, ref[:T], size[:T], K, True, f"T={T}")
    # with one order of the sum, the same bits in every size
    try:
        for rows in (16, 32, 64, 128, 256):
            gdn().gdn_debug_set_grouped_tile(rows, 0)
            ys = [gdn().gdn_linear_block(x[:T], w, sx[:T], sw, y_dtype=F32) for T in SIZES]
            torch.cuda.synchronize()
            assert all(bits_equal(y, ys[-1][:len(y)]) for y in ys), rows
    finally:
        gdn().gdn_debug_set_grouped_tile()
    status_clean()
