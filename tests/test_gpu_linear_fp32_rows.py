"""gdn_linear with wide fp32 rows: y and an fp32 residual packed, as columns of wider
buffers on and off 16 bytes, and in place, for few and many tokens."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3


@pytest.mark.parametrize("T", [3, 100, 300, 2100])
@pytest.mark.parametrize("N", [8192, 8190, 12289])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_wide_fp32_rows(T, N, dtype):
    K = 144
    g = torch.Generator(device=DEV).manual_seed(T + N)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, w, sx, sw, b, res = r(T, K), r(N, K) * K ** -0.5, None, None, r(N), r(T, N)
    if dtype == E4M3:
        (x, sx), (w, sw) = b64.quantise(x), b64.quantise(w)
    else:
        x, w = x.to(dtype), w.to(dtype)
    go = lambda **kw: gdn().gdn_linear(x, w, x_scale=sx, weight_scale=sw, bias=b, act="silu", **kw)  # noqa: E731
    y = go(residual=res, y_dtype=F32)
    ref, size = b64.linear(x, w, sx, sw, b, "silu", res)
    b64.check_linear(y, ref, size, K, dtype == E4M3)
    for off, pad in ((4, 4), (1, 2), (0, 3)):
        wide = torch.full((T + 1, N + off + pad), 3.0, device=DEV)
        cut = wide[:T, off:off + N]
        cut.copy_(res)
        go(residual=cut, y=cut)
        torch.cuda.synchronize()
        assert bits_equal(cut.contiguous(), y)
        assert torch.all(wide[T] == 3.0) and torch.all(wide[:, :off] == 3.0) and torch.all(wide[:, off + N:] == 3.0)
    status_clean()
