"""gdn_gated_rmsnorm_quant over many rows and the widest ones, against 64 bits: more
tokens than CTAs for every launch form, so that a CTA's second token, loaded ahead
of the first, is looked at, with a NaN token among them; views of z."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, b64.E4M3


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def test_z_of_one_head_with_a_free_middle_stride():
    T, dv = 9, 64
    o, wide, w = _rand(1, T, 1, dv).to(BF16), _rand(2, T, 3, dv).to(BF16), _rand(3, dv)
    z = wide[:, ::3]
    assert z.shape == (T, 1, dv) and z.stride(1) == 3 * dv
    y, scale = gdn().gdn_gated_rmsnorm_quant(o, z, w)
    p, pscale = gdn().gdn_gated_rmsnorm_quant(o, z.contiguous(), w)
    torch.cuda.synchronize()
    assert bits_equal(scale, pscale) and bits_equal(y.view(torch.uint8), p.view(torch.uint8))


# tokens, heads, dim: a vector of 8 values a thread; two, of up to 512 (fp32) or 1024
# threads; the widest rows
ROWS = [(20000, 1, 16, BF16), (5000, 4, 128, BF16), (5000, 4, 128, F32), (2000, 32, 128, BF16), (2000, 32, 128, F32),
        (2000, 32, 256, F32), (2000, 32, 256, BF16), (500, 64, 256, BF16), (500, 64, 256, F32), (400, 63, 256, F32),
        (1000, 513, 16, BF16)]


@pytest.mark.parametrize("off", [8, 4])          # z on and (bf16) off 16 bytes
@pytest.mark.parametrize("T,hv,dv,dtype", ROWS)
def test_more_tokens_than_ctas(T, hv, dv, dtype, off):
    row = hv * dv
    o, zw, w = _rand(T, T, hv, dv, scale=0.3).to(dtype), _rand(hv, T, row + 16).to(dtype), _rand(3, dv).abs() + 0.5
    z = zw[:, off:off + row]
    o[T // 2, hv // 2, 3] = float("nan")
    z[T - 2] = 0
    guard = torch.ones(T + 2, row, device=DEV).to(E4M3)
    sg = torch.full((T + 2,), -3.0, device=DEV)
    y, scale = gdn().gdn_gated_rmsnorm_quant(o, z, w, y=guard[1:T + 1].view(T, hv, dv), y_scale=sg[1:T + 1])
    torch.cuda.synchronize()
    status_clean()
    y = y.float().reshape(T, row)
    assert torch.isnan(scale[T // 2]) and torch.all(torch.isnan(y[T // 2]))
    assert scale[T - 2] == 2.0 ** -126 and torch.all(y[T - 2] == 0)
    live = torch.ones(T, dtype=torch.bool, device=DEV)
    live[T // 2] = live[T - 2] = False
    ref = b64.gated_norm(o, z.unflatten(1, (hv, dv)), w, 1e-6).reshape(T, row)
    b64.check_quant(y[live], scale[live], ref[live], b64.GATED, "y")
    assert sg[0] == -3 and sg[T + 1] == -3
    assert torch.all(guard[0].float() == 1) and torch.all(guard[T + 1].float() == 1)
    # a token's bits do not depend on where it stands
    n = min(T, 100)
    last = torch.arange(T - n, T, device=DEV)
    p, pscale = gdn().gdn_gated_rmsnorm_quant(o[last].contiguous(), z[last].contiguous(), w)
    torch.cuda.synchronize()
    ok = live[last]
    assert bits_equal(pscale[ok], scale[last][ok])
    assert torch.equal(p.float().reshape(n, row)[ok], y[last][ok])
