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
