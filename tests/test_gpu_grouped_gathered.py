"""Gathered rows of the grouped products are those that a copy of them in their order
gives, bit for bit: a stage of shared memory that a product read before the rows' copies
were there, or after the next ones, would show as another row's values."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, b64.E4M3


def _same_as_in_place(counts, K, N, dtype, n_x, rounds):
    E, R = len(counts), sum(counts)
    g = torch.Generator(device=DEV).manual_seed(R + K + N)
    w, sx, sw = torch.randn(E, N, K, generator=g, device=DEV) * K ** -0.5, None, None
    if dtype == E4M3:
        w, sw = m64.quantise_blocks(w, 128)
        sw = sw.contiguous()
    w = m64.padded(w if dtype == E4M3 else w.to(dtype), 0.0)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    for i in range(rounds):                              # other rows at the same places, of other sizes
        x = torch.randn(n_x, K, generator=g, device=DEV) * 4.0 ** (i - 2)
        if dtype == E4M3:
            x, sx = m64.quantise_blocks(x, 1)
        x = m64.padded(x if dtype == E4M3 else x.to(dtype), 0.0)
        rows = torch.randint(0, n_x, (R,), generator=g, device=DEV, dtype=torch.int32)
        at = rows.long()
        raw = torch.uint8 if dtype == E4M3 else dtype
        copy = m64.padded(x.contiguous().view(raw)[at].view(dtype), 0.0)
        want = gdn().gdn_grouped_linear(copy, w, offsets, x_scale=None if sx is None else sx[at], weight_scale=sw, y_dtype=F32)
        for _ in range(3):
            got = gdn().gdn_grouped_linear(x, w, offsets, rows=rows, x_scale=sx, weight_scale=sw, y_dtype=F32)
            torch.cuda.synchronize()
            assert bits_equal(got, want)
    status_clean()
    ref, size = m64.grouped(x, w, offsets, rows, sx, sw)
    m64.check_product(got, ref, size, K, dtype == E4M3)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("counts,K,N", [([1500, 2000, 0, 2500, 1], 2048, 2048), ([4000, 4096], 1000, 1024), ([3000] * 4, 130, 4000)])
def test_many_rows(counts, K, N, dtype):
    """Sizes of the pairs of CTAs, where one CTA's product reads rows that the other one's threads copied."""
    _same_as_in_place(counts, K, N, dtype, 5000, 4)
