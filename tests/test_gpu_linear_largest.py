"""gdn_linear at the ends of what is built: the most tokens, many channels, offsets
of y past 32 bits."""
import pytest
import torch

from tests import block64 as b64
from tests.gpu_common import DEV, gdn, status_clean

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _rand(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV, dtype=BF16)


@pytest.mark.parametrize("N", [32, 33])
def test_the_most_tokens(N):
    T, K = 65535 * 256, 16
    x, w = _rand(1, T, K), _rand(2, N, K)
    guard = torch.full((T + 1, N), 7.0, dtype=BF16, device=DEV)
    y = gdn().gdn_linear(x, w, act="silu", y=guard[:T])
    torch.cuda.synchronize()
    status_clean()
    assert torch.all(guard[T] == 7.0)
    for lo in (0, 8388480 - 1000, T // 2, T - 300000):
        rows = slice(lo, lo + 300000)
        ref, size = b64.linear(x[rows], w, None, None, None, "silu", None)
        b64.check_linear(y[rows], ref, size, K)


@pytest.mark.parametrize("T", [1, 130])
def test_many_channels(T):
    N, K = 2 ** 24 + 8, 8
    x, w, b = _rand(1, T, K), _rand(2, N, K), _rand(3, N).float()
    y = gdn().gdn_linear(x, w, bias=b)
    torch.cuda.synchronize()
    status_clean()
    for lo in (0, N // 2 + 3, N - 200000):
        at = slice(lo, lo + 200000)
        ref, size = b64.linear(x, w[at], None, None, b[at], "none", None)
        b64.check_linear(y[:, at], ref, size, K)


def test_a_long_sum():
    """n_in in the millions: k cut over a cluster, and whole."""
    K = 2 ** 22 + 8
    for T, N in ((2, 40), (200, 33)):
        x, w = _rand(1, T, K), _rand(2, N, K)
        y = gdn().gdn_linear(x, w, y_dtype=F32)
        torch.cuda.synchronize()
        status_clean()
        ref = torch.zeros(T, N, dtype=torch.float64, device=DEV)
        size = torch.zeros_like(ref)
        for lo in range(0, K, 2 ** 18):
            a, b = x[:, lo:lo + 2 ** 18].double(), w[:, lo:lo + 2 ** 18].double()
            ref += a @ b.t()
            size += a.abs() @ b.abs().t()
        b64.check_linear(y, ref, size, K)
