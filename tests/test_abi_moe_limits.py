"""The combination's limit on its size is the one its contract names: n_tokens *
ceil(hidden / 256) < 2^31, where rows are no vectors."""
import pytest

from tests.test_abi_moe import COMBINE, COMBINE0, F32, UNSUPPORTED, _call, lib  # noqa: F401


@pytest.mark.parametrize("T,H,dt", [(1 << 30, 257, 1), (1 << 30, 257, F32), ((1 << 31) - 1, 257, 1), ((1 << 31) // 5 + 1, 1025, F32)])
def test_too_many_ctas(lib, T, H, dt):  # noqa: F811
    assert T * -(-H // 256) >= 1 << 31 and T * H < 1 << 40
    assert _call(lib, "gdn_moe_combine", COMBINE, COMBINE0, T=T, H=H, k=1, xs=H, rs=H, ys=H, dt=dt) == UNSUPPORTED
