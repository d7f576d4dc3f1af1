"""Refusals of the mixture-of-experts entry points and of the block-scaled product:
the host checks return before anything touches the device."""
import ctypes

import pytest

V, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    return ctypes.CDLL(__graft_entry__._build_module().build())


def p(n):
    return V(0x10000 * n)   # never dereferenced


def _call(lib, name, types, base, **change):
    f = getattr(lib, name)
    f.argtypes = [t for t in types.values()]
    args = dict(base)
    args.update(change)
    assert set(args) == set(types)
    return f(*[args[k] for k in types])


BLOCK = dict(x=V, xs=I64, sx=V, w=V, ws=I64, sw=V, T=I64, K=I32, N=I32, y=V, ys=I64, ydt=I32, stream=V)
BLOCK0 = dict(x=p(1), xs=256, sx=p(2), w=p(3), ws=256, sw=p(4), T=0, K=256, N=128, y=p(5), ys=128, ydt=BF16, stream=None)


@pytest.mark.parametrize("want,change", [
    (OK, dict()), (OK, dict(x=None, y=None)),
    (INVALID, dict(T=-1)), (INVALID, dict(K=0)), (INVALID, dict(N=0)), (INVALID, dict(ydt=E4M3)), (INVALID, dict(ydt=7)),
    (INVALID, dict(T=4, x=None)), (INVALID, dict(T=4, w=None)), (INVALID, dict(T=4, y=None)), (INVALID, dict(T=4, sx=None)),
    (INVALID, dict(T=4, sw=None)), (INVALID, dict(T=4, y=p(1))), (INVALID, dict(T=4, y=p(3))),
    (INVALID, dict(T=4, xs=255)), (INVALID, dict(T=4, xs=264)), (INVALID, dict(T=4, ws=240)), (INVALID, dict(T=4, ws=257)),
    (INVALID, dict(T=4, ys=127)), (INVALID, dict(T=4, x=V(0x10008))), (INVALID, dict(T=4, w=V(0x10001))),
    (INVALID, dict(T=4, y=V(0x50001))), (INVALID, dict(T=4, ydt=F32, y=V(0x50002))), (INVALID, dict(T=4, sx=V(0x20002))),
    (INVALID, dict(T=4, sw=V(0x20001))), (UNSUPPORTED, dict(T=65535 * 256 + 1)), (UNSUPPORTED, dict(K=(1 << 20) + 1)),
    (UNSUPPORTED, dict(N=(1 << 20) + 1)), (UNSUPPORTED, dict(T=4, xs=1 << 36)), (UNSUPPORTED, dict(T=4, ys=1 << 36))])
def test_linear_block(lib, want, change):
    assert _call(lib, "gdn_linear_block", BLOCK, BLOCK0, **change) == want


GROUP = dict(x=V, xs=I64, sx=V, n_x=I64, rows=V, w=V, ws=I64, we=I64, sw=V, offsets=V, E=I32, R=I64, K=I32, N=I32, y=V, ys=I64,
             dt=I32, ydt=I32, stream=V)
GROUP0 = dict(x=p(1), xs=256, sx=None, n_x=8, rows=p(6), w=p(3), ws=256, we=256 * 128, sw=None, offsets=p(7), E=4, R=0, K=256,
              N=128, y=p(5), ys=128, dt=BF16, ydt=BF16, stream=None)


@pytest.mark.parametrize("want,change", [
    (OK, dict()), (INVALID, dict(R=-1)), (INVALID, dict(n_x=-1)), (INVALID, dict(K=0)), (INVALID, dict(N=-2)), (INVALID, dict(E=0)),
    (INVALID, dict(dt=9)), (UNSUPPORTED, dict(dt=F32)), (INVALID, dict(ydt=E4M3)),
    (INVALID, dict(R=9, x=None)), (INVALID, dict(R=9, w=None)), (INVALID, dict(R=9, y=None)), (INVALID, dict(R=9, offsets=None)),
    (INVALID, dict(R=9, n_x=0)), (INVALID, dict(R=9, rows=None)), (INVALID, dict(R=9, sx=p(8))), (INVALID, dict(R=9, sw=p(8))),
    (INVALID, dict(R=9, dt=E4M3)), (INVALID, dict(R=9, dt=E4M3, sx=p(8))), (INVALID, dict(R=9, xs=255)), (INVALID, dict(R=9, xs=260)),
    (INVALID, dict(R=9, ws=252)), (INVALID, dict(R=9, ws=260)), (INVALID, dict(R=9, we=256 * 127)), (INVALID, dict(R=9, we=256 * 128 + 4)),
    (INVALID, dict(R=9, ys=100)), (INVALID, dict(R=9, y=p(1))), (INVALID, dict(R=9, y=p(3))), (INVALID, dict(R=9, x=V(0x10004))),
    (INVALID, dict(R=9, rows=V(0x60002))), (INVALID, dict(R=9, offsets=V(0x70001))), (UNSUPPORTED, dict(R=65535 * 256 + 1)),
    (UNSUPPORTED, dict(n_x=1 << 31)), (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(K=(1 << 20) + 1)), (UNSUPPORTED, dict(N=(1 << 20) + 1)),
    (UNSUPPORTED, dict(R=9, we=1 << 36))])
def test_grouped_linear(lib, want, change):
    assert _call(lib, "gdn_grouped_linear", GROUP, GROUP0, **change) == want


ROUTE = dict(x=V, xs=I64, T=I64, E=I32, k=I32, renorm=I32, ids=V, w=V, offsets=V, rows=V, slots=V, dt=I32, ws=V, wsb=SZ, stream=V)
ROUTE0 = dict(x=p(1), xs=512, T=4, E=512, k=10, renorm=1, ids=p(2), w=p(3), offsets=p(4), rows=p(5), slots=p(6), dt=F32, ws=p(7),
              wsb=1 << 20, stream=None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(k=0)), (INVALID, dict(k=513)), (INVALID, dict(dt=E4M3)), (INVALID, dict(dt=5)),
    (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(k=33)), (UNSUPPORTED, dict(T=1 << 31)), (INVALID, dict(x=None)), (INVALID, dict(ids=None)),
    (INVALID, dict(w=None)), (INVALID, dict(offsets=None)), (INVALID, dict(rows=None)), (INVALID, dict(slots=None)),
    (INVALID, dict(xs=511)), (INVALID, dict(x=V(0x10002))), (INVALID, dict(dt=BF16, x=V(0x10001))), (INVALID, dict(ids=V(0x20001))),
    (INVALID, dict(offsets=V(0x40002))), (INVALID, dict(T=5000, ws=None)), (INVALID, dict(T=5000, ws=V(0x70008))),
    (INVALID, dict(T=5000, wsb=1000))])
def test_route(lib, want, change):
    assert _call(lib, "gdn_moe_route", ROUTE, ROUTE0, **change) == want


def test_route_workspace(lib):
    f = lib.gdn_moe_route_workspace_size
    f.argtypes, f.restype = [I64, I32], SZ
    assert f(0, 512) == 0
    sizes = [f(t, 512) for t in (1, 600, 20668, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[-1] < 1 << 28


QUANT = dict(x=V, xs=I64, T=I64, n=I32, glu=I32, y=V, ys=I64, s=V, dt=I32, stream=V)
QUANT0 = dict(x=p(1), xs=512, T=4, n=256, glu=0, y=p(2), ys=256, s=p(3), dt=BF16, stream=None)


@pytest.mark.parametrize("want,change", [
    (OK, dict(T=0)), (INVALID, dict(T=-1)), (INVALID, dict(n=0)), (INVALID, dict(dt=E4M3)), (INVALID, dict(x=None)), (INVALID, dict(y=None)),
    (INVALID, dict(s=None)), (INVALID, dict(y=p(1))), (INVALID, dict(s=p(1))), (INVALID, dict(s=p(2))), (INVALID, dict(xs=255)),
    (INVALID, dict(glu=1, xs=511)), (INVALID, dict(ys=255)), (INVALID, dict(x=V(0x10001))), (INVALID, dict(dt=F32, x=V(0x10002))),
    (INVALID, dict(s=V(0x30002))), (UNSUPPORTED, dict(n=(1 << 29) + 1)), (UNSUPPORTED, dict(T=1 << 31))])
def test_block_quant(lib, want, change):
    assert _call(lib, "gdn_block_quant", QUANT, QUANT0, **change) == want


COMBINE = dict(x=V, xs=I64, R=I64, slots=V, w=V, res=V, rs=I64, T=I64, k=I32, H=I32, y=V, ys=I64, dt=I32, stream=V)
COMBINE0 = dict(x=p(1), xs=64, R=40, slots=p(2), w=p(3), res=p(4), rs=64, T=4, k=10, H=64, y=p(5), ys=64, dt=BF16, stream=None)


@pytest.mark.parametrize("want,change", [
    (OK, dict(T=0)), (INVALID, dict(T=-1)), (INVALID, dict(R=-1)), (INVALID, dict(k=0)), (INVALID, dict(H=0)), (INVALID, dict(dt=E4M3)),
    (INVALID, dict(x=None)), (INVALID, dict(slots=None)), (INVALID, dict(w=None)), (INVALID, dict(y=None)), (INVALID, dict(y=p(1))),
    (INVALID, dict(xs=63)), (INVALID, dict(rs=63)), (INVALID, dict(ys=63)), (INVALID, dict(y=p(4), ys=72)), (INVALID, dict(x=V(0x10001))),
    (INVALID, dict(dt=F32, y=V(0x50002))), (INVALID, dict(slots=V(0x20002))), (UNSUPPORTED, dict(R=1 << 31)), (UNSUPPORTED, dict(k=1025)),
    (UNSUPPORTED, dict(T=1 << 30))])
def test_combine(lib, want, change):
    assert _call(lib, "gdn_moe_combine", COMBINE, COMBINE0, **change) == want
