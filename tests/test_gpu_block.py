"""The block around the layer as a serving step runs it, in 8 bits and in bf16:
residual addition and RMSNorm, the projections into the q|k|v stream, z and the
gate inputs (columns of one buffer as the layer's strided inputs), the layer
(prefill of a ragged batch, then a decode step that continues its states), the
gated RMSNorm, the output projection back onto the residual stream in place.
Every stage is held to 64 bits (the layer to the oracle) on the inputs that it
got, and a captured graph of the whole block to the eager call's bits."""
import pytest
import torch

import oracle
import workloads
from tests import block64 as b64
from tests.gpu_common import DEV, gdn, oracle_gating, status_clean
from tests.util import TOL, assert_close, bits_equal, to_np

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, b64.E4M3
HQK, HV, HIDDEN, EPS = 2, 4, 320, 1e-6
C, V = 2 * HQK * 128 + HV * 128, HV * 128


class Block:
    def __init__(self, eight, seed=5):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.eight = eight
        self.w_norm, self.w_out_norm = r(HIDDEN) * 0.1, torch.rand(128, generator=g) + 0.5
        # one projection for q|k|v and z, one each for the gate inputs a and b
        self.w = {k: self._weight(r(n, m) * m ** -0.5) for k, n, m in
                  (("qkvz", C + V, HIDDEN), ("a", HV, HIDDEN), ("b", HV, HIDDEN), ("out", HIDDEN, V))}
        self.conv_w = workloads.conv_weight(g, C, 4, BF16).to(DEV)
        self.A_log, self.dt_bias = (t.to(DEV) for t in workloads.gating_params(g, HV))
        self.w_norm, self.w_out_norm = self.w_norm.to(DEV), self.w_out_norm.to(DEV)
        self.conv_pool = torch.zeros(8, 3, C, dtype=BF16, device=DEV)
        self.pool = torch.zeros(8, HV, 128, 128, device=DEV)

    def _weight(self, w):
        if self.eight:
            q, s = b64.quantise(w.to(DEV))
            return q, s
        return w.to(BF16).to(DEV), None

    def project(self, key, x, scale, **kw):
        w, sw = self.w[key]
        return gdn().gdn_linear(x, w, x_scale=scale, weight_scale=sw, **kw)

    def __call__(self, x, stream, layer):
        """x [T, HIDDEN] the last block's output, stream the residual (updated in place)."""
        G, T = gdn(), x.shape[0]
        n, ns, _ = G.gdn_add_rmsnorm(x, self.w_norm, residual=stream, eps=EPS, weight_offset=1.0,
                                     y_dtype=E4M3 if self.eight else None, residual_out=stream)
        added = stream.clone()
        wide = self.project("qkvz", n, ns)
        a, b = self.project("a", n, ns), self.project("b", n, ns)
        o = layer(self, wide[:, :C], a, b)
        z = wide[:, C:]
        if self.eight:
            y, ys = G.gdn_gated_rmsnorm_quant(o, z, self.w_out_norm, eps=EPS)
        else:
            y, ys = G.gdn_gated_rmsnorm(o, z.unflatten(1, (HV, 128)), self.w_out_norm, eps=EPS), None
        self.project("out", y.view(T, V), ys, residual=stream, y=stream)
        return dict(n=n, ns=ns, added=added, wide=wide, a=a, b=b, o=o, y=y, ys=ys, stream=stream.clone())

    def check(self, x, before, s):
        """Every stage but the layer against 64 bits on its own inputs."""
        T = x.shape[0]
        total, ref = b64.add_rmsnorm(x, before, self.w_norm, EPS, 1.0)
        b64.check_near(s["added"], total, 2.0 ** -24, b64.HALF[BF16], "stream")
        if self.eight:
            b64.check_quant(s["n"], s["ns"], ref, b64.NORM, "norm")
        else:
            b64.check_near(s["n"], ref, b64.NORM, b64.HALF[BF16], "norm")
        for key, got in (("qkvz", s["wide"]), ("a", s["a"]), ("b", s["b"])):
            w, sw = self.w[key]
            b64.check_linear(got, *b64.linear(s["n"], w, s["ns"], sw, None, "none", None), HIDDEN, self.eight, key)
        z = s["wide"][:, C:].unflatten(1, (HV, 128))
        ref = b64.gated_norm(s["o"], z, self.w_out_norm, EPS)
        if self.eight:
            b64.check_quant(s["y"], s["ys"], ref.reshape(T, -1), b64.GATED, "gated norm")
        else:
            assert_close(s["y"], ref.cpu(), TOL[BF16], "gated norm")
        w, sw = self.w["out"]
        b64.check_linear(s["stream"], *b64.linear(s["y"].view(T, V), w, s["ys"], sw, None, "none", s["added"]), V,
                         self.eight, "out")


def _inputs(seed, T):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, HIDDEN, generator=g).to(BF16).to(DEV),
            (3 * torch.randn(T, HIDDEN, generator=g)).to(BF16).to(DEV))


@pytest.mark.parametrize("eight", [True, False])
def test_prefill_then_decode(eight):
    lens = [70, 1, 130, 0, 64]
    n, T = len(lens), sum(lens)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device=DEV)
    slots = torch.tensor([3, 0, 5, 1, 7], dtype=torch.int32, device=DEV)
    fresh, none = torch.zeros(n, dtype=torch.uint8, device=DEV), torch.full_like(slots, -1)
    block = Block(eight)

    def prefill(bl, x, a, b):
        return gdn().gdn_prefill_layer(x, bl.conv_w, bl.conv_pool, slots, fresh, a, b, bl.A_log, bl.dt_bias, cu, HQK,
                                       bl.pool, none, slots)

    x, stream = _inputs(11, T)
    before = stream.clone()
    s = block(x, stream, prefill)
    torch.cuda.synchronize()
    status_clean()
    block.check(x, before, s)
    cpu = lambda t: t.contiguous().cpu()  # noqa: E731
    o_ref = oracle.layer_prefill(cpu(s["wide"][:, :C]), cpu(cu), cpu(block.conv_w), None, torch.zeros(8, 3, C),
                                 cpu(block.A_log), cpu(block.dt_bias), cpu(s["a"]), cpu(s["b"]),
                                 torch.zeros(8, HV, 128, 128), cpu(slots), cpu(fresh), HQK, HV, 128, 128,
                                 128 ** -0.5)[0]
    assert_close(s["o"], o_ref, TOL[BF16], "layer")

    # one more token of each sequence, continuing the states; a row without a slot
    dslots = torch.tensor([3, 0, 5, -1, 7], dtype=torch.int32, device=DEV)

    def decode(bl, x, a, b):
        return gdn().gdn_decode_step_fused(x, bl.conv_w, bl.conv_pool, a, b, bl.A_log, bl.dt_bias, HQK, bl.pool, dslots)

    conv0, pool0 = block.conv_pool.clone(), block.pool.clone()
    x, stream = _inputs(12, n)
    before = stream.clone()
    s = block(x, stream, decode)
    torch.cuda.synchronize()
    status_clean()
    block.check(x, before, s)
    assert torch.all(s["o"][3] == 0)
    idx = to_np(dslots).astype(int)
    y, _ = oracle.conv1d_update(to_np(s["wide"][:, :C]), 1, to_np(block.conv_w), None, to_np(conv0), idx)
    q, k, v = oracle.split_qkv(y, HQK, HV, 128, 128)
    g, beta = oracle_gating(s["a"], s["b"], block.A_log, block.dt_bias)
    o_ref, _ = oracle.gdn_decode(q, k, v, g, beta, 1, to_np(pool0), idx, scale=128 ** -0.5)
    live = [0, 1, 2, 4]
    assert_close(s["o"][live], o_ref[live], TOL[BF16], "decode layer")


@pytest.mark.parametrize("eight", [True, False])
def test_decode_block_in_a_graph(eight):
    """Captured once, replayed on new inputs and states: the bits of the eager call."""
    n = 6
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    block = Block(eight)
    ws = torch.empty(gdn().gdn_decode_step_workspace_size(n, HQK, HV), dtype=torch.uint8, device=DEV)

    def decode(bl, x, a, b):
        return gdn().gdn_decode_step_fused(x, bl.conv_w, bl.conv_pool, a, b, bl.A_log, bl.dt_bias, HQK, bl.pool, slots,
                                           workspace=ws)

    x, stream = _inputs(21, n)
    block(x, stream, decode)                       # warm-up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, stream, decode)
    for seed in (22, 23):
        nx, ns = _inputs(seed, n)
        g = torch.Generator().manual_seed(seed)
        conv = torch.randn(8, 3, C, generator=g).to(BF16).to(DEV)
        pool = (torch.randn(8, HV, 128, 128, generator=g) * 0.02).to(DEV)
        res = []
        for replay in (False, True):
            x.copy_(nx)
            stream.copy_(ns)
            block.conv_pool.copy_(conv)
            block.pool.copy_(pool)
            if replay:
                graph.replay()
                s = got
            else:
                s = block(x, stream, decode)
            torch.cuda.synchronize()
            res.append([s["stream"].clone(), s["o"].clone(), block.pool.clone(), block.conv_pool.clone()])
        assert all(bits_equal(p, q) for p, q in zip(*res))
    status_clean()
