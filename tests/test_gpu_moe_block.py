"""The mixture-of-experts MLP of a block as a serving step runs it, in bf16 and in
8 bits: norm, router logits, router, the experts' gate and up products on gathered
rows, their gated activation, the down products, the combination onto the residual
stream.  Every stage is held to 64 bits on the inputs that it got, and a captured
graph of the whole to the eager call's bits."""
import pytest
import torch

from tests import block64 as b64
from tests import moe64 as m64
from tests.gpu_common import DEV, gdn, status_clean
from tests.util import bits_equal

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, b64.E4M3
HIDDEN, INNER, EXPERTS, TOP, EPS = 320, 192, 24, 5, 1e-6


class Mlp:
    def __init__(self, eight):
        g = torch.Generator(device=DEV).manual_seed(11)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.eight = eight
        self.norm = r(HIDDEN) * 0.1
        self.router = r(EXPERTS, HIDDEN).mul(HIDDEN ** -0.5).to(BF16)
        self.up = self._weight(r(EXPERTS, 2 * INNER, HIDDEN) * HIDDEN ** -0.5)
        self.down = self._weight(r(EXPERTS, HIDDEN, INNER) * INNER ** -0.5)

    def _weight(self, w):
        if not self.eight:
            return w.to(BF16), None
        q, s = m64.quantise_blocks(w, 128)
        return m64.padded(q, 0.0), s.contiguous()

    def __call__(self, x, stream):
        G = gdn()
        n, _, _ = G.gdn_add_rmsnorm(x, self.norm, residual=stream, eps=EPS, weight_offset=1.0, residual_out=stream)
        before = stream.clone()
        logits = G.gdn_linear(n, self.router, y_dtype=F32)
        ids, weights, offsets, rows, slots = G.gdn_moe_route(logits, TOP)
        a, sa = G.gdn_block_quant(n) if self.eight else (n, None)
        h = G.gdn_grouped_linear(a, self.up[0], offsets, rows=rows, x_scale=sa, weight_scale=self.up[1])
        if self.eight:
            b, sb = G.gdn_block_quant(h, glu=True)
        else:
            b, sb = (torch.nn.functional.silu(h[:, :INNER].float()) * h[:, INNER:].float()).to(BF16), None
        d = G.gdn_grouped_linear(b, self.down[0], offsets, x_scale=sb, weight_scale=self.down[1])
        G.gdn_moe_combine(d, slots, weights, residual=stream, y=stream)
        return dict(n=n, before=before, logits=logits, ids=ids, weights=weights, offsets=offsets, rows=rows, slots=slots,
                    a=a, sa=sa, h=h, b=b, sb=sb, d=d, out=stream.clone())

    def check(self, s):
        w64 = m64.route(s["logits"], TOP, True)
        for key, want in zip(("ids", "", "offsets", "rows", "slots"), w64):
            assert not key or torch.equal(s[key].cpu(), want), key
        m64.check_weights(s["weights"], w64[1], s["logits"], w64[0])
        b64.check_linear(s["logits"], *b64.linear(s["n"], self.router, None, None, None, "none", None), HIDDEN)
        if self.eight:
            m64.check_block_quant(s["a"], s["sa"], s["n"].double(), 4 * 2.0 ** -24, "quant")
            m64.check_block_quant(s["b"], s["sb"], m64.glu(s["h"]), b64.GATED, "glu")
        m64.check_product(s["h"], *m64.grouped(s["a"], self.up[0], s["offsets"], s["rows"], s["sa"], self.up[1]), HIDDEN,
                          self.eight, "up")
        m64.check_product(s["d"], *m64.grouped(s["b"], self.down[0], s["offsets"], None, s["sb"], self.down[1]), INNER,
                          self.eight, "down")
        m64.check_combine(s["out"], *m64.combine(s["d"], s["slots"], s["weights"], s["before"]), TOP, "combine")


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [1, 3, 64, 300, 1500])
def test_mlp(T, eight):
    mlp = Mlp(eight)
    g = torch.Generator(device=DEV).manual_seed(T)
    r = lambda: torch.randn(T, HIDDEN, generator=g, device=DEV).to(BF16)  # noqa: E731
    x, stream = r(), r()
    start = stream.clone()
    s = mlp(x, stream)
    torch.cuda.synchronize()
    status_clean()
    mlp.check(s)
    # a captured graph of the block, replayed on the same inputs and on others
    buf = start.clone()
    mlp(x, buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = mlp(x, buf)
    buf.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    for key in s:
        if s[key] is not None:
            assert bits_equal(t[key].float(), s[key].float()), key
    x.copy_(r())
    graph.replay()
    torch.cuda.synchronize()
    status_clean()
    mlp.check(t)
