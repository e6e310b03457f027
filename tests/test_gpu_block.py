"""The operators of a served MoE block run together, as they are used: norm, a projection with the requests'
adapters, the residual join with the next norm, the MoE layer under a routing rule, the closing join.
Every step is checked against the plain 64-bit evaluation of what the step before left, and the
whole run captured into a graph gives the same bits."""
import numpy as np
import pytest

import lora_ref
import mx4_ref
import norm_ref
import rule_ref
from gpu_util import to_dev
from test_gpu_mx4_moe import check as check_layer
from test_gpu_mx4_moe import upload

pytestmark = pytest.mark.gpu

H, I, E, K = 256, 128, 24, 3
RULE = dict(score="sigmoid", n_groups=4, group_top_k=2, group_score="top2", scale=2.5)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm device"
    return t


@pytest.fixture(scope="module")
def qs():
    import quantized_sparse_moe_amd as q
    q.lib()
    return q


def np64(t):
    return t.double().cpu().numpy()


class Block:
    """Weights of one block and the buffers of T tokens."""

    def __init__(self, torch, qs, T):
        self.torch, self.qs, self.T = torch, qs, T
        g = torch.Generator().manual_seed(7)
        rnd = lambda *s: torch.randn(*s, generator=g)
        bias = (0.1 * rnd(E)).numpy()
        self.layer = rule_ref.RuledLayer(dict(RULE, select_bias=bias), seed=2, hidden=H, inter=I, n_experts=E, top_k=K,
                                         gated=True)
        self.desc = upload(self.layer, torch, qs)
        self.rule = qs.RouterRule(**RULE, select_bias=torch.from_numpy(bias).cuda())
        w = lambda: (1 + 0.2 * rnd(H)).bfloat16().cuda()
        self.w = [w() for _ in range(4)]
        self.n = [qs.Norm(weight=x, eps=1e-5) for x in self.w]
        self.proj = rnd(H, H) / H ** 0.5
        self.pc, self.ps = qs.mx4_quantize(self.proj.cuda())
        self.a = (rnd(5, 16, H) / H ** 0.5).bfloat16().cuda()
        self.b = (rnd(5, H, 16) / 4).bfloat16().cuda()
        self.scales = (rnd(5) + 1.5).cuda()
        self.ad = qs.LoraAdapters(self.a, self.b, scales=self.scales)
        self.ids = torch.randint(-1, 5, (T,), generator=g, dtype=torch.int32).cuda()
        self.stream = rnd(T, H).cuda()
        self.gate = rnd(T).cuda()
        self.ws = qs.new_workspace(self.desc, T)
        self.gws = qs.mx4_new_workspace(T, H, H)
        self.aws = qs.lora_new_workspace(self.ad, T)
        self.idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
        self.wt = torch.empty(T, K, device="cuda")

    def run(self):
        qs, bf = self.qs, self.torch.bfloat16
        _, x1 = qs.moe_block_norm(residual=self.stream, pre=self.n[0], x_dtype=bf)
        p = qs.mx4_gemm(self.pc, self.ps, H, H, x1, y_dtype=bf, workspace=self.gws, adapters=self.ad, adapter_ids=self.ids,
                        adapter_workspace=self.aws)
        r1, x2 = qs.moe_block_norm(p, residual=self.stream, post=self.n[1], scale=0.5, pre=self.n[2], x_dtype=bf)
        y = qs.moe_layer_forward(self.desc, x2, y_dtype=bf, topk_idx=self.idx, topk_w=self.wt, workspace=self.ws, rule=self.rule)
        r2, x3 = qs.moe_block_norm(y, residual=r1, gate=self.gate, gate_act="sigmoid", pre=self.n[3], x_dtype=bf)
        return x1, p, r1, x2, y, r2, x3


def check_norm(b, y, r, post, gate, act, scale, pre, outs):
    e = lambda i: None if i is None else dict(kind="rms", eps=float(np.float32(1e-5)), offset=0.0, weight=np64(b.w[i]), bias=None)
    (t, bt), (v, bv) = norm_ref.block(None if y is None else np64(y), np64(r), e(post), gate, act, scale, e(pre))
    for got, want, bound, name in ((outs[0], t, bt, "f32"), (outs[1], v, bv, "bf16")):
        if got is not None:
            assert (np.abs(np64(got) - want) <= norm_ref.rounded(want, bound, name)).all()


@pytest.mark.parametrize("T", [1, 7, 40, 200])
def test_block(torch, qs, T):
    b = Block(torch, qs, T)
    x1, p, r1, x2, y, r2, x3 = b.run()
    check_norm(b, None, b.stream, None, None, "none", 1.0, 0, (None, x1))
    # the projection rounded to bf16, then the adapters
    y0 = qs.mx4_gemm(b.pc, b.ps, H, H, x1, y_dtype=torch.bfloat16)
    want, bound = lora_ref.forward(np64(b.a), np64(b.b), b.ids.cpu().numpy(), np64(x1), np64(y0), np64(b.scales))
    lora_ref.check(np64(p), want, bound, True)
    check_norm(b, p, b.stream, 1, None, "none", 0.5, 2, (r1, x2))
    check_layer(b.layer, x2.view(torch.int16).cpu().numpy().view(np.uint16), y, b.idx, b.wt, T)
    check_norm(b, y, r1, None, np64(b.gate)[:, None], "sigmoid", 1.0, 3, (r2, x3))


@pytest.mark.parametrize("T", [1, 40, 200])
def test_block_in_a_graph(torch, qs, T):
    b, own = Block(torch, qs, T), Block(torch, qs, T)
    b.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.run()
    for seed in range(4):
        torch.manual_seed(seed)
        b.stream.copy_(torch.randn(T, H))
        b.ids.copy_(torch.randint(-1, 5, (T,), dtype=torch.int32))
        own.stream.copy_(b.stream)
        own.ids.copy_(b.ids)
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, own.run()):
            assert torch.equal(got, want)
        assert torch.equal(b.idx, own.idx) and torch.equal(b.wt, own.wt)
    assert int(qs.moe_workspace_status(b.ws)) == 0


def test_two_blocks_on_two_streams(torch, qs):
    """With workspaces of their own, calls on two streams at once leave what each leaves alone."""
    one, two = Block(torch, qs, 40), Block(torch, qs, 7)
    want = [t.clone() for t in one.run()], [t.clone() for t in two.run()]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            a = one.run()
        with torch.cuda.stream(t):
            c = two.run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, want[0])) and all(torch.equal(x, y) for x, y in zip(c, want[1]))
