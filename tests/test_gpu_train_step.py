"""One training step of a whole block through the package, as a user strings it together: the
norm before the block, the router (logits from the normed rows), the MoE layer, the norm and
residual behind it, the balance and z losses, every gradient back to the stream, the router
and the experts, and the optimizer's step.  The gradients are compared with the autograd of a
64-bit form of the same block (the router's choices taken from the GPU: they carry no
gradient).

Tolerance.  x, Z = [G, U], A, O, D and dZ are rounded to bf16 between the stages and the 64-bit
form rounds nothing.  One such rounding is a relative error of at most 2^-8, spread evenly: a
standard deviation of about 0.43 2^-8.  About five of them enter an element of a gradient, a
sum of products with random signs, so its error has a standard deviation of
sqrt(5) 0.43 2^-8 = 2^-8 (rounded up) of the size of its terms' sum.  That size is the rms of
its row where the row's own factor (a channel's dZ, a token's gradient) is large, and the rms
of the whole tensor where that factor is itself a sum that cancels, whose error keeps the
common size: 2^-5 max(rms, rms of the row) is eight standard deviations, and 2e-2 |ref| on top
covers the error that goes with the element."""
import pytest
import torch

import train_oracle as R
from skew_aware_token_b200 import native as N
from skew_aware_token_b200 import synth
from skew_aware_token_b200.layer import LayerGraph, MoeLayer
from skew_aware_token_b200.synth import WORKLOADS, Workload
from skew_aware_token_b200.train import AdamW, BlockNorm, RouterLoss

pytestmark = pytest.mark.gpu
DEV = "cuda"
RES, OUT, BAL, ZC = 1.0, 0.7, 0.5, 0.05
CASES = [
    (WORKLOADS["tiny"], None, torch.float32),
    (Workload("ragged", T=515, d=512, E=12, k=4, f=384, beta=128, P=4, s=2, alpha=0.5),
     [0, 100, 100, 480], torch.bfloat16),
]


def within(got, want, what):
    got, want = got.detach().double(), want.detach().double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    rms = float(want.square().mean().sqrt()) or 1.0
    row = want.square().mean(-1, keepdim=True).sqrt().clamp(min=rms)
    over = (got - want).abs() - (2.0 ** -5 * row + 2e-2 * want.abs())
    assert float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3e} (rms {rms:.3e})"


class Block:
    """A block's parameters, its objects and one training step."""

    def __init__(self, wl, seq_off, h_dtype):
        g = torch.Generator(device=DEV)
        g.manual_seed(1)
        n = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=DEV) * scale
        self.wl = wl
        self.w1, self.w2 = synth.make_weights(wl, DEV)
        self.wr = n(wl.E, wl.d, scale=wl.d ** -0.5)
        self.w_in, self.w_out = 1 + n(wl.d, scale=0.1), 1 + n(wl.d, scale=0.1)
        self.gate = torch.rand(wl.T, generator=g, device=DEV) + 0.5
        self.h = n(wl.T, wl.d).to(h_dtype)
        self.G = n(wl.T, wl.d).to(h_dtype)      # gradient of the stream behind the block
        self.seq_off = None if seq_off is None else torch.tensor(seq_off, dtype=torch.int32,
                                                                 device=DEV)
        self.layer = MoeLayer(wl, DEV, train=True, o_rows=True)
        kw = dict(h_dtype=h_dtype, train=True, device=DEV)
        self.norm_in = BlockNorm(wl, **kw)
        self.norm_out = BlockNorm(wl, res_scale=RES, out_scale=OUT, **kw)
        self.router = RouterLoss(wl, n_seq=1 if seq_off is None else len(seq_off) - 1, device=DEV)
        self.dloss = torch.tensor([BAL, ZC], device=DEV)
        self.params = [self.w1, self.w2, self.wr, self.w_in, self.w_out]

    def gradients(self):
        b, layer = self, self.layer
        _, x = b.norm_in(b.h, w_next=b.w_in)
        logits = x.float() @ b.wr.t()
        y = layer(logits, x, b.w1, b.w2)
        losses = b.router(logits, layer.view("topk_ids"), seq_off=b.seq_off)
        h_out, _ = b.norm_out(b.h, y=y, gate=b.gate, w_post=b.w_out)
        g = b.norm_out.backward(h_out, y=y, gate=b.gate, w_post=b.w_out, dh_out=b.G)
        dx, dw1, dw2 = layer.backward(g.dy, b.w1, b.w2)
        dlogits = layer.router_backward(b.router, logits, g.dy, dloss=b.dloss,
                                        seq_off=b.seq_off)
        gin = b.norm_in.backward(b.h, w_next=b.w_in, dh_out=g.dh, dx=dx + dlogits @ b.wr)
        return dict(losses=losses, h_out=h_out, logits=logits, dh=gin.dh, dgate=g.dgate,
                    dlogits=dlogits, dw1=dw1, dw2=dw2, dwr=dlogits.t() @ x.float(),
                    dw_in=gin.dw_next, dw_out=g.dw_post)

    def grads_of(self, r):
        return [r["dw1"], r["dw2"], r["dwr"], r["dw_in"], r["dw_out"]]


def reference(b):
    """The block in 64 bits, its loss <h_out, G> + BAL balance + ZC z, and its gradients."""
    wl, ids = b.wl, b.layer.view("topk_ids").long()
    leaf = {n: t.double().requires_grad_() for n, t in
            dict(h=b.h, w1=b.w1, w2=b.w2, wr=b.wr, w_in=b.w_in, w_out=b.w_out,
                 gate=b.gate).items()}
    x = R.rms_norm(leaf["h"], leaf["w_in"], 1e-6, 0.0)
    logits = x @ leaf["wr"].t()
    logits.retain_grad()
    gates = torch.softmax(logits.gather(1, ids), 1)
    y = torch.zeros_like(x)
    for e in range(wl.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        z = x[t] @ leaf["w1"][e].t()
        a = torch.nn.functional.silu(z[:, :wl.f]) * z[:, wl.f:]
        y = y.index_add(0, t, gates[t, j][:, None] * (a @ leaf["w2"][e].t()))
    h_out, _ = R.block_norm(leaf["h"], y, leaf["gate"], leaf["w_out"], None, res_scale=RES,
                            out_scale=OUT)
    off = None if b.seq_off is None else b.seq_off.tolist()
    host = logits.cpu()
    bal, zl, *_ = R.router_losses(host, ids.cpu(), None, off)
    loss = (h_out * b.G.double()).sum() + (BAL * bal + ZC * zl).to(DEV)
    loss.backward()
    return dict(losses=torch.stack([bal, zl]).to(DEV), h_out=h_out, dh=leaf["h"].grad,
                dgate=leaf["gate"].grad, dlogits=logits.grad, dw1=leaf["w1"].grad,
                dw2=leaf["w2"].grad, dwr=leaf["wr"].grad, dw_in=leaf["w_in"].grad,
                dw_out=leaf["w_out"].grad)


@pytest.mark.parametrize("wl,seq_off,h_dtype", CASES, ids=lambda c: getattr(c, "name", None))
def test_block_gradients(wl, seq_off, h_dtype):
    b = Block(wl, seq_off, h_dtype)
    got = b.gradients()
    torch.cuda.synchronize()
    assert b.layer.read_status() == 0 and b.router.read_status() == 0
    for name, want in reference(b).items():
        within(got[name], want, name)


def test_steps_of_the_optimizer():
    """Three steps of the block's weights with the gradients that the block gives, against the
    64-bit steps on the same gradients.  A step moves a weight by at most 1.001 lr (Cauchy's
    inequality: (sum w_m g)^2 <= sum (w_m^2 / w_v) sum w_v g^2, and sum w_m^2 / w_v <= 1.002 for
    the first three steps' bias-corrected weights at 0.9 and 0.95) and the decay 1e-4 of it, so
    no weight on the way is over |end| + 4 lr in size; each step rounds it once (2^-8 of a bf16
    weight, 2^-24 of an fp32 one) and is itself off by a few 2^-24 of lr."""
    wl, lr = WORKLOADS["tiny"], 1e-3
    b = Block(wl, None, torch.float32)
    opt = AdamW(b.params, lr=lr, betas=(0.9, 0.95), weight_decay=0.1)
    ref = [(p.double(), torch.zeros_like(p, dtype=torch.float64),
            torch.zeros_like(p, dtype=torch.float64)) for p in b.params]
    for step in range(1, 4):
        grads = b.grads_of(b.gradients())
        ref = [R.adamw(p, g.double(), m, v, step, lr, 0.9, 0.95, 1e-8, 0.1)
               for (p, m, v), g in zip(ref, grads)]
        opt.step(grads)
    assert b.layer.read_status() == 0 and opt.steps.tolist()[:2] == [3, 0]
    for got, (want, _, _) in zip(b.params, ref):
        half = 2.0 ** -8 if got.dtype is torch.bfloat16 else 2.0 ** -22
        over = (got.double() - want).abs() - 3 * (half * (want.abs() + 4 * lr) + 2.0 ** -18 * lr)
        assert float(over.max()) <= 0, f"over by {float(over.max()):.3e}"


def test_layer_without_o_rows_refuses_the_router_gradient():
    wl = WORKLOADS["tiny"]
    layer = MoeLayer(wl, DEV, train=True, o_rows=False)
    with pytest.raises(ValueError, match="o_rows"):
        layer.router_backward(RouterLoss(wl, device=DEV), None, torch.zeros(wl.T, wl.d, device=DEV))


def test_router_gradient_after_other_forwards():
    """Refused after a forward that wrote no O rows; a layer that holds an O buffer gives its
    gradient after a call that wrote them; replays of a layer's graph count as its forward."""
    wl = WORKLOADS["tiny"]
    w1, w2 = synth.make_weights(wl, DEV)
    logits, x = synth.make_logits(wl).to(DEV), synth.make_x(wl).to(DEV)
    dy = torch.ones(wl.T, wl.d, device=DEV)
    router = RouterLoss(wl, device=DEV)
    layer = MoeLayer(wl, DEV, train=True, o_rows=True)
    layer(logits, x, w1, w2)
    want = layer.router_backward(router, logits, dy).clone()
    layer(logits, x, w1, w2, mode=N.MOE_FFN_ONE_LAUNCH)
    with pytest.raises(ValueError, match="o_rows"):
        layer.router_backward(router, logits, dy)
    other = MoeLayer(wl, DEV, train=True, write_o=True, o_rows=False)
    other(logits, x, w1, w2, mode=N.MOE_FFN_WRITE_O)
    assert torch.equal(other.router_backward(router, logits, dy), want)
    rows = LayerGraph(layer, w1, w2)
    fused = LayerGraph(layer, w1, w2, mode=N.MOE_FFN_ONE_LAUNCH)
    for g in (rows, fused):
        g.logits.copy_(logits)
        g.x.copy_(x)
    fused.replay()
    with pytest.raises(ValueError, match="o_rows"):
        layer.router_backward(router, logits, dy)
    rows.replay()
    assert torch.equal(layer.router_backward(router, logits, dy), want)
    torch.cuda.synchronize()
    assert layer.read_status() == 0 and other.read_status() == 0


def test_block_gradients_replayed_from_a_graph():
    """The whole of the block's forward and backward captured once, replayed on a new stream
    (x) and new experts, gives the eager call's results (sums by atomics within the last
    bits: the experts' dx)."""
    b = Block(WORKLOADS["tiny"], None, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            b.gradients()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.gradients()
    for _ in range(2):
        b.h.normal_()
        b.w2.mul_(0.5)
        graph.replay()
        replayed = {n: t.clone() for n, t in got.items()}
        eager = b.gradients()
        torch.cuda.synchronize()
        for n, t in replayed.items():
            rms = float(eager[n].double().square().mean().sqrt())
            close = (t.double() - eager[n].double()).abs() <= 2.0 ** -12 * rms + 2.0 ** -8 * \
                eager[n].double().abs()
            assert bool(close.all()), n
    assert b.layer.read_status() == 0
