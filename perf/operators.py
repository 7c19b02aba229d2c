"""The operators that train the block around the expert computation, as measured cases: the
router's balance loss, the router's gradient, the norms before and after the block with its
gate and residual scale, and the AdamW step.

`run` makes one pass through an operator: in plain torch, or with `own` set through this
package.  Sizes are those of this repository's layers (256 tokens of width 512 over 8
experts up to 16384 tokens of width 7168 over 256), with ragged ones between them.
"""
import math

import torch

own = False

DEV = "cuda"
BETA = 128                   # rows per token block of the dispatched rows
NORM_EPS = 1e-6
RES_SCALE, OUT_SCALE = 1.0, 0.7
LR, BETA1, BETA2, ADAM_EPS, WD = 1e-3, 0.9, 0.95, 1e-8, 0.1
STEPS_BEFORE = 10            # steps that the optimizer's states stand for
BLOCK = 256                  # elements that share one scale of an 8-bit state
E4M3_MAX, E4M3_TINY = 448.0, 2.0 ** -9
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest layer's router: latency is all there is
        dict(name="balance_tiny", op="balance", T=256, E=8, k=2, n_seq=1, masked=False),
        # the 128-expert layer on a packed batch: sequences of different lengths, masked
        # tokens inside them, padding behind the last one
        dict(name="balance_packed", op="balance", T=16384, E=128, k=8, n_seq=24, masked=True),
        # an odd small layer on a packed batch
        dict(name="router_grad_ragged", op="router_grad", T=1111, d=512, E=12, k=4, n_seq=3,
             masked=True),
        # the largest layer: the gates' gradient reads every expert output row
        dict(name="router_grad_wide", op="router_grad", T=16384, d=7168, E=256, k=8, n_seq=4,
             masked=False),
        # serving: a single token at the largest width; post-norm, residual, next pre-norm
        dict(name="norm_token", op="norm", T=1, d=7168, h="bf16", w="bf16", gate=False),
        # the 64-expert layer with a bf16 residual stream and a gate for each token
        dict(name="norm_mid", op="norm", T=4096, d=2048, h="bf16", w="f32", gate=True),
        # the largest layer with an fp32 residual stream
        dict(name="norm_wide", op="norm", T=16384, d=7168, h="f32", w="f32", gate=False),
        # odd token count and width, backward
        dict(name="norm_grad_ragged", op="norm_grad", T=1111, d=1000, h="f32", w="f32",
             gate=True),
        # the largest layer's backward with a bf16 residual stream
        dict(name="norm_grad_wide", op="norm_grad", T=16384, d=7168, h="bf16", w="bf16",
             gate=True),
        # many small tensors of odd sizes in one step, bf16 weights with fp32 masters
        dict(name="adamw_many", op="adamw", n=120, size=20011, bits=32, p="bf16", grad="f32",
             master=True),
        # per-expert fp32 tensors with fp32 states and bf16 gradients
        dict(name="adamw_f32", op="adamw", n=24, size=2048 * 1024, bits=32, p="f32",
             grad="bf16", master=False),
        # the 64-expert layer's weights (gate, up and down halves) with 8-bit states
        dict(name="adamw_experts_8bit", op="adamw", n=3, size=64 * 2048 * 1024, bits=8,
             p="bf16", grad="f32", master=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["balance", "router_grad", "norm", "norm_grad", "adamw"])
    if op in ("balance", "router_grad"):
        E = _spread(rng, 2, 256)
        k = rng.randint(1, min(E, 8))
        T = _spread(rng, 1, 16384)
        c = dict(op=op, T=T, E=E, k=k, n_seq=_spread(rng, 1, min(T, 48)),
                 masked=rng.random() < 0.5)
        if op == "router_grad":
            c["d"] = 8 * _spread(rng, 8, 896)
        return c
    if op in ("norm", "norm_grad"):
        return dict(op=op, T=_spread(rng, 1, 16384), d=8 * _spread(rng, 8, 896),
                    h=rng.choice(["bf16", "f32"]), w=rng.choice(["bf16", "f32"]),
                    gate=rng.random() < 0.5)
    n = _spread(rng, 1, 300)
    size = _spread(rng, 100, min(1 << 24, (1 << 26) // n))
    p = rng.choice(["bf16", "f32"])
    return dict(op=op, n=n, size=size, bits=rng.choice([8, 32]), p=p,
                grad=rng.choice(["bf16", "f32"]), master=p == "bf16" and rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype=torch.float32, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return x if scale == 1.0 else x.mul_(scale)


def _sequences(case, g):
    """seq_off [n_seq + 1] (None: the whole batch is one sequence) and token_mask (None: all
    count).  Packed batches leave about a twentieth of the rows behind the last sequence;
    cuts may coincide (an empty sequence)."""
    T, S = case["T"], case["n_seq"]
    off = mask = None
    if S > 1 or case["masked"]:
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV)
        end = T - T // 20 if case["masked"] else T
        off = torch.cat([torch.zeros(1, device=DEV, dtype=torch.int64),
                         cuts.clamp(max=end).sort().values,
                         torch.full((1,), end, device=DEV, dtype=torch.int64)]).int()
    if case["masked"]:
        mask = (torch.rand(T, generator=g, device=DEV) > 0.1).to(torch.uint8)
    return off, mask


def _router(case, g):
    """Skewed router logits with their top-k choices and gates, as the router gives them."""
    T, E, k = case["T"], case["E"], case["k"]
    rank = torch.arange(1, E + 1, device=DEV, dtype=torch.float32)
    logits = _normal((T, E), g) - rank.log()
    top, ids = logits.topk(k, dim=1)
    gates = torch.softmax(top, dim=1)
    off, mask = _sequences(case, g)
    return dict(logits=logits, topk_ids=ids.int().contiguous(), topk_gates=gates.contiguous(),
                seq_off=off, token_mask=mask)


def _rows_of(ids, E):
    """The padded row of every (token, choice) pair in expert-major, block-aligned order, and
    the row bound."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    order = flat.argsort(stable=True)
    counts = torch.bincount(flat, minlength=E)
    first = (counts.cumsum(0) - counts)[flat[order]]
    blocks = (counts + BETA - 1) // BETA
    base = (BETA * (blocks.cumsum(0) - blocks))[flat[order]]
    tok_row = torch.empty_like(flat)
    tok_row[order] = base + torch.arange(n, device=DEV) - first
    return tok_row.int().view(ids.shape), (n + min(E, n) * (BETA - 1)) // BETA * BETA


def _workload(case):
    from skew_aware_token_b200.synth import Workload
    return Workload(case.get("name", case["op"]), T=case["T"], d=case.get("d", 256),
                    E=case.get("E", 1), k=case.get("k", 1), f=128, beta=BETA, P=1, s=0)


def _sizes(case):
    return [case["size"] - 13 * (i % 7) for i in range(case["n"])]


def _up(n):
    return -(-n // BLOCK) * BLOCK


def _prepare_adamw(case, g):
    """Flat storage with every tensor on a block boundary; what pads a tensor stays zero."""
    sizes = _sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n))
    total = starts[-1]
    real = torch.ones(total, device=DEV, dtype=torch.bool)
    for n, at, end in zip(sizes, starts, starts[1:]):
        real[at + n:end] = False
    values = _normal((total,), g, scale=0.02).mul_(real)
    s = dict(case=case, sizes=sizes, starts=starts, step=STEPS_BEFORE)
    s["p"] = values.to(TYPES[case["p"]])
    s["master"] = values if case["master"] else None
    s["grad"] = _normal((total,), g, scale=1e-3).mul_(real).to(TYPES[case["grad"]])
    m = _normal((total,), g, scale=3e-4).mul_(real)
    r = _normal((total,), g, scale=1e-3).abs_().add_(1e-4).mul_(real)
    if case["bits"] == 8:
        s["m"], s["m_scale"] = _to_8bit(m, False)
        s["v"], s["v_scale"] = _to_8bit(r, True)
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, r.square_(), None, None
    if own:
        from skew_aware_token_b200.train import AdamW
        cut = lambda x, q=1: None if x is None else [  # noqa: E731
            x[at // q:at // q + -(-n // q)] for n, at in zip(sizes, starts)]
        s["opt"] = AdamW(cut(s["p"]), lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
                         weight_decay=WD, state_bits=case["bits"], master=cut(s["master"]),
                         m=cut(s["m"]), v=cut(s["v"]), m_scale=cut(s["m_scale"], BLOCK),
                         v_scale=cut(s["v_scale"], BLOCK), step=STEPS_BEFORE)
        s["grads"] = cut(s["grad"])
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(case, g)
    s = dict(case=case)
    if op in ("balance", "router_grad"):
        s.update(_router(case, g))
        if op == "router_grad":
            T, d = case["T"], case["d"]
            s["tok_row"], rows = _rows_of(s["topk_ids"], case["E"])
            s["o"] = _normal((rows, d), g, torch.bfloat16)
            s["dy"] = _normal((T, d), g, scale=1e-2)
            s["dloss"] = torch.tensor([1e-2 * T, 1e-3 * T], device=DEV)
            s["saved"] = _balance(s)
        if own:
            from skew_aware_token_b200.train import RouterLoss
            s["router"] = RouterLoss(_workload(case), n_seq=case["n_seq"], device=DEV)
            if op == "router_grad":   # the forward whose gradient is taken
                s["router"](s["logits"], s["topk_ids"], s["token_mask"], s["seq_off"])
        return s
    T, d, ht, wt = case["T"], case["d"], TYPES[case["h"]], TYPES[case["w"]]
    s["h"] = _normal((T, d), g).to(ht)          # backward: the stream behind the block
    s["y"] = _normal((T, d), g, scale=0.5)
    s["gate"] = torch.rand(T, generator=g, device=DEV) if case["gate"] else None
    s["w_post"] = (1 + _normal((d,), g, scale=0.1)).to(wt)
    s["w_next"] = (1 + _normal((d,), g, scale=0.1)).to(wt)
    if op == "norm_grad":
        s["dh_out"] = _normal((T, d), g, scale=1e-2).to(ht)
        s["dx"] = _normal((T, d), g, scale=1e-2)
    if own:
        from skew_aware_token_b200.train import BlockNorm
        s["norm"] = BlockNorm(_workload(case), h_dtype=ht, w_dtype=wt, eps=NORM_EPS,
                              res_scale=RES_SCALE, out_scale=OUT_SCALE,
                              train=op == "norm_grad", device=DEV)
    return s


# ------------------------------------------------------------------------- plain forms
def _counted(s):
    """Of each token: its sequence, and whether it counts."""
    c = s["case"]
    T, S = c["T"], c["n_seq"]
    off = s["seq_off"]
    if off is None:
        off = torch.tensor([0, T], device=DEV)
    t = torch.arange(T, device=DEV)
    seq = torch.bucketize(t, off[1:].long(), right=True)
    on = (t >= off[0]) & (seq < S)
    if s["token_mask"] is not None:
        on &= s["token_mask"] != 0
    return seq.clamp(max=S - 1), on


def _balance(s):
    c = s["case"]
    E, k, S = c["E"], c["k"], c["n_seq"]
    seq, on = _counted(s)
    x, ids = s["logits"], s["topk_ids"].long()
    top = x.amax(1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    lse = torch.where(on, (top + total.log()).squeeze(1), 0.0)
    p = torch.where(on[:, None], e / total, 0.0)
    n_s = torch.zeros(S, device=DEV, dtype=torch.float64).index_add_(0, seq, on.double())
    prob = torch.zeros(S, E, device=DEV, dtype=torch.float64).index_add_(0, seq, p.double())
    prob = prob / n_s.clamp(min=1)[:, None]
    pair = (seq[:, None] * E + ids).reshape(-1)
    counts = torch.zeros(S * E, device=DEV, dtype=torch.int32).index_add_(
        0, pair, on[:, None].expand(-1, k).reshape(-1).int()).view(S, E)
    seqs, n = (n_s > 0).sum().clamp(min=1), n_s.sum().clamp(min=1)
    per_seq = (counts * prob).sum(1) * E / (k * n_s.clamp(min=1))
    losses = torch.stack([per_seq.sum() / seqs, lse.double().square().sum() / n]).float()
    return dict(losses=losses, counts=counts, probs=prob.float(), lse=lse)


def _router_grad(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    ids = s["topk_ids"].long()
    seq, on = _counted(s)
    n_s = torch.zeros(c["n_seq"], device=DEV).index_add_(0, seq, on.float())
    seqs, n = (n_s > 0).sum().clamp(min=1), n_s.sum().clamp(min=1)
    counts, lse = s["saved"]["counts"], s["saved"]["lse"]
    a = s["dloss"][0] * E * counts / (seqs * k * n_s.clamp(min=1)[:, None] ** 2)
    a = a[seq]
    p = torch.where(on[:, None], (s["logits"] - lse[:, None]).exp(), 0.0)
    z = s["dloss"][1] * 2 / n * lse
    dlogits = p * (a - (a * p).sum(1, keepdim=True) + z[:, None])
    rows = s["o"][s["tok_row"].long().reshape(-1)].float().view(*ids.shape, -1)
    dgates = (rows * s["dy"][:, None, :]).sum(-1)
    g = s["topk_gates"]
    dlogits.scatter_add_(1, ids, g * (dgates - (g * dgates).sum(1, keepdim=True)))
    return dict(dlogits=dlogits, dgates=dgates)


def _rms(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + NORM_EPS)


def _norm(s):
    h, y, w_post, w_next = (s[n].float() for n in ("h", "y", "w_post", "w_next"))
    out = y * _rms(y) * w_post * OUT_SCALE
    if s["gate"] is not None:
        out = out * s["gate"][:, None]
    h = h * RES_SCALE + out
    x = h * _rms(h) * w_next
    return dict(h_out=h.to(s["h"].dtype), x=x.to(torch.bfloat16))


def _norm_grad(s):
    h, y, w_post, w_next, dh, dx = (s[n].float() for n in ("h", "y", "w_post", "w_next",
                                                           "dh_out", "dx"))
    d = h.shape[1]
    rh, ry = _rms(h), _rms(y)
    q = dx * w_next
    u = dh + rh * (q - h * (rh * rh) * ((q * h).sum(1, keepdim=True) / d))
    ny = y * ry
    g = s["gate"][:, None] if s["gate"] is not None else torch.ones_like(ry)
    q = u * w_post
    dy = OUT_SCALE * g * ry * (q - y * (ry * ry) * ((q * y).sum(1, keepdim=True) / d))
    dgate = OUT_SCALE * (q * ny).sum(1) if s["gate"] is not None else None
    return dict(dh=(RES_SCALE * u).to(s["h"].dtype), dy=dy, dgate=dgate,
                dw_post=(OUT_SCALE * g * u * ny).sum(0), dw_next=(dx * h * rh).sum(0))


def _to_8bit(x, root):
    """Blocks of BLOCK values as e4m3 with one scale each; a positive root keeps a code above
    zero, so that no element's denominator vanishes."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1)
    scale = top * torch.tensor(1 / E4M3_MAX, device=x.device)
    inv = torch.where(top > 0, E4M3_MAX * torch.reciprocal(top), 0.0)
    c = x * inv[:, None]
    if root:
        c = torch.where(x > 0, c.clamp(min=E4M3_TINY), c)
    return c.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1), scale


def _of_8bit(c, scale):
    return (c.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    c = s["case"]
    s["step"] += 1
    g = s["grad"].float()
    if c["bits"] == 8:
        m, r = _of_8bit(s["m"], s["m_scale"]), _of_8bit(s["v"], s["v_scale"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * (1 - BETA2) * g
    c1, c2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    root = v.sqrt()
    p = (s["p"] if s["master"] is None else s["master"]).float()
    p = p * (1 - LR * WD) - (LR / c1) * m / (root * (1 / math.sqrt(c2)) + ADAM_EPS)
    if c["bits"] == 8:
        m, m_scale = _to_8bit(m, False)
        v, v_scale = _to_8bit(root, True)
        s["m_scale"].copy_(m_scale)
        s["v_scale"].copy_(v_scale)
    s["m"].copy_(m)
    s["v"].copy_(v)
    s["p"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {n: s[n] for n in ("p", "master", "m", "v", "m_scale", "v_scale")}


PLAIN = dict(balance=_balance, router_grad=_router_grad, norm=_norm, norm_grad=_norm_grad,
             adamw=_adamw)


def _run_own(s):
    op = s["case"]["op"]
    if op == "balance":
        r = s["router"]
        r(s["logits"], s["topk_ids"], s["token_mask"], s["seq_off"])
        return dict(losses=r.losses, counts=r.counts, probs=r.probs, lse=r.lse)
    if op == "router_grad":
        r = s["router"]
        dlogits = r.backward(s["logits"], s["topk_ids"], s["topk_gates"], dloss=s["dloss"],
                             dy=s["dy"], o=s["o"], tok_row=s["tok_row"],
                             token_mask=s["token_mask"], seq_off=s["seq_off"])
        return dict(dlogits=dlogits, dgates=r.dgates)
    if op == "norm":
        h_out, x = s["norm"](s["h"], y=s["y"], gate=s["gate"], w_post=s["w_post"],
                             w_next=s["w_next"])
        return dict(h_out=h_out, x=x)
    if op == "norm_grad":
        g = s["norm"].backward(s["h"], y=s["y"], gate=s["gate"], w_post=s["w_post"],
                               w_next=s["w_next"], dh_out=s["dh_out"], dx=s["dx"])
        return dict(dh=g.dh, dy=g.dy, dgate=g.dgate, dw_post=g.dw_post, dw_next=g.dw_next)
    s["opt"].step(s["grads"])
    return _adamw_outputs(s)


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        p = 2 + 8 if case["master"] else 2 * BYTES[case["p"]]
        return dict(bytes=n * (p + BYTES[case["grad"]] + states), flops=15 * n)
    if op in ("balance", "router_grad"):
        T, E, k, S = case["T"], case["E"], case["k"], case["n_seq"]
        mask = T if case["masked"] else 0
        if op == "balance":
            return dict(bytes=T * (E + k + 1) * 4 + mask + 8 * S * E, flops=7 * T * E)
        d = case["d"]
        return dict(bytes=T * (2 * E + 4 * k + 1) * 4 + mask + 4 * S * E + T * d * (4 + 2 * k),
                    flops=2 * T * k * d + 8 * T * E)
    T, d, h, w = case["T"], case["d"], BYTES[case["h"]], BYTES[case["w"]]
    g = 4 * T if case["gate"] else 0
    if op == "norm":
        return dict(bytes=T * d * (h + 4 + h + 2) + 2 * d * w + g, flops=10 * T * d)
    return dict(bytes=T * d * (h + 4 + h + 4 + h + 4) + 2 * d * (w + 4) + 2 * g,
                flops=28 * T * d)


# ---------------------------------------------------------------- the definition, 64 bits
def _exact_sequences(s):
    """One-hot membership [S, T] of the counted tokens."""
    c = s["case"]
    t = torch.arange(c["T"], device=DEV)
    off = s["seq_off"].long() if s["seq_off"] is not None else \
        torch.tensor([0, c["T"]], device=DEV)
    member = (t >= off[:-1, None]) & (t < off[1:, None])
    if s["token_mask"] is not None:
        member = member & s["token_mask"].bool()
    return member.double()


def _exact_balance(s):
    c = s["case"]
    member = _exact_sequences(s)
    n_s = member.sum(1)
    x = s["logits"].double()
    lse = torch.logsumexp(x, 1)
    picked = torch.zeros_like(x).scatter_(1, s["topk_ids"].long(), 1.0)
    counts = member @ picked
    prob = (member @ torch.softmax(x, 1)) / n_s.clamp(min=1)[:, None]
    share = counts / (c["k"] * n_s.clamp(min=1))[:, None]
    some = (n_s > 0).sum().clamp(min=1)
    on = member.sum(0)
    losses = torch.stack([c["E"] * (share * prob).sum() / some,
                          (on * lse ** 2).sum() / n_s.sum().clamp(min=1)])
    return dict(losses=losses, counts=counts.int(), probs=prob, lse=on * lse)


def _exact_router_grad(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    member = _exact_sequences(s)
    n_s, on = member.sum(1), member.sum(0)
    x, ids, g = s["logits"].double(), s["topk_ids"].long(), s["topk_gates"].double()
    picked = torch.zeros_like(x).scatter_(1, ids, 1.0)
    weight = (member @ picked) * (E / k) / n_s.clamp(min=1)[:, None] ** 2
    b, z = s["dloss"].double() / torch.stack([(n_s > 0).sum().clamp(min=1),
                                              n_s.sum().clamp(min=1)])
    up = b * (member.T @ weight)                      # dL/dp
    p = torch.softmax(x, 1)
    dx = on[:, None] * (p * up - p * (p * up).sum(1, keepdim=True)
                        + z * 2 * torch.logsumexp(x, 1)[:, None] * p)
    dg = torch.empty(T, k, device=DEV, dtype=torch.float64)
    for j in range(k):
        for at in range(0, T, 4096):
            rows = s["o"][s["tok_row"][at:at + 4096, j].long()].double()
            dg[at:at + 4096, j] = torch.einsum("td,td->t", rows, s["dy"][at:at + 4096].double())
    soft = g * dg - g * (g * dg).sum(1, keepdim=True)
    return dict(dlogits=dx + torch.zeros_like(x).scatter_(1, ids, soft), dgates=dg)


def _exact_norm(s):
    h, y = s["h"].double(), s["y"].double()
    n = lambda v, w: v / (v.pow(2).mean(-1, keepdim=True) + NORM_EPS).sqrt() * w.double()  # noqa: E731
    g = s["gate"].double()[:, None] if s["gate"] is not None else 1.0
    h = RES_SCALE * h + OUT_SCALE * g * n(y, s["w_post"])
    return dict(h_out=h, x=n(h, s["w_next"]))


def _exact_norm_grad(s):
    """The vector-Jacobian product of the forward, by the chain rule row by row."""
    def back(v, w, q):
        inv = 1 / (v.pow(2).mean(-1, keepdim=True) + NORM_EPS).sqrt()
        unit = v * inv
        qw = q * w
        return inv * (qw - unit * (qw * unit).mean(-1, keepdim=True)), (q * unit).sum(0)

    out = {n: [] for n in ("dh", "dy", "dgate")}
    dw_post = dw_next = 0.0
    wp, wn = s["w_post"].double(), s["w_next"].double()
    for at in range(0, s["case"]["T"], 4096):
        h, y, dh, dx = (s[n][at:at + 4096].double() for n in ("h", "y", "dh_out", "dx"))
        into, part = back(h, wn, dx)
        dw_next = dw_next + part
        u = dh + into
        g = s["gate"][at:at + 4096].double()[:, None] if s["gate"] is not None else 1.0
        dy, part = back(y, wp, OUT_SCALE * g * u)
        dw_post = dw_post + part
        unit = y / (y.pow(2).mean(-1, keepdim=True) + NORM_EPS).sqrt()
        out["dh"].append(RES_SCALE * u)
        out["dy"].append(dy)
        out["dgate"].append(OUT_SCALE * (u * unit * wp).sum(1))
    out = {n: torch.cat(v) for n, v in out.items()}
    if s["gate"] is None:
        out["dgate"] = None
    return dict(out, dw_post=dw_post, dw_next=dw_next)


def _exact_8bit(x, root):
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1) / E4M3_MAX
    c = x / torch.where(scale > 0, scale, 1.0)[:, None]
    if root:
        c = torch.where(x > 0, c.clamp(min=E4M3_TINY), c)
    # the nearest e4m3 value, ties to the even mantissa
    step = torch.exp2(torch.floor(torch.log2(c.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(c / step) * step).view(-1), scale


def _exact_adamw(s):
    c = s["case"]
    t = s["step"] + 1
    g = s["grad"].double()
    m, v = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = (m.view(-1, BLOCK) * s["m_scale"].double()[:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["v_scale"].double()[:, None]).view(-1) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = (s["p"] if s["master"] is None else s["master"]).double()
    p = p - LR * WD * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    out = dict(p=p, master=p if c["master"] else None, m=m, v=v, m_scale=None, v_scale=None)
    if c["bits"] == 8:
        out["m"], out["m_scale"] = _exact_8bit(m, False)
        out["v"], out["v_scale"] = _exact_8bit(v.sqrt(), True)
    return out


EXACT = dict(balance=_exact_balance, router_grad=_exact_router_grad, norm=_exact_norm,
             norm_grad=_exact_norm_grad, adamw=_exact_adamw)


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
