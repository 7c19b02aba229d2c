"""GPU parity of the training operators (moeskew_train.h) against their 64-bit forms, through
the package's classes and the C ABI.

Tolerances, with u = 2^-24 (half a step of fp32): a sum of n fp32 terms in the kernels' order
(a thread's run of at most s terms, then log2 steps over lanes and warps) is off by at most
(s + 12) u times the sum of the terms' sizes, expf by 2 steps plus the rounding of its
argument, a root or a quotient by 2 steps.  Each check states the multiple of u it takes times
the sizes that enter (`size`, computed in 64 bits with absolute values, so that cancellation
is counted), plus half a step of the type that is stored: 2^-8 of the value for bf16, 2^-4 for
e4m3 (half its smallest step, 2^-10 of the scale, below the normal numbers)."""
import numpy as np
import pytest
import torch

import train_oracle as R
from skew_aware_token_b200 import native as N
from skew_aware_token_b200.synth import WORKLOADS, Workload
from skew_aware_token_b200.train import AdamW, BlockNorm, RouterLoss

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = 2.0 ** -8
DEV = "cuda"


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, want, tol, what):
    """|got - want| <= tol per element, all in 64 bits on the host."""
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - want).abs() - torch.as_tensor(tol, dtype=torch.float64)
    assert bool((over <= 0).all()), f"{what}: over its bound by {float(over.max()):.3e}"


def workload(T, d=256, E=8, k=2, beta=64):
    return Workload("case", T=T, d=d, E=E, k=k, f=128, beta=beta, P=1, s=0)


# ------------------------------------------------------------------------- router losses
def router_inputs(T, E, k, seed=0):
    logits = torch.randn(T, E, generator=gen(seed)) * 2 - torch.arange(1, E + 1).log()
    top, ids = logits.topk(k, dim=1)
    return logits, ids.int().contiguous(), torch.softmax(top, 1).contiguous()


LOSS_CASES = [
    # T, E, k, seq_off, mask: "none" | "some" | "all" masked
    (1, 1, 1, None, "none"), (1, 256, 8, None, "none"), (7, 33, 3, [0, 0, 7, 7], "some"),
    (256, 8, 2, None, "some"), (1111, 12, 4, [5, 300, 301, 900, 1000], "some"),
    (515, 60, 6, [0, 515], "none"), (640, 128, 8, list(range(0, 641, 5)), "some"),
    (100, 256, 8, list(range(101)), "none"), (2048, 64, 8, [0, 31, 33, 64, 2048], "some"),
    (300, 200, 5, [0, 100, 200, 300], "all"), (33, 96, 2, [33, 33], "none"),
    # more sequences than tokens, most of them empty; a batch longer than a chunk's share
    (70, 16, 2, [0] * 700 + sorted([7 * i // 100 for i in range(900)]) + [63] * 1500, "some"),
    (9500, 40, 3, [2, 31, 5000, 5000, 9400], "some"),
]


@pytest.mark.parametrize("T,E,k,off,masked", LOSS_CASES)
def test_router_losses(T, E, k, off, masked):
    logits, ids, _ = router_inputs(T, E, k)
    mask = None if masked == "none" else (torch.rand(T, generator=gen(1)) > 0.3).to(torch.uint8)
    if masked == "all":
        mask.zero_()
    elif mask is not None and off is not None and len(off) > 3:
        mask[off[1]:off[2]] = 0                       # a sequence that its mask leaves empty
    on = torch.zeros(T, dtype=torch.bool)
    for a, b in R.spans(T, off):
        on[a:b] = True
    if mask is not None:
        on &= mask.bool()
    dirty = logits.clone()
    dirty[~on] = float("nan")                          # nothing of a row that does not count
    dirty_ids = ids.clone()
    dirty_ids[~on] = 1 << 30
    S = 1 if off is None else len(off) - 1
    r = RouterLoss(workload(T, E=E, k=k), n_seq=S, device=DEV)
    r.workspace.fill_(255)
    for buf in (r.losses, r.probs, r._lse):
        buf.fill_(float("nan"))
    dev = lambda t, dt=None: None if t is None else torch.as_tensor(t, dtype=dt).to(DEV)
    args = (dev(dirty), dev(dirty_ids), dev(mask), dev(off, torch.int32))
    r(*args)
    torch.cuda.synchronize()
    assert r.read_status() == 0, N.moe_status_string(r.read_status())
    b, z, c, p, lse = R.router_losses(logits, ids, mask, off)
    assert torch.equal(r.counts.cpu().double(), c)
    n_s = [int(on[a:e].sum()) for a, e in R.spans(T, off)]
    assert r.seq_info.tolist() == n_s + [sum(n_s), sum(n > 0 for n in n_s)]
    # |x - top| < 32 here: exp's argument is off by 32 u, a row's sum of at most 8 + 5 steps
    close(r.lse, lse, 64 * U * (1 + lse.abs()), "lse")
    close(r.probs, p, 256 * U * p, "probs")
    close(r.losses, torch.stack([b, z]), 256 * U * (1 + torch.stack([b, z])), "losses")
    first = [t.clone() for t in (r.losses, r.counts, r.probs, r.lse)]
    r(*args)
    assert all(torch.equal(a, t) for a, t in zip(first, (r.losses, r.counts, r.probs, r.lse)))


@pytest.mark.parametrize("T,S", [(4000, 1 << 16), (200, 5000)])
def test_router_losses_many_empty_sequences(T, S):
    """Runs of empty sequences change nothing but the mean's place in the results, and are
    passed in steps, not one by one (65536 of them took 9.8 ms that way, 0.2 ms now)."""
    E, k = 8, 2
    logits, ids, _ = (t.to(DEV) for t in router_inputs(T, E, k, seed=4))
    mask = (torch.rand(T, generator=gen(5)) > 0.2).to(torch.uint8).to(DEV)
    at = sorted({0, T // 8, T // 5, T // 2 - 1, T // 2, T // 2 + 3, T - T // 7, T - 2})
    run = [1] * len(at)                          # how often each bound is repeated
    run[4], run[0], run[-1] = S + 1 - (len(at) - 3) - 7 - 5, 7, 5
    off = torch.tensor([a for a, n in zip(at, run) for _ in range(n)], dtype=torch.int32)
    assert off.numel() == S + 1
    full = torch.nonzero(off[1:] > off[:-1]).flatten()
    some, few = RouterLoss(workload(T), n_seq=S, device=DEV), RouterLoss(
        workload(T), n_seq=len(at) - 1, device=DEV)
    few(logits, ids, mask, torch.tensor(at, dtype=torch.int32, device=DEV))
    off, times = off.to(DEV), []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        some(logits, ids, mask, off)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert some.read_status() == 0 and few.read_status() == 0
    for name in ("counts", "probs"):
        assert torch.equal(getattr(some, name)[full], getattr(few, name)), name
        rest = torch.ones(S, dtype=torch.bool)
        rest[full] = False
        assert not bool(getattr(some, name).cpu()[rest].any()), name
    assert torch.equal(some.lse, few.lse)
    assert some.seq_info.tolist()[-2:] == few.seq_info.tolist()[-2:]
    close(some.losses, few.losses, (4 * U * few.losses.double().abs()).cpu(), "losses")
    assert min(times) < 3.0, times


def test_router_losses_lowest_values():
    """Experts masked with the type's lowest value are finite logits of no probability."""
    low = torch.finfo(torch.float32).min
    logits = torch.zeros(64, 16)
    logits[:, 4:] = low
    ids = torch.tensor([[0, 1]]).repeat(64, 1).int()
    r = RouterLoss(workload(64, E=16, k=2), device=DEV)
    r(logits.to(DEV), ids.to(DEV))
    d = r.backward(logits.to(DEV), dloss=torch.ones(2, device=DEV))
    assert r.read_status() == 0
    want = torch.tensor([0.25] * 4 + [0.0] * 12)
    close(r.probs[0], want, 8 * U, "probs")
    assert bool((d[:, 4:] == 0).all()) and bool(torch.isfinite(d).all())
    # a row of lowest values alone is a uniform row, its z loss the square's overflow
    r(torch.full((64, 16), low, device=DEV), ids.to(DEV))
    close(r.probs[0], torch.full((16,), 1 / 16), 8 * U, "probs")
    assert float(r.losses[1]) == float("inf") and bool(torch.isfinite(r.lse).all())


def test_router_losses_status():
    logits, ids, _ = router_inputs(40, 8, 2)
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = logits.clone()
        bad[17, 3] = value
        r = RouterLoss(workload(40), device=DEV)
        r(bad.to(DEV), ids.to(DEV))
        assert r.read_status() == N.MOE_STATUS_NONFINITE
    for value in (-1, 8, 1 << 30):
        bad = ids.clone()
        bad[3, 1] = value
        r = RouterLoss(workload(40), device=DEV)
        r(logits.to(DEV), bad.to(DEV))
        assert r.read_status() == N.MOE_STATUS_BAD_ID
        assert int(r.counts.sum()) == 79
    for off in ([0, 20, 10, 40], [-1, 10, 20, 40], [0, 10, 20, 41], [0, 1 << 30, 5, 40]):
        r = RouterLoss(workload(40), n_seq=3, device=DEV)
        r(logits.to(DEV), ids.to(DEV), None, torch.tensor(off, dtype=torch.int32, device=DEV))
        assert r.read_status() & N.MOET_STATUS_BAD_SEQ, off
    r = RouterLoss(workload(0), device=DEV)                # no tokens
    assert r(torch.zeros(0, 8, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)
             ).tolist() == [0, 0]
    assert r.read_status() == 0 and r.seq_info.tolist() == [0, 0, 0]


# ----------------------------------------------------------------------- router gradient
def rows_of(ids, E, beta):
    """tok_row of the block-aligned, expert-major rows, by a loop."""
    T, k = ids.shape
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    blocks = (counts + beta - 1) // beta
    base = (beta * (blocks.cumsum(0) - blocks)).tolist()
    out = torch.empty(T, k, dtype=torch.int32)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            out[t, j] = base[e]
            base[e] += 1
    return out


GRAD_CASES = [
    # T, d, E, k, seq_off, masked
    (1, 8, 1, 1, None, False), (1, 7168, 256, 8, None, False), (33, 520, 33, 3, [0, 9, 33], True),
    (257, 512, 12, 4, [3, 3, 100, 250], True), (70, 2056, 200, 8, None, False),
    (300, 64, 128, 6, [0, 150, 300], True), (5, 8192, 2, 2, None, True),
]


@pytest.mark.parametrize("T,d,E,k,off,masked", GRAD_CASES)
def test_router_gradient(T, d, E, k, off, masked):
    wl = workload(T, d=d, E=E, k=k)
    logits, ids, gates = router_inputs(T, E, k, seed=2)
    mask = (torch.rand(T, generator=gen(3)) > 0.3).to(torch.uint8) if masked else None
    R_max = N.moe_workspace_size(wl, N.MOE_WS_ROWS)
    tok_row = rows_of(ids, E, wl.beta)
    o = torch.randn(R_max, d, generator=gen(4)).bfloat16()
    dy = torch.randn(T, d, generator=gen(5))
    dloss = torch.tensor([3.0, -0.5])
    # the formula by autograd: gates are the softmax over the chosen logits
    x = logits.double().requires_grad_()
    b, z = R.router_losses(x, ids, mask, off)[:2]
    rows = o.double()[tok_row.long()]
    dg = torch.einsum("tkd,td->tk", rows, dy.double())
    g = torch.softmax(x.gather(1, ids.long()), 1)
    loss_part, = torch.autograd.grad(3.0 * b - 0.5 * z, x, allow_unused=True)
    gate_part, = torch.autograd.grad((g * dg).sum(), x)
    loss_part = torch.zeros_like(gate_part) if loss_part is None else loss_part
    S = 1 if off is None else len(off) - 1
    r = RouterLoss(wl, n_seq=S, device=DEV)
    off_d = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    mask_d = None if mask is None else mask.to(DEV)
    L, I, G = logits.to(DEV), ids.to(DEV), gates.to(DEV)
    r(L, I, mask_d, off_d)
    run = lambda **kw: r.backward(L, I, G, token_mask=mask_d, seq_off=off_d, **kw).clone()
    via = dict(dy=dy.to(DEV), o=o.to(DEV), tok_row=tok_row.to(DEV))
    r._dlogits.fill_(float("nan"))
    r._dgates.fill_(float("nan"))
    both = run(dloss=dloss.to(DEV), **via)
    # dgates: at most 8 * 4 terms a thread (d <= 8192 over 256 threads), 8 more steps
    size = torch.einsum("tkd,td->tk", rows.abs(), dy.double().abs())
    close(r.dgates, dg, 64 * U * size, "dgates")
    gd = g.detach()
    gate_size = torch.zeros_like(x).scatter_add_(
        1, ids.long(), gd * (size + (gd * size).sum(1, keepdim=True))).detach()
    p = torch.softmax(logits.double(), 1)
    # a_se by its parts: |dL/dp| is at most its largest, p is off by (64 + 32) u
    with torch.no_grad():
        _, _, c, _, lse = R.router_losses(logits, ids, mask, off)
        n_s = torch.tensor([float(sum(1 for t in range(a, e) if mask is None or mask[t]))
                            for a, e in R.spans(T, off)]).double()
        seqs, n = max(1, int((n_s > 0).sum())), max(1.0, float(n_s.sum()))
        a_max = (3.0 * E * c / (seqs * k * n_s.clamp(min=1)[:, None] ** 2)).max()
        loss_size = p * (2 * a_max + (lse / n).abs()[:, None])
    close(run(dloss=dloss.to(DEV)), loss_part, 256 * U * loss_size, "losses' part")
    close(run(**via), gate_part, 128 * U * gate_size, "gates' part")
    close(both, loss_part + gate_part, 256 * U * loss_size + 128 * U * gate_size, "both")
    assert torch.equal(both, run(dloss=dloss.to(DEV), **via))
    assert r.read_status() == 0


@pytest.mark.parametrize("T,d,E,k", [(300, 512, 12, 4), (20, 2056, 64, 8), (40, 64, 8, 2)])
@pytest.mark.parametrize("dloss", [(float("inf"), 1.0), (1.0, float("nan")), (0.0, float("-inf"))])
def test_router_gradient_of_tokens_that_do_not_count(T, d, E, k, dloss):
    """A loss gradient that is not finite (a loss scale that overflowed) reaches the tokens that
    count, and none of the others: those have their gates' part, or zeros."""
    wl = workload(T, d=d, E=E, k=k)
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k, seed=8))
    mask = (torch.arange(T) % 3 > 0).to(torch.uint8).to(DEV)
    off = torch.tensor([2, T - 4], dtype=torch.int32, device=DEV)
    o = torch.randn(N.moe_workspace_size(wl, N.MOE_WS_ROWS), d, generator=gen(1)).bfloat16().to(DEV)
    via = dict(dy=torch.randn(T, d, generator=gen(2)).to(DEV), o=o,
               tok_row=rows_of(ids.cpu(), E, wl.beta).to(DEV))
    r = RouterLoss(wl, device=DEV)
    r(logits, ids, mask, off)
    on = mask.bool()
    on[:2] = on[T - 4:] = False
    run = lambda **kw: r.backward(logits, ids, gates, token_mask=mask, seq_off=off, **kw).clone()
    gate_part = run(**via)
    bad = torch.tensor(dloss, device=DEV)
    alone, both = run(dloss=bad), run(dloss=bad, **via)
    assert bool((alone[~on] == 0).all()) and torch.equal(both[~on], gate_part[~on])
    assert not bool(torch.isfinite(alone[on]).all(1).any())


def test_router_losses_gradient_wants_a_forward():
    """Before any forward call there is nothing to take the losses' gradient of (the counts are
    zeros then, and would give zeros); the gates' part needs none."""
    T, d, E, k = 30, 64, 8, 2
    wl = workload(T, d=d, E=E, k=k)
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k))
    via = dict(dy=torch.ones(T, d, device=DEV), tok_row=rows_of(ids.cpu(), E, wl.beta).to(DEV),
               o=torch.ones(N.moe_workspace_size(wl, N.MOE_WS_ROWS), d, device=DEV).bfloat16())
    r, dloss = RouterLoss(wl, device=DEV), torch.ones(2, device=DEV)
    r.backward(topk_ids=ids, topk_gates=gates, **via)
    for kw in (dict(), dict(topk_ids=ids, topk_gates=gates, **via)):
        with pytest.raises(ValueError, match="forward"):
            r.backward(logits, dloss=dloss, **kw)
    r(logits, ids)
    assert float(r.backward(logits, dloss=dloss).abs().max()) > 0


def test_router_gradient_bad_rows_and_repeats():
    T, d, E, k = 20, 64, 8, 3
    wl = workload(T, d=d, E=E, k=k)
    R_max = N.moe_workspace_size(wl, N.MOE_WS_ROWS)
    logits, ids, gates = router_inputs(T, E, k, seed=6)
    o = torch.randn(R_max, d, generator=gen(7)).bfloat16()
    dy = torch.randn(T, d, generator=gen(8))
    tok_row = torch.randint(0, R_max, (T, k), generator=gen(9)).int()   # rows shared by tokens
    ids[4] = 5                                                        # one expert k times
    r = RouterLoss(wl, device=DEV)
    go = lambda i, t: r.backward(topk_ids=i.to(DEV), topk_gates=gates.to(DEV), dy=dy.to(DEV),
                                 o=o.to(DEV), tok_row=t.to(DEV)).cpu()
    got = go(ids, tok_row)
    dg = torch.einsum("tkd,td->tk", o.double()[tok_row.long()], dy.double())
    part = gates.double() * (dg - (gates.double() * dg).sum(1, keepdim=True))
    close(got, torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, ids.long(), part),
          64 * U * float(dg.abs().max() + 50), "repeats")
    assert r.read_status() == 0
    for bad_row in (-1, R_max, 1 << 30):
        r.clear_status()
        t = tok_row.clone()
        t[7, 2] = bad_row
        assert torch.isfinite(go(ids, t)).all() and r.read_status() == N.MOE_STATUS_BAD_ID
        assert float(r.dgates[7, 2]) == 0
    for bad_id in (-1, E, 1 << 30):
        r.clear_status()
        i = ids.clone()
        i[7, 2] = bad_id
        assert torch.isfinite(go(i, tok_row)).all() and r.read_status() == N.MOE_STATUS_BAD_ID


# ---------------------------------------------------------------------------- block norms
NORM_SHAPES = [(1, 8), (1, 7168), (3, 8192), (5, 264), (130, 512), (301, 1000), (64, 2048),
               (700, 136), (40, 4104)]
TYPES = [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
         (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)]
PARTS = ["all", "no_gate", "no_post", "no_next", "first"]


def norm_inputs(T, d, ht, wt, parts, seed=0):
    mk = lambda *s, n: torch.randn(*s, generator=gen(seed + n))
    a = dict(h=mk(T, d, n=1).to(ht), y=mk(T, d, n=2) * 0.5, gate=torch.rand(T, generator=gen(3)),
             w_post=(1 + 0.2 * mk(d, n=4)).to(wt), w_next=(1 + 0.2 * mk(d, n=5)).to(wt))
    drop = dict(all=(), no_gate=("gate",), no_post=("w_post",), no_next=("w_next",),
                first=("y", "gate", "w_post"))[parts]
    return {n: None if n in drop else t for n, t in a.items()}


def on_gpu(a):
    return {n: None if t is None else t.to(DEV) for n, t in a.items()}


def wide(a):
    return {n: None if t is None else t.double() for n, t in a.items()}


CONST = dict(eps=1e-5, w_offset=0.25, res_scale=0.8, out_scale=-0.6)


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("T,d", NORM_SHAPES)
@pytest.mark.parametrize("ht,wt", TYPES, ids=lambda t: str(t)[6:])
def test_block_norm(T, d, ht, wt, parts):
    a = norm_inputs(T, d, ht, wt, parts)
    norm = BlockNorm(workload(T, d=d), h_dtype=ht, w_dtype=wt, device=DEV, **CONST)
    for buf in (norm.h_out, norm.x):
        buf.fill_(float("nan"))
    h_out, x = norm(**on_gpu(a))
    q = wide(a)
    want_h, want_x = R.block_norm(q["h"], q["y"], q["gate"], q["w_post"], q["w_next"], **CONST)
    store = BF16 if ht is torch.bfloat16 else 0.0
    # a mean's sum: 16 terms a thread and 10 steps; the root halves it; a few products more
    size = want_h.abs() if a["y"] is None else \
        (CONST["res_scale"] * q["h"]).abs() + (want_h - CONST["res_scale"] * q["h"]).abs()
    if a["y"] is not None:
        close(h_out, want_h, store * want_h.abs() + 32 * U * size, "h_out")
    else:
        assert h_out.data_ptr() != norm.h_out.data_ptr() and torch.equal(h_out.cpu(), a["h"])
    if x is None:
        assert a["w_next"] is None
        return
    r = 1 / torch.sqrt((want_h ** 2).mean(1, keepdim=True) + CONST["eps"])
    x_size = want_x.abs() + size * r * (q["w_next"] + CONST["w_offset"]).abs()
    close(x, want_x, BF16 * want_x.abs() + 64 * U * x_size, "x")


def test_block_norm_in_place_and_zero_rows():
    a = on_gpu(norm_inputs(50, 1024, torch.float32, torch.float32, "all"))
    norm = BlockNorm(workload(50, d=1024), h_dtype=torch.float32, device=DEV, **CONST)
    h_out, x = (t.clone() for t in norm(**a))
    got, x2 = norm(**a, h_out=a["h"])
    assert got.data_ptr() == a["h"].data_ptr()
    assert torch.equal(got, h_out) and torch.equal(x2, x)
    z = dict(h=torch.zeros(50, 1024, device=DEV), y=torch.zeros(50, 1024, device=DEV),
             w_post=a["w_post"], w_next=a["w_next"])
    h_out, x = norm(**z)
    assert float(h_out.abs().max()) == 0 and float(x.float().abs().max()) == 0
    # a row's values stay its own: an infinite or NaN row leaves the others' bits alone
    b = on_gpu(norm_inputs(50, 1024, torch.float32, torch.float32, "all"))
    clean = [t.clone() for t in norm(**b)]
    b["y"][13] = float("nan")
    b["h"][20, 5] = float("inf")
    rest = [i for i in range(50) if i not in (13, 20)]
    for got, want in zip(norm(**b), clean):
        assert torch.equal(got[rest], want[rest]) and bool(torch.isnan(got[13]).all())


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("T,d", NORM_SHAPES)
@pytest.mark.parametrize("ht,wt", TYPES, ids=lambda t: str(t)[6:])
def test_block_norm_gradient(T, d, ht, wt, parts):
    a = norm_inputs(T, d, ht, wt, parts, seed=10)
    norm = BlockNorm(workload(T, d=d), h_dtype=ht, w_dtype=wt, train=True, device=DEV, **CONST)
    dh_out = torch.randn(T, d, generator=gen(20)).to(ht)
    dx = None if a["w_next"] is None else torch.randn(T, d, generator=gen(21))
    for buf in (norm.dh, norm.dy, norm.dgate, norm.dw_post, norm.dw_next):
        buf.fill_(float("nan"))
    norm.workspace.fill_(255)
    # the stream behind the block is what is stored: any row may stand for it
    b = on_gpu(a)
    run = lambda: norm.backward(b["h"], y=b["y"], gate=b["gate"], w_post=b["w_post"],
                                w_next=b["w_next"], dh_out=dh_out.to(DEV),
                                dx=None if dx is None else dx.to(DEV))
    g = run()
    # autograd of the two halves at the stored stream
    q = wide(a)
    leaf = {n: t.clone().requires_grad_() for n, t in q.items() if t is not None}
    h = leaf["h"]
    u = dh_out.double()
    zero = torch.zeros(())
    M = u.abs()
    if dx is not None:
        x = R.rms_norm(h, leaf["w_next"], CONST["eps"], CONST["w_offset"])
        gh, gw = torch.autograd.grad((x * dx.double()).sum(), (h, leaf["w_next"]))
        u = u + gh
        wn = (q["w_next"] + CONST["w_offset"]).abs()
        A = 1 / torch.sqrt((q["h"] ** 2).mean(1, keepdim=True) + CONST["eps"])
        dxa = dx.double().abs()
        M = M + A * dxa * wn + A ** 3 * q["h"].abs() * (dxa * wn * q["h"].abs()).mean(1, keepdim=True)
        # the weights' sums: at most 700 rows over 148 CTAs' groups, then 74 + 8 partial rows
        close(g.dw_next, gw, 160 * U * (dxa * A * q["h"].abs()).sum(0), "dw_next")
    store = BF16 if ht is torch.bfloat16 else 0.0
    res = CONST["res_scale"] if a["y"] is not None else 1.0
    close(g.dh, res * u, store * (res * u).abs() + 64 * U * M, "dh")
    if a["y"] is None:
        assert g.dy is None and g.dgate is None and g.dw_post is None
    else:
        names = [n for n in ("y", "gate", "w_post") if n in leaf]
        out, _ = R.block_norm(torch.zeros_like(q["h"]), leaf["y"], leaf.get("gate"),
                              leaf.get("w_post"), None, **CONST)
        grads = dict(zip(names, torch.autograd.grad((out * u).sum(), [leaf[n] for n in names])))
        y = q["y"].abs()
        ry, wp = torch.ones(T, 1).double(), torch.ones(d).double()
        if a["w_post"] is not None:
            ry = 1 / torch.sqrt((q["y"] ** 2).mean(1, keepdim=True) + CONST["eps"])
            wp = (q["w_post"] + CONST["w_offset"]).abs()
        gt = torch.ones(T, 1).double() if a["gate"] is None else q["gate"][:, None]
        c = abs(CONST["out_scale"])
        size = c * gt * ry * M * wp
        if a["w_post"] is not None:
            size = size + c * gt * ry ** 3 * y * (M * wp * y).mean(1, keepdim=True)
            close(g.dw_post, grads["w_post"], 160 * U * (c * gt * ry * M * y).sum(0), "dw_post")
        close(g.dy, grads["y"], 96 * U * size, "dy")
        if a["gate"] is not None:
            close(g.dgate, grads["gate"], 96 * U * (c * ry * M * wp * y).sum(1), "dgate")
    for name, arg in (("dgate", "gate"), ("dw_post", "w_post"), ("dw_next", "w_next")):
        assert (getattr(g, name) is None) == (a[arg] is None)
    first = [None if t is None else t.clone() for t in g]
    assert all(t is None or torch.equal(t, f) for t, f in zip(run(), first))


@pytest.mark.parametrize("T,d,ht", [(5000, 2048, torch.bfloat16), (9000, 512, torch.float32),
                                    (1500, 8192, torch.float32)])
def test_block_norm_many_rows(T, d, ht):
    """Many rows a group, both directions, against the 64-bit form on the GPU."""
    a = on_gpu(norm_inputs(T, d, ht, torch.float32, "all", seed=40))
    norm = BlockNorm(workload(T, d=d), h_dtype=ht, train=True, device=DEV, **CONST)
    q = wide(a)
    leaf = {n: t.clone().requires_grad_() for n, t in q.items()}
    want_h, want_x = R.block_norm(leaf["h"], leaf["y"], leaf["gate"], leaf["w_post"],
                                  leaf["w_next"], **CONST)
    h_out, x = norm(**a)
    store = BF16 if ht is torch.bfloat16 else 0.0
    size = CONST["res_scale"] * q["h"].abs() + (want_h - CONST["res_scale"] * q["h"]).abs()
    close(h_out, want_h, (store * want_h.abs() + 32 * U * size).detach().cpu(), "h_out")
    # the gradient at the stream as it is stored
    stored = h_out.double().requires_grad_()
    dh_out, dx = torch.randn(T, d, device=DEV).to(ht), torch.randn(T, d, device=DEV)
    xs = R.rms_norm(stored, leaf["w_next"], CONST["eps"], CONST["w_offset"])
    gh, gw = torch.autograd.grad((xs * dx.double()).sum(), (stored, leaf["w_next"]))
    u = dh_out.double() + gh
    out, _ = R.block_norm(torch.zeros_like(u), leaf["y"], leaf["gate"], leaf["w_post"], None,
                          **CONST)
    gy, gg, gp = torch.autograd.grad((out * u).sum(), [leaf[n] for n in ("y", "gate", "w_post")])
    g = norm.backward(h_out, y=a["y"], gate=a["gate"], w_post=a["w_post"], w_next=a["w_next"],
                      dh_out=dh_out, dx=dx)
    # sizes as in test_block_norm_gradient; a CTA adds at most 9000 / 148 rows, 296 CTAs at most
    A = 1 / torch.sqrt((stored.detach() ** 2).mean(1, keepdim=True) + CONST["eps"])
    wn, wp = (q[n] + CONST["w_offset"] for n in ("w_next", "w_post"))
    hs, dxa, ya = stored.detach().abs(), dx.double().abs(), q["y"].abs()
    M = dh_out.double().abs() + A * dxa * wn.abs() + A ** 3 * hs * (dxa * wn.abs() * hs).mean(
        1, keepdim=True)
    ry = 1 / torch.sqrt((q["y"] ** 2).mean(1, keepdim=True) + CONST["eps"])
    c, gt = abs(CONST["out_scale"]), q["gate"][:, None]
    ysize = c * gt * ry * M * wp.abs() + c * gt * ry ** 3 * ya * (M * wp.abs() * ya).mean(
        1, keepdim=True)
    res = CONST["res_scale"] * u
    close(g.dh, res, (store * res.abs() + 64 * U * M).cpu(), "dh")
    close(g.dy, gy, (96 * U * ysize).cpu(), "dy")
    close(g.dgate, gg, (96 * U * (c * ry * M * wp.abs() * ya).sum(1)).cpu(), "dgate")
    close(g.dw_next, gw, (192 * U * (dxa * A * hs).sum(0)).cpu(), "dw_next")
    close(g.dw_post, gp, (192 * U * (c * gt * ry * M * ya).sum(0)).cpu(), "dw_post")


@pytest.mark.parametrize("parts", PARTS[1:])
@pytest.mark.parametrize("T,d,ht", [(5000, 2048, torch.bfloat16), (9000, 512, torch.float32),
                                    (1500, 8192, torch.float32), (2500, 4104, torch.bfloat16)])
def test_block_norm_many_rows_of_parts(T, d, ht, parts):
    """Many rows a group where a row takes one sum or none (the norm before the first block,
    the one behind the last), both directions, and the same bits on every run."""
    a = on_gpu(norm_inputs(T, d, ht, torch.float32, parts, seed=60))
    norm = BlockNorm(workload(T, d=d), h_dtype=ht, train=True, device=DEV, **CONST)
    q = wide(a)
    leaf = {n: None if t is None else t.clone().requires_grad_() for n, t in q.items()}
    want_h, want_x = R.block_norm(leaf["h"], leaf["y"], leaf["gate"], leaf["w_post"],
                                  leaf["w_next"], **CONST)
    h_out, x = norm(**a)
    first = [t.clone() for t in (h_out, x) if t is not None]
    # bounds as in test_block_norm
    store = BF16 if ht is torch.bfloat16 else 0.0
    size = q["h"].abs()
    if a["y"] is not None:
        size = CONST["res_scale"] * size + (want_h - CONST["res_scale"] * q["h"]).abs()
        close(h_out, want_h, (store * want_h.abs() + 32 * U * size).detach().cpu(), "h_out")
    if a["w_next"] is not None:
        r = 1 / torch.sqrt((want_h ** 2).mean(1, keepdim=True) + CONST["eps"])
        x_size = want_x.abs() + size * r * (q["w_next"] + CONST["w_offset"]).abs()
        close(x, want_x, (BF16 * want_x.abs() + 64 * U * x_size).detach().cpu(), "x")
    for _ in range(20):
        assert all(torch.equal(t, f) for t, f in
                   zip([t for t in norm(**a) if t is not None], first))
    # the gradient at the stored stream, bounds as in test_block_norm_many_rows
    stored = h_out.double().requires_grad_()
    dh_out = torch.randn(T, d, generator=gen(61)).to(ht).to(DEV)
    dx = None if a["w_next"] is None else torch.randn(T, d, generator=gen(62)).to(DEV)
    run = lambda: norm.backward(h_out, y=a["y"], gate=a["gate"], w_post=a["w_post"],
                                w_next=a["w_next"], dh_out=dh_out, dx=dx)
    g = run()
    u, M = dh_out.double(), dh_out.double().abs()
    if dx is not None:
        xs = R.rms_norm(stored, leaf["w_next"], CONST["eps"], CONST["w_offset"])
        gh, gw = torch.autograd.grad((xs * dx.double()).sum(), (stored, leaf["w_next"]))
        A = 1 / torch.sqrt((stored.detach() ** 2).mean(1, keepdim=True) + CONST["eps"])
        hs, qa = stored.detach().abs(), dx.double().abs() * (q["w_next"] + CONST["w_offset"]).abs()
        u = u + gh
        M = M + A * qa + A ** 3 * hs * (qa * hs).mean(1, keepdim=True)
        close(g.dw_next, gw, (192 * U * (dx.double().abs() * A * hs).sum(0)).cpu(), "dw_next")
    res = u if a["y"] is None else CONST["res_scale"] * u
    close(g.dh, res, (store * res.abs() + 64 * U * M).cpu(), "dh")
    if a["y"] is not None:
        names = [n for n in ("y", "gate", "w_post") if a[n] is not None]
        out, _ = R.block_norm(torch.zeros_like(u), leaf["y"], leaf["gate"], leaf["w_post"], None,
                              **CONST)
        grads = dict(zip(names, torch.autograd.grad((out * u).sum(), [leaf[n] for n in names])))
        ya, ry, wp = q["y"].abs(), torch.ones(T, 1, device=DEV).double(), 1.0
        if a["w_post"] is not None:
            ry = 1 / torch.sqrt((q["y"] ** 2).mean(1, keepdim=True) + CONST["eps"])
            wp = (q["w_post"] + CONST["w_offset"]).abs()
        gt = 1.0 if a["gate"] is None else q["gate"][:, None]
        c = abs(CONST["out_scale"])
        ysize = c * gt * ry * M * wp
        if a["w_post"] is not None:
            ysize = ysize + c * gt * ry ** 3 * ya * (M * wp * ya).mean(1, keepdim=True)
            close(g.dw_post, grads["w_post"],
                  (192 * U * (c * gt * ry * M * ya).sum(0)).cpu(), "dw_post")
        close(g.dy, grads["y"], (96 * U * ysize).cpu(), "dy")
        if a["gate"] is not None:
            close(g.dgate, grads["gate"], (96 * U * (c * ry * M * wp * ya).sum(1)).cpu(), "dgate")
    first = [t.clone() for t in g if t is not None]
    for _ in range(5):
        assert all(torch.equal(t, f) for t, f in zip([t for t in run() if t is not None], first))


@pytest.mark.parametrize("eps", [1e-30, 1e-6])
def test_block_norm_gradient_of_small_and_large_rows(eps):
    """Rows of zeros, of tiny and of huge values, with a small eps: the formula's gradients (the
    cube of rms leaves fp32 in both directions, what it stands in does not).  Bounds as in
    test_block_norm_gradient."""
    scales = [0.0, 1e-18, 1e-16, 1e-8, 1.0, 1e6, 1e13, 1e15]
    T, d = len(scales), 512
    s = torch.tensor(scales)[:, None]
    h, y = torch.randn(T, d, generator=gen(70)) * s, torch.randn(T, d, generator=gen(71)) * s
    wp, wn = (1 + 0.2 * torch.randn(d, generator=gen(n)) for n in (72, 73))
    dh_out, dx = (torch.randn(T, d, generator=gen(n)) for n in (74, 75))
    norm = BlockNorm(workload(T, d=d), h_dtype=torch.float32, train=True, eps=eps, device=DEV)
    g = norm.backward(h.to(DEV), y=y.to(DEV), w_post=wp.to(DEV), w_next=wn.to(DEV),
                      dh_out=dh_out.to(DEV), dx=dx.to(DEV))
    h, y, wp, wn, dh_out, dx = (t.double() for t in (h, y, wp, wn, dh_out, dx))
    leaf = [t.clone().requires_grad_() for t in (h, wn, y, wp)]
    x = R.rms_norm(leaf[0], leaf[1], eps, 0.0)
    gh, gn = torch.autograd.grad((x * dx).sum(), leaf[:2])
    u = dh_out + gh
    gy, gp = torch.autograd.grad((R.rms_norm(leaf[2], leaf[3], eps, 0.0) * u).sum(), leaf[2:])
    A, ry = (1 / torch.sqrt((t ** 2).mean(1, keepdim=True) + eps) for t in (h, y))
    qa = (dx * wn).abs()
    M = dh_out.abs() + A * qa + A ** 3 * h.abs() * (qa * h.abs()).mean(1, keepdim=True)
    size = ry * M * wp.abs() + ry ** 3 * y.abs() * (M * (wp * y).abs()).mean(1, keepdim=True)
    close(g.dh, u, 64 * U * M, "dh")
    close(g.dy, gy, 96 * U * size, "dy")
    close(g.dw_next, gn, 160 * U * (dx.abs() * A * h.abs()).sum(0), "dw_next")
    close(g.dw_post, gp, 160 * U * (ry * M * y.abs()).sum(0), "dw_post")


def test_block_norm_gradient_of_no_rows_goes_to_its_stream():
    """Without rows the weights' gradients are zeros, written on the stream that is passed."""
    d = 512
    none, w = torch.zeros(0, d, device=DEV), torch.ones(d, device=DEV)
    norm = BlockNorm(workload(0, d=d), h_dtype=torch.float32, train=True, device=DEV)
    norm.dw_next.fill_(7)
    norm.dw_post.fill_(7)
    side = torch.cuda.Stream()
    big = torch.empty(1 << 28, device=DEV)
    torch.cuda.synchronize()
    for _ in range(100):
        big.fill_(1.0)                          # the current stream is busy
    g = norm.backward(none, y=none, w_post=w, w_next=w, dx=none, stream=side)
    with torch.cuda.stream(side):
        got = [t.clone() for t in (g.dw_next, g.dw_post)]
    side.synchronize()
    assert all(float(t.abs().max()) == 0 for t in got)
    norm.dw_next.fill_(7)
    norm.backward(none, w_next=w, dx=none)      # the parts alone
    assert float(norm.dw_next.abs().max()) == 0
    gate = torch.zeros(0, device=DEV)
    g = norm.backward(none, y=none, gate=gate, dh_out=none)
    assert g.dw_post is None and g.dw_next is None and g.dgate.shape == (0,)


def test_block_norm_gradient_parts_and_in_place():
    """dh_out = None is zeros; dh may take dh_out's place (C ABI)."""
    T, d = 77, 768
    a = on_gpu(norm_inputs(T, d, torch.float32, torch.float32, "all", seed=30))
    norm = BlockNorm(workload(T, d=d), h_dtype=torch.float32, train=True, device=DEV, **CONST)
    dx = torch.randn(T, d, generator=gen(31)).to(DEV)
    kw = dict(y=a["y"], gate=a["gate"], w_post=a["w_post"], w_next=a["w_next"], dx=dx)
    zero = [t.clone() for t in norm.backward(a["h"], dh_out=torch.zeros(T, d, device=DEV), **kw)]
    assert all(torch.equal(t, z) for t, z in zip(norm.backward(a["h"], **kw), zero))
    dh = torch.randn(T, d, generator=gen(32)).to(DEV)
    want = [t.clone() for t in norm.backward(a["h"], dh_out=dh, **kw)]
    N.moet_block_norm_backward(norm.cfg, norm.norm, a["h"], a["y"], a["gate"], a["w_post"],
                               a["w_next"], dh, dx, dh, norm.dy, norm.dgate, norm.dw_post,
                               norm.dw_next, norm.workspace)
    assert torch.equal(dh, want[0])
    empty = BlockNorm(workload(0, d=d), train=True, device=DEV)
    none = torch.zeros(0, d, device=DEV)
    empty.dw_next.fill_(7)
    g = empty.backward(none.bfloat16(), w_next=a["w_next"], dx=none)
    assert float(g.dw_next.abs().max()) == 0
    # through the C ABI too: no rows, weight gradients of zero
    empty.dw_next.fill_(7)
    N.moet_block_norm_backward(empty.cfg, empty.norm, a["h"], None, None, None, a["w_next"], dh,
                               dx, dh, None, None, None, empty.dw_next, empty.workspace)
    assert float(empty.dw_next.abs().max()) == 0


# --------------------------------------------------------------------------------- AdamW
SIZES = [1, 3, 255, 256, 257, 2048, 2049, 5000, 0, 70001]
KINDS = [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True)]
B1, B2, EPS, LR = 0.9, 0.95, 1e-8, 3e-3


def adam_inputs(sizes, pt, gt, seed=0):
    ps = [torch.randn(n, generator=gen(seed + i)).to(pt) for i, n in enumerate(sizes)]
    gs = [(torch.randn(n, generator=gen(seed + 100 + i)) * 0.1 ** (i % 5)).to(gt)
          for i, n in enumerate(sizes)]
    return ps, gs


@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16], ids=["g32", "g16"])
@pytest.mark.parametrize("pt,master", KINDS, ids=["f32", "bf16", "master"])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits, pt, master, gt):
    ps, gs = adam_inputs(SIZES, pt, gt)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    opt = AdamW([p.to(DEV) for p in ps], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay,
                state_bits=bits, master=True if master else None)
    host = lambda ts: [t.cpu() for t in ts]
    for step in range(1, 4):
        gd = [(g.float() * step).to(gt) for g in gs]
        before = {n: host(getattr(opt, n)) for n in ("params", "m", "v")}
        if bits == 8:
            before["m"] = [R.of_8bit(c, s) for c, s in zip(before["m"], host(opt.m_scale))]
            before["v"] = [R.of_8bit(c, s) ** 2 for c, s in zip(before["v"], host(opt.v_scale))]
        w = host(opt.master) if master else before["params"]
        opt.step([g.to(DEV) for g in gd])
        assert opt.steps.tolist()[:2] == [step, 0]
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            g, m0, v0 = gd[i].double(), before["m"][i].double(), before["v"][i].double()
            p, m, v = R.adamw(w[i].double(), g, m0, v0, step, LR, B1, B2, EPS, decay[i])
            ms = (B1 * m0).abs() + ((1 - B1) * g).abs()
            # the moment behind a cancelled sum reaches the step too
            up = ms / (1 - B1 ** step) / ((v / (1 - B2 ** step)).sqrt() + EPS)
            tol = U * (8 * p.abs() + 8 * w[i].double().abs() + 48 * LR * up)
            new = opt.params[i]
            if master:
                close(opt.master[i], p, tol, "master")
                assert torch.equal(opt.master[i].bfloat16(), new)
            close(new, p, tol + (BF16 * p.abs() if pt is torch.bfloat16 else 0), f"p[{i}]")
            if bits == 32:
                close(opt.m[i], m, 4 * U * ms, "m")
                close(opt.v[i], v, 6 * U * v, "v")
                continue
            # the stored form is defined by its fp32 roundings: the same bits
            f = lambda t: torch.tensor(t, dtype=torch.float32)
            g32 = gd[i].float()
            m32 = before["m"][i] * f(B1) + g32 * f(1 - B1)
            v32 = before["v"][i] * f(B2) + (g32 * f(1 - B2)) * g32
            # (torch's fp32 root on the CPU is up to a step off; the 64-bit one, rounded, is the
            # nearest fp32 value, since 53 >= 2 * 24 + 2 bits)
            r32 = v32.double().sqrt().float()
            for got, s, (want, ws) in ((opt.m[i], opt.m_scale[i], R.to_8bit(m32, False)),
                                       (opt.v[i], opt.v_scale[i], R.to_8bit(r32, True))):
                assert torch.equal(s.cpu(), ws)
                assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
            # and within half a step of e4m3 of the 64-bit moments
            sc = opt.m_scale[i].cpu().double().repeat_interleave(256)[:n]
            close(R.of_8bit(opt.m[i].cpu(), opt.m_scale[i].cpu()), m,
                  2.0 ** -4 * m.abs() + 2.0 ** -10 * sc + 16 * U * ms, "m")
            sc = opt.v_scale[i].cpu().double().repeat_interleave(256)[:n]
            close(R.of_8bit(opt.v[i].cpu(), opt.v_scale[i].cpu()), v.sqrt(),
                  (2.0 ** -4 + 16 * U) * v.sqrt() + 2.0 ** -9 * sc, "root of v")


@pytest.mark.parametrize("eps", [2e-38, 1e-30, 1e-20, 1e-16, 1e-12, 1e-8])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_small_gradients_and_eps(bits, eps):
    """Gradients whose squares are subnormal or next to it, over every eps that is taken: the
    step is the formula's.  v's three roundings are off by 2^-150 each there (half the smallest
    subnormal), in the root half of that relative to v."""
    n = 4096
    g = torch.randn(n, generator=gen(1)).sign() * 10 ** (-16 - 4.5 * torch.rand(n, generator=gen(2)))
    opt = AdamW([torch.zeros(n, device=DEV)], lr=1.0, betas=(B1, B2), eps=eps, weight_decay=0.0,
                state_bits=bits)
    for step in range(1, 4):
        m0, v0 = opt.m[0].cpu(), opt.v[0].cpu()
        if bits == 8:
            m0 = R.of_8bit(m0, opt.m_scale[0].cpu())
            v0 = R.of_8bit(v0, opt.v_scale[0].cpu()) ** 2
        p0 = opt.params[0].double().cpu()
        opt.step([g.to(DEV)])
        p, m, v = R.adamw(p0, g.double(), m0.double(), v0.double(), step, 1.0, B1, B2, eps, 0.0)
        ms = (B1 * m0.double()).abs() + ((1 - B1) * g.double()).abs()
        up = ms / (1 - B1 ** step) / ((v / (1 - B2 ** step)).sqrt() + eps)
        tol = U * (8 * p.abs() + 8 * p0.abs() + 48 * up) + up * 3 * 2.0 ** -150 / (2 * v) * 1.1
        close(opt.params[0], p, tol, f"p at step {step}")


@pytest.mark.parametrize("spread", [1.0, 8.0, 30.0])
def test_adamw_codes_of_many_roots(spread):
    """Four million roots, spread over up to 2^30 within a block (most of e4m3's codes, its
    subnormal ones, roots far below them, zeros): the nearest codes bit for bit.  About 60 of
    the roots lie within a few fp32 steps of a border between two codes."""
    n = 1 << 22
    g = torch.randn(n, generator=gen(1)) * torch.exp2(-spread * torch.rand(n, generator=gen(2)))
    g[::97] = 0
    opt = AdamW([torch.zeros(n, device=DEV)], lr=LR, betas=(B1, B2), state_bits=8)
    opt.step([g.to(DEV)])
    f = lambda t: torch.tensor(t, dtype=torch.float32)
    m32, v32 = g * f(1 - B1), (g * f(1 - B2)) * g
    for got, s, (want, ws) in ((opt.m[0], opt.m_scale[0], R.to_8bit(m32, False)),
                               (opt.v[0], opt.v_scale[0],
                                R.to_8bit(v32.double().sqrt().float(), True))):
        assert torch.equal(s.cpu(), ws)
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


def test_adamw_scale_skip_and_mixed_tensors():
    """grad_scale multiplies; a scale that is not finite leaves the step out; tensors of every
    kind and more of them than one launch holds step together."""
    kinds = [(pt, gt, m) for pt, m in KINDS for gt in (torch.float32, torch.bfloat16)]
    ps, gs, ms = [], [], []
    for i in range(900):
        pt, gt, m = kinds[i % 6] if i < 60 else kinds[0]
        p, g = adam_inputs([1 + 37 * i % 400], pt, gt, seed=i)
        ps += [p[0].to(DEV)]
        gs += [g[0].to(DEV)]
        ms += [p[0].float().to(DEV) if m else None]
    p0 = [p.clone() for p in ps]
    opt = AdamW(ps, lr=LR, betas=(B1, B2), weight_decay=0.1, master=ms)
    for bad in (float("nan"), float("inf")):
        opt.step(gs, grad_scale=torch.tensor([bad], device=DEV))
        assert opt.steps.tolist()[:2] == [0, 0]
        assert all(torch.equal(a, b) for a, b in zip(ps, p0))
        assert all(float(m.abs().max()) == 0 for m in opt.m)
    opt.step(gs, grad_scale=torch.tensor([0.5], device=DEV))
    assert opt.steps.tolist()[:2] == [1, 0]
    for i, (p, q, g) in enumerate(zip(ps, p0, gs)):
        q, g = q.double().cpu(), 0.5 * g.double().cpu()
        want, m, _ = R.adamw(q, g, 0 * g, 0 * g, 1, LR, B1, B2, EPS, 0.1)
        close(opt.m[i], m, 4 * U * m.abs(), "m")
        close(p, want, U * (16 * q.abs() + 64 * LR) + (BF16 * want.abs() if p.dtype is torch.bfloat16
                                                       else 0), f"p[{i}]")


def test_adamw_on_views_of_flat_storage():
    """Tensors that are views into one buffer each (scales on 4 bytes), odd ends: the result
    of tensors of their own, and nothing between the views written."""
    sizes, starts = [1, 300, 1000, 5], [0, 256, 768, 2048]
    ps, gs = adam_inputs(sizes, torch.bfloat16, torch.float32, seed=3)
    flat = dict(p=torch.full((2304,), 7, dtype=torch.bfloat16, device=DEV),
                m=torch.zeros(2304, device=DEV).to(torch.float8_e4m3fn),
                v=torch.zeros(2304, device=DEV).to(torch.float8_e4m3fn),
                ms=torch.zeros(9, device=DEV), vs=torch.zeros(9, device=DEV))
    cut = lambda x: [x[a:a + n] for a, n in zip(starts, sizes)]
    scale = lambda x: [x[a // 256:a // 256 + -(-n // 256)] for a, n in zip(starts, sizes)]
    for view, p in zip(cut(flat["p"]), ps):
        view.copy_(p)
    opt = AdamW(cut(flat["p"]), state_bits=8, m=cut(flat["m"]), v=cut(flat["v"]),
                m_scale=scale(flat["ms"]), v_scale=scale(flat["vs"]))
    alone = AdamW([p.to(DEV) for p in ps], state_bits=8)
    for _ in range(2):
        opt.step([g.to(DEV) for g in gs])
        alone.step([g.to(DEV) for g in gs])
    for name in ("params", "m", "v", "m_scale", "v_scale"):
        for a, b in zip(getattr(opt, name), getattr(alone, name)):
            assert torch.equal(a.float(), b.float()), name
    gap = torch.ones(2304, dtype=torch.bool)
    for a, n in zip(starts, sizes):
        gap[a:a + n] = False
    assert bool((flat["p"].cpu()[gap] == 7).all()) and not flat["m"].float().cpu()[gap].any()


def test_adamw_follows_a_weight_whose_storage_is_exchanged():
    """The step updates what the weight is at the step, and refuses it when it changed size,
    type or device; the states cannot be exchanged unnoticed."""
    p = torch.nn.Parameter(torch.ones(1000, device=DEV))
    opt, g = AdamW([p], lr=LR, weight_decay=0.0), [torch.ones(1000, device=DEV)]
    old = p.data
    p.data = torch.full((1000,), 2.0, device=DEV)
    opt.step(g)
    assert bool((old == 1).all()) and bool((p.data < 2).all())
    for bad, error in ((torch.ones(999, device=DEV), ValueError), (torch.ones(1000), TypeError),
                       (torch.ones(1000, device=DEV).bfloat16(), TypeError)):
        q = torch.nn.Parameter(torch.ones(1000, device=DEV))
        opt = AdamW([q], lr=LR)
        q.data = bad
        with pytest.raises(error, match=r"params\[0\]"):
            opt.step(g)
    with pytest.raises(TypeError):
        opt.m[0] = torch.zeros(1000, device=DEV)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_follows_states_whose_storage_is_exchanged(bits):
    """States moved to other storage between steps (an offload and back) are the ones that the
    next step reads and writes; what they left is not touched.  A state of another size, type
    or device is refused, and so are states that came to share memory."""
    sizes = [1000, 300, 0]
    ps, gs = adam_inputs(sizes, torch.bfloat16, torch.float32, seed=5)
    build = lambda: AdamW([p.to(DEV) for p in ps], lr=LR, state_bits=bits, master=True)
    moved, stayed, grads = build(), build(), [g.to(DEV) for g in gs]
    names = ["params", "m", "v", "master"] + (["m_scale", "v_scale"] if bits == 8 else [])
    raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t
    for turn in range(3):
        for opt in (moved, stayed):
            opt.step(grads)
        for name in names:
            for a, b in zip(getattr(moved, name), getattr(stayed, name)):
                assert torch.equal(raw(a), raw(b)), name
        left = []
        for name in names:
            for t in getattr(moved, name):
                left.append((t.data, t.data.cpu()))
                t.data = t.data.cpu().to(DEV)
        moved.step(grads)
        stayed.step(grads)
        for old, was in left:
            assert torch.equal(raw(old.cpu()), raw(was))
    for name in names[1:]:
        t = getattr(moved, name)[0]
        keep = t.data
        for bad, error in ((torch.zeros(keep.numel() + 1, device=DEV).to(keep.dtype), ValueError),
                           (keep.cpu(), TypeError), (keep.to(torch.float16), TypeError)):
            t.data = bad
            with pytest.raises(error, match=rf"{name}\[0\]"):
                moved.step(grads)
        t.data = keep
    for name, bad, error in (("steps", torch.zeros(1, dtype=torch.int32, device=DEV), ValueError),
                             ("steps", torch.zeros(4, device=DEV), TypeError),
                             ("lr", torch.zeros(4), TypeError), ("lr", 1e-3, TypeError)):
        keep = getattr(moved, name)
        setattr(moved, name, bad)
        with pytest.raises(error, match=name):
            moved.step(grads)
        setattr(moved, name, keep)
    before = moved.steps.tolist()
    keep = moved.m[1].data
    moved.m[1].data = moved.m[0].data[:300]
    for _ in range(2):
        with pytest.raises(ValueError, match="share memory"):
            moved.step(grads)
    moved.m[1].data = keep
    assert moved.steps.tolist() == before
    moved.step(grads)
    stayed.step(grads)
    for name in names:
        for a, b in zip(getattr(moved, name), getattr(stayed, name)):
            assert torch.equal(raw(a), raw(b)), name


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_without_the_states_it_had(bits):
    """States that were dropped are not stepped at the addresses that they had: the step is
    refused, or, without masters, made on the weights themselves."""
    g = [torch.ones(700, device=DEV)]
    for name in ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
        opt = AdamW([torch.ones(700, device=DEV)], lr=LR, state_bits=bits)
        opt.step(g)
        keep = getattr(opt, name)
        was = [t.clone().view(torch.uint8) for t in keep], opt.params[0].clone()
        setattr(opt, name, None)
        with pytest.raises(N.MoeError):
            opt.step(g)
        assert torch.equal(keep[0].view(torch.uint8), was[0][0])
        assert torch.equal(opt.params[0], was[1]) and opt.steps.tolist()[:2] == [1, 0]
    opt = AdamW([torch.ones(700, device=DEV).bfloat16()], lr=LR, state_bits=bits, master=True)
    opt.step(g)
    keep, opt.master = opt.master, None
    was, w = keep[0].clone(), opt.params[0].clone()
    opt.step(g)
    assert torch.equal(keep[0], was) and not torch.equal(opt.params[0], w)


def test_exchanged_buffers_are_written_where_they_are():
    """An object's own buffers that were exchanged (the attribute or its .data) are the ones that
    the next call writes; one of another size or type is refused."""
    T, d, E, k = 70, 512, 16, 4
    wl = workload(T, d=d, E=E, k=k)
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k))
    a = on_gpu(norm_inputs(T, d, torch.bfloat16, torch.float32, "all"))
    dx = torch.randn(T, d, generator=gen(1)).to(DEV)
    dloss = torch.ones(2, device=DEV)
    r, n = RouterLoss(wl, device=DEV), BlockNorm(wl, train=True, device=DEV)
    calls = {
        r: (lambda: r(logits, ids), ("losses", "counts", "probs", "seq_info", "_lse", "workspace",
                                     "status")),
        n: (lambda: n(**a), ("h_out", "x")),
    }
    back = {
        r: (lambda: r.backward(logits, dloss=dloss), ("counts", "seq_info", "_lse", "_dlogits",
                                                      "_dgates", "status")),
        n: (lambda: n.backward(a["h"], y=a["y"], gate=a["gate"], w_post=a["w_post"],
                               w_next=a["w_next"], dx=dx),
            ("dh", "dy", "dgate", "dw_post", "dw_next", "workspace")),
    }
    for table in (calls, back):
        for obj, (go, names) in table.items():
            go()
            torch.cuda.synchronize()
            want = {name: getattr(obj, name).clone() for name in names}
            left = []
            for i, name in enumerate(names):
                t = getattr(obj, name)
                left.append((t.data, t.clone()))
                new = t.clone() if name in ("counts", "seq_info", "_lse", "status") and \
                    table is back else torch.zeros_like(t)
                if i % 2:
                    t.data = new
                else:
                    setattr(obj, name, new)
            for old, _ in left:
                old.fill_(3)
            go()
            torch.cuda.synchronize()
            for old, _ in left:
                assert bool((old == 3).all())
            for name in names:
                if name not in ("workspace", "_dgates"):
                    assert torch.equal(getattr(obj, name), want[name]), name
            for name in names:
                keep = getattr(obj, name)
                for bad, error in ((keep.flatten()[:-1], ValueError), (keep.cpu(), TypeError),
                                   (keep.half(), TypeError)):
                    setattr(obj, name, bad)
                    with pytest.raises(error, match=name):
                        go()
                setattr(obj, name, keep)


def test_adamw_raises_the_weights_versions():
    """A weight that autograd saved in a forward before the step is an error in the backward
    behind it; weights made in inference mode, which have no version, step too."""
    p = torch.nn.Parameter(torch.ones(500, device=DEV))
    q = torch.nn.Parameter(torch.ones(300, device=DEV).bfloat16())
    opt = AdamW([p, q], lr=LR, master=True)
    x = torch.randn(500, device=DEV, requires_grad=True)
    y = (x * p).sum()
    grads = [torch.ones(500, device=DEV), torch.ones(300, device=DEV)]
    was = p._version, q._version
    with pytest.raises(ValueError):
        opt.step([grads[0], grads[0]])
    assert (p._version, q._version) == was
    opt.step(grads)
    assert p._version > was[0] and q._version > was[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    (x * p).sum().backward()
    assert torch.equal(x.grad, p.detach())
    with torch.inference_mode():
        w = torch.ones(500, device=DEV)
    inner = AdamW([w], lr=LR)
    inner.step(grads[:1])
    with torch.inference_mode():
        inner.step(grads[:1])
        opt.step(grads)
    assert bool((w < 1).all()) and opt.steps.tolist()[0] == 2


def test_first_use_on_another_stream():
    """An object used at once on a stream other than the one it was built on."""
    wl = workload(700, d=1024, E=64, k=8)
    logits, ids, _ = (t.to(DEV) for t in router_inputs(700, 64, 8))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    want = None
    for _ in range(5):
        big = torch.empty(1 << 28, device=DEV)
        for _ in range(20):
            big.fill_(1.0)                      # the building stream is busy
        r = RouterLoss(wl, device=DEV)
        with torch.cuda.stream(side):
            r(logits, ids)
        side.synchronize()
        got = (r.losses.clone(), r.counts.clone(), r.probs.clone())
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_adamw_bad_gradients_stay_in_their_block():
    n = 1024
    for bits in (32, 8):
        p = torch.ones(n, device=DEV)
        opt = AdamW([p], lr=LR, state_bits=bits)
        g = torch.randn(n, generator=gen(0)).to(DEV)
        g[300], g[301] = float("nan"), float("inf")
        opt.step([g])
        assert not bool(torch.isfinite(p[300:302]).any())
        rest = torch.ones(n, dtype=torch.bool)
        rest[300:302] = False
        assert bool(torch.isfinite(p.cpu()[rest]).all())
        if bits == 8:
            ok = torch.isfinite(opt.m_scale[0]).cpu().tolist()
            assert ok == [True, False, True, True]
    # blocks of nothing, and of next to nothing
    p = torch.ones(600, device=DEV)
    opt = AdamW([p], lr=LR, state_bits=8, weight_decay=0.0)
    g = torch.zeros(600, device=DEV)
    g[256:] = 1e-25
    opt.step([g])
    assert bool((p[:256] == 1).all()) and bool(torch.isfinite(p).all())
    assert opt.v_scale[0].tolist()[0] == 0 and bool(torch.isfinite(opt.v[0].float()).all())


def test_adamw_refuses_shared_and_wrong_tensors():
    buf = torch.zeros(1024, device=DEV)
    with pytest.raises(ValueError, match="share memory"):
        AdamW([buf[:512], buf[256:]])
    with pytest.raises(ValueError, match="share memory"):
        AdamW([buf, buf])
    with pytest.raises(ValueError, match="contiguous"):
        AdamW([torch.zeros(8, 8, device=DEV).t()])
    with pytest.raises(TypeError):
        AdamW([torch.zeros(8, device=DEV, dtype=torch.float16)])
    opt = AdamW([buf])
    for bad in ([], [torch.zeros(1023, device=DEV)] , [buf, buf]):
        with pytest.raises(ValueError):
            opt.step(bad)
    for bad in (torch.zeros(1024), torch.zeros(1024, device=DEV, dtype=torch.float16), None):
        with pytest.raises(TypeError):
            opt.step([bad])
    with pytest.raises(N.MoeError):                     # an address off its 16 bytes
        AdamW([buf[1:1000]]).step([torch.zeros(999, device=DEV)])


# -------------------------------------------------------------------- streams and graphs
def test_captured_step_replays_with_new_data():
    """Every operator captured in one graph on a side stream, replayed on new inputs, against
    eager calls on the same inputs."""
    T, d, E, k = 200, 512, 16, 4
    wl = workload(T, d=d, E=E, k=k)
    a = on_gpu(norm_inputs(T, d, torch.bfloat16, torch.float32, "all"))
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k))
    R_max = N.moe_workspace_size(wl, N.MOE_WS_ROWS)
    o = torch.randn(R_max, d, generator=gen(1)).bfloat16().to(DEV)
    tok_row = rows_of(ids.cpu(), E, wl.beta).to(DEV)
    dh, dx = torch.randn(T, d, generator=gen(2)).bfloat16().to(DEV), torch.randn(T, d, device=DEV)
    dloss = torch.ones(2, device=DEV)

    def build():
        r, n = RouterLoss(wl, device=DEV), BlockNorm(wl, train=True, device=DEV)
        w = [torch.ones(5000, device=DEV), torch.ones(300, device=DEV, dtype=torch.bfloat16)]
        opt = AdamW(w, lr=LR, state_bits=8)

        def step():
            n(**a)
            r(logits, ids)
            g = n.backward(n.h_out, y=a["y"], gate=a["gate"], w_post=a["w_post"],
                           w_next=a["w_next"], dh_out=dh, dx=dx)
            r.backward(logits, ids, gates, dloss=dloss, dy=g.dy, o=o, tok_row=tok_row)
            opt.step([g.dy.view(-1)[:5000], g.dy.view(-1)[5000 + 24:5324]])
            return [n.h_out, n.x, r.losses, r.counts, *g, r.dlogits, r.dgates, *w, *opt.m,
                    *opt.v_scale, opt.steps]
        return step, opt

    eager, e_opt = build()
    step, g_opt = build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    eager()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        a["y"].normal_()
        logits.normal_()
        for opt in (e_opt, g_opt):
            opt.set_lr(LR / (turn + 1))
        graph.replay()
        want = eager()
        torch.cuda.synchronize()
        assert g_opt.steps.tolist()[:2] == [turn + 2, 0]
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x,
                               y.view(torch.uint8) if y.element_size() == 1 else y)


def test_two_streams_at_once():
    """Objects of their own on two streams, many calls in flight: the results of one stream."""
    wl = workload(3000, d=1024, E=64, k=8)
    logits, ids, _ = (t.to(DEV) for t in router_inputs(3000, 64, 8))
    a = on_gpu(norm_inputs(3000, 1024, torch.bfloat16, torch.bfloat16, "all"))
    dx = torch.randn(3000, 1024, generator=gen(1)).to(DEV)

    def work(obj):
        r, n = obj
        r(logits, ids)
        n(**a)
        n.backward(n.h_out, y=a["y"], gate=a["gate"], w_post=a["w_post"], w_next=a["w_next"],
                   dx=dx)

    objs = [(RouterLoss(wl, device=DEV),
             BlockNorm(wl, w_dtype=torch.bfloat16, train=True, device=DEV)) for _ in range(3)]
    work(objs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for s, obj in zip(streams, objs[1:]):
            with torch.cuda.stream(s):
                work(obj)
    torch.cuda.synchronize()
    for r, n in objs[1:]:
        for x, y in ((r.losses, objs[0][0].losses), (r.probs, objs[0][0].probs),
                     (n.x, objs[0][1].x), (n.dy, objs[0][1].dy),
                     (n.dw_post, objs[0][1].dw_post), (n.dw_next, objs[0][1].dw_next)):
            assert torch.equal(x, y)
    # a stream that is passed, and one of no device of these arrays
    with torch.cuda.stream(streams[0]):
        objs[1][0](logits, ids, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(objs[1][0].losses, objs[0][0].losses)


# ----------------------------------------------------------------------- refused arguments
def test_wrong_arguments_are_refused():
    T, d, E, k = 64, 256, 8, 2
    wl = workload(T, d=d, E=E, k=k)
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k))
    r = RouterLoss(wl, n_seq=2, device=DEV)
    off = torch.tensor([0, 30, T], dtype=torch.int32, device=DEV)
    r(logits, ids, None, off)
    for bad in (dict(logits=logits.half()), dict(logits=logits.cpu()), dict(logits=None),
                dict(topk_ids=ids.long()), dict(seq_off=None), dict(seq_off=off.long()),
                dict(token_mask=torch.ones(T, device=DEV))):
        with pytest.raises(TypeError):
            r(**{**dict(logits=logits, topk_ids=ids, seq_off=off), **bad})
    for bad in (dict(logits=logits[:-1]), dict(logits=logits.t().contiguous().t()),
                dict(seq_off=off[:2]), dict(topk_ids=ids[:, :1]),
                dict(logits=torch.zeros(T, 2 * E, device=DEV))):
        with pytest.raises(ValueError):
            r(**{**dict(logits=logits, topk_ids=ids, seq_off=off), **bad})
    with pytest.raises(ValueError):
        r.backward(logits, ids, gates)
    with pytest.raises(TypeError):
        r.backward(logits, ids, gates, dy=torch.zeros(T, d, device=DEV))
    a = on_gpu(norm_inputs(T, d, torch.bfloat16, torch.float32, "all"))
    n = BlockNorm(wl, device=DEV)
    for bad in (dict(h=a["h"].float()), dict(y=a["y"].bfloat16()), dict(w_post=a["w_post"].half()),
                dict(gate=a["gate"].cpu())):
        with pytest.raises(TypeError):
            n(**{**a, **bad})
    for bad in (dict(y=None), dict(w_next=a["w_next"][:-8]), dict(h=a["h"][:, ::2]),
                dict(gate=a["gate"][:-1])):
        with pytest.raises(ValueError):
            n(**{**a, **bad})
    with pytest.raises(ValueError):
        n(a["h"])
    with pytest.raises(ValueError):
        n.backward(a["h"], dh_out=a["h"])                # built without train
    t = BlockNorm(wl, train=True, device=DEV)
    for bad in (dict(), dict(dh_out=a["h"], dx=a["y"]), dict(w_next=a["w_next"]),
                dict(dh_out=a["h"], gate=a["gate"])):
        with pytest.raises(ValueError):
            t.backward(a["h"], **bad)


def test_longer_arguments_are_refused():
    """A vector that is too long is refused as a short one is; MoeLayer's flat buffers, which are
    longer than their contents, are taken."""
    T, d, E, k = 64, 256, 8, 2
    wl = workload(T, d=d, E=E, k=k)
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k))
    r = RouterLoss(wl, n_seq=2, device=DEV)
    more = lambda t, n=1: torch.cat([t.reshape(-1), t.reshape(-1)[:n]])
    off = torch.tensor([0, 30, T], dtype=torch.int32, device=DEV)
    three = torch.tensor([0, 20, 40, T], dtype=torch.int32, device=DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    dloss = torch.ones(2, device=DEV)
    for name, bad in (("seq_off", three), ("token_mask", more(mask)), ("logits", more(logits))):
        with pytest.raises(ValueError, match=name):
            r(**{**dict(logits=logits, topk_ids=ids, seq_off=off), name: bad})
        with pytest.raises(ValueError, match=name):
            r.backward(**{**dict(logits=logits, dloss=dloss, seq_off=off), name: bad})
    with pytest.raises(ValueError, match="dloss"):
        r.backward(logits, dloss=torch.ones(3, device=DEV), seq_off=off)
    a = on_gpu(norm_inputs(T, d, torch.bfloat16, torch.float32, "all"))
    n = BlockNorm(wl, train=True, device=DEV)
    dx = torch.randn(T, d, device=DEV)
    for name in ("h", "gate", "w_post", "w_next"):
        with pytest.raises(ValueError, match=name):
            n(**{**a, name: more(a[name])})
    for name in ("gate", "w_post", "w_next", "dh_out"):
        b = dict(y=a["y"], gate=a["gate"], w_post=a["w_post"], w_next=a["w_next"],
                 dh_out=a["h"], dx=dx)
        with pytest.raises(ValueError, match=name):
            n.backward(a["h"], **{**b, name: more(b[name])})
    n_p = 300
    p = lambda dt=torch.float32: torch.zeros(n_p, dtype=dt, device=DEV)
    z = lambda n, dt=torch.float32: [torch.zeros(n, device=DEV).to(dt)]
    e4 = torch.float8_e4m3fn
    for kw in (dict(m=z(301)), dict(v=z(301)), dict(state_bits=8, m=z(301, e4)),
               dict(state_bits=8, m_scale=z(3)), dict(state_bits=8, v_scale=z(3))):
        with pytest.raises(ValueError, match="contiguous with"):
            AdamW([p()], **kw)
    with pytest.raises(ValueError, match="master"):
        AdamW([p(torch.bfloat16)], master=z(301))
    with pytest.raises(ValueError, match="grad_scale"):
        AdamW([p()]).step([p()], grad_scale=torch.ones(2, device=DEV))
    # what MoeLayer owns
    want = r(logits, ids, None, off).clone()
    assert torch.equal(r(logits, more(ids, 7), None, off), want)
    R_max = N.moe_workspace_size(wl, N.MOE_WS_ROWS)
    o = torch.randn(R_max, d, generator=gen(1)).bfloat16().to(DEV)
    rows = rows_of(ids.cpu(), E, wl.beta).to(DEV)
    want = r.backward(topk_ids=ids, topk_gates=gates, dy=dx, o=o, tok_row=rows).clone()
    got = r.backward(topk_ids=more(ids, 7), topk_gates=more(gates, 7), dy=dx, o=more(o, 9),
                     tok_row=more(rows, 5))
    assert torch.equal(got, want)
    want = n(**a)[1].clone()
    assert torch.equal(n(**{**a, "y": more(a["y"], 4)})[1], want)


def test_rows_around_the_outputs_stay():
    """Guard elements around every output of the C ABI calls stay as they were."""
    T, d, E, k, G = 37, 264, 12, 3, 64
    wl = workload(T, d=d, E=E, k=k)
    cfg = N.MoeCfg.of(wl)
    a = on_gpu(norm_inputs(T, d, torch.bfloat16, torch.float32, "all"))
    logits, ids, gates = (t.to(DEV) for t in router_inputs(T, E, k))
    guards = []

    def out(n, dt=torch.float32):
        buf = torch.full((G + n + G,), 77, dtype=dt, device=DEV)
        guards.append((buf, n))
        return buf[G:G + n]

    status = torch.zeros(4, dtype=torch.int32, device=DEV)
    ws = out(N.moet_workspace_size(wl, 1, N.MOET_WS_BALANCE), torch.uint8)
    losses, counts, probs = out(4), out(E, torch.int32), out(E)
    info, lse, dlogits, dgates = out(3, torch.int32), out(T), out(T * E), out(T * k)
    N.moet_balance_loss(cfg, logits, ids, None, None, 1, losses, counts, probs, info, lse, ws,
                        status)
    R_max = N.moe_workspace_size(wl, N.MOE_WS_ROWS)
    o = torch.zeros(R_max, d, dtype=torch.bfloat16, device=DEV)
    N.moet_router_backward(cfg, logits, ids, gates, a["y"], o, rows_of(ids.cpu(), E, 64).to(DEV),
                           None, None, 1, counts, info, lse, losses, dgates, dlogits, status)
    norm = N.MoetNorm(1e-6, 0, 1, 1, N.MOET_BF16, N.MOET_F32)
    h_out, x = out(T * d, torch.bfloat16), out(T * d, torch.bfloat16)
    N.moet_block_norm(cfg, norm, a["h"], a["y"], a["gate"], a["w_post"], a["w_next"], h_out, x)
    dh, dy, dgate, dwp, dwn = out(T * d, torch.bfloat16), out(T * d), out(T), out(d), out(d)
    ws2 = out(N.moet_workspace_size(wl, 1, N.MOET_WS_NORM_BWD), torch.uint8)
    N.moet_block_norm_backward(cfg, norm, h_out, a["y"], a["gate"], a["w_post"], a["w_next"],
                               a["h"], a["y"], dh, dy, dgate, dwp, dwn, ws2)
    for n in (1, 255, 257, 4099):
        for bits, dt in ((32, torch.float32), (8, torch.uint8)):
            nb = -(-n // 256)
            p, m, v = out(n, torch.bfloat16), out(n, dt), out(n, dt)
            sm, sv = (out(nb), out(nb)) if bits == 8 else (None, None)
            mw = out(n)
            for t in (m, v, sm, sv):
                if t is not None:
                    t.zero_()
            g = torch.ones(n, device=DEV)
            ptr = lambda t: None if t is None else t.data_ptr()
            e = (N.MoetAdamwTensor * 1)(N.MoetAdamwTensor(
                ptr(p), ptr(g), ptr(m), ptr(v), ptr(sm), ptr(sv), ptr(mw), n, 0.1, N.MOET_BF16,
                N.MOET_F32, N.MOET_F32 if bits == 32 else N.MOET_E4M3))
            steps = torch.zeros(4, dtype=torch.int32, device=DEV)
            N.moet_adamw_step(e, 1, N.MoetAdamw(0.9, 0.95, 1e-8),
                              torch.full((4,), 1e-3, device=DEV), None, steps)
            torch.cuda.synchronize()
            assert bool((mw < 77).all())
    torch.cuda.synchronize()
    for buf, n in guards:
        assert bool((buf[:G] == 77).all()) and bool((buf[G + n:] == 77).all())
