"""Host-side checks of the training operators: exports, constants, workspace sizes, and the
refusals (before anything is launched), on the CPU; and the 64-bit forms that the GPU tests
compare with, against differences."""
import ctypes
import re
import subprocess

import pytest
import torch

import train_oracle as R
from skew_aware_token_b200 import build as B
from skew_aware_token_b200 import native as N
from skew_aware_token_b200.synth import WORKLOADS

NO_GPU = not torch.cuda.is_available()
no_gpu = pytest.mark.skipif(not NO_GPU, reason="fake pointers are only passed where no GPU exists")
OK = 1 << 20
INVALID, UNSUPPORTED = N.MOE_ERR_INVALID_ARG, N.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built_library():
    B.build()
    return N.lib()


def cfg(**kw):
    return ctypes.byref(N.MoeCfg.of(WORKLOADS["tiny"].with_(**kw)))


def test_header_binding_and_exports_agree():
    text = open(N.TRAIN_HEADER_PATH).read()
    declared = set(re.findall(r"MOE_API\s+[\w\s\*]+?\b(moet_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", N.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {w for w in (line.split()[-1] for line in out.splitlines() if " T " in line)
                if w.startswith("moet_")}
    assert declared == exported == {n for n in N._SIGNATURES if n.startswith("moet_")}
    enum = {m.group(1): int(m.group(2)) for m in re.finditer(r"\b(MOET_\w+)\s*=\s*(\d+)", text)}
    enum.update({m.group(1): int(m.group(2))
                 for m in re.finditer(r"#define (MOET_\w+) (\d+)", text)})
    for name, val in enum.items():
        assert getattr(N, name) == val, name
    assert N.moe_status_string(N.MOET_STATUS_BAD_SEQ) not in ("", "unknown code",
                                                              "several device status bits")


def test_workspace_sizes():
    size = N.moet_workspace_size
    for wl in (WORKLOADS["tiny"], WORKLOADS["dsv3_a1"]):
        assert size(wl, 1, N.MOET_WS_BALANCE) > 0
        assert size(wl, 700, N.MOET_WS_BALANCE) > size(wl, 1, N.MOET_WS_BALANCE)
        assert size(wl, 1, N.MOET_WS_NORM_BWD) >= 2 * wl.d * 4
        assert size(wl, 0, N.MOET_WS_BALANCE) == 0
        assert size(wl, (1 << 20) + 1, N.MOET_WS_BALANCE) == 0
        assert size(wl, 1, 2) == 0
    for bad in (dict(d=516), dict(d=N.MOET_MAX_NORM_D + 8), dict(k=9)):
        assert size(WORKLOADS["tiny"].with_(**bad), 1, N.MOET_WS_NORM_BWD) == 0


BALANCE = dict(logits=OK, ids=OK, mask=None, off=None, n_seq=1, losses=OK, counts=OK, probs=OK,
               info=OK, lse=OK, ws=OK, status=OK)
ROUTER = dict(logits=OK, ids=OK, gates=OK, dy=OK, o=OK, tok_row=OK, mask=None, off=None, n_seq=1,
              counts=OK, info=OK, lse=OK, dloss=OK, dgates=OK, dlogits=OK, status=OK)
NORM = dict(h=OK, y=OK, gate=OK, w_post=OK, w_next=OK, h_out=OK, x=OK)
NORM_BWD = dict(h_out=OK, y=OK, gate=OK, w_post=OK, w_next=OK, dh_out=OK, dx=OK, dh=OK, dy=OK,
                dgate=OK, dw_post=OK, dw_next=OK, ws=OK)


def call(fn, base, c=None, first=(), **change):
    args = dict(base)
    assert not set(change) - set(args)
    args.update(change)
    return getattr(N.lib(), fn)(c or cfg(), *first, *args.values(), None)


@no_gpu
def test_balance_loss_refusals():
    f = "moet_balance_loss"
    for name in ("logits", "ids", "losses", "counts", "probs", "info", "lse", "ws", "status"):
        assert call(f, BALANCE, **{name: None}) == INVALID, name
        assert call(f, BALANCE, **{name: OK + 4}) == UNSUPPORTED, name
    assert call(f, BALANCE, mask=OK + 1) == UNSUPPORTED
    assert call(f, BALANCE, off=OK + 4) == UNSUPPORTED
    for n in (0, -1, (1 << 20) + 1):
        assert call(f, BALANCE, off=OK, n_seq=n) == INVALID
    assert call(f, BALANCE, n_seq=2) == INVALID          # sequences without their bounds
    assert call(f, BALANCE, cfg(k=9)) == INVALID
    assert call(f, BALANCE, cfg(E=300)) == UNSUPPORTED
    assert N.lib().moet_balance_loss(None, *BALANCE.values(), None) == INVALID


@no_gpu
def test_router_backward_refusals():
    f = "moet_router_backward"
    for name in ("ids", "gates", "dy", "o", "tok_row", "dlogits", "status", "logits", "lse",
                 "counts", "info"):
        assert call(f, ROUTER, **{name: None}) == INVALID, name
        assert call(f, ROUTER, **{name: OK + 8}) == UNSUPPORTED, name
    for name in ("mask", "off", "dgates", "dloss"):
        assert call(f, ROUTER, **{name: OK + 4}) == UNSUPPORTED, name
    nothing = dict(dy=None, o=None, tok_row=None)
    assert call(f, ROUTER, dloss=None, dgates=None, **nothing) == INVALID
    assert call(f, ROUTER, **nothing) == INVALID         # dgates without the gates' part
    assert call(f, ROUTER, n_seq=2) == INVALID
    assert call(f, ROUTER, cfg(d=516)) == UNSUPPORTED


def norm_of(**kw):
    a = dict(eps=1e-6, w_offset=0.0, res_scale=1.0, out_scale=1.0, h_dtype=1, w_dtype=0)
    a.update(kw)
    return ctypes.byref(N.MoetNorm(*a.values()))


@no_gpu
def test_block_norm_refusals():
    f, n = "moet_block_norm", norm_of()
    for name in ("h", "h_out", "x", "w_next"):
        assert call(f, NORM, first=(n,), **{name: None}) == INVALID, name
    for name in NORM:
        assert call(f, NORM, first=(n,), **{name: OK + 8}) == UNSUPPORTED, name
    assert call(f, NORM, first=(None,)) == INVALID
    alone = dict(y=None, gate=None, w_post=None, h_out=None)
    for name in ("gate", "w_post", "h_out"):
        assert call(f, NORM, first=(n,), **{**alone, name: OK}) == INVALID, name
    assert call(f, NORM, first=(n,), **alone, w_next=None, x=None) == INVALID
    for bad in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(h_dtype=2),
                dict(w_dtype=-1), dict(out_scale=float("inf")), dict(res_scale=float("nan"))):
        assert call(f, NORM, first=(norm_of(**bad),)) == INVALID, bad
    for d in (516, N.MOET_MAX_NORM_D + 8):
        assert call(f, NORM, cfg(d=d), first=(n,)) == UNSUPPORTED


@no_gpu
def test_block_norm_backward_refusals():
    f, n = "moet_block_norm_backward", norm_of()
    for name in ("h_out", "dh", "ws", "dy", "dx", "w_next", "dgate", "dw_post", "dw_next",
                 "gate", "w_post"):
        assert call(f, NORM_BWD, first=(n,), **{name: None}) == INVALID, name
    for name in NORM_BWD:
        assert call(f, NORM_BWD, first=(n,), **{name: OK + 8}) == UNSUPPORTED, name
    assert call(f, NORM_BWD, first=(n,), y=None) == INVALID
    assert call(f, NORM_BWD, first=(n,), dh_out=None, dx=None, w_next=None,
                dw_next=None) == INVALID


def tensors(**kw):
    a = dict(p=OK, g=OK, m=OK, v=OK, m_scale=None, v_scale=None, master=None, n=100,
             weight_decay=0.1, p_dtype=0, g_dtype=0, state_dtype=0)
    a.update(kw)
    return (N.MoetAdamwTensor * 1)(N.MoetAdamwTensor(*a.values()))


@no_gpu
def test_adamw_refusals():
    step = N.lib().moet_adamw_step
    opt = N.MoetAdamw(0.9, 0.99, 1e-8)

    def go(ts=None, n=1, o=opt, lr=OK, gs=None, st=OK):
        return step(tensors() if ts is None else ts, n, ctypes.byref(o), lr, gs, st, None)

    for name in ("p", "g", "m", "v"):
        assert go(tensors(**{name: None})) == INVALID, name
        assert go(tensors(**{name: OK + 4})) == UNSUPPORTED, name
    assert go(tensors(master=OK)) == INVALID             # fp32 weights have none
    assert go(tensors(master=OK + 2, p_dtype=1)) == UNSUPPORTED
    assert go(tensors(m_scale=OK, v_scale=OK)) == INVALID
    assert go(tensors(state_dtype=2)) == INVALID         # 8-bit states without scales
    assert go(tensors(state_dtype=2, m_scale=OK)) == INVALID
    assert go(tensors(v_scale=OK)) == INVALID
    assert go(tensors(state_dtype=2, m_scale=OK + 2, v_scale=OK)) == UNSUPPORTED
    for bad in (dict(n=-1), dict(p_dtype=2), dict(g_dtype=2), dict(g_dtype=-1),
                dict(state_dtype=1), dict(weight_decay=float("nan"))):
        assert go(tensors(**bad)) == INVALID, bad
    assert go(tensors(n=(1 << 40) + 1)) == UNSUPPORTED
    for bad in ((1.0, 0.9, 1e-8), (-0.1, 0.9, 1e-8), (0.9, 1.0, 1e-8), (0.9, 0.9, 0.0),
                (0.9, 0.9, -1.0), (0.9, 0.9, 1e-40), (float("nan"), 0.9, 1e-8),
                (0.9, 0.9, float("inf"))):
        assert go(o=N.MoetAdamw(*bad)) == INVALID, bad
    assert go(lr=None) == INVALID and go(st=None) == INVALID
    assert go(lr=OK + 4) == UNSUPPORTED and go(gs=OK + 4) == UNSUPPORTED
    assert go(n=-1) == INVALID
    assert step(None, 1, ctypes.byref(opt), OK, None, OK, None) == INVALID
    assert step(tensors(), 1, None, OK, None, OK, None) == INVALID


@no_gpu
def test_adamw_refuses_an_eps_without_a_reciprocal():
    """An eps whose fp32 reciprocal the step's approximate one flushes to 0."""
    for far in (2.0 ** 101, 1e38, 3e38):
        opt = N.MoetAdamw(0.9, 0.9, far)
        assert N.lib().moet_adamw_step(tensors(), 1, ctypes.byref(opt), OK, None, OK,
                                       None) == INVALID, far


def test_classes_refuse_the_cpu():
    from skew_aware_token_b200 import train
    wl = WORKLOADS["tiny"]
    with pytest.raises(ValueError):
        train.RouterLoss(wl, device="cpu")
    with pytest.raises(ValueError):
        train.BlockNorm(wl, device="cpu")
    with pytest.raises(TypeError):
        train.AdamW([torch.zeros(4)])
    with pytest.raises(ValueError):
        train.AdamW([])
    for bad in (dict(n_seq=0), dict(n_seq=-3)):
        with pytest.raises(ValueError):
            train.RouterLoss(wl, **bad)
    with pytest.raises(ValueError):
        train.BlockNorm(wl.with_(d=516))
    with pytest.raises(ValueError):
        train.BlockNorm(wl, h_dtype=torch.float16)


def test_router_gradient_wants_the_last_forwards_rows(monkeypatch):
    """A layer's router gradient runs after a forward that wrote O rows, and is refused before
    any, after one that wrote none, and once the next batch has been routed."""
    from skew_aware_token_b200.layer import MoeLayer
    for name in ("moe_route_hist", "moe_block_offsets", "moe_plan_blocks", "moe_combine",
                 "moe_dispatch_permute", "moe_expert_ffn"):
        monkeypatch.setattr(N, name, lambda *a, **kw: None)
    taken = []

    class Router:
        def backward(self, *a, **kw):
            taken.append(kw["o"])

    refused = lambda: pytest.raises(ValueError, match="o_rows")
    go = lambda layer: layer.router_backward(Router(), None, None)
    forward = lambda layer, mode: layer(None, None, None, None, mode=mode, stream=1)
    fused, one, wide = N.MOE_FFN_FUSED_COMBINE, N.MOE_FFN_ONE_LAUNCH, N.MOE_FFN_WRITE_O
    layer = MoeLayer(WORKLOADS["tiny"], "cpu", train=True, o_rows=True)
    with refused():
        go(layer)                               # no forward yet
    forward(layer, fused)
    go(layer)
    assert taken[-1] is layer.o
    forward(layer, one)                         # fuses the combine whatever o_rows says
    with refused():
        go(layer)
    forward(layer, fused)
    go(layer)
    layer.pre_ffn(None, None, stream=1)         # the next batch's row maps
    with refused():
        go(layer)
    layer = MoeLayer(WORKLOADS["tiny"], "cpu", train=True, write_o=True, o_rows=False)
    forward(layer, wide)
    go(layer)
    assert len(taken) == 3 and taken[-1] is layer.o
    forward(layer, fused)
    with refused():
        go(layer)


def test_gradient_lists_are_checked():
    """The native reader of gradient lists refuses what is not a list of the right tensors and
    says which one it is."""
    sizes, t = (ctypes.c_int64 * 3)(5, 5, 5), (N.MoetAdamwTensor * 3)()
    host = [torch.zeros(5) for _ in range(3)]
    for bad, error, text in (
            (host, TypeError, r"grads\[0\] must be on cuda:0"),
            ([1, 2, 3], TypeError, r"grads\[0\] must be a torch"), (host[:2], ValueError, "list of 3"),
            ((None,) * 3, TypeError, r"grads\[0\]"), (torch.zeros(3), ValueError, "list of 3"),
            ([torch.zeros(5, dtype=torch.int32)] * 3, TypeError, r"grads\[0\] must be a torch"),
            ([torch.zeros(5, dtype=torch.float64)] * 3, TypeError, r"grads\[0\]"),
            ([torch.zeros(5, device="meta")] * 3, TypeError, r"grads\[0\] must be on"),
            ([torch.zeros(5).to_sparse()] * 3, TypeError, r"grads\[0\] must be on")):
        with pytest.raises(error, match=text):
            N.read_step(bad, host, sizes, 0, t)
    assert all(not e.g for e in t)


def test_args_library_belongs_to_one_torch(monkeypatch):
    """The library that reads torch's objects says which torch and interpreter it was built for;
    for another one it is built again, and not loaded before that."""
    target = B.args_target()
    assert torch.__version__ in target and B.args_built_for() == target
    assert B._args_up_to_date() and B.up_to_date()
    N._args()
    monkeypatch.setattr(B, "args_target", lambda: target.replace(torch.__version__, "1.0.0"))
    assert not B._args_up_to_date() and not B.up_to_date()
    monkeypatch.setattr(N, "_args_lib", None)
    with pytest.raises(RuntimeError, match="was built for"):
        N._args()


@pytest.mark.parametrize("lacking", ["torch", "headers", "compiler", "nothing"])
def test_the_library_builds_without_torch(monkeypatch, tmp_path, capsys, lacking):
    """libmoeskew.so needs neither torch nor g++: without them the build makes it and leaves
    libmoeskew_args.so out.  (Stand-ins for the compilers that write what they are asked for.)"""
    import stat
    for name in ("nvcc", "g++"):
        tool = tmp_path / name
        tool.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\necho made > "$2"\n')
        tool.chmod(tool.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / ("none" if lacking == "compiler" else "g++")))
    for name in ("LIB", "ARGS_LIB", "BUILD"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    if lacking == "torch":
        find = B.importlib.util.find_spec
        monkeypatch.setattr(B.importlib.util, "find_spec",
                            lambda n: None if n == "torch" else find(n))
    elif lacking == "headers":
        monkeypatch.setattr(B, "_torch_dir", lambda: str(tmp_path))
    for force in (False, True):
        assert B.build(force=force) == B.LIB and (tmp_path / "LIB").exists()
    out = capsys.readouterr().err
    if lacking == "nothing":
        assert (tmp_path / "ARGS_LIB").exists() and not out
    else:
        assert not (tmp_path / "ARGS_LIB").exists() and "is left out" in out
        assert B.up_to_date()


def test_state_lists_are_checked():
    """A step's state lists are read with it: one of another length is named."""
    sizes, t = (ctypes.c_int64 * 3)(5, 5, 5), (N.MoetAdamwTensor * 3)()
    host = [torch.zeros(5) for _ in range(3)]
    for j, name in enumerate(("m", "v", "m_scale", "v_scale", "master")):
        states = [None] * 5
        states[j] = host[:2]
        with pytest.raises(ValueError, match=f"list of 3 {name} is needed"):
            N.read_step(host, host, sizes, 0, t, tuple(states))


# ---- the 64-bit forms, against differences ----
def _g(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def test_router_losses_differences():
    x = torch.randn(9, 5, generator=_g(0), dtype=torch.float64, requires_grad=True)
    ids = torch.randint(0, 5, (9, 2), generator=_g(1))
    mask, off = [1, 0, 1, 1, 1, 1, 0, 1, 1], [1, 4, 4, 8]
    f = lambda x: R.router_losses(x, ids, mask, off)[:2]
    assert torch.autograd.gradcheck(f, (x,), eps=1e-6, atol=1e-8)
    # by hand: uniform logits give P = 1/E, so the balance loss is 1 and z = (log E)^2
    b, z, c, p, _ = R.router_losses(torch.zeros(9, 5), ids, None, None)
    assert abs(float(b) - 1) < 1e-12 and abs(float(z) - torch.log(torch.tensor(5.0).double()) ** 2) < 1e-12
    assert float(c.sum()) == 18 and abs(float(p.sum()) - 1) < 1e-12


def test_block_norm_differences():
    mk = lambda *s, seed: torch.randn(*s, generator=_g(seed), dtype=torch.float64,
                                      requires_grad=True)
    h, y, g = mk(3, 8, seed=1), mk(3, 8, seed=2), mk(3, seed=3)
    wp, wn = mk(8, seed=4), mk(8, seed=5)
    f = lambda h, y, g, wp, wn: R.block_norm(h, y, g, wp, wn, eps=1e-2, w_offset=1.0,
                                             res_scale=0.5, out_scale=0.7)
    assert torch.autograd.gradcheck(f, (h, y, g, wp, wn), eps=1e-6, atol=1e-7)


def test_8bit_form_round_trip():
    x = torch.randn(1000, generator=_g(7)) * torch.logspace(-6, 0, 1000)
    for v, root in ((x, False), (x.abs(), True)):
        c, s = R.to_8bit(v, root)
        back = R.of_8bit(c, s)
        scale = s.repeat_interleave(256)[:1000]
        floor = scale * 2.0 ** (-9 if root else -10)
        # half an e4m3 step, or half (a clamped root: one) smallest subnormal
        assert bool(((back - v).abs() <= v.abs() * 2.0 ** -4 * 1.001 + floor * 1.001).all())
    assert int((R.to_8bit(x.abs(), True)[0].float() == 0).sum()) == 0
    c, s = R.to_8bit(torch.zeros(300), True)
    assert s.tolist() == [0, 0] and float(c.float().abs().max()) == 0
