"""Training the block around the expert computation: the router's losses and gradient, the
norms before and after the block, and the weights' AdamW step.  Each class owns its output
buffers, as MoeLayer does, and calls the library's kernels (include/moeskew_train.h) on the
current CUDA stream of its device, or on `stream`.  One object serves one stream at a time;
its outputs are views that the next call overwrites.

    norm_in, norm_out = BlockNorm(wl, train=True), BlockNorm(wl, train=True)
    router = RouterLoss(wl, n_seq=3)
    opt = AdamW([w1, w2], lr=1e-3, state_bits=8)
    layer = MoeLayer(wl, train=True, o_rows=True)

    _, x = norm_in(h, w_next=w_in)                     # the norm before the block
    y = layer(logits, x, w1, w2)
    losses = router(logits, layer.view("topk_ids"), seq_off=seq_off)
    h_out, _ = norm_out(h, y=y, w_post=w_out)          # the norm and residual behind it
    ...
    g = norm_out.backward(h_out, y=y, w_post=w_out, dh_out=dh_out)
    dx, dw1, dw2 = layer.backward(g.dy, w1, w2)
    dlogits = layer.router_backward(router, logits, g.dy, dloss=dloss, seq_off=seq_off)
    opt.step([dw1, dw2])
"""
from __future__ import annotations

import collections
import ctypes

import torch

from . import native as N

_TYPES = {torch.float32: N.MOET_F32, torch.bfloat16: N.MOET_BF16,
          torch.float8_e4m3fn: N.MOET_E4M3}


def _device(device) -> torch.device:
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("the training operators run on a CUDA device")
    return torch.device("cuda", torch.cuda.current_device()) if dev.index is None else dev


# The current device and its current stream's handle without the objects around them (a fifth
# of a small call's time).
_device_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _OnDevice:
    """Runs a call with the object's device current and the stream resolved on it."""

    def _on(self, device):
        self.device = device
        self._index = device.index

    def _settle(self):
        """The buffers' first fill is done when the object is, whatever stream it is used on."""
        with torch.cuda.device(self._index):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def _call(self, fn, args, stream):
        index = self._index
        if stream is None:
            stream = _raw_stream(index)
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device != self.device:
                raise ValueError(f"the stream is on {stream.device}, the arrays on {self.device}")
            stream = stream.cuda_stream
        else:
            stream = int(stream)
        if _device_index() == index:
            N.call(fn, *args, stream)
        else:
            with torch.cuda.device(index):
                N.call(fn, *args, stream)


class RouterLoss(_OnDevice):
    """Balance loss, z loss, per-expert counts and the gradient of the router's logits, for a
    batch of `n_seq` packed sequences (moet_balance_loss, moet_router_backward)."""

    def __init__(self, wl, n_seq: int = 1, device="cuda"):
        self.cfg = wl if isinstance(wl, N.MoeCfg) else N.MoeCfg.of(wl)
        self.n_seq = int(n_seq)
        size = N.moet_workspace_size(self.cfg, self.n_seq, N.MOET_WS_BALANCE)
        if size == 0:
            raise ValueError("configuration or n_seq rejected by moet_workspace_size")
        dev = _device(device)
        self._on(dev)
        self._cfg = ctypes.byref(self.cfg)
        T, E, k, S = self.cfg.T, self.cfg.E, self.cfg.k, self.n_seq
        z = lambda *shape, dt=torch.float32: torch.zeros(shape, dtype=dt, device=dev)
        new = lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=dev)
        self.losses, self.probs = new(2), new(S, E)
        self.counts, self.seq_info = z(S, E, dt=torch.int32), z(S + 2, dt=torch.int32)
        self._lse = z(max(T, 1))
        self._dgates, self._dlogits = new(max(T * k, 1)), new(max(T * E, 1))
        self.lse = self._lse[:T]
        self.dgates = self._dgates[:T * k].view(T, k)
        self.dlogits = self._dlogits[:T * E].view(T, E)
        self.workspace = new(size, dt=torch.uint8)
        self.status = z(4, dt=torch.int32)
        f32, i32, rows = torch.float32, torch.int32, N.moe_workspace_size(self.cfg, N.MOE_WS_ROWS)
        flat, opt = N.ARG_FLAT, N.ARG_OPTIONAL  # flat: what MoeLayer hands out
        batch = (("token_mask", torch.uint8, T, opt), ("seq_off", i32, S + 1, opt * (S == 1)))
        x, ids = ("logits", f32, T * E, 0), ("topk_ids", i32, T * k, flat)
        through_gates = (ids, ("topk_gates", f32, T * k, flat), ("dy", f32, T * self.cfg.d, 0),
                         ("o", torch.bfloat16, rows * self.cfg.d, flat),
                         ("tok_row", i32, T * k, flat))
        through_losses = (("dloss", f32, 2, 0), x, *batch)
        # the buffers above are read with each call's arguments, in the entry points' order:
        # an exchanged one is written where it is, or refused
        own = lambda name, dt=f32: (name, dt, getattr(self, name).numel(), 0)
        saved = (own("counts", i32), own("seq_info", i32), own("_lse"))
        grads = (own("_dgates"), own("_dlogits"), own("status", i32))
        index = self._index
        self._loss_args = N.Arguments(index, x, ids, *batch, own("losses"), own("counts", i32),
                                      own("probs"), own("seq_info", i32), own("_lse"),
                                      own("workspace", torch.uint8), own("status", i32))
        self._gate_args = N.Arguments(index, *through_gates, *saved, *grads)
        self._dloss_args = N.Arguments(index, *through_losses, *saved, *grads)
        self._both_args = N.Arguments(index, *through_gates, *through_losses, *saved, *grads)
        self._forward_ran = False
        self._settle()

    def __call__(self, logits, topk_ids, token_mask=None, seq_off=None, stream=None):
        """fp32 [2]: balance loss and z loss of logits fp32 [T, E] and the router's topk_ids
        int32 [T, k].  token_mask uint8 [T] leaves tokens out; seq_off int32 [n_seq + 1] are
        the sequences' bounds (None with one sequence: the whole batch)."""
        a = self._loss_args.read(logits, topk_ids, token_mask, seq_off, self.losses, self.counts,
                                 self.probs, self.seq_info, self._lse, self.workspace, self.status)
        if self.cfg.T == 0:  # empty tensors have no address
            a[0] = a[1] = a[4]
        # (taken one by one: to unpack the array costs a microsecond)
        self._call("moet_balance_loss", (self._cfg, a[0], a[1], a[2], a[3], self.n_seq, a[4], a[5],
                                         a[6], a[7], a[8], a[9], a[10]), stream)
        self._forward_ran = True
        return self.losses

    def backward(self, logits=None, topk_ids=None, topk_gates=None, dloss=None, dy=None, o=None,
                 tok_row=None, token_mask=None, seq_off=None, stream=None):
        """dlogits fp32 [T, E]: the losses' part with dloss (fp32 [2], their gradient; after
        the forward call on the same logits, ids, mask and sequences), the gates' part with
        dy (fp32 [T, d]), o (the expert output rows, bf16 [R_max, d]) and tok_row, or both.
        The gates' gradient is in `dgates` then."""
        gates = dy is not None or o is not None or tok_row is not None
        own = (self.counts, self.seq_info, self._lse, self._dgates, self._dlogits, self.status)
        if gates and dloss is not None:
            a = self._both_args.read(topk_ids, topk_gates, dy, o, tok_row, dloss, logits,
                                     token_mask, seq_off, *own)
            via, dl, x, mask, off, at = (a[0], a[1], a[2], a[3], a[4]), a[5], a[6], a[7], a[8], 9
        elif gates:
            a = self._gate_args.read(topk_ids, topk_gates, dy, o, tok_row, *own)
            via, dl, x, mask, off, at = (a[0], a[1], a[2], a[3], a[4]), None, None, None, None, 5
        elif dloss is not None:
            a = self._dloss_args.read(dloss, logits, token_mask, seq_off, *own)
            via, dl, x, mask, off, at = (None,) * 5, a[0], a[1], a[2], a[3], 4
        else:
            raise ValueError("nothing to take the gradient of: give dloss, or dy, o and tok_row")
        if dloss is not None and not self._forward_ran:
            raise ValueError("the losses' gradient follows a forward call: it reads what that left")
        if self.cfg.T == 0:
            return self.dlogits
        self._call("moet_router_backward",
                   (self._cfg, x, *via, mask, off, self.n_seq, a[at], a[at + 1], a[at + 2], dl,
                    a[at + 3] if gates else None, a[at + 4], a[at + 5]), stream)
        return self.dlogits

    def clear_status(self):
        self.status.zero_()

    def read_status(self) -> int:
        return int(self.status[0].item())


BlockNormGrads = collections.namedtuple("BlockNormGrads", "dh dy dgate dw_post dw_next")


class BlockNorm(_OnDevice):
    """The norms before and after a block with the block's gate and residual scale, over T
    rows of width d (moet_block_norm, moet_block_norm_backward):

        h_out = res_scale h + out_scale gate norm(y; w_post),   x = bf16(norm(h_out; w_next))

    `train` holds the backward's buffers too."""

    def __init__(self, wl, h_dtype=torch.bfloat16, w_dtype=torch.float32, eps: float = 1e-6,
                 w_offset: float = 0.0, res_scale: float = 1.0, out_scale: float = 1.0,
                 train: bool = False, device="cuda"):
        self.cfg = wl if isinstance(wl, N.MoeCfg) else N.MoeCfg.of(wl)
        for t in (h_dtype, w_dtype):
            if t not in (torch.float32, torch.bfloat16):
                raise ValueError("h_dtype and w_dtype are torch.float32 or torch.bfloat16")
        if not eps > 0:
            raise ValueError("eps must be above 0")
        size = N.moet_workspace_size(self.cfg, 1, N.MOET_WS_NORM_BWD)
        if size == 0:
            raise ValueError("configuration rejected by moet_workspace_size (d % 8 == 0 and "
                             f"d <= {N.MOET_MAX_NORM_D} are needed)")
        dev = _device(device)
        self._on(dev)
        T, d = self.cfg.T, self.cfg.d
        self.h_dtype, self.w_dtype, self.train = h_dtype, w_dtype, bool(train)
        self.norm = N.MoetNorm(eps, w_offset, res_scale, out_scale, _TYPES[h_dtype],
                               _TYPES[w_dtype])
        new = lambda dt, *shape: torch.empty(shape, dtype=dt, device=dev)
        rows = max(T, 1)
        self.h_out, self.x = new(h_dtype, rows, d)[:T], new(torch.bfloat16, rows, d)[:T]
        if train:
            self.dh, self.dy = new(h_dtype, rows, d)[:T], new(torch.float32, rows, d)[:T]
            self.dgate = new(torch.float32, rows)[:T]
            self.dw_post, self.dw_next = new(torch.float32, d), new(torch.float32, d)
            self.workspace = new(torch.uint8, size)
        self._refs = (ctypes.byref(self.cfg), ctypes.byref(self.norm))
        f32, rows = torch.float32, T * d
        opt, flat = N.ARG_OPTIONAL, N.ARG_OPTIONAL | N.ARG_FLAT  # flat: what MoeLayer hands out
        inputs = (("h", h_dtype, rows, 0), ("y", f32, rows, flat), ("gate", f32, T, opt),
                  ("w_post", w_dtype, d, opt), ("w_next", w_dtype, d, opt))
        # with the object's own buffers, in the entry points' order: an exchanged one is written
        # where it is, or refused
        self._args = N.Arguments(self._index, *inputs, ("h_out", h_dtype, rows, opt),
                                 ("x", torch.bfloat16, rows, opt))
        self._grad_args = N.Arguments(
            self._index, *inputs, ("dh_out", h_dtype, rows, opt), ("dx", f32, rows, flat),
            ("dh", h_dtype, rows, 0), ("dy", f32, rows, opt), ("dgate", f32, T, opt),
            ("dw_post", f32, d, opt), ("dw_next", f32, d, opt),
            ("workspace", torch.uint8, size, 0))
        self._settle()

    def __call__(self, h, y=None, gate=None, w_post=None, w_next=None, h_out=None, stream=None):
        """(h_out, x): the residual stream behind the block and, with w_next, the next
        block's bf16 rows.  Without y, h_out is h itself (a norm before the first block).
        `h_out=` takes the result's place in the caller's buffer; it may be h itself."""
        if y is None:
            if w_next is None:
                raise ValueError("nothing to compute: give y, w_next or both")
            if gate is not None or w_post is not None or h_out is not None:
                raise ValueError("gate, w_post and h_out belong to y")
        elif h_out is None:
            h_out = self.h_out
        x = None if w_next is None else self.x
        arrays = self._args.read(h, y, gate, w_post, w_next, h_out, x)
        if self.cfg.T:
            self._call("moet_block_norm", (*self._refs, *arrays), stream)
        return (h if y is None else h_out), x

    def backward(self, h_out, y=None, gate=None, w_post=None, w_next=None, dh_out=None, dx=None,
                 stream=None) -> BlockNormGrads:
        """The gradients of one forward call: `h_out` is the stream it returned, dh_out the
        gradient of that, dx (fp32 [T, d]) of x; dh_out = None is 0.  Fields that belong to
        an argument that is None are None."""
        if not self.train:
            raise ValueError("built without train=True")
        if y is None and (gate is not None or w_post is not None):
            raise ValueError("gate and w_post belong to y")
        if (w_next is None) != (dx is None):
            raise ValueError("dx and w_next are given together")
        if dh_out is None and dx is None:
            raise ValueError("give dh_out, dx or both")
        only = lambda buf, arg: None if arg is None else buf
        g = BlockNormGrads(self.dh, only(self.dy, y), only(self.dgate, gate),
                           only(self.dw_post, w_post), only(self.dw_next, w_next))
        given = (h_out, y, gate, w_post, w_next, dh_out, dx, *g, self.workspace)
        arrays = self._grad_args.read(*given)
        if self.cfg.T == 0:  # empty tensors have no address; the weights' gradients become 0
            arrays = [None if t is None else a or arrays[-1] for t, a in zip(given, arrays)]
        self._call("moet_block_norm_backward", (*self._refs, *arrays), stream)
        return g


class AdamW(_OnDevice):
    """AdamW over `params` (fp32 or bf16 tensors on one device), updated in place
    (moet_adamw_step).

    `weight_decay`: one number, or one a tensor.  `state_bits`: 32 (fp32 moments) or 8 (e4m3
    codes with an fp32 scale per 256 elements; `v` then holds the second moment's root).
    `master`: True keeps fp32 masters of bf16 weights, made from the weights here; or a list
    of them.  `m`, `v`, `m_scale`, `v_scale`: lists to take as states (a checkpoint's, or
    views of a flat buffer); zeros by default.  `step`: steps that they have seen.  Each step
    takes the weights and states as it finds them: their storage may be exchanged between steps
    (`.data`), not their size or type.

    Steps taken and learning rate live on the device (`steps`, `lr`), so a captured step
    replays with their current values: set_lr() between replays."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, state_bits: int = 32, master=None, m=None, v=None,
                 m_scale=None, v_scale=None, step: int = 0):
        self.params = tuple(params)
        if not self.params:
            raise ValueError("no parameters")
        if not all(isinstance(p, torch.Tensor) for p in self.params):
            raise TypeError("params must be CUDA tensors")
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        if not all(0 <= b < 1 for b in betas) or not eps > 0 or step < 0:
            raise ValueError("betas in [0, 1), eps > 0 and step >= 0 are needed")
        first = self.params[0]
        if not first.is_cuda:
            raise TypeError("params must be CUDA tensors")
        dev = first.device
        self._on(dev)
        count = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else \
            [float(weight_decay)] * count
        state = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        sizes = [p.numel() for p in self.params]
        blocks = [-(-n // N.MOET_ADAMW_BLOCK) for n in sizes]
        if master is True:
            master = [p.detach().float() if p.dtype is torch.bfloat16 else None
                      for p in self.params]
        zeros = lambda ns, dt: tuple(torch.zeros(n, dtype=dt, device=dev) for n in ns)
        self.m = zeros(sizes, state) if m is None else tuple(m)
        self.v = zeros(sizes, state) if v is None else tuple(v)
        self.m_scale = self.v_scale = None
        if state_bits == 8:
            self.m_scale = zeros(blocks, torch.float32) if m_scale is None else tuple(m_scale)
            self.v_scale = zeros(blocks, torch.float32) if v_scale is None else tuple(v_scale)
        elif m_scale is not None or v_scale is not None:
            raise ValueError("scales belong to 8-bit states")
        self.master = None if master is None else tuple(master)
        for name, ts in (("weight_decay", decay), ("m", self.m), ("v", self.v),
                         ("m_scale", self.m_scale), ("v_scale", self.v_scale),
                         ("master", self.master)):
            if ts is not None and len(ts) != count:
                raise ValueError(f"{name}: {len(ts)} of them for {count} parameters")
        specs, tensors, self._spans = [], [], []
        self._tensors = (N.MoetAdamwTensor * count)()
        for i, p in enumerate(self.params):
            if p.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError("params must be torch.float32 or torch.bfloat16")
            own = [("m", self.m[i], state, sizes[i]), ("v", self.v[i], state, sizes[i])]
            if state_bits == 8:
                own += [("m_scale", self.m_scale[i], torch.float32, blocks[i]),
                        ("v_scale", self.v_scale[i], torch.float32, blocks[i])]
            w = None if self.master is None else self.master[i]
            if w is not None:
                if p.dtype is not torch.bfloat16:
                    raise ValueError("fp32 weights have no master")
                own.append(("master", w, torch.float32, sizes[i]))
            own.append(("params", p, p.dtype, sizes[i]))
            specs += [(f"{name}[{i}]", dt, n, 0) for name, _, dt, n in own]
            tensors += [t for _, t, _, _ in own]
            e = self._tensors[i]
            e.n, e.weight_decay = sizes[i], decay[i]
            e.p_dtype, e.state_dtype = _TYPES[p.dtype], _TYPES[state]
        for (name, dt, n, _), at in zip(specs, N.Arguments(dev.index, *specs).read(*tensors)):
            field, i = name[:-1].split("[")
            field = "p" if field == "params" else field
            setattr(self._tensors[int(i)], field, at)
            if n:
                self._spans.append((int(i), field, n * dt.itemsize, name))
        self._apart()
        self._sizes = (ctypes.c_int64 * count)(*sizes)
        self._step_args = N.Arguments(dev.index, ("lr", torch.float32, 1, N.ARG_FLAT),
                                      ("grad_scale", torch.float32, 1, N.ARG_OPTIONAL),
                                      ("steps", torch.int32, 2, N.ARG_FLAT))
        self._opt = N.MoetAdamw(float(betas[0]), float(betas[1]), float(eps))
        self.lr = torch.full((4,), float(lr), device=dev)
        self.steps = torch.tensor([step, 0, 0, 0], dtype=torch.int32, device=dev)
        self._settle()

    def _apart(self):
        """Refuses weights and states that share memory."""
        self._known_apart = False
        spans = sorted((at, at + size, name) for at, size, name in (
            (getattr(self._tensors[i], field), size, name)
            for i, field, size, name in self._spans))
        for (_, end, a), (begin, _, b) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError(f"{a} and {b} share memory")
        self._known_apart = True

    def set_lr(self, lr: float) -> None:
        """Sets the learning rate of the steps that follow on the current stream."""
        self.lr.fill_(float(lr))

    def step(self, grads, grad_scale=None, stream=None) -> None:
        """One step with `grads` (fp32 or bf16, one a parameter, of its size).  `grad_scale`:
        fp32 device tensor that multiplies them (a clip or a loss scale's inverse); when it
        is not finite, the step is left out.  Autograd counts the step as a change of the
        weights."""
        grads = grads if isinstance(grads, (list, tuple)) else list(grads)
        a = self._step_args.read(self.lr, grad_scale, self.steps)
        moved = N.read_step(grads, self.params, self._sizes, self._index, self._tensors,
                            (self.m, self.v, self.m_scale, self.v_scale, self.master))
        if moved or not self._known_apart:
            self._apart()
        self._call("moet_adamw_step",
                   (self._tensors, len(self._sizes), ctypes.byref(self._opt), a[0], a[1], a[2]),
                   stream)
