"""Plain 64-bit forms of the training operators, written for autograd: a gradient is the
autograd of these forward forms (and those are checked against differences on the CPU)."""
from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn


def spans(T, seq_off):
    off = [0, T] if seq_off is None else [int(v) for v in seq_off]
    return list(zip(off[:-1], off[1:]))


def router_losses(logits, topk_ids, token_mask=None, seq_off=None):
    """(balance loss, z loss, counts, probs, lse) by a loop over sequences, in 64 bits."""
    x = logits.double()
    T, E = x.shape
    k = topk_ids.shape[1]
    lse = torch.zeros(T, dtype=torch.float64)
    counts, probs, bal, n_all, z = [], [], [], 0, 0.0
    for a, b in spans(T, seq_off):
        rows = [t for t in range(a, b) if token_mask is None or int(token_mask[t])]
        n_all += len(rows)
        c = torch.zeros(E, dtype=torch.float64)
        P = torch.zeros(E, dtype=torch.float64)
        if rows:
            r = torch.tensor(rows)
            for e in topk_ids[r].reshape(-1).tolist():
                c[e] += 1
            l = torch.logsumexp(x[r], 1)
            P = torch.exp(x[r] - l[:, None]).sum(0) / len(rows)
            lse = lse.index_put((r,), l)
            z = z + (l ** 2).sum()
            bal.append(E / (k * len(rows)) * (c * P).sum())
        counts.append(c)
        probs.append(P)
    balance = torch.stack(bal).mean() if bal else torch.zeros((), dtype=torch.float64)
    zloss = z / n_all if n_all else torch.zeros((), dtype=torch.float64)
    return balance, zloss, torch.stack(counts), torch.stack(probs), lse


def rms_norm(v, w, eps, offset):
    return v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + eps) * (w + offset)


def block_norm(h, y, gate, w_post, w_next, eps=1e-6, w_offset=0.0, res_scale=1.0,
               out_scale=1.0):
    """(h_out, x) in 64 bits; absent arguments are None."""
    if y is not None:
        o = y if w_post is None else rms_norm(y, w_post, eps, w_offset)
        if gate is not None:
            o = o * gate[:, None]
        h = res_scale * h + out_scale * o
    return h, None if w_next is None else rms_norm(h, w_next, eps, w_offset)


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p - lr * wd * p - lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    return p, m, v


def to_8bit(x, root):
    """fp32 moments -> (e4m3 codes, scales), each operation rounded by itself (the stored
    form is defined by these fp32 roundings)."""
    n = x.numel()
    pad = torch.zeros(-(-n // 256) * 256, dtype=torch.float32)
    pad[:n] = x
    b = pad.view(-1, 256)
    top = b.abs().amax(1)
    some = ~(top < 1e-30)
    inv = torch.where(some, torch.tensor(448.0) * (torch.ones(()) / top), torch.zeros(()))
    scale = torch.where(some, top * torch.tensor(1 / 448.0), torch.zeros(()))
    c = b * inv[:, None]
    if root:
        c = torch.where(b > 0, c.clamp(min=2.0 ** -9), c)
    return c.clamp(-448, 448).to(E4M3).view(-1)[:n], scale


def of_8bit(c, scale):
    n = c.numel()
    return c.float() * scale.repeat_interleave(256)[:n]
