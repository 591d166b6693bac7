"""fp64 CPU definitions of the calls around the scan in a recurrent block: the
gated linear recurrence token by token, layer norm, and the causal conv's
gradients.  Gradients come from reverse-mode differentiation of these
definitions, so they share no formula with the kernels' backward passes.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def _f64(t, grad=False):
    if t is None:
        return None
    return t.detach().cpu().to(F64).clone().requires_grad_(grad)


def _sigma(z):
    # through its logarithm: the derivative of torch.sigmoid is formed as
    # s (1 - s), which loses what is left of 1 - s for large z even in fp64
    return torch.exp(torch.nn.functional.logsigmoid(z))


def _gated(x, ga, gx, A, ba, bx, h0, lens):
    """(y [B, L, D] with zeros behind a row's end, state after each row's last token)."""
    B, L, D = x.shape
    h = h0 if h0 is not None else torch.zeros(B, D, dtype=F64)
    ys = []
    for t in range(L):
        r = _sigma(ga[:, t] + (ba if ba is not None else 0.0))
        i = _sigma(gx[:, t] + (bx if bx is not None else 0.0))
        new = torch.exp(A * r) * h + torch.sqrt(-torch.expm1(2 * A * r)) * i * x[:, t]
        there = (torch.arange(B) < B) if lens is None else t < lens
        h = torch.where(there[:, None], new, h)
        ys.append(torch.where(there[:, None], new, torch.zeros_like(new)))
    y = torch.stack(ys, 1) if L else torch.zeros(B, 0, D, dtype=F64)
    return y, h


def _lens(seq_lens, L):
    return None if seq_lens is None else seq_lens.cpu().to(torch.int64).clamp(0, L)


def gated_scan(x, gate_a, gate_x, A, bias_a=None, bias_x=None, h0=None, seq_lens=None):
    return _gated(*(_f64(t) for t in (x, gate_a, gate_x, A, bias_a, bias_x, h0)),
                  _lens(seq_lens, x.shape[1]))


def gated_scan_states(x, gate_a, gate_x, A, bias_a=None, bias_x=None, h0=None, tile=128):
    """The state before token 0, tile, 2 tile, ...: [B, ceil(L / tile), D]."""
    y, _ = gated_scan(x, gate_a, gate_x, A, bias_a, bias_x, h0)
    B, L, D = x.shape
    first = _f64(h0) if h0 is not None else torch.zeros(B, D, dtype=F64)
    return torch.stack([first] + [y[:, t - 1] for t in range(tile, L, tile)], 1)


def gated_scan_bwd(x, gate_a, gate_x, A, dy, bias_a=None, bias_x=None, h0=None, dh_last=None,
                   seq_lens=None):
    """Gradients of sum(dy * y) + sum(dh_last * h_last) for every input given."""
    names = ["x", "gate_a", "gate_x", "A", "bias_a", "bias_x", "h0"]
    v = [_f64(t, True) for t in (x, gate_a, gate_x, A, bias_a, bias_x, h0)]
    y, h = _gated(*v, _lens(seq_lens, x.shape[1]))
    lens = _lens(seq_lens, x.shape[1])
    g = _f64(dy)
    if lens is not None:                       # the padding may hold anything
        there = torch.arange(x.shape[1])[None, :, None] < lens[:, None, None]
        g = torch.where(there, g, torch.zeros_like(g))
    loss = (g * y).sum()
    if dh_last is not None:
        loss = loss + (_f64(dh_last) * h).sum()
    given = [(n, t) for n, t in zip(names, v) if t is not None]
    grads = torch.autograd.grad(loss, [t for _, t in given], allow_unused=True)
    return {"d" + n: torch.zeros_like(t) if gr is None else gr
            for (n, t), gr in zip(given, grads)}


def _norm(x, weight, bias, residual, eps):
    s = x if residual is None else x + residual
    mean = s.mean(-1)
    var = (s - mean[..., None]).pow(2).mean(-1)
    n = (s - mean[..., None]) / torch.sqrt(var + eps)[..., None]
    y = n if weight is None else n * weight
    return (y if bias is None else y + bias), mean, 1 / torch.sqrt(var + eps), s


def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5):
    return _norm(*(_f64(t) for t in (x, weight, bias, residual)), eps)


def layer_norm_bwd(x, dy, weight=None, bias=None, residual=None, dresidual_out=None, eps=1e-5):
    """Gradients of sum(dy * y) + sum(dresidual_out * (x + residual))."""
    v = [_f64(t, True) for t in (x, weight, bias)]
    y, _, _, s = _norm(*v, _f64(residual), eps)
    loss = (_f64(dy) * y).sum()
    if dresidual_out is not None:
        loss = loss + (_f64(dresidual_out) * s).sum()
    given = [(n, t) for n, t in zip(("x", "weight", "bias"), v) if t is not None]
    grads = torch.autograd.grad(loss, [t for _, t in given], allow_unused=True)
    return {"d" + n: torch.zeros_like(t) if g is None else g for (n, t), g in zip(given, grads)}


def causal_conv1d_silu_bwd(x, weight, du, bias=None, state=None, silu=True, dstate_out=None):
    """Gradients of sum(du * u) + sum(dstate_out * state_out) for every input given."""
    B, L, D = x.shape
    K = weight.shape[1]
    v = [_f64(t, True) for t in (x, weight, bias, state)]
    xs, w, b, st = v
    first = st if st is not None else torch.zeros(B, D, K - 1, dtype=F64)
    full = torch.cat([first, xs.transpose(1, 2)], 2)
    s = sum(w[:, k, None] * full[:, :, k:k + L] for k in range(K))
    if b is not None:
        s = s + b[:, None]
    u = (s * _sigma(s) if silu else s).transpose(1, 2)
    loss = (_f64(du) * u).sum()
    if dstate_out is not None:
        loss = loss + (_f64(dstate_out) * full[:, :, L:]).sum()
    given = [(n, t) for n, t in zip(("x", "weight", "bias", "state"), v) if t is not None]
    grads = torch.autograd.grad(loss, [t for _, t in given], allow_unused=True)
    return {"d" + n: torch.zeros_like(t) if g is None else g for (n, t), g in zip(given, grads)}
