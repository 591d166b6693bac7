"""fp64 CPU definitions of linear attention with a decay for each head (token by
token), the norm of queries and keys with rotary positions, and the moves of
states between a pool's slots.  Gradients come from reverse-mode
differentiation of these definitions, so they share no formula with the
kernels' backward passes.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def _f64(t, grad=False):
    if t is None:
        return None
    return t.detach().cpu().to(F64).clone().requires_grad_(grad)


def _linear(q, k, v, g, scale, h0, lens):
    """(o [B, L, H, Dv] with zeros behind a row's end, the state after each row's last token)."""
    B, L, G, Dk = q.shape
    H, Dv = v.shape[2:]
    q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
    g = g.expand(B, L, H)
    h = h0 if h0 is not None else torch.zeros(B, H, Dk, Dv, dtype=F64)
    out = []
    for t in range(L):
        new = torch.exp(g[:, t])[..., None, None] * h + k[:, t, :, :, None] * v[:, t, :, None, :]
        o = scale * (q[:, t, :, :, None] * new).sum(2)
        if lens is None:
            h = new
        else:
            there = (t < lens)[:, None, None]
            h = torch.where(there[..., None], new, h)
            o = torch.where(there, o, torch.zeros_like(o))
        out.append(o)
    return (torch.stack(out, 1) if L else torch.zeros(B, 0, H, Dv, dtype=F64)), h


def _lens(seq_lens, L):
    return None if seq_lens is None else seq_lens.cpu().to(torch.int64).clamp(0, L)


def _zero_padding(t, lens):
    """The padding may hold anything: what is behind a row's end counts as zero."""
    if lens is None or t is None or t.dim() < 2:
        return t
    there = torch.arange(t.shape[1]) < lens[:, None]
    return torch.where(there.view(*there.shape, *[1] * (t.dim() - 2)), t, torch.zeros_like(t))


def linear_attention(q, k, v, log_decay, scale, h0=None, seq_lens=None):
    lens = _lens(seq_lens, q.shape[1])
    q, k, v, g = (_zero_padding(_f64(t), lens) for t in (q, k, v, log_decay))
    return _linear(q, k, v, g, scale, _f64(h0), lens)


def linear_attention_bwd(q, k, v, log_decay, do, scale, h0=None, dh_last=None, seq_lens=None):
    """Gradients of sum(do * o) + sum(dh_last * h_last) for every input given."""
    lens = _lens(seq_lens, q.shape[1])
    t = {n: _zero_padding(_f64(x), lens).requires_grad_(True)
         for n, x in (("dq", q), ("dk", k), ("dv", v), ("dlog_decay", log_decay))}
    if h0 is not None:
        t["dh0"] = _f64(h0, True)
    o, h = _linear(t["dq"], t["dk"], t["dv"], t["dlog_decay"], scale, t.get("dh0"), lens)
    loss = (o * _zero_padding(_f64(do), lens)).sum()
    if dh_last is not None:
        loss = loss + (h * _f64(dh_last)).sum()
    got = torch.autograd.grad(loss, list(t.values()), allow_unused=True)
    return {n: (torch.zeros_like(x) if d is None else d) for (n, x), d in zip(t.items(), got)}


def linear_step(state, q, k, v, log_decay, scale, slots=None):
    """(o, the pool afterwards): rows in order, each against state[slots[b]]."""
    S = _f64(state)
    q, k, v, g = (_f64(t) for t in (q, k, v, log_decay))
    B, G, Dk = q.shape
    H, Dv = v.shape[1:]
    g = g.expand(B, H)
    o = torch.zeros(B, H, Dv, dtype=F64)
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < S.shape[0]:
            continue
        for h in range(H):
            grp = h // (H // G)
            S[s, h] = torch.exp(g[b, h]) * S[s, h] + torch.outer(k[b, grp], v[b, h])
            o[b, h] = scale * (q[b, grp] @ S[s, h])
    return o, S


def _turned(y, angle, interleaved):
    """The first 2 * angle.shape[-1] elements of [..., heads, width], in pairs, as complex numbers times e^{i angle}."""
    half = angle.shape[-1]
    first = torch.arange(half) * 2 if interleaved else torch.arange(half)
    second = first + (1 if interleaved else half)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)[..., None, :]
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _qk(q, k, wq, wk, positions, inv_freq, interleaved, eps):
    out = []
    for x, w in ((q, wq), (k, wk)):
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w
        if inv_freq is not None:
            y = _turned(y, positions.cpu().to(F64)[..., None] * inv_freq, interleaved)
        out.append(y)
    return out


def qk_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, interleaved=False, eps=1e-6):
    return _qk(*(_f64(t) for t in (q, k, q_weight, k_weight)), positions, _f64(inv_freq), interleaved, eps)


def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                     interleaved=False, eps=1e-6):
    t = {n: _f64(x, True) for n, x in (("dq", q), ("dk", k), ("dq_weight", q_weight), ("dk_weight", k_weight))
         if x is not None}
    y, z = _qk(t["dq"], t["dk"], t.get("dq_weight"), t.get("dk_weight"), positions, _f64(inv_freq), interleaved, eps)
    loss = (y * _f64(dq_out)).sum() + (z * _f64(dk_out)).sum()
    got = torch.autograd.grad(loss, list(t.values()), allow_unused=True)
    return {n: (torch.zeros_like(x) if d is None else d) for (n, x), d in zip(t.items(), got)}


def slots_copy(pool, src, dst, dim=0):
    """One assignment: every source is read before any destination is written."""
    before = pool.detach().cpu().movedim(dim, 0)
    after = before.clone()
    for s, d in zip(src.tolist(), dst.tolist()):
        if 0 <= d < before.shape[0] and s < before.shape[0]:
            after[d] = before[s] if s >= 0 else torch.zeros_like(before[0])
    return after.movedim(0, dim)
