"""How far an element of a linear-attention call may be from its fp64 value,
worked out from the inputs.  Every value is a sum of products of the inputs and
decays, so running the definition over absolute values (all terms positive)
gives the size that its roundings are relative to.

fp32: an operation rounds by 2^-24, hardware exp2 by 2^-23; a value passes at
most as many as its sum has terms: tokens, the contracted width, and for each
chunk of 32 tokens the decay's exponential, its product and the addition.  All
are counted at 2^-23.  bf16 (half a step: 2^-8): the stored output, and the two
operands (scores, state) that are rounded where only bf16 comes of them: in o
and dv always (each term of their sums is a product of two factors off by half
a step at most), in dq and dk where no decay's gradient is formed of them.
"""
import torch

from oracle import linear as O

U = 2.0 ** -23
HALF = 2.0 ** -8


def _abs(t):
    return None if t is None else t.detach().cpu().double().abs()


def roundings(L, Dk, Dv):
    return L + Dk + Dv + 6 * (L // 32 + 1) + 64


def _wide(t, H):
    return t.repeat_interleave(H // t.shape[2], 2)


def _padded(t, lens):
    return t if lens is None else O._zero_padding(t, lens.cpu().long().clamp(0, t.shape[1]))


def forward(q, k, v, log_decay, scale, h0=None, seq_lens=None):
    """Allowances for (o, h_last)."""
    q_, k_, v_ = (_padded(_abs(t), seq_lens) for t in (q, k, v))
    o, h = O.linear_attention(q_, k_, v_, log_decay, abs(scale), _abs(h0), seq_lens)
    exact, _ = O.linear_attention(q, k, v, log_decay, scale, h0, seq_lens)
    n = roundings(q.shape[1], q.shape[3], v.shape[3]) * U
    extra = (2 * HALF + HALF * n) * o + HALF * exact.abs() if q.dtype == torch.bfloat16 else 0.0
    return n * o + extra + 1e-37, n * h + 1e-37


def backward(q, k, v, log_decay, do, scale, h0=None, dh_last=None, seq_lens=None, split=True):
    """Allowances for every gradient; split: the decay's is formed too."""
    H, G = v.shape[2], q.shape[2]
    a = [_padded(t, seq_lens) for t in (_wide(_abs(q), H), _wide(_abs(k), H), _abs(v))]
    m = O.linear_attention_bwd(*a, log_decay, _padded(_abs(do), seq_lens), abs(scale), _abs(h0), _abs(dh_last),
                               seq_lens)
    x = O.linear_attention_bwd(q, k, v, log_decay, do, scale, h0, dh_last, seq_lens)
    n = roundings(q.shape[1], q.shape[3], v.shape[3]) * U
    bf = q.dtype == torch.bfloat16
    out = {}
    for name in ("dq", "dk", "dv"):
        size = m[name] if name == "dv" else m[name].unflatten(2, (G, H // G)).sum(3)
        out[name] = n * size + 1e-37
        if bf:
            out[name] += HALF * x[name].abs() + HALF * n * size + (0.0 if split and name != "dv" else 2 * HALF * size)
    if h0 is not None:
        out["dh0"] = n * m["dh0"] + 1e-37
    # sums of q . dq and k . dk over the tokens from t on, from <dh_last, h_last>
    per = (a[0] * m["dq"] + a[1] * m["dk"]).sum(3)
    if dh_last is not None:
        _, h = O.linear_attention(*a, log_decay, abs(scale), _abs(h0), seq_lens)
        per[:, -1:] += (h * _abs(dh_last)).sum((2, 3))[:, None]
    tail = per.flip(1).cumsum(1).flip(1)
    out["dlog_decay"] = 2 * n * (tail if log_decay.dim() == 3 else tail.sum((0, 1))) + 1e-37
    return out


def check(name, got, want, allowed):
    got = got.detach().cpu().double()
    want = want.double()
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), name
    over = (got - want).abs() - allowed
    assert (over <= 0).all(), (name, float(over.max()), float(((got - want).abs() / allowed).max()))


def near(name, got, want, bar):
    """Normwise: the 2-norm of the difference over the result's."""
    got, want = got.detach().cpu().double(), want.double()
    n = float(want.norm())
    assert float((got - want).norm()) <= bar * (n if n else 1.0), (name, float((got - want).norm()), n)
