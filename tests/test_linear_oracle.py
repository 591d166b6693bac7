"""Pins of oracle/linear.py (fp64 definitions of linear attention, the head norm
with rotary positions and the moves between slots) against code that shares
nothing with it: closed forms, the masked product, and central differences for
every gradient."""
import math

import pytest
import torch

from oracle import linear as O

F64 = torch.float64


def make(B=2, L=9, H=4, G=2, Dk=3, Dv=5, seed=0, ragged=False, by_head=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)                 # noqa: E731
    t = dict(q=r(B, L, G, Dk), k=r(B, L, G, Dk), v=r(B, L, H, Dv),
             log_decay=-torch.rand(*((H,) if by_head else (B, L, H)), generator=g, dtype=F64), scale=0.7,
             h0=r(B, H, Dk, Dv))
    if ragged:
        t["seq_lens"] = torch.tensor([L - 2, 0, L + 5][:B], dtype=torch.int32)
    return t, r(B, L, H, Dv), r(B, H, Dk, Dv)


def test_masked_product():
    """o = (q k^T o M) v + e^G q h0 with M_ij = e^{G_i - G_j} for j <= i: the whole sequence at once."""
    t, _, _ = make()
    q, k = (t[x].repeat_interleave(2, 2).transpose(1, 2) for x in ("q", "k"))
    v, G = t["v"].transpose(1, 2), t["log_decay"].transpose(1, 2).cumsum(2)
    M = torch.exp(G[..., :, None] - G[..., None, :]).tril()
    o = t["scale"] * (((q @ k.transpose(2, 3)) * M) @ v + torch.exp(G)[..., None] * (q @ t["h0"]))
    got, h = O.linear_attention(**t)
    assert torch.allclose(got, o.transpose(1, 2), rtol=1e-12, atol=1e-12)
    w = torch.exp(G[..., -1:] - G)[..., None]
    want = torch.exp(G[..., -1])[..., None, None] * t["h0"] + (k * w).transpose(2, 3) @ v
    assert torch.allclose(h, want, rtol=1e-12, atol=1e-12)


def test_constant_decay_is_a_geometric_sum():
    L, a = 40, 0.9
    one = torch.ones(1, L, 1, 1, dtype=F64)
    o, h = O.linear_attention(one, one, one, torch.tensor([math.log(a)], dtype=F64), 2.0)
    want = torch.tensor([(1 - a ** (t + 1)) / (1 - a) for t in range(L)], dtype=F64)
    assert torch.allclose(o.flatten(), 2 * want, rtol=1e-12) and abs(h.item() - want[-1].item()) < 1e-12


def test_chained_calls_and_steps_are_one_call():
    t, _, _ = make(ragged=False)
    o, h = O.linear_attention(**t)
    a, b = ({**t, **{n: t[n][:, s] for n in ("q", "k", "v", "log_decay")}} for s in (slice(0, 4), slice(4, None)))
    o1, h1 = O.linear_attention(**a)
    o2, h2 = O.linear_attention(**{**b, "h0": h1})
    assert torch.allclose(torch.cat([o1, o2], 1), o) and torch.allclose(h2, h)
    state = t["h0"]
    for i in range(9):
        oi, state = O.linear_step(state, t["q"][:, i], t["k"][:, i], t["v"][:, i], t["log_decay"][:, i], t["scale"])
        assert torch.allclose(oi, o[:, i])
    assert torch.allclose(state, h)


def test_ragged_rows_are_short_calls():
    t, _, _ = make(B=3, ragged=True)
    o, h = O.linear_attention(**t)
    for b, n in enumerate([7, 0, 9]):
        ob, hb = O.linear_attention(t["q"][b:b + 1, :n], t["k"][b:b + 1, :n], t["v"][b:b + 1, :n],
                                    t["log_decay"][b:b + 1, :n], t["scale"], t["h0"][b:b + 1])
        assert torch.equal(o[b, :n], ob[0]) and torch.equal(h[b], hb[0]) and not o[b, n:].any()


def _differences(loss, x, eps=1e-6):
    d = torch.zeros_like(x)
    for i in range(x.numel()):
        for s in (1, -1):
            y = x.clone().flatten()
            y[i] += s * eps
            d.view(-1)[i] += s * loss(y.view_as(x)) / (2 * eps)
    return d


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("by_head", [False, True])
def test_gradients_against_differences(ragged, by_head):
    t, do, dh = make(L=5, Dk=2, Dv=2, H=2, G=1, ragged=ragged, by_head=by_head)
    got = O.linear_attention_bwd(t["q"], t["k"], t["v"], t["log_decay"], do, t["scale"], t["h0"], dh, t.get("seq_lens"))
    for n in ("q", "k", "v", "log_decay", "h0"):
        def loss(x):
            o, h = O.linear_attention(**{**t, n: x})
            return ((o * do).sum() + (h * dh).sum()).item()
        assert torch.allclose(got["d" + n], _differences(loss, t[n]), rtol=1e-6, atol=1e-6), n


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_its_matrix(interleaved):
    g = torch.Generator().manual_seed(1)
    q, w = torch.randn(3, 2, 6, generator=g, dtype=F64), torch.rand(6, generator=g, dtype=F64)
    pos, freq = torch.tensor([0, 5, 700000], dtype=torch.int32), torch.tensor([1.0, 0.25], dtype=F64)
    y, _ = O.qk_norm_rope(q, q, w, w, pos, freq, interleaved)
    for r in range(3):
        for h in range(2):
            x = q[r, h] / math.sqrt(float(q[r, h] @ q[r, h]) / 6 + 1e-6) * w
            for p in range(2):
                a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + 2)
                c, s = math.cos(float(pos[r]) * float(freq[p])), math.sin(float(pos[r]) * float(freq[p]))
                assert abs(y[r, h, a] - (x[a] * c - x[b] * s)) < 1e-12
                assert abs(y[r, h, b] - (x[b] * c + x[a] * s)) < 1e-12
            assert torch.allclose(y[r, h, 4:], x[4:])


def test_rotation_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)                 # noqa: E731
    t = dict(q=r(2, 2, 4), k=r(2, 1, 4), q_weight=r(4), k_weight=r(4))
    more = dict(positions=torch.tensor([3, 11], dtype=torch.int32), inv_freq=torch.tensor([0.5], dtype=F64))
    dq, dk = r(2, 2, 4), r(2, 1, 4)
    got = O.qk_norm_rope_bwd(t["q"], t["k"], dq, dk, t["q_weight"], t["k_weight"], **more)
    for n in t:
        def loss(x):
            y, z = O.qk_norm_rope(**{**t, n: x}, **more)
            return ((y * dq).sum() + (z * dk).sum()).item()
        assert torch.allclose(got["d" + n], _differences(loss, t[n]), rtol=1e-6, atol=1e-7), n


def test_slots_are_one_assignment():
    pool = torch.arange(12.0).view(2, 6)
    out = O.slots_copy(pool, torch.tensor([1, 0, -1, 7, 5]), torch.tensor([0, 1, 3, 4, 3]), dim=1)
    assert out.tolist() == [[1, 0, 2, 5, 4, 5], [7, 6, 8, 11, 10, 11]]
