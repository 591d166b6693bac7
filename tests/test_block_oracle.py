"""Pins of oracle/block.py (fp64 definitions of the gated recurrence, layer
norm and the conv's gradients) against code that shares nothing with it:
closed forms, library routines, and central differences for every gradient."""
import math

import pytest
import torch

import oracle
from oracle import block as O

F64 = torch.float64


def _gated(B=2, L=7, D=3, seed=0, ragged=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)                 # noqa: E731
    t = dict(x=r(B, L, D), gate_a=r(B, L, D), gate_x=r(B, L, D),
             A=-torch.rand(D, generator=g, dtype=F64) - 0.05, bias_a=r(D), bias_x=r(D), h0=r(B, D))
    if ragged:
        t["seq_lens"] = torch.tensor([0, L - 2, L + 5][:B], dtype=torch.int32)
    return t


def test_one_token_closed_form():
    t = _gated(B=1, L=1, D=1)
    y, h = O.gated_scan(**t)
    r = 1 / (1 + math.exp(-(t["gate_a"] + t["bias_a"]).item()))
    i = 1 / (1 + math.exp(-(t["gate_x"] + t["bias_x"]).item()))
    a = math.exp(t["A"].item() * r)
    want = a * t["h0"].item() + math.sqrt(1 - a * a) * i * t["x"].item()
    assert abs(y.item() - want) < 1e-15 and abs(h.item() - want) < 1e-15


def test_constant_gates_are_a_geometric_sum():
    L, A = 50, -0.3
    ones = torch.ones(1, L, 1, dtype=F64)
    y, _ = O.gated_scan(ones, 0 * ones, 0 * ones, torch.tensor([A], dtype=F64))
    a = math.exp(A / 2)
    w = math.sqrt(1 - a * a) / 2
    want = torch.tensor([w * (1 - a ** (t + 1)) / (1 - a) for t in range(L)], dtype=F64)
    assert torch.allclose(y[0, :, 0], want, rtol=1e-12, atol=0)


def test_chained_calls_and_ragged_rows():
    t = _gated(B=3, L=9, ragged=True)
    y, h = O.gated_scan(**t)
    for b, n in enumerate([0, 7, 9]):
        one = {k: (v[b:b + 1, :n] if v.dim() == 3 else v[b:b + 1] if k == "h0" else v)
               for k, v in t.items() if k != "seq_lens"}
        y1, h1 = O.gated_scan(**one)
        assert torch.equal(y[b:b + 1, :n], y1) and torch.equal(h[b:b + 1], h1)
        assert not y[b, n:].any()
    s = O.gated_scan_states(**{k: v for k, v in t.items() if k != "seq_lens"}, tile=4)
    y, _ = O.gated_scan(**{k: v for k, v in t.items() if k != "seq_lens"})
    assert torch.equal(s[:, 0], t["h0"]) and torch.equal(s[:, 2], y[:, 7])


def _differences(f, given, grads, step=1e-6, tol=1e-6):
    for name, t in given.items():
        flat = t.view(-1)
        for k in range(0, flat.numel(), max(1, flat.numel() // 7)):
            keep = flat[k].item()
            flat[k] = keep + step
            up = f()
            flat[k] = keep - step
            down = f()
            flat[k] = keep
            want = (up - down) / (2 * step)
            got = grads["d" + name].reshape(-1)[k].item()
            assert abs(got - want) <= tol * max(1.0, abs(want)), (name, k, got, want)


@pytest.mark.parametrize("ragged", [False, True])
def test_gated_gradients_by_differences(ragged):
    t = _gated(B=3, L=6, ragged=ragged)
    dy, dh = torch.randn(3, 6, 3, dtype=F64), torch.randn(3, 3, dtype=F64)
    grads = O.gated_scan_bwd(t["x"], t["gate_a"], t["gate_x"], t["A"], dy, t["bias_a"], t["bias_x"],
                             t["h0"], dh, t.get("seq_lens"))

    def f():
        y, h = O.gated_scan(**t)
        return float((y * dy).sum() + (h * dh).sum())

    _differences(f, {k: v for k, v in t.items() if k != "seq_lens"}, grads)


def test_layer_norm_is_the_library_routine_and_gradients_by_differences():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)                 # noqa: E731
    x, w, b, res, dy, ds = r(4, 9), r(9), r(9), r(4, 9), r(4, 9), r(4, 9)
    y, mean, rstd, s = O.layer_norm(x, w, b, res, eps=1e-3)
    want = torch.nn.functional.layer_norm(x + res, (9,), w, b, eps=1e-3)
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-13) and torch.equal(s, x + res)
    assert torch.allclose(mean, (x + res).mean(1), rtol=1e-12)
    assert torch.allclose(rstd, ((x + res).var(1, unbiased=False) + 1e-3).rsqrt(), rtol=1e-12)
    grads = O.layer_norm_bwd(x, dy, w, b, res, ds, eps=1e-3)

    def f():
        y, _, _, s = O.layer_norm(x, w, b, res, eps=1e-3)
        return float((y * dy).sum() + (s * ds).sum())

    _differences(f, {"x": x, "weight": w, "bias": b}, grads)


@pytest.mark.parametrize("K,L", [(1, 5), (2, 1), (3, 8), (4, 2), (4, 11)])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradients_by_differences(K, L, silu):
    g = torch.Generator().manual_seed(K)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)                 # noqa: E731
    t = dict(x=r(2, L, 3), weight=r(3, K), bias=r(3), state=r(2, 3, K - 1))
    du, ds = r(2, L, 3), r(2, 3, K - 1)
    grads = O.causal_conv1d_silu_bwd(t["x"], t["weight"], du, t["bias"], t["state"], silu, ds)

    def f():                                   # the forward oracle: separate code (numpy)
        u, s = oracle.causal_conv1d_silu(t["x"], t["weight"], t["bias"], state=t["state"], silu=silu)
        s = torch.as_tensor(s) if K > 1 else torch.zeros(2, 3, 0, dtype=F64)
        return float((torch.as_tensor(u) * du).sum() + (s * ds).sum())

    _differences(f, {k: v for k, v in t.items() if v.numel()}, grads)
