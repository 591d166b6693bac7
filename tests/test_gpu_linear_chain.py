"""The calls run together as a layer of linear attention uses them -- queries,
keys and values out of one projection, normed and rotated, attention, and back
through both -- against reverse-mode differentiation of the whole in fp64; and
as a server does: prompts read into a pool's slots, a prefix forked, single
tokens, a beam's reorder, against whole sequences."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import linear as O

import _linear_bounds as Bd

pytestmark = pytest.mark.gpu

F64 = torch.float64


def make(B, L, H, G, Dk, Dv, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)                            # noqa: E731
    return dict(wide=r(B, L, 2 * G * Dk + H * Dv).to(dtype), wq=1 + 0.1 * r(Dk), wk=1 + 0.1 * r(Dk),
                g=-torch.exp(r(B, L, H) - 2), pos=torch.arange(L, dtype=torch.int32).repeat(B, 1) + 100000,
                freq=10000.0 ** (-torch.arange(Dk // 4) * 4.0 / Dk), do=r(B, L, H, Dv).to(dtype))


def parts(wide, H, G, Dk, Dv):
    return (wide[..., :G * Dk].unflatten(-1, (G, Dk)), wide[..., G * Dk:2 * G * Dk].unflatten(-1, (G, Dk)),
            wide[..., 2 * G * Dk:].unflatten(-1, (H, Dv)))


def layer(t, size):
    """Forward and every gradient through the library."""
    q, k, v = parts(t["wide"], *size)
    q1, k1 = ssm.qk_norm_rope_fwd(q, k, t["wq"], t["wk"], t["pos"], t["freq"])
    o, h = ssm.linear_attention_fwd(q1, k1, v, t["g"])
    r = ssm.linear_attention_bwd(q1, k1, v, t["g"], t["do"])
    n = ssm.qk_norm_rope_bwd(q, k, r["dq"], r["dk"], t["wq"], t["wk"], t["pos"], t["freq"])
    wide = torch.cat([n["dq"].flatten(2), n["dk"].flatten(2), r["dv"].flatten(2)], 2)
    return dict(o=o, h=h, wide=wide, wq=n["dq_weight"], wk=n["dk_weight"], g=r["dlog_decay"])


def exact(t, size):
    leaves = {n: t[n].cpu().to(F64).requires_grad_(True) for n in ("wide", "wq", "wk", "g")}
    q, k, v = parts(leaves["wide"], *size)
    q, k = O._qk(q, k, leaves["wq"], leaves["wk"], t["pos"], t["freq"].cpu().to(F64), False, 1e-6)
    o, h = O._linear(q, k, v, leaves["g"], size[2] ** -0.5, None, None)
    grads = torch.autograd.grad((o * t["do"].cpu().to(F64)).sum(), list(leaves.values()))
    return dict(o=o.detach(), h=h.detach(), **dict(zip(leaves, grads)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B, L, size", [(2, 90, (4, 2, 64, 64)), (1, 200, (2, 2, 32, 96)), (3, 33, (3, 1, 128, 48))])
def test_layer_gradients(B, L, size, dtype):
    """fp32: 1e-5 of the norm.  bf16: at most four tensors on a path are rounded by half a step (2^-8 each):
    queries and keys, scores and state, the attention's gradients, the layer's."""
    t = make(B, L, *size, dtype)
    got = layer({n: x.cuda() for n, x in t.items()}, size)
    want = exact(t, size)
    for n in want:
        Bd.near(n, got[n], want[n], 1e-5 if dtype == torch.float32 else 4 * 2.0 ** -8)


def test_gradients_against_differences_along_them():
    """The loss, formed in fp64 of the library's outputs, moves along the gradient as it says."""
    size = (2, 1, 32, 32)
    t = {n: x.cuda() for n, x in make(1, 70, *size, torch.float32, seed=4).items()}
    grads = layer(t, size)
    for n in ("wide", "g"):
        d = grads[n].double()
        step = 1e-3 / float(d.norm())
        losses = []
        for s in (1, -1):
            moved = {**t, n: (t[n].double() + s * step * d).float()}
            losses.append(float((layer(moved, size)["o"].double() * t["do"].double()).sum()))
        # second differences cancel; outputs off by 1e-6 of the loss's terms over a step of 1e-3
        slope, want = (losses[0] - losses[1]) / (2 * step), float(d.norm()) ** 2
        terms = float((grads["o"].double() * t["do"].double()).abs().sum())
        assert abs(slope - want) <= 1e-3 * want + 1e-6 * terms / step, n


def test_layer_captured_and_replayed_while_another_runs():
    size = (4, 2, 64, 64)
    t = {n: x.cuda() for n, x in make(2, 200, *size, torch.bfloat16).items()}
    other = {n: x.cuda() for n, x in make(2, 200, *size, torch.bfloat16, seed=7).items()}
    want_other = layer(other, size)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(t, size)
    for n in range(4):
        t["wide"].copy_(torch.randn(t["wide"].shape, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            beside = layer(other, size)
        torch.cuda.synchronize()
        got = {k: x.clone() for k, x in out.items()}
        want = layer(t, size)
        assert all(torch.equal(got[k], want[k]) for k in want), n
        assert all(torch.equal(beside[k], want_other[k]) for k in beside), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_served_beams(dtype):
    """Two layers' states in one pool.  A prompt of 50 tokens is read into slot 2, forked to 0 and 4, every beam goes on
    with its own tokens, then beam 4 takes over beam 0's state, and 2 is cleared and takes a new sequence."""
    H, G, Dk, Dv, slots = 2, 1, 64, 32, 5
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g)                            # noqa: E731
    L = 62
    toks = [dict(q=r(3, L, G, Dk).to(dtype), k=r(3, L, G, Dk).to(dtype), v=r(3, L, H, Dv).to(dtype),
                 log_decay=-torch.exp(r(3, L, H) - 2)) for _ in range(2)]
    for t in toks:                                                # one prompt
        for x in t.values():
            x[1:, :50] = x[:1, :50]
    pool = torch.full((2, slots, H, Dk, Dv), 9.0).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()             # noqa: E731
    for n, t in enumerate(toks):
        _, h = ssm.linear_attention_fwd(*(t[x][:1, :50].contiguous().cuda() for x in ("q", "k", "v", "log_decay")))
        pool[n, 2] = h[0]
    ssm.state_slots_copy(pool, i32(2, 2), i32(0, 4), dim=1)       # beams 0, 1, 2 in slots 0, 2, 4
    outs = [[[] for _ in range(3)] for _ in range(2)]

    def go(at, rows, where):
        for n, t in enumerate(toks):
            o = ssm.linear_state_update(pool[n], *(t[x][rows, at].contiguous().cuda() for x in ("q", "k", "v", "log_decay")),
                                        slots=i32(*where))
            for b, row in enumerate(rows):
                outs[n][row].append(o[b])
    for at in range(50, 56):
        go(at, [0, 1, 2], [0, 2, 4])
    ssm.state_slots_copy(pool, i32(0, -1), i32(4, 2), dim=1)      # beam 2 takes beam 0's place; slot 2 starts anew
    for at in range(56, L):
        go(at, [0, 1, 2], [0, 2, 4])
    assert (pool[:, 1] == 9).all() and (pool[:, 3] == 9).all()
    for n, t in enumerate(toks):
        whole = {x: y.clone() for x, y in t.items()}
        for y in whole.values():
            y[2, 50:56] = y[0, 50:56]
        for row, first in ((0, 0), (1, 56), (2, 0)):
            one = {x: y[row:row + 1, first:] for x, y in whole.items()}
            want, h = O.linear_attention(**one, scale=Dk ** -0.5)
            allow_o, allow_h = Bd.forward(**one, scale=Dk ** -0.5)
            at = slice(56 - first, None)
            got = torch.stack(outs[n][row][6:], 0)[None]
            Bd.check("o", got, want[:, at], allow_o[:, at])
            Bd.check("state", pool[n, [0, 2, 4][row]][None], h, allow_h)
