"""The gated linear recurrence on the GPU against the fp64 oracle, element by
element within the bounds of _block_bounds (worked out from the inputs)."""
import numpy as np
import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import block as O

import _block_bounds as Bd

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(B, L, D, dtype, seed=0, state=True, bias=True, lens=None, slow=False, gates=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)                            # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g)                             # noqa: E731
    A = -torch.exp(u(D) * 5 - 4.8) if not slow else -torch.exp(u(D) * 10 - 14)
    t = dict(x=r(B, L, D).to(dtype), gate_a=(r(B, L, D) * gates).to(dtype),
             gate_x=(r(B, L, D) * gates).to(dtype), A=A,
             bias_a=u(D) * 2 - 1 if bias else None, bias_x=u(D) * 2 - 1 if bias else None,
             h0=r(B, D) if state else None,
             seq_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return t, r(B, L, D).to(dtype), (r(B, D) if state else None)


def dev(t):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


SHAPES = [
    # B, L, D, row lengths
    (1, 1, 1, None), (1, 1, 64, None), (2, 3, 5, None), (3, 127, 64, None), (1, 128, 64, None),
    (2, 129, 60, None), (1, 255, 68, None), (2, 257, 130, None), (1, 640, 33, None),
    (4, 300, 72, [0, 1, 299, 300]), (5, 260, 67, [128, 129, 127, 256, 0]),
    (3, 131, 4, [-4, 1000, 130]), (2, 1500, 8, None), (2, 1300, 3, [1300, 5]),
    (2, 32, 66, None), (3, 33, 64, [33, 32, 0]), (2, 64, 65, [64, 31]), (3, 65, 128, [65, 64, 1]),
    (2, 97, 62, [97, 96]),
]


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    B, L, D, lens = shape
    for state, bias in ((True, True), (False, False)):
        t, dy, dh = make(B, L, D, dtype, seed=L + D, state=state, bias=bias, lens=lens)
        d = dev(t)
        yr, hr = O.gated_scan(**t)
        ey, eh, keep = Bd.gated(**t)
        y = torch.full((B, L, D), 7.0, dtype=dtype, device="cuda")
        y, h, ck = ssm.gated_scan_fwd_ckpt(**d, out=y)
        there = torch.ones(B, L, dtype=torch.bool)
        if lens is not None:
            there = torch.arange(L)[None] < torch.tensor(lens)[:, None]
        assert torch.all(y.cpu()[~there] == 7.0)                 # padding untouched
        Bd.check(torch.where(there[..., None], y.cpu(), torch.zeros(1, dtype=dtype)), yr, ey, "y")
        Bd.check(h, hr, eh, "h_last")
        y2, h2 = ssm.gated_scan_fwd(**d, out=torch.full_like(y, 7.0))
        assert torch.equal(y2, y) and torch.equal(h2, h)
        assert torch.equal(ck[:, 0], d["h0"] if state else torch.zeros(B, D, device="cuda"))

        gr = O.gated_scan_bwd(t["x"], t["gate_a"], t["gate_x"], t["A"], dy, t["bias_a"], t["bias_x"],
                              t["h0"], dh, t["seq_lens"])
        eg = Bd.gated_bwd(keep, dy, dh)
        got = {}
        for c in (ck, None):
            got[c is None] = ssm.gated_scan_bwd(
                **d, dy=dy.cuda(), dh_last=None if dh is None else dh.cuda(), ckpt=c)
            assert set(got[c is None]) == set(gr)
        for k, ref in gr.items():
            Bd.check(got[False][k], ref, eg[k], k)
            # the call's own sweep saves what the forward saved
            assert torch.equal(got[False][k], got[True][k]), k


@pytest.mark.parametrize("dtype", [F, BF])
def test_slow_decay_and_shut_gates(dtype):
    """A from e^-14: 1 - a^2 down to 1e-8; gates from -30 to 30."""
    B, L, D = 2, 400, 64
    t, dy, dh = make(B, L, D, dtype, seed=5, slow=True, gates=10.0)
    t["gate_a"].clamp_(-30, 30)
    t["gate_x"].clamp_(-30, 30)
    yr, hr = O.gated_scan(**t)
    ey, eh, keep = Bd.gated(**t)
    d = dev(t)
    y, h, ck = ssm.gated_scan_fwd_ckpt(**d)
    Bd.check(y, yr, ey, "y")
    Bd.check(h, hr, eh, "h_last")
    gr = O.gated_scan_bwd(t["x"], t["gate_a"], t["gate_x"], t["A"], dy, t["bias_a"], t["bias_x"],
                          t["h0"], dh)
    eg = Bd.gated_bwd(keep, dy, dh)
    g = ssm.gated_scan_bwd(**d, dy=dy.cuda(), dh_last=dh.cuda(), ckpt=ck)
    for k, ref in gr.items():
        Bd.check(g[k], ref, eg[k], k)


def test_limits_are_finite():
    """Gates beyond what exp can hold, a decay of exactly one and of exactly zero."""
    B, L, D = 1, 200, 64
    x = torch.ones(B, L, D, device="cuda")
    for ga, gx, A in ((-300.0, 300.0, -1.0), (300.0, -300.0, -1.0), (0.0, 0.0, 0.0),
                      (300.0, 0.0, -1e6), (-88.0, 0.0, -1e-30)):
        a = dict(x=x, gate_a=torch.full_like(x, ga), gate_x=torch.full_like(x, gx),
                 A=torch.full((D,), A, device="cuda"), h0=torch.full((B, D), 2.0, device="cuda"))
        y, h, ck = ssm.gated_scan_fwd_ckpt(**a)
        g = ssm.gated_scan_bwd(**a, dy=torch.ones_like(x), ckpt=ck)
        assert torch.isfinite(y).all() and all(torch.isfinite(v).all() for v in g.values())
        if A == 0.0 or A == -1e-30:
            assert (y - 2.0).abs().max() < 1e-6 and (g["dh0"] == L).all()
        if A == 0.0:
            assert not g["dA"].any()
        if A == -1e6:
            assert torch.equal(y, torch.full_like(y, 0.5))       # a = 0, w = 1, i = 1/2


def test_padding_is_never_read():
    B, L, D = 3, 200, 64
    for dtype in (F, BF):
        t, dy, dh = make(B, L, D, dtype, seed=9, lens=[77, 0, 130])
        clean = ssm.gated_scan_bwd(**dev(t), dy=dy.cuda(), dh_last=dh.cuda())
        yc, hc = ssm.gated_scan_fwd(**dev(t), out=torch.zeros(B, L, D, dtype=dtype, device="cuda"))
        for k in ("x", "gate_a", "gate_x"):
            for b, n in enumerate(t["seq_lens"].tolist()):
                t[k][b, n:] = float("nan")
        for b, n in enumerate(t["seq_lens"].tolist()):
            dy[b, n:] = float("inf")
        y, h = ssm.gated_scan_fwd(**dev(t), out=torch.zeros(B, L, D, dtype=dtype, device="cuda"))
        g = ssm.gated_scan_bwd(**dev(t), dy=dy.cuda(), dh_last=dh.cuda())
        assert torch.equal(y, yc) and torch.equal(h, hc)
        for k in clean:
            assert torch.equal(g[k], clean[k]), k
        for k in ("dx", "dgate_a", "dgate_x"):
            assert not g[k][0, 77:].any() and not g[k][1].any() and not g[k][2, 130:].any()


def test_no_tokens():
    d = dev(make(2, 0, 12, BF)[0])
    y, h, ck = ssm.gated_scan_fwd_ckpt(**d)
    assert y.shape == (2, 0, 12) and ck.shape == (2, 0, 12) and torch.equal(h, d["h0"])
    _, h = ssm.gated_scan_fwd(**dict(d, h0=None))
    assert not h.any()
    dh = torch.randn(2, 12, device="cuda")
    g = ssm.gated_scan_bwd(**d, dy=d["x"], dh_last=dh)
    assert torch.equal(g["dh0"], dh) and not any(g[k].any() for k in ("dA", "dbias_a", "dbias_x"))
    g = ssm.gated_scan_bwd(**d, dy=d["x"], ckpt=ck)
    assert not g["dh0"].any()


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("shape", [(1, 1), (1, 1536), (3, 7), (64, 100), (5, 2562)])
def test_step(shape, dtype):
    B, D = shape
    t, _, _ = make(B, 1, D, dtype, seed=B)
    d = dev(t)
    state = d["h0"].clone()
    y = ssm.gated_state_update(state, d["x"][:, 0].contiguous(), d["gate_a"][:, 0].contiguous(),
                               d["gate_x"][:, 0].contiguous(), d["A"], d["bias_a"], d["bias_x"])
    ys, hs = ssm.gated_scan_fwd(**d)
    assert torch.equal(y, ys[:, 0]) and torch.equal(state, hs)      # the scan's arithmetic
    yr, hr = O.gated_scan(**t)
    ey, eh, _ = Bd.gated(**t)
    Bd.check(y, yr[:, 0], ey[:, 0], "y")
    Bd.check(state, hr, eh, "state")


def test_tokens_one_by_one_are_the_scan():
    """Prefill, then decode: the scan over a prompt and steps over the rest
    against one scan over both."""
    B, L, D, n = 2, 300, 96, 290
    t, _, _ = make(B, L, D, BF, seed=2)
    d = dev(t)
    cut = lambda a, b: {k: (v[:, a:b].contiguous() if v is not None and v.dim() == 3 else v)  # noqa: E731
                        for k, v in d.items()}
    _, state = ssm.gated_scan_fwd(**cut(0, n))
    ys = []
    for k in range(n, L):
        c = cut(k, k + 1)
        ys.append(ssm.gated_state_update(state, c["x"][:, 0], c["gate_a"][:, 0].contiguous(),
                                         c["gate_x"][:, 0].contiguous(), c["A"], c["bias_a"],
                                         c["bias_x"]))
    yr, hr = O.gated_scan(**t)
    ey, eh, _ = Bd.gated(**t)
    Bd.check(torch.stack(ys, 1), yr[:, n:], ey[:, n:], "y")
    Bd.check(state, hr, eh, "state")


def test_writes_stay_inside():
    B, L, D, pad = 2, 137, 68, 64
    t, dy, dh = make(B, L, D, BF, seed=1, lens=[137, 90])
    n = B * L * D
    guard = torch.full((n + 2 * pad,), 9.0, device="cuda", dtype=BF)
    ssm.gated_scan_fwd(**dev(t), out=guard[pad:pad + n].view(B, L, D))
    assert torch.all(guard[:pad] == 9) and torch.all(guard[pad + n:] == 9)
    n = B * 2 * D
    guard = torch.full((n + 2 * pad,), 9.0, device="cuda")
    ssm.gated_scan_fwd_ckpt(**dev(t), ckpt=guard[pad:pad + n].view(B, 2, D))
    assert torch.all(guard[:pad] == 9) and torch.all(guard[pad + n:] == 9)
    assert torch.all(guard[pad + n - D:pad + n] == 9)             # a state behind a row's end: not written
    need = ssm.gated_scan_bwd_workspace_bytes(B, L, D, BF)
    ws = torch.full((need + 512,), 3, dtype=torch.uint8, device="cuda")
    a = ssm.gated_scan_bwd(**dev(t), dy=dy.cuda(), dh_last=dh.cuda(), workspace=ws[256:256 + need])
    assert torch.all(ws[:256] == 3) and torch.all(ws[256 + need:] == 3)
    b = ssm.gated_scan_bwd(**dev(t), dy=dy.cuda(), dh_last=dh.cuda())
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("walkers", ["1", "2", "5"])
def test_workspace_is_cleared_and_kept_within(walkers, monkeypatch):
    """A workspace full of anything, and one that a longer call has used,
    between guards."""
    monkeypatch.setenv("SSM_GATED_WALKERS", walkers)
    B, L, D = 2, 2100, 100
    t, dy, dh = make(B, L, D, BF, seed=1, lens=[2100, 1300])
    d, dy, dh = dev(t), dy.cuda(), dh.cuda()
    y, h = ssm.gated_scan_fwd(**d, out=torch.zeros(B, L, D, dtype=BF, device="cuda"))
    g = ssm.gated_scan_bwd(**d, dy=dy, dh_last=dh)
    need = ssm.gated_scan_workspace_bytes(B, L, D, BF)
    assert (need > 0) == (walkers != "1")
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            y2, h2 = ssm.gated_scan_fwd(**d, workspace=ws[256:256 + need],
                                        out=torch.zeros(B, L, D, dtype=BF, device="cuda"))
            assert torch.equal(y, y2) and torch.equal(h, h2)
        assert torch.all(ws[:256] == fill) and torch.all(ws[256 + need:] == fill)
    need = ssm.gated_scan_bwd_workspace_bytes(B, L, D, BF)
    for fill in (0, 0xFF):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            g2 = ssm.gated_scan_bwd(**d, dy=dy, dh_last=dh, workspace=ws[256:256 + need])
            assert all(torch.equal(g[k], g2[k]) for k in g)
        assert torch.all(ws[:256] == fill) and torch.all(ws[256 + need:] == fill)


def test_two_graphs_share_a_workspace():
    """Two captured calls of different lengths over one workspace, replayed in
    turn with eager work between."""
    t1, _, _ = make(1, 3000, 64, BF, seed=1)
    t2, _, _ = make(2, 1700, 96, F, seed=2)
    d1, d2 = dev(t1), dev(t2)
    need = max(ssm.gated_scan_workspace_bytes(1, 3000, 64, BF), ssm.gated_scan_workspace_bytes(2, 1700, 96, F))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    w1, w2 = ssm.gated_scan_fwd(**d1), ssm.gated_scan_fwd(**d2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ssm.gated_scan_fwd(**d1, workspace=ws)
        ssm.gated_scan_fwd(**d2, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = ssm.gated_scan_fwd(**d1, workspace=ws)
    with torch.cuda.graph(g2):
        o2 = ssm.gated_scan_fwd(**d2, workspace=ws)
    for _ in range(4):
        g1.replay()
        g2.replay()
        ws.random_(0, 255)
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1[0], w1[0]) and torch.equal(o1[1], w1[1])
        assert torch.equal(o2[0], w2[0]) and torch.equal(o2[1], w2[1])


def test_odd_values_pass_between_workgroups(monkeypatch):
    """States and decays that are zero, denormal, infinite or NaN go through
    the hand-over as through one workgroup (a slot's zero means empty)."""
    B, L, D = 1, 1500, 64
    base, dy, _ = make(B, L, D, F, seed=6)
    base = dev(base)
    dy = dy.cuda()
    for case in range(5):
        d = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in base.items()}
        if case == 0:
            d["x"].zero_()
            d["h0"].zero_()
        elif case == 1:
            d["A"].fill_(-1e5)                       # every decay zero
            d["x"].mul_(torch.rand(L, 1, device="cuda") < 0.01)
        elif case == 2:
            d["x"].fill_(-1e-42)
            d["h0"].fill_(-1e-44)
        elif case == 3:
            d["x"][0, 300, 5] = float("inf")
            d["x"][0, 700, 6] = float("nan")
        else:
            d["x"].neg_().mul_(0.0)                  # zeros of both signs
        got = []
        for w in ("1", "3"):
            monkeypatch.setenv("SSM_GATED_WALKERS", w)
            y, h, ck = ssm.gated_scan_fwd_ckpt(**d)
            g = ssm.gated_scan_bwd(**d, dy=dy * (0.0 if case == 0 else 1.0), ckpt=ck)
            got.append({"y": y, "h": h, "ck": ck, **g})
        torch.cuda.synchronize()
        for k in got[0]:
            a, b = got[0][k], got[1][k]
            same = (a.view(torch.int32) == b.view(torch.int32)) | (a.isnan() & b.isnan())
            assert same.all(), (case, k)


def test_misaligned_views_are_refused():
    t = dev(make(1, 8, 8, BF)[0])
    flat = torch.zeros(65, dtype=BF, device="cuda")
    t["x"] = flat[1:].view(1, 8, 8)
    with pytest.raises(ssm.SSMError, match="MISALIGNED"):
        ssm.gated_scan_fwd(**t)
    t["x"] = torch.zeros(1, 8, 16, dtype=BF, device="cuda")[:, :, ::2]
    with pytest.raises(ValueError, match="contiguous"):
        ssm.gated_scan_fwd(**t)


@pytest.mark.parametrize("B,L,D", [(2, 700, 128), (1, 3000, 64)])
def test_graph_replays_with_new_inputs_and_two_graphs(B, L, D):
    """Captured forward and backward on a stream of their own, replayed over
    changed inputs with eager work between, against the eager calls."""
    t, dy, dh = make(B, L, D, BF, seed=3)
    d, dy, dh = dev(t), dy.cuda(), dh.cuda()

    def both():
        y, h, ck = ssm.gated_scan_fwd_ckpt(**d)
        return {"y": y, "h": h, **ssm.gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck)}

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    for k in range(4):
        gen = torch.Generator().manual_seed(k)
        d["x"].copy_(torch.randn(B, L, D, generator=gen))
        d["gate_a"].copy_(torch.randn(B, L, D, generator=gen))
        want = both()
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            for n in want:
                assert torch.equal(out[n], want[n]), (k, n)


def test_two_streams_at_once():
    t1, _, _ = make(1, 5000, 64, BF, seed=1)
    t2, _, _ = make(3, 4000, 96, F, seed=2)
    d1, d2 = dev(t1), dev(t2)
    w1, w2 = ssm.gated_scan_fwd(**d1), ssm.gated_scan_fwd(**d2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            got.append((ssm.gated_scan_fwd(**d1), w1))
        with torch.cuda.stream(s2):
            got.append((ssm.gated_scan_fwd(**d2), w2))
    torch.cuda.synchronize()
    for g, w in got:
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("dtype", [F, BF])
def test_long_sequence_sampled(dtype):
    """One long row, the oracle on a few of its channels."""
    B, L, D, ch = 1, 20000, 512, [0, 63, 64, 300, 511]
    t, dy, dh = make(B, L, D, dtype, seed=11)
    d = dev(t)
    y, h, ck = ssm.gated_scan_fwd_ckpt(**d)
    g = ssm.gated_scan_bwd(**d, dy=dy.cuda(), dh_last=dh.cuda(), ckpt=ck)
    sub = {k: (None if v is None else v[..., ch].contiguous()) for k, v in t.items() if k != "seq_lens"}
    yr, hr = O.gated_scan(**sub)
    ey, eh, keep = Bd.gated(**sub)
    Bd.check(y[..., ch], yr, ey, "y")
    Bd.check(h[..., ch], hr, eh, "h_last")
    dys, dhs = dy[..., ch].contiguous(), dh[..., ch].contiguous()
    gr = O.gated_scan_bwd(sub["x"], sub["gate_a"], sub["gate_x"], sub["A"], dys, sub["bias_a"],
                          sub["bias_x"], sub["h0"], dhs)
    eg = Bd.gated_bwd(keep, dys, dhs)
    for k, ref in gr.items():
        Bd.check(g[k][..., ch], ref, eg[k], k)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("shape", [(1, 129, 64, None), (2, 700, 68, None), (1, 2600, 33, None),
                                   (4, 1100, 128, [0, 1100, 129, 640]), (3, 3000, 8, [2999, 1, 1500])])
def test_walkers_agree(shape, dtype, monkeypatch):
    """Any number of workgroups per strip gives the same bits as one."""
    B, L, D, lens = shape
    t, dy, dh = make(B, L, D, dtype, seed=L, lens=lens)
    d, dy, dh = dev(t), dy.cuda(), dh.cuda()

    def run():
        y, h, ck = ssm.gated_scan_fwd_ckpt(**d, out=torch.zeros(B, L, D, dtype=dtype, device="cuda"),
                                           ckpt=torch.zeros(B, -(-L // 128), D, device="cuda"))
        r = {"y": y, "h": h, "ck": ck}
        r.update(ssm.gated_scan_bwd(**d, dy=dy, dh_last=dh, ckpt=ck))
        r.update({"own " + k: v for k, v in ssm.gated_scan_bwd(**d, dy=dy, dh_last=dh).items()})
        torch.cuda.synchronize()
        return r

    monkeypatch.setenv("SSM_GATED_WALKERS", "1")
    assert ssm.gated_scan_walkers(B, L, D) == 1 and ssm.gated_scan_workspace_bytes(B, L, D) == 0
    want = run()
    for n in (2, 3, 7, 64):
        monkeypatch.setenv("SSM_GATED_WALKERS", str(n))
        tiles = -(-L // 256)
        assert ssm.gated_scan_walkers(B, L, D) == min(n, tiles)
        assert ssm.gated_scan_bwd_walkers(B, L, D) == min(n, -(-L // 128))
        assert ssm.gated_scan_workspace_bytes(B, L, D) >= (B * -(-D // 64) * (tiles * 64 * 12 + 4) if tiles > 1 else 0)
        got = run()
        for k in want:
            assert torch.equal(got[k], want[k]), (n, k)


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 elements: its last rows against the same
    rows alone, bit for bit."""
    L, D = 70000, 32768
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, L, D, dtype=BF, device="cuda").normal_(generator=gen)
    A = -torch.rand(D, generator=gen, device="cuda") - 0.01
    # a cut at a tile's border: the second call starts from the first's state
    cut = 128 * 546
    y, h = ssm.gated_scan_fwd(x, x, x, A)
    _, first = ssm.gated_scan_fwd(x[:, :cut], x[:, :cut], x[:, :cut], A)
    tail = x[:, cut:].contiguous()
    y2, h2 = ssm.gated_scan_fwd(tail, tail, tail, A, h0=first)
    assert torch.equal(y[:, cut:], y2) and torch.equal(h, h2)
