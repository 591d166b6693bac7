"""Linear attention on the GPU against the fp64 definition, element by element
within the allowances of _linear_bounds (worked out from the inputs)."""
import math

import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import linear as O

import _linear_bounds as Bd

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(B, L, H, G, Dk, Dv, dtype, seed=0, state=True, by_head=False, lens=None, rate=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)                            # noqa: E731
    t = dict(q=r(B, L, G, Dk).to(dtype), k=r(B, L, G, Dk).to(dtype), v=r(B, L, H, Dv).to(dtype),
             log_decay=-torch.exp(2 * r(*((H,) if by_head else (B, L, H))) - 3) * rate, scale=Dk ** -0.5,
             h0=r(B, H, Dk, Dv) if state else None,
             seq_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return t, r(B, L, H, Dv).to(dtype), (r(B, H, Dk, Dv) if state else None)


def dev(t):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


def run_both(t, do, dh, decay_grad=True):
    """Forward and backward of one set of inputs, both checked."""
    d, lens, by_head = dev(t), t["seq_lens"], t["log_decay"].dim() == 1
    out = torch.full(do.shape, 7.0, dtype=do.dtype).cuda()
    o, h = ssm.linear_attention_fwd(**d, out=out)
    grads = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], d["log_decay"], do.cuda(), scale=t["scale"], h0=d["h0"],
                                     dh_last=None if dh is None else dh.cuda(), seq_lens=d["seq_lens"],
                                     decay_grad=decay_grad)
    torch.cuda.synchronize()
    want_o, want_h = O.linear_attention(**t)
    allow_o, allow_h = Bd.forward(**t)
    if lens is not None:
        there = torch.arange(do.shape[1]) < lens.clamp(0, do.shape[1])[:, None]
        assert (o.cpu()[~there] == 7.0).all()                     # the padding is left alone
        o = torch.where(there[..., None, None].cuda(), o, 0.0)
    Bd.check("o", o, want_o, allow_o)
    Bd.check("h_last", h, want_h, allow_h)
    Bd.near("h_last", h, want_h, 1e-5)
    bar = 1e-5 if do.dtype == F else 5e-3
    Bd.near("o", o, want_o, bar)
    args = dict(q=t["q"], k=t["k"], v=t["v"], log_decay=t["log_decay"], do=do, scale=t["scale"], h0=t["h0"],
                dh_last=dh, seq_lens=lens)
    want = O.linear_attention_bwd(**args)
    allow = Bd.backward(**args, split=decay_grad)
    if not decay_grad:
        del want["dlog_decay"]
    assert set(grads) == set(want)
    for n in want:
        Bd.check(n, grads[n], want[n], allow[n])
        # a decay's gradient by head is a sum over all tokens that may cancel to any part of its terms' size:
        # no bar relative to the result follows from the roundings, the allowance above does
        if n != "dlog_decay" or not by_head:
            Bd.near(n, grads[n], want[n], 1e-5 if grads[n].dtype == F else bar)
        if lens is not None and n in ("dq", "dk", "dv"):
            assert not grads[n].cpu()[~there].any()
    return o, h, grads


SHAPES = [
    # B, L, H, G, Dk, Dv, row lengths
    (1, 1, 1, 1, 16, 16, None), (2, 2, 2, 2, 64, 64, None), (1, 31, 3, 1, 48, 32, None), (2, 32, 2, 2, 32, 80, None),
    (1, 33, 2, 1, 64, 112, None), (2, 63, 1, 1, 128, 64, None), (1, 64, 2, 2, 96, 128, None), (1, 65, 4, 2, 128, 128, None),
    (2, 127, 3, 3, 16, 48, None), (1, 129, 2, 2, 80, 16, None), (1, 200, 2, 1, 256, 64, None), (1, 97, 1, 1, 256, 256, None),
    (1, 130, 2, 2, 64, 256, None), (4, 150, 2, 1, 64, 64, [0, 1, 150, 149]), (5, 100, 2, 2, 112, 48, [64, 65, 63, 32, 0]),
    (3, 70, 4, 4, 16, 16, [-3, 1000, 33]), (2, 700, 2, 1, 64, 64, None), (2, 600, 1, 1, 128, 96, [600, 130]),
]


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    *size, lens = shape
    for state, by_head in ((True, False), (False, True)):
        run_both(*make(*size, dtype, seed=sum(size), state=state, by_head=by_head, lens=lens))


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("size", [(2, 100, 2, 1, 64, 64), (1, 90, 2, 2, 128, 48), (1, 70, 2, 2, 256, 144)])
def test_without_the_decays_gradient(size, dtype):
    run_both(*make(*size, dtype), decay_grad=False)


@pytest.mark.parametrize("segments", [2, 3, 5])
@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("size, lens", [((2, 330, 2, 1, 64, 64), None), ((4, 300, 1, 1, 128, 80), [300, 64, 0, 129]),
                                        ((1, 257, 2, 2, 48, 256), None)])
def test_forced_segments(size, lens, dtype, segments, monkeypatch):
    monkeypatch.setenv("SSM_LINEAR_SEGMENTS", str(segments))
    tokens = -(-(-(-size[1] // segments)) // 64) * 64             # of a segment: whole blocks of 64
    assert ssm.linear_attention_segments(*size[:3], *size[4:], dtype=dtype) == -(-size[1] // tokens)
    for by_head in (False, True):
        run_both(*make(*size, dtype, seed=segments, by_head=by_head, lens=lens))


def test_planned_segments():
    assert ssm.linear_attention_segments(1, 1024, 2, 32, 32, dtype=F) > 1
    run_both(*make(1, 1024, 2, 2, 32, 32, F))
    run_both(*make(1, 1024, 2, 1, 32, 32, BF, lens=[900]))


@pytest.mark.parametrize("dtype", [F, BF])
def test_strong_and_absent_decays(dtype):
    """Decays of zero (nothing is forgotten), of minus infinity and far below (all is), among ordinary ones."""
    t, do, dh = make(2, 140, 2, 2, 64, 32, dtype, seed=5)
    g = t["log_decay"]
    g[0, :70] = 0.0
    g[1, ::3] = -300.0
    g[1, 1::7] = -1e30
    g[:, 100] = -90.0
    run_both(t, do, dh)
    hard = {**t, "log_decay": g.clone()}
    hard["log_decay"][:, 33] = -math.inf                          # exp is zero: as if the row began there
    o, h = ssm.linear_attention_fwd(**dev(hard))
    grads = ssm.linear_attention_bwd(*(dev(hard)[n] for n in ("q", "k", "v", "log_decay")), do.cuda(), h0=t["h0"].cuda())
    soft = {**t, "log_decay": g.clone()}
    soft["log_decay"][:, 33] = -2000.0
    Bd.check("o", o, O.linear_attention(**soft)[0], Bd.forward(**soft)[0])
    for n, x in grads.items():
        assert torch.isfinite(x).all(), n
    allow = Bd.backward(*(soft[n] for n in ("q", "k", "v", "log_decay")), do, t["scale"], t["h0"])["dlog_decay"]
    assert (grads["dlog_decay"][:, 33].cpu().double().abs() <= allow[:, 33]).all()    # zero, of sums that cancel


def test_growing_state():
    t, do, dh = make(1, 80, 2, 2, 32, 32, F, rate=-0.05)          # log decays above zero
    assert (t["log_decay"] > 0).all()
    run_both(t, do, dh)


@pytest.mark.parametrize("dtype", [F, BF])
def test_a_nan_decay_starts_at_its_token(dtype):
    t, _, _ = make(1, 100, 2, 1, 64, 64, dtype)
    clean, _ = ssm.linear_attention_fwd(**dev(t))
    t["log_decay"][0, 40, 1] = math.nan
    o, h = ssm.linear_attention_fwd(**dev(t))
    assert torch.equal(o[:, :40], clean[:, :40]) and torch.equal(o[:, :, 0], clean[:, :, 0])
    assert o[0, 40:, 1].isnan().all() and h[0, 1].isnan().all() and not h[0, 0].isnan().any()


@pytest.mark.parametrize("dtype", [F, BF])
def test_padding_is_never_read(dtype):
    t, do, dh = make(3, 150, 2, 1, 64, 80, dtype, lens=[0, 77, 128])
    there = torch.arange(150) < t["seq_lens"][:, None]
    first = run_both(t, do, dh)
    for x in (t["q"], t["k"], t["v"], do):
        x[~there] = math.nan
    t["log_decay"][~there] = math.inf
    d = dev(t)
    o, h = ssm.linear_attention_fwd(**d)
    assert torch.equal(h, first[1]) and torch.equal(torch.where(there[..., None, None].cuda(), o, 0.0), first[0])
    grads = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], d["log_decay"], do.cuda(), scale=t["scale"], h0=d["h0"],
                                     dh_last=dh.cuda(), seq_lens=d["seq_lens"])
    for n, x in grads.items():
        assert torch.equal(x, first[2][n]), n


@pytest.mark.parametrize("dtype", [F, BF])
def test_parts_of_a_projection(dtype):
    """Queries, keys and values as parts of one wider tensor: the same bits as their dense copies."""
    B, L, H, G, Dk, Dv = 2, 70, 4, 2, 32, 48
    wide = torch.randn(B, L, 2 * G * Dk + H * Dv + 40, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    q, k, v = (wide[..., a:a + n].unflatten(2, s) for a, n, s in
               ((8, G * Dk, (G, Dk)), (8 + G * Dk, G * Dk, (G, Dk)), (16 + 2 * G * Dk, H * Dv, (H, Dv))))
    t, do, _ = make(B, L, H, G, Dk, Dv, dtype)
    g = t["log_decay"].cuda()
    do = do.cuda()
    a = ssm.linear_attention_fwd(q, k, v, g)
    b = ssm.linear_attention_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = ssm.linear_attention_bwd(q, k, v, g, do)
    b = ssm.linear_attention_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g, do)
    assert all(torch.equal(a[n], b[n]) for n in b)
    state = torch.zeros(B, H, Dk, Dv).cuda()
    a = ssm.linear_state_update(state.clone(), q[:, 5], k[:, 5], v[:, 5], g[:, 5].contiguous())
    b = ssm.linear_state_update(state, q[:, 5].contiguous(), k[:, 5].contiguous(), v[:, 5].contiguous(),
                                g[:, 5].contiguous())
    assert torch.equal(a, b)


def test_dirty_workspace_and_its_end():
    """Whatever the workspace holds, the results are the same, and nothing behind it is written."""
    t, do, dh = make(2, 400, 2, 1, 64, 64, BF)
    d = dev(t)
    need = ssm.linear_attention_bwd_workspace_bytes(2, 400, 2, 1, 64, 64)
    need_f = ssm.linear_attention_workspace_bytes(2, 400, 2, 64, 64)
    outs = []
    for fill in (0, 255):
        ws = torch.full((max(need, need_f) + 4096,), fill, dtype=torch.uint8).cuda()
        g = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], d["log_decay"], do.cuda(), h0=d["h0"], dh_last=dh.cuda(),
                                     workspace=ws[:need])
        o, h = ssm.linear_attention_fwd(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"], workspace=ws[:need_f])
        torch.cuda.synchronize()
        assert (ws[max(need, need_f):] == fill).all()
        outs.append([*g.values(), o, h])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_no_tokens():
    z = dict(dtype=BF, device="cuda")
    h0, dh = torch.randn(2, 3, 16, 32).cuda(), torch.randn(2, 3, 16, 32).cuda()
    q, v = torch.empty(2, 0, 1, 16, **z), torch.empty(2, 0, 3, 32, **z)
    for g in (torch.empty(2, 0, 3).cuda(), torch.full((3,), -0.1).cuda()):
        o, h = ssm.linear_attention_fwd(q, q, v, g, h0=h0)
        assert o.shape == (2, 0, 3, 32) and torch.equal(h, h0)
        assert not ssm.linear_attention_fwd(q, q, v, g)[1].any()
        r = ssm.linear_attention_bwd(q, q, v, g, v, h0=h0, dh_last=dh)
        assert torch.equal(r["dh0"], dh) and not r["dlog_decay"].any()


# ---- single tokens

@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("B, H, G, Dk, Dv", [(1, 1, 1, 16, 16), (3, 4, 2, 64, 80), (2, 3, 3, 256, 256), (5, 2, 1, 96, 112),
                                             (300, 2, 2, 32, 48)])
def test_step(B, H, G, Dk, Dv, dtype):
    for by_head, n in ((False, 0), (True, B + 4)):
        t, _, _ = make(B, 1, H, G, Dk, Dv, dtype, seed=B + Dv, by_head=by_head)
        q, k, v, g = t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["log_decay"] if by_head else t["log_decay"][:, 0]
        gen = torch.Generator().manual_seed(9)
        pool = torch.randn(n or B, H, Dk, Dv, generator=gen)
        slots = torch.randperm(n, generator=gen)[:B].int() if n else None
        if n and B > 2:
            slots[1] = -1                                         # a padded row
            slots[2] = n + 3                                      # a slot that is not there
            slots[-1] = slots[0]                                  # two tokens of one sequence
        state = pool.clone().cuda()
        o = ssm.linear_state_update(state, q.cuda(), k.cuda(), v.cuda(), g.cuda(),
                                    slots=None if slots is None else slots.cuda())
        want, after = O.linear_step(pool, q, k, v, g, Dk ** -0.5, slots)
        size, bound = O.linear_step(pool.abs(), q.abs(), k.abs(), v.abs(), g, Dk ** -0.5, slots)
        n32 = (Dk + 24) * Bd.U
        half = Bd.HALF if dtype == BF else 0.0
        Bd.check("o", o, want, n32 * size + half * want.abs() + 1e-37)
        Bd.check("state", state, after, 12 * Bd.U * bound + 1e-37)
        if n:
            untouched = [i for i in range(n) if i not in slots.tolist()]
            assert torch.equal(state.cpu()[untouched], pool[untouched])


@pytest.mark.parametrize("dtype", [F, BF])
def test_steps_continue_a_prompt(dtype):
    t, _, _ = make(2, 75, 2, 1, 64, 64, dtype)
    d = dev(t)
    whole, h = ssm.linear_attention_fwd(**d)
    part = {n: (x[:, :70].contiguous() if n in ("q", "k", "v", "log_decay") else x) for n, x in d.items()}
    _, state = ssm.linear_attention_fwd(**part)
    allow_o, allow_h = Bd.forward(**t)
    for i in range(70, 75):
        o = ssm.linear_state_update(state, d["q"][:, i], d["k"][:, i], d["v"][:, i], d["log_decay"][:, i].contiguous())
        assert ((o.cpu().double() - whole[:, i].cpu().double()).abs() <= 2 * allow_o[:, i]).all()
    assert ((state.cpu().double() - h.cpu().double()).abs() <= 2 * allow_h).all()


def test_many_rows_of_one_slot():
    """All rows name one slot: they are its tokens, in order."""
    t, _, _ = make(1, 40, 2, 2, 32, 32, F)
    d = dev(t)
    state = torch.stack([d["h0"][0], torch.ones_like(d["h0"][0])])
    o = ssm.linear_state_update(state, d["q"][0], d["k"][0], d["v"][0], d["log_decay"][0].contiguous(),
                                slots=torch.zeros(40, dtype=torch.int32).cuda())
    want, h = O.linear_attention(**t)
    allow_o, allow_h = Bd.forward(**t)
    Bd.check("o", o, want[0], allow_o[0])
    Bd.check("state", state[:1], h, allow_h)
    assert (state[1] == 1).all()


# ---- how it is called

def test_same_bits_every_time():
    t, do, dh = make(2, 300, 4, 2, 64, 64, BF)
    d = dev(t)
    args = (d["q"], d["k"], d["v"], d["log_decay"], do.cuda())
    first = ssm.linear_attention_bwd(*args, h0=d["h0"], dh_last=dh.cuda())
    for _ in range(3):
        again = ssm.linear_attention_bwd(*args, h0=d["h0"], dh_last=dh.cuda())
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_two_streams_at_once():
    calls = []
    for seed in (1, 2):
        t, do, dh = make(2, 500, 4, 2, 64, 64, BF, seed=seed)
        d = dev(t)
        args = (d["q"], d["k"], d["v"], d["log_decay"], do.cuda())
        calls.append((args, dict(h0=d["h0"], dh_last=dh.cuda())))
    want = [ssm.linear_attention_bwd(*a, **k) for a, k in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(5):
        got.clear()
        for s, (a, k) in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(ssm.linear_attention_bwd(*a, **k))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(x[n], y[n]) for n in y)


def test_captured_and_replayed():
    t, do, dh = make(2, 400, 2, 1, 64, 64, BF, lens=[400, 123])
    d = dev(t)
    do, dh = do.cuda(), dh.cuda()
    state, token = torch.randn(3, 2, 64, 64).cuda(), torch.randn(2, 1, 64).to(BF).cuda()
    v1, g1 = torch.randn(2, 2, 64).to(BF).cuda(), torch.full((2, 2), -0.1).cuda()
    slots = torch.tensor([2, 0], dtype=torch.int32).cuda()

    there = (torch.arange(400) < t["seq_lens"][:, None])[..., None, None].cuda()

    def work():
        o, h = ssm.linear_attention_fwd(**d)
        r = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], d["log_decay"], do, h0=d["h0"], dh_last=dh,
                                     seq_lens=d["seq_lens"])
        y = ssm.linear_state_update(state, token, token, v1, g1, slots=slots)
        return [torch.where(there, o, 0), h, y, *r.values()]

    held = state.clone()
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for n in range(4):
        for x in (d["q"], d["v"], do):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(n)).to(BF))
        state.copy_(held)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        after = state.clone()
        state.copy_(held)
        want = work()
        assert torch.equal(after, state)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


def test_offsets_past_32_bits():
    """Values 2^31 elements apart: a long stride between tokens, and many rows."""
    L, H, Dv = 1030, 1, 16
    row = 1 << 21
    big = torch.empty(L * row, dtype=BF, device="cuda")            # 2.2e9 elements
    v = big.as_strided((1, L, H, Dv), (L * row, row, Dv, 1))
    t, do, _ = make(1, L, H, 1, 16, Dv, BF, state=False)
    d = dev(t)
    v.copy_(d["v"])
    a = ssm.linear_attention_fwd(d["q"], d["k"], v, d["log_decay"])
    b = ssm.linear_attention_fwd(**d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = ssm.linear_attention_bwd(d["q"], d["k"], v, d["log_decay"], do.cuda())
    b = ssm.linear_attention_bwd(d["q"], d["k"], d["v"], d["log_decay"], do.cuda())
    assert all(torch.equal(a[n], b[n]) for n in b)


def test_outputs_past_32_bits():
    """2^31 output elements and more: the last rows as a call of their own."""
    B, L, H, Dv = 2, 4200, 2048, 128
    q = torch.randn(B, L, 1, 16, dtype=BF, device="cuda")
    v = torch.randn(B, L, H, Dv, dtype=BF, device="cuda")
    g = torch.full((H,), -0.05, device="cuda")
    assert v.numel() > 2 ** 31
    o, h = ssm.linear_attention_fwd(q, q, v, g)
    for b, heads in ((0, slice(0, 2)), (1, slice(H - 2, H))):
        x, y = ssm.linear_attention_fwd(q[b:b + 1], q[b:b + 1], v[b:b + 1, :, heads].contiguous(), g[:2].contiguous())
        near = (o[b:b + 1, :, heads].float() - x.float()).norm() / x.float().norm()
        assert float(near) < 5e-3 and float((h[b:b + 1, heads] - y).norm() / y.norm()) < 1e-5


def test_the_most_heads():
    """2^20 heads of the widest values: one launch of 2^31 work-items, every output of it exact."""
    B, H, Dk, Dv = 64, 16384, 16, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randint(-2, 3, (B, 1, 1, Dk), generator=g, device="cuda").to(BF) for _ in range(2))
    v = torch.randint(-4, 5, (B, 1, H, Dv), generator=g, device="cuda", dtype=torch.int8).to(BF)
    o, _ = ssm.linear_attention_fwd(q, k, v, torch.zeros(H, device="cuda"), scale=1.0, return_last_state=False)
    dots = (q.float() * k.float()).sum(-1)                        # at most 64 in size: products with v are exact in bf16
    assert torch.equal(o, (dots.reshape(B, 1, 1, 1) * v.float()).to(BF))
