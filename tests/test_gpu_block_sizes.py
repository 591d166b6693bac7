"""The calls around the scan at sizes past what one launch, 32-bit offsets or
the GPU's workgroups at once can hold."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import block as O

import _block_bounds as Bd

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def randn(*shape, dtype=F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=g)


def test_more_strips_than_one_launch_takes():
    """2^24 batch rows of one short tile, a strip each: 256 threads a strip
    would be 2^32 work-items.  The rows against the same rows in two calls."""
    B, L, D = (1 << 24) + 3, 1, 1
    x, ga, gx, dy = (randn(B, L, D, seed=k) for k in range(4))
    h0, dh = randn(B, D, seed=4), randn(B, D, seed=5)
    lens = (torch.arange(B, device="cuda") % 5 != 0).to(torch.int32)
    A, ba, bx = (torch.full((D,), v, device="cuda") for v in (-0.5, 0.1, -0.2))
    y, h, ck = ssm.gated_scan_fwd_ckpt(x, ga, gx, A, ba, bx, h0, seq_lens=lens, out=torch.zeros_like(x))
    g = ssm.gated_scan_bwd(x, ga, gx, A, dy, ba, bx, h0, dh, seq_lens=lens, ckpt=ck)
    own = ssm.gated_scan_bwd(x, ga, gx, A, dy, ba, bx, h0, dh, seq_lens=lens)
    assert all(torch.equal(g[k], own[k]) for k in g)
    half = B // 2 // 8 * 8                                     # (a view has to begin at 16 bytes)
    for s in (slice(0, half), slice(half, B)):
        y2, h2, ck2 = ssm.gated_scan_fwd_ckpt(x[s], ga[s], gx[s], A, ba, bx, h0[s], seq_lens=lens[s],
                                              out=torch.zeros_like(x[s]))
        assert torch.equal(y[s], y2) and torch.equal(h[s], h2) and torch.equal(ck[s], ck2)
        g2 = ssm.gated_scan_bwd(x[s], ga[s], gx[s], A, dy[s], ba, bx, h0[s], dh[s], seq_lens=lens[s], ckpt=ck2)
        for k in ("dx", "dgate_a", "dgate_x", "dh0"):
            assert torch.equal(g[k][s], g2[k]), k
    # a sum: a term passes at most B / 16 + 16 additions, of 2^-24 each of what
    # is summed so far
    for k, terms in (("dbias_a", g["dgate_a"]), ("dbias_x", g["dgate_x"])):
        terms = terms.double()
        off = abs(float(g[k].double() - terms.sum()))
        assert off <= (B / 16 + 16) * 2.0 ** -24 * float(terms.abs().sum()), k


def test_more_rows_of_one_tile_than_one_launch_takes():
    """1024 threads a strip: the limit of one launch is at 2^22 strips."""
    B, L, D = (1 << 22) + 1, 129, 1
    x = randn(B, L, D, dtype=BF)
    A = torch.full((D,), -0.5, device="cuda")
    y, h = ssm.gated_scan_fwd(x, x, x, A)
    half = B // 2 // 8 * 8
    for s in (slice(0, half), slice(half, B)):
        y2, h2 = ssm.gated_scan_fwd(x[s], x[s], x[s], A)
        assert torch.equal(y[s], y2) and torch.equal(h[s], h2)


def test_step_of_more_items_than_one_launch_takes():
    """A decode step of 2^32 single channels (an odd width)."""
    B, D = 858993460, 5
    assert B * D > 1 << 32
    x, state = randn(B, D, dtype=BF), randn(B, D, seed=1)
    A = -torch.rand(D, device="cuda")
    cuts = [0, 8, B // 2 // 8 * 8, B // 8 * 8 - 64, B]
    before = [(state[a:b][:1000].clone(), state[a:b][-1000:].clone()) for a, b in zip(cuts, cuts[1:])]
    y = ssm.gated_state_update(state, x, x, x, A)
    for (a, b), ends in zip(zip(cuts, cuts[1:]), before):
        for s0, xs, ys, ss in ((ends[0], x[a:b][:1000], y[a:b][:1000], state[a:b][:1000]),
                               (ends[1], x[a:b][-1000:], y[a:b][-1000:], state[a:b][-1000:])):
            xs = xs.clone()
            y2 = ssm.gated_state_update(s0, xs, xs, xs, A)
            assert torch.equal(ys, y2) and torch.equal(ss, s0)


def test_more_norm_rows_than_one_launch_takes():
    """2^29 rows of two elements, eight threads a row; the rows against the
    same rows in calls of their own."""
    rows, D = (1 << 29) + 37, 2
    x = randn(rows, D, dtype=BF)
    w, b = randn(D, seed=1), randn(D, seed=2)
    r = ssm.layer_norm_fwd(x, w, b, out=torch.full_like(x, 7.0))
    step = 1 << 27
    for a in range(0, rows, step):
        e = ssm.layer_norm_fwd(x[a:a + step], w, b)
        for k in e:
            assert torch.equal(e[k], r[k][a:a + step]), (k, a)


def test_sums_of_more_columns_than_one_launch_takes():
    """The parameters' gradients of 2^28 columns, 16 threads a column."""
    D = (1 << 28) + 5
    x, dy = randn(1, D, dtype=BF), randn(1, D, dtype=BF, seed=1)
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 0.5, device="cuda")
    w = torch.ones(D, device="cuda")
    g = ssm.layer_norm_bwd(x, dy, mean, rstd, weight=w, bias=w)
    assert torch.equal(g["dbias"], dy[0].float())
    n = (x[0].float() - 0.25) * 0.5
    assert torch.equal(g["dweight"], dy[0].float() * n)


@pytest.mark.parametrize("state", [False, True])
def test_more_conv_rows_than_one_launch_takes(state):
    """2^23 batch rows of a workgroup of 512 threads each."""
    B, L, D, K = (1 << 23) + 3, 1, 1, 3
    x, du = randn(B, L, D), randn(B, L, D, seed=1)
    w = torch.tensor([[0.5, -0.25, 2.0]], device="cuda")
    b = torch.tensor([0.1], device="cuda")
    kw = dict(state=randn(B, D, K - 1, seed=2), dstate_out=randn(B, D, K - 1, seed=3)) if state else {}
    g = ssm.causal_conv1d_silu_bwd(x, w, du, bias=b, **kw)
    half = B // 2 // 8 * 8
    for s in (slice(0, half), slice(half, B)):
        g2 = ssm.causal_conv1d_silu_bwd(x[s], w, du[s], bias=b, **{k: v[s] for k, v in kw.items()})
        for k in ("dx",) + (("dstate",) if state else ()):
            assert torch.equal(g[k][s], g2[k]), k
    # dx holds w[2] g here and the state's gradient; dbias is the sum of g: a
    # term passes at most B / 16 + 16 additions
    if not state:
        terms = (g["dx"] / 2.0).double()
        off = abs(float(g["dbias"].double() - terms.sum()))
        assert off <= (B / 16 + 17) * 2.0 ** -24 * float(terms.abs().sum())


def test_states_of_more_items_than_one_launch_takes():
    """The carried state's gradient without tokens: 2^32 channels, copied."""
    B, D, K = (1 << 25) + 1, 128, 2
    assert B * D > 1 << 32
    st = randn(B, D, K - 1)
    x = torch.empty(B, 0, D, device="cuda")
    g = ssm.causal_conv1d_silu_bwd(x, torch.ones(D, K, device="cuda"), x, state=st, dstate_out=st)
    assert torch.equal(g["dstate"], st) and not g["dweight"].any()


@pytest.mark.parametrize("B,L,D,direction", [(1, 2048, 19200, "fwd"), (3, 1100, 6400, "fwd"), (1, 2048, 19200, "bwd"),
                                             (2, 1000, 11500, "bwd")])
def test_more_walkers_than_the_gpu_runs_at_once(B, L, D, direction, monkeypatch):
    """Sizes at which the planner itself lets several workgroups walk a strip
    and asks for more of them than there are CUs (one runs on a CU at a time),
    against one workgroup to a strip, bit for bit."""
    monkeypatch.delenv("SSM_GATED_WALKERS", raising=False)
    query = ssm.gated_scan_walkers if direction == "fwd" else ssm.gated_scan_bwd_walkers
    w = query(B, L, D)
    assert w > 1 and w * B * -(-D // 64) > 256
    x, ga, gx, dy = (randn(B, L, D, dtype=BF, seed=k) for k in range(4))
    A, ba, bx = -torch.rand(D, device="cuda") - 0.001, randn(D, seed=5), randn(D, seed=6)
    h0, dh = randn(B, D, seed=7), randn(B, D, seed=8)
    lens = torch.tensor([L, L - 300, 7][:B], dtype=torch.int32, device="cuda")

    def run():
        y, h, ck = ssm.gated_scan_fwd_ckpt(x, ga, gx, A, ba, bx, h0, seq_lens=lens, out=torch.zeros_like(x),
                                           ckpt=torch.zeros(B, -(-L // 128), D, device="cuda"))
        r = {"y": y, "h": h, "ck": ck}
        if direction == "bwd":
            r.update(ssm.gated_scan_bwd(x, ga, gx, A, dy, ba, bx, h0, dh, ckpt=ck, seq_lens=lens))
            r.update({"own " + k: v for k, v in
                      ssm.gated_scan_bwd(x, ga, gx, A, dy, ba, bx, h0, dh, seq_lens=lens).items()})
        return r

    got = run()
    monkeypatch.setenv("SSM_GATED_WALKERS", "1")
    want = run()
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_backward_offsets_past_32_bits():
    """Gradients of tensors of more than 2^31 elements: the first and the last
    rows against calls over those rows alone, which meet in the state and its
    gradient, bit for bit."""
    L, D = 70000, 32768
    x = randn(1, L, D, dtype=BF, seed=1)
    A = -torch.rand(D, device="cuda") - 0.01
    cut = 128 * 546                                # a border of saved states
    _, _, ck = ssm.gated_scan_fwd_ckpt(x, x, x, A)
    g = ssm.gated_scan_bwd(x, x, x, A, x, ckpt=ck)
    tail = x[:, cut:].contiguous()
    first = ck[:, 546].contiguous()
    g2 = ssm.gated_scan_bwd(tail, tail, tail, A, tail, h0=first)
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.equal(g[k][:, cut:], g2[k]), k
    head = x[:, :cut]
    g1 = ssm.gated_scan_bwd(head, head, head, A, head, dh_last=g2["dh0"], ckpt=ck[:, :546])
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.equal(g[k][:, :cut], g1[k]), k


def test_conv_offsets_past_32_bits():
    L, D, K = 70000, 32768, 4
    x = randn(1, L, D, dtype=BF, seed=1)
    w, b = randn(D, K, seed=2) * 0.5, randn(D, seed=3)
    dso = randn(1, D, K - 1, seed=4)
    g = ssm.causal_conv1d_silu_bwd(x, w, x, bias=b, dstate_out=dso)
    cut = 256 * 273                                # a border of the workgroups' blocks
    tail = x[:, cut:].contiguous()
    state = x[:, cut - (K - 1):cut].float().transpose(1, 2).contiguous()
    g2 = ssm.causal_conv1d_silu_bwd(tail, w, tail, bias=b, state=state, dstate_out=dso)
    assert torch.equal(g["dx"][:, cut:], g2["dx"])


@pytest.mark.parametrize("residual", [False, True])
def test_norm_offsets_past_32_bits(residual):
    rows, D = (1 << 21) + 37, 1024
    x, dy = randn(rows, D, dtype=BF, seed=1), randn(rows, D, dtype=BF, seed=2)
    w, b = randn(D, seed=3), randn(D, seed=4)
    last = slice(rows - 1000, rows)

    def run(x, dy, res, dres):
        n = ssm.layer_norm_fwd(x, w, b, residual=res)
        g = ssm.layer_norm_bwd(n.get("residual_out", x), dy, n["mean"], n["rstd"], weight=w, bias=b,
                               dresidual_out=dres, return_dresidual=residual)
        return {**n, **g}

    res, dres = (randn(rows, D, seed=5), randn(rows, D, seed=6)) if residual else (None, None)
    got = run(x, dy, res, dres)
    cut = lambda t: None if t is None else t[last].clone()                    # noqa: E731
    want = run(cut(x), cut(dy), cut(res), cut(dres))
    for k in want:
        if k not in ("dweight", "dbias"):
            assert torch.equal(got[k][last], want[k]), k


# each thread layout of the backward, by the row's length, with more rows than
# its 256 workgroups take in one round: 1024 / (threads to a row) rows each
ROUNDS = [(F, 8, 33000), (F, 64, 33000), (F, 200, 20000), (F, 500, 9000), (F, 1030, 5000), (F, 2052, 2100),
          (F, 4104, 1100), (F, 8200, 600), (F, 20001, 300), (BF, 8, 70000), (BF, 100, 40000), (BF, 250, 20000),
          (BF, 768, 9000), (BF, 1030, 4200), (BF, 2052, 2100), (BF, 4104, 1100), (BF, 8200, 600), (BF, 20001, 300)]


@pytest.mark.parametrize("dtype,D,rows", ROUNDS)
def test_norm_backward_over_several_rounds_of_rows(dtype, D, rows):
    gen = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=gen)                             # noqa: E731
    x, dy, w, b = (r(rows, D) * 2 + 0.3).to(dtype), r(rows, D).to(dtype), 1 + 0.2 * r(D), 0.3 * r(D)
    for res in (None, r(rows, D) * 3):
        up = lambda t: None if t is None else t.cuda()                        # noqa: E731
        n = ssm.layer_norm_fwd(up(x), up(w), up(b), residual=up(res))
        g = ssm.layer_norm_bwd(n.get("residual_out", up(x)), up(dy), n["mean"], n["rstd"], weight=up(w), bias=up(b))
        ref = O.layer_norm_bwd(x, dy, w, b, res)
        err = Bd.norm_bwd(Bd.norm(x, w, b, res)[1], dy)
        for k, v in ref.items():
            Bd.check(g[k], v, err[k], k)
