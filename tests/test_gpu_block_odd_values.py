"""Values a caller does not expect in the calls around the scan: what is not a
number stays visible in the gradients, and what is infinite stays where it
belongs."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import block as O

import _block_bounds as Bd
from test_gpu_gated import dev, make

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def compare_nan(got, ref, err):
    """NaN exactly where the definition has it, the other elements within the
    bounds of the same call without the NaN (which they do not depend on)."""
    for k, r in ref.items():
        g = got[k].cpu()
        assert torch.equal(g.isnan(), r.isnan()), (k, int(g.isnan().sum()), int(r.isnan().sum()))
        zero = torch.zeros((), dtype=torch.float64)
        Bd.check(torch.where(g.isnan(), zero.to(g.dtype), g), torch.where(r.isnan(), zero, r), err[k], k)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("shape", [(1, 20, 64), (2, 60, 33), (1, 128, 66), (2, 700, 64), (1, 1500, 33)])
@pytest.mark.parametrize("which", ["gate_a", "gate_x", "bias_a", "bias_x"])
def test_nan_in_a_gate_is_nan_in_the_gradients(which, shape, dtype):
    B, L, D = shape
    t, dy, dh = make(B, L, D, dtype, seed=L)
    err = Bd.gated_bwd(Bd.gated(**t)[2], dy, dh)
    if which.startswith("gate"):
        t[which][0, L // 3, 5] = NAN
        t[which][B - 1, L - 2, D - 1] = NAN
    else:
        t[which][3] = NAN
    ref = O.gated_scan_bwd(t["x"], t["gate_a"], t["gate_x"], t["A"], dy, t["bias_a"], t["bias_x"],
                           t["h0"], dh)
    assert any(v.isnan().any() for v in ref.values())
    d = dev(t)
    _, _, ck = ssm.gated_scan_fwd_ckpt(**d)
    for c in (ck, None):
        compare_nan(ssm.gated_scan_bwd(**d, dy=dy.cuda(), dh_last=dh.cuda(), ckpt=c), ref, err)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("L", [20, 40, 128, 129, 700])
def test_a_positive_decay_rate_is_nan_in_the_gradients(L, dtype):
    """A > 0 has no weight sqrt(1 - a^2): NaN in the outputs, and in every
    gradient of those channels that the weight enters."""
    B, D = 2, 66
    t, dy, dh = make(B, L, D, dtype, seed=L)
    t["A"][7], t["A"][65] = 0.5, 1e-3
    d = dev(t)
    y, _, ck = ssm.gated_scan_fwd_ckpt(**d)
    for c in (ck, None):
        g = ssm.gated_scan_bwd(**d, dy=dy.cuda(), dh_last=dh.cuda(), ckpt=c)
        for k in ("dx", "dgate_a", "dgate_x", "dA", "dbias_a", "dbias_x"):
            bad = g[k].isnan()
            assert bad[..., 7].all() and bad[..., 65].all(), k
            assert int(bad.sum()) == bad.numel() // D * 2, k
    assert y[..., 7].isnan().all() and y[..., 65].isnan().all()


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("L,walkers", [(20, None), (50, None), (128, None), (200, None), (1500, "1"), (1500, "3")])
def test_rows_without_tokens_do_not_reach_the_gradients(L, walkers, dtype, value, monkeypatch):
    """An unused slot of a batch, whose carried state and whose state's
    gradient hold anything: zeros in its rows, nothing of it in the sums, and
    its state's gradient handed through."""
    if walkers:
        monkeypatch.setenv("SSM_GATED_WALKERS", walkers)
    B, D = 4, 66
    t, dy, dh = make(B, L, D, dtype, seed=L, lens=[0, L, 0, L - 3])
    clean = ssm.gated_scan_bwd(**dev(t), dy=dy.cuda(), dh_last=dh.cuda())
    t["h0"][0], dh[0] = value, value
    t["h0"][2, 5], dh[2, 9] = value, value
    d = dev(t)
    _, h, ck = ssm.gated_scan_fwd_ckpt(**d)
    same = lambda a, b: torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))      # noqa: E731
    assert same(h[[0, 2]], d["h0"][[0, 2]]) and torch.isfinite(h[[1, 3]]).all()
    for c in (ck, None):
        g = ssm.gated_scan_bwd(**d, dy=dy.cuda(), dh_last=dh.cuda(), ckpt=c)
        for k in ("dx", "dgate_a", "dgate_x"):
            assert not g[k][[0, 2]].any() and not g[k][3, L - 3:].any(), k
            assert torch.equal(g[k], clean[k]), k
        for k in ("dA", "dbias_a", "dbias_x"):
            assert torch.equal(g[k], clean[k]), k
        assert same(g["dh0"][[0, 2]].cpu(), dh[[0, 2]]) and torch.equal(g["dh0"][[1, 3]], clean["dh0"][[1, 3]])


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("L", [32, 64, 100, 300, 1500])
def test_padding_is_zero_under_an_infinite_adjoint(L, dtype):
    B, D = 3, 33
    n = [L - 1, 1, L // 2]
    t, dy, dh = make(B, L, D, dtype, seed=L, lens=n)
    dh[0], dh[1, 4], dh[2, 7] = INF, NAN, -INF
    t["h0"][1, 8] = INF
    d = dev(t)
    for c in (ssm.gated_scan_fwd_ckpt(**d)[2], None):
        g = ssm.gated_scan_bwd(**d, dy=dy.cuda(), dh_last=dh.cuda(), ckpt=c)
        for k in ("dx", "dgate_a", "dgate_x"):
            for b in range(B):
                assert not g[k][b, n[b]:].any(), (k, b)
            assert not torch.isfinite(g[k][0, n[0] - 1]).any()     # the row's own tokens show it


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("D", [1, 64])
def test_conv_gradient_of_huge_arguments(D, dtype):
    """The derivative of s sigma(s) is 0 far below zero and 1 far above (for
    s < -200 it is below |s| e^-200, nothing in fp32), however large s is."""
    low, high = [-200.0, -1e4, -1e20, -1e30, -1e35, -1e37, -1e38], [200.0, 1e20, 1e35, 1e38]
    x = torch.tensor(low + high).to(dtype)[None, :, None].repeat(2, 30, D).cuda()
    du = torch.full_like(x, 3.0)
    g = ssm.causal_conv1d_silu_bwd(x, torch.ones(D, 1, device="cuda"), du, bias=torch.zeros(D, device="cuda"))
    want = torch.tensor([0.0] * len(low) + [3.0] * len(high))[None, :, None].repeat(2, 30, D)
    assert torch.equal(g["dx"].float().cpu(), want)
    assert torch.equal(g["dbias"].cpu(), torch.full((D,), 2 * 30 * len(high) * 3.0))
    # and through the carried state's kernel: weights of the last inputs
    w = torch.tensor([1.0, 0.5]).repeat(D, 1).cuda()
    st = torch.full((1, D, 1), -1e38, device="cuda")
    g = ssm.causal_conv1d_silu_bwd(torch.zeros(1, 2, D, dtype=dtype, device="cuda"), w,
                                   torch.full((1, 2, D), 2.0, dtype=dtype, device="cuda"), state=st)
    assert not g["dstate"].any()
    # dx[0] = w[1] g[0] + w[0] g[1] with g[0] = 0, g[1] = 2 * sigma(0) = 1
    assert torch.equal(g["dx"].float().cpu()[0], torch.tensor([[1.0], [0.5]]).repeat(1, D))
    # what is not a number, or infinite, is not hidden
    x = torch.tensor([NAN, -INF, INF]).to(dtype)[None, :, None].repeat(1, 1, D).cuda()
    g = ssm.causal_conv1d_silu_bwd(x, torch.ones(D, 1, device="cuda"), torch.ones_like(x))
    assert not torch.isfinite(g["dx"]).any()


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("L", [1, 7, 8, 31, 32, 33, 300])
def test_conv_tokens_behind_the_end_do_not_count(L, dtype):
    """The last input times the first weight is an argument of a token that
    does not exist: beyond fp32 it must not reach the tokens that do."""
    for D in (64, 33):
        for K in (2, 3, 4):
            x = torch.zeros(1, L, D, dtype=dtype, device="cuda")
            x[:, -1] = 1e30
            w = torch.ones(D, K, device="cuda")
            w[:, 0] = 1e20
            g = ssm.causal_conv1d_silu_bwd(x, w, torch.full_like(x, 2.0), bias=torch.zeros(D, device="cuda"))
            # silu' is 1 at the last token and 1/2 at the others; what follows it counts nothing
            gs = torch.ones(L + K, dtype=torch.float64)
            gs[L - 1], gs[L:] = 2.0, 0.0
            want = sum(w[0, k].double().item() * gs[K - 1 - k:K - 1 - k + L] for k in range(K))
            half = torch.finfo(dtype).eps / 2
            off = (g["dx"].double().cpu() - want[None, :, None]).abs()
            assert (off <= (half + K * 2.0 ** -24) * want.abs()[None, :, None]).all(), (D, K)
            assert torch.equal(g["dbias"].cpu(), torch.full((D,), L + 1.0))


@pytest.mark.parametrize("L", [1, 3, 8, 9, 31, 32, 40, 257])
def test_conv_sums_do_not_take_inputs_of_tokens_behind_the_end(L):
    """Without SiLU an infinite last input meets only the last weight of the
    last token."""
    for D in (64, 33):
        for K in (2, 4):
            x, du = torch.ones(2, L, D, device="cuda"), torch.full((2, L, D), 2.0, device="cuda")
            x[:, -1] = 0.0
            w = torch.ones(D, K, device="cuda")
            want = ssm.causal_conv1d_silu_bwd(x, w, du, bias=w[:, 0].contiguous(), silu=False)
            x[0, -1], x[1, -1] = INF, NAN
            got = ssm.causal_conv1d_silu_bwd(x, w, du, bias=w[:, 0].contiguous(), silu=False)
            assert torch.equal(got["dweight"][:, :-1], want["dweight"][:, :-1]), (D, K)
            assert not torch.isfinite(got["dweight"][:, -1]).any()
            assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dbias"], want["dbias"])


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("L,walkers", [(20, None), (100, None), (256, None), (1500, "1"), (1500, "4")])
def test_rows_without_tokens_keep_their_state_whatever_the_parameters(L, walkers, dtype, monkeypatch):
    if walkers:
        monkeypatch.setenv("SSM_GATED_WALKERS", walkers)
    D = 66
    t, _, dh = make(3, L, D, dtype, seed=L, lens=[0, L, 0])
    t["bias_a"][3] = t["bias_x"][4] = NAN
    t["A"][5] = 0.5
    d = dev(t)
    y, h, ck = ssm.gated_scan_fwd_ckpt(**d, out=torch.full((3, L, D), 7.0, dtype=dtype, device="cuda"))
    assert torch.equal(h[[0, 2]], d["h0"][[0, 2]]) and torch.equal(ck[[0, 2], 0], d["h0"][[0, 2]])
    assert torch.all(y[[0, 2]] == 7.0)
    assert y[1, :, 3:6].isnan().all() and h[1, 3:6].isnan().all() and int(h.isnan().sum()) == 3
    g = ssm.gated_scan_bwd(**d, dy=torch.ones_like(y), dh_last=dh.cuda(), ckpt=ck)
    assert torch.equal(g["dh0"][[0, 2]].cpu(), dh[[0, 2]]) and not g["dx"][[0, 2]].any()
