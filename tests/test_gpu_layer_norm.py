"""Layer norm on the GPU against the fp64 oracle, element by element within
the bounds of _block_bounds."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import block as O

import _block_bounds as Bd

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def make(rows, D, dtype, seed=0, mean=0.3, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)                            # noqa: E731
    return dict(x=(r(rows, D) * scale + mean).to(dtype), w=1 + 0.2 * r(D), b=0.3 * r(D),
                res=r(rows, D) * 3, dy=r(rows, D).to(dtype), dres=r(rows, D))


SHAPES = [(1, 1), (3, 2), (1, 64), (5, 63), (7, 257), (2, 512), (6, 768), (4, 1000), (3, 1024),
          (2, 1537), (3, 2048), (5, 2561), (2, 4096), (3, 4104), (2, 5120), (2, 8192), (3, 8193),
          (2, 12296), (1, 16384), (2, 16385), (2, 40000), (700, 40), (2100, 8), (1030, 1024)]


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    rows, D = shape
    t = make(rows, D, dtype, seed=D)
    d = {k: v.cuda() for k, v in t.items()}
    for res, params in ((False, True), (True, True), (True, False)):
        w, b = (t["w"], t["b"]) if params else (None, None)
        r = t["res"] if res else None
        dw, db = (d["w"], d["b"]) if params else (None, None)
        got = ssm.layer_norm_fwd(d["x"], dw, db, residual=d["res"] if res else None)
        ref = dict(zip(("y", "mean", "rstd", "s"), O.layer_norm(t["x"], w, b, r)))
        err, keep = Bd.norm(t["x"], w, b, r)
        for k in ("y", "mean", "rstd"):
            Bd.check(got[k], ref[k], err[k], (k, res, params))
        assert ("residual_out" in got) == res
        if res:
            Bd.check(got["residual_out"], ref["s"], err["s"], "residual_out")
        dro = t["dres"] if res else None
        g = ssm.layer_norm_bwd(got.get("residual_out", d["x"]), d["dy"], got["mean"], got["rstd"],
                               weight=dw, bias=db, dresidual_out=d["dres"] if res else None,
                               return_dresidual=res)
        gr = O.layer_norm_bwd(t["x"], t["dy"], w, b, r, dro)
        eg = Bd.norm_bwd(keep, t["dy"], dro)
        for k, v in gr.items():
            Bd.check(g[k], v, eg[k], (k, res, params))
        if res:
            Bd.check(g["dresidual"], gr["dx"], eg["dx"], "dresidual")
            assert torch.equal(g["dresidual"].to(dtype), g["dx"])
        assert set(g) == set(gr) | ({"dresidual"} if res else set())


@pytest.mark.parametrize("D", [64, 100, 3000, 8200, 20001])
def test_far_from_zero_and_constant_rows(D):
    """Rows whose mean is far larger than their spread, and rows of one value
    (variance zero: y is the bias, the input's gradient finite)."""
    t = make(4, D, F, seed=1, mean=1000.0, scale=0.5)
    t["x"][1] = 3.0
    t["x"][2] = 0.0
    d = {k: v.cuda() for k, v in t.items()}
    got = ssm.layer_norm_fwd(d["x"], d["w"], d["b"])
    ref = dict(zip(("y", "mean", "rstd"), O.layer_norm(t["x"], t["w"], t["b"])))
    err, keep = Bd.norm(t["x"], t["w"], t["b"])
    for k in ref:
        Bd.check(got[k], ref[k], err[k], k)
    g = ssm.layer_norm_bwd(d["x"], d["dy"], got["mean"], got["rstd"], weight=d["w"], bias=d["b"])
    gr = O.layer_norm_bwd(t["x"], t["dy"], t["w"], t["b"])
    eg = Bd.norm_bwd(keep, t["dy"])
    for k in gr:
        Bd.check(g[k], gr[k], eg[k], k)


def test_shapes_eps_and_no_rows():
    x = torch.randn(2, 3, 5, 48, device="cuda")
    r = ssm.layer_norm_fwd(x, eps=0.5)
    assert r["y"].shape == x.shape and r["mean"].shape == (2, 3, 5)
    y, mean, rstd, _ = O.layer_norm(x.reshape(30, 48), eps=0.5)
    err, _ = Bd.norm(x.reshape(30, 48), eps=0.5)
    Bd.check(r["y"].reshape(30, 48), y, err["y"], "y")
    Bd.check(r["rstd"].reshape(30), rstd, err["rstd"], "rstd")
    assert "mean" not in ssm.layer_norm_fwd(x, return_stats=False)
    one = ssm.layer_norm_fwd(x[0, 0, 0])
    assert one["mean"].shape == ()
    e = torch.empty(0, 48, device="cuda")
    r = ssm.layer_norm_fwd(e)
    w = torch.ones(48, device="cuda")
    g = ssm.layer_norm_bwd(e, e, r["mean"], r["rstd"], weight=w, bias=w)
    assert g["dx"].shape == (0, 48) and not g["dweight"].any() and not g["dbias"].any()


def test_writes_stay_inside_and_repeat():
    rows, D, pad = 37, 776, 64
    t = {k: v.cuda() for k, v in make(rows, D, BF, seed=4).items()}
    n = rows * D
    gy = torch.full((n + 2 * pad,), 9.0, device="cuda", dtype=BF)
    gr = torch.full((n + 2 * pad,), 9.0, device="cuda")
    r = ssm.layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["res"], out=gy[pad:pad + n].view(rows, D),
                           residual_out=gr[pad:pad + n].view(rows, D))
    for g in (gy, gr):
        assert torch.all(g[:pad] == 9) and torch.all(g[pad + n:] == 9)
    need = ssm.layer_norm_bwd_workspace_bytes(rows, D)
    ws = torch.full((need + 512,), 3, dtype=torch.uint8, device="cuda")
    a = dict(x=r["residual_out"], dy=t["dy"], mean=r["mean"], rstd=r["rstd"], weight=t["w"], bias=t["b"])
    one = ssm.layer_norm_bwd(**a, workspace=ws[256:256 + need])
    assert torch.all(ws[:256] == 3) and torch.all(ws[256 + need:] == 3)
    two = ssm.layer_norm_bwd(**a)
    assert all(torch.equal(one[k], two[k]) for k in one)


def test_graph_replays():
    rows, D = 300, 768
    t = {k: v.cuda() for k, v in make(rows, D, BF, seed=4).items()}

    def both():
        r = ssm.layer_norm_fwd(t["x"], t["w"], t["b"], residual=t["res"])
        g = ssm.layer_norm_bwd(r["residual_out"], t["dy"], r["mean"], r["rstd"], weight=t["w"],
                               bias=t["b"], dresidual_out=t["dres"], return_dresidual=True)
        return {**r, **g}

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for k in range(3):
        t["x"].copy_(torch.randn(rows, D, generator=torch.Generator().manual_seed(k)))
        want = both()
        g.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), (k, n)
