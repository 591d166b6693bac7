"""Refusals of the calls around the scan, on the host: the C ABI rejects bad
arguments before any HIP call, and the Python wrappers raise before anything
reaches the library (only invalid calls are made here; nothing is launched)."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from selective_state_space_21_amd import _native

FAKE = 0x10000          # never dereferenced: validation fails before any use
MIS = 0x10002
ODD = 0x10001
HUGE = 1 << 61


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def fwd(lib, **kw):
    a = dict(x=FAKE, ga=FAKE, gx=FAKE, A=FAKE, ba=None, bx=None, h0=None, y=FAKE, h=None, ck=None,
             lens=None, B=2, L=300, D=128, dt=1, ws=FAKE, n=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.ssm_gated_scan_fwd(*list(a.values()), None)


def bwd(lib, **kw):
    a = dict(x=FAKE, ga=FAKE, gx=FAKE, A=FAKE, ba=None, bx=None, h0=None, ck=None, dy=FAKE, dh=None,
             dx=FAKE, dga=FAKE, dgx=FAKE, dA=FAKE, dba=None, dbx=None, dh0=None, lens=None, B=2,
             L=300, D=128, dt=1, ws=FAKE, n=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.ssm_gated_scan_bwd(*list(a.values()), None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_gated_refusals(lib, call):
    for name in ("x", "ga", "gx", "A"):
        assert call(lib, **{name: None}) == 1
    assert call(lib, B=0) == 2 and call(lib, D=0) == 2 and call(lib, L=-1) == 2 and call(lib, D=-7) == 2
    assert call(lib, B=1 << 40, L=1 << 20, D=1 << 20) == 2
    assert call(lib, L=HUGE) == 2 and call(lib, D=HUGE) == 2 and call(lib, B=HUGE) == 2
    assert call(lib, dt=2) == 3 and call(lib, dt=-1) == 3
    assert call(lib, B=1 << 26, L=1, D=1) == 4                    # strips
    assert call(lib, B=1, L=1 << 40, D=1) == 4                    # tiles
    assert call(lib, B=1, L=1, D=(1 << 20) + 1) == 4              # a tile's rows
    for name in ("x", "ga", "gx", "ck"):
        assert call(lib, **{name: MIS}) == 5
    for name in ("A", "ba", "bx", "h0", "lens"):
        assert call(lib, **{name: MIS}) == 5


def test_gated_output_refusals(lib):
    assert fwd(lib, y=None) == 1 and fwd(lib, y=MIS) == 5 and fwd(lib, h=ODD) == 5
    for name in ("dy", "dx", "dga", "dgx", "dA"):
        assert bwd(lib, **{name: None}) == 1
        assert bwd(lib, **{name: MIS}) == 5
    for name in ("dh", "dba", "dbx", "dh0"):
        assert bwd(lib, **{name: ODD}) == 5


def test_gated_workspace_refusals(lib):
    for ck in (None, FAKE):
        need = lib.ssm_gated_scan_bwd_workspace_bytes(2, 300, 128, 1, int(ck is not None))
        assert need > 0
        assert bwd(lib, ck=ck, ws=None) == 6 and bwd(lib, ck=ck, n=need - 1) == 6
        assert bwd(lib, ck=ck, ws=FAKE + 128) == 5
    full = lib.ssm_gated_scan_bwd_workspace_bytes(2, 300, 128, 1, 0)
    assert full >= need + lib.ssm_gated_scan_ckpt_bytes(2, 300, 128, 1)
    assert lib.ssm_gated_scan_ckpt_bytes(2, 300, 128, 1) == 2 * 3 * 128 * 4
    assert lib.ssm_gated_scan_ckpt_bytes(2, 0, 128, 1) == 0
    for bad in ((0, 5, 5, 1), (5, -1, 5, 1), (1, 1, 1, 9), (HUGE, HUGE, HUGE, 0)):
        assert lib.ssm_gated_scan_workspace_bytes(*bad) == 0
        assert lib.ssm_gated_scan_bwd_workspace_bytes(*bad, 0) == 0
        assert lib.ssm_gated_scan_ckpt_bytes(*bad) == 0
    assert lib.ssm_gated_scan_walkers(0, 5, 5) == 0 and lib.ssm_gated_scan_walkers(1, HUGE, HUGE) == 0


def test_step_refusals(lib):
    def step(**kw):
        a = dict(state=FAKE, x=FAKE, ga=FAKE, gx=FAKE, A=FAKE, ba=None, bx=None, y=FAKE, B=2, D=8, dt=0)
        a.update(kw)
        return lib.ssm_gated_state_update(*list(a.values()), None)
    for name in ("state", "x", "ga", "gx", "A", "y"):
        assert step(**{name: None}) == 1 and step(**{name: MIS}) == 5
    assert step(ba=ODD) == 5 and step(bx=ODD) == 5
    assert step(B=0) == 2 and step(D=-1) == 2 and step(B=1 << 40, D=1 << 40) == 2
    assert step(B=1 << 30, D=1 << 20) == 4 and step(dt=5) == 3


def test_norm_refusals(lib):
    def f(**kw):
        a = dict(x=FAKE, res=None, w=None, b=None, eps=1e-5, y=FAKE, ro=None, m=None, r=None, rows=4, D=8, dt=1)
        a.update(kw)
        return lib.ssm_layer_norm_fwd(*list(a.values()), None)

    def g(**kw):
        a = dict(x=FAKE, xdt=1, dy=FAKE, m=FAKE, r=FAKE, w=None, dro=None, dx=FAKE, dr=None, dw=None,
                 db=None, rows=4, D=8, dt=1, ws=FAKE, n=1 << 40)
        a.update(kw)
        return lib.ssm_layer_norm_bwd(*list(a.values()), None)
    for call in (f, g):
        assert call(x=None) == 1 and call(x=MIS) == 5
        assert call(rows=-1) == 2 and call(D=0) == 2 and call(D=HUGE, rows=1) == 2
        assert call(rows=1 << 31) == 4 and call(dt=2) == 3
    assert f(y=None) == 1 and f(ro=FAKE) == 1                     # residual_out without residual
    for eps in (-1e-9, float("nan"), float("inf")):
        assert f(eps=eps) == 4
    for name in ("res", "w", "b", "m", "r"):
        assert f(**{name: MIS}) == 5
    for name in ("dy", "m", "r", "dx"):
        assert g(**{name: None}) == 1 and g(**{name: MIS}) == 5
    for name in ("w", "dro", "dr", "dw", "db"):
        assert g(**{name: MIS}) == 5
    assert g(xdt=3) == 3 and g(xdt=1, dt=0) == 4
    need = lib.ssm_layer_norm_bwd_workspace_bytes(4, 8)
    assert need > 0 and g(ws=None) == 6 and g(n=need - 1) == 6 and g(ws=FAKE + 64) == 5
    assert lib.ssm_layer_norm_bwd_workspace_bytes(-1, 8) == 0


def test_conv_bwd_refusals(lib):
    def g(**kw):
        a = dict(x=FAKE, w=FAKE, b=None, st=None, silu=1, du=FAKE, dso=None, dx=FAKE, dw=FAKE, db=None,
                 ds=None, B=2, L=9, D=8, K=4, dt=1, ws=FAKE, n=1 << 40)
        a.update(kw)
        return lib.ssm_causal_conv1d_silu_bwd(*list(a.values()), None)
    for name in ("x", "w", "du", "dx", "dw"):
        assert g(**{name: None}) == 1 and g(**{name: MIS}) == 5
    for name in ("b", "st", "dso", "db", "ds"):
        assert g(**{name: MIS}) == 5
    assert g(K=0) == 2 and g(K=5) == 4 and g(B=0) == 2 and g(L=-1) == 2 and g(L=HUGE) == 2 and g(dt=4) == 3
    assert g(B=1 << 20, L=1 << 20, D=1 << 10) == 4 and g(D=(1 << 21) + 1) == 4
    need = lib.ssm_causal_conv1d_silu_bwd_workspace_bytes(2, 9, 8, 4)
    assert need > 0 and g(ws=None) == 6 and g(n=need - 1) == 6 and g(ws=FAKE + 64) == 5


# ---- the wrappers: everything here is on the CPU, so a call that passes every
# other check is refused for its device

def _scan(**kw):
    t = dict(x=torch.zeros(2, 5, 8), gate_a=torch.zeros(2, 5, 8), gate_x=torch.zeros(2, 5, 8),
             A=-torch.ones(8), bias_a=torch.zeros(8), bias_x=torch.zeros(8), h0=torch.zeros(2, 8))
    t.update(kw)
    return t


BAD_SCAN = [
    (dict(x=torch.zeros(2, 8)), ValueError), (dict(x=torch.zeros(2, 5, 8).half()), TypeError),
    (dict(x=[1.0]), TypeError), (dict(x=torch.zeros(2, 5, 8, dtype=torch.float64)), TypeError),
    (dict(gate_a=torch.zeros(2, 5, 7)), ValueError), (dict(gate_x=torch.zeros(2, 5, 8).bfloat16()), TypeError),
    (dict(gate_a=None), TypeError), (dict(A=None), TypeError), (dict(A=torch.zeros(8, 1)), ValueError),
    (dict(A=torch.zeros(8).bfloat16()), TypeError), (dict(bias_a=torch.zeros(7)), ValueError),
    (dict(bias_x=torch.zeros(8).bfloat16()), TypeError), (dict(h0=torch.zeros(8)), ValueError),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError), (dict(), ValueError),
]


@pytest.mark.parametrize("kw,err", BAD_SCAN)
def test_gated_wrapper_refusals(kw, err):
    with pytest.raises(err):
        ssm.gated_scan_fwd(**_scan(**kw))
    with pytest.raises(err):
        ssm.gated_scan_fwd_ckpt(**_scan(**kw))
    with pytest.raises(err):
        ssm.gated_scan_bwd(dy=torch.zeros(2, 5, 8), **_scan(**kw))


@pytest.mark.parametrize("kw", [dict(out=torch.zeros(2, 5, 9)), dict(out=torch.zeros(2, 5, 8).bfloat16())])
def test_gated_wrapper_output_refusals(kw):
    with pytest.raises((TypeError, ValueError)):
        ssm.gated_scan_fwd(**_scan(), **kw)
    with pytest.raises(ValueError, match="ckpt"):
        ssm.gated_scan_fwd_ckpt(**_scan(), ckpt=torch.zeros(2, 2, 8))
    with pytest.raises(ValueError, match="dy"):
        ssm.gated_scan_bwd(dy=torch.zeros(2, 4, 8), **_scan())
    with pytest.raises(TypeError):
        ssm.gated_scan_bwd(dy=None, **_scan())
    with pytest.raises(ValueError, match="dh_last"):
        ssm.gated_scan_bwd(dy=torch.zeros(2, 5, 8), dh_last=torch.zeros(2, 9), **_scan())


def test_other_wrapper_refusals():
    z = torch.zeros
    with pytest.raises(ValueError):
        ssm.gated_state_update(z(2, 8), z(2, 8), z(2, 8), z(2, 8), -torch.ones(8))
    with pytest.raises(TypeError):
        ssm.gated_state_update(z(2, 8).bfloat16(), z(2, 8), z(2, 8), z(2, 8), -torch.ones(8))
    with pytest.raises(TypeError):
        ssm.gated_state_update(None, z(2, 8), z(2, 8), z(2, 8), -torch.ones(8))
    with pytest.raises(ValueError):
        ssm.gated_state_update(z(2, 8), z(2, 1, 8), z(2, 8), z(2, 8), -torch.ones(8))
    for bad in (dict(weight=z(7)), dict(bias=z(8, 1)), dict(residual=z(8)), dict(residual_out=z(3, 8)), {}):
        with pytest.raises(ValueError):
            ssm.layer_norm_fwd(z(3, 8), **bad)
    with pytest.raises(TypeError):
        ssm.layer_norm_fwd(z(3, 8), residual=z(3, 8).bfloat16())
    with pytest.raises(TypeError):
        ssm.layer_norm_bwd(z(3, 8).bfloat16(), z(3, 8), z(3), z(3))
    with pytest.raises(ValueError):
        ssm.layer_norm_bwd(z(3, 8), z(3, 8), z(3, 1), z(3))
    with pytest.raises(TypeError):
        ssm.layer_norm_bwd(z(3, 8), z(3, 8), None, z(3))
    for bad in (dict(weight=z(8)), dict(weight=z(7, 4)), dict(du=z(2, 5, 7)), dict(state=z(2, 8, 4)), {}):
        t = dict(x=z(2, 5, 8), weight=z(8, 4), du=z(2, 5, 8))
        t.update(bad)
        with pytest.raises(ValueError):
            ssm.causal_conv1d_silu_bwd(**t)
    with pytest.raises(TypeError):
        ssm.causal_conv1d_silu_bwd(z(2, 5, 8), z(8, 4), None)


def test_every_new_name_is_public():
    for name in ("gated_scan_fwd", "gated_scan_fwd_ckpt", "gated_scan_bwd", "gated_state_update",
                 "layer_norm_fwd", "layer_norm_bwd", "causal_conv1d_silu_bwd"):
        assert name in ssm.__all__ and callable(getattr(ssm, name))
