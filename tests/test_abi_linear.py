"""Refusals of linear attention, the head norm with rotary positions and the
moves between slots, on the host: the C ABI rejects bad arguments before any
HIP call, and the Python wrappers raise before anything reaches the library
(only invalid calls are made here; nothing is launched)."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from selective_state_space_21_amd import _native, linear_attention

FAKE = 0x10000          # never dereferenced: validation fails before any use
MIS = 0x10002
ODD = 0x10001
HUGE = 1 << 61


@pytest.fixture(scope="module")
def lib():
    return _native.load()


SIZES = dict(q_row=256, k_row=256, v_row=512, B=2, L=300, H=4, G=2, Dk=128, Dv=128, dt=1)


def fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, by=0, scale=1.0, h0=None, o=FAKE, h=None, lens=None, **SIZES, ws=FAKE,
             n=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.ssm_linear_attention_fwd(*list(a.values()), None)


def bwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, by=0, scale=1.0, h0=None, do=FAKE, dh=None, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE,
             dh0=None, lens=None, **SIZES, ws=FAKE, n=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.ssm_linear_attention_bwd(*list(a.values()), None)


def step(lib, **kw):
    a = dict(state=FAKE, q=FAKE, k=FAKE, v=FAKE, g=FAKE, by=0, scale=1.0, slots=None, o=FAKE, q_row=256, k_row=256, v_row=512,
             B=2, n_slots=2, H=4, G=2, Dk=128, Dv=128, dt=1)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.ssm_linear_state_update(*list(a.values()), None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_sizes_and_pointers(lib, call):
    for name in ("q", "k", "v", "g"):
        assert call(lib, **{name: None}) == 1
    for name in ("B", "H", "G", "Dk", "Dv"):
        assert call(lib, **{name: 0}) == 2 and call(lib, **{name: -16}) == 2 and call(lib, **{name: HUGE}) in (2, 4)
    assert call(lib, G=3) == 2 and call(lib, G=8) == 2            # heads do not share them evenly
    assert call(lib, dt=2) == 3 and call(lib, dt=-1) == 3
    for name in ("Dk", "Dv"):
        for n in (8, 24, 100, 272, 512):
            assert call(lib, **{name: n}) in (2, 4)
    assert call(lib, Dk=24) == 4 and call(lib, Dv=272) == 4
    assert call(lib, B=1 << 22) == 4
    for name in ("q_row", "k_row", "v_row"):
        assert call(lib, **{name: 255}) == 2                      # tokens overlap
        assert call(lib, **{name: 513}) == 2 and call(lib, **{name: 516}) == 2     # not 16 bytes
        assert call(lib, **{name: (1 << 22) + 8}) == 2
    assert call(lib, q_row=516, dt=0) != 2 or call(lib, q_row=516, dt=0, q=None) == 1
    assert call(lib, scale=float("nan")) == 4 and call(lib, scale=float("inf")) == 4
    for name in ("q", "k", "v"):
        assert call(lib, **{name: MIS}) == 5
    assert call(lib, g=ODD) == 5


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_heads_of_one_launch(lib, call):
    """Four column tiles of 512 threads a head stay below 2^32 work-items: past 2^20 heads the call is refused."""
    more = {"slots": FAKE} if call is step else {"L": 1}
    assert call(lib, B=1 << 18, H=4, q=None, **more) == 1
    assert call(lib, B=(1 << 18) + 1, H=4, q=None, **more) == 4


def test_outputs(lib):
    assert fwd(lib, o=None) == 1 and fwd(lib, o=MIS) == 5
    for name in ("h0", "h", "lens"):
        assert fwd(lib, **{name: ODD}) == 5
    for name in ("do", "dq", "dk", "dv"):
        assert bwd(lib, **{name: None}) == 1 and bwd(lib, **{name: MIS}) == 5
    for name in ("h0", "dh", "dg", "dh0", "lens"):
        assert bwd(lib, **{name: ODD}) == 5
    assert fwd(lib, L=-1) == 2 and bwd(lib, L=-1) == 2 and fwd(lib, L=(1 << 30) + 1) == 4 and fwd(lib, L=HUGE) == 2
    assert step(lib, o=None) == 1 and step(lib, state=None) == 1 and step(lib, state=MIS) == 5 and step(lib, o=MIS) == 5
    assert step(lib, slots=ODD) == 5 and step(lib, n_slots=0) == 2 and step(lib, n_slots=1) == 2
    assert step(lib, n_slots=1 << 31, slots=FAKE) == 4


def test_workspaces(lib):
    need = lib.ssm_linear_attention_workspace_bytes(1, 8192, 4, 128, 128, 1)
    assert need > 0
    more = dict(B=1, L=8192)
    assert fwd(lib, ws=None, **more) == 6 and fwd(lib, n=need - 1, **more) == 6 and fwd(lib, ws=FAKE + 16, n=need, **more) == 5
    need = lib.ssm_linear_attention_bwd_workspace_bytes(2, 300, 4, 2, 128, 128, 0, 1)
    assert bwd(lib, ws=None) == 6 and bwd(lib, n=need - 1) == 6 and bwd(lib, ws=FAKE + 128, n=need) == 5
    shared = lib.ssm_linear_attention_bwd_workspace_bytes(2, 300, 4, 4, 128, 128, 0, 1)
    assert need - shared == 2 * 2 * 300 * 4 * 128 * 4             # the heads' gradients of shared keys
    assert lib.ssm_linear_attention_workspace_bytes(1, 100, 2, 24, 64, 1) == 0
    assert lib.ssm_linear_attention_bwd_workspace_bytes(1, 100, 2, 3, 64, 64, 0, 1) == 0


def test_segments(lib, monkeypatch):
    monkeypatch.delenv("SSM_LINEAR_SEGMENTS", raising=False)
    seg = lib.ssm_linear_attention_segments
    assert seg(1, 0, 1, 64, 64, 1) == 1 and seg(1, 64, 1, 64, 64, 1) == 1 and seg(0, 64, 1, 64, 64, 1) == 0
    assert seg(64, 2048, 16, 64, 64, 1) == 1                      # the GPU is full
    for L in (1000, 5000, 70000, 1 << 30):
        n = seg(1, L, 2, 64, 64, 1)
        assert 1 < n <= 256
        assert lib.ssm_linear_attention_workspace_bytes(1, L, 2, 64, 64, 1) >= n * 2 * 64 * 64 * 4
    monkeypatch.setenv("SSM_LINEAR_SEGMENTS", "7")
    assert seg(4, 7000, 2, 64, 64, 1) == 7 and seg(4, 100, 2, 64, 64, 1) == 2
    monkeypatch.setenv("SSM_LINEAR_SEGMENTS", "1000")
    assert seg(64, 2048, 16, 64, 64, 1) == 1


def norm(lib, bwd=False, **kw):
    a = dict(q=FAKE, k=FAKE)
    if bwd:
        a |= dict(dyq=FAKE, dyk=FAKE)
    a |= dict(wq=FAKE, wk=FAKE, pos=FAKE, freq=FAKE, inter=0, eps=1e-6, oq=FAKE, ok=FAKE)
    if bwd:
        a |= dict(dwq=FAKE, dwk=FAKE)
    a |= dict(q_row=512, k_row=256, rows=5, Hq=4, Hk=2, width=128, rotary=64, dt=1)
    if bwd:
        a |= dict(ws=FAKE, n=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return (lib.ssm_qk_norm_rope_bwd if bwd else lib.ssm_qk_norm_rope_fwd)(*list(a.values()), None)


@pytest.mark.parametrize("bwd", [False, True])
def test_head_norm(lib, bwd):
    for name in ("q", "k", "oq", "ok", "pos", "freq"):
        assert norm(lib, bwd, **{name: None}) == 1
    for name in ("rows", "Hq", "Hk", "rotary"):
        assert norm(lib, bwd, **{name: -2}) == 2
    assert norm(lib, bwd, width=0) == 2 and norm(lib, bwd, rotary=130) == 2 and norm(lib, bwd, rotary=63) == 2
    assert norm(lib, bwd, q_row=511) == 2 and norm(lib, bwd, k_row=0) == 2 and norm(lib, bwd, rows=HUGE) == 2
    assert norm(lib, bwd, dt=5) == 3
    assert norm(lib, bwd, width=127) == 4 and norm(lib, bwd, width=514, q_row=4096, k_row=4096) == 4
    assert norm(lib, bwd, rows=(1 << 24) + 1) == 4 and norm(lib, bwd, Hq=65537, q_row=1 << 24) == 4
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(lib, bwd, eps=eps) == 4
    for name in ("oq", "ok"):
        assert norm(lib, bwd, **{name: MIS}) == 5
    for name in ("q", "k", "wq", "wk", "pos", "freq"):
        assert norm(lib, bwd, **{name: ODD}) == 5
    assert norm(lib, bwd, q=MIS, dt=0) == 5
    if bwd:
        need = lib.ssm_qk_norm_rope_bwd_workspace_bytes(5, 128)
        assert norm(lib, True, ws=None) == 6 and norm(lib, True, n=need - 1) == 6 and norm(lib, True, ws=FAKE + 8) == 5
        assert norm(lib, True, dyq=None) == 1 and norm(lib, True, dyk=MIS) == 5 and norm(lib, True, dwq=MIS) == 5
        assert lib.ssm_qk_norm_rope_bwd_workspace_bytes(-1, 128) == 0


def slots(lib, **kw):
    a = dict(pool=FAKE, src=FAKE, dst=FAKE, layers=2, n_slots=8, size=4096, n=3)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.ssm_state_slots_copy(*list(a.values()), None)


def test_slots(lib):
    for name in ("pool", "src", "dst"):
        assert slots(lib, **{name: None}) == 1
    for name in ("layers", "size", "n"):
        assert slots(lib, **{name: -1}) == 2 and slots(lib, **{name: 0}) == 0     # nothing to do
    assert slots(lib, n_slots=0) == 2 and slots(lib, size=HUGE) == 2 and slots(lib, layers=1 << 40, size=1 << 30) == 2
    assert slots(lib, n=2049) == 4 and slots(lib, n_slots=1 << 31) == 4 and slots(lib, layers=1 << 26, size=1 << 20, n_slots=1) == 4
    assert slots(lib, src=MIS) == 5 and slots(lib, dst=ODD) == 5


# ---- the wrappers: CPU tensors never reach the library

def cpu(**kw):
    a = dict(q=torch.zeros(2, 5, 2, 16), k=torch.zeros(2, 5, 2, 16), v=torch.zeros(2, 5, 4, 32), log_decay=torch.zeros(2, 5, 4))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw, err", [
    (dict(), ValueError), (dict(q=None), TypeError), (dict(k=None), TypeError), (dict(v=None), TypeError),
    (dict(log_decay=None), TypeError), (dict(q=torch.zeros(2, 5, 32)), ValueError), (dict(v=torch.zeros(2, 6, 4, 32)), ValueError),
    (dict(q=torch.zeros(2, 5, 3, 16)), ValueError), (dict(k=torch.zeros(2, 5, 2, 32)), ValueError),
    (dict(k=torch.zeros(2, 5, 2, 16, dtype=torch.bfloat16)), TypeError), (dict(q=torch.zeros(2, 5, 2, 16).half()), TypeError),
])
def test_attention_wrappers(kw, err):
    a = cpu(**kw)
    with pytest.raises(err):
        ssm.linear_attention_fwd(**a)
    with pytest.raises(err):
        ssm.linear_attention_bwd(**a, do=torch.zeros(2, 5, 4, 32))
    if all(x is None or (isinstance(x, torch.Tensor) and x.dim() >= 3) for x in a.values()):
        b = {n: None if x is None else x[:, 0] for n, x in a.items()}
        with pytest.raises((err, ValueError)):
            ssm.linear_state_update(torch.zeros(2, 4, 16, 32), **b)


def test_other_wrappers():
    z = torch.zeros(5, 2, 16)
    for kw, err in ((dict(), ValueError), (dict(k=None), TypeError), (dict(k=[z]), TypeError), (dict(q=torch.zeros(5, 2, 16).half()), TypeError),
                    (dict(k=torch.zeros(4, 2, 16)), ValueError), (dict(k=torch.zeros(5, 16)), ValueError),
                    (dict(inv_freq=torch.zeros(8)), (TypeError, ValueError))):
        with pytest.raises(err):
            ssm.qk_norm_rope_fwd(**{**dict(q=z, k=z), **kw})
        with pytest.raises(err):
            ssm.qk_norm_rope_bwd(**{**dict(q=z, k=z, dq_out=z, dk_out=z), **kw})
    i = torch.zeros(3, dtype=torch.int32)
    for a, err in (((torch.zeros(4, 8), i, i), ValueError), ((None, i, i), TypeError), ((torch.zeros(4, 8), i, None), TypeError),
                   ((torch.zeros(4, 8), i, i[:2]), ValueError), ((torch.zeros(4, 8), i.long(), i.long()), TypeError),
                   ((torch.zeros(0, 8), i, i), ValueError)):
        with pytest.raises(err):
            ssm.state_slots_copy(*a)
    with pytest.raises(ValueError):
        ssm.state_slots_copy(torch.zeros(4, 8), i, i, dim=2)


def test_row_strides():
    """What counts as tokens a fixed stride apart (device aside)."""
    base = torch.zeros(2, 5, 100)
    dev = torch.device("meta")

    def rows(t, shape):
        class Device:                                             # stands for a device tensor
            pass
        d = Device()
        d.shape, d.dtype, d.is_cuda, d.device = t.shape, t.dtype, True, dev
        d.is_contiguous, d.stride = t.is_contiguous, t.stride
        return linear_attention._row("q", d, shape, dev)
    assert rows(torch.zeros(2, 5, 2, 16), (2, 5, 2, 16)) == 32
    assert rows(base[..., 4:36].unflatten(2, (2, 16)), (2, 5, 2, 16)) == 100
    assert rows(base[:, :1, :32].unflatten(2, (2, 16)), (2, 1, 2, 16)) == 500
    assert rows(base[:1, :1, :32].unflatten(2, (2, 16)), (1, 1, 2, 16)) == 32
    for bad in (base[..., :32].unflatten(2, (2, 16)).transpose(0, 1), base[..., :64:2].unflatten(2, (2, 16)),
                base[..., :64].unflatten(2, (2, 32))[..., :16], base[:, :4, :32].unflatten(2, (2, 16)),
                torch.zeros(1, 1, 2, 16).expand(2, 5, 2, 16)):
        with pytest.raises(ValueError):
            rows(bad, bad.shape)


def test_every_new_name_is_public():
    for n in linear_attention.__all__:
        assert n in ssm.__all__ and getattr(ssm, n).__doc__ or "workspace_bytes" in n, n
