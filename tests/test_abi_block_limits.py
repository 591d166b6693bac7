"""Sizes that the calls around the scan refuse because no launch can take them:
on the host, before any HIP call (only refused calls are made here)."""
import pytest

from selective_state_space_21_amd import _native

FAKE = 0x10000          # never dereferenced: validation fails before any use
U = 4                   # SSM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def test_step_rows_that_no_launch_takes(lib):
    def step(B, D):
        return lib.ssm_gated_state_update(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, B, D, 1, None)
    assert step(1, 1 << 33) == U and step(1, (1 << 32) + 1) == U and step(3, 1 << 40) == U


def test_walkers_asked_for_fit_a_launch(lib, monkeypatch):
    monkeypatch.setenv("SSM_GATED_WALKERS", "64")
    for B in (1, 1 << 16, 1 << 17, 1 << 20, 1 << 21, (1 << 22) + 1, (1 << 25) - 1):
        for query in (lib.ssm_gated_scan_walkers, lib.ssm_gated_scan_bwd_walkers):
            w = query(B, 100000, 64)
            assert 1 <= w <= 64 and (w == 1 or w * B * 1024 < 1 << 32), (B, w)
    assert lib.ssm_gated_scan_walkers(1, 100000, 64) == 64


def test_norm_backward_rows_that_no_launch_takes(lib):
    def g(rows, D):
        return lib.ssm_layer_norm_bwd(FAKE, 1, FAKE, FAKE, FAKE, None, None, FAKE, None, None, None, rows, D, 1,
                                      FAKE, 1 << 62, None)
    assert g(1, 1 << 32) == U and g(5, (1 << 32) - 255) == U
    assert lib.ssm_layer_norm_bwd_workspace_bytes(1, 1 << 32) == 0
    assert lib.ssm_layer_norm_bwd_workspace_bytes(1, (1 << 32) - 256) > 0


def test_conv_backward_rows_that_no_launch_takes(lib):
    def g(B, L, D):
        return lib.ssm_causal_conv1d_silu_bwd(FAKE, FAKE, None, None, 1, FAKE, None, FAKE, FAKE, None, None, B, L,
                                              D, 4, 1, FAKE, 1 << 62, None)
    assert g(1, 1 << 31, 1) == U and g(2, (1 << 31) - 255, 64) == U and g(1, 1 << 30, 65) == U
    assert lib.ssm_causal_conv1d_silu_bwd_workspace_bytes(1, 1 << 31, 1, 4) == 0
    assert lib.ssm_causal_conv1d_silu_bwd_workspace_bytes(1, (1 << 31) - 256, 1, 4) > 0
