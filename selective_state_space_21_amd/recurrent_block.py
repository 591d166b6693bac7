"""The calls around the scan in a recurrent block: the gated linear recurrence
(forward, training pair, decode step), layer norm with the fp32 residual
stream, and the backward of the causal conv1d + SiLU.

Python entry points of the C ABI in include/ssm.h, by the rules of the
package's other wrappers: they check every argument, allocate outputs and
workspace on the caller's stream, and marshal; the arithmetic runs in the
library's HIP kernels.
"""
from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch

from . import _args, _native

__all__ = ["gated_scan_fwd", "gated_scan_fwd_ckpt", "gated_scan_bwd", "gated_state_update",
           "gated_scan_walkers", "gated_scan_bwd_walkers", "gated_scan_workspace_bytes", "gated_scan_ckpt_bytes",
           "gated_scan_bwd_workspace_bytes", "layer_norm_fwd", "layer_norm_bwd",
           "layer_norm_bwd_workspace_bytes", "causal_conv1d_silu_bwd",
           "causal_conv1d_silu_bwd_workspace_bytes"]

_F32 = torch.float32
_DT = _args.DTYPES
_ptr = _args.ptr


_HERE = contextlib.nullcontext()


def _on(device):
    """The kernels are launched on the current device: make it the tensors'."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def gated_scan_walkers(B: int, L: int, D: int) -> int:
    """Workgroups that walk one strip of 64 channels together at these sizes."""
    return int(_native.load().ssm_gated_scan_walkers(B, L, D))


def gated_scan_bwd_walkers(B: int, L: int, D: int) -> int:
    """The same for the backward."""
    return int(_native.load().ssm_gated_scan_bwd_walkers(B, L, D))


def gated_scan_workspace_bytes(B: int, L: int, D: int, dtype=torch.bfloat16) -> int:
    return int(_native.load().ssm_gated_scan_workspace_bytes(B, L, D, _DT[dtype]))


def gated_scan_ckpt_bytes(B: int, L: int, D: int, dtype=torch.bfloat16) -> int:
    return int(_native.load().ssm_gated_scan_ckpt_bytes(B, L, D, _DT[dtype]))


def gated_scan_bwd_workspace_bytes(B: int, L: int, D: int, dtype=torch.bfloat16,
                                   with_ckpt: bool = False) -> int:
    return int(_native.load().ssm_gated_scan_bwd_workspace_bytes(B, L, D, _DT[dtype],
                                                                 int(bool(with_ckpt))))


def _gated_args(x, gate_a, gate_x, A, bias_a, bias_x, h0, seq_lens, *more):
    dt = _args.act_dtype("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [B, L, D]")
    Bt, L, Dm = x.shape
    dev = x.device
    _args.need(gate_a=gate_a, gate_x=gate_x, A=A)
    _args.check_args(dev, ("x", x, (Bt, L, Dm), dt), ("gate_a", gate_a, (Bt, L, Dm), dt),
                     ("gate_x", gate_x, (Bt, L, Dm), dt), ("A", A, (Dm,), _F32),
                     ("bias_a", bias_a, (Dm,), _F32), ("bias_x", bias_x, (Dm,), _F32),
                     ("h0", h0, (Bt, Dm), _F32), ("seq_lens", seq_lens, (Bt,), torch.int32), *more)
    return dt, dev, Bt, L, Dm


def _gated_fwd(x, gate_a, gate_x, A, bias_a, bias_x, h0, return_last_state, out, ckpt, save,
               workspace, seq_lens):
    tiles = 0
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        tiles = -(-x.shape[1] // _native.GATED_TILE)
        shape = tuple(x.shape)
    else:
        shape = (0, 0, 0)                                # refused in _gated_args
    dt, dev, Bt, L, Dm = _gated_args(
        x, gate_a, gate_x, A, bias_a, bias_x, h0, seq_lens,
        ("out", out, shape, getattr(x, "dtype", None)),
        ("ckpt", ckpt, (shape[0], tiles, shape[2]), _F32))
    lib = _native.load()
    need = int(lib.ssm_gated_scan_workspace_bytes(Bt, L, Dm, _DT[dt]))
    workspace, ws_bytes = _args.workspace(workspace, need, dev)
    y = out if out is not None else torch.empty((Bt, L, Dm), dtype=dt, device=dev)
    h_last = torch.empty((Bt, Dm), dtype=_F32, device=dev) if return_last_state else None
    if save and ckpt is None:
        ckpt = torch.empty((Bt, tiles, Dm), dtype=_F32, device=dev)
    with _on(dev):
        rc = lib.ssm_gated_scan_fwd(
            _ptr(x), _ptr(gate_a), _ptr(gate_x), _ptr(A), _ptr(bias_a), _ptr(bias_x), _ptr(h0),
            _ptr(y), _ptr(h_last), _ptr(ckpt), _ptr(seq_lens), Bt, L, Dm, _DT[dt],
            _ptr(workspace), ws_bytes, _args.stream_handle(dev))
    _native.check(rc, "ssm_gated_scan_fwd")
    return y, h_last, ckpt


def gated_scan_fwd(x: torch.Tensor, gate_a: torch.Tensor, gate_x: torch.Tensor, A: torch.Tensor,
                   bias_a: Optional[torch.Tensor] = None, bias_x: Optional[torch.Tensor] = None,
                   h0: Optional[torch.Tensor] = None, return_last_state: bool = True,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   seq_lens: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence, forward (ssm_gated_scan_fwd).

    x, gate_a, gate_x: [Bt, L, Dm]; A: [Dm] fp32, not positive; bias_a,
    bias_x: [Dm] fp32; h0: [Bt, Dm] fp32.  Returns (y, h_last).
    seq_lens: optional int32 [Bt] -- row b runs its first seq_lens[b] tokens;
    later positions of y are left untouched.
    """
    return _gated_fwd(x, gate_a, gate_x, A, bias_a, bias_x, h0, return_last_state, out, None,
                      False, workspace, seq_lens)[:2]


def gated_scan_fwd_ckpt(x: torch.Tensor, gate_a: torch.Tensor, gate_x: torch.Tensor,
                        A: torch.Tensor, bias_a: Optional[torch.Tensor] = None,
                        bias_x: Optional[torch.Tensor] = None,
                        h0: Optional[torch.Tensor] = None, return_last_state: bool = True,
                        out: Optional[torch.Tensor] = None, ckpt: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        seq_lens: Optional[torch.Tensor] = None):
    """The forward for training: gated_scan_fwd that also saves the state
    entering every 128-token tile for gated_scan_bwd(..., ckpt=...).  ckpt:
    optional fp32 [Bt, ceil(L/128), Dm] to fill.  Returns (y, h_last, ckpt)."""
    return _gated_fwd(x, gate_a, gate_x, A, bias_a, bias_x, h0, return_last_state, out, ckpt,
                      True, workspace, seq_lens)


def gated_scan_bwd(x: torch.Tensor, gate_a: torch.Tensor, gate_x: torch.Tensor, A: torch.Tensor,
                   dy: torch.Tensor, bias_a: Optional[torch.Tensor] = None,
                   bias_x: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                   dh_last: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   ckpt: Optional[torch.Tensor] = None,
                   seq_lens: Optional[torch.Tensor] = None) -> dict:
    """Gradients of the gated recurrence (ssm_gated_scan_bwd).

    Inputs as gated_scan_fwd plus dy [Bt, L, Dm] (dtype of x) and dh_last
    [Bt, Dm] fp32.  ckpt: fp32 [Bt, ceil(L/128), Dm] from gated_scan_fwd_ckpt
    over the same inputs; without it the call recomputes the states.  With
    seq_lens the gradients behind a row's end are zeros.  Returns a dict with
    dx, dgate_a, dgate_x (dtype of x), dA [Dm], and dbias_a, dbias_x, dh0 for
    the optional inputs that were given.
    """
    _args.need(dy=dy)
    shape = tuple(x.shape) if isinstance(x, torch.Tensor) and x.dim() == 3 else (0, 0, 0)
    tiles = -(-shape[1] // _native.GATED_TILE)
    dt, dev, Bt, L, Dm = _gated_args(
        x, gate_a, gate_x, A, bias_a, bias_x, h0, seq_lens,
        ("dy", dy, shape, getattr(x, "dtype", None)), ("dh_last", dh_last, (shape[0], shape[2]), _F32),
        ("ckpt", ckpt, (shape[0], tiles, shape[2]), _F32))
    lib = _native.load()
    with_ckpt = ckpt is not None and L > 0
    need = int(lib.ssm_gated_scan_bwd_workspace_bytes(Bt, L, Dm, _DT[dt], int(with_ckpt)))
    workspace, ws_bytes = _args.workspace(workspace, need, dev)
    out = {"dx": torch.empty_like(x), "dgate_a": torch.empty_like(x),
           "dgate_x": torch.empty_like(x), "dA": torch.empty((Dm,), dtype=_F32, device=dev)}
    if bias_a is not None:
        out["dbias_a"] = torch.empty((Dm,), dtype=_F32, device=dev)
    if bias_x is not None:
        out["dbias_x"] = torch.empty((Dm,), dtype=_F32, device=dev)
    if h0 is not None:
        out["dh0"] = torch.empty((Bt, Dm), dtype=_F32, device=dev)
    with _on(dev):
        rc = lib.ssm_gated_scan_bwd(
            _ptr(x), _ptr(gate_a), _ptr(gate_x), _ptr(A), _ptr(bias_a), _ptr(bias_x), _ptr(h0),
            _ptr(ckpt) if with_ckpt else None, _ptr(dy), _ptr(dh_last), _ptr(out["dx"]),
            _ptr(out["dgate_a"]), _ptr(out["dgate_x"]), _ptr(out["dA"]),
            _ptr(out.get("dbias_a")), _ptr(out.get("dbias_x")), _ptr(out.get("dh0")),
            _ptr(seq_lens), Bt, L, Dm, _DT[dt], _ptr(workspace), ws_bytes,
            _args.stream_handle(dev))
    _native.check(rc, "ssm_gated_scan_bwd")
    return out


def gated_state_update(state: torch.Tensor, x: torch.Tensor, gate_a: torch.Tensor,
                       gate_x: torch.Tensor, A: torch.Tensor,
                       bias_a: Optional[torch.Tensor] = None,
                       bias_x: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step of the gated recurrence (ssm_gated_state_update).

    state: [Bt, Dm] fp32, updated in place; x, gate_a, gate_x: [Bt, Dm];
    A, bias_a, bias_x: [Dm] fp32.  Returns y [Bt, Dm].
    """
    dt = _args.act_dtype("x", x)
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    Bt, Dm = x.shape
    dev = x.device
    _args.need(state=state, gate_a=gate_a, gate_x=gate_x, A=A)
    _args.check_args(dev, ("state", state, (Bt, Dm), _F32), ("x", x, (Bt, Dm), dt),
                     ("gate_a", gate_a, (Bt, Dm), dt), ("gate_x", gate_x, (Bt, Dm), dt),
                     ("A", A, (Dm,), _F32), ("bias_a", bias_a, (Dm,), _F32),
                     ("bias_x", bias_x, (Dm,), _F32), ("out", out, (Bt, Dm), dt))
    y = out if out is not None else torch.empty_like(x)
    with _on(dev):
        rc = _native.load().ssm_gated_state_update(
            _ptr(state), _ptr(x), _ptr(gate_a), _ptr(gate_x), _ptr(A), _ptr(bias_a), _ptr(bias_x),
            _ptr(y), Bt, Dm, _DT[dt], _args.stream_handle(dev))
    _native.check(rc, "ssm_gated_state_update")
    return y


def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   return_stats: bool = True, out: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None) -> dict:
    """Layer norm over the last axis (ssm_layer_norm_fwd), of x or, with
    `residual`, of their sum.

    x: [..., D]; weight, bias: [D] fp32; residual: fp32, the shape of x (the
    residual stream).  Returns a dict with y (dtype of x), mean and rstd
    (fp32, the shape of x without its last axis) unless return_stats is off,
    and residual_out = x + residual (fp32) with a residual.
    """
    dt = _args.act_dtype("x", x)
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    shape, D, dev = tuple(x.shape), x.shape[-1], x.device
    rows = x.numel() // D if D else 0
    _args.check_args(dev, ("x", x, shape, dt), ("weight", weight, (D,), _F32),
                     ("bias", bias, (D,), _F32), ("residual", residual, shape, _F32),
                     ("out", out, shape, dt), ("residual_out", residual_out, shape, _F32))
    if residual_out is not None and residual is None:
        raise ValueError("residual_out needs a residual")
    r = {"y": out if out is not None else torch.empty_like(x)}
    if return_stats:
        r["mean"] = torch.empty(shape[:-1], dtype=_F32, device=dev)
        r["rstd"] = torch.empty(shape[:-1], dtype=_F32, device=dev)
    if residual is not None:
        r["residual_out"] = residual_out if residual_out is not None else torch.empty_like(residual)
    with _on(dev):
        rc = _native.load().ssm_layer_norm_fwd(
            _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), float(eps), _ptr(r["y"]),
            _ptr(r.get("residual_out")), _ptr(r.get("mean")), _ptr(r.get("rstd")), rows, D,
            _DT[dt], _args.stream_handle(dev))
    _native.check(rc, "ssm_layer_norm_fwd")
    return r


def layer_norm_bwd_workspace_bytes(rows: int, D: int) -> int:
    return int(_native.load().ssm_layer_norm_bwd_workspace_bytes(rows, D))


def layer_norm_bwd(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   dresidual_out: Optional[torch.Tensor] = None, return_dresidual: bool = False,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of layer_norm_fwd (ssm_layer_norm_bwd).

    x: the tensor that was normalised -- the forward's x (dtype of dy), or its
    residual_out (fp32); dy: [..., D]; mean, rstd: as the forward returned
    them; dresidual_out: fp32, the gradient of residual_out.  Returns a dict
    with dx (dtype of dy), dresidual (the same gradient in fp32) if asked for,
    and dweight, dbias [D] (fp32) for the parameters that were given (the bias
    itself is not read).
    """
    dt = _args.act_dtype("dy", dy)
    xdt = _args.act_dtype("x", x)
    if dy.dim() < 1:
        raise ValueError("dy must be [..., D]")
    if xdt not in (dt, _F32):
        raise TypeError(f"x must be {dt} or float32 (got {xdt})")
    shape, D, dev = tuple(dy.shape), dy.shape[-1], dy.device
    rows = dy.numel() // D if D else 0
    _args.need(mean=mean, rstd=rstd)
    _args.check_args(dev, ("x", x, shape, xdt), ("dy", dy, shape, dt),
                     ("mean", mean, shape[:-1], _F32), ("rstd", rstd, shape[:-1], _F32),
                     ("weight", weight, (D,), _F32), ("bias", bias, (D,), _F32),
                     ("dresidual_out", dresidual_out, shape, _F32))
    lib = _native.load()
    workspace, ws_bytes = _args.workspace(
        workspace, int(lib.ssm_layer_norm_bwd_workspace_bytes(rows, D)), dev)
    r = {"dx": torch.empty_like(dy)}
    if return_dresidual:
        r["dresidual"] = torch.empty(shape, dtype=_F32, device=dev)
    if weight is not None:
        r["dweight"] = torch.empty((D,), dtype=_F32, device=dev)
    if bias is not None:
        r["dbias"] = torch.empty((D,), dtype=_F32, device=dev)
    with _on(dev):
        rc = lib.ssm_layer_norm_bwd(
            _ptr(x), _DT[xdt], _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(weight),
            _ptr(dresidual_out), _ptr(r["dx"]), _ptr(r.get("dresidual")), _ptr(r.get("dweight")),
            _ptr(r.get("dbias")), rows, D, _DT[dt], _ptr(workspace), ws_bytes,
            _args.stream_handle(dev))
    _native.check(rc, "ssm_layer_norm_bwd")
    return r


def causal_conv1d_silu_bwd_workspace_bytes(B: int, L: int, D: int, K: int) -> int:
    return int(_native.load().ssm_causal_conv1d_silu_bwd_workspace_bytes(B, L, D, K))


def causal_conv1d_silu_bwd(x: torch.Tensor, weight: torch.Tensor, du: torch.Tensor,
                           bias: Optional[torch.Tensor] = None,
                           state: Optional[torch.Tensor] = None, silu: bool = True,
                           dstate_out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of causal_conv1d_silu (ssm_causal_conv1d_silu_bwd).

    x, weight, bias, state, silu: as the forward; du: [Bt, L, Dm] (dtype of
    x), the gradient of u; dstate_out: [Bt, Dm, K-1] fp32, the gradient of the
    state that the forward handed on.  Returns a dict with dx (dtype of x),
    dweight [Dm, K], and dbias, dstate for the optional inputs that were given.
    """
    dt = _args.act_dtype("x", x)
    if x.dim() != 3 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [B, L, D] and weight [D, K]")
    Bt, L, Dm = x.shape
    K, dev = weight.shape[1], x.device
    _args.need(du=du)
    _args.check_args(dev, ("x", x, (Bt, L, Dm), dt), ("weight", weight, (Dm, K), _F32),
                     ("du", du, (Bt, L, Dm), dt), ("bias", bias, (Dm,), _F32),
                     ("state", state, (Bt, Dm, K - 1), _F32),
                     ("dstate_out", dstate_out, (Bt, Dm, K - 1), _F32))
    lib = _native.load()
    workspace, ws_bytes = _args.workspace(
        workspace, int(lib.ssm_causal_conv1d_silu_bwd_workspace_bytes(Bt, L, Dm, K)), dev)
    r = {"dx": torch.empty_like(x), "dweight": torch.empty_like(weight)}
    if bias is not None:
        r["dbias"] = torch.empty_like(bias)
    if state is not None:
        r["dstate"] = torch.empty_like(state)
    with _on(dev):
        rc = lib.ssm_causal_conv1d_silu_bwd(
            _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), int(bool(silu)), _ptr(du),
            _ptr(dstate_out), _ptr(r["dx"]), _ptr(r["dweight"]), _ptr(r.get("dbias")),
            _ptr(r.get("dstate")), Bt, L, Dm, K, _DT[dt], _ptr(workspace), ws_bytes,
            _args.stream_handle(dev))
    _native.check(rc, "ssm_causal_conv1d_silu_bwd")
    return r
