"""Selective state space scan, its short causal convolution and the group norm: the binding of the
``efla_causal_conv*``, ``efla_ssm_*`` and ``efla_group_norm*`` calls of ``include/efla.h`` (argument
marshalling only).

    y_t = silu(bias + sum_j w_j x_{t-W+1+j})                                       (causal_conv)
    delta_t = softplus(dt_t + dt_bias),  h_t = exp(-exp(A_log) delta_t) h_{t-1} + delta_t x_t B_t,
    y_t = (C_t . h_t + D x_t) silu(z_t)                                            (ssm_scan)
    y = silu(w (x - mean) / sqrt(var + eps) + b) over the channels of a group      (group_norm)

The calls are plain functions: gradients come from the ``*_bwd`` calls, and nothing is recorded for
autograd.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _check, load
from .gated import (_DT, _INT_MAX, _bad, _empty, _empty_as, _first, _given, _need, _ptr, _stream, _too_large, _workspace)
from .gated import _on_device as _refuse_device

_vp, _ip, _sz, _fl = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SIGNATURES = {
    "efla_causal_conv": [_vp] * 7 + [_ip] * 7 + [_vp],
    "efla_causal_conv_bwd": [_vp] * 10 + [_ip] * 6 + [_vp, _sz, _vp],
    "efla_causal_conv_bwd_workspace": [_ip] * 4 + [ctypes.POINTER(_sz)],
    "efla_causal_conv_step": [_vp] * 5 + [_ip] * 5 + [_vp],
    "efla_ssm_scan": [_vp] * 12 + [_ip] * 7 + [_vp, _sz, _vp],
    "efla_ssm_scan_workspace": [_ip] * 7 + [ctypes.POINTER(_sz)],
    "efla_ssm_scan_train": [_vp] * 11 + [_ip] * 6 + [_vp, _sz, _vp],
    "efla_ssm_bwd_workspace": [_ip] * 5 + [ctypes.POINTER(_sz)],
    "efla_ssm_scan_bwd": [_vp] * 20 + [_ip] * 7 + [_vp, _sz, _vp],
    "efla_ssm_step": [_vp] * 10 + [_ip] * 5 + [_vp],
    "efla_group_norm": [_vp] * 5 + [_ip] * 6 + [_fl, _vp, _sz, _vp],
    "efla_group_norm_workspace": [_ip] * 6 + [ctypes.POINTER(_sz)],
    "efla_group_norm_bwd": [_vp] * 8 + [_ip] * 6 + [_vp, _sz, _vp],
}
_ACTIVATIONS = {None: 0, "silu": 1}
_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = load()
        for name, types in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = _ip, types
        _bound = L
    return _bound


def _all(like: torch.Tensor, *args):
    """``_need`` of every (name, tensor or None, shape, dtype), 0.5 us each where nothing is amiss."""
    device = like.get_device()
    for name, t, shape, dtype in args:
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous()):
            _need(name, t, shape, dtype, like)


def _on_device(t: torch.Tensor):
    """The check of ``gated._on_device``, without what torch.cuda.current_device() does around it."""
    if not t.is_cuda or t.get_device() != torch._C._cuda_getDevice():
        _refuse_device(t)


def _activation(activation) -> int:
    code = _ACTIVATIONS.get(activation, -1)
    if code < 0:
        _bad(f"unknown activation {activation!r} (None or 'silu')")
    return code


@functools.lru_cache(maxsize=4096)
def _bytes(name: str, *sizes: int) -> int:
    """A workspace query, which depends on nothing but its sizes: asked once for each."""
    n = _sz(0)
    _check(getattr(_lib(), name)(*sizes, ctypes.byref(n)))
    return n.value


def _sequences(cu_seqlens, B: int, x) -> int:
    if cu_seqlens is None:
        return B
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        _bad("cu_seqlens must be a 1-D int32 tensor of at least one bound")
    _need("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, x)
    if B != 1:
        _bad(f"cu_seqlens given with B={B} (must be 1)")
    return cu_seqlens.shape[0] - 1


def _conv_args(x, w, bias, dims):
    code = _first("x", x, dims)
    if w.dim() != 2:
        _bad(f"w must be [D, W], got {list(w.shape)}")
    shape = x.shape
    D, W = shape[-1], w.shape[1]
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX or D > _INT_MAX or W > _INT_MAX:
        _too_large(*shape, W)
    _all(x, ("x", x, shape, x.dtype), ("w", w, (D, W), torch.float32), ("bias", bias, (D,), torch.float32))
    return code, D, W


def causal_conv(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                state0: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                activation: Optional[str] = "silu", y: Optional[torch.Tensor] = None,
                state_T: Optional[torch.Tensor] = None, stream=None,
                return_state: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The short causal convolution over whole sequences with its activation (``efla_causal_conv``).

    x [B,T,D] (bf16 or fp32), w [D,W] (the newest token's weight last) and bias [D] fp32; state0
    [N,W-1,D] in x's dtype, the inputs before each sequence; cu_seqlens [N+1] int32 (then B == 1).
    Returns (y [B,T,D], state_T [N,W-1,D] -- the last W-1 inputs -- or None when ``return_state`` is False).
    """
    code, D, W = _conv_args(x, w, bias, 3)
    act = _activation(activation)
    B, T, _ = x.shape
    N = _sequences(cu_seqlens, B, x)
    if state0 is not None:
        _need("state0", state0, (N, W - 1, D), x.dtype, x)
    _on_device(x)
    L = _lib()
    y = _given("y", y, x.shape, x.dtype, x, stream)
    if state_T is not None or return_state:
        state_T = _given("state_T", state_T, (N, max(W - 1, 0), D), x.dtype, x, stream)
    _check(L.efla_causal_conv(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(state0), _ptr(cu_seqlens), y.data_ptr(),
                              _ptr(state_T), B, T, D, W, N, code, act, _stream(stream, x)))
    return y, state_T


def causal_conv_bwd(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor], state0: Optional[torch.Tensor],
                    dy: torch.Tensor, dstate_T: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                    need_dstate0: bool = True, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``causal_conv`` (no cu_seqlens) from dy [B,T,D] and dstate_T [B,W-1,D] (or None) in x's dtype
    (``efla_causal_conv_bwd``): a dict with dx, dstate0 (None unless asked for) in x's dtype, dw [D,W] and dbias [D]
    (None without a bias) fp32."""
    code, D, W = _conv_args(x, w, bias, 3)
    act = _activation(activation)
    B, T, _ = x.shape
    _need("dy", dy, x.shape, x.dtype, x)
    for name, t in (("state0", state0), ("dstate_T", dstate_T)):
        if t is not None:
            _need(name, t, (B, W - 1, D), x.dtype, x)
    _on_device(x)
    L = _lib()
    ws = _workspace(workspace, _bytes("efla_causal_conv_bwd_workspace", B, T, D, W), x, stream)
    out = {"dx": _empty_as(x, x.dtype, stream), "dw": _empty_as(w, torch.float32, stream),
           "dbias": None if bias is None else _empty_as(bias, torch.float32, stream),
           "dstate0": _empty((B, max(W - 1, 0), D), x.dtype, x, stream) if need_dstate0 else None}
    _check(L.efla_causal_conv_bwd(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(state0), dy.data_ptr(), _ptr(dstate_T),
                                  *(_ptr(t) for t in out.values()), B, T, D, W, code, act, ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream(stream, x)))
    return out


def causal_conv_step(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor], state: torch.Tensor, *,
                     activation: Optional[str] = "silu", y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token per sequence (``efla_causal_conv_step``): x [B,D], state [B,W-1,D] in x's dtype, shifted in place.
    Returns y [B,D]."""
    code, D, W = _conv_args(x, w, bias, 2)
    act = _activation(activation)
    B = x.shape[0]
    _need("state", state, (B, W - 1, D), x.dtype, x)
    _on_device(x)
    y = _given("y", y, x.shape, x.dtype, x, stream)
    _check(_lib().efla_causal_conv_step(x.data_ptr(), w.data_ptr(), _ptr(bias), state.data_ptr(), y.data_ptr(), B, D, W,
                                        code, act, _stream(stream, x)))
    return y


def _ssm_args(x, dt, A_log, B, C, D, dt_bias, z, lead: int):
    """Shapes of the scan's inputs with `lead` leading dimensions; (lead shape, channels, state, groups, dtype code)."""
    code = _first("x", x, lead + 1)
    if A_log.dim() != 2 or B.dim() != lead + 2:
        _bad(f"A_log must be [D, d_state] and B {lead + 2}-D, got {list(A_log.shape)} and {list(B.shape)}")
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    *at, ch = shape
    N, G = A_log.shape[1], B.shape[lead]
    if shape[0] > _INT_MAX or shape[lead - 1] > _INT_MAX or ch > _INT_MAX or N > _INT_MAX or G > _INT_MAX:
        _too_large(*shape, N, G)
    each, shared = (ch,), (*at, G, N)
    _all(x, ("x", x, shape, dtype), ("dt", dt, shape, dtype), ("A_log", A_log, (ch, N), f32), ("B", B, shared, dtype),
         ("C", C, shared, dtype), ("D", D, each, f32), ("dt_bias", dt_bias, each, f32), ("z", z, shape, dtype))
    return at, ch, N, G, code


def _inputs(x, dt, A_log, B, C, D, dt_bias, z):
    return (x.data_ptr(), dt.data_ptr(), A_log.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(dt_bias), _ptr(z))


def ssm_scan_workspace(B: int, T: int, D: int, d_state: int, G: int = 1, N: Optional[int] = None) -> int:
    """Workspace bytes of ``ssm_scan``; N: the number of sequences of cu_seqlens, if that is given."""
    if max(B, T, D, d_state, G, N or 0) > _INT_MAX:
        _too_large(B, T, D, d_state, G, N or 0)
    return _bytes("efla_ssm_scan_workspace", B, T, D, d_state, G, B if N is None else N, int(N is not None))


def ssm_bwd_workspace(B: int, T: int, D: int, d_state: int, G: int = 1) -> int:
    """Workspace bytes of ``ssm_scan_train`` and ``ssm_scan_bwd``."""
    if max(B, T, D, d_state, G) > _INT_MAX:
        _too_large(B, T, D, d_state, G)
    return _bytes("efla_ssm_bwd_workspace", B, T, D, d_state, G)


def ssm_scan(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             S0: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
             workspace: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
             S_T: Optional[torch.Tensor] = None, stream=None,
             return_state: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The selective state space scan over whole sequences (``efla_ssm_scan``).

    x, dt, z [B,T,D] and B, C [B,T,G,d_state] (bf16 or fp32; the D / G channels of a group share B and C), A_log
    [D,d_state], D and dt_bias [D] fp32; S0 [N,D,d_state] fp32; cu_seqlens [N+1] int32 (then the batch is 1).
    Returns (y [B,T,D] in x's dtype, S_T [N,D,d_state] fp32 or None when ``return_state`` is False).  ``workspace`` (of
    ``ssm_scan_workspace(...)`` bytes) is allocated here when not given.  How packed sequences are cut goes by their mean
    length: one that is far longer than many short ones is faster in a call of its own.
    """
    (rows, T), ch, N, G, code = _ssm_args(x, dt, A_log, B, C, D, dt_bias, z, 2)
    seqs = _sequences(cu_seqlens, rows, x)
    if S0 is not None:
        _need("S0", S0, (seqs, ch, N), torch.float32, x)
    _on_device(x)
    L = _lib()
    need = _bytes("efla_ssm_scan_workspace", rows, T, ch, N, G, seqs, int(cu_seqlens is not None))
    ws = _workspace(workspace, need, x, stream) if need else workspace
    y = _given("y", y, x.shape, x.dtype, x, stream)
    if S_T is not None or return_state:
        S_T = _given("S_T", S_T, (seqs, ch, N), torch.float32, x, stream)
    _check(L.efla_ssm_scan(*_inputs(x, dt, A_log, B, C, D, dt_bias, z), _ptr(S0), _ptr(cu_seqlens), y.data_ptr(), _ptr(S_T),
                           rows, T, ch, N, G, seqs, code, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                           _stream(stream, x)))
    return y, S_T


def ssm_scan_train(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, S0: Optional[torch.Tensor] = None, *,
                   workspace: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   S_T: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``ssm_scan`` over rows of [B, T] that also fills ``workspace`` for one ``ssm_scan_bwd(..., workspace=...,
    saved=True)`` of the same inputs.  Returns (y, S_T, workspace)."""
    (rows, T), ch, N, G, code = _ssm_args(x, dt, A_log, B, C, D, dt_bias, z, 2)
    if S0 is not None:
        _need("S0", S0, (rows, ch, N), torch.float32, x)
    _on_device(x)
    L = _lib()
    ws = _workspace(workspace, _bytes("efla_ssm_bwd_workspace", rows, T, ch, N, G), x, stream)
    y = _given("y", y, x.shape, x.dtype, x, stream)
    S_T = _given("S_T", S_T, (rows, ch, N), torch.float32, x, stream)
    _check(L.efla_ssm_scan_train(*_inputs(x, dt, A_log, B, C, D, dt_bias, z), _ptr(S0), y.data_ptr(), S_T.data_ptr(), rows, T,
                                 ch, N, G, code, ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream, x)))
    return y, S_T, ws


def ssm_scan_bwd(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                 D: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor], z: Optional[torch.Tensor],
                 S0: Optional[torch.Tensor], dy: torch.Tensor, dS_T: Optional[torch.Tensor] = None, *,
                 need_dS0: bool = True, workspace: Optional[torch.Tensor] = None, saved: bool = False,
                 stream=None) -> dict:
    """Gradients of ``ssm_scan`` (no cu_seqlens) from dy [B,T,D] in x's dtype and dS_T [B,D,d_state] fp32 (or None),
    ``efla_ssm_scan_bwd``: a dict with dx, ddt, dB, dC, dz in x's dtype, dA_log, dD, ddt_bias and dS0 fp32 (None for an
    input that is None, and for dS0 unless asked for).  ``saved=True`` takes the workspace that ``ssm_scan_train``
    filled for these inputs and does not run the forward again; it serves one backward."""
    (rows, T), ch, N, G, code = _ssm_args(x, dt, A_log, B, C, D, dt_bias, z, 2)
    if saved and workspace is None:
        _bad("saved=True needs the workspace that ssm_scan_train filled")
    _need("dy", dy, x.shape, x.dtype, x)
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _need(name, t, (rows, ch, N), torch.float32, x)
    _on_device(x)
    L = _lib()
    ws = _workspace(workspace, _bytes("efla_ssm_bwd_workspace", rows, T, ch, N, G), x, stream)
    f32 = torch.float32
    out = {"dx": _empty_as(x, x.dtype, stream), "ddt": _empty_as(x, x.dtype, stream), "dA_log": _empty_as(A_log, f32, stream),
           "dB": _empty_as(B, x.dtype, stream), "dC": _empty_as(B, x.dtype, stream),
           "dD": None if D is None else _empty_as(D, f32, stream),
           "ddt_bias": None if dt_bias is None else _empty_as(dt_bias, f32, stream),
           "dz": None if z is None else _empty_as(x, x.dtype, stream),
           "dS0": _empty((rows, ch, N), f32, x, stream) if need_dS0 else None}
    _check(L.efla_ssm_scan_bwd(*_inputs(x, dt, A_log, B, C, D, dt_bias, z), _ptr(S0), dy.data_ptr(), _ptr(dS_T),
                               *(_ptr(t) for t in out.values()), rows, T, ch, N, G, code, int(saved), ws.data_ptr(),
                               ws.numel() * ws.element_size(), _stream(stream, x)))
    return out


def ssm_step(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             D: Optional[torch.Tensor], dt_bias: Optional[torch.Tensor], z: Optional[torch.Tensor], S: torch.Tensor, *,
             y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token per sequence; S [B,D,d_state] fp32 is updated in place (``efla_ssm_step``).  x, dt, z [B,D], B, C
    [B,G,d_state].  Returns y [B,D]."""
    (rows,), ch, N, G, code = _ssm_args(x, dt, A_log, B, C, D, dt_bias, z, 1)
    _need("S", S, (rows, ch, N), torch.float32, x)
    _on_device(x)
    y = _given("y", y, x.shape, x.dtype, x, stream)
    _check(_lib().efla_ssm_step(*_inputs(x, dt, A_log, B, C, D, dt_bias, z), S.data_ptr(), y.data_ptr(), rows, ch, N, G, code,
                                _stream(stream, x)))
    return y


def _group_norm_args(x, w, b, groups):
    if x.dim() < 2:
        _bad(f"x must be [rows, ..., C], got {list(x.shape)}")
    code = _first("x", x, x.dim())
    rows, C = x.shape[0], x.shape[-1]
    L = 1
    for n in x.shape[1:-1]:
        L *= n
    if max(rows, L, C, groups) > _INT_MAX:
        _too_large(rows, L, C, groups)
    if groups < 1 or C % groups:
        _bad(f"x's {C} channels must be a multiple of groups={groups}")
    _need("x", x, x.shape, x.dtype, x)
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _need(name, t, (C,), torch.float32, x)
    return code, rows, L, C


def group_norm_workspace(rows: int, L: int, C: int, groups: int, dtype: torch.dtype, backward: bool = False) -> int:
    """Workspace bytes of ``group_norm`` and, with ``backward``, of ``group_norm_bwd``."""
    if dtype not in _DT:
        _bad(f"unsupported dtype {dtype}")
    if max(rows, L, C, groups) > _INT_MAX:
        _too_large(rows, L, C, groups)
    return _bytes("efla_group_norm_workspace", rows, L, C, groups, _DT[dtype], int(backward))


def group_norm(x: torch.Tensor, w: Optional[torch.Tensor], b: Optional[torch.Tensor], groups: int, *, eps: float = 1e-5,
               activation: Optional[str] = None, y: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
               return_stats: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """The group norm with its activation, channels last (``efla_group_norm``).

    x [rows, ..., C] (bf16 or fp32), normalised over everything between and the C / groups channels of a group: a
    token's heads for x [tokens, C], a feature map for x [batch, height, width, C].  w, b [C] fp32 or None.  ``y`` may
    be x.  Returns y, or (y, stats) -- stats [rows, groups, 2] fp32 for ``group_norm_bwd`` -- where ``stats`` is given
    or asked for."""
    code, rows, L, C = _group_norm_args(x, w, b, groups)
    act = _activation(activation)
    _on_device(x)
    Lb = _lib()
    y = _given("y", y, x.shape, x.dtype, x, stream)
    if stats is not None or return_stats:
        stats = _given("stats", stats, (rows, groups, 2), torch.float32, x, stream)
    need = _bytes("efla_group_norm_workspace", rows, L, C, groups, code, 0)
    ws = _workspace(workspace, need, x, stream) if need else None
    _check(Lb.efla_group_norm(x.data_ptr(), _ptr(w), _ptr(b), y.data_ptr(), _ptr(stats), rows, L, C, groups, code, act, eps,
                              _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream, x)))
    return y if stats is None else (y, stats)


def group_norm_bwd(x: torch.Tensor, w: Optional[torch.Tensor], b: Optional[torch.Tensor], groups: int,
                   stats: torch.Tensor, dy: torch.Tensor, *, activation: Optional[str] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``group_norm`` from dy in x's dtype and the forward's stats (``efla_group_norm_bwd``): a dict with dx
    in x's dtype, dw and db [C] fp32 (None without w, b)."""
    code, rows, L, C = _group_norm_args(x, w, b, groups)
    act = _activation(activation)
    _need("stats", stats, (rows, groups, 2), torch.float32, x)
    _need("dy", dy, x.shape, x.dtype, x)
    _on_device(x)
    Lb = _lib()
    ws = _workspace(workspace, _bytes("efla_group_norm_workspace", rows, L, C, groups, code, 1), x, stream)
    out = {"dx": _empty_as(x, x.dtype, stream), "dw": None if w is None else _empty_as(w, torch.float32, stream),
           "db": None if b is None else _empty_as(b, torch.float32, stream)}
    _check(Lb.efla_group_norm_bwd(x.data_ptr(), _ptr(w), _ptr(b), stats.data_ptr(), dy.data_ptr(),
                                  *(_ptr(t) for t in out.values()), rows, L, C, groups, code, act, ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream(stream, x)))
    return out
