"""Gated delta rule and the norms around it: the binding of the ``efla_gated_*`` and
``efla_norm_gate*`` calls of ``include/efla.h`` (argument marshalling only).

    S_t = e^{g_t} (I - alpha_t k_t k_t^T) S_{t-1} + alpha_t k_t v_t^T,   o_t = S_t^T q_t

H value heads read H_k query/key heads (value head h reads key head ``h // (H // H_k)``);
``update="euler"`` (alpha = beta) is the gated delta rule, ``update="exact"`` the exact gate with the
same decay.  The calls are plain functions: gradients come from the ``*_bwd*`` calls, and nothing is recorded
for autograd.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import UPDATES, EflaError, _check, load

_DT = {torch.bfloat16: 0, torch.float32: 1}
_vp, _ip, _sz, _ll, _fl = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_float
_SIGNATURES = {
    "efla_gated_fwd_chunked": [_vp] * 9 + [_ip] * 10 + [_vp],
    "efla_gated_fwd_chunked_train": [_vp] * 8 + [_ip] * 8 + [_vp, _sz, _vp],
    "efla_gated_bwd_workspace": [_ip] * 7 + [ctypes.POINTER(_sz)],
    "efla_gated_bwd_chunked": [_vp] * 14 + [_ip] * 9 + [_vp, _sz, _vp],
    "efla_gated_decode_step": [_vp] * 7 + [_ip] * 8 + [_vp],
    "efla_gated_decode_tokens": [_vp] * 7 + [_ip] * 9 + [_vp],
    "efla_gated_prep": [_vp] * 10 + [_ll] + [_ip] * 4 + [_fl, _fl, _vp],
    "efla_gated_prep_bwd": [_vp] * 16 + [_ll] + [_ip] * 4 + [_fl, _fl, _vp, _sz, _vp],
    "efla_gated_prep_bwd_workspace": [_ll, _ip, ctypes.POINTER(_sz)],
    "efla_norm_gate": [_vp] * 4 + [_ll, _ip, _ip, _fl, _vp],
    "efla_norm_gate_bwd": [_vp] * 7 + [_ll, _ip, _ip, _fl, _vp, _sz, _vp],
    "efla_norm_gate_bwd_workspace": [_ip, ctypes.POINTER(_sz)],
}
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


def _bad(msg: str):
    raise EflaError(1, msg)


_INT_MAX = 2147483647  # ctypes would pass the low 32 bits of a larger size


def _too_large(*sizes: int):
    _bad(f"a size of {max(sizes)} exceeds {_INT_MAX}")


def _need(name: str, t: torch.Tensor, shape, dtype, like: torch.Tensor):
    """`t` is a contiguous tensor of this shape and dtype on `like`'s device."""
    if t.dtype is not dtype or t.shape != shape:
        _bad(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != like.get_device():
        _bad(f"{name} is on {t.device}, the first argument on {like.device}")
    if not t.is_contiguous():
        _bad(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _first(name: str, t: torch.Tensor, dims: int) -> int:
    """Checks of the argument the others are held to; its dtype's code.  The device is checked last,
    so that every other fault is reported on a machine without a GPU too."""
    if t.dim() != dims or (code := _DT.get(t.dtype)) is None:
        _bad(f"{name} must be a {dims}-D bfloat16 or float32 tensor, got {t.dtype} {list(t.shape)}")
    return code


def _on_device(t: torch.Tensor):
    if not t.is_cuda:
        _bad("the tensors must be CUDA tensors")
    if t.get_device() != torch.cuda.current_device():
        _bad(f"the tensors are on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _stream(stream, like: torch.Tensor) -> int:
    """The handle of `stream`, or of the current one (of `like`'s device, which is current) without the
    Stream object that torch.cuda.current_stream() makes: 0.1 us in place of 2.9."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(like.get_device())
    if stream.device_index != like.get_device():
        _bad(f"the stream is on cuda:{stream.device_index}, the tensors on {like.device}")
    return stream.cuda_stream


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An allocation the call's kernels use on `stream`: from that stream's memory, so that it waits for
    whatever used it before, and not handed out again before the current stream is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _empty_as(t: torch.Tensor, dtype, stream) -> torch.Tensor:
    """``_empty`` with the shape of `t` (torch.empty_like takes a third of torch.empty's time)."""
    return torch.empty_like(t, dtype=dtype) if stream is None else _empty(t.shape, dtype, t, stream)


def _update(update: str) -> int:
    code = UPDATES.get(update)
    if code is None:
        _bad(f"unknown update rule {update!r}")
    return code


def _heads(q, k, v, g, beta, lead: int):
    """Shapes of the mixer's inputs with `lead` leading dimensions; (lead shape, Hk, H, dk, dv, dtype code)."""
    code = _first("q", q, lead + 2)
    if v.dim() != lead + 2:
        _bad(f"v must be {lead + 2}-D, got {list(v.shape)}")
    qs = q.shape
    *at, Hk, dk = qs
    H, dv = v.shape[lead:]
    if dk > _INT_MAX or dv > _INT_MAX or H > _INT_MAX:
        _too_large(dk, dv, H)
    if Hk < 1 or H % Hk:
        _bad(f"v's {H} heads must be a multiple of q's and k's {Hk}")
    per_head = (*at, H)
    _need("q", q, qs, q.dtype, q)
    _need("k", k, qs, q.dtype, q)
    _need("v", v, (*at, H, dv), q.dtype, q)
    _need("g", g, per_head, torch.float32, q)
    _need("beta", beta, per_head, torch.float32, q)
    return at, Hk, H, dk, dv, code


def _given(name: str, t: Optional[torch.Tensor], shape, dtype, like, stream) -> torch.Tensor:
    """An output: the caller's, checked, or a new one."""
    if t is None:
        return _empty_as(like, dtype, stream) if like.shape == shape else _empty(shape, dtype, like, stream)
    _need(name, t, shape, dtype, like)
    return t


def _o_dtype(o, o_dtype, q) -> torch.dtype:
    dtype = o.dtype if o is not None else q.dtype if o_dtype is None else o_dtype
    if dtype not in _DT:
        _bad(f"o must be bfloat16 or float32, not {dtype}")
    return dtype


def gated_fwd_chunked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                      S0: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                      o: Optional[torch.Tensor] = None, S_T: Optional[torch.Tensor] = None,
                      o_dtype: Optional[torch.dtype] = None, stream=None, return_state: bool = True,
                      update: str = "euler") -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gated delta rule over whole sequences (``efla_gated_fwd_chunked``).

    q, k [B,T,H_k,dk], v [B,T,H,dv] (bf16 or fp32); g (log decay, <= 0), beta [B,T,H] fp32;
    S0 [N,H,dk,dv] fp32; cu_seqlens [N+1] int32 (then B == 1).  Returns (o [B,T,H,dv], S_T
    [N,H,dk,dv] fp32 or None when ``return_state`` is False).
    """
    (B, T), Hk, H, dk, dv, code = _heads(q, k, v, g, beta, 2)
    rule = _update(update)
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            _bad("cu_seqlens must be a 1-D int32 tensor of at least one bound")
        _need("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, q)
        if B != 1:
            _bad(f"cu_seqlens given with B={B} (must be 1)")
        N = cu_seqlens.shape[0] - 1
    if S0 is not None:
        _need("S0", S0, (N, H, dk, dv), torch.float32, q)
    od = _o_dtype(o, o_dtype, q)
    _on_device(q)
    L = _lib()
    o = _given("o", o, v.shape, od, v, stream)
    if S_T is not None or return_state:
        S_T = _given("S_T", S_T, (N, H, dk, dv), torch.float32, q, stream)
    _check(L.efla_gated_fwd_chunked(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(S0),
                                    _ptr(cu_seqlens), o.data_ptr(), _ptr(S_T), B, T, Hk, H, dk, dv, N, code, _DT[od],
                                    rule, _stream(stream, q)))
    return o, S_T


def gated_bwd_workspace(B: int, T: int, Hk: int, H: int, dk: int, dv: int, dtype: torch.dtype) -> int:
    """Workspace bytes of ``gated_fwd_chunked_train`` and ``gated_bwd_chunked``."""
    if dtype not in _DT:
        _bad(f"unsupported dtype {dtype}")
    if max(B, T, Hk, H, dk, dv) > _INT_MAX:
        _too_large(B, T, Hk, H, dk, dv)
    n = _sz(0)
    _check(_lib().efla_gated_bwd_workspace(B, T, Hk, H, dk, dv, _DT[dtype], ctypes.byref(n)))
    return n.value


def _workspace(ws: Optional[torch.Tensor], need: int, like: torch.Tensor, stream) -> torch.Tensor:
    if ws is None:
        return _empty((max(need, 16),), torch.uint8, like, stream)
    if ws.device != like.device or not ws.is_contiguous():
        _bad(f"workspace must be a contiguous tensor on {like.device}")
    if ws.numel() * ws.element_size() < need:
        _bad(f"workspace of {need} bytes needed, got {ws.numel() * ws.element_size()}")
    return ws


def gated_fwd_chunked_train(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                            S0: Optional[torch.Tensor] = None, *, workspace: Optional[torch.Tensor] = None,
                            o: Optional[torch.Tensor] = None, S_T: Optional[torch.Tensor] = None, stream=None,
                            update: str = "euler") -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``gated_fwd_chunked`` over rows of [B, T] (o in q's dtype) that also fills ``workspace`` for one
    ``gated_bwd_chunked(..., workspace=..., saved=True)`` of the same inputs.  Returns (o, S_T, workspace)."""
    (B, T), Hk, H, dk, dv, code = _heads(q, k, v, g, beta, 2)
    rule = _update(update)
    if S0 is not None:
        _need("S0", S0, (B, H, dk, dv), torch.float32, q)
    _on_device(q)
    L = _lib()
    o = _given("o", o, v.shape, q.dtype, v, stream)
    S_T = _given("S_T", S_T, (B, H, dk, dv), torch.float32, q, stream)
    need = gated_bwd_workspace(B, T, Hk, H, dk, dv, q.dtype)
    ws = _workspace(workspace, need, q, stream)
    _check(L.efla_gated_fwd_chunked_train(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                          _ptr(S0), o.data_ptr(), S_T.data_ptr(), B, T, Hk, H, dk, dv, code, rule,
                                          ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream, q)))
    return o, S_T, ws


def gated_bwd_chunked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                      S0: Optional[torch.Tensor], dO: torch.Tensor, dS_T: Optional[torch.Tensor] = None, *,
                      need_dS0: bool = True, workspace: Optional[torch.Tensor] = None, saved: bool = False,
                      stream=None, update: str = "euler") -> dict:
    """Gradients of ``gated_fwd_chunked`` (no cu_seqlens) from dO [B,T,H,dv] in q's dtype and dS_T
    [B,H,dk,dv] fp32 (or None): dq, dk, dv in q's dtype, dg, dbeta and dS0 fp32
    (``efla_gated_bwd_chunked``).  ``saved=True`` takes the workspace ``gated_fwd_chunked_train``
    filled for these inputs and does not run the forward again; it serves one backward."""
    (B, T), Hk, H, dk, dv, code = _heads(q, k, v, g, beta, 2)
    rule = _update(update)
    if saved and workspace is None:
        _bad("saved=True needs the workspace that gated_fwd_chunked_train filled")
    _need("dO", dO, v.shape, q.dtype, q)
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _need(name, t, (B, H, dk, dv), torch.float32, q)
    _on_device(q)
    L = _lib()
    need = gated_bwd_workspace(B, T, Hk, H, dk, dv, q.dtype)
    ws = _workspace(workspace, need, q, stream)
    out = {"dq": _empty_as(q, q.dtype, stream), "dk": _empty_as(q, q.dtype, stream), "dv": _empty_as(v, q.dtype, stream),
           "dg": _empty_as(g, torch.float32, stream), "dbeta": _empty_as(g, torch.float32, stream),
           "dS0": _empty((B, H, dk, dv), torch.float32, q, stream) if need_dS0 else None}
    _check(L.efla_gated_bwd_chunked(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(S0),
                                    dO.data_ptr(), _ptr(dS_T), *(_ptr(t) for t in out.values()), B, T, Hk, H, dk, dv,
                                    code, rule, int(saved), ws.data_ptr(), ws.numel() * ws.element_size(),
                                    _stream(stream, q)))
    return out


def _decode(fn, lead, q, k, v, g, beta, S, o, o_dtype, stream, update):
    at, Hk, H, dk, dv, code = _heads(q, k, v, g, beta, lead)
    rule = _update(update)
    _need("S", S, (at[0], H, dk, dv), torch.float32, q)
    od = _o_dtype(o, o_dtype, q)
    _on_device(q)
    o = _given("o", o, v.shape, od, v, stream)
    _check(getattr(_lib(), fn)(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), S.data_ptr(),
                               o.data_ptr(), *at, Hk, H, dk, dv, code, _DT[od], rule, _stream(stream, q)))
    return o


def gated_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                      S: torch.Tensor, *, o: Optional[torch.Tensor] = None, o_dtype: Optional[torch.dtype] = None,
                      stream=None, update: str = "euler") -> torch.Tensor:
    """One token per sequence; S [B,H,dk,dv] fp32 is updated in place (``efla_gated_decode_step``).
    q, k [B,H_k,dk], v [B,H,dv], g, beta [B,H] fp32.  Returns o [B,H,dv]."""
    return _decode("efla_gated_decode_step", 1, q, k, v, g, beta, S, o, o_dtype, stream, update)


def gated_decode_tokens(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                        S: torch.Tensor, *, o: Optional[torch.Tensor] = None, o_dtype: Optional[torch.dtype] = None,
                        stream=None, update: str = "euler") -> torch.Tensor:
    """m tokens per sequence appended to the state, S [B,H,dk,dv] fp32 updated in place
    (``efla_gated_decode_tokens``).  q, k [B,m,H_k,dk], v [B,m,H,dv], g, beta [B,m,H] fp32.
    Returns o [B,m,H,dv].  The formulas of m ``gated_decode_step`` calls, which are fp32 arithmetic throughout; bf16
    inputs with dk = dv = 128 run on the tensor cores here (operands in two bf16 parts, about 3e-6)."""
    return _decode("efla_gated_decode_tokens", 2, q, k, v, g, beta, S, o, o_dtype, stream, update)


def _prep_args(q, k, a, b, A_log, dt_bias):
    code = _first("q", q, q.dim())
    if q.dim() < 3 or a.dim() != q.dim() - 1:
        _bad(f"q must be [..., H_k, dk] and a [..., H], got {list(q.shape)} and {list(a.shape)}")
    lead, H = tuple(q.shape[:-2]), a.shape[-1]
    if H > _INT_MAX or q.shape[-1] > _INT_MAX:
        _too_large(H, q.shape[-1])
    _need("q", q, q.shape, q.dtype, q)
    _need("k", k, q.shape, q.dtype, q)
    _need("a", a, (*lead, H), q.dtype, q)
    _need("b", b, (*lead, H), q.dtype, q)
    _need("A_log", A_log, (H,), torch.float32, q)
    _need("dt_bias", dt_bias, (H,), torch.float32, q)
    tokens = 1
    for n in lead:
        tokens *= n
    return code, tokens, H


def gated_prep(q: torch.Tensor, k: torch.Tensor, a: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
               dt_bias: torch.Tensor, *, scale: float = 1.0, eps: float = 1e-6, stream=None) -> dict:
    """The norms and gates before the mixer (``efla_gated_prep``): q^ = scale q / sqrt(|q|^2 + eps), k^
    likewise without the scale, g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b).

    q, k [..., H_k, dk] and a, b [..., H] (bf16 or fp32), A_log, dt_bias [H] fp32.  Returns a dict
    with q and k in q's dtype and g, beta [..., H] fp32."""
    code, tokens, H = _prep_args(q, k, a, b, A_log, dt_bias)
    _on_device(q)
    out = {"q": _empty_as(q, q.dtype, stream), "k": _empty_as(q, q.dtype, stream),
           "g": _empty_as(a, torch.float32, stream), "beta": _empty_as(a, torch.float32, stream)}
    _check(_lib().efla_gated_prep(q.data_ptr(), k.data_ptr(), a.data_ptr(), b.data_ptr(), A_log.data_ptr(),
                                  dt_bias.data_ptr(), *(t.data_ptr() for t in out.values()), tokens, q.shape[-2], H,
                                  q.shape[-1], code, scale, eps, _stream(stream, q)))
    return out


def gated_prep_bwd(q: torch.Tensor, k: torch.Tensor, a: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
                   dt_bias: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dg: torch.Tensor, dbeta: torch.Tensor, *,
                   scale: float = 1.0, eps: float = 1e-6, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``gated_prep`` from those of its outputs (``efla_gated_prep_bwd``): a dict with dq,
    dk, da, db in q's dtype and dA_log, ddt_bias [H] fp32."""
    code, tokens, H = _prep_args(q, k, a, b, A_log, dt_bias)
    _need("dq", dq, q.shape, q.dtype, q)
    _need("dk", dk, q.shape, q.dtype, q)
    _need("dg", dg, a.shape, torch.float32, q)
    _need("dbeta", dbeta, a.shape, torch.float32, q)
    _on_device(q)
    L = _lib()
    need = _sz(0)
    _check(L.efla_gated_prep_bwd_workspace(tokens, H, ctypes.byref(need)))
    ws = _workspace(workspace, need.value, q, stream)
    out = {"dq": _empty_as(q, q.dtype, stream), "dk": _empty_as(q, q.dtype, stream), "da": _empty_as(a, q.dtype, stream),
           "db": _empty_as(a, q.dtype, stream), "dA_log": _empty_as(A_log, torch.float32, stream),
           "ddt_bias": _empty_as(A_log, torch.float32, stream)}
    _check(L.efla_gated_prep_bwd(q.data_ptr(), k.data_ptr(), a.data_ptr(), b.data_ptr(), A_log.data_ptr(),
                                 dt_bias.data_ptr(), dq.data_ptr(), dk.data_ptr(), dg.data_ptr(), dbeta.data_ptr(),
                                 *(t.data_ptr() for t in out.values()), tokens, q.shape[-2], H, q.shape[-1], code,
                                 scale, eps, ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream, q)))
    return out


def _norm_args(o, z, w):
    if o.dim() < 1:
        _bad("o must have at least one dimension")
    code = _first("o", o, o.dim())
    d = o.shape[-1]
    if d > _INT_MAX:
        _too_large(d)
    _need("o", o, o.shape, o.dtype, o)
    _need("z", z, o.shape, o.dtype, o)
    _need("w", w, (d,), torch.float32, o)
    rows = 1
    for n in o.shape[:-1]:
        rows *= n
    return code, rows, d


def norm_gate(o: torch.Tensor, z: torch.Tensor, w: torch.Tensor, *, eps: float = 1e-6,
              y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The norm after the mixer fused with its output gate (``efla_norm_gate``):
    y = o / sqrt(mean(o^2) + eps) * w * silu(z) over the last dimension.  o, z [..., d] (bf16 or
    fp32), w [d] fp32; ``y`` may be o or z."""
    code, rows, d = _norm_args(o, z, w)
    _on_device(o)
    y = _given("y", y, o.shape, o.dtype, o, stream)
    _check(_lib().efla_norm_gate(o.data_ptr(), z.data_ptr(), w.data_ptr(), y.data_ptr(), rows, d, code, eps,
                                 _stream(stream, o)))
    return y


def norm_gate_bwd(o: torch.Tensor, z: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, *, eps: float = 1e-6,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``norm_gate`` (``efla_norm_gate_bwd``): a dict with do, dz in o's dtype and dw [d] fp32."""
    code, rows, d = _norm_args(o, z, w)
    _need("dy", dy, o.shape, o.dtype, o)
    _on_device(o)
    L = _lib()
    need = _sz(0)
    _check(L.efla_norm_gate_bwd_workspace(d, ctypes.byref(need)))
    ws = _workspace(workspace, need.value, o, stream)
    out = {"do": _empty_as(o, o.dtype, stream), "dz": _empty_as(o, o.dtype, stream), "dw": _empty_as(w, torch.float32, stream)}
    _check(L.efla_norm_gate_bwd(o.data_ptr(), z.data_ptr(), w.data_ptr(), dy.data_ptr(),
                                *(t.data_ptr() for t in out.values()), rows, d, code, eps, ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream(stream, o)))
    return out
